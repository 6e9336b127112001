"""GPU parity of the attention calls (include/ttt_attention.h) against the fp64 oracle
(oracle/ttt_attention.py), element by element, on seeded inputs.

Bars.  H is the half step of the output's type relative to the value (bf16 2^-8, fp32 2^-24,
e4m3 2^-4 and 2^-10 below its normal range); U = 2^-24 that of fp32 arithmetic.
* norm and rotation: the sum of D <= 1024 squares runs over chains of at most 16 + 6 additions
  of positive terms (22 U, half of it after the root), the mean, eps, root and division add
  4 U, the two scalings 2 U; the angle in turns is rounded once to fp32 (|turn| <= 1/2: 2 pi U
  / 2 in radians), its sine and cosine to 4 U, the rotation's products and sum 3 U: below 32 U
  (|n0| + |n1|) together, n the normed pair.  |y - y_ref| <= H |y_ref| + 2^-19 (|n0| + |n1|).
* its backward: the gradient turned back g carries 2^-20 (|dy0| + |dy1|), x r 17 U; the mean
  of u x r over D terms sums absolute values the same way: |dx - ref| <= H |dx_ref| + 2^-18 r
  (G w + |x r| mean(G w |x r|)), G = |dy0| + |dy1| of the pair.  The scale's gradient is a
  sum of N products in some fixed order: (N + 64) U sum G |x r|.
* paged attention: a score's fp32 sum of D products is within D U sum |q k| scale, the base-2
  argument within 4 U |s|; call the sum of both d.  A probability is then off by d relative,
  by 2^-16 from its two bf16 parts, and the same for the normaliser: |o - o_ref| <= H |o_ref|
  + (2 d + 2^-15) max |v|.  lse: d + 4 U (|lse| + 1).
* window training: out as the window attention's own bar (the probabilities are rounded to
  bf16); lse as above.  Gradients: p and ds rounded to bf16 (2^-8 relative each), delta from
  the rounded out (2^-8 sum |dout out|), fp32 parts below 2^-14 of the absolute sums:
  |dv - ref| <= H |ref| + (2^-8 + 2^-14) sum p |dout|,
  |dq - ref| <= H |ref| + scale sum_j (2^-8 |ds_j| + p_j (2^-8 e + 2^-14 (|dp_j| + e))) |k_j|
  with e = sum |dout out|, dk the same over queries; the term 2^-8 e falls away where no row
  sees more than 64 tokens (delta is then summed as p dp).
"""
import numpy as np
import pytest
import torch

import attention_bars as bars
import oracle.ttt_attention as oa
import oracle.ttt_block as blk
import weight_sequence_layers_amd as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def np64(t):
    return t.detach().double().cpu().numpy()


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ------------------------------------------------------------------------ norm and rotation
class Rope:
    """A case's configuration and inputs: queries, keys and values as parts of one row."""

    def __init__(self, T, Hq, Hk, D, rot, axes=1, pairing="halves", norm="rms", act="bf16", weights=True,
                 eps=1e-6, far=False, seed=1):
        say(f"rope T={T} Hq={Hq} Hk={Hk} D={D} rot={rot} axes={axes} {pairing} {norm} {act} far={far}")
        self.T, self.Hq, self.Hk, self.D, self.rot, self.axes = T, Hq, Hk, D, rot, axes
        self.pairing, self.eps = pairing, (eps if norm == "rms" else None)
        self.dt = torch.bfloat16 if act == "bf16" else torch.float32
        self.cfg = W.make_rope_config(q_heads=Hq, k_heads=Hk, head_dim=D, rot_dim=rot, axes=axes,
                                      pairing=pairing, norm=norm, act=act, eps=eps)
        g = gen(seed)
        pad = 8
        self.ld = (Hq + 2 * Hk) * D + pad
        self.x = torch.randn(T, self.ld, generator=g, device=DEV).to(self.dt)
        self.q, self.k, self.v = self.x, self.x[:, Hq * D:], self.x[:, (Hq + Hk) * D:]
        hi = 2 ** 31 - 1 if far else 5000
        self.pos = torch.randint(-hi, hi, (axes, T), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        self.freq = torch.rand(axes, rot // 2, generator=g, device=DEV) ** 4
        if rot == 0:
            self.pos = self.freq = None
        use = weights and norm == "rms"
        self.qw = (1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(self.dt) if use else None
        self.kw = (1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(self.dt) if use else None
        self.ang = (np.zeros((T, 0)) if rot == 0 else oa.angles(np64(self.pos), np64(self.freq)))

    def heads(self, which):
        o, n = {"q": (0, self.Hq), "k": (self.Hq, self.Hk), "v": (self.Hq + self.Hk, self.Hk)}[which]
        return np64(self.x[:, o * self.D:(o + n) * self.D]).reshape(self.T, n, self.D)

    def weight(self, which):
        w = self.qw if which == "q" else self.kw
        return None if w is None else np64(w)

    def both(self, x):
        """|x0| + |x1| of each element's pair (|x| where nothing turns)."""
        y = np.abs(x)
        i0, i1 = oa.pair_index(self.rot, self.pairing)
        s = y[..., i0] + y[..., i1]
        y[..., i0], y[..., i1] = s, s
        return y

    def ref(self, which):
        """The rotated heads and their bar."""
        x, w = self.heads(which), self.weight(which)
        y = oa.norm_rope(x, w, self.ang, self.pairing, self.eps)
        n = oa.norm_rope(x, w, np.zeros((self.T, 0)), self.pairing, self.eps)
        return y, H[self.dt] * np.abs(y) + 2.0 ** -19 * self.both(n) + 1e-38

    def out(self, n, extra=3):
        """Rows for n heads with some behind them that must stay."""
        return torch.full((self.T + extra, n * self.D + 16), 7.0, dtype=self.dt, device=DEV)

    def call(self, qo=None, ko=None, **kw):
        qo = self.out(self.Hq) if qo is None else qo
        ko = self.out(self.Hk) if ko is None else ko
        W.ttt_qk_norm_rope(self.cfg, self.q, self.ld, self.k, self.ld, self.qw, self.kw, self.freq, self.pos,
                           qo, qo.stride(0), ko, ko.stride(0), self.T, **kw)
        return qo, ko

    def check(self, qo, ko):
        torch.cuda.synchronize()
        for which, o, n in (("q", qo, self.Hq), ("k", ko, self.Hk)):
            y, bar = self.ref(which)
            got = np64(o[:self.T, :n * self.D]).reshape(y.shape)
            worst = np.max(np.abs(got - y) / bar) if y.size else 0.0
            assert worst <= 1, (which, worst)
            assert bool((o[self.T:] == 7).all()) and bool((o[:, n * self.D:] == 7).all())


ROPES = [
    dict(T=1, Hq=1, Hk=1, D=16, rot=16),
    dict(T=5, Hq=3, Hk=1, D=48, rot=16, pairing="pairs"),
    dict(T=37, Hq=8, Hk=2, D=128, rot=128),
    dict(T=37, Hq=8, Hk=2, D=128, rot=128, act="f32", pairing="pairs"),
    dict(T=33, Hq=2, Hk=2, D=80, rot=32, axes=2, act="f32"),
    dict(T=21, Hq=6, Hk=6, D=128, rot=96, axes=3, pairing="pairs"),
    dict(T=9, Hq=1, Hk=2, D=1024, rot=1024, axes=4),
    dict(T=9, Hq=2, Hk=1, D=512, rot=256, act="f32"),
    dict(T=12, Hq=4, Hk=4, D=64, rot=0, norm="rms"),
    dict(T=12, Hq=4, Hk=4, D=64, rot=64, norm="none"),
    dict(T=12, Hq=4, Hk=4, D=64, rot=32, weights=False, eps=0.1),
    dict(T=40, Hq=2, Hk=2, D=64, rot=64, act="f32", far=True),
    dict(T=5003, Hq=2, Hk=1, D=64, rot=64),
    dict(T=40001, Hq=1, Hk=1, D=32, rot=32, axes=3, act="f32"),
]


@pytest.mark.parametrize("kw", ROPES)
def test_norm_rope_matches_oracle(kw):
    r = Rope(**kw)
    r.check(*r.call())


def test_norm_rope_in_place_in_a_projections_rows():
    r = Rope(T=70, Hq=4, Hk=2, D=64, rot=64)
    refs = {w: r.ref(w) for w in "qk"}
    v = r.v.clone()
    W.ttt_qk_norm_rope(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, r.q, r.ld, r.k, r.ld, r.T)
    torch.cuda.synchronize()
    for w in "qk":
        assert np.all(np.abs(r.heads(w) - refs[w][0]) <= refs[w][1])
    assert torch.equal(r.v, v)


def test_norm_rope_zero_rows_and_large_values():
    r = Rope(T=4, Hq=2, Hk=1, D=64, rot=64)
    r.x[1] = 0
    r.x[2] *= 1e15     # squares up to 1e31
    r.check(*r.call())


def test_norm_rope_keeps_nan_and_inf_to_their_heads():
    r = Rope(T=3, Hq=2, Hk=2, D=64, rot=64)
    clean = r.call()
    r.x[1, 5] = float("nan")
    r.x[2, 2 * 64 + 7] = float("inf")   # a key's
    qo, ko = r.call()
    torch.cuda.synchronize()
    assert bool(qo[1, :64].isnan().all())
    qo[1, :64] = clean[0][1, :64]
    assert torch.equal(qo, clean[0])
    assert bool((~ko[2, :64].isfinite()).any())
    ko[2, :64] = clean[1][2, :64]
    assert torch.equal(ko, clean[1])


def test_no_tokens_leaves_the_outputs():
    r = Rope(T=4, Hq=2, Hk=1, D=64, rot=64)
    qo, ko = r.out(2), r.out(1)
    W.ttt_qk_norm_rope(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, qo, 144, ko, 80, 0)
    torch.cuda.synchronize()
    assert bool((qo == 7).all()) and bool((ko == 7).all())


def rope_backward(r, dq_w=True, dk_w=True, in_place=False, work=None, seed=9):
    g = gen(seed)
    gq = torch.randn(r.T, r.Hq * r.D + 8, generator=g, device=DEV).to(r.dt)
    gk = torch.randn(r.T, r.Hk * r.D, generator=g, device=DEV).to(r.dt)
    refs = [np64(gq[:, :r.Hq * r.D]).reshape(r.T, r.Hq, r.D), np64(gk).reshape(r.T, r.Hk, r.D)]
    dq, dk = (gq, gk) if in_place else (r.out(r.Hq), r.out(r.Hk))
    dqw = torch.full((r.D,), 5.0, device=DEV) if dq_w and r.qw is not None else None
    dkw = torch.full((r.D,), 5.0, device=DEV) if dk_w and r.kw is not None else None
    n = W.ttt_qk_norm_rope_backward_work(r.cfg, r.T)
    work = torch.empty(n, dtype=torch.uint8, device=DEV) if work is None else work
    W.ttt_qk_norm_rope_backward(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, gq, gq.stride(0), gk,
                                gk.stride(0), dq, dq.stride(0), dk, dk.stride(0), dqw, dkw, work, r.T)
    return refs, dq, dk, dqw, dkw


def check_rope_backward(r, refs, dq, dk, dqw, dkw, behind=True):
    torch.cuda.synchronize()
    for which, dy, d, dw in (("q", refs[0], dq, dqw), ("k", refs[1], dk, dkw)):
        x, w = r.heads(which), r.weight(which)
        dx_ref, dw_ref = oa.norm_rope_vjp(x, w, r.ang, r.pairing, r.eps, dy)
        G = r.both(dy)
        if r.eps is None:
            inner = G
        else:
            rr = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + r.eps)
            xh, Gw = np.abs(x * rr), G * (1 if w is None else np.abs(w))
            inner = rr * (Gw + xh * np.mean(Gw * xh, -1, keepdims=True))
        bar = H[r.dt] * np.abs(dx_ref) + 2.0 ** -18 * inner + 1e-38
        n = dx_ref.shape[1] * r.D
        got = np64(d[:r.T, :n]).reshape(dx_ref.shape)
        assert np.max(np.abs(got - dx_ref) / bar) <= 1, (which, np.max(np.abs(got - dx_ref) / bar))
        if behind:
            assert bool((d[r.T:] == 7).all()) and bool((d[:, n:] == 7).all())
        if dw is not None:
            N = r.T * dx_ref.shape[1]
            bar = (N + 64) * U * np.sum(G * xh, axis=(0, 1)) + 2.0 ** -18 * np.sum(G * xh, axis=(0, 1))
            assert np.all(np.abs(np64(dw) - dw_ref) <= bar), which


@pytest.mark.parametrize("kw", ROPES)
def test_norm_rope_backward_matches_oracle(kw):
    r = Rope(**kw)
    check_rope_backward(r, *rope_backward(r))


@pytest.mark.parametrize("dq_w,dk_w", [(True, False), (False, True), (False, False)])
def test_norm_rope_backward_of_some_scales_in_place(dq_w, dk_w):
    r = Rope(T=55, Hq=4, Hk=2, D=64, rot=32, pairing="pairs")
    check_rope_backward(r, *rope_backward(r, dq_w, dk_w, in_place=True), behind=False)


def test_norm_rope_backward_against_differences():
    """The kernel's own forward in fp32, differenced: the rounding of the sum (about 1e-3 of its
    terms' size over the step) leaves four digits."""
    r = Rope(T=6, Hq=2, Hk=2, D=32, rot=32, act="f32", axes=2)
    refs, dq, dk, dqw, dkw = rope_backward(r)
    d = torch.randn(r.x.shape, generator=gen(2), device=DEV)
    x0, f = r.x.clone(), []
    for s in (1, -1):
        r.x.copy_(x0 + s * 2.0 ** -6 * d)
        qo, ko = r.call()
        torch.cuda.synchronize()
        f.append(sum(np.sum(np64(o[:r.T, :64]).reshape(dy.shape) * dy) for o, dy in zip((qo, ko), refs)))
    got = (f[0] - f[1]) / 2.0 ** -5
    dd = np64(d)
    want = np.sum(np64(dq[:r.T, :64]) * dd[:, :64]) + np.sum(np64(dk[:r.T, :64]) * dd[:, 64:128])
    # third derivatives of the norm are bounded by 15 / rms^3 per unit, rms ~ 1 here, the step
    # cubed 2^-18 / 6 times 24 rows: below 1e-3 of the gradients' scale; checked at 1e-2
    scale = np.sqrt(np.sum(np64(dq[:r.T, :64]) ** 2) + np.sum(np64(dk[:r.T, :64]) ** 2))
    assert abs(got - want) <= 1e-2 * scale


def test_no_tokens_give_zero_scale_gradients():
    r = Rope(T=3, Hq=2, Hk=1, D=64, rot=64)
    a, b = torch.full((64,), 5.0, device=DEV), torch.full((64,), 5.0, device=DEV)
    W.ttt_qk_norm_rope_backward(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, r.q, r.ld, r.k, r.ld,
                                r.out(2), 144, r.out(1), 80, a, b, None, 0)
    torch.cuda.synchronize()
    assert bool((a == 0).all()) and bool((b == 0).all())


def test_norm_rope_backward_replayed():
    r = Rope(T=3001, Hq=3, Hk=1, D=64, rot=64)
    work = torch.empty(W.ttt_qk_norm_rope_backward_work(r.cfg, r.T), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    gq, gk = (torch.randn(r.T, n * r.D, generator=gen(3), device=DEV).to(r.dt) for n in (r.Hq, r.Hk))
    dq, dk, a, b = torch.empty_like(gq), torch.empty_like(gk), torch.empty(64, device=DEV), torch.empty(64, device=DEV)

    def call():
        W.ttt_qk_norm_rope_backward(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, gq, r.Hq * r.D, gk,
                                    r.Hk * r.D, dq, r.Hq * r.D, dk, r.Hk * r.D, a, b, work, r.T)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dq, dk, a, b)]
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in (dq, dk, a, b):
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, (dq, dk, a, b)))
        torch.randn(1000, device=DEV).sum().item()


def test_norm_rope_backward_is_the_same_every_time():
    r = Rope(T=30011, Hq=3, Hk=1, D=64, rot=64)
    first = rope_backward(r)
    again = rope_backward(r)
    torch.cuda.synchronize()
    for a, b in zip(first[1:], again[1:]):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------ cache
def new_cache(pages, heads, size, dim, dtype, together=False, fill=float("nan")):
    """k, v [pages, heads, size, dim] full of NaN: two arrays, or in turn in one."""
    if together:
        both = torch.full((pages, 2, heads, size, dim), fill, device=DEV).to(dtype)
        return both[:, 0], both[:, 1]
    return tuple(torch.full((pages, heads, size, dim), fill, device=DEV).to(dtype) for _ in range(2))


@pytest.mark.parametrize("kw,size,dtype,together", [
    (dict(T=1, Hq=2, Hk=1, D=64, rot=64), 1, "bf16", False),
    (dict(T=37, Hq=8, Hk=2, D=128, rot=128), 16, "bf16", True),
    (dict(T=37, Hq=4, Hk=4, D=128, rot=64, pairing="pairs", axes=3), 24, "e4m3", False),
    (dict(T=29, Hq=1, Hk=3, D=48, rot=16, norm="none"), 7, "e4m3", True),
    (dict(T=29, Hq=2, Hk=1, D=256, rot=256), 5, "e4m3", False),
    (dict(T=5003, Hq=2, Hk=2, D=64, rot=64), 64, "bf16", False),
])
@pytest.mark.parametrize("scaled", [False, True])
def test_append_matches_oracle(kw, size, dtype, together, scaled):
    r = Rope(**kw)
    ct = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    pages = r.T // size + 4
    k, v = new_cache(pages, r.Hk, size, r.D, ct, together, fill=3.0)
    g = gen(5)
    slot = torch.randperm(pages * size, generator=g, device=DEV)[:r.T].to(torch.int64)
    if r.T > 4:
        slot[2], slot[3], slot[4] = -1, pages * size, 2 ** 62
    if scaled and dtype == "e4m3":
        ks = 0.01 + 0.02 * torch.rand(r.Hk, generator=g, device=DEV)
        vs = 0.001 + 0.01 * torch.rand(r.Hk, generator=g, device=DEV)   # some values pass 448
    else:
        ks = vs = None
    cache = W.make_kv_cache(k, v, k_scale=ks, v_scale=vs)
    qo = r.out(r.Hq)
    W.ttt_qk_norm_rope_append(r.cfg, r.q, r.ld, r.k, r.ld, r.v, r.ld, r.qw, r.kw, r.freq, r.pos, cache, slot, qo,
                              qo.stride(0), r.T)
    torch.cuda.synchronize()
    y, bar = r.ref("q")
    assert np.all(np.abs(np64(qo[:r.T, :r.Hq * r.D]).reshape(y.shape) - y) <= bar)
    assert bool((qo[r.T:] == 7).all())
    at = slot.cpu().numpy()
    ok = (at >= 0) & (at < pages * size)
    kref, kbar = r.ref("k")
    vref = r.heads("v")
    for c, ref, inner, sc in ((k, kref, kbar - H[r.dt] * np.abs(kref), ks), (v, vref, 0 * vref, vs)):
        flat = np64(c.float()).transpose(0, 2, 1, 3).reshape(pages * size, r.Hk, r.D)
        s = 1.0 if sc is None else np64(sc)[:, None]
        got = flat[at[ok]]
        want = ref[ok] / s
        if dtype == "e4m3":
            want = np.clip(want, -448, 448)
            b = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
            b = b + 1.125 * (inner[ok] / s + 2 * U * np.abs(want))
        else:
            b = H[torch.bfloat16] * np.abs(want) + inner[ok]
            if c is v:
                b = 0 * b
        assert np.all(np.abs(got - want) <= b), float(np.max(np.abs(got - want) - b))
        rest = np.ones(pages * size, bool)
        rest[at[ok]] = False
        assert np.all(flat[rest] == 3.0)


def test_append_e4m3_keeps_nan_and_holds_infinity():
    r = Rope(T=2, Hq=1, Hk=1, D=16, rot=0, norm="none")
    r.x[0, 32], r.x[0, 33], r.x[0, 34] = float("nan"), float("inf"), -float("inf")
    k, v = new_cache(1, 1, 2, 16, torch.float8_e4m3fn, fill=0.0)
    W.ttt_qk_norm_rope_append(r.cfg, r.q, r.ld, r.k, r.ld, r.v, r.ld, None, None, None, None, W.make_kv_cache(k, v),
                              torch.tensor([1, 0], device=DEV), r.out(1), 32, 2)
    torch.cuda.synchronize()
    row = v.float()[0, 0, 1]
    assert bool(row[0].isnan()) and float(row[1]) == 448 and float(row[2]) == -448


# ------------------------------------------------------------------------ paged attention
class Paged:
    def __init__(self, lens, Hq, Hk, D, size, dtype="bf16", scaled=False, together=False, qscale=1.5, seed=3,
                 max_pages=None, spare=3):
        say(f"paged lens={lens[:8]}.. S={len(lens)} Hq={Hq} Hk={Hk} D={D} size={size} {dtype}")
        g = gen(seed)
        S = len(lens)
        self.S, self.Hq, self.Hk, self.D, self.size = S, Hq, Hk, D, size
        used = [max(0, -(-n // size)) for n in lens]
        self.width = max(max(used), 1) if max_pages is None else max_pages
        pages = sum(used) + spare
        ct = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
        self.k, self.v = new_cache(pages, Hk, size, D, ct, together)   # NaN wherever nothing is stored
        order = torch.randperm(pages, generator=g, device=DEV).cpu().tolist()
        table = np.full((S, self.width), -1, np.int32)
        bits = torch.int16 if dtype == "bf16" else torch.uint8
        at = 0
        for s, n in enumerate(lens):
            for i in range(used[s]):
                table[s, i] = order[at]
                m = min(size, n - i * size)
                for c in (self.k, self.v):
                    c.view(bits)[order[at], :, :m] = torch.randn(Hk, m, D, generator=g, device=DEV).to(ct).view(bits)
                at += 1
        self.table = torch.from_numpy(table).to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.ks = 0.5 + torch.rand(Hk, generator=g, device=DEV) if scaled else None
        self.vs = 0.5 + torch.rand(Hk, generator=g, device=DEV) if scaled else None
        self.q = (qscale * torch.randn(S, Hq * D + 8, generator=g, device=DEV)).to(torch.bfloat16)
        self.cache = W.make_kv_cache(self.k, self.v, k_scale=self.ks, v_scale=self.vs)
        self.out = torch.full((S + 2, Hq * D + 16), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((S + 2, Hq), 7.0, device=DEV)

    def work(self, window=0):
        n = W.ttt_paged_attention_work(self.cache, self.S, self.Hq, self.width, window)
        return torch.full((max(n, 1) // 4 + 1,), float("nan"), device=DEV)   # never read unwritten

    def call(self, window=0, scale=0.0, work=None, lse=True, **kw):
        work = self.work(window) if work is None else work
        W.ttt_paged_attention(self.q, self.q.stride(0), self.cache, self.table, self.lens, self.out,
                              self.out.stride(0), self.lse if lse else None, self.S, self.Hq, self.width, window,
                              scale, work, **kw)

    def values(self):
        k, v = np64(self.k.float()), np64(self.v.float())
        if self.ks is not None:
            k, v = k * np64(self.ks)[:, None, None], v * np64(self.vs)[:, None, None]
        return k, v

    def check(self, window=0, scale=0.0, lse=True):
        torch.cuda.synchronize()
        scale = scale or 1 / np.sqrt(self.D)
        k, v = self.values()
        q = np64(self.q[:, :self.Hq * self.D]).reshape(self.S, self.Hq, self.D)
        ref, rl = oa.paged_attention(q, k, v, self.table.cpu().numpy(), self.lens.cpu().numpy(), window, scale)
        qmax = np.sqrt(np.sum(q * q, -1)).max() if q.size else 0
        kmax = np.sqrt(np.nanmax(np.sum(np.where(np.isnan(k), 0, k) ** 2, -1)))
        d = scale * qmax * kmax * (self.D + 4) * U       # sum |q k| <= |q| |k|
        got = np64(self.out[:self.S, :self.Hq * self.D]).reshape(ref.shape)
        bar = 2.0 ** -8 * np.abs(ref) + (2 * d + 2.0 ** -15) * np.nanmax(np.abs(v)) if np.any(~np.isnan(v)) else 0
        worst = np.abs(got - ref) - bar
        assert not np.isnan(got).any() and np.all(worst <= 0), float(worst.max())
        assert bool((self.out[self.S:] == 7).all()) and bool((self.out[:, self.Hq * self.D:] == 7).all())
        if lse:
            gl = np64(self.lse[:self.S])
            empty = np.isinf(rl)
            assert np.array_equal(np.isneginf(gl), empty)
            assert np.all(np.abs(gl[~empty] - rl[~empty]) <= d + 4 * U * (np.abs(rl[~empty]) + 1))
            assert bool((self.lse[self.S:] == 7).all())
        # an empty row is exactly zero
        assert np.all(got[np.isinf(rl)] == 0)


PAGEDS = [
    (dict(lens=[1], Hq=1, Hk=1, D=64, size=1), 0),
    (dict(lens=[5], Hq=2, Hk=2, D=128, size=16), 0),
    (dict(lens=[0, 31, 32, 33, 127, 128, 129, 1], Hq=8, Hk=8, D=128, size=16), 0),
    (dict(lens=[200, 77, 0], Hq=8, Hk=2, D=128, size=7, together=True), 0),
    (dict(lens=[200, 77, 0], Hq=8, Hk=2, D=128, size=7, dtype="e4m3"), 0),
    (dict(lens=[200, 77, 300], Hq=6, Hk=2, D=64, size=24, dtype="e4m3", scaled=True, together=True), 0),
    (dict(lens=[200, 77, 300], Hq=34, Hk=2, D=64, size=24), 0),        # 17 queries to a key head
    (dict(lens=[200, 513], Hq=40, Hk=1, D=256, size=3), 0),
    (dict(lens=[200, 513], Hq=3, Hk=3, D=256, size=64, dtype="e4m3", scaled=True), 0),
    (dict(lens=[3000, 1, 0, 600], Hq=4, Hk=2, D=128, size=16), 0),     # split and joined
    (dict(lens=[3000, 1, 0, 600], Hq=4, Hk=2, D=64, size=128, dtype="e4m3"), 0),
    (dict(lens=[1500, 700], Hq=4, Hk=1, D=256, size=16), 0),
    (dict(lens=[3000, 1, 0, 600, 100], Hq=4, Hk=2, D=128, size=16), 100),
    (dict(lens=[3000, 1, 0, 600, 2048], Hq=2, Hk=2, D=64, size=24), 1024),
    (dict(lens=[300, 1, 2], Hq=2, Hk=2, D=128, size=24, dtype="e4m3"), 1),
    (dict(lens=[300], Hq=2, Hk=2, D=128, size=24), 2 ** 31 - 1),
    (dict(lens=[20000], Hq=1, Hk=1, D=128, size=64), 0),
]


@pytest.mark.parametrize("kw,window", PAGEDS)
def test_paged_attention_matches_oracle(kw, window):
    p = Paged(**kw)
    p.call(window)
    p.check(window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 1, 17, 64])
def test_paged_attention_heads_of_256_around_a_step(dtype, window):
    """Lengths around the 16 tokens of a wave's step and the 64 of a workgroup's, whose last page
    numbers lie outside the cache for one of them."""
    p = Paged([0, 1, 15, 16, 17, 31, 63, 64, 65, 129, 400], 4, 2, 256, 7, dtype=dtype)
    p.table[9, 18] = -1        # tokens 126 .. 128
    p.call(window)
    p.check(window)


def test_paged_attention_large_scores_and_own_scale():
    p = Paged([700, 40], 4, 2, 128, 16, qscale=30.0)
    p.call(scale=0.3)
    p.check(scale=0.3)
    p.out.fill_(7.0)
    p.call(scale=0.3, lse=False)
    p.check(scale=0.3, lse=False)


def test_paged_attention_many_sequences():
    rng = np.random.default_rng(1)
    p = Paged([int(n) for n in rng.integers(0, 90, 300)], 4, 4, 64, 16)
    p.call()
    p.check()


def test_paged_attention_bad_pages_and_lengths():
    """Page numbers outside the cache are left out, lengths are held to the table's width."""
    p = Paged([300, 300, 300, 64, 300], 4, 2, 128, 16, max_pages=19)
    t = p.table
    pages = p.k.shape[0]
    t[0, 3], t[0, 18], t[1, 0], t[1, 7] = -1, pages, 2 ** 31 - 1, -2 ** 31
    t[2] = -5                                  # nothing left
    p.lens[3] = -7
    p.lens[4] = 2 ** 31 - 1                    # 304 places, the last ones not stored: NaN
    row = int(t[4, 18])
    p.k[row], p.v[row] = 0.5, 0.25
    p.call()
    p.check()
    assert bool((p.out[2, :512] == 0).all()) and bool((p.lse[2] == -float("inf")).all())


@pytest.mark.parametrize("n", [50, 3000])
def test_paged_attention_keeps_nan_to_what_sees_it(n):
    """A NaN key reaches the query heads that share it (out and lse), a NaN value one element of
    them; other heads and sequences are as without."""
    p = Paged([n, 60], 4, 2, 128, 16)
    p.call()
    torch.cuda.synchronize()
    clean, lse = p.out.clone(), p.lse.clone()
    p.k[int(p.table[0, 1]), 1, 3, 7] = float("nan")      # heads 2 and 3 of sequence 0
    p.v[int(p.table[1, 0]), 0, 2, 9] = float("nan")      # element 9 of heads 0 and 1 of sequence 1
    p.call()
    torch.cuda.synchronize()
    assert bool(p.out[0, 256:512].isnan().all()) and bool(p.lse[0, 2:].isnan().all())
    assert bool(p.out[1, 9].isnan()) and bool(p.out[1, 128 + 9].isnan())
    p.out[0, 256:512], p.lse[0, 2:] = clean[0, 256:512], lse[0, 2:]
    p.out[1, 9], p.out[1, 128 + 9] = clean[1, 9], clean[1, 128 + 9]
    assert torch.equal(p.out, clean) and torch.equal(p.lse, lse)


def test_paged_attention_one_long_sequence_among_short_ones():
    p = Paged([20000] + [40] * 20, 4, 1, 128, 64)
    p.call()
    p.check()


def test_two_streams_with_a_workspace_each():
    """Two decoding calls in flight at once, each on its own stream with its own workspace, ten
    times over."""
    ps = [Paged([3000, 700], 4, 2, 128, 16, seed=s) for s in (21, 22)]
    works = [p.work() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, w, s in zip(ps, works, streams):
            p.call(work=w, stream=s)
    for p in ps:
        p.check()


def test_paged_attention_two_sequences_share_pages():
    p = Paged([300, 200], 2, 2, 64, 16)
    p.table[1, :13] = p.table[0, :13]
    p.call()
    p.check()


def test_paged_attention_no_pages_at_all():
    p = Paged([5, 6], 2, 2, 64, 16, max_pages=None)
    out = torch.full((2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, 2), 7.0, device=DEV)
    W.ttt_paged_attention(p.q, p.q.stride(0), p.cache, None, p.lens, out, 128, lse, 2, 2, 0, 0, 0.0, None)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_paged_attention_past_32_bit_offsets():
    """Pages past 2^32 bytes and 2^32 elements into the cache."""
    pages, size = 34000, 64
    both = torch.empty(pages, 2, 8, size, 128, dtype=torch.bfloat16, device=DEV)   # 8.9 GB
    k, v = both[:, 0], both[:, 1]
    rows = [33999, 3, 33000]
    g = gen(4)
    for p in rows:
        both[p] = torch.randn(2, 8, size, 128, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, 8 * 128, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    cache = W.make_kv_cache(k, v)
    W.ttt_paged_attention(q, 1024, cache, torch.tensor([rows], dtype=torch.int32, device=DEV),
                          torch.tensor([180], dtype=torch.int32, device=DEV), out, 1024, None, 1, 8, 3, 0, 0.0,
                          torch.empty(max(1, W.ttt_paged_attention_work(cache, 1, 8, 3, 0)), dtype=torch.uint8,
                                      device=DEV))
    kk, vv = (np64(torch.stack([c[p] for p in rows])) for c in (k, v))
    ref, _ = oa.paged_attention(np64(q).reshape(1, 8, 128), kk, vv, np.array([[0, 1, 2]]), [180], 0, 128 ** -0.5)
    assert np.all(np.abs(np64(out).reshape(ref.shape) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * np.abs(vv).max())
    # append there too
    r = Rope(T=2, Hq=1, Hk=8, D=128, rot=0, norm="none")
    W.ttt_qk_norm_rope_append(r.cfg, r.q, r.ld, r.k, r.ld, r.v, r.ld, None, None, None, None, cache,
                              torch.tensor([33998 * size + 1, 5 * size + 63], device=DEV), r.out(1), 144, 2)
    torch.cuda.synchronize()
    assert np.array_equal(np64(k[33998, :, 1]), r.heads("k")[0]) and np.array_equal(np64(v[5, :, 63]), r.heads("v")[1])


def test_paged_attention_on_another_stream_and_replayed():
    p = Paged([3000, 1, 0, 600], 4, 2, 128, 16)
    work = p.work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.call(work=work, stream=s)
    s.synchronize()
    p.check()
    eager = p.out.clone(), p.lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call(work=work)
    for i in range(4):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        if i == 2:      # other lengths than the captured ones
            p.lens[0] = 2000
        g.replay()
        torch.cuda.synchronize()
        if i < 2:
            assert torch.equal(p.out, eager[0]) and torch.equal(p.lse, eager[1])
        else:
            p.check()
        torch.randn(1000, device=DEV).sum().item()


# ------------------------------------------------------------------------ window training
class Window:
    def __init__(self, B, H, T, window, mode, qscale=1.0, seed=2):
        say(f"window training B={B} H={H} T={T} window={window} {mode}")
        self.B, self.H, self.T, self.window, self.mode, self.D = B, H, T, window, mode, H * 128
        g = gen(seed)
        self.x = torch.randn(B, T, 3 * self.D + 8, generator=g, device=DEV).to(torch.bfloat16)
        self.x[..., :self.D] *= qscale
        self.go = torch.randn(B, T, self.D + 16, generator=g, device=DEV).to(torch.bfloat16)
        self.out = torch.full((B, T, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((B, H, T), 7.0, device=DEV)
        self.dx = torch.full((B * T + 2, 3 * self.D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        self.work = torch.full((B, H, T), float("nan"), device=DEV)

    def forward(self, **kw):
        D = self.D
        W.ttt_window_attention_lse(self.x, self.x[..., D:], self.x[..., 2 * D:], 3 * D + 8, self.out, D, self.lse,
                                   self.B, self.H, self.T, self.window, self.mode, **kw)

    def backward(self, **kw):
        D, dx = self.D, self.dx
        W.ttt_window_attention_backward(
            self.x, self.x[..., D:], self.x[..., 2 * D:], 3 * D + 8, self.out, D, self.lse, self.go, D + 16, dx,
            dx[:, D:], dx[:, 2 * D:], 3 * D + 8, self.work, self.B, self.H, self.T, self.window, self.mode, **kw)

    def check(self, problems=None):
        """problems: the (batch, head) pairs to compare, all by default."""
        torch.cuda.synchronize()
        T, D = self.T, self.D
        x, go, out, lse = np64(self.x), np64(self.go), np64(self.out), np64(self.lse)
        dx = np64(self.dx[:self.B * T]).reshape(self.B, T, -1)
        assert np.all(dx[..., 3 * D:] == 7) and bool((self.dx[self.B * T:] == 7).all())
        worst = {}
        for b in range(self.B):
            for h in range(self.H):
                if problems and (b, h) not in problems:
                    continue
                Q, K, V = (x[b, :, i * D + h * 128:i * D + h * 128 + 128] for i in range(3))
                dO, O = go[b, :, h * 128:h * 128 + 128], out[b, :, h * 128:h * 128 + 128]
                sc = 1 / np.sqrt(128)
                d = 132 * U * sc * np.sqrt((Q * Q).sum(1).max() * (K * K).sum(1).max())
                rl = oa.window_lse(Q, K, self.window, self.mode)
                assert np.all(np.abs(lse[b, h] - rl) <= d + 4 * U * (np.abs(rl) + 1))
                ro = blk.window_attention(Q, K, V, self.window, self.mode)
                assert np.all(np.abs(O - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -7 * np.abs(V).max() + 1e-6)
                P = oa.window_probs(Q, K, self.window, self.mode)
                dP = dO @ V.T
                dS = P * (dP - np.sum(P * dP, 1, keepdims=True))
                e = np.sum(np.abs(dO * O), 1, keepdims=True)
                # where no row sees more than 64 tokens delta does not come from the rounded out
                eo = 0 if min(self.window, T) <= 64 else 2.0 ** -8
                es = sc * (2.0 ** -8 * np.abs(dS) + P * (eo * e + 2.0 ** -14 * (np.abs(dP) + e)))
                refs = oa.window_attention_vjp(Q, K, V, dO, self.window, self.mode)
                bars = es @ np.abs(K), es.T @ np.abs(Q), (2.0 ** -8 + 2.0 ** -14) * (P.T @ np.abs(dO))
                for i, n in enumerate(("dq", "dk", "dv")):
                    got = dx[b, :, i * D + h * 128:i * D + h * 128 + 128]
                    r = np.max(np.abs(got - refs[i]) / (2.0 ** -8 * np.abs(refs[i]) + bars[i] + 1e-30))
                    worst[n] = max(worst.get(n, 0), r)
        say("  worst error / bar", {k: round(float(v), 3) for k, v in worst.items()})
        assert max(worst.values()) <= 1


WINDOWS = [(1, 1, 1, 5, "sliding"), (1, 1, 1, 5, "block"), (2, 2, 300, 37, "sliding"), (1, 1, 300, 1, "sliding"),
           (1, 2, 129, 64, "sliding"), (1, 1, 520, 128, "sliding"), (1, 1, 300, 1000, "sliding"), (2, 3, 257, 200, "sliding"),
           (1, 1, 300, 2 ** 31 - 1, "sliding"), (2, 2, 300, 50, "block"), (1, 1, 300, 64, "block"),
           (1, 1, 300, 1, "block"), (1, 2, 333, 300, "block"), (1, 1, 300, 2 ** 31 - 1, "block"), (3, 2, 777, 250, "block")]


@pytest.mark.parametrize("B,H,T,window,mode", WINDOWS)
def test_window_training_matches_oracle(B, H, T, window, mode):
    w = Window(B, H, T, window, mode, qscale=2.0 if T == 520 else 1.0)
    w.forward()
    w.backward()
    w.check()


@pytest.mark.parametrize("window,mode", [(500, "sliding"), (700, "block"), (50, "sliding"), (33, "block"),
                                         (4000, "sliding")])
def test_window_training_of_a_full_launch(window, mode):
    """More than 256 workgroups of 64 rows (the kernels' form for launches that fill the CUs)."""
    w = Window(2, 4, 2100, window, mode)
    w.forward()
    w.backward()
    w.check([(0, 0), (1, 3)])


@pytest.mark.parametrize("B,T,window,mode", [(2, 1000, 300, "sliding"), (2, 1000, 300, "block"),
                                             (4, 4200, 900, "sliding")])
def test_window_lse_output_is_the_window_attentions(B, T, window, mode):
    """Both within their bar of the exact row, so within twice the bar of each other."""
    w = Window(B, 2, T, window, mode)
    w.forward()
    plain = torch.empty_like(w.out)
    D = w.D
    W.ttt_window_attention(w.x, w.x[..., D:], w.x[..., 2 * D:], 3 * D + 8, plain, D, B, 2, T, window, mode)
    torch.cuda.synchronize()
    bar = 2 * (2.0 ** -8 * plain.float().abs() + 2.0 ** -7 * w.x.float().abs().max() + 1e-6)
    assert bool(((plain.float() - w.out.float()).abs() <= bar).all())


def test_window_training_with_growing_and_large_scores():
    """Scores that keep passing the running maximum by far, and scores of several hundred."""
    w = Window(1, 1, 700, 400, "sliding", qscale=30.0)
    w.x[0, :, 128:256] *= torch.linspace(0.1, 3.0, 700, device=DEV)[:, None].to(torch.bfloat16)
    w.forward()
    w.backward()
    w.check()


def test_window_backward_against_differences():
    """The fp64 forward differenced along one direction against the kernel's gradients: bf16
    gradients carry 2^-7 of the sum of their products with the direction."""
    w = Window(1, 1, 200, 60, "sliding")
    w.forward()
    w.backward()
    torch.cuda.synchronize()
    x, go, dx = np64(w.x[0]), np64(w.go[0, :, :128]), np64(w.dx[:200])
    d = np.random.default_rng(1).standard_normal((200, 384))

    def f(s):
        y = x[:, :384] + s * d
        return np.sum(go * blk.window_attention(y[:, :128], y[:, 128:256], y[:, 256:], 60, "sliding"))
    got, want = (f(1e-5) - f(-1e-5)) / 2e-5, np.sum(dx[:, :384] * d)
    assert abs(got - want) <= 2.0 ** -7 * np.sqrt(np.sum((dx[:, :384] * d) ** 2)) * 4


def test_window_training_repeats_and_replays():
    w = Window(1, 2, 700, 256, "sliding")
    w.forward()
    w.backward()
    torch.cuda.synchronize()
    eager = w.out.clone(), w.lse.clone(), w.dx.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.forward()
        w.backward()
    for _ in range(3):
        for t in (w.out, w.lse, w.dx):
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (w.out, w.lse, w.dx)):
            assert torch.equal(a, b)
        torch.randn(1000, device=DEV).sum().item()


# ------------------------------------------------------------------------ as they are used
def test_training_run_of_the_attention_sublayer():
    """Norm and rotation, window attention, and both backwards, on one projection's rows,
    against the chained fp64 formulas.  Bar: relative 2-norm 2^-6 per tensor (four bf16 stages,
    each at most 2^-8 of its own output per element)."""
    T, Hn, D, window = 300, 2, 128, 90
    r = Rope(T=T, Hq=Hn, Hk=Hn, D=D, rot=D, seed=11)
    qo, ko = (torch.empty(T, Hn * D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    W.ttt_qk_norm_rope(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, qo, Hn * D, ko, Hn * D, T)
    v = r.v[:, :Hn * D].contiguous()
    out, lse = torch.empty_like(qo), torch.empty(1, Hn, T, device=DEV)
    n = Hn * D
    W.ttt_window_attention_lse(qo, ko, v, n, out, n, lse, 1, Hn, T, window)
    go = torch.randn(T, n, generator=gen(12), device=DEV).to(torch.bfloat16)
    gq, gk, gv = (torch.empty_like(qo) for _ in range(3))
    W.ttt_window_attention_backward(qo, ko, v, n, out, n, lse, go, n, gq, gk, gv, n,
                                    torch.empty_like(lse), 1, Hn, T, window)
    dqw, dkw = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    work = torch.empty(W.ttt_qk_norm_rope_backward_work(r.cfg, T), dtype=torch.uint8, device=DEV)
    dq, dk = torch.empty_like(gq), torch.empty_like(gk)
    W.ttt_qk_norm_rope_backward(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, gq, n, gk, n, dq, n, dk,
                                n, dqw, dkw, work, T)
    torch.cuda.synchronize()
    q, k, vv = (r.heads(x) for x in "qkv")
    qr, kr = (oa.norm_rope(x, r.weight(w), r.ang, r.pairing, r.eps) for w, x in (("q", q), ("k", k)))
    g = np64(go).reshape(T, Hn, D)
    ref_o = np.stack([blk.window_attention(qr[:, h], kr[:, h], vv[:, h], window, "sliding") for h in range(Hn)], 1)
    grads = [oa.window_attention_vjp(qr[:, h], kr[:, h], vv[:, h], g[:, h], window, "sliding") for h in range(Hn)]
    rq, rk, rv = (np.stack([x[i] for x in grads], 1) for i in range(3))
    rq, rqw = oa.norm_rope_vjp(q, r.weight("q"), r.ang, r.pairing, r.eps, rq)
    rk, rkw = oa.norm_rope_vjp(k, r.weight("k"), r.ang, r.pairing, r.eps, rk)
    for name, got, ref in (("out", out, ref_o), ("dq", dq, rq), ("dk", dk, rk), ("dv", gv, rv), ("dqw", dqw, rqw),
                           ("dkw", dkw, rkw)):
        e = np.linalg.norm(np64(got).ravel() - ref.ravel()) / np.linalg.norm(ref)
        say(name, e)
        assert e <= 2.0 ** -6, (name, e)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_serving_run_prefill_then_decode(dtype):
    """A prompt appended to the cache, then tokens one by one, each attending to the cache
    through the window: every row is the window attention's row over the whole sequence (bf16
    cache: the same rounded keys and values; e4m3: those the cache holds)."""
    T, P, Hn, D, size, window = 150, 140, 2, 128, 16, 64
    r = Rope(T=T, Hq=Hn, Hk=Hn, D=D, rot=D, seed=13)
    r.pos.copy_(torch.arange(T, device=DEV, dtype=torch.int32)[None])
    r.ang = oa.angles(np64(r.pos), np64(r.freq))
    pages = 12
    ct = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k, v = new_cache(pages, Hn, size, D, ct)
    cache = W.make_kv_cache(k, v)
    order = torch.randperm(pages, generator=gen(14), device=DEV)
    table = order[None, :10].to(torch.int32).contiguous()
    t = torch.arange(T, device=DEV)
    slot = order[t // size] * size + t % size
    n = Hn * D
    qo = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
    W.ttt_qk_norm_rope_append(r.cfg, r.q, r.ld, r.k, r.ld, r.v, r.ld, r.qw, r.kw, r.freq, r.pos, cache, slot, qo, n, P)
    out = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
    work = torch.empty(max(1, W.ttt_paged_attention_work(cache, 1, Hn, 10, window)), dtype=torch.uint8, device=DEV)
    for i in range(P, T):
        x = r.x[i:i + 1]
        W.ttt_qk_norm_rope_append(r.cfg, x, r.ld, x[:, n:], r.ld, x[:, 2 * n:], r.ld, r.qw, r.kw, r.freq,
                                  r.pos[:, i].clone(), cache, slot[i:i + 1].clone(), qo[i:i + 1], n, 1)
        W.ttt_paged_attention(qo[i:i + 1], n, cache, table, torch.tensor([i + 1], dtype=torch.int32, device=DEV),
                              out[i:i + 1], n, None, 1, Hn, 10, window, 0.0, work)
    torch.cuda.synchronize()
    q = np64(qo).reshape(T, Hn, D)
    rows = [c.float()[order[t // size], :, t % size] for c in (k, v)]
    kk, vv = (np64(x) for x in rows)
    assert not np.isnan(kk).any() and not np.isnan(vv).any()
    y, bar = r.ref("q")
    assert np.all(np.abs(q[P:] - y[P:])[:] <= bar[P:])
    for h in range(Hn):
        ref = blk.window_attention(q[:, h], kk[:, h], vv[:, h], window, "sliding")[P:]
        got = np64(out[P:]).reshape(T - P, Hn, D)[:, h]
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * np.abs(vv).max())


# ------------------------------------------------------------------------ the binding's checks
def test_binding_refuses_wrong_tensors():
    r = Rope(T=4, Hq=2, Hk=1, D=64, rot=64)
    qo, ko = r.out(2), r.out(1)

    def call(**kw):
        a = dict(q=r.q, k=r.k, qw=r.qw, kw=r.kw, freq=r.freq, pos=r.pos, qo=qo, ko=ko)
        a.update(kw)
        W.ttt_qk_norm_rope(r.cfg, a["q"], r.ld, a["k"], r.ld, a["qw"], a["kw"], a["freq"], a["pos"], a["qo"], 144,
                           a["ko"], 80, 4)
    call()
    for kw, code in ((dict(q=r.q.cpu()), 4), (dict(q=r.q.float()), 3), (dict(pos=r.pos.long()), 3),
                     (dict(pos=r.pos[:, :3].contiguous()), 2), (dict(freq=r.freq.double()), 3),
                     (dict(qw=r.qw[:32]), 2), (dict(ko=ko[:1]), 2), (dict(qw=torch.ones(64, 2, device=DEV).bfloat16()[:, 0]), 2)):
        with pytest.raises(W.TTTError) as e:
            call(**kw)
        assert e.value.status == code, kw
    for shape, dt in (((2, 1, 4, 64), torch.float32), ((0, 1, 4, 64), torch.bfloat16), ((2, 4, 64), torch.bfloat16)):
        with pytest.raises(W.TTTError):
            W.make_kv_cache(torch.zeros(shape, device=DEV, dtype=dt), torch.zeros(shape, device=DEV, dtype=dt))
    x = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    W.make_kv_cache(x, x)      # one head: the same memory order
    x = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    with pytest.raises(W.TTTError):
        W.make_kv_cache(x, x)


def test_binding_refuses_rows_past_the_memory():
    """Row strides that lead past a tensor's memory, a cache or a stream of another device."""
    r = Rope(T=4, Hq=2, Hk=1, D=64, rot=64)
    flat = torch.zeros(3 * 256 + 128, device=DEV, dtype=torch.bfloat16)   # 4 rows 256 apart, to the element
    ko = r.out(1)

    def call(qo, ld):
        W.ttt_qk_norm_rope(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, qo, ld, ko, 80, 4)
    call(flat, 256)
    third = torch.zeros(4, 384, device=DEV, dtype=torch.bfloat16)
    call(third[:, 256:], 384)
    for qo, ld in ((flat, 264), (flat[:-8], 256), (third[:, 256:], 392), (third[:, :128].contiguous(), 136)):
        with pytest.raises(W.TTTError) as e:
            call(qo, ld)
        assert e.value.status == 2

    kv = torch.zeros(2, 1, 4, 64, device=DEV, dtype=torch.bfloat16)
    c = W.make_kv_cache(kv, torch.zeros_like(kv))
    q = torch.zeros(2, 64, device=DEV, dtype=torch.bfloat16)
    out, table = torch.ones_like(q), torch.zeros(2, 1, device=DEV, dtype=torch.int32)
    lens = torch.zeros(2, device=DEV, dtype=torch.int32)

    def attend(ld=64, **kw):
        W.ttt_paged_attention(q, ld, c, table, lens, out, 64, None, 2, 1, 1, 0, 0.0, None, **kw)
    attend()
    assert not out.any()
    x = torch.zeros(6, 128, device=DEV, dtype=torch.bfloat16)
    stat = torch.zeros(6, device=DEV)

    def window(ld, ld_out):
        W.ttt_window_attention_lse(x, x, x, ld, torch.zeros_like(x), ld_out, stat, 2, 1, 3, 2)
    window(128, 128)
    other = type("Stream", (), dict(device=torch.device("cuda", c.device + 1), cuda_stream=0))
    c.device += 1
    for bad, code in ((lambda: attend(ld=72), 2), (attend, 4), (lambda: attend(stream=other), 4),
                      (lambda: window(136, 128), 2), (lambda: window(128, 136), 2)):
        with pytest.raises(W.TTTError) as e:
            bad()
        assert e.value.status == code


def test_binding_refuses_tables_of_another_layout():
    """Tables whose rows would be read with another length than they have: a page table wider than
    max_pages, positions for more tokens than the call's, statistics with their axes turned."""
    p = Paged([40, 33, 20], 4, 2, 64, 16)
    wide = torch.nn.functional.pad(p.table, (0, 5), value=-1).contiguous()
    turned = torch.zeros(4, 3, device=DEV)
    r = Rope(T=4, Hq=2, Hk=1, D=64, rot=64, axes=2)
    w = Window(2, 3, 5, 2, "sliding")
    stat, pos, lse = torch.zeros(2, 5, 3, device=DEV), torch.cat((r.pos, r.pos), 1).contiguous(), p.lse

    def attend(table, lse):
        W.ttt_paged_attention(p.q, p.q.stride(0), p.cache, table, p.lens, p.out, p.out.stride(0), lse, 3, 4,
                              p.width, 0, 0.0, p.work())

    def bad_pos():
        r.pos = pos
        r.call()

    def bad_stat(call):
        w.lse = stat
        call()
    p.call()
    w.forward()
    for bad in (lambda: attend(wide, lse), lambda: attend(p.table, turned), bad_pos, lambda: bad_stat(w.forward),
                lambda: bad_stat(w.backward)):
        with pytest.raises(W.TTTError) as e:
            bad()
        assert e.value.status == 2
    attend(p.table.flatten(), lse)
    p.check()
    # one sequence: the rest of its row is not read
    one = Paged([40], 4, 2, 64, 16)
    W.ttt_paged_attention(one.q, one.q.stride(0), one.cache, torch.nn.functional.pad(one.table, (0, 5)), one.lens,
                          one.out, one.out.stride(0), one.lse, 1, 4, one.width, 0, 0.0, one.work())
    one.check()


def test_binding_refuses_rows_of_another_layout():
    """Tensors whose own rows are not ld apart, which would be read as if they were."""
    T, Hn, D = 6, 4, 64
    r = Rope(T=T, Hq=Hn, Hk=Hn, D=D, rot=64)
    n = Hn * D
    qo, ko = (torch.zeros(T, n, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    x = r.x[:, :n].contiguous().view(T, Hn, D)

    def call(q, qo):
        W.ttt_qk_norm_rope(r.cfg, q, n, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, qo, n, ko, n, T)
    call(x, qo)
    r.check(torch.cat((qo, torch.full_like(qo, 7.0))), torch.cat((ko, torch.full_like(ko, 7.0))))
    first = qo.clone()
    call(x.transpose(0, 1), qo)     # the heads named before the tokens: the same memory
    torch.cuda.synchronize()
    assert torch.equal(qo, first)
    turned = torch.zeros(Hn, T, D, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    for q, o in ((turned, qo), (x, turned), (torch.zeros(T, 2 * n, dtype=torch.bfloat16, device=DEV), qo)):
        with pytest.raises(W.TTTError) as e:
            call(q, o)
        assert e.value.status == 2


@pytest.mark.parametrize("n,window,D,size", [(50, 0, 128, 16), (3000, 0, 128, 16), (3000, 700, 64, 24), (400, 0, 256, 7)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_paged_attention_keeps_infinities_to_what_sees_them(bad, n, window, D, size):
    """An infinite key, whose scores are +inf for one query head and -inf for another, gives NaN
    for both, out and lse; an infinite value NaN in its element; tokens outside the window, other
    heads and other sequences are as without."""
    p = Paged([n, 60, 60, 0], 4, 2, D, size)
    at = n - 20                                       # a token of sequence 0 that the window holds
    p.q[0, 2 * D + 5], p.q[0, 3 * D + 5] = 1.0, -1.0
    p.call(window)
    torch.cuda.synchronize()
    clean, lse = p.out.clone(), p.lse.clone()
    p.k[int(p.table[0, at // size]), 1, at % size, 5] = bad              # heads 2 and 3 of sequence 0
    for j in (0, 7, 59):                                                 # elements of weights of all sizes
        p.v[int(p.table[1, j // size]), 0, j % size, j] = bad            # heads 0 and 1 of sequence 1
    if window:
        p.k[int(p.table[0, 1]), 0, 3, 5] = p.v[int(p.table[0, 1]), 0, 4, 5] = bad    # before the window
    p.call(window)
    torch.cuda.synchronize()
    h2 = slice(2 * D, 4 * D)
    assert bool(p.out[0, h2].isnan().all()) and bool(p.lse[0, 2:].isnan().all())
    p.out[0, h2], p.lse[0, 2:] = clean[0, h2], lse[0, 2:]
    for j in (0, 7, 59):
        for h in (0, 1):
            assert bool(p.out[1, h * D + j].isnan()), (j, h)
            p.out[1, h * D + j] = clean[1, h * D + j]
    assert torch.equal(p.out, clean) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("n", [3, 3000])
def test_paged_attention_of_keys_that_are_all_infinite_is_not_an_empty_sequence(n):
    p = Paged([n, 0], 2, 2, 64, 16)
    p.q[0, 5], p.q[0, 64 + 5] = 1.0, -1.0
    for i in range(-(-n // 16)):
        p.k[int(p.table[0, i]), :, :, 5] = -float("inf")
    p.call()
    torch.cuda.synchronize()
    assert bool(p.out[0, :128].isnan().all()) and bool(p.lse[0].isnan().all())
    assert bool((p.out[1, :128] == 0).all()) and bool((p.lse[1] == -float("inf")).all())


def test_paged_attention_of_an_infinite_query_is_nan():
    p = Paged([50, 60], 4, 2, 128, 16)
    p.call()
    torch.cuda.synchronize()
    clean, lse = p.out.clone(), p.lse.clone()
    p.q[0, 128 + 3] = float("inf")
    p.call()
    torch.cuda.synchronize()
    assert bool(p.out[0, 128:256].isnan().all()) and bool(p.lse[0, 1].isnan())
    p.out[0, 128:256], p.lse[0, 1] = clean[0, 128:256], lse[0, 1]
    assert torch.equal(p.out, clean) and torch.equal(p.lse, lse)


# ------------------------------------------------------------------------ bars from the launch's own sums
@pytest.mark.parametrize("kw", [
    dict(T=5003, Hq=2, Hk=1, D=64, rot=64), dict(T=40001, Hq=1, Hk=1, D=32, rot=32, axes=3, act="f32"),
    dict(T=6001, Hq=3, Hk=2, D=128, rot=64, pairing="pairs"), dict(T=33000, Hq=2, Hk=1, D=64, rot=0, act="f32"),
    dict(T=9001, Hq=1, Hk=5, D=80, rot=32, axes=2, act="f32"), dict(T=2500, Hq=1, Hk=2, D=1024, rot=1024),
    dict(T=700, Hq=33, Hk=7, D=48, rot=48, act="f32")])
def test_scale_gradients_within_the_bar_of_their_chains(kw):
    """The scales' gradients against a bar that losing one token exceeds (the bar of the other
    tests grows with the tokens)."""
    r = Rope(**kw)
    refs, _, _, dqw, dkw = rope_backward(r)
    torch.cuda.synchronize()
    for which, dy, dw in (("q", refs[0], dqw), ("k", refs[1], dkw)):
        x = r.heads(which)
        _, ref = oa.norm_rope_vjp(x, r.weight(which), r.ang, r.pairing, r.eps, dy)
        xh = np.abs(x) / np.sqrt(np.mean(x * x, -1, keepdims=True) + r.eps)
        case, sizes, err = (r.T, x.shape[1], r.D, r.rot), r.both(dy) * xh, np64(dw) - ref
        worst = float(np.max(np.abs(err) / bars.scale_grad_bar(*case, np.sum(sizes, axis=(0, 1)), ref)))
        norm = float(np.linalg.norm(err) / bars.scale_grad_norm_bar(*case, np.sum(sizes ** 2, axis=(0, 1))))
        say("  error / bar", which, round(worst, 4), "of the norms", round(norm, 4))
        assert worst <= 1 and norm <= 1


@pytest.mark.parametrize("B,Hn,T,window,mode,problems", [
    (1, 1, 2100, 4000, "sliding", [(0, 0)]), (1, 1, 2100, 500, "sliding", [(0, 0)]),     # the form of few workgroups
    (1, 2, 700, 300, "block", [(0, 1)]), (1, 1, 300, 37, "sliding", [(0, 0)]), (1, 1, 65, 64, "sliding", [(0, 0)]),
    (2, 4, 2100, 4000, "sliding", [(0, 0), (1, 3)]), (2, 4, 2100, 500, "sliding", [(1, 2)]),    # of full launches
    (2, 4, 2100, 700, "block", [(0, 1)]), (2, 4, 2100, 50, "sliding", [(1, 3)]), (2, 4, 2100, 33, "block", [(0, 3)]),
    (2, 4, 2177, 2177, "block", [(1, 0)]),
])
def test_window_training_errors_are_those_of_its_roundings(B, Hn, T, window, mode, problems):
    """Every block of 32 rows of out, dq, dk and dv is as far off in the 2-norm as the bf16 roundings
    make it; one key or query left out is several times that."""
    w = Window(B, Hn, T, window, mode)
    w.forward()
    w.backward()
    torch.cuda.synchronize()
    D = w.D
    x, go, o, dx = np64(w.x), np64(w.go), np64(w.out), np64(w.dx[:B * T]).reshape(B, T, -1)
    for b, h in problems:
        cols = slice(h * 128, h * 128 + 128)
        Q, K, V = (x[b, :, i * D:(i + 1) * D][:, cols] for i in range(3))
        dO, P = go[b, :, cols], oa.window_probs(Q, K, window, mode)
        out = P @ V
        refs = (out, *oa.window_attention_vjp(Q, K, V, dO, window, mode))
        models = bars.window_models(Q, K, V, dO, P, out, min(window, T) <= 64)
        got = (o[b, :, cols], *(dx[b, :, i * D:(i + 1) * D][:, cols] for i in range(3)))
        assert np.all(np.abs(got[0] - out) <= bars.window_out_bar(P, V, out))
        worst = {n: bars.worst_block(*a) for n, *a in zip(("out", "dq", "dk", "dv"), got, refs, models)}
        say("  worst block / bar", {n: round(v, 3) for n, v in worst.items()})
        assert max(worst.values()) <= 1


@pytest.mark.parametrize("B,T,window,mode", [(2, 1000, 300, "sliding"), (2, 1000, 300, "block"), (4, 2200, 900, "sliding")])
def test_window_lse_output_and_the_window_attentions_differ_by_their_roundings(B, T, window, mode):
    """The training forward and the block's window attention: each within its roundings of the exact
    rows (the block's normaliser sums the rounded probabilities: their errors count once more)."""
    w = Window(B, 2, T, window, mode)
    w.forward()
    plain = torch.empty_like(w.out)
    D = w.D
    W.ttt_window_attention(w.x, w.x[..., D:], w.x[..., 2 * D:], 3 * D + 8, plain, D, B, 2, T, window, mode)
    torch.cuda.synchronize()
    x = np64(w.x[B - 1])
    Q, K, V = (x[:, i * D + 128:i * D + 256] for i in range(3))
    P = oa.window_probs(Q, K, window, mode)
    out = P @ V
    model = bars.window_models(Q, K, V, V, P, out, True)[0]
    norm = bars.R / np.sqrt(3) * np.sqrt(np.sum(P * P, 1, keepdims=True)) * np.abs(out)
    a, b = np64(w.out[B - 1, :, 128:256]), np64(plain[B - 1, :, 128:256])
    assert bars.worst_block(a, out, model) <= 1
    assert bars.worst_block(b, out, np.hypot(model, norm)) <= 1
    assert bars.worst_block(a, b, np.sqrt(2) * np.hypot(model, norm)) <= 1


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (64, "e4m3"), (128, "bf16"), (128, "e4m3"), (256, "bf16"), (256, "e4m3")])
@pytest.mark.parametrize("window", [0, 9001])
def test_paged_attention_counts_every_token_of_a_long_sequence(D, dtype, window):
    """Small scores: every token weighs about one part in its sequence's length, and the bar of
    lse, which goes with the scores' size, is below a third of what a lost token moves it by."""
    lens = [20011, 4097, 2049, 2048, 2047, 513, 0]
    p = Paged(lens, 4, 2, D, 24, dtype=dtype, qscale=0.01)
    q = np64(p.q[:, :4 * D]).reshape(-1, 4, D)
    kmax = np.sqrt(np.nansum(p.values()[0] ** 2, -1).max())
    d = np.sqrt(np.sum(q * q, -1).max()) * kmax * (D + 4) * U / np.sqrt(D)     # as check() has it
    longest = min(lens[0], window or lens[0])
    least = np.exp(-2 * np.sqrt(np.sum(q * q, -1).max()) * kmax / np.sqrt(D)) / longest
    assert d + 4 * U * (np.log(longest) + 2) < least / 3
    p.call(window)
    p.check(window)


def test_rotation_angles_keep_more_than_32_bits():
    """Unit pairs (1, 0) turn into (cos, sin) of their angles. Bar, in half steps U of fp32 at 1: the
    sine and cosine of a 32-bit angle are within one unit in the last place (1 U), the turn by
    the rest of the angle rounds once more (U / 2); the rounding of the angle itself (up to pi / 2
    U) must not be seen."""
    T, D = 4000, 128
    r = Rope(T=T, Hq=1, Hk=1, D=D, rot=D, axes=2, act="f32", norm="none")
    r.x.zero_()
    r.x[:, :D // 2], r.x[:, D:D + D // 2] = 1, 1
    qo, ko = r.call()
    torch.cuda.synchronize()
    for o in (qo, ko):
        y = np64(o[:T, :D])
        for got, want in ((y[:, :D // 2], np.cos(r.ang)), (y[:, D // 2:], np.sin(r.ang))):
            worst = float(np.abs(got - want).max() / U)
            say("  worst half steps", round(worst, 3))
            assert worst <= 1.75


# ------------------------------------------------------------------------ whole steps in a graph
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_decoding_step_captured_once_serves_every_token(dtype):
    """Append and attention of one new token for three sequences in one graph, replayed with the
    tokens, positions, slots and lengths changed in place, beside the same calls made eagerly on
    caches of their own, on another stream; a sequence that pauses has slot -1."""
    S, Hq, Hk, D, size, width, steps = 3, 4, 2, 128, 7, 40, 9
    r = Rope(T=S * steps, Hq=Hq, Hk=Hk, D=D, rot=D, seed=31)
    ct = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    scale = (0.02 + 0.02 * torch.rand(Hk, generator=gen(32), device=DEV)) if dtype == "e4m3" else None
    pages = S * width
    order = torch.randperm(pages, generator=gen(33), device=DEV).to(torch.int32).view(S, width)
    start = torch.tensor([270, 0, 13], dtype=torch.int32, device=DEV)
    fill = [torch.randn(pages, Hk, size, D, generator=gen(34 + i), device=DEV).to(ct) for i in range(2)]

    class Side:
        def __init__(self):
            self.kv = [f.clone() for f in fill]
            self.cache = W.make_kv_cache(*self.kv, k_scale=scale, v_scale=scale)
            self.x = torch.zeros(S, r.ld, dtype=r.dt, device=DEV)
            self.pos = torch.zeros(1, S, dtype=torch.int32, device=DEV)
            self.slot = torch.zeros(S, dtype=torch.int64, device=DEV)
            self.lens = start.clone()
            self.q, self.out = (torch.empty(S, Hq * D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            self.lse = torch.empty(S, Hq, device=DEV)
            self.work = torch.empty(max(1, W.ttt_paged_attention_work(self.cache, S, Hq, width, 0)),
                                    dtype=torch.uint8, device=DEV)

        def step(self, i):
            """The next token's inputs; sequence 1 pauses at step 4."""
            self.x.copy_(r.x[S * i:S * i + S])
            self.pos.copy_(self.lens[None])
            at = self.lens.long()
            page = order.gather(1, (at // size)[:, None])[:, 0].long()
            self.slot.copy_(page * size + at % size)
            self.lens.add_(1)
            if i == 4:
                self.slot[1] = -1
                self.lens[1] -= 1

        def call(self, **kw):
            n = Hq * D
            W.ttt_qk_norm_rope_append(r.cfg, self.x, r.ld, self.x[:, n:], r.ld, self.x[:, n + Hk * D:], r.ld, r.qw, r.kw,
                                      r.freq, self.pos, self.cache, self.slot, self.q, n, S, **kw)
            W.ttt_paged_attention(self.q, n, self.cache, order, self.lens, self.out, n, self.lse, S, Hq, width, 0, 0.0,
                                  self.work, **kw)

        def results(self):
            return [t.view(torch.uint8) if t.element_size() == 1 else t for t in (self.q, self.out, self.lse, *self.kv)]

    eager, replayed = Side(), Side()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        replayed.call()
    for i in range(steps):
        eager.step(i)
        side.wait_stream(torch.cuda.current_stream())
        eager.call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        replayed.step(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.results(), replayed.results()):
            assert torch.equal(a, b), i
        torch.randn(1000, device=DEV).sum().item()
    assert bool(eager.out.isfinite().all())


@pytest.mark.parametrize("T,window,mode", [(300, 90, "sliding"), (3000, 40, "block")])
def test_a_training_step_captured_serves_other_inputs(T, window, mode):
    """Norm and rotation, window attention and both backwards in one graph on one projection's rows,
    replayed with other inputs, against the calls made eagerly on a stream of their own."""
    Hn, D = 6, 128
    n = Hn * D
    r = Rope(T=T, Hq=Hn, Hk=Hn, D=D, rot=D, seed=41)
    go = torch.empty(T, n, dtype=r.dt, device=DEV)

    def side():
        t = dict(qkv=torch.empty(T, 3 * n, dtype=r.dt, device=DEV), out=torch.empty(T, n, dtype=r.dt, device=DEV),
                 lse=torch.empty(1, Hn, T, device=DEV), g=torch.empty(T, 3 * n, dtype=r.dt, device=DEV),
                 dqw=torch.empty(D, device=DEV), dkw=torch.empty(D, device=DEV))
        stat = torch.empty(1, Hn, T, device=DEV)
        work = torch.empty(W.ttt_qk_norm_rope_backward_work(r.cfg, T), dtype=torch.uint8, device=DEV)

        def call(**kw):
            q, g = t["qkv"], t["g"]
            W.ttt_qk_norm_rope(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, q, 3 * n, q[:, n:], 3 * n, T, **kw)
            W.ttt_window_attention_lse(q, q[:, n:], q[:, 2 * n:], 3 * n, t["out"], n, t["lse"], 1, Hn, T, window, mode, **kw)
            W.ttt_window_attention_backward(q, q[:, n:], q[:, 2 * n:], 3 * n, t["out"], n, t["lse"], go, n, g, g[:, n:],
                                            g[:, 2 * n:], 3 * n, stat, 1, Hn, T, window, mode, **kw)
            W.ttt_qk_norm_rope_backward(r.cfg, r.q, r.ld, r.k, r.ld, r.qw, r.kw, r.freq, r.pos, g, 3 * n, g[:, n:], 3 * n,
                                        g, 3 * n, g[:, n:], 3 * n, t["dqw"], t["dkw"], work, T, **kw)
        return t, call
    (a, eager), (b, captured) = side(), side()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured()
    for i in range(4):
        r.x.copy_(torch.randn(r.x.shape, generator=gen(50 + i), device=DEV))
        go.copy_(torch.randn(go.shape, generator=gen(60 + i), device=DEV))
        for t in (a, b):
            t["qkv"][:, 2 * n:] = r.v[:, :n]
        stream.wait_stream(torch.cuda.current_stream())
        eager(stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
        graph.replay()
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k], b[k]) and bool(a[k].isfinite().all()), (i, k)
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.parametrize("axes", [1, 2, 4])
def test_rotation_angles_of_far_positions(axes):
    """Positions anywhere in int32 against angles in 60 decimal digits (64 bits leave up to 2^-22
    radians of 2^31): the bar of near ones, and 2^-30 for the reference's own steps."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    tau = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    T, rot = 60, 64
    r = Rope(T=T, Hq=1, Hk=1, D=rot, rot=rot, axes=axes, act="f32", norm="none", far=True)
    r.freq[:, ::3] = torch.rand(r.freq[:, ::3].shape, generator=gen(71), device=DEV) * 0.5 + 0.5
    r.pos[:, :2], r.pos[:, 2:4] = 2 ** 31 - 1, -2 ** 31
    r.x.zero_()
    r.x[:, :rot // 2], r.x[:, rot:rot + rot // 2] = 1, 1
    pos, freq = r.pos.cpu().tolist(), [[Decimal(x) for x in row] for row in r.freq.double().cpu().tolist()]
    ang = np.empty((T, rot // 2))
    for t in range(T):
        for j in range(rot // 2):
            x = sum(pos[a][t] * freq[a][j] for a in range(axes)) / tau
            ang[t, j] = float((x - x.to_integral_value()) * tau)
    qo, ko = r.call()
    torch.cuda.synchronize()
    for o in (qo, ko):
        y = np64(o[:T, :rot])
        worst = max(float(np.abs(y[:, :rot // 2] - np.cos(ang)).max()), float(np.abs(y[:, rot // 2:] - np.sin(ang)).max()))
        say("  worst half steps", round(worst / U, 3))
        assert worst <= 1.75 * U + 2.0 ** -30
