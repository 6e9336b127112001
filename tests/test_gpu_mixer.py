"""GPU parity of the mixer calls (include/ttt_mixer.h) against the fp64 oracle (oracle/ttt_mixer.py),
element by element, within the error models of mixer_bars.py."""
import numpy as np
import pytest
import torch

import mixer_bars as bars
import oracle.ttt_mixer as om
import weight_sequence_layers_amd as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF = torch.bfloat16


def np64(t):
    return t.detach().double().cpu().numpy()


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def worst(got, ref, bar):
    e = np.abs(got - ref) / bar
    return float(np.max(e)) if e.size else 0.0


# ------------------------------------------------------------------------ linear attention
class Linear:
    """A case: sequences of `lens` tokens, packed with `gap` rows that belong to none after each (with a gap
    or unequal lengths the call takes starts), q, k and v parts of one row."""

    def __init__(self, lens, heads=2, K=64, V=64, gap=0, decay=None, scale=0.0, seed=1, pad=8, dense=False):
        say(f"linear lens={lens} heads={heads} K={K} V={V} gap={gap} decay={decay}")
        self.lens, self.heads, self.K, self.V, self.dense = list(lens), heads, K, V, dense
        self.B, self.T = len(lens), max(list(lens) + [0])
        self.cfg = W.make_linear_attention_config(heads=heads, dim_k=K, dim_v=V, scale=scale)
        self.scale = scale or K ** -0.5
        self.first = np.concatenate([[0], np.cumsum([n + gap for n in lens])]).astype(np.int64)
        self.rows = int(self.first[-1])
        g = gen(seed)
        self.ld = heads * (2 * K + V) + pad
        self.x = torch.randn(self.rows, self.ld, generator=g, device=DEV).to(BF)
        self.q, self.k, self.v = self.x, self.x[:, heads * K:], self.x[:, 2 * heads * K:]
        d = [0.9, 0.5, 1.0, 0.99, 0.0] if decay is None else decay
        self.decay = torch.tensor([d[h % len(d)] for h in range(heads)], device=DEV)
        # the rows of a gap are sequences of their own, which the checks leave out
        self.starts = None
        if not dense:
            cut = [0]
            for n in lens:
                cut += [cut[-1] + n] + ([cut[-1] + n + gap] if gap else [])
            self.seqs = list(range(0, len(cut) - 1, 2 if gap else 1))
            self.starts = torch.tensor(cut, device=DEV, dtype=torch.int32)
            if gap:
                self.B = len(cut) - 1
        else:
            self.seqs = list(range(self.B))

    def states(self, seed=2, slots=None):
        return 3 * torch.randn(self.B if slots is None else slots, self.heads, self.K, self.V, generator=gen(seed),
                               device=DEV)

    def out(self, n, extra=3):
        return torch.full((self.rows + extra, self.heads * n + 8), 7.0, dtype=BF, device=DEV)

    def work(self, backward=False):
        f = W.ttt_linear_attention_backward_work if backward else W.ttt_linear_attention_work
        return torch.empty(f(self.cfg, self.B, self.T), dtype=torch.uint8, device=DEV)

    def call(self, sin=None, sout=None, slot=None, out=None, work=None, **kw):
        out = self.out(self.V) if out is None else out
        W.ttt_linear_attention(self.cfg, self.q, self.ld, self.k, self.ld, self.v, self.ld, self.decay, self.starts, sin,
                               sout, slot, out, out.stride(0), self.rows, self.B, self.T,
                               self.work() if work is None else work, **kw)
        return out

    def back(self, dout, sin=None, ds=None, dsin=None, grads=None, work=None):
        dq, dk, dv = grads or (self.out(self.K), self.out(self.K), self.out(self.V))
        W.ttt_linear_attention_backward(self.cfg, self.q, self.ld, self.k, self.ld, self.v, self.ld, self.decay,
                                        self.starts, sin, dout, dout.stride(0), ds, dq, dq.stride(0), dk, dk.stride(0),
                                        dv, dv.stride(0), dsin, self.rows, self.B, self.T,
                                        self.work(True) if work is None else work)
        return dq, dk, dv

    def part(self, t, i, h, n):
        """Rows of sequence i (of lens) and head h of t, whose heads have n elements."""
        a = int(self.first[i])
        return np64(t[a:a + self.lens[i], h * n:(h + 1) * n])

    def qkv(self, i, h):
        return self.part(self.q, i, h, self.K), self.part(self.k, i, h, self.K), self.part(self.v, i, h, self.V)

    def lam(self, h):
        return float(np64(self.decay)[h])

    def kept(self, t, n):
        """Rows of no sequence, rows behind the last and columns behind the heads stay."""
        mine = torch.zeros(len(t), dtype=torch.bool, device=DEV)
        for i, m in enumerate(self.lens):
            mine[int(self.first[i]):int(self.first[i]) + m] = True
        return bool((t[~mine] == 7).all()) and bool((t[:, self.heads * n:] == 7).all())

    def check(self, out, sout=None, sin=None, entry=None):
        torch.cuda.synchronize()
        zero = np.zeros((self.K, self.V))
        for i, b in enumerate(self.seqs):
            at = b if entry is None else entry[b]
            for h in range(self.heads):
                s0 = zero if sin is None or at is None else np64(sin[at, h])
                (o, bar), (S, sbar) = bars.forward(*self.qkv(i, h), self.lam(h), s0, self.scale)
                w = worst(self.part(out, i, h, self.V), o, bar)
                assert w <= 1, ("out", i, h, w)
                if sout is not None and at is not None:
                    w = worst(np64(sout[at, h]), S, sbar)
                    assert w <= 1, ("state", i, h, w)


# dense batches, ragged ones, one and more segments, every pair of dims
LINEAR = [
    dict(lens=[1], heads=1, K=64, V=64, dense=True), dict(lens=[1, 1, 1], heads=3, K=128, V=64, dense=True),
    dict(lens=[31], K=128, V=128), dict(lens=[32, 32], K=64, V=128, dense=True), dict(lens=[33], K=256, V=64),
    dict(lens=[5, 0, 64, 1], K=128, V=128), dict(lens=[0], K=64, V=64), dict(lens=[0, 0, 3], K=64, V=256),
    dict(lens=[257, 100, 511], K=256, V=256, heads=1), dict(lens=[777, 777], K=128, V=128, dense=True),
    dict(lens=[1000, 3, 0, 2500, 512], K=64, V=64, heads=5), dict(lens=[3001], K=128, V=256, heads=1),
    dict(lens=[2048], K=256, V=128, heads=1, decay=[0.9995]), dict(lens=[513, 512, 511], gap=5, K=64, V=128),
    dict(lens=[700] * 3, heads=1, K=128, V=128, scale=2.5, decay=[1.0]),
    dict(lens=[40] * 130, heads=2, K=64, V=64),
]


@pytest.mark.parametrize("kw", LINEAR)
@pytest.mark.parametrize("states", [False, True])
def test_linear_attention_matches_oracle(kw, states):
    c = Linear(**kw)
    sin = c.states() if states else None
    sout = torch.full_like(sin, 7.0) if states else None
    out = c.call(sin, sout)
    c.check(out, sout, sin)
    if not kw.get("gap"):
        assert c.kept(out, c.V)


@pytest.mark.parametrize("kw", LINEAR)
@pytest.mark.parametrize("states", [False, True])
def test_linear_attention_backward_matches_oracle(kw, states):
    c = Linear(**kw)
    g = gen(5)
    dout = torch.randn(c.rows, c.heads * c.V + 16, generator=g, device=DEV).to(BF)
    sin, ds = (c.states(), c.states(3)) if states else (None, None)
    dsin = torch.full_like(ds, 7.0) if states else None
    dq, dk, dv = c.back(dout, sin, ds, dsin)
    torch.cuda.synchronize()
    zero = np.zeros((c.K, c.V))
    for i, b in enumerate(c.seqs):
        for h in range(c.heads):
            s0, d1 = (np64(sin[b, h]), np64(ds[b, h])) if states else (zero, zero)
            ref = bars.backward(*c.qkv(i, h), c.lam(h), s0, c.scale, c.part(dout, i, h, c.V), d1)
            got = [c.part(dq, i, h, c.K), c.part(dk, i, h, c.K), c.part(dv, i, h, c.V)]
            for name, x, (y, bar) in zip(("dq", "dk", "dv"), got, ref):
                w = worst(x, y, bar)
                assert w <= 1, (name, i, h, w)
            if states:
                w = worst(np64(dsin[b, h]), *ref[3])
                assert w <= 1, ("dstate_in", i, h, w)
    if not kw.get("gap"):
        assert c.kept(dq, c.K) and c.kept(dk, c.K) and c.kept(dv, c.V)


def test_linear_attention_keeps_rows_of_no_sequence():
    """starts that leave rows out before the first and behind the last sequence."""
    c = Linear(lens=[70, 40], K=64, V=64)
    c.starts = torch.tensor([20, 70, 100], dtype=torch.int32, device=DEV)
    out = c.out(64)
    c.call(out=out)
    torch.cuda.synchronize()
    assert bool((out[:20] == 7).all()) and bool((out[100:] == 7).all())
    c.lens, c.first = [50, 30], np.array([20, 70, 100])
    c.check(out)
    d = Linear(lens=[70, 40], K=64, V=64)
    d.starts = c.starts
    grads = d.back(torch.randn(d.rows, 128, generator=gen(3), device=DEV).to(BF))
    torch.cuda.synchronize()
    for g in grads:
        assert bool((g[:20] == 7).all()) and bool((g[100:] == 7).all())


def test_linear_attention_of_starts_that_are_out_of_order():
    """Starts outside the rows count as the nearer end, an end before its start as an empty sequence and
    a sequence longer than seq_len as that long."""
    c = Linear(lens=[60, 60], K=64, V=64)
    c.starts = torch.tensor([-5, 30, 1000, 990], dtype=torch.int32, device=DEV)
    c.B, c.T, c.seqs = 3, 50, [0, 1, 2]
    sin, sout = c.states(), torch.full((3, 2, 64, 64), 7.0, device=DEV)
    out = c.call(sin, sout)
    c.lens, c.first = [30, 50, 0], np.array([0, 30, 120, 120])
    c.check(out, sout, sin)
    assert bool((out[80:] == 7).all())


def test_linear_attention_slots():
    c = Linear(lens=[300, 3, 0, 64, 33], K=128, V=64)
    sin = c.states(slots=9)
    sout = torch.full_like(sin, 7.0)
    slot = torch.tensor([4, -1, 8, 0, 9], dtype=torch.int32, device=DEV)   # two of them nowhere
    entry = [4, None, 8, 0, None]
    out = c.call(sin, sout, slot)
    c.check(out, sout, sin, entry)
    others = [i for i in range(9) if i not in entry]
    assert bool((sout[others] == 7).all())
    assert torch.equal(sout[8], sin[8])          # an empty sequence's
    pool = sin.clone()
    again = c.call(pool, pool, slot)             # in place
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(pool[[4, 0]], sout[[4, 0]])
    assert torch.equal(pool[others], sin[others])
    last = c.call(None, sout, slot)              # from zeros
    c.check(last, sout, None, entry)
    c.check(c.call(sin, None, slot), None, sin, entry)    # no state asked for


@pytest.mark.parametrize("T,K,V", [(700, 128, 128), (2500, 64, 64)])
def test_linear_attention_in_place_over_several_segments(T, K, V):
    c = Linear(lens=[T, T // 2], K=K, V=V, heads=1)
    pool, sout = c.states(), c.states(9)
    want = c.call(pool, sout)
    got = c.call(pool, pool)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(pool, sout)


def test_linear_attention_continues_where_it_stopped():
    """A prompt in two calls, the state carried between them, is the prompt in one."""
    T, cut = 1000, 417
    c = Linear(lens=[T], K=128, V=128, decay=[0.99, 1.0])
    state = c.states()
    sin = state.clone()
    out, work = c.out(128), c.work()
    for a, b in ((0, cut), (cut, T)):
        W.ttt_linear_attention(c.cfg, c.q[a:b], c.ld, c.k[a:b], c.ld, c.v[a:b], c.ld, c.decay, None, state, state, None,
                               out[a:b], out.stride(0), b - a, 1, b - a, work)
    c.check(out, state, sin)


@pytest.mark.parametrize("heads,K,V", [(2, 128, 128), (3, 64, 256), (1, 256, 64)])
def test_linear_attention_steps_are_a_prompt(heads, K, V):
    """Single tokens one after another against the oracle's recurrence."""
    S, T = 3, 40
    c = Linear(lens=[T] * S, heads=heads, K=K, V=V, dense=True)
    sin = c.states()
    state, out = sin.clone(), c.out(V)
    for t in range(T):
        at = lambda x: x[t:S * T:T]  # noqa: E731
        q, k, v = (at(x).contiguous() for x in (c.q, c.k, c.v))
        o = torch.empty(S, heads * V, dtype=BF, device=DEV)
        W.ttt_linear_attention_step(c.cfg, q, q.stride(0), k, k.stride(0), v, v.stride(0), c.decay, state, state, None,
                                    o, heads * V, S)
        out[t:S * T:T, :heads * V] = o
    c.check(out, state, sin)


STEPS = [dict(S=1, heads=1, K=64, V=64), dict(S=1, heads=8, K=128, V=128), dict(S=61, heads=3, K=64, V=128),
         dict(S=300, heads=4, K=128, V=64), dict(S=130, heads=4, K=256, V=256), dict(S=5, heads=2, K=128, V=256),
         dict(S=1000, heads=2, K=64, V=64), dict(S=7, heads=1, K=256, V=64)]


@pytest.mark.parametrize("kw", STEPS)
@pytest.mark.parametrize("pool", [True, False])
def test_linear_attention_step_matches_oracle(kw, pool):
    S, heads, K, V = kw["S"], kw["heads"], kw["K"], kw["V"]
    c = Linear(lens=[1] * S, heads=heads, K=K, V=V, dense=True, decay=[0.9, 0.0, 1.0])
    sin = c.states(slots=S + 2) if pool else None
    sout = torch.full((S + 2, heads, K, V), 7.0, device=DEV)
    slot = torch.randperm(S + 2, generator=gen(3), device=DEV)[:S].to(torch.int32)
    if S > 2:
        slot[1] = -1
    if S > 4:
        slot[3] = S + 2
    out = c.out(V)
    W.ttt_linear_attention_step(c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay, sin, sout, slot, out, out.stride(0), S)
    torch.cuda.synchronize()
    assert c.kept(out, V)
    at = [int(x) if 0 <= int(x) < S + 2 else None for x in slot.cpu()]
    some = list(range(S)) if S <= 64 else [0, 1, 3, S // 2, S - 1]
    for b in some:
        for h in range(heads):
            q, k, v = (x[0] for x in c.qkv(b, h))
            s0 = np.zeros((K, V)) if sin is None or at[b] is None else np64(sin[at[b], h])
            new = c.lam(h) * s0 + np.outer(k, v)
            size = np.abs(c.lam(h) * s0) + np.abs(np.outer(k, v))
            ref, bar = c.scale * (new.T @ q), c.scale * (size.T @ np.abs(q))
            # the state two roundings, the sum K more in some order, the scale
            got = np64(out[b, h * V:(h + 1) * V])
            assert worst(got, ref, 2.0 ** -8 * np.abs(ref) + (K + 4) * 2.0 ** -24 * bar + 1e-30) <= 1
            if at[b] is not None:
                assert worst(np64(sout[at[b], h]), new, 2 * 2.0 ** -24 * size + 1e-30) <= 1
    others = [i for i in range(S + 2) if i not in at]
    assert bool((sout[others] == 7).all())


def test_linear_attention_step_in_place_and_without_a_state():
    c = Linear(lens=[1] * 6, heads=2, K=128, V=128, dense=True)
    sin, a, b, d = c.states(), c.out(128), c.out(128), c.out(128)
    args = (c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay)
    sout = torch.empty_like(sin)
    W.ttt_linear_attention_step(*args, sin, sout, None, a, a.stride(0), 6)
    W.ttt_linear_attention_step(*args, sin, None, None, d, d.stride(0), 6)
    pool = sin.clone()
    W.ttt_linear_attention_step(*args, pool, pool, None, b, b.stride(0), 6)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, d) and torch.equal(pool, sout)


def test_linear_attention_step_keeps_what_is_not_finite_to_its_head():
    c = Linear(lens=[1] * 4, heads=2, K=64, V=64, dense=True)
    sin = c.states()
    args = (c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay)
    clean, sclean, out, sout = c.out(64), torch.empty_like(sin), c.out(64), torch.empty_like(sin)
    W.ttt_linear_attention_step(*args, sin, sclean, None, clean, clean.stride(0), 4)
    sin[1, 0, 3, 5] = float("inf")
    c.x[2, 64 + 7] = float("nan")        # a query of sequence 2, head 1
    W.ttt_linear_attention_step(*args, sin, sout, None, out, out.stride(0), 4)
    torch.cuda.synchronize()
    assert not bool(out[1, 5].isfinite()) and bool(out[2, 64:128].isnan().all())
    out[1, 5], out[2, 64:128] = clean[1, 5], clean[2, 64:128]
    sout[1, 0, 3, 5] = sclean[1, 0, 3, 5]
    assert torch.equal(out, clean) and torch.equal(sout, sclean)


def test_linear_attention_keeps_nan_to_its_sequence_and_head():
    c = Linear(lens=[100, 70, 100], heads=2, K=64, V=64)
    sin, sout, s2 = c.states(), c.states(4), c.states(4)
    clean = c.call(sin, sout)
    c.x[130, 64 + 3] = float("nan")      # sequence 1, head 1's query of its token 30
    c.x[130, 4 * 64 + 5] = float("nan")  # head 0's value
    out = c.call(sin, s2)
    torch.cuda.synchronize()
    assert bool(out[130, :128].isnan().any())
    out[100:170] = clean[100:170]
    s2[1] = sout[1]
    assert torch.equal(out, clean) and torch.equal(s2, sout)


def test_linear_attention_far_rows():
    """Rows more than 2^32 bytes behind the first."""
    ld, far = 1 << 20, 2200
    x = torch.empty(far + 40, ld, dtype=BF, device=DEV)          # 4.7 GB
    c = Linear(lens=[40, 40], K=64, V=64)
    for a, b in ((0, 0), (far, 40)):
        x[a:a + 40, :c.ld] = c.x[b:b + 40]
    out = torch.empty(far + 40, 128, dtype=BF, device=DEV)
    near = c.call()
    starts = torch.tensor([0, 40, far, far + 40], dtype=torch.int32, device=DEV)
    W.ttt_linear_attention(c.cfg, x, ld, x[:, 128:], ld, x[:, 256:], ld, c.decay, starts[[0, 1, 1]].contiguous(), None,
                           None, None, out, 128, far + 40, 2, 40, c.work())
    W.ttt_linear_attention(c.cfg, x, ld, x[:, 128:], ld, x[:, 256:], ld, c.decay, starts[[2, 3, 3]].contiguous(), None,
                           None, None, out, 128, far + 40, 2, 40, c.work())
    torch.cuda.synchronize()
    assert torch.equal(out[:40], near[:40, :128]) and torch.equal(out[far:], near[40:80, :128])


@pytest.mark.parametrize("lens", [[40, 33, 0, 64], [900, 20, 1500]])
def test_linear_attention_captured(lens):
    """Forward and backward in one graph, replayed with other inputs and starts beside eager calls on another
    stream with a workspace of their own."""
    c = Linear(lens=lens, heads=2, K=64, V=64)
    sin, ds = c.states(), c.states(3)
    sout, dsin = torch.empty_like(sin), torch.empty_like(sin)
    dout = torch.randn(c.rows, 128, generator=gen(8), device=DEV).to(BF)
    w, wb = c.work(), c.work(True)
    outs = [c.out(64), c.out(64), c.out(64), c.out(64)]

    def both(o, so, dso, w, wb):
        c.call(sin, so, out=o[0], work=w)
        c.back(dout, sin, ds, dso, grads=o[1:], work=wb)
    both(outs, sout, dsin, w, wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(outs, sout, dsin, w, wb)
    other = torch.cuda.Stream()
    eager = [c.out(64) for _ in range(4)]
    es, ed, ew, ewb = torch.empty_like(sin), torch.empty_like(sin), c.work(), c.work(True)
    base = c.starts.clone()
    for i in range(4):
        c.x.copy_(torch.randn(c.x.shape, generator=gen(20 + i), device=DEV).to(BF))
        c.starts.copy_(base)
        if i == 2:
            c.starts[1:-1] -= 7
        for t in (*outs, *eager):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            both(eager, es, ed, ew, ewb)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*outs, sout, dsin), (*eager, es, ed)))
        torch.randn(1000, device=DEV).sum().item()


def test_linear_attention_is_the_same_every_time():
    c = Linear(lens=[3000, 1234], K=128, V=128)
    sin, ds = c.states(), c.states(3)
    dout = torch.randn(c.rows, 256, generator=gen(8), device=DEV).to(BF)
    runs = []
    for _ in range(3):
        sout, dsin = torch.empty_like(sin), torch.empty_like(sin)
        junk = torch.full((W.ttt_linear_attention_backward_work(c.cfg, c.B, c.T),), 255, dtype=torch.uint8, device=DEV)
        runs.append([c.call(sin, sout, work=junk), *c.back(dout, sin, ds, dsin, work=junk), sout, dsin])
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_linear_attention_without_sequences_or_tokens():
    c = Linear(lens=[5], K=64, V=64)
    out = c.out(64)
    W.ttt_linear_attention(c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay, None, None, None, None, out, out.stride(0), 0, 0,
                           5, None)
    sin = c.states()
    sout = torch.full_like(sin, 7.0)
    W.ttt_linear_attention(c.cfg, None, c.ld, None, c.ld, None, c.ld, c.decay, None, sin, sout, None, None, c.ld, 0, 1, 0,
                           None)
    dsin = torch.full_like(sin, 7.0)
    W.ttt_linear_attention_backward(c.cfg, None, c.ld, None, c.ld, None, c.ld, c.decay, None, None, None, c.ld, sin,
                                    *(None, c.ld) * 3, dsin, 0, 1, 0, None)
    W.ttt_linear_attention_step(c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay, sin, sin, None, out, out.stride(0), 0)
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and torch.equal(sout, sin) and torch.equal(dsin, sin)


def test_linear_attention_of_the_largest_batch():
    """65535 sequences of one token, 2^20 sequences and heads together: out = scale (q . k) v; the weight in
    fp32 (64 roundings of 2^-24 of the products' sizes) and as two bf16 numbers (2^-16), out rounded."""
    B, heads, D = 65535, 16, 64
    cfg = W.make_linear_attention_config(heads=heads, dim_k=D)
    q, k, v = (torch.randn(B, heads * D, generator=gen(i), device=DEV).to(BF) for i in range(3))
    out, decay = torch.empty_like(q), torch.ones(heads, device=DEV)
    W.ttt_linear_attention(cfg, q, heads * D, k, heads * D, v, heads * D, decay, None, None, None, None, out, heads * D, B,
                           B, 1, None)
    torch.cuda.synchronize()
    q, k, v, o = (t.view(B, heads, D).double() for t in (q, k, v, out))
    p, size = (q * k).sum(-1, keepdim=True) / 8, (q * k).abs().sum(-1, keepdim=True) / 8
    assert bool(((o - p * v).abs() <= 2.0 ** -8 * (p * v).abs() + 2.0 ** -15 * size * v.abs()).all())


@pytest.mark.parametrize("lens", [[90, 64], [600]])
def test_linear_attention_of_decays_outside_the_unit_interval(lens):
    """Negative ones and ones past 1 are taken by the formula: (-a)^n = (-1)^n a^n, so that the results are
    those of a with every other key and query and the first state turned, within their bars."""
    c = Linear(lens=lens, heads=3, K=64, V=64, decay=[-0.9, 1.004, -1.0])
    sin, sout = c.states(), c.states()
    out = c.call(sin, sout)
    torch.cuda.synchronize()
    for i, n in enumerate(lens):
        for h, a in enumerate([-0.9, 1.004, -1.0]):
            q, k, v = c.qkv(i, h)
            sign, last = 1.0, 1.0
            if a < 0:      # S_t of -a is (-1)^(t + 1) times that of a
                sign, last = -1.0, 1.0 if n % 2 else -1.0
                turn = np.where(np.arange(n) % 2, -1.0, 1.0)[:, None]
                q, k = q * turn, k * turn
            (o, bar), (S, sbar) = bars.forward(q, k, v, abs(c.lam(h)), sign * np64(sin[i, h]), c.scale)
            assert worst(c.part(out, i, h, 64), o, bar) <= 1 and worst(np64(sout[i, h]), last * S, sbar) <= 1


def test_linear_attention_gradients_against_differences():
    """The kernel's own forward, differenced along one direction of v and of the initial state, in which the
    output is linear: the outputs' roundings, R / sqrt(3) of each, are all that is left."""
    c = Linear(lens=[120], heads=1, K=64, V=64, decay=[0.97])
    sin = c.states()
    dout = torch.randn(c.rows, 64, generator=gen(8), device=DEV).to(BF)
    dsin, zero = torch.empty_like(sin), torch.zeros_like(sin)
    dv = c.back(dout, sin, zero, dsin)[2]
    step = torch.randn(c.rows, 64, generator=gen(9), device=DEV).to(BF)
    ss = torch.randn(sin.shape, generator=gen(10), device=DEV)
    v0, f, size = c.x[:, 128:192].clone(), [], []
    for s in (1, -1):
        c.x[:, 128:192] = (v0.float() + s * step.float()).to(BF)
        o = c.call(sin + s * ss)
        torch.cuda.synchronize()
        f.append(float(np.sum(np64(o[:120, :64]) * np64(dout))))
        size.append(np.sum((np64(o[:120, :64]) * np64(dout)) ** 2))
        moved = np64(c.x[:, 128:192]) - np64(v0)
        if s == 1:
            up = moved
    down = moved
    got = f[0] - f[1]
    want = np.sum(np64(dv[:120, :64]) * (up - down)) + 2 * np.sum(np64(dsin) * np64(ss))
    noise = np.sqrt(sum(size)) * 2.0 ** -8 / np.sqrt(3)
    grads = np.sqrt(np.sum((np64(dv[:120, :64]) * (up - down)) ** 2)) * 2.0 ** -8 / np.sqrt(3)
    assert abs(got - want) <= 6 * (noise + grads), (got, want, noise, grads)


# ------------------------------------------------------------------------ norms between sub-layers
class Norm:
    def __init__(self, T, D, act="bf16", groups=1, norm_y=True, kind="none", h=True, scales=True, n=True, pad=8, eps=1e-6,
                 seed=1):
        say(f"norm T={T} D={D} {act} groups={groups} norm_y={norm_y} {kind} h={h} scales={scales} n={n}")
        self.T, self.D, self.groups, self.norm_y, self.kind, self.eps, self.n = T, D, groups, norm_y, kind, eps, n
        self.dt = BF if act == "bf16" else torch.float32
        self.cfg = W.make_residual_norm_config(dim=D, groups=groups, norm_y=norm_y, gate=kind, act=act, eps=eps)
        g = gen(seed)
        self.ld = D + pad

        def rows(f=1.0):
            return (f * torch.randn(T, self.ld, generator=g, device=DEV)).to(self.dt)

        def scale(m):
            return (m + 0.2 * torch.randn(D, generator=g, device=DEV)).to(self.dt) if scales else None
        self.y, self.h, self.gate = rows(0.5), rows(2.0) if h else None, rows(2.0) if kind != "none" else None
        self.wy, self.rs, self.wn = scale(1) if norm_y else None, scale(0.5), scale(1) if n else None
        self.dho, self.dn = rows(), rows() if n else None

    def kw(self):
        c = lambda x: None if x is None else np64(x[:, :self.D] if x.dim() == 2 else x)  # noqa: E731
        return dict(h=c(self.h), gate=c(self.gate), wy=c(self.wy), rs=c(self.rs), wn=c(self.wn), groups=self.groups,
                    norm_y=self.norm_y, kind=self.kind, eps=self.eps)

    def new(self, extra=2):
        return torch.full((self.T + extra, self.ld), 7.0, dtype=self.dt, device=DEV)

    def call(self, ho=None, no=None, want_h=True):
        ho = (self.new() if ho is None else ho) if want_h else None
        no = (self.new() if no is None else no) if self.n else None
        W.ttt_residual_norm(self.cfg, self.h, self.ld, self.y, self.ld, self.gate, self.ld, self.wy, self.rs, self.wn, ho,
                            self.ld, no, self.ld, self.T)
        return ho, no

    def check(self, ho, no, kw=None, y=None, behind=True):
        torch.cuda.synchronize()
        kw, y = kw or self.kw(), np64(self.y[:, :self.D]) if y is None else y
        f = om.residual_norm(y, **kw)
        hb, nb = bars.norm(f, y, kw["h"], kw["rs"], kw["wn"], H[self.dt])
        for name, o, ref, bar in (("h", ho, f["h_out"], hb), ("n", no, f["n_out"], nb)):
            if o is not None:
                w = worst(np64(o[:self.T, :self.D]), ref, bar)
                assert w <= 1, (name, w)
                if behind:
                    assert bool((o[self.T:] == 7).all()) and bool((o[:, self.D:] == 7).all())

    def sums(self):
        return [None if w is None else torch.full((self.D,), 5.0, device=DEV) for w in (self.wy, self.rs, self.wn)]

    def back(self, dh=None, dy=None, dg=None, sums=None, dho=True, work=None):
        n = W.ttt_residual_norm_backward_work(self.cfg, self.T)
        work = torch.empty(n, dtype=torch.uint8, device=DEV) if work is None else work
        dh = (self.new() if dh is None else dh) if self.h is not None else None
        dy = self.new() if dy is None else dy
        dg = (self.new() if dg is None else dg) if self.gate is not None else None
        sums = self.sums() if sums is None else sums
        W.ttt_residual_norm_backward(self.cfg, self.h, self.ld, self.y, self.ld, self.gate, self.ld, self.wy, self.rs,
                                     self.wn, self.dho if dho else None, self.ld, self.dn, self.ld, dh, self.ld, dy,
                                     self.ld, dg, self.ld, *sums, work, self.T)
        return dh, dy, dg, sums

    def check_back(self, dh, dy, dg, sums, dho=None, dn=None, behind=True):
        torch.cuda.synchronize()
        kw, y = self.kw(), np64(self.y[:, :self.D])
        zero = np.zeros_like(y)
        dho = np64(self.dho[:, :self.D]) if dho is None else dho
        dn = (np64(self.dn[:, :self.D]) if self.n else zero) if dn is None else dn
        f, ref = om.residual_norm(y, **kw), om.residual_norm_vjp(y, dho, dn, **kw)
        bar = bars.norm_backward(f, ref, y, kw["h"], kw["gate"], kw["wy"], kw["rs"], kw["wn"], dho, dn, self.groups,
                                 self.norm_y, H[self.dt])
        for name, o in (("dh", dh), ("dy", dy), ("dgate", dg), ("dwy", sums[0]), ("drs", sums[1]), ("dwn", sums[2])):
            if o is None:
                continue
            got = np64(o if o.dim() == 1 else o[:self.T, :self.D])
            w = worst(got, ref[name], bar[name])
            assert w <= 1, (name, w)
            if o.dim() == 2 and behind:
                assert bool((o[self.T:] == 7).all()) and bool((o[:, self.D:] == 7).all())


NORMS = [
    dict(T=1, D=8), dict(T=3, D=16, act="f32", kind="silu"), dict(T=37, D=64, groups=8, kind="sigmoid"),
    dict(T=5, D=72, h=False), dict(T=130, D=136, act="f32", kind="sigmoid", scales=False),
    dict(T=77, D=512, groups=1, kind="silu", n=False), dict(T=33, D=768, groups=6, kind="silu"),
    dict(T=33, D=768, groups=12, act="f32"), dict(T=21, D=1024, groups=2, kind="silu"), dict(T=9, D=1032),
    dict(T=9, D=1536, act="f32", groups=3, kind="silu"), dict(T=9, D=2048, groups=16, act="f32", kind="sigmoid"),
    dict(T=7, D=2056), dict(T=5, D=4096, groups=32, kind="silu", act="f32"), dict(T=4, D=5000, kind="sigmoid"),
    dict(T=5, D=8192, act="f32", kind="silu"), dict(T=3, D=8192, groups=16), dict(T=20, D=256, norm_y=False),
    dict(T=20, D=256, norm_y=False, h=False, scales=False, n=False), dict(T=20, D=40, groups=5, eps=0.1),
    dict(T=5003, D=64, kind="silu"), dict(T=4999, D=128, groups=2, act="f32", kind="sigmoid"),
]


@pytest.mark.parametrize("kw", NORMS)
def test_residual_norm_matches_oracle(kw):
    c = Norm(**kw)
    c.check(*c.call())
    if c.n:
        c.check(*c.call(want_h=False))


@pytest.mark.parametrize("kw", NORMS)
def test_residual_norm_backward_matches_oracle(kw):
    c = Norm(**kw)
    c.check_back(*c.back())


@pytest.mark.parametrize("h_as,n_as", [("h", "y"), ("y", "h"), ("gate", "y"), ("h", "gate")])
def test_residual_norm_in_place(h_as, n_as):
    c = Norm(T=70, D=256, groups=2, kind="silu")
    kw, y = c.kw(), np64(c.y[:, :256])
    ho, no = c.call(getattr(c, h_as), getattr(c, n_as))
    c.check(ho, no, kw, y, behind=False)


def test_residual_norm_backward_in_place_and_of_some_gradients():
    c = Norm(T=70, D=256, groups=2, kind="silu")
    dho, dn = np64(c.dho[:, :256]), np64(c.dn[:, :256])
    dh, dy, dg, sums = c.back(dh=c.dho, dy=c.dn, sums=[None, torch.empty(256, device=DEV), None])
    c.check_back(dh, dy, dg, sums, dho, dn, behind=False)
    c = Norm(T=70, D=256, groups=2, kind="silu")
    W.ttt_residual_norm_backward(c.cfg, c.h, c.ld, c.y, c.ld, c.gate, c.ld, c.wy, c.rs, c.wn, c.dho, c.ld, c.dn, c.ld, None, 0,
                                 None, 0, (g := c.new()), c.ld, None, None, None, None, c.T)
    c.check_back(None, None, g, [None] * 3)
    c = Norm(T=30, D=64)
    c.check_back(*c.back(dho=False), dho=np.zeros((30, 64)))


def test_residual_norm_keeps_what_is_not_finite_to_its_row():
    c = Norm(T=40, D=64, kind="silu")
    clean, cback = c.call(), c.back()
    c.y[3, 5], c.h[17, 9], c.gate[30, 60] = float("nan"), float("inf"), float("nan")
    got, back = c.call(), c.back()
    torch.cuda.synchronize()
    for a, b in zip((*got, *back[:3]), (*clean, *cback[:3])):
        for row in (3, 17, 30):
            assert not bool(a[row, :64].isfinite().all())
            a[row] = b[row]
        assert torch.equal(a, b)


def test_residual_norm_of_zero_and_large_rows():
    c = Norm(T=4, D=128, act="f32")
    c.y[1], c.h[1] = 0, 0
    c.y[2] *= 1e15
    c.h[2] *= 1e15
    c.check(*c.call())


def test_residual_norm_of_no_rows():
    c = Norm(T=3, D=64, kind="sigmoid")
    ho, no = c.new(), c.new()
    c.T = 0
    c.call(ho, no)
    _, _, _, sums = c.back(c.new(), c.new(), c.new())
    torch.cuda.synchronize()
    assert bool((ho == 7).all()) and bool((no == 7).all()) and all(bool((s == 0).all()) for s in sums)


def test_residual_norm_far_rows():
    """Rows more than 2^32 bytes behind the first."""
    ld, T = 1 << 24, 160
    x = torch.zeros(T, ld, dtype=BF, device=DEV)      # 5.4 GB
    c = Norm(T=T, D=64, h=False)
    x[:, :64] = c.y[:, :64]
    near = c.call()
    far = c.new(), c.new()
    W.ttt_residual_norm(c.cfg, None, 0, x, ld, None, 0, c.wy, c.rs, c.wn, far[0], c.ld, far[1], c.ld, T)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(near, far))


def test_residual_norm_of_more_rows_than_a_launch():
    """2^20 workgroups of one row each, and five more, in place."""
    D, T = 1032, (1 << 20) + 5
    c = Norm(T=61, D=D, kind="silu", pad=0)
    near = c.call()
    x = [t.repeat(T // 61 + 1, 1)[:T].contiguous() for t in (c.y, c.h, c.gate)]   # 2.2 GB each
    y, h, gate = x
    W.ttt_residual_norm(c.cfg, h, D, y, D, gate, D, c.wy, c.rs, c.wn, h, D, y, D, T)
    torch.cuda.synchronize()
    for got, ref in zip((h, y), near):
        for a in (0, (1 << 20) // 61 * 61 - 61):      # the first rows, and those around the launch's end
            assert torch.equal(got[a:a + 61], ref[:61])
        for r in range((1 << 20) - 3, T):
            assert torch.equal(got[r], ref[r % 61])


def test_residual_norm_backward_captured():
    c = Norm(T=3001, D=256, groups=4, kind="silu")
    work = torch.empty(W.ttt_residual_norm_backward_work(c.cfg, c.T), dtype=torch.uint8, device=DEV)
    outs = [c.new(), c.new(), c.new(), c.new(), c.new(), c.sums()]

    def both(o, w):
        c.call(o[0], o[1])
        c.back(o[2], o[3], o[4], o[5], work=w)
    both(outs, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(outs, work)
    other, w2 = torch.cuda.Stream(), torch.empty_like(work)
    eager = [c.new(), c.new(), c.new(), c.new(), c.new(), c.sums()]
    for i in range(4):
        for j, t in enumerate((c.y, c.h, c.gate, c.dho, c.dn)):
            t.copy_(torch.randn(t.shape, generator=gen(10 * i + j), device=DEV).to(BF))
        for t in (*outs[:5], *outs[5], *eager[:5], *eager[5]):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            both(eager, w2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*outs[:5], *outs[5]), (*eager[:5], *eager[5])))
        torch.randn(1000, device=DEV).sum().item()


def test_residual_norm_gradients_against_differences():
    """The kernel's own forward in fp32, differenced: third derivatives of the norms are bounded by 15 / rms^3
    a unit, rms near 1 here, and the step 2^-6: below 1e-3 of the gradients' scale; checked at 1e-2."""
    c = Norm(T=6, D=64, act="f32", groups=2, kind="silu")
    dh, dy, dg, _ = c.back()
    f = []
    ins = [c.y, c.h, c.gate]
    base = [t.clone() for t in ins]
    d = [torch.randn(t.shape, generator=gen(30 + i), device=DEV) for i, t in enumerate(ins)]
    for s in (1, -1):
        for t, b, x in zip(ins, base, d):
            t.copy_(b + s * 2.0 ** -6 * x)
        ho, no = c.call()
        torch.cuda.synchronize()
        f.append(sum(np.sum(np64(o[:6, :64]) * np64(g[:, :64])) for o, g in ((ho, c.dho), (no, c.dn))))
    got = (f[0] - f[1]) * 2.0 ** 5
    grads = [np64(t[:6, :64]) for t in (dy, dh, dg)]
    want = sum(np.sum(g * np64(x[:, :64])) for g, x in zip(grads, d))
    assert abs(got - want) <= 1e-2 * np.sqrt(sum(np.sum(g * g) for g in grads))


# ------------------------------------------------------------------------ together
class Layer:
    """A pre-norm sub-layer of linear attention at width heads * D, as a program makes one of the calls: projection
    to queries, keys, values and gate, the layer, the norm of each head with its gate, projection back, residual
    and the next sub-layer's norm."""

    def __init__(self, heads, D, seed=1):
        self.heads, self.D, self.N = heads, D, heads * D
        g = gen(seed)
        w = lambda o, i: (torch.randn(o, i, generator=g, device=DEV) / i ** 0.5).to(BF)  # noqa: E731
        self.w_in, self.w_out = w(4 * self.N, self.N), w(self.N, self.N)
        self.scales = [(1 + 0.1 * torch.randn(self.N, generator=g, device=DEV)).to(BF) for _ in range(3)]
        self.decay = 1 - 2.0 ** -(3 + torch.arange(heads, device=DEV, dtype=torch.float32))
        self.la = W.make_linear_attention_config(heads=heads, dim_k=D)
        self.inner = W.make_residual_norm_config(dim=self.N, groups=heads, norm_y=True, gate="silu")
        self.outer = W.make_residual_norm_config(dim=self.N)

    def start(self, x):
        n = torch.empty_like(x)
        W.ttt_residual_norm(self.outer, None, 0, x, self.N, None, 0, None, None, self.scales[0], None, 0, n, self.N, len(x))
        return n

    def finish(self, x, p, o):
        T, N = len(x), self.N
        z, y, h, n = (torch.empty_like(x) for _ in range(4))
        W.ttt_residual_norm(self.inner, None, 0, o, N, p[:, 3 * N:], 4 * N, self.scales[1], None, None, z, N, None, 0, T)
        W.ttt_linear(z, self.w_out, None, y, T, N, N)
        W.ttt_residual_norm(self.outer, x, N, y, N, None, 0, None, None, self.scales[2], h, N, n, N, T)
        return h, n

    def prompt(self, x, starts, state, slot, longest, work):
        T, N, B = len(x), self.N, len(starts) - 1
        p, o = torch.empty(T, 4 * N, dtype=BF, device=DEV), torch.empty(T, N, dtype=BF, device=DEV)
        W.ttt_linear(self.start(x), self.w_in, None, p, T, N, 4 * N)
        W.ttt_linear_attention(self.la, p, 4 * N, p[:, N:], 4 * N, p[:, 2 * N:], 4 * N, self.decay, starts, state, state, slot,
                               o, N, T, B, longest, work)
        return self.finish(x, p, o)

    def token(self, x, state, slot):
        T, N = len(x), self.N
        p, o = torch.empty(T, 4 * N, dtype=BF, device=DEV), torch.empty(T, N, dtype=BF, device=DEV)
        W.ttt_linear(self.start(x), self.w_in, None, p, T, N, 4 * N)
        W.ttt_linear_attention_step(self.la, p, 4 * N, p[:, N:], 4 * N, p[:, 2 * N:], 4 * N, self.decay, state, state, slot, o,
                                    N, T)
        return self.finish(x, p, o)


def test_a_layer_serves_a_prompt_and_then_tokens():
    """Two ragged prompts and then five tokens of each, one captured step replayed, against the same tokens as
    prompts: every value is the same sums in another order and rounded to bf16 five times on its way (the
    projection's inputs, q, k, v, the layer's output, the gated norm, the projection back, h), a flip of a
    rounding there moves it by some 2^-8; the states by 2^-9 of their size on average."""
    L = Layer(heads=4, D=64)
    lens, more = [70, 33], 5
    g = gen(3)
    xs = [torch.randn(n + more, L.N, generator=g, device=DEV).to(BF) for n in lens]
    slot = torch.tensor([2, 0], dtype=torch.int32, device=DEV)

    def prompt(parts, pool):
        n = [len(p) for p in parts]
        starts = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV)
        work = torch.empty(W.ttt_linear_attention_work(L.la, 2, max(n)), dtype=torch.uint8, device=DEV)
        return L.prompt(torch.cat(parts), starts, pool, slot, max(n), work)
    whole = torch.zeros(3, 4, 64, 64, device=DEV)
    h1, n1 = prompt(xs, whole)
    pool = torch.zeros_like(whole)
    prompt([x[:n] for x, n in zip(xs, lens)], pool)
    token = torch.empty(2, L.N, dtype=BF, device=DEV)
    before = pool.clone()
    L.token(token.zero_(), pool, slot)       # warm
    pool.copy_(before)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h2, n2 = L.token(token, pool, slot)
    pool.copy_(before)
    ends = [0, lens[0] + more]
    for i in range(more):
        token.copy_(torch.stack([x[n + i] for x, n in zip(xs, lens)]))
        graph.replay()
        torch.cuda.synchronize()
        for s in range(2):
            row = ends[s] + lens[s] + i
            for a, b in ((h2[s], h1[row]), (n2[s], n1[row])):
                assert float((a.float() - b.float()).norm() / b.float().norm()) < 2.0 ** -6
    # the states: products of keys and values that are themselves the same bf16 numbers or a step apart
    assert float((pool - whole).norm() / whole.norm()) < 2.0 ** -7
    assert bool((pool[1] == 0).all())


def test_a_layers_training_step():
    """Gradients through norm, layer, gated norm and residual, each from the values that the calls themselves
    made: each call's own bars hold along the way."""
    heads, D, T = 2, 64, 300
    N = heads * D
    c = Linear(lens=[T], heads=heads, K=D, V=D, dense=True, pad=0, decay=[0.95, 0.999])
    o = c.call(out=torch.empty(T, N, dtype=BF, device=DEV))
    m = Norm(T=T, D=N, groups=heads, kind="silu", pad=0)
    m.y = o
    m.check_back(*(r := m.back()))
    dq, dk, dv = c.back(r[1][:T])
    torch.cuda.synchronize()
    zero = np.zeros((D, D))
    for h in range(heads):
        ref = bars.backward(*c.qkv(0, h), c.lam(h), zero, c.scale, np64(r[1][:T, h * D:(h + 1) * D]), zero)
        for x, (y, bar) in zip((dq, dk, dv), ref):
            assert worst(c.part(x, 0, h, D), y, bar) <= 1


def test_calls_on_another_device_are_refused():
    c = Linear(lens=[4], K=64, V=64)
    with pytest.raises(W.TTTError) as e:
        W.ttt_linear_attention_step(c.cfg, c.q, c.ld, c.k, c.ld, c.v, c.ld, c.decay.cpu(), None, None, None, c.out(64), 136, 4)
    assert e.value.status == 4
    m = Norm(T=3, D=64)
    m.wy = m.wy.cpu()
    with pytest.raises(W.TTTError):
        m.call()
