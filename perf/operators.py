"""The attention operators around the window attention, as cases to measure: per-head norms with
the position rotation (and their backward), the same pass into a paged key-value cache, attention
of one new token over that cache, and the window attention's training step.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` makes what a program holds before the
call, `run(state)` is one call: in plain torch operations, or with `own` set through the library.
`exact(case, seed)` computes the outputs in 64 bits from the definitions, `work(case)` the bytes
and operations that a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ cases
def listed():
    rot = {"op": "rotate", "axes": 1, "pairing": "halves", "norm": "rms"}
    grad = {"op": "rotate_grad", "axes": 1, "pairing": "halves", "norm": "rms"}
    app = {"op": "append", "axes": 1, "pairing": "halves", "norm": "rms"}
    dec = {"op": "decode", "window": 0}
    win = {"op": "window_train"}
    return [
        # one decoding step of four sequences of the LM block (8 heads of 128)
        dict(rot, name="rotate_step", tokens=4, q_heads=8, k_heads=8, dim=128, rot_dim=128,
             act="bf16"),
        # eight images of 8040 tokens of the image set's block (6 heads), positions view, row
        # and column, three quarters of each head rotated, in 32 bits
        dict(rot, name="rotate_images", tokens=8 * 8040, q_heads=6, k_heads=6, dim=128,
             rot_dim=96, axes=3, pairing="pairs", act="f32"),
        # the LM block's training sequence of 32768 tokens
        dict(grad, name="rotate_grad_text", tokens=32768, q_heads=8, k_heads=8, dim=128,
             rot_dim=128, act="bf16"),
        # three images and a ragged rest, 32 bits, shared keys, heads of 64
        dict(grad, name="rotate_grad_images", tokens=3 * 8040 + 77, q_heads=12, k_heads=4, dim=64,
             rot_dim=64, axes=3, pairing="halves", act="f32"),
        # a decoding step of 61 sequences, shared keys, into an 8-bit cache
        dict(app, name="append_step", tokens=61, q_heads=32, k_heads=8, dim=128, rot_dim=128,
             page=16, pages=256, cache="e4m3"),
        # a prompt of 8192 tokens of the LM block into a 16-bit cache
        dict(app, name="append_prompt", tokens=8192, q_heads=8, k_heads=8, dim=128, rot_dim=128,
             page=64, pages=160, cache="bf16"),
        # two short conversations: latency
        dict(dec, name="decode_short", seqs=2, max_len=130, q_heads=8, k_heads=8, dim=128, page=16,
             cache="bf16"),
        # a serving batch of ragged lengths, four queries sharing a key head
        dict(dec, name="decode_batch", seqs=64, max_len=8192, q_heads=32, k_heads=8, dim=128,
             page=16, cache="bf16"),
        # one long context of the long workload (131072 tokens) of the LM block's heads
        dict(dec, name="decode_long", seqs=1, max_len=131072, q_heads=8, k_heads=8, dim=128, page=64,
             cache="bf16"),
        # the LM block's sliding window of 2048 over longer sequences, 8-bit cache, a page size
        # that no tile size divides
        dict(dec, name="decode_window", seqs=96, max_len=5000, q_heads=16, k_heads=4, dim=128, page=24,
             window=2048, cache="e4m3"),
        # a short ragged training batch, one window per image
        dict(win, name="window_train_small", batch=3, tokens=777, heads=2, window=250, mode="block"),
        # the LM block's training sequence: 32768 tokens, 8 heads, sliding window of 2048
        dict(win, name="window_train_text", batch=1, tokens=32768, heads=8, window=2048,
             mode="sliding"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_grad", "append", "decode", "decode", "window_train"])
    if op == "window_train":
        heads, batch = rng.choice([1, 2, 3, 6, 8]), rng.choice([1, 1, 2, 4])
        tokens = _log(rng, 1, 16384 // batch)
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads,
                "window": _log(rng, 1, 2048), "mode": rng.choice(["sliding", "block"])}
    k_heads = rng.choice([1, 2, 4, 6, 8])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "decode":
        seqs = _log(rng, 1, 128)
        max_len = _log(rng, 1, min(131072, 2097152 // (seqs * k_heads)))
        return {"op": op, "seqs": seqs, "max_len": max_len, "q_heads": k_heads * group,
                "k_heads": k_heads, "dim": rng.choice([64, 128, 256]), "page": rng.choice([1, 7, 16, 24, 64, 128]),
                "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "cache": cache}
    dim = rng.choice([64, 128, 128, 256])
    case = {"op": op, "q_heads": k_heads * group, "k_heads": k_heads, "dim": dim,
            "rot_dim": rng.choice([0, dim // 2, dim, dim]), "axes": rng.choice([1, 2, 3]),
            "pairing": rng.choice(["halves", "pairs"]), "norm": rng.choice(["rms", "rms", "none"])}
    tokens = _log(rng, 1, max(64, 16777216 // ((group + 1) * k_heads * dim)))
    if op == "append":
        page = rng.choice([1, 7, 16, 24, 64])
        case.update(tokens=tokens, page=page, pages=tokens // page + 3, cache=cache)
    else:
        case.update(tokens=tokens, act=rng.choice(["bf16", "bf16", "f32"]))
    return case


def _lens(c):
    """The sequences' cached lengths: spread over 0 .. max_len, the first at max_len, and with
    eight or more sequences one that is still empty."""
    out = [c["max_len"]]
    for i in range(1, c["seqs"]):
        out.append(0 if i == 5 and c["seqs"] >= 8 else
                   1 + int((c["max_len"] - 1) * math.modf(0.6180339887 * i)[0]))
    return out


def work(c):
    op = c["op"]
    if op == "window_train":
        T, w = c["tokens"], min(c["window"], c["tokens"])
        if c["mode"] == "sliding":
            pairs = w * (w + 1) // 2 + (T - w) * w
        else:
            pairs = (T // w) * w * w + (T % w) ** 2
        n = c["batch"] * T * c["heads"]
        # q, k, v and dO read, out, dq, dk, dv written in 16 bits, lse in 32
        return {"bytes": n * (8 * 128 * 2 + 4), "flops": 14 * 128 * pairs * c["batch"] * c["heads"]}
    if op == "decode":
        size = 2 if c["cache"] == "bf16" else 1
        keys = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        rows = c["seqs"] * c["q_heads"]
        return {"bytes": keys * c["k_heads"] * c["dim"] * 2 * size + rows * (c["dim"] * 4 + 4),
                "flops": 4 * keys * c["q_heads"] * c["dim"]}
    n = c["tokens"] * c["dim"]
    nq, nk, heads = n * c["q_heads"], n * c["k_heads"], c["q_heads"] + c["k_heads"]
    pos = 4 * c["axes"] * c["tokens"]
    if op == "append":
        size = 2 if c["cache"] == "bf16" else 1
        return {"bytes": 4 * nq + (2 + size) * 2 * nk + pos + 8 * c["tokens"],
                "flops": 8 * n * heads}
    size = 2 if c["act"] == "bf16" else 4
    if op == "rotate":
        return {"bytes": 2 * size * n * heads + pos, "flops": 8 * n * heads}
    return {"bytes": 3 * size * n * heads + pos, "flops": 16 * n * heads}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    c = dict(case)
    if c["op"] == "window_train":
        B, T, D = c["batch"], c["tokens"], c["heads"] * 128
        bf = torch.bfloat16
        new = lambda *s: torch.empty(*s, dtype=bf, device=DEV)  # noqa: E731
        return {"case": c, "qkv": randn(B, T, 3 * D).to(bf), "dout": randn(B, T, D).to(bf),
                "out": new(B, T, D), "dqkv": new(B, T, 3 * D),
                "lse": torch.empty(B, c["heads"], T, device=DEV),
                "work": torch.empty(B, c["heads"], T, device=DEV)}
    Hq, Hk, D = c["q_heads"], c["k_heads"], c["dim"]
    if c["op"] == "decode":
        S, page = c["seqs"], c["page"]
        lens = _lens(c)
        used = [-(-n // page) for n in lens]
        width, pages = max(used), sum(used) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)   # -1: no page
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        k, v = randn(pages, Hk, page, D), randn(pages, Hk, page, D)
        k_scale = v_scale = None
        if c["cache"] == "bf16":
            k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        else:
            k_scale = 0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV)
            v_scale = 0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV)
            k = (k / k_scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            v = (v / v_scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        q = (1.5 * randn(S, Hq * D)).to(torch.bfloat16)
        return {"case": c, "q": q, "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale,
                "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
                "out": torch.empty_like(q), "lse": torch.empty(S, Hq, device=DEV)}
    T, rot, axes = c["tokens"], c["rot_dim"], c["axes"]
    dt = torch.float32 if c.get("act") == "f32" else torch.bfloat16
    # positions: text counts on from somewhere; images have view, row and column of a grid of
    # 120 x 67 patches
    t = torch.arange(T, device=DEV)
    if axes == 1:
        start = int(torch.randint(0, 30000, (1,), generator=g, device=DEV))
        pos = (t + start)[None]
    else:
        pos = torch.stack([t // 8040, t % 8040 // 120, t % 120])[3 - axes:]
    # frequencies base^(-2 j / rot); with several axes pair j turns with axis j mod axes
    j = torch.arange(rot // 2, device=DEV)
    freq = torch.zeros(axes, rot // 2, device=DEV)
    freq[j % axes, j] = torch.pow(torch.tensor(10000.0, device=DEV), -2.0 * j / max(rot, 1)).float()
    norm = c["norm"] == "rms"
    state = {"case": c, "pos": pos.to(torch.int32).contiguous(), "freq": freq,
             "q_weight": (1 + 0.1 * randn(D)).to(dt) if norm else None,
             "k_weight": (1 + 0.1 * randn(D)).to(dt) if norm else None,
             # queries, keys and values as one projection's output rows
             "qkv": (0.7 * randn(T, (Hq + 2 * Hk) * D)).to(dt)}
    if c["op"] == "rotate":
        state.update(q_out=torch.empty(T, Hq * D, dtype=dt, device=DEV),
                     k_out=torch.empty(T, Hk * D, dtype=dt, device=DEV))
    elif c["op"] == "rotate_grad":
        state.update(dq_out=randn(T, Hq * D).to(dt), dk_out=randn(T, Hk * D).to(dt),
                     dq=torch.empty(T, Hq * D, dtype=dt, device=DEV),
                     dk=torch.empty(T, Hk * D, dtype=dt, device=DEV),
                     dq_weight=torch.empty(D, device=DEV) if norm else None,
                     dk_weight=torch.empty(D, device=DEV) if norm else None)
    else:
        page, pages = c["page"], c["pages"]
        slot = torch.randperm(page * pages, generator=g, device=DEV)[:T].to(torch.int64)
        if T >= 8:
            slot[T - 2] = -1     # a padding token of the batch
        ct = torch.bfloat16 if c["cache"] == "bf16" else torch.float8_e4m3fn
        scaled = c["cache"] == "e4m3"
        state.update(slot=slot, q_out=torch.empty(T, Hq * D, dtype=dt, device=DEV),
                     k=torch.zeros(pages, Hk, page, D, device=DEV).to(ct),
                     v=torch.zeros(pages, Hk, page, D, device=DEV).to(ct),
                     k_scale=0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV) if scaled else None,
                     v_scale=0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV) if scaled else None)
    return state


# ------------------------------------------------------------------------------------ plain forms
def _thirds(s):
    """Queries, keys and values [tokens, heads, dim] of the projection's rows."""
    c = s["case"]
    T, Hq, Hk, D = c["tokens"], c["q_heads"], c["k_heads"], c["dim"]
    x = s["qkv"]
    return (x[:, :Hq * D].view(T, Hq, D), x[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D),
            x[:, (Hq + Hk) * D:].view(T, Hk, D))


def _turns(s):
    """cos and sin [tokens, 1, rot / 2] of every pair's angle."""
    angle = (s["pos"].double()[:, :, None] * s["freq"].double()[:, None, :]).sum(0)[:, None, :]
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, c):
    """The pairs of x's first rot_dim elements turned by the angles."""
    rot = c["rot_dim"]
    y = x.clone()
    a, b = ((slice(0, rot // 2), slice(rot // 2, rot)) if c["pairing"] == "halves"
            else (slice(0, rot, 2), slice(1, rot, 2)))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _normed(x, w, c):
    x = x.float()
    if c["norm"] == "none":
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_rotate(s):
    c, (q, k, _), (cos, sin) = s["case"], _thirds(s), _turns(s)
    q = _turn(_normed(q, s["q_weight"], c), cos, sin, c)
    k = _turn(_normed(k, s["k_weight"], c), cos, sin, c)
    dt = s["qkv"].dtype
    return q.flatten(1).to(dt), k.flatten(1).to(dt)


def _plain_grad_of(x, w, dy, cos, sin, c):
    g = _turn(dy.float().view(x.shape), cos, -sin, c)
    if c["norm"] == "none":
        return g, None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    xh = x * r
    dw = (g * xh).double().sum((0, 1)).float()
    u = g * w.float()
    return r * (u - xh * (u * xh).mean(-1, keepdim=True)), dw


def _plain_rotate_grad(s):
    c, (q, k, _), (cos, sin) = s["case"], _thirds(s), _turns(s)
    dt = s["qkv"].dtype
    dq, dwq = _plain_grad_of(q, s["q_weight"], s["dq_out"], cos, sin, c)
    dk, dwk = _plain_grad_of(k, s["k_weight"], s["dk_out"], cos, sin, c)
    return dq.flatten(1).to(dt), dk.flatten(1).to(dt), dwq, dwk


def _plain_append(s):
    c, (_, _, v) = s["case"], _thirds(s)
    q, k = _plain_rotate(dict(s, qkv=s["qkv"].float()))
    k, v = k.view(v.shape), v.float()
    if c["cache"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
    keep = s["slot"] >= 0
    page, at = s["slot"][keep] // c["page"], s["slot"][keep] % c["page"]
    for name, x in (("k", k), ("v", v)):
        bits = torch.int16 if c["cache"] == "bf16" else torch.uint8
        s[name].view(bits)[page, :, at] = x[keep].to(s[name].dtype).view(bits)
    return q.to(torch.bfloat16), s["k"], s["v"]


def _plain_decode(s):
    c = s["case"]
    S, Hq, Hk, D = c["seqs"], c["q_heads"], c["k_heads"], c["dim"]
    table = s["table"].long().clamp_min(0)
    L = table.shape[1] * c["page"]

    def cached(x, scale):   # [S, Hk, L, D] in 32 bits
        bits = torch.int16 if c["cache"] == "bf16" else torch.uint8
        y = x.view(bits)[table].view(x.dtype).permute(0, 2, 1, 3, 4).reshape(S, Hk, L, D).float()
        return y if scale is None else y * scale[:, None, None]

    k, v = cached(s["k"], s["k_scale"]), cached(s["v"], s["v_scale"])
    j = torch.arange(L, device=DEV)[None]
    n = s["lens"].long()[:, None]
    seen = (j < n) & ((j >= n - c["window"]) if c["window"] else (j >= 0))
    seen = seen[:, None, None, :]
    q = s["q"].float().view(S, Hk, Hq // Hk, D)
    sc = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(D))
    sc = torch.where(seen, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))   # empty sequences: all zero
    z = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(z == 0, 1.0, z)
    return out.reshape(S, Hq * D).to(torch.bfloat16), (m + torch.log(z)).reshape(S, Hq)


def _plain_window_train(s):
    c = s["case"]
    B, T, H, W = c["batch"], c["tokens"], c["heads"], min(c["window"], c["tokens"])
    nb = -(-T // W)
    sliding = c["mode"] == "sliding"

    def blocks(x):   # [B, T, H * 128] -> [B * H, blocks, W, 128]
        x = x.float().view(B, T, H, 128).transpose(1, 2).reshape(B * H, T, 128)
        return torch.nn.functional.pad(x, (0, 0, 0, nb * W - T)).view(B * H, nb, W, 128)

    def seen_of(x):  # the keys of a block's queries: with a sliding window the block before, too
        if not sliding:
            return x
        return torch.cat([torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1), x], 2)

    def back(dx):    # the gradients of seen_of's blocks, added up
        if not sliding:
            return dx
        before, here = dx[:, :, :W], dx[:, :, W:]
        return here + torch.cat([before[:, 1:], torch.zeros_like(before[:, :1])], 1)

    def rows(x):     # [B * H, blocks, W, 128] -> [B, T, H * 128]
        x = x.reshape(B, H, nb * W, 128)[:, :, :T].transpose(1, 2)
        return x.reshape(B, T, H * 128).to(torch.bfloat16)

    q, k, v = (blocks(x) for x in s["qkv"].chunk(3, -1))
    do = blocks(s["dout"])
    kk, vv = seen_of(k), seen_of(v)
    t = torch.arange(nb * W, device=DEV).view(nb, W, 1)
    j = torch.arange(kk.shape[2], device=DEV) + (torch.arange(nb, device=DEV)[:, None] - int(sliding)) * W
    j = j[:, None, :]
    seen = (j >= 0) & (j < T)
    if sliding:
        seen = seen & (j <= t) & (j > t - W)
    seen = seen | (t >= T)    # rows of the padding: any mask without an empty row
    scale = 1 / math.sqrt(128)
    sc = torch.where(seen, (q @ kk.transpose(-1, -2)) * scale, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    p = p / z
    out = p @ vv
    lse = (m + torch.log(z)).reshape(B, H, nb * W)[:, :, :T]
    dp = do @ vv.transpose(-1, -2)
    ds = p * (dp - (do * out).sum(-1, keepdim=True)) * scale
    dq = ds @ kk
    dk = back(ds.transpose(-1, -2).contiguous() @ q)
    dv = back(p.transpose(-1, -2).contiguous() @ do)
    return rows(out), lse, torch.cat([rows(dq), rows(dk), rows(dv)], -1)


# ------------------------------------------------------------------------------------ the library
def _own_rotate(s):
    import weight_sequence_layers_amd as W
    c, x = s["case"], s["qkv"]
    Hq, Hk, D = c["q_heads"], c["k_heads"], c["dim"]
    cfg = W.make_rope_config(q_heads=Hq, k_heads=Hk, head_dim=D, rot_dim=c["rot_dim"],
                             axes=c["axes"], pairing=c["pairing"], norm=c["norm"], act=c.get("act", "bf16"))
    ld = x.shape[1]
    q, k, v = x, x[:, Hq * D:], x[:, (Hq + Hk) * D:]
    if c["op"] == "rotate":
        W.ttt_qk_norm_rope(cfg, q, ld, k, ld, s["q_weight"], s["k_weight"], s["freq"], s["pos"],
                           s["q_out"], Hq * D, s["k_out"], Hk * D, c["tokens"])
        return s["q_out"], s["k_out"]
    if c["op"] == "rotate_grad":
        if "work" not in s:
            n = W.ttt_qk_norm_rope_backward_work(cfg, c["tokens"])
            s["work"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        W.ttt_qk_norm_rope_backward(cfg, q, ld, k, ld, s["q_weight"], s["k_weight"], s["freq"],
                                    s["pos"], s["dq_out"], Hq * D, s["dk_out"], Hk * D, s["dq"],
                                    Hq * D, s["dk"], Hk * D, s["dq_weight"], s["dk_weight"],
                                    s["work"], c["tokens"])
        return s["dq"], s["dk"], s["dq_weight"], s["dk_weight"]
    cache = W.make_kv_cache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    W.ttt_qk_norm_rope_append(cfg, q, ld, k, ld, v, ld, s["q_weight"], s["k_weight"], s["freq"],
                              s["pos"], cache, s["slot"], s["q_out"], Hq * D, c["tokens"])
    return s["q_out"], s["k"], s["v"]


def _own_decode(s):
    import weight_sequence_layers_amd as W
    c = s["case"]
    S, Hq, D, width = c["seqs"], c["q_heads"], c["dim"], s["table"].shape[1]
    cache = W.make_kv_cache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if "work" not in s:
        n = W.ttt_paged_attention_work(cache, S, Hq, width, c["window"])
        s["work"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    W.ttt_paged_attention(s["q"], Hq * D, cache, s["table"], s["lens"], s["out"], Hq * D, s["lse"],
                          S, Hq, width, c["window"], 0.0, s["work"])
    return s["out"], s["lse"]


def _own_window_train(s):
    import weight_sequence_layers_amd as W
    c, x, dx = s["case"], s["qkv"], s["dqkv"]
    B, T, H = c["batch"], c["tokens"], c["heads"]
    D = H * 128
    k, v = x[..., D:], x[..., 2 * D:]
    W.ttt_window_attention_lse(x, k, v, 3 * D, s["out"], D, s["lse"], B, H, T, c["window"], c["mode"])
    W.ttt_window_attention_backward(x, k, v, 3 * D, s["out"], D, s["lse"], s["dout"], D,
                                    dx, dx[..., D:], dx[..., 2 * D:], 3 * D, s["work"],
                                    B, H, T, c["window"], c["mode"])
    return s["out"], s["lse"], dx


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotate": _own_rotate, "rotate_grad": _own_rotate, "append": _own_rotate,
                "decode": _own_decode, "window_train": _own_window_train}[op](state)
    return {"rotate": _plain_rotate, "rotate_grad": _plain_rotate_grad, "append": _plain_append,
            "decode": _plain_decode, "window_train": _plain_window_train}[op](state)


# ------------------------------------------------------------------------------------ 64 bits
def _exact_pairs(c):
    """Index pairs [rot / 2] of the elements that turn together."""
    j = torch.arange(c["rot_dim"] // 2, device=DEV)
    return (j, j + c["rot_dim"] // 2) if c["pairing"] == "halves" else (2 * j, 2 * j + 1)


def _exact_rotation(s, back=False):
    """The turn as complex factors [tokens, 1, rot / 2]."""
    angle = torch.einsum("at,aj->tj", s["pos"].double(), s["freq"].double())[:, None]
    return torch.polar(torch.ones_like(angle), -angle if back else angle)


def _exact_turned(x, turn, c):
    i0, i1 = _exact_pairs(c)
    z = torch.complex(x[..., i0], x[..., i1]) * turn
    y = x.clone()
    y[..., i0], y[..., i1] = z.real, z.imag
    return y


def _exact_heads(s):
    c = s["case"]
    Hq, Hk, D = c["q_heads"], c["k_heads"], c["dim"]
    x = s["qkv"].double().view(c["tokens"], Hq + 2 * Hk, D)
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


def _exact_rms(x):
    return torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)


def _exact_e4m3(x, scale):
    """x / scale rounded to the nearest e4m3 value, ties to even: three mantissa bits, the
    smallest step 2^-9, values past 448 held there."""
    x = (x / scale.double()[:, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "window_train":
        return _exact_window(s)
    if c["op"] == "decode":
        return _exact_decode(s)
    q, k, v = _exact_heads(s)
    wq, wk = ((s["q_weight"].double(), s["k_weight"].double()) if c["norm"] == "rms" else (None, None))
    if c["op"] == "rotate_grad":
        turn, res, dws = _exact_rotation(s, True), [], []
        for x, w, dy in ((q, wq, s["dq_out"]), (k, wk, s["dk_out"])):
            g = _exact_turned(dy.double().view(x.shape), turn, c)
            if w is None:
                res.append(g.flatten(1))
                dws.append(None)
                continue
            m = _exact_rms(x)
            dws.append((g * x / m).sum((0, 1)))
            g = g * w
            res.append((g / m - x * (g * x).sum(-1, keepdim=True) / (x.shape[-1] * m ** 3)).flatten(1))
        return res[0], res[1], dws[0], dws[1]
    turn = _exact_rotation(s)
    q, k = (_exact_turned(x if w is None else x / _exact_rms(x) * w, turn, c)
            for x, w in ((q, wq), (k, wk)))
    if c["op"] == "rotate":
        return q.flatten(1), k.flatten(1)
    if c["cache"] == "e4m3":
        k, v = _exact_e4m3(k, s["k_scale"]), _exact_e4m3(v, s["v_scale"])
    caches = []
    for x in (k, v):
        flat = torch.zeros(c["pages"] * c["page"], c["k_heads"], c["dim"], dtype=torch.float64, device=DEV)
        flat[s["slot"][s["slot"] >= 0]] = x[s["slot"] >= 0]
        caches.append(flat.view(c["pages"], c["page"], c["k_heads"], c["dim"]).transpose(1, 2).contiguous())
    return q.flatten(1), caches[0], caches[1]


def _exact_decode(s):
    c = s["case"]
    S, Hq, Hk, D = c["seqs"], c["q_heads"], c["k_heads"], c["dim"]
    out = torch.zeros(S, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((S, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lens(c)):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        ids = s["table"][i, :-(-n // c["page"])].long()
        k, v = (torch.cat([x[a].double() for a in ids.split(2048)]).transpose(1, 2).reshape(-1, Hk, D)[lo:n]
                if x.dtype == torch.bfloat16 else
                x.view(torch.uint8)[ids].view(x.dtype).double().transpose(1, 2).reshape(-1, Hk, D)[lo:n]
                for x in (s["k"], s["v"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        for h in range(Hk):
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            z = s["q"][i].double().view(Hq, D)[g] @ k[:, h].T / math.sqrt(D)
            lse[i, g] = torch.logsumexp(z, -1)
            out[i, g] = torch.softmax(z, -1) @ v[:, h]
    return out.view(S, Hq * D), lse


def _exact_window(s):
    c = s["case"]
    B, T, H, W = c["batch"], c["tokens"], c["heads"], c["window"]
    out = torch.zeros(B, T, H, 128, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, H, T, dtype=torch.float64, device=DEV)
    dqkv = torch.zeros(B, T, 3, H, 128, dtype=torch.float64, device=DEV)
    x = s["qkv"].view(B, T, 3, H, 128)
    step = max(1024, W) // W * W if c["mode"] == "block" else 2048
    for b in range(B):
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            lo = t0 if c["mode"] == "block" else max(0, t0 - W + 1)
            q = x[b, t0:t1, 0].double().transpose(0, 1).contiguous()
            k, v = (x[b, lo:t1, i].double().transpose(0, 1).contiguous() for i in (1, 2))
            do = s["dout"][b, t0:t1].double().view(t1 - t0, H, 128).transpose(0, 1).contiguous()
            ti = torch.arange(t0, t1, device=DEV)[:, None]
            tj = torch.arange(lo, t1, device=DEV)[None]
            ok = (ti // W == tj // W) if c["mode"] == "block" else (tj <= ti) & (ti - tj < W)
            z = torch.bmm(q, k.transpose(1, 2)) / math.sqrt(128)
            z = z.masked_fill(~ok, -math.inf)
            lse[b, :, t0:t1] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            o = torch.bmm(p, v)
            out[b, t0:t1] = o.transpose(0, 1)
            dp = torch.bmm(do, v.transpose(1, 2))
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(128)
            dqkv[b, t0:t1, 0] += torch.bmm(ds, k).transpose(0, 1)
            dqkv[b, lo:t1, 1] += torch.bmm(ds.transpose(1, 2), q).transpose(0, 1)
            dqkv[b, lo:t1, 2] += torch.bmm(p.transpose(1, 2), do).transpose(0, 1)
    return out.view(B, T, -1), lse, dqkv.view(B, T, -1)
