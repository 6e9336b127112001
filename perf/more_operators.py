"""The linear attention with a decay for each head (a prompt, a training step, single tokens) and
the norms, gate and residual between two sub-layers (and their backward), as cases to measure.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` makes what a program holds before the
call, `run(state)` is one call: in plain torch operations, or with `own` set through the library.
`exact(case, seed)` computes the outputs in 64 bits from the definitions, `work(case)` the bytes
and operations that a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 128     # tokens of a chunk of the plain form


# ------------------------------------------------------------------------------------ cases
def listed():
    step = {"op": "step", "dim_k": 128, "dim_v": 128}
    prompt = {"op": "prompt", "dim_k": 128, "dim_v": 128, "carry": True}
    train = {"op": "train", "dim_k": 128, "dim_v": 128, "carry": False}
    text = {"dim": 1024, "groups": 1, "act": "bf16", "norm_y": True, "gate": "none", "residual": True,
            "scale": True, "norm_n": True}
    return [
        # a single conversation's next token: 8 heads of 128, the LM block's
        dict(step, name="step_one", seqs=1, heads=8),
        # a decoding step of a serving batch
        dict(step, name="step_batch", seqs=256, heads=8),
        # heads of 64 (the small chunk's 12), an odd number of sequences
        dict(step, name="step_narrow", seqs=61, heads=12, dim_k=64, dim_v=64),
        # three short prompts of a chat, ragged, each continuing a state
        dict(prompt, name="prompt_short", seqs=3, max_len=130, heads=8),
        # a serving batch's prompts of ragged lengths, the small chunk's heads
        dict(prompt, name="prompt_ragged", seqs=24, max_len=4096, heads=12, dim_k=64, dim_v=64),
        # the long workload's 131072 tokens
        dict(prompt, name="prompt_long", seqs=1, max_len=131072, heads=8),
        # a short ragged training batch whose sequences go on from a state
        dict(train, name="train_small", batch=3, tokens=777, heads=2, carry=True),
        # the LM block's training sequence of 32768 tokens
        dict(train, name="train_text", batch=1, tokens=32768, heads=8),
        # one decoding step of four sequences between two sub-layers of the LM block
        dict(text, op="norm", name="norm_step", tokens=4),
        # eight images of 8040 tokens of the image set's block, in 32 bits
        dict(text, op="norm", name="norm_images", tokens=8 * 8040, dim=768, act="f32"),
        # the LM block's training sequence: the norm of each head of a sequence layer's output,
        # gated, then residual and next norm, backward
        dict(text, op="norm_grad", name="norm_grad_text", tokens=32768, groups=8, gate="silu"),
        # three images and a ragged rest, 32 bits
        dict(text, op="norm_grad", name="norm_grad_images", tokens=3 * 8040 + 77, dim=768, act="f32",
             gate="sigmoid", scale=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "step", "prompt", "prompt", "train", "train", "norm", "norm_grad"])
    if op in ("norm", "norm_grad"):
        groups, wide = rng.choice([(1, 0), (1, 0), (4, 64), (6, 128), (8, 128), (5, 16), (3, 256)])
        dim = groups * wide if wide else rng.choice([8 * _log(rng, 1, 1024), 64, 768, 1024, 2048])
        parts = {k: rng.random() < 0.75 for k in ("norm_y", "residual", "scale", "norm_n")}
        if not parts["norm_y"]:
            groups = 1
        return {"op": op, "tokens": _log(rng, 1, max(64, 33554432 // dim)), "dim": dim, "groups": groups,
                "act": rng.choice(["bf16", "bf16", "f32"]), "gate": rng.choice(["none", "sigmoid", "silu"]), **parts}
    heads = rng.choice([1, 2, 3, 4, 8, 12])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64), (256, 256), (256, 64), (64, 256)])
    case = {"op": op, "heads": heads, "dim_k": dk, "dim_v": dv}
    if op == "step":
        case.update(seqs=_log(rng, 1, 256 * 8 * 128 * 128 // (heads * dk * dv)))
    elif op == "prompt":
        seqs = _log(rng, 1, 64)
        most = 131072 * 8 * 128 // (heads * max(dk, dv) * seqs)
        case.update(seqs=seqs, max_len=_log(rng, 1, min(65536, most)), carry=rng.random() < 0.7)
    else:
        batch = rng.choice([1, 1, 2, 3, 4])
        case.update(batch=batch, tokens=_log(rng, 1, 32768 * 8 * 128 // (heads * max(dk, dv) * batch)),
                    carry=rng.random() < 0.5)
    return case


def _lens(c):
    """The prompts' lengths: spread over 1 .. max_len, the first at max_len, and with eight or more
    one that is empty."""
    return [c["max_len"]] + [
        0 if i == 5 and c["seqs"] >= 8 else 1 + int((c["max_len"] - 1) * math.modf(0.6180339887 * i)[0])
        for i in range(1, c["seqs"])]


def work(c):
    op = c["op"]
    if op in ("norm", "norm_grad"):
        n, size = c["tokens"] * c["dim"], 2 if c["act"] == "bf16" else 4
        read = 1 + (c["gate"] != "none") + c["residual"]
        if op == "norm":    # the residual sum (or the sub-layer's own output) and the norm
            return {"bytes": n * size * (read + 1 + c["norm_n"]), "flops": 12 * n}
        return {"bytes": n * size * (2 * read + 1 + c["norm_n"]), "flops": 30 * n}
    H, K, V = c["heads"], c["dim_k"], c["dim_v"]
    if op == "step":        # the state read and written in 32 bits, the token's rows in 16
        return {"bytes": c["seqs"] * H * (8 * K * V + 4 * K + 4 * V), "flops": 5 * c["seqs"] * H * K * V}
    # a token's product with the state and its own with it: 4 K V, whatever the chunks
    if op == "prompt":
        n = sum(_lens(c)) * H
        return {"bytes": n * 4 * (K + V) + 4 * c["seqs"] * H * K * V * (1 + c["carry"]), "flops": 4 * K * V * n}
    n = c["batch"] * c["tokens"] * H
    return {"bytes": n * 2 * (4 * K + 4 * V) + 4 * c["batch"] * H * K * V * 3 * c["carry"], "flops": 12 * K * V * n}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    c, bf = dict(case), torch.bfloat16
    if c["op"] in ("norm", "norm_grad"):
        T, D = c["tokens"], c["dim"]
        dt = torch.float32 if c["act"] == "f32" else bf
        new = lambda: torch.empty(T, D, dtype=dt, device=DEV)  # noqa: E731
        s = {"case": c, "y": (0.5 * randn(T, D)).to(dt), "h": (2 * randn(T, D)).to(dt) if c["residual"] else None,
             "gate": (1.5 * randn(T, D)).to(dt) if c["gate"] != "none" else None,
             "y_weight": (1 + 0.1 * randn(D)).to(dt) if c["norm_y"] else None,
             "res_scale": (0.5 + 0.1 * randn(D)).to(dt) if c["scale"] else None,
             "n_weight": (1 + 0.1 * randn(D)).to(dt) if c["norm_n"] else None}
        if c["op"] == "norm":
            s.update(h_out=new(), n_out=new() if c["norm_n"] else None)
        else:
            sums = lambda w: torch.empty(D, device=DEV) if w is not None else None  # noqa: E731
            s.update(dh_out=randn(T, D).to(dt), dn=randn(T, D).to(dt) if c["norm_n"] else None,
                     dh=new() if c["residual"] else None, dy=new(), dgate=new() if c["gate"] != "none" else None,
                     dy_weight=sums(s["y_weight"]), dres_scale=sums(s["res_scale"]), dn_weight=sums(s["n_weight"]))
        return s
    H, K, V = c["heads"], c["dim_k"], c["dim_v"]
    # the heads' memories from 4 tokens to about a thousand, as such layers are set up
    reach = 2 + 8 * torch.arange(H, device=DEV) / max(1, H - 1) + 0.3 * torch.rand(H, generator=g, device=DEV)
    s = {"case": c, "decay": 1 - torch.exp2(-reach)}
    rows = {"step": c.get("seqs"), "prompt": sum(_lens(c)) if c["op"] == "prompt" else 0,
            "train": c.get("batch", 0) * c.get("tokens", 0)}[c["op"]]
    # queries, keys and values as one projection's rows
    s["qkv"] = (0.7 * randn(rows, H * (2 * K + V))).to(bf)
    s["out"] = torch.empty(rows, H * V, dtype=bf, device=DEV)
    if c["op"] == "train":
        B = c["batch"]
        s.update(dout=randn(rows, H * V).to(bf), dqkv=torch.empty_like(s["qkv"]),
                 state=4 * randn(B, H, K, V) if c["carry"] else None,
                 dstate=randn(B, H, K, V) if c["carry"] else None,
                 dstate_in=torch.empty(B, H, K, V, device=DEV) if c["carry"] else None)
        return s
    # states of sequences in a pool that has some to spare; the new ones go to a pool of their own,
    # so that a guessed token can be taken back
    n = c["seqs"]
    s["slot"] = torch.randperm(n + 3, generator=g, device=DEV)[:n].to(torch.int32)
    s["state"] = 4 * randn(n + 3, H, K, V) if c.get("carry", True) else None
    s["state_out"] = torch.zeros(n + 3, H, K, V, device=DEV)
    if c["op"] == "prompt":
        starts = torch.tensor([0] + _lens(c), device=DEV).cumsum(0)
        s["starts"] = starts.to(torch.int32)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _thirds(x, c):
    H, K, V = c["heads"], c["dim_k"], c["dim_v"]
    return x[:, :H * K].reshape(-1, H, K), x[:, H * K:2 * H * K].reshape(-1, H, K), x[:, 2 * H * K:].reshape(-1, H, V)


def _powers(decay, n):
    """decay^n [H, ...] of whole numbers n >= 0, in 64 bits."""
    d = decay.double().reshape(-1, *[1] * n.dim())
    return d ** n.double()


def _recur(q, k, v, decay):
    """sum over j <= i of decay^(i - j) (q_i . k_j) v_j, for q, k, v [B, H, T, .] in 32 bits, and
    sum over j of decay^(T - 1 - j) k_j v_j^T: chunks with zeros before the first token, each
    chunk's state from all before it."""
    B, H, T, K = k.shape
    N = max(1, -(-T // CHUNK))
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, N * CHUNK - T, 0)).reshape(B, H, N, CHUNK, -1)  # noqa: E731
    q, k, v = pad(q), pad(k), pad(v)
    i = torch.arange(CHUNK, device=DEV)
    near = (i[:, None] - i[None]).clamp_min(0)
    mask = torch.where(i[:, None] >= i[None], _powers(decay, near), 0.0).float()
    out = ((q @ k.transpose(-1, -2)) * mask[:, None]) @ v
    tail = _powers(decay, CHUNK - 1 - i).float()[:, None, :, None]
    local = ((k * tail).transpose(-1, -2) @ v).reshape(B, H, N, -1)
    n = torch.arange(N + 1, device=DEV)
    far = n[:, None] - 1 - n[None, :-1]
    join = torch.where(far >= 0, _powers(decay, CHUNK * far.clamp_min(0)), 0.0).float()
    states = (join @ local).reshape(B, H, N + 1, K, -1)
    head = _powers(decay, 1 + i).float()[:, None, :, None]
    out = out + head * (q @ states[:, :, :N])
    return out.reshape(B, H, N * CHUNK, -1)[:, :, N * CHUNK - T:], states[:, :, N]


def _plain_step(s):
    c = s["case"]
    q, k, v = (x.float() for x in _thirds(s["qkv"], c))
    at = s["slot"].long()
    new = s["state"][at] * s["decay"][:, None, None] + k[..., :, None] * v[..., None, :]
    out = (q[..., :, None] * new).sum(-2) * (1 / math.sqrt(c["dim_k"]))
    s["state_out"][at] = new
    return out.flatten(1).to(torch.bfloat16), s["state_out"]


def _plain_prompt(s):
    c, starts, lam = s["case"], s["starts"].long(), s["decay"]
    S, L = c["seqs"], c["max_len"]
    lens = starts[1:] - starts[:-1]
    # prompts at the ends of rows of max_len places
    at = torch.arange(L, device=DEV)[None] - (L - lens[:, None])
    seen = at >= 0
    row = (starts[:-1, None] + at).clamp_min(0)
    q, k, v = (torch.where(seen[..., None, None], x.float()[row], 0.0).transpose(1, 2) for x in _thirds(s["qkv"], c))
    out, state = _recur(q, k, v, lam)
    if s["state"] is not None:
        first = s["state"][s["slot"].long()]
        past = _powers(lam, (at + 1).clamp_min(0)).float().transpose(0, 1)
        out = out + past[..., None] * (q @ first)
        state = state + _powers(lam, lens).float().t()[..., None, None] * first
    out = (out * (1 / math.sqrt(c["dim_k"]))).transpose(1, 2)[seen]
    s["state_out"][s["slot"].long()] = state
    return out.flatten(1).to(torch.bfloat16), s["state_out"]


def _plain_train(s):
    c, lam = s["case"], s["decay"]
    B, T, H, scale = c["batch"], c["tokens"], c["heads"], 1 / math.sqrt(c["dim_k"])
    heads = lambda x: x.float().reshape(B, T, H, -1).transpose(1, 2)  # noqa: E731
    rows = lambda x: x.transpose(1, 2).reshape(B * T, -1).to(torch.bfloat16)  # noqa: E731
    back = lambda x: x.flip(2)  # noqa: E731
    q, k, v = (heads(x) for x in _thirds(s["qkv"], c))
    do = heads(s["dout"])
    out, _ = _recur(q, k, v, lam)
    dq, _ = _recur(do, v, k, lam)
    dk, _ = _recur(back(v), back(do), back(q), lam)
    dv, _ = _recur(back(k), back(q), back(do), lam)
    out, dq, dk, dv = scale * out, scale * dq, scale * back(dk), scale * back(dv)
    if s["state"] is None:
        return rows(out), torch.cat([rows(dq), rows(dk), rows(dv)], -1)
    t = torch.arange(T, device=DEV)
    past, rest = _powers(lam, t + 1).float()[..., None], _powers(lam, T - 1 - t).float()[..., None]
    first, last = s["state"], s["dstate"]
    out = out + scale * past * (q @ first)
    dq = dq + scale * past * (do @ first.transpose(-1, -2))
    dk = dk + rest * (v @ last.transpose(-1, -2))
    dv = dv + rest * (k @ last)
    before = _powers(lam, torch.tensor(T, device=DEV)).float()[:, None, None] * last
    before = before + scale * (past * q).transpose(-1, -2) @ do
    return rows(out), torch.cat([rows(dq), rows(dk), rows(dv)], -1), before


def _acts(s):
    """The gate's value and slope."""
    if s["gate"] is None:
        return 1.0, None
    g = s["gate"].float()
    sig = 1 / (1 + torch.exp(-g))
    if s["case"]["gate"] == "sigmoid":
        return sig, sig * (1 - sig)
    return g * sig, sig * (1 + g * (1 - sig))


def _normed(x, w, groups):
    """x over the root mean square of its groups, that times w, and 1 / root."""
    x = x.reshape(len(x), groups, -1)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = (x * r).flatten(1)
    return n, n * w.float(), r


def _norm_parts(s):
    c = s["case"]
    y = s["y"].float()
    u = _normed(y, s["y_weight"], c["groups"])[1] if c["norm_y"] else y
    z = u * _acts(s)[0]
    hh = z if s["res_scale"] is None else z * s["res_scale"].float()
    return u, z, hh if s["h"] is None else s["h"].float() + hh


def _plain_norm(s):
    dt = s["y"].dtype
    h = _norm_parts(s)[2]
    if s["n_weight"] is None:
        return h.to(dt)
    return h.to(dt), _normed(h, s["n_weight"], 1)[1].to(dt)


def _norm_back(x, w, groups, d):
    """Gradients of x and w for the gradient d of _normed(x, w, groups)[1]."""
    n, _, r = _normed(x, w, groups)
    u = (d * w.float()).reshape(len(x), groups, -1)
    xh = n.reshape(u.shape)
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    return dx.flatten(1), (d * n).double().sum(0).float()


def _plain_norm_grad(s):
    c, dt = s["case"], s["y"].dtype
    u, z, h = _norm_parts(s)
    act, slope = _acts(s)
    d, dgate, dyw, drs, dnw = s["dh_out"].float(), None, None, None, None
    if s["dn"] is not None:
        dx, dnw = _norm_back(h, s["n_weight"], 1, s["dn"].float())
        d = d + dx
    dz = d
    if s["res_scale"] is not None:
        drs = (d * z).double().sum(0).float()
        dz = d * s["res_scale"].float()
    if slope is not None:
        dgate = (dz * u * slope).to(dt)
    dy = dz * act
    if c["norm_y"]:
        dy, dyw = _norm_back(s["y"].float(), s["y_weight"], c["groups"], dy)
    return {"dh": None if s["h"] is None else d.to(dt), "dy": dy.to(dt), "dgate": dgate, "dy_weight": dyw,
            "dres_scale": drs, "dn_weight": dnw}


# ------------------------------------------------------------------------------------ the library
def _own_linear(s):
    import weight_sequence_layers_amd as W
    c, x = s["case"], s["qkv"]
    H, K, V = c["heads"], c["dim_k"], c["dim_v"]
    cfg = W.make_linear_attention_config(heads=H, dim_k=K, dim_v=V)
    ld, q, k, v = x.shape[1], x, x[:, H * K:], x[:, 2 * H * K:]
    if c["op"] == "step":
        W.ttt_linear_attention_step(cfg, q, ld, k, ld, v, ld, s["decay"], s["state"], s["state_out"], s["slot"],
                                    s["out"], H * V, c["seqs"])
        return s["out"], s["state_out"]
    if c["op"] == "prompt":
        S, L, T = c["seqs"], c["max_len"], len(x)
        if "work" not in s:
            s["work"] = torch.empty(W.ttt_linear_attention_work(cfg, S, L), dtype=torch.uint8, device=DEV)
        W.ttt_linear_attention(cfg, q, ld, k, ld, v, ld, s["decay"], s["starts"], s["state"], s["state_out"],
                               s["slot"], s["out"], H * V, T, S, L, s["work"])
        return s["out"], s["state_out"]
    B, T, dx = c["batch"], c["tokens"], s["dqkv"]
    if "work" not in s:
        n = max(W.ttt_linear_attention_work(cfg, B, T), W.ttt_linear_attention_backward_work(cfg, B, T))
        s["work"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    W.ttt_linear_attention(cfg, q, ld, k, ld, v, ld, s["decay"], None, s["state"], None, None, s["out"], H * V,
                           B * T, B, T, s["work"])
    W.ttt_linear_attention_backward(cfg, q, ld, k, ld, v, ld, s["decay"], None, s["state"], s["dout"], H * V,
                                    s["dstate"], dx, ld, dx[:, H * K:], ld, dx[:, 2 * H * K:], ld, s["dstate_in"],
                                    B * T, B, T, s["work"])
    return (s["out"], dx) if s["state"] is None else (s["out"], dx, s["dstate_in"])


def _own_norm(s):
    import weight_sequence_layers_amd as W
    c = s["case"]
    T, D = c["tokens"], c["dim"]
    cfg = W.make_residual_norm_config(dim=D, groups=c["groups"], norm_y=c["norm_y"], gate=c["gate"], act=c["act"])
    ins = (s["h"], D, s["y"], D, s["gate"], D, s["y_weight"], s["res_scale"], s["n_weight"])
    if c["op"] == "norm":
        W.ttt_residual_norm(cfg, *ins, s["h_out"], D, s["n_out"], D, T)
        return s["h_out"] if s["n_out"] is None else (s["h_out"], s["n_out"])
    if "work" not in s:
        s["work"] = torch.empty(W.ttt_residual_norm_backward_work(cfg, T), dtype=torch.uint8, device=DEV)
    W.ttt_residual_norm_backward(cfg, *ins, s["dh_out"], D, s["dn"], D, s["dh"], D, s["dy"], D, s["dgate"], D,
                                 s["dy_weight"], s["dres_scale"], s["dn_weight"], s["work"], T)
    return {k: s[k] for k in ("dh", "dy", "dgate", "dy_weight", "dres_scale", "dn_weight")}


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_norm if op.startswith("norm") else _own_linear)(state)
    return {"step": _plain_step, "prompt": _plain_prompt, "train": _plain_train, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad}[op](state)


# ------------------------------------------------------------------------------------ 64 bits
def _exact_layer(q, k, v, lam, first, lens, scale):
    """The recurrence token by token: q, k, v [B, T, H, .], first [B, H, K, V] or None, lens [B].
    Returns (out [B, T, H, V], the state behind each sequence's last token)."""
    B, T, H, K = q.shape
    state = torch.zeros(B, H, K, v.shape[-1], dtype=torch.float64, device=DEV) if first is None else first.double().clone()
    out, same = torch.empty_like(v), bool((lens == T).all())
    for t in range(T):
        new = torch.addcmul(state * lam[:, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
        state = new if same else torch.where((t < lens)[:, None, None, None], new, state)
        out[:, t] = (q[:, t, :, :, None] * state).sum(-2)
    return out * scale, state


def _exact_train(s, q, k, v, lam, scale):
    """Gradients token by token: the states forward for dq, their cotangents backward for dk, dv."""
    c = s["case"]
    B, T, H = c["batch"], c["tokens"], c["heads"]
    do = s["dout"].double().reshape(B, T, H, -1)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    state = torch.zeros(B, H, q.shape[-1], v.shape[-1], dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].double()
    for t in range(T):
        state = torch.addcmul(state * lam[:, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
        dq[:, t] = scale * (state * do[:, t, :, None, :]).sum(-1)
    cot = torch.zeros_like(state) if s["dstate"] is None else s["dstate"].double()
    for t in range(T - 1, -1, -1):
        cot = torch.addcmul(cot, scale * q[:, t, :, :, None], do[:, t, :, None, :])
        dk[:, t] = (cot * v[:, t, :, None, :]).sum(-1)
        dv[:, t] = (cot * k[:, t, :, :, None]).sum(-2)
        cot = cot * lam[:, None, None]
    return torch.cat([x.reshape(B * T, -1) for x in (dq, dk, dv)], -1), cot


def _exact_linear(s):
    c, lam = s["case"], s["decay"].double()
    H, K, V, scale = c["heads"], c["dim_k"], c["dim_v"], c["dim_k"] ** -0.5
    x = s["qkv"].double()
    q, k, v = x[:, :H * K].view(-1, H, K), x[:, H * K:2 * H * K].view(-1, H, K), x[:, 2 * H * K:].view(-1, H, V)
    if c["op"] == "train":
        B, T = c["batch"], c["tokens"]
        q, k, v = (y.reshape(B, T, H, -1) for y in (q, k, v))
        out, _ = _exact_layer(q, k, v, lam, s["state"], torch.full((B,), T, device=DEV), scale)
        grads, cot = _exact_train(s, q, k, v, lam, scale)
        out = out.reshape(B * T, H * V)
        return (out, grads) if s["state"] is None else (out, grads, cot)
    lens = [1] * c["seqs"] if c["op"] == "step" else _lens(c)
    most, at = max(lens), 0
    padded = [torch.zeros(c["seqs"], most, H, y.shape[-1], dtype=torch.float64, device=DEV) for y in (q, k, v)]
    for b, n in enumerate(lens):
        for p, y in zip(padded, (q, k, v)):
            p[b, :n] = y[at:at + n]
        at += n
    slot = s["slot"].long()
    out, last = _exact_layer(*padded, lam, None if s["state"] is None else s["state"][slot],
                             torch.tensor(lens, device=DEV), scale)
    pool = s["state_out"].double()
    pool[slot] = last
    return torch.cat([out[b, :n] for b, n in enumerate(lens)]).reshape(-1, H * V), pool


def _exact_norm(s):
    c = s["case"]
    x = {k: None if s[k] is None else s[k].double() for k in ("h", "y", "gate", "y_weight", "res_scale", "n_weight")}
    T, D, G = c["tokens"], c["dim"], c["groups"]
    one = torch.ones(D, dtype=torch.float64, device=DEV)
    root = lambda z, g: torch.sqrt((z.view(T, g, D // g) ** 2).sum(-1, keepdim=True) / (D // g) + 1e-6).expand(T, g, D // g).reshape(T, D)  # noqa: E731
    ry = root(x["y"], G) if c["norm_y"] else 1.0
    wy = x["y_weight"] if c["norm_y"] else one
    sig = torch.sigmoid(x["gate"]) if c["gate"] != "none" else None
    act = 1.0 if sig is None else sig if c["gate"] == "sigmoid" else x["gate"] * sig
    rs = one if x["res_scale"] is None else x["res_scale"]
    z = x["y"] / ry * wy * act
    h = z * rs + (0 if x["h"] is None else x["h"])
    rh = root(h, 1)
    if c["op"] == "norm":
        return h if x["n_weight"] is None else (h, h / rh * x["n_weight"])
    d, dnw = s["dh_out"].double(), None
    if s["dn"] is not None:
        dn = s["dn"].double()
        dnw = (dn * h / rh).sum(0)
        a = dn * x["n_weight"]
        d = d + a / rh - h * (a * h).sum(-1, keepdim=True) / (D * rh ** 3)
    dz = d * rs
    dgate = None
    if sig is not None:
        slope = sig * (1 - sig) if c["gate"] == "sigmoid" else sig + x["gate"] * sig * (1 - sig)
        dgate = dz * x["y"] / ry * wy * slope
    du, dyw = dz * act, None
    if c["norm_y"]:
        dyw = (du * x["y"] / ry).sum(0)
        a = du * wy
        part = (a * x["y"]).view(T, G, D // G).sum(-1, keepdim=True).expand(T, G, D // G).reshape(T, D)
        du = a / ry - x["y"] * part / ((D // G) * ry ** 3)
    return {"dh": None if x["h"] is None else d, "dy": du, "dgate": dgate, "dy_weight": dyw,
            "dres_scale": None if x["res_scale"] is None else (d * z).sum(0), "dn_weight": dnw}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_linear(s)
