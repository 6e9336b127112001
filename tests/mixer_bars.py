"""Error models of the mixer calls, shared by the GPU tests and by the CPU tests that plant mistakes in
the oracle and see them exceed the bars.

U = 2^-24 and R = 2^-8 are the half steps of fp32 and bf16 relative to the value.

Linear attention, for one head, in chunks of C = 64 tokens from the sequence's first (backward in
time: last) token.  Every sum is bounded by that of its terms' absolute values, A.  A state takes
per chunk a product with a power (2 U), at most 3 C additions of products of bf16 numbers (the decayed
value in three parts: 3 C U), the decayed value's own roundings (power, scale, product: 4 U), and one
join of a segment's sum with the state before it (2 U):
  E' = a^n E + (3 n + 8) U A'.
Where only outputs follow from it the decayed value enters in two parts, which leave 2^-16 of it: F, as E
and 2^-16 (A' - a^n A) a chunk.  An output takes the state in two bf16 parts (each leaves at most 2^-8 of what it is given: 2^-16) in a
sum of 2 D products, the power and scale (3 U); and the chunk's own scores, sums of D products (D U),
with the mask's factor (3 U), in two bf16 parts (2^-16) in a sum of 2 C products.  It is rounded to bf16
at the end.

Norms.  The sum of squares runs over chains of at most 32 + 9 additions of positive terms (half
of it after the root), mean, eps, root and division 4 U: r within 26 U.  u = y r w 28 U, the gate's
value 8 U and its product 2 U, the residual's sum U: h' is within e = 41 U |s z| + U |h'|.  p is
within 26 U and sum |h'| e / sum h'^2; n adds 2 U.  Backward, with X = p (|h| + |s z|) for |x|, which
is then within 71 U X; a mean of a x takes 41 U more for its sum: d = dh' + p (a - x m) is within
2^-16 (|dh'| + p |a| + p X mean(|a| X)) = 2^-16 D.  What follows are products of it with numbers within
60 U, and one more mean: 2^-15 of the same terms.  The scales' gradients: chains of a few additions a
lane, the others in 64 bits: 2^-14 of the sum of the terms' bounds.
"""
import numpy as np

U = 2.0 ** -24
R = 2.0 ** -8
C = 64


def layer(q, k, v, decay, x0, scale_p, scale_s, scale_w, forward):
    """One recurrence as the kernel has it, in 64 bits, with its bars: (out, bar), (state, bar).
    forward: x0 is the state before the first token and the last token's state is given; else the
    operands are in reversed order, x0 is what the first of them meets and the state is given as the
    next would meet it."""
    K, V = k.shape[1], v.shape[1]
    S, A, E, F = np.array(x0, np.float64), np.abs(x0), np.zeros((K, V)), np.zeros((K, V))
    out, bar = np.zeros((len(q), V)), np.zeros((len(q), V))
    for t0 in range(0, len(q), C):
        n = min(C, len(q) - t0)
        qq, kk, vv = q[t0:t0 + n], k[t0:t0 + n], v[t0:t0 + n]
        e0 = 1 if forward or t0 > 0 else 0
        i = np.arange(n)
        near = np.where(i[:, None] >= i, np.power(decay, np.maximum(i[:, None] - i, 0)), 0.0) * scale_p
        past = np.power(decay, i + e0)[:, None] * scale_s
        out[t0:t0 + n] = past * (qq @ S) + (near * (qq @ kk.T)) @ vv
        bar[t0:t0 + n] = (past * (np.abs(qq) @ (F + (2.0 ** -16 + (2 * K + 8) * U) * A)) +
                          (2.0 ** -16 + (K + 2 * C + 8) * U) * ((near * (np.abs(qq) @ np.abs(kk).T)) @ np.abs(vv)))
        w = np.power(decay, n - 1 - i)[:, None] * scale_w
        f = decay ** (n - 1 + e0)
        S = f * S + kk.T @ (w * vv)
        new = np.abs(kk).T @ (w * np.abs(vv))
        A = f * A + new
        E = f * E + (3 * n + 8) * U * A
        F = f * F + (3 * n + 8) * U * A + 2.0 ** -16 * new
    if not forward and len(q):
        S, A, E = decay * S, decay * A, decay * E + U * decay * A
    return (out, bar + R * np.abs(out) + 1e-30), (S, E + U * np.abs(S) + 1e-30)


def forward(q, k, v, decay, s0, scale):
    return layer(q, k, v, decay, s0, scale, scale, 1.0, True)


def backward(q, k, v, decay, s0, scale, do, ds):
    """[(dq, bar), (dk, bar), (dv, bar), (ds0, bar)]."""
    turn = lambda x: x[::-1]  # noqa: E731
    dq = layer(do, v, k, decay, s0.T, scale, scale, 1.0, True)[0]
    dk = layer(turn(v), turn(do), turn(q), decay, ds.T, scale, 1.0, scale, False)[0]
    dv, d0 = layer(turn(k), turn(q), turn(do), decay, ds, scale, 1.0, scale, False)
    return [dq, tuple(turn(x) for x in dk), tuple(turn(x) for x in dv), d0]


def norm(f, y, h, rs, wn, H):
    """Bars of h_out and n_out from the oracle's values f; H: half step of the output's type."""
    sz = np.abs((1 if rs is None else rs) * f["z"])
    e = 41 * U * sz + U * np.abs(f["h_out"])
    sq = np.sum(f["h_out"] ** 2, -1, keepdims=True)
    rel = 28 * U + np.sum(np.abs(f["h_out"]) * e, -1, keepdims=True) / np.maximum(sq, 1e-300)
    n = np.abs(f["n_out"])
    return (H * np.abs(f["h_out"]) + e + 1e-38,
            H * n + (1 if wn is None else np.abs(wn)) * f["p"] * e + rel * n + 1e-38)


def norm_backward(f, ref, y, h, gate, wy, rs, wn, dho, dn, groups, norm_y, H):
    """Bars of a backward's outputs by name."""
    one = lambda x: 1.0 if x is None else np.abs(x)  # noqa: E731
    X = f["p"] * ((0 if h is None else np.abs(h)) + one(rs) * np.abs(f["z"]))
    a = np.abs(dn) * one(wn)
    D = np.abs(dho) + f["p"] * (a + X * np.mean(a * X, -1, keepdims=True))
    dz = D * one(rs)
    du = dz * np.abs(f["act"])
    yr = np.abs(y * f["r"])
    b = du * one(wy)
    dy = b
    if norm_y:
        m = (b * yr).reshape(len(y), groups, -1)
        m = np.broadcast_to(np.mean(m, -1, keepdims=True), m.shape).reshape(y.shape)
        dy = f["r"] * (b + yr * m)
    bars = dict(dh=2.0 ** -16 * D, dy=2.0 ** -15 * dy, dwy=2.0 ** -14 * np.sum(du * yr, 0),
                drs=2.0 ** -14 * np.sum(D * np.abs(f["z"]), 0), dwn=2.0 ** -14 * np.sum(np.abs(dn) * X, 0))
    if gate is not None:
        s = 1 / (1 + np.exp(-gate))
        bars["dgate"] = 2.0 ** -15 * dz * np.abs(f["u"]) * s * (1 + np.abs(gate))
    for k in ("dh", "dy", "dgate"):
        if bars.get(k) is not None:
            bars[k] = bars[k] + H * np.abs(ref[k])
    return {k: v + 1e-38 for k, v in bars.items()}
