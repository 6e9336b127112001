"""Error models of the attention calls, shared by the GPU tests and by the CPU tests that plant
mistakes in the oracle and see them exceed the bars.

U = 2^-24 and R = 2^-8 are the half steps of fp32 and bf16 relative to the value. Rounded once, a
number is off by at most its half step; over many numbers the error's root mean square is at most
R / sqrt(3) of theirs (evenly spread over the step, at the low end of a binade, where the step
is largest against the value).
"""
import numpy as np

U = 2.0 ** -24
R = 2.0 ** -8
BLOCK = 32      # rows that a 2-norm is taken over: those of one wave


def scale_grad_chain(tokens, heads, dim, rot):
    """fp32 additions that one lane makes for a scale's gradient, as the launch lays them out: a
    workgroup of 256 lanes takes blocks of tb tokens, its groups of lph lanes a head each; the
    lanes', workgroups' and launch's sums are joined in 64 bits."""
    lph = 1
    while lph * 16 < dim:
        lph *= 2
    groups = 256 // lph
    fit = min(16, 2048 // (rot // 2)) if rot else 16
    tb = max(1, min(fit, tokens // 2048))
    blocks = -(-tokens // tb)
    return -(-blocks // min(blocks, 512)) * -(-tb * heads // groups)


def scale_grad_bar(tokens, heads, dim, rot, terms, ref):
    """Bar of a scale's gradient [dim]: terms = sum over tokens and heads of G |x r|. A term's
    gradient carries 16 U of G (the turn back), its x r 17 U; every addition of a chain rounds a
    partial sum, which the terms' sum bounds; a workgroup's sum and the result are rounded once
    more."""
    return (33 + scale_grad_chain(tokens, heads, dim, rot) + 1) * U * terms + U * np.abs(ref)


def scale_grad_norm_bar(tokens, heads, dim, rot, squares):
    """Bar of the 2-norm over the columns of that gradient's error: the terms' errors, each at its
    bound, and those of a chain's additions, independent of each other.  squares = sum over
    tokens and heads of (G |x r|)^2."""
    return (33 + np.sqrt(scale_grad_chain(tokens, heads, dim, rot))) * U * np.sqrt(np.sum(squares))


def block_norms(x):
    """2-norms of BLOCK rows each of x [rows, n]; the last block takes what is left, at least
    BLOCK rows where there are as many."""
    n = max(1, len(x) // BLOCK)
    return np.array([np.linalg.norm(x[BLOCK * i:(BLOCK * (i + 1) if i + 1 < n else len(x))]) for i in range(n)])


def window_models(Q, K, V, dO, P, out, summed):
    """Root mean squares [T, 128] of the errors of out, dq, dk, dv of one head, from the
    definition's P and out: each bf16 rounding taken as an error of R / sqrt(3) of what is
    rounded, independent of the others (out; p for the products with v and dout; ds; out again in
    delta = dout . out, unless it is summed as p dp)."""
    c = 1 / np.sqrt(Q.shape[1])
    r = R / np.sqrt(3)
    dP = dO @ V.T
    dS = P * (dP - np.sum(dO * out, 1, keepdims=True))
    d2 = 0 if summed else np.sum((dO * out) ** 2, 1, keepdims=True)   # delta's, over r
    dq, dk, dv = c * (dS @ K), c * (dS.T @ Q), P.T @ dO
    sq = (out ** 2 + P ** 2 @ V ** 2,
          dq ** 2 + c * c * (dS ** 2 @ K ** 2 + d2 * (P @ K) ** 2),
          dk ** 2 + c * c * (dS ** 2).T @ Q ** 2 + c * c * (P ** 2 * d2).T @ Q ** 2,
          dv ** 2 + (P ** 2).T @ dO ** 2)
    return [r * np.sqrt(x) for x in sq]


def window_out_bar(P, V, out):
    """Every element of out: its rounding, and each probability's for the product with v."""
    return R * np.abs(out) + (R + 2.0 ** -14) * (P @ np.abs(V)) + 1e-30


def worst_block(got, ref, model):
    """The largest error of a block of rows against 1.5 times the model's (a block has thousands of
    roundings, whose sum of squares does not leave its mean by half; the model takes every step
    at its largest, 1.4 times the mean over a binade), and 2^-14 of the values for fp32's parts."""
    bar = 1.5 * block_norms(model) + 2.0 ** -14 * block_norms(ref)
    return float(np.max(block_norms(got - ref) / np.maximum(bar, 1e-30)))
