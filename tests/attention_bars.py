"""Error models of the attention calls, shared by the GPU tests and by the CPU tests that plant
mistakes in the oracle and see them exceed the bars.

U = 2^-24 is the half step of fp32 relative to the value.
"""
import numpy as np

U = 2.0 ** -24


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
