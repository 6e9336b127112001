"""The bars of the attention calls' GPU tests catch the mistakes they are there for: small ones,
planted here in the oracle, exceed them, and the roundings that the kernels make do not."""
import numpy as np
import pytest
import torch

import attention_bars as bars
import oracle.ttt_attention as oa


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def scale_terms(T, H, D, rot, seed=1):
    """Terms [T, H, D] of a scale's gradient and their sizes G |x r|."""
    rng = np.random.default_rng(seed)
    x, dy = rng.standard_normal((2, T, H, D))
    ang = oa.angles(rng.integers(-5000, 5000, (1, T)), rng.random((1, rot // 2)) ** 4)
    xh = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
    G = np.abs(dy)
    i0, i1 = oa.pair_index(rot, "halves")
    s = G[..., i0] + G[..., i1]
    G[..., i0], G[..., i1] = s, s
    return oa.turn(dy, ang, "halves", -1.0) * xh, G * np.abs(xh)


@pytest.mark.parametrize("T,H,D,rot", [(5003, 2, 64, 64), (40001, 1, 32, 32), (6001, 3, 128, 64), (33000, 2, 64, 0)])
def test_scale_gradient_bar_catches_what_a_launch_may_lose(T, H, D, rot):
    terms, sizes = scale_terms(T, H, D, rot)
    ref = terms.sum((0, 1))
    bar = bars.scale_grad_bar(T, H, D, rot, sizes.sum((0, 1)), ref)
    assert np.all(bar < 0.01 * np.sqrt(np.mean(ref ** 2)))
    tb = max(1, min(16, T // 2048))
    lost = {"the last token": terms[-1:], "the last block": terms[-(T % tb or tb):],
            "one head of the first token": terms[:1, :1], "a workgroup's tokens": terms[7 * tb::512 * tb]}
    for name, part in lost.items():
        assert np.max(np.abs(part.sum((0, 1))) / bar) > 5, name
    # twice the same workgroup, and a sum in the launch's order
    assert np.max(np.abs(terms[:tb].sum((0, 1))) / bar) > 5
    # the sum itself, in chains of fp32 additions of the launch's length joined in 64 bits
    n = bars.scale_grad_chain(T, H, D, rot)
    assert 1 <= n < 64
    flat = terms.reshape(-1, D).astype(np.float32)
    flat = np.concatenate((flat, np.zeros((-len(flat) % n, D), np.float32))).reshape(-1, n, D)
    chain = np.zeros((len(flat), D), np.float32)
    for i in range(n):
        chain += flat[:, i]
    err = chain.astype(np.float64).sum(0) - ref
    assert np.all(np.abs(err) <= bar)
    norm = bars.scale_grad_norm_bar(T, H, D, rot, (sizes ** 2).sum((0, 1)))
    assert np.linalg.norm(err) <= norm < 1e-5 * np.linalg.norm(ref)
    assert np.linalg.norm(terms[:1, :1]) > 20 * norm


def head(T, window, mode, seed=2):
    rng = np.random.default_rng(seed)
    Q, K, V, dO = (bf16(rng.standard_normal((T, 128))) for _ in range(4))
    return Q, K, V, dO, oa.window_probs(Q, K, window, mode)


def grads(Q, K, V, dO, P, delta):
    c = 1 / np.sqrt(128)
    dS = P * (dO @ V.T - delta)
    return c * (dS @ K), c * (dS.T @ Q), P.T @ dO


@pytest.mark.parametrize("T,window,mode", [(2100, 4000, "sliding"), (2100, 500, "sliding"), (1400, 700, "block"),
                                           (300, 37, "sliding"), (300, 1, "sliding"), (520, 128, "block")])
def test_window_models_hold_for_the_roundings_and_catch_one_key(T, window, mode):
    Q, K, V, dO, P = head(T, window, mode)
    out, summed = P @ V, min(window, T) <= 64
    delta = np.sum(dO * out, 1, keepdims=True)
    refs = (out, *grads(Q, K, V, dO, P, delta))
    model = bars.window_models(Q, K, V, dO, P, out, summed)
    # the kernels' roundings: p, ds and the results to bf16, delta of the rounded out
    o16 = bf16(bf16(P) @ V)
    d16 = delta if summed else np.sum(dO * o16, 1, keepdims=True)
    c = 1 / np.sqrt(128)
    dS = bf16(P * (dO @ V.T - d16))
    got = (o16, bf16(c * (dS @ K)), bf16(c * (dS.T @ Q)), bf16(bf16(P).T @ dO))
    assert np.all(np.abs(o16 - out) <= bars.window_out_bar(P, V, out))
    for g, r, m in zip(got, refs, model):
        assert bars.worst_block(g, r, m) <= 1
    if window == 1:
        return
    # one key left out of the products, for the rows of the last block that see it; one query left
    # out of a key's sums
    t0 = T - 32
    lost = P.copy()
    j = T - 33 if mode == "sliding" else T - 40
    lost[t0:, j] = 0
    assert bars.worst_block(lost @ V, out, model[0]) > 2
    assert bars.worst_block(grads(Q, K, V, dO, lost, delta)[0], refs[1], model[1]) > 2
    lost = P.copy()
    lost[T - 20, T - 32:] = 0
    for i, x in enumerate(grads(Q, K, V, dO, lost, delta)[1:]):
        assert bars.worst_block(x, refs[2 + i], model[2 + i]) > 2
    # a row's mask one token short
    shifted = oa.window_probs(Q, K, max(1, min(window, T) - 1), mode) if mode == "sliding" and window < T else None
    if shifted is not None:
        assert bars.worst_block(shifted @ V, out, model[0]) > 2
