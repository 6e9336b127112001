"""Pins of the attention oracle: its gradients against differences, its special cases against
the block oracle and against sums written out."""
import numpy as np
import pytest

import oracle.ttt_attention as oa
import oracle.ttt_block as blk


def _diff(f, x, dx, h=1e-5):
    return (f(x + h * dx) - f(x - h * dx)) / (2 * h)


@pytest.mark.parametrize("pairing", ["halves", "pairs"])
@pytest.mark.parametrize("eps,weighted,rot", [(1e-6, True, 16), (1e-2, False, 32), (None, False, 16)])
def test_norm_rope_gradients_against_differences(pairing, eps, weighted, rot):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((5, 3, 32)), rng.standard_normal((5, 3, 32))
    w = 1 + 0.2 * rng.standard_normal(32) if weighted else None
    ang = oa.angles(rng.integers(0, 999, (2, 5)), rng.standard_normal((2, rot // 2)))
    dx, dw = oa.norm_rope_vjp(x, w, ang, pairing, eps, dy)
    for _ in range(3):
        d = rng.standard_normal(x.shape)
        got = _diff(lambda z: np.sum(dy * oa.norm_rope(z, w, ang, pairing, eps)), x, d)
        assert abs(got - np.sum(dx * d)) <= 1e-7 * (1 + abs(got))
    if weighted:
        d = rng.standard_normal(32)
        got = _diff(lambda z: np.sum(dy * oa.norm_rope(x, z, ang, pairing, eps)), w, d)
        assert abs(got - np.sum(dw * d)) <= 1e-7 * (1 + abs(got))


def test_rotation_keeps_lengths_and_depends_on_differences():
    rng = np.random.default_rng(4)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    freq = rng.standard_normal((1, 8))

    def dot(a, b):
        return np.sum(oa.turn(q, oa.angles([[a]], freq), "pairs") *
                      oa.turn(k, oa.angles([[b]], freq), "pairs"))
    assert abs(dot(7, 3) - dot(104, 100)) < 1e-9
    y = oa.turn(q, oa.angles([[12345]], freq), "halves")
    assert abs(np.sum(y * y) - np.sum(q * q)) < 1e-9


@pytest.mark.parametrize("mode,window", [("sliding", 4), ("sliding", 1), ("block", 5), ("block", 50)])
def test_window_gradients_against_differences(mode, window):
    rng = np.random.default_rng(5)
    Q, K, V, dO = (rng.standard_normal((11, 8)) for _ in range(4))
    grads = oa.window_attention_vjp(Q, K, V, dO, window, mode)
    for i in range(3):
        d = rng.standard_normal(Q.shape)

        def f(x):
            a = [Q, K, V]
            a[i] = x
            return np.sum(dO * blk.window_attention(*a, window, mode))
        got = _diff(f, (Q, K, V)[i], d)
        assert abs(got - np.sum(grads[i] * d)) <= 1e-7 * (1 + abs(got))


def test_window_lse_of_one_token_is_its_score():
    rng = np.random.default_rng(6)
    Q, K = rng.standard_normal((6, 8)), rng.standard_normal((6, 8))
    assert np.allclose(oa.window_lse(Q, K, 1, "sliding"), np.sum(Q * K, 1) / np.sqrt(8))


def test_paged_attention_is_the_window_attentions_last_row():
    rng = np.random.default_rng(7)
    T, D, size = 13, 16, 4
    Q, K, V = (rng.standard_normal((T, D)) for _ in range(3))
    table = np.array([[2, 0, 3, 1]])
    kc, vc = np.full((4, 1, size, D), np.nan), np.full((4, 1, size, D), np.nan)
    for t in range(T):
        kc[table[0, t // size], 0, t % size], vc[table[0, t // size], 0, t % size] = K[t], V[t]
    for window in (0, 1, 5, 40):
        out, lse = oa.paged_attention(Q[-1][None, None], kc, vc, table, [T], window, 1 / np.sqrt(D))
        ref = blk.window_attention(Q, K, V, window or T, "sliding")[-1]
        assert np.allclose(out[0, 0], ref)
        assert np.allclose(lse[0, 0], oa.window_lse(Q, K, window or T, "sliding")[-1])


def test_paged_attention_leaves_out_bad_pages_and_empty_sequences():
    rng = np.random.default_rng(8)
    q, kc, vc = rng.standard_normal((3, 2, 4)), rng.standard_normal((2, 1, 3, 4)), rng.standard_normal((2, 1, 3, 4))
    table = np.array([[1, 7], [-1, 2], [0, 1]])
    out, lse = oa.paged_attention(q, kc, vc, table, [5, 6, -2], 0, 0.5)
    z = 0.5 * kc[1, 0] @ q[0, 0]
    assert np.allclose(out[0, 0], np.exp(z) @ vc[1, 0] / np.exp(z).sum())
    assert np.all(out[1:] == 0) and np.all(lse[1:] == -np.inf)


def test_e4m3_rounding():
    assert list(oa.e4m3([0, 1, 17, 25, 26, 449, -1e9, 2.0 ** -10, 1.5 * 2.0 ** -9, 3e-3])) == [
        0, 1, 16, 24, 26, 448, -448, 0, 2.0 ** -8, 2.0 ** -8]
