"""Plain fp64 CPU oracle of the attention calls (include/ttt_attention.h).

TEST INFRASTRUCTURE. Only the tests may import or run this module. It shares no code with the
HIP library.

The TTT-E2E page trains its window attention with normalised queries
and keys and rotary positions; the formulas here are the header's:
* per-head norm n = x / sqrt(mean(x^2) + eps) * w, pairs turned by sum_a pos_a freq_a,j;
* the backward of both, as formulas;
* a paged cache (dict of page, head, place), attention of one token over it;
* the window attention's log-sum-exp and gradients.
"""
from __future__ import annotations

import numpy as np

from oracle.ttt_block import window_mask


def angles(pos, freq):
    """[tokens, rot / 2] from pos [axes, tokens] and freq [axes, rot / 2]."""
    return np.asarray(pos, np.float64).T @ np.asarray(freq, np.float64)


def pair_index(rot: int, pairing: str):
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if pairing == "halves" else (2 * j, 2 * j + 1)


def turn(x, ang, pairing: str, sign: float = 1.0):
    """x [tokens, heads, dim] with the pairs of its first 2 * ang.shape[1] elements turned."""
    y = np.array(x, np.float64)
    i0, i1 = pair_index(2 * ang.shape[1], pairing)
    c, s = np.cos(ang)[:, None, :], sign * np.sin(ang)[:, None, :]
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i0] * s + x[..., i1] * c
    return y


def norm_rope(x, w, ang, pairing: str, eps):
    """x [tokens, heads, dim]; w [dim] or None; eps None: no norm."""
    x = np.asarray(x, np.float64)
    if eps is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if w is not None:
            x = x * w
    return turn(x, ang, pairing)


def norm_rope_vjp(x, w, ang, pairing: str, eps, dy):
    """(dx, dw) of sum <dy, norm_rope(x)>; dw None without norm."""
    x, g = np.asarray(x, np.float64), turn(np.asarray(dy, np.float64), ang, pairing, -1.0)
    if eps is None:
        return g, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xh = x * r
    u = g if w is None else g * w
    return r * (u - xh * np.mean(u * xh, axis=-1, keepdims=True)), np.sum(g * xh, axis=(0, 1))


def seen_tokens(length: int, window: int, limit: int):
    """First and past-the-last cached token that the new token sees."""
    n = min(max(int(length), 0), limit)
    return (max(0, n - window) if window else 0), n


def paged_attention(q, k_cache, v_cache, table, lens, window: int, scale: float):
    """q [seqs, heads, dim]; caches [pages, kv_heads, page_size, dim] of values; table
    [seqs, max_pages]. Returns (out, lse)."""
    S, H, D = q.shape
    P, Hk, size, _ = k_cache.shape
    out, lse = np.zeros((S, H, D)), np.full((S, H), -np.inf)
    for s in range(S):
        lo, n = seen_tokens(lens[s], window, table.shape[1] * size)
        rows = [(int(table[s, j // size]), j % size) for j in range(lo, n)]
        rows = [(p, i) for p, i in rows if 0 <= p < P]
        if not rows:
            continue
        p, i = (np.array(x) for x in zip(*rows))
        for h in range(H):
            kk, vv = k_cache[p, h * Hk // H, i], v_cache[p, h * Hk // H, i]
            z = scale * (kk @ q[s, h])
            m = z.max()
            e = np.exp(z - m)
            lse[s, h] = m + np.log(e.sum())
            out[s, h] = (e / e.sum()) @ vv
    return out, lse


def window_lse(Q, K, window: int, mode: str):
    """log sum exp of each row's scaled scores for one head."""
    z = np.where(window_mask(len(Q), window, mode), Q @ K.T / np.sqrt(Q.shape[1]), -np.inf)
    m = z.max(axis=1)
    return m + np.log(np.exp(z - m[:, None]).sum(axis=1))


def window_probs(Q, K, window: int, mode: str):
    z = np.where(window_mask(len(Q), window, mode), Q @ K.T / np.sqrt(Q.shape[1]), -np.inf)
    e = np.exp(z - z.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def window_attention_vjp(Q, K, V, dO, window: int, mode: str):
    """(dQ, dK, dV) of sum <dO, window_attention(Q, K, V)> for one head."""
    P = window_probs(Q, K, window, mode)
    dP = dO @ V.T
    dS = P * (dP - np.sum(P * dP, axis=1, keepdims=True)) / np.sqrt(Q.shape[1])
    return dS @ K, dS.T @ Q, P.T @ dO


def e4m3(x):
    """Nearest e4m3 value (ties to even), values past 448 held there."""
    x = np.clip(np.asarray(x, np.float64), -448, 448)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.round(x / step) * step
