"""Plain fp64 CPU oracle of the mixer calls (include/ttt_mixer.h).

TEST INFRASTRUCTURE. Only the tests may import or run this module. It shares no code with the
HIP library. Everything is written token by token from the header's formulas, for one head of one
sequence (linear attention) or for a matrix of rows (the norms).
"""
from __future__ import annotations

import numpy as np


def linear_attention(q, k, v, decay, s0, scale):
    """out [T, V] and the final state [K, V] of one head."""
    S = np.array(s0, np.float64)
    out = np.zeros((len(q), v.shape[1]))
    for t in range(len(q)):
        S = decay * S + np.outer(k[t], v[t])
        out[t] = scale * (S.T @ q[t])
    return out, S


def linear_attention_vjp(q, k, v, decay, s0, scale, do, ds):
    """(dq, dk, dv, ds0) of sum <do, out> + <ds, final state>."""
    T = len(q)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S = np.array(s0, np.float64)
    for t in range(T):
        S = decay * S + np.outer(k[t], v[t])
        dq[t] = scale * (S @ do[t])
    P = np.array(ds, np.float64)
    for t in range(T - 1, -1, -1):
        P = P + scale * np.outer(q[t], do[t])
        dk[t], dv[t] = P @ v[t], P.T @ k[t]
        P = decay * P
    return dq, dk, dv, P


def _inv_rms(x, groups, eps):
    """1 / root mean square of each element's group."""
    g = x.reshape(len(x), groups, -1)
    r = 1 / np.sqrt(np.mean(g * g, -1, keepdims=True) + eps)
    return np.broadcast_to(r, g.shape).reshape(x.shape)


def _group_mean(x, groups):
    g = x.reshape(len(x), groups, -1)
    return np.broadcast_to(np.mean(g, -1, keepdims=True), g.shape).reshape(x.shape)


def gate_value(g, kind):
    """The gate's value and slope."""
    if kind == "none":
        return np.float64(1.0), None
    s = 1 / (1 + np.exp(-g))
    return (s, s * (1 - s)) if kind == "sigmoid" else (g * s, s + g * s * (1 - s))


def residual_norm(y, *, h=None, gate=None, wy=None, rs=None, wn=None, groups=1, norm_y=False, kind="none", eps=1e-6):
    """A dict of the values along the way: r, u, act, slope, z, h_out, p, n_out."""
    r = _inv_rms(y, groups, eps) if norm_y else np.ones_like(y)
    u = y * r * (1 if wy is None else wy)
    act, slope = gate_value(gate, kind)
    z = u * act
    h_out = (0 if h is None else h) + (1 if rs is None else rs) * z
    p = _inv_rms(h_out, 1, eps)
    return dict(r=r, u=u, act=act, slope=slope, z=z, h_out=h_out, p=p, n_out=h_out * p * (1 if wn is None else wn))


def residual_norm_vjp(y, dho, dn, *, h=None, gate=None, wy=None, rs=None, wn=None, groups=1, norm_y=False,
                      kind="none", eps=1e-6):
    """Gradients of sum <dho, h_out> + <dn, n_out>."""
    f = residual_norm(y, h=h, gate=gate, wy=wy, rs=rs, wn=wn, groups=groups, norm_y=norm_y, kind=kind, eps=eps)
    x, a = f["h_out"] * f["p"], dn * (1 if wn is None else wn)
    d = dho + f["p"] * (a - x * np.mean(a * x, -1, keepdims=True))
    dz = d * (1 if rs is None else rs)
    du = dz * f["act"]
    yr = y * f["r"]
    b = du * (1 if wy is None else wy)
    dy = f["r"] * (b - yr * _group_mean(b * yr, groups)) if norm_y else b
    return dict(dh=d, dy=dy, dgate=None if f["slope"] is None else dz * f["u"] * f["slope"],
                dwy=np.sum(du * yr, 0), drs=np.sum(d * f["z"], 0), dwn=np.sum(dn * x, 0))
