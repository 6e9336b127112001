"""Pins of the mixer oracle: against sums written out, torch's gradients in 64 bits and differences;
and planted mistakes that exceed the error models' bars."""
import numpy as np
import pytest
import torch

import mixer_bars as bars
import oracle.ttt_mixer as om


def data(T, K, V, seed=0):
    g = np.random.default_rng(seed)
    q, k, v = g.standard_normal((T, K)), g.standard_normal((T, K)), g.standard_normal((T, V))
    return q, k, v, g.standard_normal((K, V)), g.standard_normal((T, V)), g.standard_normal((K, V))


@pytest.mark.parametrize("T", [0, 1, 7, 33, 100])
@pytest.mark.parametrize("decay", [0.0, 0.3, 0.97, 1.0])
def test_linear_attention_is_the_sum_over_earlier_tokens(T, decay):
    q, k, v, s0, do, ds = data(T, 5, 3)
    out, S = om.linear_attention(q, k, v, decay, s0, 0.7)
    for i in range(T):
        want = decay ** (i + 1) * (s0.T @ q[i]) + sum(decay ** (i - j) * (q[i] @ k[j]) * v[j] for j in range(i + 1))
        assert np.allclose(out[i], 0.7 * want, rtol=1e-12, atol=1e-12)
    want = decay ** T * s0 + sum((decay ** (T - 1 - j) * np.outer(k[j], v[j]) for j in range(T)), 0 * s0)
    assert np.allclose(S, want, rtol=1e-12, atol=1e-12)
    (o2, _), (s2, _) = bars.forward(q, k, v, decay, s0, 0.7)
    assert np.allclose(o2, out, rtol=1e-11, atol=1e-11) and np.allclose(s2, S, rtol=1e-11, atol=1e-11)
    ref = om.linear_attention_vjp(q, k, v, decay, s0, 0.7, do, ds)
    for (got, _), want in zip(bars.backward(q, k, v, decay, s0, 0.7, do, ds), ref):
        assert np.allclose(got, want, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("decay", [0.0, 0.6, 1.0])
def test_linear_attention_gradients(decay):
    q, k, v, s0, do, ds = data(9, 4, 6, 1)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, s0)]
    S, loss = t[3], 0.0
    for i in range(9):
        S = decay * S + torch.outer(t[1][i], t[2][i])
        loss = loss + 0.4 * (S.T @ t[0][i]) @ torch.tensor(do[i])
    (loss + (S * torch.tensor(ds)).sum()).backward()
    for got, x in zip(om.linear_attention_vjp(q, k, v, decay, s0, 0.4, do, ds), t):
        assert np.allclose(got, x.grad.numpy(), rtol=1e-12, atol=1e-12)


def planted(name, q, k, v, decay, s0):
    """The layer with a mistake."""
    S, out = s0.copy(), np.zeros((len(q), v.shape[1]))
    for t in range(len(q)):
        if name == "token lost" and t == 40:
            S = decay * S
        elif name == "token late":       # read before its own token is added
            out[t] = S.T @ q[t]
            S = decay * S + np.outer(k[t], v[t])
            continue
        elif name == "state not decayed over a chunk's end" and t % 32 == 0 and t:
            S = S + np.outer(k[t], v[t])
        elif name == "state in 8 bits" and t % 32 == 0:
            S = decay * np.round(S * 64) / 64 + np.outer(k[t], v[t])
        else:
            S = decay * S + np.outer(k[t], v[t])
        out[t] = S.T @ q[t]
    return out, S


@pytest.mark.parametrize("name", ["token lost", "token late", "state not decayed over a chunk's end",
                                  "state in 8 bits", "state forgotten"])
def test_planted_mistakes_exceed_the_bars(name):
    q, k, v, s0, _, _ = data(100, 16, 16, 2)
    (out, bar), (S, sbar) = bars.forward(q, k, v, 0.98, s0, 1.0)
    got, S2 = planted(name, q, k, v, 0.98, 0 * s0 if name == "state forgotten" else s0)
    assert np.max(np.abs(got - out) / bar) > 3
    if name != "token late":
        assert np.max(np.abs(S2 - S) / sbar) > 3


PARTS = [dict(), dict(norm_y=True), dict(norm_y=True, groups=4), dict(kind="sigmoid"), dict(kind="silu", norm_y=True),
         dict(kind="silu", norm_y=True, groups=2, no_h=True), dict(no_scales=True, norm_y=True, kind="sigmoid")]


def rows(parts, T=5, D=16, seed=3):
    g = np.random.default_rng(seed)
    p = dict(parts)
    no_h, no_scales = p.pop("no_h", False), p.pop("no_scales", False)
    kw = dict(h=None if no_h else g.standard_normal((T, D)),
              gate=g.standard_normal((T, D)) if p.get("kind", "none") != "none" else None,
              wy=1 + 0.2 * g.standard_normal(D) if p.get("norm_y") and not no_scales else None,
              rs=None if no_scales else 0.5 + 0.2 * g.standard_normal(D),
              wn=None if no_scales else 1 + 0.2 * g.standard_normal(D), eps=1e-3, **p)
    return g.standard_normal((T, D)), g.standard_normal((T, D)), g.standard_normal((T, D)), kw


def torch_norm(y, kw):
    def rms(x, groups):
        g = x.reshape(len(x), groups, -1)
        return (g / torch.sqrt((g * g).mean(-1, keepdim=True) + kw["eps"])).reshape(x.shape)
    u = rms(y, kw.get("groups", 1)) if kw.get("norm_y") else y
    u = u if kw["wy"] is None else u * kw["wy"]
    kind = kw.get("kind", "none")
    z = u if kind == "none" else u * (torch.sigmoid(kw["gate"]) if kind == "sigmoid" else torch.nn.functional.silu(kw["gate"]))
    z = z if kw["rs"] is None else z * kw["rs"]
    h = z if kw["h"] is None else kw["h"] + z
    n = rms(h, 1)
    return h, n if kw["wn"] is None else n * kw["wn"]


@pytest.mark.parametrize("parts", PARTS)
def test_residual_norm_and_its_gradients(parts):
    y, dho, dn, kw = rows(parts)
    t = {k: torch.tensor(x, requires_grad=True) if isinstance(x, np.ndarray) else x for k, x in kw.items()}
    ty = torch.tensor(y, requires_grad=True)
    h, n = torch_norm(ty, t)
    f = om.residual_norm(y, **kw)
    assert np.allclose(f["h_out"], h.detach().numpy(), rtol=1e-12) and np.allclose(f["n_out"], n.detach().numpy(), rtol=1e-12)
    ((h * torch.tensor(dho)).sum() + (n * torch.tensor(dn)).sum()).backward()
    got = om.residual_norm_vjp(y, dho, dn, **kw)
    for name, x in (("dy", ty), ("dh", t["h"]), ("dgate", t["gate"]), ("dwy", t["wy"]), ("drs", t["rs"]), ("dwn", t["wn"])):
        if x is not None:
            assert np.allclose(got[name], x.grad.numpy(), rtol=1e-11, atol=1e-12), name


@pytest.mark.parametrize("wrong", ["mean over the row", "no mean of the gradient", "gate's value for its slope", "a row lost",
                                   "scale left out"])
def test_planted_norm_mistakes_exceed_the_bars(wrong):
    y, dho, dn, kw = rows(dict(kind="silu", norm_y=True, groups=2), T=200, D=32)
    f, ref = om.residual_norm(y, **kw), om.residual_norm_vjp(y, dho, dn, **kw)
    bar = bars.norm_backward(f, ref, y, kw["h"], kw["gate"], kw["wy"], kw["rs"], kw["wn"], dho, dn, 2, True, bars.R)
    if wrong == "mean over the row":
        got, what = om.residual_norm_vjp(y, dho, dn, **{**kw, "groups": 1}), "dy"
    elif wrong == "no mean of the gradient":
        got, what = dict(dh=dho + f["p"] * dn * kw["wn"]), "dh"
    elif wrong == "gate's value for its slope":
        got, what = dict(dgate=ref["dgate"] / f["slope"] * f["act"]), "dgate"
    elif wrong == "a row lost":
        cut = {**kw, "h": kw["h"][1:], "gate": kw["gate"][1:]}
        got, what = om.residual_norm_vjp(y[1:], dho[1:], dn[1:], **cut), "dwn"
    else:
        got, what = om.residual_norm_vjp(y, dho, dn, **{**kw, "rs": None}), "dy"
    assert np.max(np.abs(got[what] - ref[what]) / bar[what]) > 3
