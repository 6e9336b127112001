"""The gates of the norms between sub-layers (include/ttt_mixer.h) over the whole range of their types: the
gate's value and slope against 64 bits, and whole calls with gates as masks have them."""
import numpy as np
import pytest
import torch

import oracle.ttt_mixer as om
import weight_sequence_layers_amd as W
from test_gpu_mixer import BF, DEV, H, Norm, gen, np64, say

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:overflow encountered")]
U = 2.0 ** -24
# half of the least number that the type holds besides 0
LEAST = {BF: 2.0 ** -134, torch.float32: 2.0 ** -150}


def parts(g):
    """sigmoid(g) and sigmoid(-g), each without cancellation."""
    return 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))


def stable(g, kind):
    """The oracle's gate_value with a slope that does not cancel, and silu's limit 0 at -infinity."""
    if kind == "none":
        return np.float64(1.0), None
    s, o = parts(g)
    if kind == "sigmoid":
        return s, s * o
    far = np.maximum(g, -1000.0)
    return far * s, s * (1 + np.clip(g, -1000.0, 1000.0) * o)


def every_gate(act):
    """All numbers of bf16, infinities and NaN among them; in fp32 the same and as many others."""
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32)
    if act == "bf16":
        return bits.to(torch.int16).view(BF)
    low = torch.randint(0, 1 << 16, (1 << 16,), generator=gen(4), device=DEV, dtype=torch.int32)
    return torch.cat([bits << 16, (bits << 16) | low]).view(torch.float32)


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_the_gates_value_of_every_number(kind, act):
    """h_out = act(gate) of y = 1.  exp(-|g|) within 7 half steps of fp32 (the square of an exponential within
    3), the quotient 3 more, silu's product one: 12 U with the output's rounding; and, where the value is
    below the type's normal numbers, half of its least one, for silu times |g| < 110 before the product."""
    g = every_gate(act).view(-1, 64)
    say(f"gate values {kind} {act} {len(g)}")
    cfg = W.make_residual_norm_config(dim=64, gate=kind, act=act)
    out = torch.empty_like(g)
    W.ttt_residual_norm(cfg, None, 0, torch.ones_like(g), 64, g, 64, None, None, None, out, 64, None, 64, len(g))
    torch.cuda.synchronize()
    g, got = np64(g), np64(out)
    nan = np.isnan(g)
    assert np.array_equal(np.isnan(got), nan)
    g, got = g[~nan], got[~nan]
    ref = stable(g, kind)[0]
    with np.errstate(invalid="ignore"):
        bar = (H[out.dtype] + 12 * U) * np.abs(ref) + LEAST[out.dtype] + 110 * 2.0 ** -150
        e = np.where(got == ref, 0.0, np.abs(got - ref) / bar)
    assert np.max(e) <= 1, (g[np.argmax(e)], got[np.argmax(e)], ref[np.argmax(e)])


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_the_gates_slope_of_every_number(kind, act):
    """dgate of y = dh_out = 1.  s and 1 - s within 10 U each: s (1 - s) 21 U, and s + g s (1 - s) 22 U of the
    sum of its terms' sizes; the output's rounding on top, and half of the least numbers as in the value's test."""
    g = every_gate(act).view(-1, 64)
    say(f"gate slopes {kind} {act} {len(g)}")
    cfg = W.make_residual_norm_config(dim=64, gate=kind, act=act)
    out, one = torch.empty_like(g), torch.ones_like(g)
    W.ttt_residual_norm_backward(cfg, None, 0, one, 64, g, 64, None, None, None, one, 64, None, 0, None, 0, None, 0, out, 64,
                                 None, None, None, None, len(g))
    torch.cuda.synchronize()
    g, got = np64(g), np64(out)
    nan = np.isnan(g)
    assert np.array_equal(np.isnan(got), nan)
    g, got = g[~nan], got[~nan]
    ref, (s, o) = stable(g, kind)[1], parts(g)
    size = s * o if kind == "sigmoid" else s * (1 + np.clip(np.abs(g), 0, 1000) * o)
    e = np.abs(got - ref) / (H[out.dtype] * np.abs(ref) + 22 * U * size + LEAST[out.dtype] + 220 * 2.0 ** -150)
    assert np.max(e) <= 1, (g[np.argmax(e)], got[np.argmax(e)], ref[np.argmax(e)])


# one gate a row, beside ordinary ones
SMALL = [-80.0, -87.3, -88.0, -100.0, -104.0, -150.0, -1e4, -4.72e7, -1e8, -1e9, -1e10, -1e12, -1e30, -3e38, "min", "-inf"]
LARGE = [20.0, 88.0, 150.0, 1e4, 1e8, 1e12, 1e30, 2.4e38, 3e38, "max", "inf"]


def masked(kind, act, T, **kw):
    """A case whose rows have one gate of the lists each, the last row only the lowest number; and the oracle's
    arguments, infinities as numbers whose value and slope are the same."""
    c = Norm(T=T, D=256, act=act, groups=4, kind=kind, **kw)
    f = torch.finfo(c.dt)
    names = {"min": f.min, "max": f.max, "-inf": -float("inf"), "inf": float("inf")}
    for i, x in enumerate(SMALL + (LARGE if kind == "sigmoid" else [])):
        c.gate[i, 37 + i] = names.get(x, x)
    c.gate[T - 1, :256] = f.min
    args = c.kw()
    args["gate"] = np.clip(args["gate"], -1e300, 1e300)
    return c, args


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_rows_with_masked_gates(kind, act, monkeypatch):
    monkeypatch.setattr(om, "gate_value", stable)
    c, kw = masked(kind, act, 40)
    c.check(*c.call(), kw)


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_gradients_of_rows_with_masked_gates(kind, act, monkeypatch):
    """The sums over the rows among them."""
    monkeypatch.setattr(om, "gate_value", stable)
    c, kw = masked(kind, act, 40)
    monkeypatch.setattr(c, "kw", lambda: kw)
    c.check_back(*c.back())


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_gradients_of_rows_whose_squares_pass_the_range(act):
    """The norm of a row whose squares add up past fp32 is zeros, and its gradient has no part in the row's others or in
    the sums: all as with a gradient of zeros there, bit by bit."""
    c = Norm(T=30, D=256, act=act, groups=2, kind="silu")
    c.h[7, :256] = 1e38
    c.h[11, :256] = -3e37
    c.h[19, :100] = 2e19
    c.dn[[7, 11, 19]] *= 1000
    got = c.back()
    c.dn[[7, 11, 19]] = 0
    want = c.back()
    torch.cuda.synchronize()
    for a, b in zip((*got[:3], *got[3]), (*want[:3], *want[3])):
        assert bool(b.isfinite().all()) and torch.equal(a, b)
    assert bool((c.call()[1][[7, 11, 19], :256] == 0).all())
