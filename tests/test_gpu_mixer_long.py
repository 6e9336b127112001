"""Linear attention (include/ttt_mixer.h) over long memories, and over rows that the last-level cache cannot keep."""
import numpy as np
import pytest
import torch

import mixer_bars as bars
import weight_sequence_layers_amd as W
from test_gpu_mixer import BF, DEV, Linear, gen, np64, say, worst

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("power,T,lens", [(12, 32768, 1), (16, 131072, 1), (16, 131072, 0)])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_linear_attention_of_a_long_memory(power, T, lens, K, V):
    """Keys of 0: the last state is decay^T times the first, and so is the gradient of the first of the last's.
    Each chunk rounds the state's product with the decay's power once, up or down alike for states that are
    not the same: n chunks move the mean of N elements by 6 U sqrt(n / N) at most (six standard deviations of U
    / sqrt(3) each, with room); the powers together, and a join of segments, are off by no more than 4 U on
    top.  One sequence among empty ones (a batch of more workgroups than run at once, so that it is not cut),
    and one alone, which is."""
    a = np.float32(1 - 2.0 ** -power)
    heads, B = 2, 600 if lens else 1
    say(f"long memory 1 - 2^-{power} T={T} B={B} K={K} V={V}")
    cfg = W.make_linear_attention_config(heads=heads, dim_k=K, dim_v=V)
    x = torch.zeros(T, heads * max(K, V), dtype=BF, device=DEV)
    out, ld = torch.empty_like(x), x.stride(0)
    starts = torch.tensor([0] * B + [T], dtype=torch.int32, device=DEV)
    decay = torch.full((heads,), float(a), device=DEV)
    s = 1 + torch.rand(B, heads, K, V, generator=gen(1), device=DEV)
    so, work = torch.empty_like(s), torch.empty(W.ttt_linear_attention_work(cfg, B, T), dtype=torch.uint8, device=DEV)
    assert (len(work) == 0) == bool(lens)
    W.ttt_linear_attention(cfg, x, ld, x, ld, x, ld, decay, starts, s, so, None, out, ld, T, B, T, work)
    torch.cuda.synchronize()
    want = float(a) ** T * np64(s[B - 1])
    e = np.mean((np64(so[B - 1]) - want) / want)
    n, N = T / 64, heads * K * V
    bar = 4 * U + 6 * U * np.sqrt(n / N)
    say(f"mean error of the state {e:.2e} (bar {bar:.2e})")
    assert abs(e) <= bar
    assert torch.equal(so[:B - 1], s[:B - 1])
    g = [torch.empty_like(x) for _ in range(3)]
    work = torch.empty(W.ttt_linear_attention_backward_work(cfg, B, T), dtype=torch.uint8, device=DEV)
    W.ttt_linear_attention_backward(cfg, x, ld, x, ld, x, ld, decay, starts, None, x, ld, s, g[0], ld, g[1], ld, g[2], ld, so,
                                    T, B, T, work)
    torch.cuda.synchronize()
    e = np.mean((np64(so[B - 1]) - want) / want)
    say(f"mean error of its gradient {e:.2e}")
    assert abs(e) <= bar
    assert torch.equal(so[:B - 1], s[:B - 1])


def test_linear_attention_past_the_last_level_cache():
    """11100 tokens of 64 heads of 64 (273 MB of rows), two ragged sequences of many chunks: forward, and backward in
    time, against the oracle at three of the heads."""
    c = Linear(lens=[9001, 2099], heads=64, K=64, V=64, pad=0, decay=[0.9, 0.99, 1.0, 0.999])
    assert 2 * c.rows * c.ld > 1 << 28
    sin, ds = c.states(), c.states(3)
    sout, dsin = torch.full_like(sin, 7.0), torch.full_like(ds, 7.0)
    dout = torch.randn(c.rows, 64 * 64, generator=gen(5), device=DEV).to(BF)
    out, grads = c.call(sin, sout), c.back(dout, sin, ds, dsin)
    torch.cuda.synchronize()
    assert c.kept(out, 64) and all(c.kept(g, 64) for g in grads)
    for i in range(2):
        for h in (0, 31, 63):
            ops = (*c.qkv(i, h), c.lam(h), np64(sin[i, h]), c.scale)
            (o, bar), state = bars.forward(*ops)
            assert worst(c.part(out, i, h, 64), o, bar) <= 1 and worst(np64(sout[i, h]), *state) <= 1, (i, h)
            ref = bars.backward(*ops, c.part(dout, i, h, 64), np64(ds[i, h]))
            for x, (y, bar) in zip(grads, ref):
                assert worst(c.part(x, i, h, 64), y, bar) <= 1, (i, h)
            assert worst(np64(dsin[i, h]), *ref[3]) <= 1, (i, h)
