"""The norms' backward (include/ttt_mixer.h) over more rows than the workgroups of a launch take at once."""
import pytest
import torch

import weight_sequence_layers_amd as W
from test_gpu_mixer import BF, DEV, Norm, gen, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# 768 workgroups of 256 / lanes rows up to rows of 2048 elements, 512 and 256 of one row beyond; the last round not
# full, with 1 to 3 sums over each row
ROUNDS = [
    dict(T=768 * 32 * 2 + 9, D=64, groups=4, kind="silu"), dict(T=768 * 4 + 1, D=512, act="f32", norm_y=False),
    dict(T=768 * 2 * 2 + 1, D=1024, kind="silu"), dict(T=768 * 2 + 1, D=1024, act="f32", groups=8, kind="sigmoid"),
    dict(T=2 * 768 + 5, D=2048, act="f32", kind="sigmoid"), dict(T=3 * 768 + 2, D=2048, n=False),
    dict(T=3 * 384 + 7, D=4096, kind="silu"), dict(T=384 + 1, D=2056, act="f32"),
    dict(T=2 * 512 + 3, D=2056, act="f32", groups=257), dict(T=512 + 1, D=4096, kind="sigmoid"),
    dict(T=3 * 256 + 1, D=8192), dict(T=2 * 256 + 3, D=4104, act="f32", kind="silu"),
]


@pytest.mark.parametrize("kw", ROUNDS)
def test_residual_norm_backward_of_several_rounds(kw):
    c = Norm(**kw)
    c.check_back(*c.back())


def integers(T, D, seed, low=-8, high=9):
    return torch.randint(low, high, (T, D), generator=gen(seed), device=DEV).float()


@pytest.mark.parametrize("T,D", [(768 * 256 * 3 + 77, 8), (768 * 32 * 3 + 5, 64), (768 * 2 * 5 + 1, 1024),
                                 (768 * 3 + 2, 2048), (384 * 70 + 3, 2056), (512 * 66 + 3, 2056), (256 * 65 + 1, 4104)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_residual_norm_backward_adds_up_every_row(T, D, act):
    """Sums of small whole numbers: exact in 32 bits in any order, so that no row may be lost or taken twice.
    Rows of +-1 have the norm 1 / sqrt(1 + eps), which is 1 for an eps of 1e-30."""
    say(f"whole numbers T={T} D={D} {act}")
    dt = BF if act == "bf16" else torch.float32
    y = (2 * integers(T, D, 1, 0, 2) - 1).to(dt)
    d, one = integers(T, D, 2).to(dt), torch.ones(D, dtype=dt, device=DEV)
    dy, sums = torch.empty_like(y), torch.zeros(3, D, device=DEV)
    want = (d.float() * y.float()).double().sum(0)
    cfg = W.make_residual_norm_config(dim=D, norm_y=True, act=act, eps=1e-30)
    work = torch.empty(W.ttt_residual_norm_backward_work(cfg, T), dtype=torch.uint8, device=DEV)
    W.ttt_residual_norm_backward(cfg, None, 0, y, D, None, 0, one, one, None, d, D, None, 0, None, 0, dy, D, None, 0,
                                 sums[0], sums[1], None, work, T)
    cfg = W.make_residual_norm_config(dim=D, act=act, eps=1e-30)
    W.ttt_residual_norm_backward(cfg, None, 0, y, D, None, 0, None, None, one, None, 0, d, D, None, 0, dy, D, None, 0,
                                 None, None, sums[2], work, T)
    torch.cuda.synchronize()
    assert all(torch.equal(s.double(), want) for s in sums)


@pytest.mark.parametrize("T,D", [(768 * 1024 + 5, 1032), (384 * 1024 + 5, 2056)])
def test_residual_norm_backward_of_equal_rows(T, D):
    """Equal terms, which a long sum in 32 bits rounds to one side at every addition: 1 + 2^-15 - 2^-20 added to a sum
    between 512 and 1024, whose numbers are 2^-14 apart, adds 1.  The sums are chains of at most 64 additions (64 U),
    what joins them (U) and one rounding at the end."""
    say(f"equal rows T={T} D={D}")
    c = 1 + 2.0 ** -15 - 2.0 ** -20
    y, d, one = (torch.full(s, x, device=DEV) for s, x in (((T, D), 1.0), ((T, D), c), ((D,), 1.0)))
    cfg = W.make_residual_norm_config(dim=D, act="f32")
    work = torch.empty(W.ttt_residual_norm_backward_work(cfg, T), dtype=torch.uint8, device=DEV)
    got = torch.empty(D, device=DEV)
    dy = torch.empty(T, D, device=DEV)
    W.ttt_residual_norm_backward(cfg, None, 0, y, D, None, 0, None, one, None, d, D, None, 0, None, 0, dy, D, None, 0, None,
                                 got, None, work, T)
    torch.cuda.synchronize()
    e = float(((got.double() - T * c) / (T * c)).abs().max())
    assert e <= 66 * U, e


def test_residual_norm_backward_of_several_launches_captured():
    """Rows past 64 to a workgroup go into launches of their own: replayed with other rows beside the same eager call on
    another stream; work between the calls holds anything."""
    c = Norm(T=256 * 64 * 2 + 9, D=4104, kind="silu", pad=0)
    n = W.ttt_residual_norm_backward_work(c.cfg, c.T)
    outs, eager = [c.new(0), c.new(0), c.new(0), c.sums()], [c.new(0), c.new(0), c.new(0), c.sums()]
    work, other = (torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    c.back(*outs, work=work)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        c.back(*outs, work=work)
    for i in range(3):
        c.y.copy_(torch.randn(c.y.shape, generator=gen(10 + i), device=DEV))
        for t in (*outs[:3], *outs[3], *eager[:3], *eager[3]):
            t.fill_(7.0)
        work.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            c.back(*eager, work=other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*outs[:3], *outs[3]), (*eager[:3], *eager[3])))
