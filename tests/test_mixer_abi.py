"""The mixer calls reject bad arguments on the host before any HIP call, their workspace sizes and index rules
hold, and the binding refuses tensors that would be misread (no compute call is made here)."""
import ctypes
import os
import subprocess

import pytest
import torch

import weight_sequence_layers_amd as W
import weight_sequence_layers_amd.build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20   # pointers that no call reads here


def P(i, off=0):
    return ctypes.c_void_p(A * (i + 1) * 64 + off)


def lin(heads=2, dim_k=64, dim_v=128, scale=0.0):
    return W.ttt_linear_attention_config(heads, dim_k, dim_v, scale)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(heads=0), 2), (dict(heads=4097), 2), (dict(dim_k=32), 5), (dict(dim_v=96), 5), (dict(dim_k=512), 5),
    (dict(scale=-1.0), 4), (dict(scale=float("nan")), 4), (dict(scale=float("inf")), 4), (dict(scale=2.0), 0),
    (dict(dim_k=256, dim_v=256), 0)])
def test_linear_config(kw, code):
    assert W.lib().ttt_validate_linear_attention_config(ctypes.byref(lin(**kw))) == code
    if code:
        with pytest.raises(W.TTTError) as e:
            W.ttt_validate_linear_attention_config(lin(**kw))
        assert e.value.status == code and len(str(e.value)) > 12
    assert ctypes.sizeof(W.ttt_linear_attention_config) == 16


def forward(cfg=None, **kw):
    a = dict(q=P(0), ld_q=128, k=P(1), ld_k=128, v=P(2), ld_v=256, decay=P(3), starts=P(4), sin=P(5), sout=P(6), slot=P(7),
             slots=4, out=P(8), ld_out=256, tokens=100, batch=3, seq_len=40, work=P(9), bytes=1 << 40)
    a.update(kw)
    return W.lib().ttt_linear_attention(ctypes.byref(cfg or lin()), *a.values(), None)


BAD = [(dict(batch=-1), 2), (dict(batch=65536), 2), (dict(seq_len=-1), 2), (dict(seq_len=(1 << 30) + 1), 2),
       (dict(tokens=-1), 2), (dict(tokens=1 << 31), 2), (dict(starts=None), 2), (dict(ld_q=120), 2), (dict(ld_k=132), 2),
       (dict(ld_v=128), 2), (dict(ld_v=1 << 24), 2), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
       (dict(decay=None), 1), (dict(q=P(0, 8)), 9), (dict(decay=P(3, 4)), 9), (dict(starts=P(4, 4)), 9),
       (dict(batch=0, q=None), 0)]


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(ld_out=128), 2), (dict(out=None), 1), (dict(slots=-1), 2), (dict(slot=None, slots=2), 2), (dict(slot=P(7, 4)), 9),
    (dict(sin=P(5, 8)), 9), (dict(out=P(0)), 4), (dict(out=P(2)), 4), (dict(sout=P(0)), 4), (dict(sout=P(5, 16)), 4),
    (dict(sout=P(8)), 4), (dict(out=P(5)), 4), (dict(sout=P(3)), 4), (dict(out=P(4)), 4), (dict(sout=P(7)), 4),
    (dict(seq_len=100000, work=None), 1), (dict(seq_len=100000, bytes=64), 2), (dict(seq_len=100000, work=P(5)), 4),
    (dict(seq_len=100000, work=P(0)), 4),
])
def test_linear_arguments(kw, code):
    assert forward(**kw) == code, W.lib().ttt_last_error()


def test_linear_sizes_of_many_heads():
    assert forward(lin(heads=4096), ld_q=4096 * 64, ld_k=4096 * 64, ld_v=4096 * 128, ld_out=4096 * 128, batch=300) == 2


def backward(cfg=None, **kw):
    a = dict(q=P(0), ld_q=128, k=P(1), ld_k=128, v=P(2), ld_v=256, decay=P(3), starts=P(4), sin=P(5), dout=P(6), ld_dout=256,
             ds=P(7), dq=P(8), ld_dq=128, dk=P(9), ld_dk=128, dv=P(10), ld_dv=256, dsin=P(11), tokens=100, batch=3,
             seq_len=40, work=P(12), bytes=1 << 40)
    a.update(kw)
    return W.lib().ttt_linear_attention_backward(ctypes.byref(cfg or lin()), *a.values(), None)


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(ld_dout=128), 2), (dict(ld_dq=64), 2), (dict(ld_dk=64), 2), (dict(ld_dv=128), 2), (dict(dout=None), 1),
    (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(dsin=P(11, 4)), 9), (dict(dq=P(0)), 4),
    (dict(dk=P(8)), 4), (dict(dv=P(6)), 4), (dict(dsin=P(7)), 4), (dict(dsin=P(5)), 4), (dict(dsin=P(8)), 4),
    (dict(seq_len=100000, work=None), 1), (dict(seq_len=100000, bytes=64), 2), (dict(seq_len=100000, work=P(10)), 4),
])
def test_linear_backward_arguments(kw, code):
    assert backward(**kw) == code, W.lib().ttt_last_error()


def step(cfg=None, **kw):
    a = dict(q=P(0), ld_q=128, k=P(1), ld_k=128, v=P(2), ld_v=256, decay=P(3), sin=P(5), sout=P(6), slot=P(7), slots=4,
             out=P(8), ld_out=256, seqs=3)
    a.update(kw)
    return W.lib().ttt_linear_attention_step(ctypes.byref(cfg or lin()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(seqs=-1), 2), (dict(seqs=(1 << 20) + 1), 2), (dict(ld_q=64), 2), (dict(ld_out=130), 2), (dict(slots=-1), 2),
    (dict(slot=None, slots=2), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(decay=None), 1), (dict(slot=P(7, 4)), 9),
    (dict(sout=P(6, 4)), 9), (dict(out=P(1)), 4), (dict(sout=P(2)), 4), (dict(sout=P(5, 16)), 4), (dict(out=P(5)), 4),
    (dict(out=P(6)), 4), (dict(seqs=0, q=None), 0)])
def test_linear_step_arguments(kw, code):
    assert step(**kw) == code, W.lib().ttt_last_error()


def test_linear_step_sizes_of_many_heads():
    assert step(lin(heads=4096), ld_q=4096 * 64, ld_k=4096 * 64, ld_v=4096 * 128, ld_out=4096 * 128, seqs=1025) == 2


@pytest.mark.parametrize("fn", [W.ttt_linear_attention_work, W.ttt_linear_attention_backward_work])
def test_linear_work(fn):
    for heads in (1, 8, 64):
        for batch in (0, 1, 7, 1000):
            for T in (0, 1, 255, 256, 5000, 1 << 20, 1 << 30):
                c = W.make_linear_attention_config(heads=heads, dim_k=128)
                n = fn(c, batch, T)
                assert 0 <= n <= 1 << 29
                if batch == 0 or T < 256:
                    assert n == 0
    for bad in ((-1, 5), (5, -1), (5, (1 << 30) + 1)):
        with pytest.raises(W.TTTError):
            fn(lin(), *bad)
    with pytest.raises(W.TTTError):
        fn(lin(), 1 << 32, 5)
    assert W.lib().ttt_linear_attention_work(ctypes.byref(lin()), 1, 1, None) == 1


def norm(**kw):
    a = dict(dim=64, groups=1, norm_y=1, gate=1, act=1, eps=1e-6)
    a.update(kw)
    return W.ttt_residual_norm_config(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(dim=0), 2), (dict(dim=12), 2), (dict(dim=8200), 2), (dict(dim=8192), 0), (dict(groups=0), 2),
    (dict(groups=3), 2), (dict(groups=16), 2), (dict(groups=8), 0), (dict(dim=96, groups=2), 2), (dict(dim=2048, groups=2), 2),
    (dict(dim=96, groups=3), 0), (dict(dim=96), 0), (dict(norm_y=2), 4), (dict(norm_y=-1), 4), (dict(gate=3), 4),
    (dict(gate=-1), 4), (dict(act=2), 3), (dict(eps=0.0), 4), (dict(eps=float("inf")), 4), (dict(eps=float("nan")), 4)])
def test_norm_config(kw, code):
    assert W.lib().ttt_validate_residual_norm_config(ctypes.byref(norm(**kw))) == code
    if code:
        with pytest.raises(W.TTTError) as e:
            W.ttt_validate_residual_norm_config(norm(**kw))
        assert e.value.status == code and len(str(e.value)) > 12
    assert ctypes.sizeof(W.ttt_residual_norm_config) == 24


def rnorm(cfg=None, **kw):
    a = dict(h=P(0), ld_h=64, y=P(1), ld_y=64, g=P(2), ld_g=64, wy=P(3), rs=P(4), wn=P(5), ho=P(6), ld_ho=64, n=P(7), ld_n=64,
             tokens=10)
    a.update(kw)
    return W.lib().ttt_residual_norm(ctypes.byref(cfg or norm()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(tokens=(1 << 25) + 1), 2), (dict(ld_h=56), 2), (dict(ld_y=68), 2), (dict(ld_n=(1 << 28) + 8), 2),
    (dict(y=None), 1), (dict(g=None), 1), (dict(ho=None, n=None, wn=None), 1), (dict(n=None), 4), (dict(y=P(1, 8)), 9),
    (dict(wy=P(3, 2)), 9), (dict(ho=P(0, 16)), 4), (dict(ho=P(0), ld_ho=72), 4), (dict(n=P(6)), 4), (dict(n=P(3)), 4),
    (dict(ho=P(5)), 4), (dict(tokens=0, y=None, g=None, ho=None, n=None, wn=None), 0)])
def test_norm_arguments(kw, code):
    assert rnorm(**kw) == code, W.lib().ttt_last_error()


def test_norm_parts_that_the_configuration_lacks():
    assert rnorm(norm(gate=0)) == 4
    assert rnorm(norm(norm_y=0)) == 4


def nback(cfg=None, **kw):
    a = dict(h=P(0), ld_h=64, y=P(1), ld_y=64, g=P(2), ld_g=64, wy=P(3), rs=P(4), wn=P(5), dho=P(6), ld_dho=64, dn=P(7), ld_dn=64,
             dh=P(8), ld_dh=64, dy=P(9), ld_dy=64, dg=P(10), ld_dg=64, dwy=P(11), drs=P(12), dwn=P(13), work=P(14),
             bytes=1 << 30, tokens=10)
    a.update(kw)
    return W.lib().ttt_residual_norm_backward(ctypes.byref(cfg or norm()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(ld_dho=8), 2), (dict(ld_dn=8), 2), (dict(ld_dh=8), 2), (dict(ld_dy=8), 2), (dict(ld_dg=8), 2),
    (dict(y=None), 1), (dict(g=None), 1), (dict(dho=None, dn=None, wn=None, dwn=None), 1), (dict(dn=None), 4),
    (dict(h=None), 4), (dict(wy=None), 4), (dict(rs=None), 4), (dict(wn=None), 4), (dict(work=None), 1), (dict(bytes=8), 2),
    (dict(dwy=P(11, 4)), 9), (dict(dh=P(0)), 4), (dict(dy=P(1)), 4), (dict(dg=P(2)), 4), (dict(dy=P(8)), 4),
    (dict(dh=P(6), ld_dh=72), 4), (dict(dwy=P(6)), 4), (dict(work=P(7)), 4), (dict(work=P(9)), 4), (dict(dwn=P(5)), 4),
    (dict(drs=P(11)), 4)])
def test_norm_backward_arguments(kw, code):
    assert nback(**kw) == code, W.lib().ttt_last_error()


def test_norm_backward_parts_that_the_configuration_lacks():
    assert nback(norm(gate=0), g=None) == 4
    assert nback(norm(norm_y=0)) == 4


def test_norm_backward_work():
    for dim in (8, 768, 2048, 2056, 8192):
        sizes = [W.ttt_residual_norm_backward_work(norm(dim=dim), t) for t in (0, 1, 100, 1 << 25)]
        assert sizes[0] == 0 and sizes == sorted(sizes) and sizes[1] >= 12 * dim and sizes[-1] <= 1 << 27
    for bad in (-1, (1 << 25) + 1):
        with pytest.raises(W.TTTError):
            W.ttt_residual_norm_backward_work(norm(), bad)
    assert W.lib().ttt_residual_norm_backward_work(ctypes.byref(norm()), 1, None) == 1


# ------------------------------------------------------------------------ the binding
BIG = (1 << 32) + 4


@pytest.mark.parametrize("field", ["heads", "dim_k", "dim_v"])
def test_linear_config_numbers_past_32_bits_are_refused(field):
    with pytest.raises(W.TTTError) as e:
        W.make_linear_attention_config(**{**dict(heads=2, dim_k=64, dim_v=64), field: BIG})
    assert e.value.status == 2


def test_other_numbers_past_32_bits_are_refused():
    c = W.make_linear_attention_config(heads=2, dim_k=64)
    n = None
    for call in (lambda: W.make_residual_norm_config(dim=BIG), lambda: W.make_residual_norm_config(dim=64, groups=BIG),
                 lambda: W.ttt_linear_attention(c, n, 128, n, 128, n, 128, n, n, n, n, n, n, 128, 5, BIG, 5, n),
                 lambda: W.ttt_linear_attention_backward(c, n, 128, n, 128, n, 128, n, n, n, n, 128, n, n, 128, n, 128, n, 128, n,
                                                         5, BIG, 5, n),
                 lambda: W.ttt_linear_attention_step(c, n, 128, n, 128, n, 128, n, n, n, n, n, 128, BIG)):
        with pytest.raises(W.TTTError) as e:
            call()
        assert e.value.status == 2 and "2^31" in str(e.value)
    for scale in (1e-50, -1e-300):
        with pytest.raises(W.TTTError) as e:
            W.make_linear_attention_config(heads=2, dim_k=64, scale=scale)
        assert e.value.status == 4


@pytest.mark.parametrize("shape,ok", [
    ((5, 2, 64, 128), True), ((0, 2, 64, 128), True), ((5, 2, 128, 64), False), ((5, 3, 64, 128), False), ((2, 64, 128), False),
    ((10, 64, 128), False), ((1, 5, 2, 64, 128), False)])
def test_pools_of_another_shape_are_refused(shape, ok):
    t = torch.zeros(shape)
    if ok:
        assert W._pool(t, "state", lin(), -1, torch) == (t.data_ptr(), shape[0])
    else:
        with pytest.raises(W.TTTError) as e:
            W._pool(t, "state", lin(), -1, torch)
        assert e.value.status == 2


def test_pools_that_are_not_dense_or_of_another_type_or_number_are_refused():
    for t, code in ((torch.zeros(5, 2, 128, 64).transpose(2, 3), 2), (torch.zeros(5, 2, 64, 128, dtype=torch.bfloat16), 3),
                    (torch.zeros(10, 2, 64, 128)[::2], 2)):
        with pytest.raises(W.TTTError) as e:
            W._pool(t, "state", lin(), -1, torch)
        assert e.value.status == code
    with pytest.raises(W.TTTError):
        W._pools(torch.zeros(5, 2, 64, 128), torch.zeros(4, 2, 64, 128), lin(), -1, torch)
    assert W._pools(None, None, lin(), -1, torch) == (None, None, 0)


def test_mixer_index_rules(tmp_path):
    """Spans of sequences and entries of pools for numbers that no sane program passes."""
    src = tmp_path / "index.cpp"
    src.write_text(r'''
#include <hip/hip_runtime.h>
#include <cstdio>
#include <cstdlib>
#include "ttt_mixer_internal.h"
using namespace ttt;
#define CHECK(x) do { if (!(x)) { printf("line %d\n", __LINE__); exit(1); } } while (0)
int main() {
  const int32_t lo = INT32_MIN, hi = INT32_MAX;
  const int32_t starts[] = {lo, -1, 0, 5, 5, 3, 40, 100, 101, hi, lo, hi};
  for (int64_t tokens : {(int64_t)0, (int64_t)1, (int64_t)100, (int64_t)hi})
    for (int32_t T : {0, 1, 30, 1 << 30})
      for (int b = 0; b < 11; ++b) {
        int64_t row0; int32_t len;
        lin_span(starts, b, tokens, T, row0, len);
        CHECK(row0 >= 0 && row0 <= tokens && len >= 0 && len <= T && row0 + len <= tokens);
        if (starts[b + 1] <= starts[b]) CHECK(len == 0);
      }
  int64_t row0; int32_t len;
  lin_span(starts, 5, 100, 1000, row0, len);
  CHECK(row0 == 3 && len == 37);
  lin_span(nullptr, 65534, 0, 1 << 30, row0, len);
  CHECK(row0 == (int64_t)65534 << 30 && len == 1 << 30);
  for (int32_t i : starts)
    for (int32_t slots : {0, 1, 6, hi}) {
      const int64_t s = lin_slot(&i, 0, slots);
      CHECK(s == -1 || (s == i && s >= 0 && s < slots));
      if (i >= 0 && i < slots) CHECK(s == i);
    }
  CHECK(lin_slot(nullptr, 3, 4) == 3 && lin_slot(nullptr, 4, 4) == -1);
  return 0;
}
''')
    _run_host(src, tmp_path)


def test_norm_launches_of_many_rows(tmp_path):
    """A launch has fewer than 2^32 threads, and the launches that follow one another have the rows in turn."""
    src = tmp_path / "index.cpp"
    src.write_text(r'''
#include <hip/hip_runtime.h>
#include <cstdio>
#include <cstdlib>
#include "ttt_mixer_internal.h"
using namespace ttt;
#define CHECK(x) do { if (!(x)) { printf("line %d\n", __LINE__); exit(1); } } while (0)
int main() {
  CHECK(NORM_LAUNCH * 1024 < (int64_t)1 << 32);
  NormArgs a = {};
  a.y = (const void*)4096; a.ldy = 1 << 20;
  a.n = (void*)8192; a.ldn = 8;
  a.tokens = (1 << 25) - 3;
  int64_t rows = 0;
  for (int64_t first = 0; first < a.tokens; first += 1 << 20) {
    const NormArgs p = norm_part(a, first, 1 << 20, 2);
    CHECK(!p.h && !p.gate && !p.ho && p.tokens > 0 && p.tokens <= 1 << 20);
    CHECK((int64_t)p.y == 4096 + (first << 21) && (int64_t)p.n == 8192 + first * 16 && p.ldy == a.ldy);
    rows += p.tokens;
  }
  CHECK(rows == a.tokens);
  return 0;
}
''')
    _run_host(src, tmp_path)


def _run_host(src, tmp_path):
    exe = tmp_path / "index"
    r = subprocess.run([B.HIPCC, "--offload-arch=gfx950", "-std=c++17", "-w", "-x", "hip", str(src), "-I" + os.path.join(ROOT, "include"),
                        "-I" + B.CSRC, "-o", str(exe)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert r.returncode == 0, r.stdout
