"""The attention calls reject bad arguments on the host before any HIP call, and their
workspace sizes and index rules hold (no compute call is made here)."""
import ctypes
import os
import subprocess

import pytest

import weight_sequence_layers_amd as W
import weight_sequence_layers_amd.build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20   # pointers that no call reads here


def P(i, off=0):
    return ctypes.c_void_p(A * (i + 1) * 64 + off)


def rope(**kw):
    base = dict(q_heads=4, k_heads=2, head_dim=64, rot_dim=32, axes=2)
    base.update(kw)
    return W.make_rope_config(**base)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(q_heads=0), 2), (dict(k_heads=0), 2), (dict(k_heads=4097), 2),
    (dict(head_dim=8), 2), (dict(head_dim=72), 2), (dict(head_dim=1040), 2), (dict(rot_dim=24), 2),
    (dict(rot_dim=80), 2), (dict(rot_dim=-16), 2), (dict(rot_dim=0), 0), (dict(axes=0), 2),
    (dict(axes=5), 2), (dict(pairing=2), 4), (dict(norm=2), 4), (dict(act=2), 3),
    (dict(eps=0.0), 4), (dict(eps=-1.0), 4), (dict(eps=float("nan")), 4), (dict(eps=float("inf")), 4),
    (dict(eps=0.0, norm="none"), 0), (dict(head_dim=1024, rot_dim=1024, act="f32"), 0),
])
def test_rope_config(kw, code):
    assert W.lib().ttt_validate_rope_config(ctypes.byref(rope(**kw))) == code
    if code:
        with pytest.raises(W.TTTError) as e:
            W.ttt_validate_rope_config(rope(**kw))
        assert e.value.status == code and len(str(e.value)) > 12


def test_rope_config_layout():
    assert ctypes.sizeof(W.ttt_rope_config) == 36
    assert ctypes.sizeof(W.ttt_kv_cache) == 4 * 8 + 8 + 6 * 4
    assert W.lib().ttt_validate_rope_config(None) == 1


def forward(cfg=None, **kw):
    a = dict(q=P(0), ld_q=256, k=P(1), ld_k=128, qw=P(2), kw=P(3), freq=P(4), pos=P(5), qo=P(6), ld_qo=256,
             ko=P(7), ld_ko=128, tokens=10)
    a.update(kw)
    return W.lib().ttt_qk_norm_rope(ctypes.byref(cfg or rope()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(tokens=(1 << 25) + 1), 2), (dict(tokens=1 << 31), 2), (dict(ld_q=248), 2), (dict(ld_k=127), 2),
    (dict(ld_qo=255), 2), (dict(ld_ko=132), 2), (dict(ld_q=(1 << 28) + 8), 2), (dict(q=None), 1),
    (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(freq=None), 1), (dict(pos=None), 1),
    (dict(q=P(0, 2)), 9), (dict(kw=P(3, 8)), 9), (dict(pos=P(5, 4)), 9), (dict(tokens=0, q=None), 0),
    (dict(qo=P(0), ld_qo=264), 4),          # in place with another stride
    (dict(qo=P(0, 16)), 4),                 # part of q's own rows
    (dict(qo=P(1)), 4), (dict(ko=P(0)), 4), (dict(qo=P(7)), 4),
])
def test_rope_arguments(kw, code):
    assert forward(**kw) == code, W.lib().ttt_last_error()


def test_rope_scales_need_a_norm():
    assert forward(rope(norm="none")) == 4
    assert forward(rope(norm="none"), qw=None) == 4


def backward(cfg=None, **kw):
    a = dict(q=P(0), ld_q=256, k=P(1), ld_k=128, qw=P(2), kw=P(3), freq=P(4), pos=P(5), gq=P(6), ld_gq=256,
             gk=P(7), ld_gk=128, dq=P(8), ld_dq=256, dk=P(9), ld_dk=128, dqw=P(10), dkw=P(11), work=P(12),
             bytes=1 << 30, tokens=10)
    a.update(kw)
    return W.lib().ttt_qk_norm_rope_backward(ctypes.byref(cfg or rope()), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(ld_gq=8), 2), (dict(ld_gk=8), 2), (dict(ld_dq=8), 2), (dict(ld_dk=8), 2),
    (dict(q=None), 1), (dict(gk=None), 1), (dict(dk=None), 1), (dict(work=None), 1), (dict(bytes=8), 2),
    (dict(qw=None), 4), (dict(kw=None), 4), (dict(dq=P(0)), 4), (dict(dk=P(6)), 4), (dict(dq=P(9)), 4),
    (dict(dq=P(6), ld_dq=512), 4), (dict(dqw=P(10, 4)), 9),
])
def test_rope_backward_arguments(kw, code):
    assert backward(**kw) == code, W.lib().ttt_last_error()


def test_rope_backward_work():
    assert W.ttt_qk_norm_rope_backward_work(rope(norm="none"), 100) == 0
    assert W.ttt_qk_norm_rope_backward_work(rope(), 0) == 0
    one, many = (W.ttt_qk_norm_rope_backward_work(rope(), n) for n in (1, 1 << 24))
    assert 0 < one <= many <= 1 << 24
    for bad in (-1, 1 << 31):
        with pytest.raises(W.TTTError):
            W.ttt_qk_norm_rope_backward_work(rope(), bad)
    assert W.lib().ttt_qk_norm_rope_backward_work(ctypes.byref(rope()), 1, None) == 1


def cache(**kw):
    c = W.ttt_kv_cache()
    a = dict(k=P(20).value, v=P(21).value, k_scale=None, v_scale=None, page_stride=2 * 16 * 64, pages=10,
             page_size=16, kv_heads=2, head_dim=64, dtype=0, reserved=0)
    a.update(kw)
    for n, x in a.items():
        setattr(c, n, x)
    return c


def append(c=None, cfg=None, **kw):
    a = dict(q=P(0), ld_q=256, k=P(1), ld_k=128, v=P(2), ld_v=128, qw=None, kw=None, freq=P(4), pos=P(5),
             cache=ctypes.byref(c or cache()), slot=P(6), qo=P(7), ld_qo=256, tokens=10)
    a.update(kw)
    return W.lib().ttt_qk_norm_rope_append(ctypes.byref(cfg or rope()), *a.values(), None)


BAD_CACHES = [
    (dict(dtype=2), 3), (dict(reserved=1), 4), (dict(pages=0), 2), (dict(page_size=0), 2),
    (dict(page_size=65537), 2), (dict(kv_heads=0), 2), (dict(head_dim=24), 2), (dict(page_stride=2047), 2),
    (dict(page_stride=2052), 2), (dict(k_scale=P(30).value), 4), (dict(page_stride=1 << 40, pages=1 << 30), 2),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(kv_heads=1, page_stride=4096), 2), (dict(head_dim=32), 2), (dict(k=None), 1), (dict(v=P(21, 8).value), 9),
    (dict(dtype=1, v_scale=P(30, 4).value), 9), (dict(v=P(20).value), 4), (dict(k=P(7).value), 4),
    (dict(v=P(2).value), 4)])
def test_append_cache(kw, code):
    assert append(cache(**kw)) == code, W.lib().ttt_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), 2), (dict(ld_v=64), 2), (dict(v=None), 1), (dict(slot=None), 1), (dict(slot=P(6, 8)), 9),
    (dict(qo=P(1)), 4), (dict(qo=P(2)), 4), (dict(cache=None), 1), (dict(tokens=0, q=None), 0)])
def test_append_arguments(kw, code):
    assert append(**kw) == code, W.lib().ttt_last_error()


def test_append_takes_bf16_only():
    assert append(cfg=rope(act="f32")) == 3


def paged(c=None, **kw):
    a = dict(q=P(0), ld_q=256, cache=ctypes.byref(c or cache()), table=P(1), lens=P(2), out=P(3), ld_out=256,
             lse=P(4), seqs=3, heads=4, max_pages=8, window=0, scale=0.0, work=P(5), bytes=1 << 30)
    a.update(kw)
    return W.lib().ttt_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(head_dim=32, page_stride=4096), 5), (dict(k=None), 1), (dict(v=P(3).value), 4)])
def test_paged_cache(kw, code):
    assert paged(cache(**kw)) == code, W.lib().ttt_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(seqs=-1), 2), (dict(seqs=(1 << 20) + 1), 2), (dict(heads=3), 2), (dict(heads=0), 2),
    (dict(heads=65538), 2), (dict(seqs=1 << 20, heads=16), 2), (dict(max_pages=-1), 2), (dict(max_pages=(1 << 26) + 1), 2), (dict(window=-1), 2),
    (dict(scale=-1.0), 4), (dict(scale=float("nan")), 4), (dict(scale=float("inf")), 4), (dict(ld_q=128), 2),
    (dict(ld_out=260), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(lse=P(4, 4)), 9), (dict(out=P(0)), 4), (dict(seqs=0, q=None), 0),
    (dict(max_pages=1 << 20, work=None), 1), (dict(max_pages=1 << 20, bytes=100), 2), (dict(cache=None), 1),
])
def test_paged_arguments(kw, code):
    assert paged(**kw) == code, W.lib().ttt_last_error()


def test_paged_work_covers_every_split_and_is_small():
    n = ctypes.c_int64()
    for seqs in (1, 7, 1000, 1 << 20):
        for pages in (0, 1, 40, 1 << 20):
            for window in (0, 1, 2048):
                assert W.lib().ttt_paged_attention_work(ctypes.byref(cache()), seqs, 4, pages, window,
                                                        ctypes.byref(n)) == 0
                assert 0 <= n.value < 1 << 26
    assert W.lib().ttt_paged_attention_work(ctypes.byref(cache()), 1, 4, 1, 0, None) == 1


def window(fn, **kw):
    a = dict(q=P(0), k=P(0, 512), v=P(0, 1024), ld=768, out=P(1), ld_out=256, lse=P(2))
    if fn == "backward":
        a.update(dout=P(3), ld_dout=256, dq=P(4), dk=P(4, 512), dv=P(4, 1024), ld_d=768, work=P(5))
    a.update(batch=1, heads=2, seq_len=20, window=8, mode=0)
    a.update(kw)
    return getattr(W.lib(), "ttt_window_attention_" + fn)(*a.values(), None)


@pytest.mark.parametrize("fn,kw,code", [
    *[(f, kw, code) for f in ("lse", "backward") for kw, code in [
        (dict(batch=0), 2), (dict(heads=0), 2), (dict(window=0), 2), (dict(mode=2), 4), (dict(seq_len=-1), 2),
        (dict(ld=260), 2), (dict(ld=128), 2), (dict(ld_out=128), 2), (dict(ld_out=(1 << 28) + 8), 2),
        (dict(ld=1 << 24), 2), (dict(q=None), 1), (dict(lse=None), 1), (dict(lse=P(2, 4)), 9),
        (dict(seq_len=0, q=None), 0)]],
    ("lse", dict(out=P(0)), 4), ("lse", dict(lse=P(0)), 4), ("lse", dict(lse=P(1)), 4),
    ("backward", dict(ld_dout=128), 2), ("backward", dict(ld_d=128), 2), ("backward", dict(dout=None), 1),
    ("backward", dict(work=None), 1), ("backward", dict(dq=P(0)), 4), ("backward", dict(dk=P(1)), 4),
    ("backward", dict(dv=P(3)), 4), ("backward", dict(dk=P(4, 256)), 4), ("backward", dict(work=P(2)), 4),
    ("backward", dict(work=P(4)), 4), ("backward", dict(dv=P(4)), 4),
])
def test_window_training_arguments(fn, kw, code):
    assert window(fn, **kw) == code, W.lib().ttt_last_error()


INDEX_PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ttt_attention_internal.h"
using namespace ttt;
#define CHECK(x) do { if (!(x)) { printf("%s failed (len %d pages %d size %d window %d splits %d)\n", #x, len, mp, ps, win, sp); return 1; } } while (0)
int main() {
  unsigned s = 1;
  auto rnd = [&](int n) { s = s * 1664525u + 1013904223u; return (int)((s >> 8) % (unsigned)n); };
  for (int it = 0; it < 200000; ++it) {
    const int ps = 1 + rnd(it % 3 ? 70 : 65536);
    const int most = (1 << 30) / ps;
    const int mp = it % 5 ? rnd(20) : most - rnd(2);
    const int len = it % 7 ? rnd(2000) - 5 : (it % 2 ? 0x7fffffff : (int)0x80000000);
    const int win = it % 2 ? 0 : 1 + rnd(it % 4 ? 300 : 0x7ffffffe), sp = 1 + rnd(1024);
    int lo, hi;
    paged_span(len, mp, ps, win, lo, hi);
    CHECK(0 <= lo && lo <= hi && hi <= mp * ps);
    CHECK(hi == (len < 0 ? 0 : len < mp * ps ? len : mp * ps));
    CHECK(hi - lo == (win && win < hi ? win : hi));
    const int part = paged_part(hi - lo, sp);
    CHECK(part >= 0 && part % PG_BLOCK == 0 && (hi == lo || part > 0));
    long covered = 0;
    int live = 0;
    for (int i = 0; i < sp; ++i) {   // the kernel's own expressions
      const long at = (long)i * part;
      CHECK(at < 0x7fffffffL);
      const int b0 = lo + (hi - lo < at ? hi - lo : (int)at), b1 = hi < b0 + part ? hi : b0 + part;
      CHECK((long)b0 + part < 0x7fffffffL && b0 >= lo && b1 <= hi);
      covered += b1 > b0 ? b1 - b0 : 0;
      live += b1 > b0;
    }
    CHECK(covered == hi - lo);
    CHECK(part >= hi - lo ? live <= 1 : live == (hi - lo + part - 1) / part);
  }
  const int len = 0, mp = 0, win = 0, sp = 0;
  for (int ps : {1, 7, 64})
    for (int page : {-2147483647 - 1, -1, 0, 5, 9, 10, 2147483647})
      for (int head : {0, 2})
        for (int place = 0; place < ps; ++place) {
          const int rb = 256, heads = 3;
          const int64_t stride = (int64_t)heads * ps * rb + ((int64_t)1 << 33);
          const int64_t off = paged_row(page, 10, stride, head, ps, place, rb);
          if (page < 0 || page >= 10) CHECK(off == -1);
          else CHECK(off == page * stride + (int64_t)(head * ps + place) * rb && off + rb <= 9 * stride + (int64_t)heads * ps * rb);
        }
  printf("ok\n");
  return 0;
}
"""


def test_paged_index_rules(tmp_path):
    """The functions that the kernels use for a sequence's span, its parts and a token's row,
    compiled for the host: every token once, nothing outside the cache, whatever the lengths and
    page numbers hold."""
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(INDEX_PROGRAM)
    subprocess.run([B.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-I" + os.path.join(ROOT, "include"),
                    "-I" + B.CSRC, "-x", "hip", str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.parametrize("call,kw", [
    *[(forward, dict(qo=P(i))) for i in (2, 3, 4, 5)], *[(forward, dict(ko=P(i))) for i in (2, 3, 4, 5)],
    (forward, dict(pos=P(6, 256 * 2 * 9 + 496))),     # the output's last elements
    *[(backward, {out: P(i)}) for out in ("dqw", "dkw", "work") for i in range(10)],
    *[(backward, {out: P(i)}) for out in ("dq", "dk") for i in (2, 3, 4, 5)],
    (backward, dict(dqw=P(11))), (backward, dict(work=P(10))), (backward, dict(work=P(11))),
    (backward, dict(dqw=P(11), tokens=0)),
    *[(append, dict(qo=P(i))) for i in (4, 5, 6, 20, 21)], *[(append, {n: P(20)}) for n in ("freq", "pos", "slot", "qw")],
    *[(paged, dict(out=P(i))) for i in (0, 1, 2, 20, 21)], *[(paged, dict(lse=P(i))) for i in (0, 1, 2, 3, 20, 21)],
    *[(paged, dict(work=P(i), max_pages=1000)) for i in (0, 1, 2, 3, 4, 20, 21)],
])
def test_nothing_written_overlaps_what_is_read(call, kw):
    assert call(**kw) == 4, W.lib().ttt_last_error()


def test_scales_of_an_e4m3_cache_are_not_written_over():
    for n in ("k_scale", "v_scale"):
        assert append(cache(dtype=1, **{n: P(7).value})) == 4
        assert append(cache(dtype=1, **{n: P(21).value})) == 4
        for at in (3, 4):
            assert paged(cache(dtype=1, **{n: P(at).value})) == 4


@pytest.mark.parametrize("fn", ["lse", "backward", ""])
@pytest.mark.parametrize("batch,heads,seq_len,code", [
    ((1 << 24) - 1, 1, 128, 1), (1 << 24, 1, 1, 2), ((1 << 23) + 1, 1, 129, 2), (1 << 12, 1 << 12, 1, 2),
    ((1 << 12) - 1, 1 << 12, 1, 1), (1, 1, (1 << 31) - 128, 1), (1, 1, (1 << 31) - 127, 2),
    (1 << 24, 1 << 16, (1 << 31) - 1, 2),     # the product of the three passes 64 bits
    ((1 << 31) - 1, (1 << 17) - 1, (1 << 31) - 1, 2), ((1 << 31) - 1, 1, 0, 0),
])
def test_window_launches_count_their_threads_in_32_bits(fn, batch, heads, seq_len, code):
    """256 threads to every 128 rows of a head: 2^24 such workgroups are refused before any launch,
    one fewer passes on to the pointers (code 1: q is NULL)."""
    ld = heads * 128
    kw = dict(q=None, ld=ld, ld_out=ld, batch=batch, heads=heads, seq_len=seq_len)
    if fn == "":
        got = W.lib().ttt_window_attention(None, P(0), P(0), ld, P(1), ld, batch, heads, seq_len, 8, 0, None)
    else:
        got = window(fn, **kw, **(dict(ld_dout=ld, ld_d=ld) if fn == "backward" else {}))
    assert got == code, W.lib().ttt_last_error()
