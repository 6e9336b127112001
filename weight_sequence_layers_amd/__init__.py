"""Python binding of libttt, the large-chunk TTT layer forward for MI355X (gfx950).

Argument marshalling only: every step of the layer runs in the HIP kernels of libttt.so.
PyTorch supplies device memory and the current stream. The functions carry the C names
(ttt_init_state, ttt_chunk_forward, ttt_sequence_forward, ...) and raise TTTError on any
non-OK status. If libttt.so is missing or cannot be loaded, every call raises: there is
no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
# LIBTTT_PATH selects another build of the library (the host-sanitized copy of the CPU tests)
LIB_PATH = os.environ.get("LIBTTT_PATH") or os.path.join(PKG, "libttt.so")

FW = {"swiglu": 0, "gelu": 1, "linear": 2}
LOSS = {"dot": 0, "mse": 1}
ACT = {"f32": 0, "bf16": 1}
ORDER = {"apply_then_update": 0, "update_then_apply": 1}

STATUS = {0: "TTT_OK", 1: "TTT_E_NULL", 2: "TTT_E_SHAPE", 3: "TTT_E_DTYPE", 4: "TTT_E_CONFIG",
          5: "TTT_E_UNSUPPORTED", 6: "TTT_E_ALLOC", 7: "TTT_E_HIP", 8: "TTT_E_NONFINITE",
          9: "TTT_E_ALIGN"}

# bf16 planes per operand class (apply, grad, ns) and the mask of Newton-Schulz iterations
# run on one plane (ns_one_plane) for the named workloads; chosen as the cheapest setting
# whose end-to-end error stays well inside the parity bound.
PRECISION = {
    "tiny": (3, 3, 3, 0),
    "lm": (1, 2, 2, 0b00011),
    "long": (1, 3, 3, 0),
    "long_alt": (1, 3, 3, 0),
    "imageset": (1, 1, 2, 0),
    "smallchunk": (1, 1, 1, 0),
}


class TTTError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class ttt_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "heads", "dim", "hidden", "chunk", "fw", "loss", "act", "order", "ns_steps",
        "row_renorm", "apply_planes", "grad_planes", "ns_planes", "ns_one_plane", "path")
    ] + [("lr", ctypes.c_float * 3), ("weight_decay", ctypes.c_float), ("replay", ctypes.c_int32),
         ("momentum", ctypes.c_float)]


class ttt_block_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "dim", "window", "window_mode", "ffn_hidden", "reserved")
    ] + [("max_seq_len", ctypes.c_int64), ("ttt", ttt_config)]


BLOCK_WEIGHTS = ("attn_qkv", "attn_out", "ttt_qkv", "ttt_eta", "ttt_out", "ffn_up", "ffn_down")


class ttt_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BLOCK_WEIGHTS]


class ttt_rope_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "q_heads", "k_heads", "head_dim", "rot_dim", "axes", "pairing", "norm", "act")
    ] + [("eps", ctypes.c_float)]


class ttt_kv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")
    ] + [("page_stride", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in (
        "pages", "page_size", "kv_heads", "head_dim", "dtype", "reserved")]
    device = None   # of the tensors, where make_kv_cache filled the struct


HEAD_NORM = {"none": 0, "rms": 1}
PAIRING = {"halves": 0, "pairs": 1}
WINDOW = {"sliding": 0, "block": 1}
LINEAR_EPI = {"plain": 0, "residual": 1, "gelu": 2}
ATTN_HEAD_DIM = 128

_lib = None


def lib() -> ctypes.CDLL:
    """Load libttt.so (built in-tree by build.py). Raises if it is not there."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run weight_sequence_layers_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        cfgp, vp, i64 = ctypes.POINTER(ttt_config), ctypes.c_void_p, ctypes.c_int64
        i32 = ctypes.c_int32
        ropep, cachep = ctypes.POINTER(ttt_rope_config), ctypes.POINTER(ttt_kv_cache)
        sig = {
            "ttt_validate_config": [cfgp],
            "ttt_state_numel": [cfgp, ctypes.POINTER(i64)],
            "ttt_init_state": [cfgp, vp, vp, ctypes.POINTER(vp)],
            "ttt_chunk_forward": [vp, vp, vp, vp, vp, vp, vp],
            "ttt_sequence_forward": [vp, vp, vp, vp, vp, vp, i64, vp],
            "ttt_sequence_forward_masked": [vp, vp, vp, vp, vp, vp, i64, vp, vp],
            "ttt_apply_backward": [vp, vp, vp, vp, vp, vp],
            "ttt_chunk_backward": [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
            "ttt_get_state": [vp, vp, vp],
            "ttt_set_state": [vp, vp, vp],
            "ttt_state_health": [vp],
            "ttt_destroy_state": [vp],
            "ttt_sequence_forward_noalloc": [cfgp, vp, vp, vp, vp, vp, vp, i64, vp],
            "ttt_profile_begin": [vp, ctypes.c_int32, ctypes.c_int32],
            "ttt_profile_end": [vp, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)],
            "ttt_window_attention": [vp, vp, vp, i64, vp, i64, i32, i32, i64, i32, i32, vp],
            "ttt_linear": [vp, vp, vp, vp, i64, i32, i32, i32, vp],
            "ttt_block_init": [ctypes.POINTER(ttt_block_config),
                               ctypes.POINTER(ttt_block_weights), vp, vp, ctypes.POINTER(vp)],
            "ttt_block_forward": [vp, vp, vp, i64, vp],
            "ttt_block_destroy": [vp],
            "ttt_validate_rope_config": [ropep],
            "ttt_qk_norm_rope": [ropep, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, i64,
                                 vp],
            "ttt_qk_norm_rope_backward_work": [ropep, i64, ctypes.POINTER(i64)],
            "ttt_qk_norm_rope_backward": [ropep, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp,
                                          i64, vp, i64, vp, i64, vp, vp, vp, i64, i64, vp],
            "ttt_qk_norm_rope_append": [ropep, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, cachep,
                                        vp, vp, i64, i64, vp],
            "ttt_paged_attention_work": [cachep, i32, i32, i32, i32, ctypes.POINTER(i64)],
            "ttt_paged_attention": [vp, i64, cachep, vp, vp, vp, i64, vp, i32, i32, i32, i32,
                                    ctypes.c_float, vp, i64, vp],
            "ttt_window_attention_lse": [vp, vp, vp, i64, vp, i64, vp, i32, i32, i64, i32, i32,
                                         vp],
            "ttt_window_attention_backward": [vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp, vp,
                                              i64, vp, i32, i32, i64, i32, i32, vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.ttt_block_ttt_state.argtypes = [vp]
        L.ttt_block_ttt_state.restype = vp
        L.ttt_status_str.argtypes = [ctypes.c_int]
        L.ttt_status_str.restype = ctypes.c_char_p
        L.ttt_last_error.argtypes = []
        L.ttt_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(st: int):
    if st != 0:
        raise TTTError(st, lib().ttt_last_error().decode())


PATH = {"auto": 0, "staged": 1, "resident": 2}


def make_config(cfg=None, *, planes=None, **kw) -> ttt_config:
    """ttt_config from an object with the workload fields (batch, heads, dim, hidden, chunk,
    fw, loss, act, order, ns_steps, renorm and optionally lr, weight_decay), overridden by
    keyword arguments. `planes` is (apply, grad, ns, ns_one_plane); by default the preset of
    the workload's name, else 0s. `path` is "auto", "staged" or "resident". `lr` is a
    sequence of up to 3 step sizes in the state's matrix order (0 or missing: 1). `replay`
    records each call's launches in a HIP graph and replays it for repeated pointers."""
    f = {}
    if cfg is not None:
        for k in ("batch", "heads", "dim", "hidden", "chunk", "fw", "loss", "act", "order",
                  "ns_steps", "renorm"):
            f[k] = getattr(cfg, k)
        for k in ("lr", "weight_decay", "momentum"):
            if hasattr(cfg, k):
                f[k] = getattr(cfg, k)
        if planes is None:
            planes = PRECISION.get(getattr(cfg, "name", ""), None)
    f.update(kw)
    planes = planes or (0, 0, 0, 0)
    c = ttt_config()
    c.batch, c.heads, c.dim, c.hidden, c.chunk = (int(f["batch"]), int(f["heads"]), int(f["dim"]),
                                                  int(f["hidden"]), int(f["chunk"]))
    c.fw = FW[f["fw"]] if isinstance(f["fw"], str) else int(f["fw"])
    c.loss = LOSS[f["loss"]] if isinstance(f["loss"], str) else int(f["loss"])
    c.act = ACT[f["act"]] if isinstance(f["act"], str) else int(f["act"])
    c.order = ORDER[f["order"]] if isinstance(f["order"], str) else int(f["order"])
    c.ns_steps = int(f.get("ns_steps", 0))
    c.row_renorm = int(bool(f.get("renorm", False)))
    c.apply_planes, c.grad_planes, c.ns_planes, c.ns_one_plane = (int(p) for p in planes)
    path = f.get("path", "auto")
    c.path = PATH[path] if isinstance(path, str) else int(path)
    lr = list(f.get("lr", ()) or ())
    if len(lr) > 3:
        raise ValueError("at most 3 step sizes")
    for i, x in enumerate(lr):
        c.lr[i] = float(x)
    c.weight_decay = float(f.get("weight_decay", 0.0))
    c.replay = int(bool(f.get("replay", False)))
    c.momentum = float(f.get("momentum", 0.0))
    return c


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return int(getattr(stream, "cuda_stream", stream)) or None


def ttt_validate_config(cfg: ttt_config) -> None:
    _check(lib().ttt_validate_config(ctypes.byref(cfg)))


def ttt_state_numel(cfg: ttt_config) -> int:
    n = ctypes.c_int64()
    _check(lib().ttt_state_numel(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


class State:
    """Owns a ttt_state handle (freed by destroy() or garbage collection), or, with
    owner set, refers to one that object owns (destroy() then only drops the reference)."""

    def __init__(self, handle: int, cfg: ttt_config, owner=None):
        self.handle = ctypes.c_void_p(handle)
        self.cfg = cfg
        self.owner = owner

    def destroy(self):
        if self.handle:
            h, self.handle = self.handle, None
            if self.owner is None:
                _check(lib().ttt_destroy_state(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def ttt_init_state(cfg: ttt_config, w0, stream=None) -> State:
    """w0: contiguous fp32 device tensor with the per-head initial matrices, matrix by
    matrix (see include/libttt.h)."""
    h = ctypes.c_void_p()
    _check(lib().ttt_init_state(ctypes.byref(cfg), _ptr(w0), _stream(stream), ctypes.byref(h)))
    return State(h.value, cfg)


def ttt_chunk_forward(st: State, q, k, v, eta, out, stream=None) -> None:
    _check(lib().ttt_chunk_forward(st.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(out),
                                   _stream(stream)))


def ttt_apply_backward(st: State, q, dout, dq, dw, stream=None) -> None:
    """Backward of one chunk's apply step with the state as it stands: dq [B,H,chunk,d] and
    dw (state-shaped fp32) of sum <dout, f_W(q)> (see include/libttt.h)."""
    _check(lib().ttt_apply_backward(st.handle, _ptr(q), _ptr(dout), _ptr(dq), _ptr(dw),
                                    _stream(stream)))


def ttt_chunk_backward(st: State, q, k, v, eta, dout, dw, dq, dk, dv, deta, stream=None) -> None:
    """Backward through one chunk with the state as it stands (the state before the chunk):
    dw holds the cotangent of the state after the chunk and receives that of the state
    before it; dq, dk, dv, deta receive the input gradients (see include/libttt.h)."""
    _check(lib().ttt_chunk_backward(st.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(dout),
                                    _ptr(dw), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(deta),
                                    _stream(stream)))


def ttt_sequence_forward(st: State, q, k, v, eta, out, seq_len: int, stream=None) -> None:
    _check(lib().ttt_sequence_forward(st.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                      _ptr(out), int(seq_len), _stream(stream)))


# workspace bytes the allocation-free call holds per GPU (TTT_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 << 20


def ttt_sequence_forward_noalloc(cfg: ttt_config, state, q, k, v, eta, out, seq_len: int,
                                 stream=None) -> None:
    """ttt_sequence_forward with no state object and no allocation: `state` (fp32 device
    tensor, the ttt_get_state layout) holds the initial weights and receives the final ones
    (see include/libttt.h)."""
    _check(lib().ttt_sequence_forward_noalloc(ctypes.byref(cfg), _ptr(state), _ptr(q), _ptr(k),
                                              _ptr(v), _ptr(eta), _ptr(out), int(seq_len),
                                              _stream(stream)))


def ttt_sequence_forward_masked(st: State, q, k, v, eta, out, seq_len: int, update,
                                stream=None) -> None:
    """ttt_sequence_forward in which chunk c updates the state only if update[c] is true
    (a sequence of seq_len/chunk flags, or None for all; see include/libttt.h)."""
    n = int(seq_len) // st.cfg.chunk
    arr = None
    if update is not None:
        flags = [1 if u else 0 for u in update]
        if len(flags) != n:
            raise ValueError(f"{len(flags)} update flags for {n} chunks")
        arr = (ctypes.c_uint8 * max(n, 1))(*flags)
    _check(lib().ttt_sequence_forward_masked(st.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(eta),
                                             _ptr(out), int(seq_len),
                                             ctypes.cast(arr, ctypes.c_void_p) if arr else None,
                                             _stream(stream)))


def ttt_get_state(st: State, dst, stream=None) -> None:
    _check(lib().ttt_get_state(st.handle, _ptr(dst), _stream(stream)))


def ttt_set_state(st: State, src, stream=None) -> None:
    _check(lib().ttt_set_state(st.handle, _ptr(src), _stream(stream)))


def ttt_state_health(st: State) -> None:
    _check(lib().ttt_state_health(st.handle))


def ttt_destroy_state(st: State) -> None:
    st.destroy()


STAGES = {"front_q": 0, "front_k": 1, "out": 2, "contract": 3, "ns_gram": 4, "ns_poly": 5,
          "ns_update": 6, "renorm": 7, "split": 8, "mse": 9, "resident": 10, "dq": 11,
          "tfront": 12, "ns_bwd": 13, "ns_small": 14}


def ttt_profile_begin(st: State, stage, max_launches: int = 4096) -> None:
    """Bracket every launch of one stage kernel with HIP events (see include/libttt.h)."""
    sid = STAGES[stage] if isinstance(stage, str) else int(stage)
    _check(lib().ttt_profile_begin(st.handle, sid, int(max_launches)))


def ttt_profile_end(st: State):
    """Returns (timed launches, total milliseconds)."""
    n = ctypes.c_int64()
    ms = ctypes.c_double()
    _check(lib().ttt_profile_end(st.handle, ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value


def matrix_shapes(cfg: ttt_config):
    d, dh = cfg.dim, cfg.hidden
    return {0: [(dh, d), (dh, d), (d, dh)], 1: [(dh, d), (d, dh)], 2: [(d, d)]}[cfg.fw]


def split_state(cfg: ttt_config, flat):
    """Views of a flat state buffer as per-matrix [batch, heads, rows, cols] tensors: the
    fast weights, then (with momentum) their buffers."""
    out, o = [], 0
    shapes = matrix_shapes(cfg)
    for r, c in shapes + (shapes if cfg.momentum > 0 else []):
        n = cfg.batch * cfg.heads * r * c
        out.append(flat[o:o + n].view(cfg.batch, cfg.heads, r, c))
        o += n
    return out


# ---------------------------------------------------------------- the LaCT block (ttt_block.h)
def ttt_window_attention(q, k, v, ld: int, out, ld_out: int, batch: int, heads: int,
                         seq_len: int, window: int, mode="sliding", stream=None) -> None:
    """Window attention over heads of 128: q, k, v, out bf16 device tensors whose element
    (b, t, h, e) sits at (b seq_len + t) ld + 128 h + e (ld_out for out); mode "sliding" or
    "block" (see include/ttt_block.h)."""
    m = WINDOW[mode] if isinstance(mode, str) else int(mode)
    _check(lib().ttt_window_attention(_ptr(q), _ptr(k), _ptr(v), int(ld), _ptr(out),
                                      int(ld_out), int(batch), int(heads), int(seq_len),
                                      int(window), m, _stream(stream)))


def ttt_linear(x, w, resid, y, rows: int, in_features: int, out_features: int,
               epilogue="plain", stream=None) -> None:
    """y = epilogue(x w^T) in bf16 with fp32 accumulation; epilogue "plain", "residual"
    (adds resid) or "gelu" (see include/ttt_block.h)."""
    e = LINEAR_EPI[epilogue] if isinstance(epilogue, str) else int(epilogue)
    _check(lib().ttt_linear(_ptr(x), _ptr(w), _ptr(resid), _ptr(y), int(rows), int(in_features),
                            int(out_features), e, _stream(stream)))


def make_block_config(ttt: ttt_config, *, dim: int, window: int, mode="sliding",
                      ffn_hidden: int = 0, max_seq_len: int) -> ttt_block_config:
    c = ttt_block_config()
    c.batch = ttt.batch
    c.dim = int(dim)
    c.window = int(window)
    c.window_mode = WINDOW[mode] if isinstance(mode, str) else int(mode)
    c.ffn_hidden = int(ffn_hidden)
    c.reserved = 0
    c.max_seq_len = int(max_seq_len)
    c.ttt = ttt
    return c


class Block:
    """Owns a ttt_block handle and keeps the weight tensors it references alive."""

    def __init__(self, handle: int, cfg: ttt_block_config, weights):
        self.handle = ctypes.c_void_p(handle)
        self.cfg = cfg
        self.weights = weights

    def destroy(self):
        if self.handle:
            h, self.handle = self.handle, None
            _check(lib().ttt_block_destroy(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def ttt_block_init(cfg: ttt_block_config, weights, w0, stream=None) -> Block:
    """weights: mapping from the names in BLOCK_WEIGHTS to contiguous bf16 device tensors;
    w0: the TTT sub-layer's initial matrices (the layout ttt_init_state takes)."""
    w = ttt_block_weights()
    for n in BLOCK_WEIGHTS:
        setattr(w, n, _ptr(weights[n]))
    h = ctypes.c_void_p()
    _check(lib().ttt_block_init(ctypes.byref(cfg), ctypes.byref(w), _ptr(w0), _stream(stream),
                                ctypes.byref(h)))
    return Block(h.value, cfg, dict(weights))


def ttt_block_forward(blk: Block, x, y, seq_len: int, stream=None) -> None:
    _check(lib().ttt_block_forward(blk.handle, _ptr(x), _ptr(y), int(seq_len), _stream(stream)))


def ttt_block_ttt_state(blk: Block) -> State:
    """The block's TTT state, for ttt_get_state and the other state calls."""
    return State(lib().ttt_block_ttt_state(blk.handle), blk.cfg.ttt, owner=blk)


def ttt_block_destroy(blk: Block) -> None:
    blk.destroy()


# ------------------------------------------- attention around the block (ttt_attention.h)
def _here(stream):
    """torch, the current device's number and the handle of `stream` (None: its current
    stream)."""
    import torch
    dev = torch._C._cuda_getDevice()   # the tensors have initialised torch.cuda: 0.2 us less than asking it
    if stream is None:   # the handle without a Stream object around it: 1 us less per call
        return torch, dev, torch._C._cuda_getCurrentRawStream(dev) or None
    if getattr(getattr(stream, "device", None), "index", dev) != dev:
        raise TTTError(4, f"a stream of {stream.device}, not of the current HIP device")
    return torch, dev, _stream(stream)


def _cache(c, dev: int):
    """The cache as an argument; make_kv_cache noted the device of its tensors."""
    if c.device is not None and c.device != dev:
        raise TTTError(4, f"the cache is on cuda:{c.device}, not on the current HIP device")
    return ctypes.byref(c)


def _arg(t, name: str, dtype, n: int, dev: int, dense: bool = True) -> Optional[int]:
    """The pointer of a device tensor argument, after the checks that the library cannot make:
    a tensor of the current device dev, of its dtype, with at least n elements (dense:
    contiguous). None passes as NULL."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise TTTError(4, f"{name} is on {t.device}, not on the current HIP device")
    if t.dtype is not dtype:
        raise TTTError(3, f"{name} is {t.dtype}, not {dtype}")
    if t.numel() < n:
        raise TTTError(2, f"{name} has {t.numel()} elements, {n} needed")
    if dense and not t.is_contiguous():
        raise TTTError(2, f"{name} is not contiguous")
    return t.data_ptr()


def _table(t, name: str, dtype, shape, dev: int) -> Optional[int]:
    """_arg of a table read as `shape`: flat, or of a shape whose rows fall where those of `shape`
    do (more rows may follow). A wider table, or one with its axes in another order, would be
    read with the wrong row length."""
    if t is not None and t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    n = 1
    for x in shape:
        n *= x
    p = _arg(t, name, dtype, n, dev)
    if p is not None and n and t.dim() > 1:
        def apart(dims):   # elements between neighbours along each dim of more than one
            at, m = [], 1
            for x in reversed(dims):
                if x > 1:
                    at.append(m)
                    m *= x
            return at
        have, want = apart(t.shape), apart(shape)
        if len(have) < len(want):
            want = want[:len(have)]   # flat, or some of the outer dims as one
        if not set(have).issuperset(want):
            raise TTTError(2, f"{name} is {list(t.shape)}, read as {list(shape)}")
    return p


def _rows_fit(t, rows: int, width: int, ld: int) -> bool:
    """Whether t holds `rows` rows of `width` elements ld apart as its own strides have it: dims
    that are dense up to a row, then one of stride ld, and dense in rows before it, in whatever
    order the tensor names them (heads before tokens: the same memory); or contiguous rows given
    flat or with the row's dims among the outer ones. One row needs to be dense."""
    dims = [(s, n) for n, s in zip(reversed(t.shape), reversed(t.stride())) if n > 1]
    if rows > 1:
        dims.sort()
    at, inner, outer, dense = 1, 1, 1, True
    for s, n in dims:
        if dense and rows > 1 and s == ld and ld >= at:
            at, dense = ld, False
        if s != at:
            return inner >= width and (outer >= rows if not dense else rows <= 1)
        at *= n
        if dense:
            inner *= n
        else:
            outer *= n
    if not dense:
        return outer >= rows and inner >= width
    return rows <= 1 or len(dims) < 2 or (
        len(dims) == 2 and ld == width and ld % dims[0][1] == 0 and t.is_contiguous())


def _rows(t, name: str, dtype, rows: int, width: int, ld: int, dev: int) -> Optional[int]:
    """_arg of a matrix of rows ld elements apart: a flat tensor, or one whose own rows are. The
    last must end within a contiguous tensor, or within the memory that another is a view of (a
    third of a projection's rows)."""
    if t is None:
        return None
    here = t.dtype is dtype and t.get_device() == dev
    shape = t.shape
    if here and len(shape) == 2 and rows <= shape[0] and width <= shape[1] and t.stride() == (ld, 1):
        return t.data_ptr()   # most calls: the tests below cost 0.2 us a tensor
    last, have = (rows - 1) * ld + width, t.numel()
    if here and have >= rows * width:
        if rows > 0 and not _rows_fit(t, rows, width, ld):
            raise TTTError(2, f"{name}: {list(shape)} of strides {list(t.stride())}, read as {rows} rows of {width}, "
                              f"{ld} apart")
        if not t.is_contiguous():
            have = t.untyped_storage().nbytes() // dtype.itemsize - t.storage_offset()
        if have >= last:
            return t.data_ptr()
    _arg(t, name, dtype, rows * width, dev, False)
    raise TTTError(2, f"{name}: {rows} rows {ld} apart take {last} elements, {have} are there")


def _int32(x: int) -> None:
    """Refuses what ctypes would wrap: x is the bitwise or of numbers passed as int32 (a negative
    one among them is the library's to refuse)."""
    if x >> 31 > 0:
        raise TTTError(2, "a number of 2^31 or more")


def _work(t, dev: int):
    """Pointer and bytes of a workspace tensor of any dtype (None: none)."""
    return (None, 0) if t is None else (_arg(t, "work", t.dtype, 0, dev), t.nbytes)


def make_rope_config(*, q_heads: int, k_heads: int, head_dim: int, rot_dim: Optional[int] = None,
                     axes: int = 1, pairing="halves", norm="rms", act="bf16",
                     eps: float = 1e-6) -> ttt_rope_config:
    """ttt_rope_config; rot_dim None rotates whole heads."""
    _int32(int(q_heads) | int(k_heads) | int(head_dim) | int(rot_dim or 0) | int(axes))
    c = ttt_rope_config()
    c.q_heads, c.k_heads, c.head_dim = int(q_heads), int(k_heads), int(head_dim)
    c.rot_dim = int(head_dim if rot_dim is None else rot_dim)
    c.axes = int(axes)
    c.pairing = PAIRING[pairing] if isinstance(pairing, str) else int(pairing)
    c.norm = HEAD_NORM[norm] if isinstance(norm, str) else int(norm)
    c.act = ACT[act] if isinstance(act, str) else int(act)
    c.eps = float(eps)
    return c


def ttt_validate_rope_config(cfg: ttt_rope_config) -> None:
    _check(lib().ttt_validate_rope_config(ctypes.byref(cfg)))


def _rope_inputs(cfg, q_weight, k_weight, freq, pos, tokens, dev, dt, torch):
    D, half, axes = cfg.head_dim, cfg.rot_dim // 2, cfg.axes
    return (_arg(q_weight, "q_weight", dt, D, dev), _arg(k_weight, "k_weight", dt, D, dev),
            _table(freq, "freq", torch.float32, (axes, half), dev),
            _table(pos, "pos", torch.int32, (axes, tokens if half else 0), dev))


def ttt_qk_norm_rope(cfg: ttt_rope_config, q, ld_q: int, k, ld_k: int, q_weight, k_weight, freq,
                     pos, q_out, ld_qo: int, k_out, ld_ko: int, tokens: int,
                     stream=None) -> None:
    """Per-head norm and position rotation of queries and keys: element (t, h, e) of q at
    t ld_q + h head_dim + e (k, q_out and k_out with theirs); freq fp32 [axes, rot_dim / 2],
    pos int32 [axes, tokens] (see include/ttt_attention.h)."""
    torch, dev, st = _here(stream)
    D, dt = cfg.head_dim, torch.bfloat16 if cfg.act == 1 else torch.float32
    wq, wk = cfg.q_heads * D, cfg.k_heads * D
    _check(lib().ttt_qk_norm_rope(
        ctypes.byref(cfg), _rows(q, "q", dt, tokens, wq, ld_q, dev), ld_q,
        _rows(k, "k", dt, tokens, wk, ld_k, dev), ld_k,
        *_rope_inputs(cfg, q_weight, k_weight, freq, pos, tokens, dev, dt, torch),
        _rows(q_out, "q_out", dt, tokens, wq, ld_qo, dev), ld_qo,
        _rows(k_out, "k_out", dt, tokens, wk, ld_ko, dev), ld_ko, tokens, st))


def ttt_qk_norm_rope_backward_work(cfg: ttt_rope_config, tokens: int) -> int:
    """Bytes of the workspace that ttt_qk_norm_rope_backward takes."""
    n = ctypes.c_int64()
    _check(lib().ttt_qk_norm_rope_backward_work(ctypes.byref(cfg), tokens, ctypes.byref(n)))
    return n.value


def ttt_qk_norm_rope_backward(cfg: ttt_rope_config, q, ld_q: int, k, ld_k: int, q_weight, k_weight,
                              freq, pos, dq_out, ld_dqo: int, dk_out, ld_dko: int, dq, ld_dq: int,
                              dk, ld_dk: int, dq_weight, dk_weight, work, tokens: int,
                              stream=None) -> None:
    """Backward of ttt_qk_norm_rope: dq, dk (activation dtype) and dq_weight, dk_weight (fp32
    [head_dim], or None); work: device tensor of at least ttt_qk_norm_rope_backward_work bytes
    (see include/ttt_attention.h)."""
    torch, dev, st = _here(stream)
    D, dt = cfg.head_dim, torch.bfloat16 if cfg.act == 1 else torch.float32
    wq, wk = cfg.q_heads * D, cfg.k_heads * D
    f32 = torch.float32
    _check(lib().ttt_qk_norm_rope_backward(
        ctypes.byref(cfg), _rows(q, "q", dt, tokens, wq, ld_q, dev), ld_q,
        _rows(k, "k", dt, tokens, wk, ld_k, dev), ld_k,
        *_rope_inputs(cfg, q_weight, k_weight, freq, pos, tokens, dev, dt, torch),
        _rows(dq_out, "dq_out", dt, tokens, wq, ld_dqo, dev), ld_dqo,
        _rows(dk_out, "dk_out", dt, tokens, wk, ld_dko, dev), ld_dko,
        _rows(dq, "dq", dt, tokens, wq, ld_dq, dev), ld_dq,
        _rows(dk, "dk", dt, tokens, wk, ld_dk, dev), ld_dk,
        _arg(dq_weight, "dq_weight", f32, D, dev), _arg(dk_weight, "dk_weight", f32, D, dev),
        *_work(work, dev), tokens, st))


def make_kv_cache(k, v, *, k_scale=None, v_scale=None) -> ttt_kv_cache:
    """ttt_kv_cache over k and v, device tensors [pages, kv_heads, page_size, head_dim] of bf16
    or float8_e4m3fn whose pages are contiguous and equally far apart (two tensors, or the
    halves of one [pages, 2, ...]); the scales are fp32 [kv_heads] or None. The tensors stay
    alive with the struct."""
    import torch
    shape, stride = k.shape, k.stride()
    if len(shape) != 4 or shape != v.shape or k.dtype is not v.dtype or stride != v.stride():
        raise TTTError(2, "k and v: two tensors [pages, kv_heads, page_size, head_dim] of one "
                          "dtype and layout")
    pages, heads, size, dim = shape
    _int32(pages | heads | size | dim)
    if pages < 1 or not ((stride[3] == 1 or dim == 1) and (stride[2] == dim or size == 1) and
                         (stride[1] == size * dim or heads == 1)):
        raise TTTError(2, "at least one page, and each contiguous")
    if k.dtype is torch.bfloat16:
        dtype = 0
    elif k.dtype is torch.float8_e4m3fn:
        dtype = 1
    else:
        raise TTTError(3, f"cache of {k.dtype}: bfloat16 or float8_e4m3fn")
    dev = torch._C._cuda_getDevice()
    c = ttt_kv_cache(_arg(k, "k", k.dtype, 0, dev, False), _arg(v, "v", k.dtype, 0, dev, False),
                     _arg(k_scale, "k_scale", torch.float32, heads, dev),
                     _arg(v_scale, "v_scale", torch.float32, heads, dev),
                     stride[0] if pages > 1 else heads * size * dim, pages, size, heads, dim, dtype, 0)
    c.tensors = (k, v, k_scale, v_scale)
    c.device = dev
    return c


def ttt_qk_norm_rope_append(cfg: ttt_rope_config, q, ld_q: int, k, ld_k: int, v, ld_v: int,
                            q_weight, k_weight, freq, pos, cache: ttt_kv_cache, slot, q_out,
                            ld_qo: int, tokens: int, stream=None) -> None:
    """ttt_qk_norm_rope of new tokens, keys and values going to the cache: slot int64 [tokens],
    page * page_size + place, or negative for a token that is not stored
    (see include/ttt_attention.h)."""
    torch, dev, st = _here(stream)
    D, dt = cfg.head_dim, torch.bfloat16 if cfg.act == 1 else torch.float32
    wq, wk = cfg.q_heads * D, cfg.k_heads * D
    _check(lib().ttt_qk_norm_rope_append(
        ctypes.byref(cfg), _rows(q, "q", dt, tokens, wq, ld_q, dev), ld_q,
        _rows(k, "k", dt, tokens, wk, ld_k, dev), ld_k,
        _rows(v, "v", dt, tokens, wk, ld_v, dev), ld_v,
        *_rope_inputs(cfg, q_weight, k_weight, freq, pos, tokens, dev, dt, torch),
        _cache(cache, dev), _arg(slot, "slot", torch.int64, tokens, dev),
        _rows(q_out, "q_out", dt, tokens, wq, ld_qo, dev), ld_qo, tokens, st))


def ttt_paged_attention_work(cache: ttt_kv_cache, seqs: int, heads: int, max_pages: int,
                             window: int) -> int:
    """Bytes of the workspace that ttt_paged_attention takes."""
    _int32(seqs | heads | max_pages | window)
    n = ctypes.c_int64()
    _check(lib().ttt_paged_attention_work(ctypes.byref(cache), seqs, heads, max_pages, window,
                                          ctypes.byref(n)))
    return n.value


def ttt_paged_attention(q, ld_q: int, cache: ttt_kv_cache, table, lens, out, ld_out: int, lse,
                        seqs: int, heads: int, max_pages: int, window: int, scale: float, work,
                        stream=None) -> None:
    """Attention of one new token per sequence over its cached tokens: table int32
    [seqs, max_pages], lens int32 [seqs]; window 0: all of them; scale 0: 1 / sqrt(head_dim);
    lse fp32 [seqs, heads] or None (see include/ttt_attention.h)."""
    _int32(seqs | heads | max_pages | window)
    if scale and -2.0 ** -150 <= scale <= 2.0 ** -150:
        raise TTTError(4, f"scale {scale} is 0 in 32 bits, which selects another")
    torch, dev, st = _here(stream)
    bf, n = torch.bfloat16, heads * cache.head_dim
    _check(lib().ttt_paged_attention(
        _rows(q, "q", bf, seqs, n, ld_q, dev), ld_q, _cache(cache, dev),
        _table(table, "table", torch.int32, (seqs, max_pages), dev), _arg(lens, "lens", torch.int32, seqs, dev),
        _rows(out, "out", bf, seqs, n, ld_out, dev), ld_out,
        _table(lse, "lse", torch.float32, (seqs, heads), dev), seqs, heads, max_pages, window, scale,
        *_work(work, dev), st))


def ttt_window_attention_lse(q, k, v, ld: int, out, ld_out: int, lse, batch: int, heads: int,
                             seq_len: int, window: int, mode="sliding", stream=None) -> None:
    """ttt_window_attention that also stores lse, fp32 [batch, heads, seq_len], for the backward
    (see include/ttt_attention.h)."""
    _int32(batch | heads | window)
    m = WINDOW[mode] if isinstance(mode, str) else int(mode)
    torch, dev, st = _here(stream)
    bf, rows, n = torch.bfloat16, batch * seq_len, heads * ATTN_HEAD_DIM
    _check(lib().ttt_window_attention_lse(
        _rows(q, "q", bf, rows, n, ld, dev), _rows(k, "k", bf, rows, n, ld, dev),
        _rows(v, "v", bf, rows, n, ld, dev), ld,
        _rows(out, "out", bf, rows, n, ld_out, dev), ld_out,
        _table(lse, "lse", torch.float32, (batch, heads, seq_len), dev), batch, heads, seq_len, window, m, st))


def ttt_window_attention_backward(q, k, v, ld: int, out, ld_out: int, lse, dout, ld_dout: int, dq,
                                  dk, dv, ld_d: int, work, batch: int, heads: int, seq_len: int,
                                  window: int, mode="sliding", stream=None) -> None:
    """Backward of ttt_window_attention: dq, dk, dv with row stride ld_d; work fp32
    [batch, heads, seq_len] (see include/ttt_attention.h)."""
    _int32(batch | heads | window)
    m = WINDOW[mode] if isinstance(mode, str) else int(mode)
    torch, dev, st = _here(stream)
    bf, f32, rows, n = torch.bfloat16, torch.float32, batch * seq_len, heads * ATTN_HEAD_DIM
    _check(lib().ttt_window_attention_backward(
        _rows(q, "q", bf, rows, n, ld, dev), _rows(k, "k", bf, rows, n, ld, dev),
        _rows(v, "v", bf, rows, n, ld, dev), ld,
        _rows(out, "out", bf, rows, n, ld_out, dev), ld_out,
        _table(lse, "lse", f32, (batch, heads, seq_len), dev),
        _rows(dout, "dout", bf, rows, n, ld_dout, dev), ld_dout, _rows(dq, "dq", bf, rows, n, ld_d, dev),
        _rows(dk, "dk", bf, rows, n, ld_d, dev), _rows(dv, "dv", bf, rows, n, ld_d, dev), ld_d,
        _arg(work, "work", f32, rows * heads, dev), batch, heads, seq_len, window, m, st))
