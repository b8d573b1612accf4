"""Python binding of libyoco.so, the B200 (sm_100a) attention core of the
YOCO / YOCO++ decoder-decoder architecture.

Argument marshalling only: every function passes torch CUDA tensors as raw
device pointers, plus the current CUDA stream, to the C ABI declared in
include/yoco.h, and raises YocoError on a non-OK status.  Every computation
runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing a function fails loudly when libyoco.so is missing.

Entry points (same names as the C ABI, without the ``yoco_`` prefix):
kv_project_blend, swa_prefill, swa_decode, cross_prefill, cross_decode,
attention_prefill,
gret_prefill, gret_decode, kv_quantize_i8, cross_decode_i8,
rope (with rope_config), cross_decode_tree, swa_decode_tree, cross_tree_commit,
swa_tree_commit,
plus linear, workspace sizes, cache_bytes, device_status and the test-only
debug_tile_schedule.
"""
import ctypes
import functools
import os

import torch

__all__ = ["YocoError", "load", "lib_path", "kv_project_blend", "linear", "swa_prefill",
           "swa_decode", "swa_decode_step", "swa_decode_step_workspace_size", "cross_prefill",
           "cross_decode", "cross_decode_workspace_size",
           "swa_decode_workspace_size", "cache_bytes", "device_status", "launch_count", "AttnCfg",
           "debug_tile_schedule", "SCHEDULE_PREFILL", "SCHEDULE_DECODE", "gret_prefill", "gret_decode",
           "kv_i8_row_bytes", "kv_quantize_i8", "cross_decode_i8",
           "attention_prefill", "debug_exp2_poly", "gret_prefill_workspace_size",
           "RopeCfg", "rope_config", "rope", "cross_decode_tree", "cross_decode_tree_workspace_size",
           "swa_decode_tree", "swa_decode_tree_workspace_size", "cross_tree_commit", "swa_tree_commit"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = range(6)
BF16, FP32 = 0, 1
SCHEDULE_PREFILL, SCHEDULE_DECODE = 0, 1
_DT = {torch.bfloat16: BF16, torch.float32: FP32}


class YocoError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _LIB.yoco_status_string(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


class AttnCfg(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class RopeCfg(ctypes.Structure):
    """yoco_rope_cfg: what yoco_rope turns by (rope_config fills one)."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("mscale", ctypes.c_double),
                ("inv_freq", ctypes.c_double * 64)]


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


def lib_path():
    return os.path.join(_HERE, "libyoco.so")


def load():
    """Load libyoco.so (built in-tree by shared_kv_decoder_b200.build)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libyoco.so not found at {path}; build it with "
                           "`python -m shared_kv_decoder_b200.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    f64 = ctypes.c_double
    cfgp = ctypes.POINTER(AttnCfg)
    st = ctypes.c_int
    sigs = {
        "yoco_kv_project_blend": (st, [vp, i64, i32, vp, i32, f32, vp, vp, f32, f32, vp, vp, vp,
                                       cfgp, vp]),
        "yoco_linear": (st, [vp, i64, i32, vp, i32, i32, f32, vp, f32, vp, i32, vp]),
        "yoco_swa_prefill": (st, [vp, vp, vp, i32, i64, i32, vp, vp, vp, vp, vp, cfgp, vp]),
        "yoco_swa_decode": (st, [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, cfgp, vp]),
        "yoco_swa_decode_step": (st, [vp, i32, vp, i32, f32, vp, vp, f32, f32, vp, vp, i32, i32, vp, vp, vp,
                                      vp, vp, vp, vp, sz, cfgp, vp]),
        "yoco_swa_decode_step_workspace_size": (sz, [i32, i32, cfgp]),
        "yoco_cross_prefill": (st, [vp, vp, vp, i32, i64, i64, i64, vp, vp, cfgp, vp]),
        "yoco_attention_prefill": (st, [vp, vp, vp, i32, i64, i64, i64, i32, vp, vp, cfgp, vp]),
        "yoco_cross_decode": (st, [vp, vp, vp, i64, vp, vp, i32, i64, vp, vp, vp, sz, cfgp, vp]),
        "yoco_cross_decode_static": (st, [vp, vp, vp, i64, vp, vp, i32, i64, vp, vp, cfgp, vp]),
        "yoco_cross_decode_workspace_size": (sz, [i32, i64, cfgp]),
        "yoco_swa_decode_workspace_size": (sz, [i32, i32, cfgp]),
        "yoco_cache_bytes": (ctypes.c_double, [i32, i32, i64, cfgp]),
        "yoco_gret_prefill": (st, [vp, vp, vp, vp, i32, i64, f32, vp, vp, vp, sz, cfgp, vp]),
        "yoco_gret_prefill_workspace_size": (sz, [i32, i64, cfgp]),
        "yoco_kv_i8_row_bytes": (i64, [cfgp]),
        "yoco_kv_quantize_i8": (st, [vp, vp, i64, vp, vp, vp, cfgp, vp]),
        "yoco_cross_decode_i8": (st, [vp, vp, vp, i64, vp, vp, i32, i64, vp, vp, vp, sz, cfgp, vp]),
        "yoco_gret_decode": (st, [vp, vp, vp, vp, i32, f32, vp, vp, cfgp, vp]),
        "yoco_rope_init": (st, [ctypes.POINTER(RopeCfg), i32, i32, f64, i32, f64, f64, f64, f64, f64]),
        "yoco_rope": (st, [vp, vp, i32, i64, vp, i64, i32, vp, vp, ctypes.POINTER(RopeCfg), cfgp, vp]),
        "yoco_cross_decode_tree": (st, [vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, i32, i32, i64, vp, vp, vp, sz, cfgp,
                                        vp]),
        "yoco_cross_decode_tree_workspace_size": (sz, [i32, i32, i64, cfgp]),
        "yoco_swa_decode_tree": (st, [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, cfgp, vp]),
        "yoco_swa_decode_tree_workspace_size": (sz, [i32, i32, i32, cfgp]),
        "yoco_cross_tree_commit": (st, [vp, vp, vp, vp, i32, i32, vp, vp, i64, vp, vp, vp, vp, cfgp, vp]),
        "yoco_swa_tree_commit": (st, [vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, cfgp, vp]),
        "yoco_debug_tile_schedule": (st, [i32, cfgp, i32, i64, i64, i64, i32, vp, vp, i64, i32, vp,
                                          i64, ctypes.POINTER(ctypes.c_int64)]),
        "yoco_get_device_status": (st, [vp]),
        "yoco_debug_wait_timeout_probe": (st, [vp]),
        "yoco_debug_exp2_poly": (st, [vp, vp, i64, vp]),
        "yoco_status_string": (ctypes.c_char_p, [st]),
        "yoco_version": (ctypes.c_char_p, []),
        "yoco_launch_count": (ctypes.c_uint64, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = L
    return L


def _check(status, where):
    if status != OK:
        raise YocoError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("libyoco takes CUDA tensors only")
            if not t.is_contiguous():
                raise ValueError("libyoco takes contiguous tensors only")


def _cfg(Hq, Hkv, D, dtype, scale=0.0):
    return AttnCfg(int(Hq), int(Hkv), int(D), float(scale), _DT[dtype])


def kv_project_blend(x, w_kv, Hkv, D, k_base=None, v_base=None, w_k=0.0, w_v=0.0,
                     dst_rows=None, k_out=None, v_out=None, apply_ln=True, eps=1e-5):
    """[K | V] = LN(x) W_kv^T (+ w_k K_base, + w_v V_base), fused epilogue.
    x [n, d]; w_kv [2*Hkv*D, d]; bases [n, Hkv, D]; returns (k_out, v_out)."""
    L = load()
    n, d = x.shape
    if k_out is None:
        k_out = torch.empty((n, Hkv, D), dtype=x.dtype, device=x.device)
    if v_out is None:
        v_out = torch.empty((n, Hkv, D), dtype=x.dtype, device=x.device)
    _dev(x, w_kv, k_base, v_base, dst_rows, k_out, v_out)
    cfg = _cfg(Hkv, Hkv, D, x.dtype)
    _check(L.yoco_kv_project_blend(_ptr(x), n, d, _ptr(w_kv), int(bool(apply_ln)), eps,
                                   _ptr(k_base), _ptr(v_base), float(w_k), float(w_v),
                                   _ptr(dst_rows), _ptr(k_out), _ptr(v_out), ctypes.byref(cfg),
                                   _stream()), "yoco_kv_project_blend")
    return k_out, v_out


def linear(x, w, base=None, base_w=1.0, apply_ln=False, eps=1e-5, out=None):
    """out = N(x) W^T + base_w * base.  x [n, d_in]; w [d_out, d_in]."""
    L = load()
    n, d_in = x.shape
    d_out = w.shape[0]
    if out is None:
        out = torch.empty((n, d_out), dtype=x.dtype, device=x.device)
    _dev(x, w, base, out)
    _check(L.yoco_linear(_ptr(x), n, d_in, _ptr(w), d_out, int(bool(apply_ln)), eps, _ptr(base),
                         float(base_w), _ptr(out), _DT[x.dtype], _stream()), "yoco_linear")
    return out


def swa_prefill(q, k, v, window, ring=None, want_lse=False, scale=0.0, o=None):
    """Sliding-window prefill.  q [B, T, Hq, D]; k, v [B, T, Hkv, D].
    ring: None, or a tuple (ring_k, ring_v, slot_pos) to fill.
    Returns o (and lse [B, Hq, T] when want_lse)."""
    L = load()
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    if o is None:
        o = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device) if want_lse else None
    rk, rv, sp = ring if ring is not None else (None, None, None)
    _dev(q, k, v, o, lse, rk, rv, sp)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_swa_prefill(_ptr(q), _ptr(k), _ptr(v), B, T, int(window), _ptr(o), _ptr(lse),
                              _ptr(rk), _ptr(rv), _ptr(sp), ctypes.byref(cfg), _stream()),
           "yoco_swa_prefill")
    return (o, lse) if want_lse else o


def swa_decode_workspace_size(B, window, Hq, Hkv, D, dtype):
    cfg = _cfg(Hq, Hkv, D, dtype)
    return int(load().yoco_swa_decode_workspace_size(B, window, ctypes.byref(cfg)))


def swa_decode(q, k_new, v_new, pos, ring_k, ring_v, slot_pos, window, workspace=None,
               scale=0.0, o=None):
    """One sliding-window decode step.  q [B, Hq, D]; k_new, v_new [B, Hkv, D];
    pos int64 [B]; ring_k, ring_v [B, window, Hkv, D]; slot_pos int32 [B, window]."""
    L = load()
    B, Hq, D = q.shape
    Hkv = k_new.shape[1]
    if workspace is None:
        workspace = torch.empty(swa_decode_workspace_size(B, window, Hq, Hkv, D, q.dtype),
                                dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    _dev(q, k_new, v_new, pos, ring_k, ring_v, slot_pos, o, workspace)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_swa_decode(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(pos), B, int(window),
                             _ptr(ring_k), _ptr(ring_v), _ptr(slot_pos), _ptr(o), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), ctypes.byref(cfg),
                             _stream()), "yoco_swa_decode")
    return o


def swa_decode_step_workspace_size(B, window, Hq, Hkv, D, dtype):
    cfg = _cfg(Hq, Hkv, D, dtype)
    return int(load().yoco_swa_decode_step_workspace_size(B, window, ctypes.byref(cfg)))


def swa_decode_step(x, w_kv, q, pos, ring_k, ring_v, slot_pos, window, k_base=None, v_base=None,
                    w_k=0.0, w_v=0.0, apply_ln=True, eps=1e-5, o=None, k_out=None, v_out=None,
                    workspace=None, scale=0.0):
    """One self-decoder decode step: kv_project_blend of the B new tokens, then
    swa_decode with that K/V.  x [B, d]; w_kv [2*Hkv*D, d]; q [B, Hq, D];
    pos int64 [B]; ring_k, ring_v [B, window, Hkv, D]; slot_pos int32 [B, window];
    k_out / v_out [B, Hkv, D] (optional) receive the blended new K / V."""
    L = load()
    B, Hq, D = q.shape
    Hkv = ring_k.shape[2]
    d = x.shape[1]
    if workspace is None:
        workspace = torch.empty(swa_decode_step_workspace_size(B, window, Hq, Hkv, D, q.dtype),
                                dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    _dev(x, w_kv, q, pos, ring_k, ring_v, slot_pos, k_base, v_base, o, k_out, v_out, workspace)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_swa_decode_step(_ptr(x), d, _ptr(w_kv), int(bool(apply_ln)), eps, _ptr(k_base),
                                  _ptr(v_base), float(w_k), float(w_v), _ptr(q), _ptr(pos), B, int(window),
                                  _ptr(ring_k), _ptr(ring_v), _ptr(slot_pos), _ptr(o), _ptr(k_out),
                                  _ptr(v_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  ctypes.byref(cfg), _stream()), "yoco_swa_decode_step")
    return o


def cross_prefill(q, k, v, q_pos0=0, want_lse=False, scale=0.0, o=None):
    """Causal cross-attention over the shared KV.  q [B, Tq, Hq, D];
    k, v [B, Tkv, Hkv, D]; query row i at absolute position q_pos0 + i."""
    L = load()
    B, Tq, Hq, D = q.shape
    Tkv, Hkv = k.shape[1], k.shape[2]
    if o is None:
        o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if want_lse else None
    _dev(q, k, v, o, lse)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_cross_prefill(_ptr(q), _ptr(k), _ptr(v), B, Tq, Tkv, int(q_pos0), _ptr(o),
                                _ptr(lse), ctypes.byref(cfg), _stream()), "yoco_cross_prefill")
    return (o, lse) if want_lse else o


def cross_decode_workspace_size(B, max_len, Hq, Hkv, D, dtype):
    cfg = _cfg(Hq, Hkv, D, dtype)
    return int(load().yoco_cross_decode_workspace_size(B, max_len, ctypes.byref(cfg)))


def cross_decode(q, k_cache, v_cache, seq_start, seq_len, max_len, workspace=None,
                 want_lse=False, scale=0.0, o=None):
    """One cross-decoder decode step over the packed shared cache.
    q [B, Hq, D]; caches [rows, Hkv, D]; seq_start int64 [B]; seq_len int32 [B]."""
    L = load()
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if workspace is None:
        workspace = torch.empty(cross_decode_workspace_size(B, max_len, Hq, Hkv, D, q.dtype),
                                dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if want_lse else None
    _dev(q, k_cache, v_cache, seq_start, seq_len, o, lse, workspace)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_cross_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(seq_start),
                               _ptr(seq_len), B, int(max_len), _ptr(o), _ptr(lse),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               ctypes.byref(cfg), _stream()), "yoco_cross_decode")
    return (o, lse) if want_lse else o


def cache_bytes(L_self, window, N, Hkv, D, dtype=torch.bfloat16):
    cfg = _cfg(Hkv, Hkv, D, dtype)
    return float(load().yoco_cache_bytes(L_self, window, N, ctypes.byref(cfg)))


def launch_count():
    """Kernels launched by the library so far in this process."""
    return int(load().yoco_launch_count())


def device_status():
    """Synchronise the current stream and return the device status code."""
    return int(load().yoco_get_device_status(_stream()))


def debug_tile_schedule(kind, Hq, Hkv, D, dtype=torch.bfloat16, B=1, Tq=0, Tkv=0, q_pos0=0, window=0,
                        seq_start=None, seq_len=None, max_len=1, n_cta=0):
    """The kernels' work plan, computed on the host (test-only; see
    yoco_debug_tile_schedule).  Returns an int64 numpy array [n, 6]:
    prefill {cta, b, head, query tile, KV tile, masked};
    decode {cta, b, split, first row, tokens, stages}.  seq_start / seq_len
    are host sequences (decode only)."""
    import numpy as np
    L = load()
    cfg = _cfg(Hq, Hkv, D, dtype)
    ss = sl = None
    if kind == SCHEDULE_DECODE:
        ss = np.ascontiguousarray(np.asarray(seq_start, dtype=np.int64))
        sl = np.ascontiguousarray(np.asarray(seq_len, dtype=np.int32))
    n = ctypes.c_int64(0)
    args = lambda rec, cap: (int(kind), ctypes.byref(cfg), int(B), int(Tq), int(Tkv), int(q_pos0),
                             int(window), None if ss is None else ss.ctypes.data_as(ctypes.c_void_p),
                             None if sl is None else sl.ctypes.data_as(ctypes.c_void_p), int(max_len),
                             int(n_cta), rec, cap, ctypes.byref(n))
    _check(L.yoco_debug_tile_schedule(*args(None, 0)), "yoco_debug_tile_schedule")
    out = np.zeros((n.value, 6), dtype=np.int64)
    _check(L.yoco_debug_tile_schedule(*args(out.ctypes.data_as(ctypes.c_void_p), n.value)),
           "yoco_debug_tile_schedule")
    return out


def gret_prefill_workspace_size(B, T, H, D, dtype=torch.bfloat16):
    cfg = _cfg(H, H, D, dtype)
    return int(load().yoco_gret_prefill_workspace_size(B, int(T), ctypes.byref(cfg)))


def gret_prefill(q, k, v, g, tau, state=None, scale=0.0, o=None, workspace="auto"):
    """Chunkwise gated retention over a prompt.  q, k, v [B, T, H, D] bf16;
    g [B, T, H] fp32 gate logits; state [B, H, D, D] fp32 initial state,
    overwritten with the final state (None: start from zero).
    workspace: a uint8 CUDA tensor for the split over superchunks, "auto" to
    allocate one of the size the library asks for, or None (no split).
    Returns o."""
    L = load()
    B, T, H, D = q.shape
    if o is None:
        o = torch.empty_like(q)
    if isinstance(workspace, str):
        n = gret_prefill_workspace_size(B, T, H, D, q.dtype)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None
    _dev(q, k, v, g, state, o, workspace)
    cfg = _cfg(H, H, D, q.dtype, scale)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(L.yoco_gret_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), B, T, float(tau), _ptr(state), _ptr(o),
                               _ptr(workspace), ws_bytes, ctypes.byref(cfg), _stream()), "yoco_gret_prefill")
    return o


def gret_decode(q, k, v, g, tau, state, scale=0.0, o=None):
    """One recurrent gated-retention step.  q, k, v [B, H, D]; g [B, H] fp32;
    state [B, H, D, D] fp32, updated in place.  Returns o [B, H, D]."""
    L = load()
    B, H, D = q.shape
    if o is None:
        o = torch.empty_like(q)
    _dev(q, k, v, g, state, o)
    cfg = _cfg(H, H, D, q.dtype, scale)
    _check(L.yoco_gret_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), B, float(tau), _ptr(state), _ptr(o),
                              ctypes.byref(cfg), _stream()), "yoco_gret_decode")
    return o


def kv_i8_row_bytes(Hkv, D):
    """Bytes of one row of an 8-bit K or V cache (codes, then padded scales)."""
    return int(load().yoco_kv_i8_row_bytes(ctypes.byref(_cfg(Hkv, Hkv, D, torch.bfloat16))))


def kv_quantize_i8(k, v, k_i8=None, v_i8=None, dst_rows=None):
    """8-bit quantisation of K, V [n, Hkv, D] into cache rows (uint8 tensors
    [rows, row_bytes]); dst_rows (int64, device) places row i at dst_rows[i].
    Returns (k_i8, v_i8)."""
    L = load()
    n, Hkv, D = k.shape
    rb = kv_i8_row_bytes(Hkv, D)
    if k_i8 is None:
        k_i8 = torch.empty((n, rb), dtype=torch.uint8, device=k.device)
    if v_i8 is None:
        v_i8 = torch.empty((n, rb), dtype=torch.uint8, device=k.device)
    _dev(k, v, dst_rows, k_i8, v_i8)
    cfg = _cfg(Hkv, Hkv, D, k.dtype)
    _check(L.yoco_kv_quantize_i8(_ptr(k), _ptr(v), n, _ptr(dst_rows), _ptr(k_i8), _ptr(v_i8), ctypes.byref(cfg),
                                 _stream()), "yoco_kv_quantize_i8")
    return k_i8, v_i8


def cross_decode_i8(q, k_i8, v_i8, Hkv, seq_start, seq_len, max_len, workspace=None, o=None, want_lse=False,
                    scale=0.0):
    """cross_decode over 8-bit caches (uint8 rows from kv_quantize_i8)."""
    L = load()
    B, Hq, D = q.shape
    if o is None:
        o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if want_lse else None
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    if workspace is None:
        n = L.yoco_cross_decode_workspace_size(B, int(max_len), ctypes.byref(cfg))
        workspace = torch.empty(max(int(n), 16), dtype=torch.uint8, device=q.device)
    _dev(q, k_i8, v_i8, seq_start, seq_len, o, lse, workspace)
    if v_i8.shape != k_i8.shape:
        raise ValueError("k_i8 and v_i8 must have the same shape")
    _check(L.yoco_cross_decode_i8(_ptr(q), _ptr(k_i8), _ptr(v_i8), k_i8.shape[0], _ptr(seq_start), _ptr(seq_len), B,
                                  int(max_len), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                  ctypes.byref(cfg), _stream()), "yoco_cross_decode_i8")
    return (o, lse) if want_lse else o


def attention_prefill(q, k, v, q_pos0=0, window=0, o=None, want_lse=False, scale=0.0):
    """Causal (window 0) or windowed attention of q [B, Tq, Hq, D] over keys
    k, v [B, Tkv, Hkv, D], query row i at key position q_pos0 + i."""
    L = load()
    B, Tq, Hq, D = q.shape
    Tkv, Hkv = k.shape[1], k.shape[2]
    if o is None:
        o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if want_lse else None
    _dev(q, k, v, o, lse)
    cfg = _cfg(Hq, Hkv, D, q.dtype, scale)
    _check(L.yoco_attention_prefill(_ptr(q), _ptr(k), _ptr(v), B, Tq, Tkv, int(q_pos0), int(window), _ptr(o),
                                    _ptr(lse), ctypes.byref(cfg), _stream()), "yoco_attention_prefill")
    return (o, lse) if want_lse else o


def debug_exp2_poly(x, y=None):
    """Test-only: the prefill softmax's polynomial 2^x (the FMA-pipe half of its
    exponentials) applied elementwise to an fp32 CUDA tensor."""
    L = load()
    if y is None:
        y = torch.empty_like(x)
    _dev(x, y)
    if x.dtype != torch.float32 or y.dtype != torch.float32 or y.numel() != x.numel():
        raise ValueError("debug_exp2_poly takes fp32 tensors of one size")
    _check(L.yoco_debug_exp2_poly(_ptr(x), _ptr(y), x.numel(), _stream()), "yoco_debug_exp2_poly")
    return y


# ---------------------------------------------- rotary positions, drafted tokens
def _want(t, name, dtype, shape, device):
    """One tensor argument: its type, shape, device (an index) and layout."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    raise ValueError("libyoco takes contiguous tensors only")


def _cuda_float(t, name):
    """The device index of the tensor that the others go by."""
    if not t.is_cuda:
        raise ValueError("libyoco takes CUDA tensors only")
    if t.dtype not in _DT:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in _DT)}")
    if not t.is_contiguous():
        raise ValueError("libyoco takes contiguous tensors only")
    return t.get_device()


_I32, _I64 = torch.int32, torch.int64


@functools.lru_cache(maxsize=256)
def _cfg_ref(Hq, Hkv, D, dtype, scale=0.0):
    return ctypes.byref(_cfg(Hq, Hkv, D, dtype, scale))


def _addr(t):
    return None if t is None else t.data_ptr()


def _call(device, name, *args):
    """A library call on CUDA device `device` and its current stream."""
    fn = getattr(_LIB or load(), name)
    if device == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != OK:
        raise YocoError(status, name)


def rope_config(rot_dim, theta=10000.0, layout="half", scaling="none", factor=1.0, orig_len=0, beta_fast=32.0,
                beta_slow=1.0, mscale=0.0):
    """The pairs, frequencies and magnitude that rope() turns by.  layout
    "half" (elements i, i + rot_dim / 2) or "interleaved" (2i, 2i + 1); scaling
    "none", "linear", "ntk" or "by_parts" (its mscale 0: 0.1 ln(factor) + 1).
    The returned RopeCfg's inv_freq (radians a position) may be set freely."""
    if layout not in _ROPE_LAYOUTS or scaling not in _ROPE_SCALINGS:
        raise ValueError(f"layout is one of {list(_ROPE_LAYOUTS)}, scaling one of {list(_ROPE_SCALINGS)}")
    cfg = RopeCfg()
    _check(load().yoco_rope_init(ctypes.byref(cfg), int(rot_dim), _ROPE_LAYOUTS[layout], float(theta),
                                 _ROPE_SCALINGS[scaling], float(factor), float(orig_len), float(beta_fast),
                                 float(beta_slow), float(mscale)), "yoco_rope_init")
    return cfg


def rope(q, k, rope_cfg, pos=None, pos0=0, q_out=None, k_out=None, backward=False):
    """Rotary positions.  q [B, T, Hq, D] and k [B, T, Hkv, D], or one token a
    sequence as [B, Hq, D] and [B, Hkv, D]; either may be None.  pos int64
    [B, T] ([B]); None: token t of every sequence is at pos0 + t.  backward: q
    and k are gradients of the rotated Q and K, the result those before it.
    Returns (q_out, k_out), new tensors unless given (q_out = q: in place)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("rope needs q or k")
    device = _cuda_float(x, "q" if q is not None else "k")
    dtype, shape = x.dtype, x.shape
    if len(shape) == 4:
        B, T, Hq, D = shape
        lead = (B, T)
    elif len(shape) == 3:
        B, Hq, D = shape
        T, lead = 1, (B,)
    else:
        raise ValueError("rope takes [B, T, heads, D] or [B, heads, D]")
    Hkv = Hq
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q)
        elif q_out is not q:
            _want(q_out, "q_out", dtype, shape, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        if k is not x:
            Hkv = k.shape[-2] if k.dim() == len(shape) else -1
            _want(k, "k", dtype, (*lead, Hkv, D), device)
        if k_out is None:
            k_out = torch.empty_like(k)
        elif k_out is not k:
            _want(k_out, "k_out", dtype, k.shape, device)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if pos is not None:
        _want(pos, "pos", _I64, lead, device)
    _call(device, "yoco_rope", _addr(q), _addr(k), B, T, _addr(pos), int(pos0), int(bool(backward)), _addr(q_out),
          _addr(k_out), ctypes.byref(rope_cfg), _cfg_ref(Hq, Hkv, D, dtype))
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _tree_ws(device_index, B, N, max_len, Hq, Hkv, D, dtype):
    with torch.cuda.device(device_index):
        return int(load().yoco_cross_decode_tree_workspace_size(B, N, max_len, _cfg_ref(Hq, Hkv, D, dtype)))


def cross_decode_tree_workspace_size(B, N, max_len, Hq, Hkv, D, dtype):
    return int(load().yoco_cross_decode_tree_workspace_size(B, N, int(max_len), _cfg_ref(Hq, Hkv, D, dtype)))


def swa_decode_tree_workspace_size(B, N, window, Hq, Hkv, D, dtype):
    return int(load().yoco_swa_decode_tree_workspace_size(B, N, int(window), _cfg_ref(Hq, Hkv, D, dtype)))


def _tree_args(q, k_nodes, v_nodes, tree_mask, n_nodes, context, workspace, o, want_lse):
    """What both trees check and allocate.  The workspace itself comes last, to be
    kept until the call is on its stream."""
    device = _cuda_float(q, "q")
    if q.dim() != 4 or k_nodes.dim() != 4:
        raise ValueError("q is [B, N, Hq, D], k_nodes and v_nodes [B, N, Hkv, D]")
    dtype, shape = q.dtype, q.shape
    B, N, Hq, D = shape
    Hkv = k_nodes.shape[2]
    nodes = (B, N, Hkv, D)
    _want(k_nodes, "k_nodes", dtype, nodes, device)
    _want(v_nodes, "v_nodes", dtype, nodes, device)
    if tree_mask is not None:
        _want(tree_mask, "tree_mask", torch.uint64 if tree_mask.dtype is torch.uint64 else _I64, (B, N), device)
    if n_nodes is not None:
        _want(n_nodes, "n_nodes", _I32, (B,), device)
    if workspace is None:
        ws_bytes = _tree_ws(device, B, N, context, Hq, Hkv, D, dtype)
        if ws_bytes > 0:
            workspace = q.new_empty(ws_bytes, dtype=torch.uint8)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{device}")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    if o is None:
        o = torch.empty_like(q)
    else:
        _want(o, "o", dtype, shape, device)
    lse = q.new_empty((B, Hq, N), dtype=torch.float32) if want_lse else None
    return B, N, Hq, Hkv, D, device, _addr(workspace), ws_bytes, o, lse, workspace


def cross_decode_tree(q, k_nodes, v_nodes, k_cache, v_cache, seq_start, seq_len, max_len, tree_mask=None,
                      n_nodes=None, workspace=None, want_lse=False, scale=0.0, o=None):
    """Attention of drafted tokens over the packed shared cache.  q [B, N, Hq, D];
    k_nodes, v_nodes [B, N, Hkv, D]; caches [rows, Hkv, D]; seq_start int64 [B];
    seq_len int32 [B] (committed tokens); tree_mask int64 / uint64 [B, N]: bit j
    lets node i see node j (None: a chain); n_nodes int32 [B] or None (N).
    Returns o (and lse [B, Hq, N] when want_lse)."""
    max_len, dtype = int(max_len), q.dtype
    B, N, Hq, Hkv, D, device, ws, ws_bytes, o, lse, keep = _tree_args(q, k_nodes, v_nodes, tree_mask, n_nodes, max_len,
                                                                      workspace, o, want_lse)
    rows = (k_cache.shape[0], Hkv, D)
    _want(k_cache, "k_cache", dtype, rows, device)
    _want(v_cache, "v_cache", dtype, rows, device)
    _want(seq_start, "seq_start", _I64, (B,), device)
    _want(seq_len, "seq_len", _I32, (B,), device)
    _call(device, "yoco_cross_decode_tree", q.data_ptr(), k_nodes.data_ptr(), v_nodes.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), rows[0], seq_start.data_ptr(), seq_len.data_ptr(), _addr(tree_mask), _addr(n_nodes), B, N,
          max_len, o.data_ptr(), _addr(lse), ws, ws_bytes, _cfg_ref(Hq, Hkv, D, dtype, float(scale)))
    return (o, lse) if want_lse else o


def swa_decode_tree(q, k_nodes, v_nodes, node_pos, ring_k, ring_v, slot_pos, window, tree_mask=None, n_nodes=None,
                    workspace=None, want_lse=False, scale=0.0, o=None):
    """Attention of drafted tokens over the sliding-window ring, which is only
    read.  node_pos int64 [B, N]; ring_k, ring_v [B, window, Hkv, D]; slot_pos
    int32 [B, window]; the rest as in cross_decode_tree."""
    W, dtype = int(window), q.dtype
    B, N, Hq, Hkv, D, device, ws, ws_bytes, o, lse, keep = _tree_args(q, k_nodes, v_nodes, tree_mask, n_nodes, W,
                                                                      workspace, o, want_lse)
    ring = (B, W, Hkv, D)
    _want(node_pos, "node_pos", _I64, (B, N), device)
    _want(ring_k, "ring_k", dtype, ring, device)
    _want(ring_v, "ring_v", dtype, ring, device)
    _want(slot_pos, "slot_pos", _I32, (B, W), device)
    _call(device, "yoco_swa_decode_tree", q.data_ptr(), k_nodes.data_ptr(), v_nodes.data_ptr(), node_pos.data_ptr(),
          _addr(tree_mask), _addr(n_nodes), B, N, W, ring_k.data_ptr(), ring_v.data_ptr(), slot_pos.data_ptr(),
          o.data_ptr(), _addr(lse), ws, ws_bytes, _cfg_ref(Hq, Hkv, D, dtype, float(scale)))
    return (o, lse) if want_lse else o


def _commit_args(k_nodes, v_nodes, path, n_path):
    device = _cuda_float(k_nodes, "k_nodes")
    if k_nodes.dim() != 4:
        raise ValueError("k_nodes and v_nodes are [B, N, Hkv, D]")
    B, N = k_nodes.shape[:2]
    _want(v_nodes, "v_nodes", k_nodes.dtype, k_nodes.shape, device)
    _want(path, "path", _I32, (B, N), device)
    _want(n_path, "n_path", _I32, (B,), device)
    return (*k_nodes.shape, device)


def cross_tree_commit(k_nodes, v_nodes, path, n_path, k_cache, v_cache, seq_start, seq_len, seq_cap=None, new_len=None):
    """Appends the accepted nodes path[b][:n_path[b]] (int32 [B, N], [B]) to each
    sequence of the packed cache; seq_cap int32 [B] bounds a sequence's rows.
    Returns new_len int32 [B]; seq_len stays as it is."""
    B, N, Hkv, D, device = _commit_args(k_nodes, v_nodes, path, n_path)
    rows = (k_cache.shape[0], Hkv, D)
    _want(k_cache, "k_cache", k_nodes.dtype, rows, device)
    _want(v_cache, "v_cache", k_nodes.dtype, rows, device)
    _want(seq_start, "seq_start", _I64, (B,), device)
    _want(seq_len, "seq_len", _I32, (B,), device)
    if seq_cap is not None:
        _want(seq_cap, "seq_cap", _I32, (B,), device)
    if new_len is None:
        new_len = torch.empty_like(seq_len)
    else:
        _want(new_len, "new_len", _I32, (B,), device)
    _call(device, "yoco_cross_tree_commit", k_nodes.data_ptr(), v_nodes.data_ptr(), path.data_ptr(), n_path.data_ptr(),
          B, N, k_cache.data_ptr(), v_cache.data_ptr(), rows[0], seq_start.data_ptr(), seq_len.data_ptr(),
          _addr(seq_cap), new_len.data_ptr(), _cfg_ref(Hkv, Hkv, D, k_nodes.dtype))
    return new_len


def swa_tree_commit(k_nodes, v_nodes, node_pos, path, n_path, ring_k, ring_v, slot_pos, window):
    """Pushes the accepted nodes path[b][:n_path[b]] into the ring, in order:
    slot node_pos mod window, slot_pos updated."""
    B, N, Hkv, D, device = _commit_args(k_nodes, v_nodes, path, n_path)
    W = int(window)
    _want(node_pos, "node_pos", _I64, (B, N), device)
    _want(ring_k, "ring_k", k_nodes.dtype, (B, W, Hkv, D), device)
    _want(ring_v, "ring_v", k_nodes.dtype, (B, W, Hkv, D), device)
    _want(slot_pos, "slot_pos", _I32, (B, W), device)
    _call(device, "yoco_swa_tree_commit", k_nodes.data_ptr(), v_nodes.data_ptr(), node_pos.data_ptr(), path.data_ptr(),
          n_path.data_ptr(), B, N, W, ring_k.data_ptr(), ring_v.data_ptr(), slot_pos.data_ptr(),
          _cfg_ref(Hkv, Hkv, D, k_nodes.dtype))
