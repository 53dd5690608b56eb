"""GB300 (sm_103a) FlashAttention-style attention forward.

Python binding of the C ABI declared in ``include/attn.h``: argument
marshalling only.  Every step of the computation runs in the CUDA library
``_build/libattn_fwd_gb300.so`` (built by ``attention_attn_fwd_gb300.build``);
there is no fallback, and every entry point raises ``AttnError`` when the
library is missing.

Layouts follow the host launcher of "Flash Attention in CUDA Tile (cuTile)":
Q, O are [B, Hq, Sq, D] and K, V are [B, Hkv, Skv, D], contiguous.
"""
import contextlib
import ctypes
import math
import os
import struct
import threading

__all__ = [
    "ATTN_F16", "ATTN_BF16", "ATTN_E4M3", "AttnError", "attn_fwd",
    "attn_fwd_window", "attn_fwd_fp8",
    "attn_fwd_splitkv", "attn_fwd_splitkv_window",
    "attn_splitkv_plan", "attn_fwd_splitkv_noalloc",
    "attn_noalloc_scratch_bytes", "attn_status_string", "attn_device_status",
    "attn_stream_status", "attn_selftest_wait_timeout", "attn_dispatch",
    "attn_tile_config", "attn_unit_plan", "attn_version", "attn_bwd",
    "attn_bwd_workspace_bytes",
    "fwd", "fwd_splitkv", "fwd_fp8", "bwd",
    "attn_kv8_append", "attn_kv8_fwd", "attn_kv8_workspace_bytes",
    "attn_kv8_evict",
    "KV8Cache", "kv8_append", "kv8_fwd", "kv8_workspace", "kv8_evict",
    "attn_rope_phase", "attn_qk_rope", "attn_qk_rope_bwd",
    "attn_qk_rope_bwd_workspace_bytes",
    "Rope", "qk_rope", "qk_rope_bwd", "qk_rope_bwd_workspace",
    "attn_prefix_fwd", "attn_prefix_workspace_bytes",
    "attn_selftest_prefix_timeout",
    "PrefixCache", "prefix_fwd", "prefix_workspace",
    "library_path", "load_library",
]

ATTN_F16 = 0
ATTN_BF16 = 1
ATTN_E4M3 = 2

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_ALIGNMENT = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_TIMEOUT = 5

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libattn_fwd_gb300.so")
_lib = None
_lock = threading.Lock()


class AttnError(RuntimeError):
    """A non-OK status from the C ABI, or the library is not available."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


class _Dispatch(ctypes.Structure):
    """attn_dispatch_t of include/attn.h."""
    _fields_ = [(n, ctypes.c_int) for n in (
        "block_m", "block_n", "q_tiles", "paired", "s_buffers", "stages",
        "order", "o_store", "hold_scores", "num_splits", "units",
        "smem_bytes", "merge")] + [("name", ctypes.c_char_p)]


class _KV8(ctypes.Structure):
    """attn_kv8_t of include/attn.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k", "v", "k_scale", "v_scale", "lens")] + [
            (n, ctypes.c_int) for n in ("B", "Hkv", "capacity", "D", "block")]


class _RopeStruct(ctypes.Structure):
    """attn_rope_t of include/attn.h."""
    _fields_ = [("phase", ctypes.c_void_p), ("axis", ctypes.c_void_p)] + [
        (n, ctypes.c_int) for n in ("D", "rot", "axes", "interleaved")]


# attn_heads_t of include/attn.h: pointer, stride_b, stride_s, stride_h.
_heads = struct.Struct("@Pqqq").pack


class _Prefix(ctypes.Structure):
    """attn_prefix_cache_t of include/attn.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "prefix_k", "prefix_v", "prefix_len", "k", "v", "lens")] + [
            (n, ctypes.c_int) for n in ("B", "Hkv", "prefix_capacity",
                                        "capacity", "D")]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the CUDA library (once).  Raises AttnError if it is not built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise AttnError(
                "CUDA library not built (%s); run "
                "`python -m attention_attn_fwd_gb300.build`" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i = ctypes.c_void_p, ctypes.c_int
        ip = ctypes.POINTER(ctypes.c_int)
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                 ctypes.c_float, i, i, i, vp]
        lib.attn_fwd.restype = i
        lib.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                        ctypes.c_float, i, i, i, i, vp]
        lib.attn_fwd_window.restype = i
        lib.attn_status_string.argtypes = [i]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        lib.attn_device_status.restype = i
        lib.attn_tile_config.argtypes = [i, i, i, i, i, i, i, i, i,
                                         ip, ip, ip, ip, ip]
        lib.attn_tile_config.restype = i
        lib.attn_version.argtypes = []
        lib.attn_version.restype = i
        sz = ctypes.c_size_t
        lib.attn_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                         ctypes.c_float, i, i, i, i, vp, sz,
                                         vp]
        lib.attn_fwd_splitkv.restype = i
        lib.attn_fwd_splitkv_window.argtypes = [vp, vp, vp, vp, vp, i, i, i,
                                                i, i, i, ctypes.c_float, i, i,
                                                i, i, i, vp, sz, vp]
        lib.attn_fwd_splitkv_window.restype = i
        lib.attn_splitkv_plan.argtypes = [i, i, i, i, i, i, i, i, i, ip,
                                          ctypes.POINTER(sz)]
        lib.attn_splitkv_plan.restype = i
        lib.attn_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i,
                                                 i, i, i, ctypes.c_float, i,
                                                 i, i, i, vp]
        lib.attn_fwd_splitkv_noalloc.restype = i
        lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i,
                                 i, i, i, ctypes.c_float, i, i, i, i, vp, sz,
                                 vp]
        lib.attn_bwd.restype = i
        lib.attn_bwd_workspace_bytes.argtypes = [i, i, i]
        lib.attn_bwd_workspace_bytes.restype = sz
        f = ctypes.c_float
        lib.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                     f, f, f, f, i, i, i, i, vp, sz, vp]
        lib.attn_fwd_fp8.restype = i
        lib.attn_noalloc_scratch_bytes.argtypes = []
        lib.attn_noalloc_scratch_bytes.restype = sz
        lib.attn_dispatch.argtypes = [i, i, i, i, i, i, i, i, i, i, i,
                                      ctypes.POINTER(_Dispatch)]
        lib.attn_dispatch.restype = i
        lp = ctypes.POINTER(ctypes.c_longlong)
        lib.attn_unit_plan.argtypes = [i] * 10 + [ip, lp, lp, ip, ip]
        lib.attn_unit_plan.restype = i
        lib.attn_stream_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
        lib.attn_stream_status.restype = i
        lib.attn_selftest_wait_timeout.argtypes = [
            vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, i, i,
            ctypes.c_ulonglong, vp]
        lib.attn_selftest_wait_timeout.restype = i
        cp = ctypes.POINTER(_KV8)
        lib.attn_kv8_append.argtypes = [cp, vp, vp, i, vp, i, vp]
        lib.attn_kv8_append.restype = i
        lib.attn_kv8_fwd.argtypes = [cp, vp, vp, vp, vp, i, i, vp, f, i, i,
                                     vp, sz, vp]
        lib.attn_kv8_fwd.restype = i
        lib.attn_kv8_workspace_bytes.argtypes = [i] * 7
        lib.attn_kv8_workspace_bytes.restype = sz
        lib.attn_kv8_evict.argtypes = [cp, cp, vp, vp, i, i, vp, vp]
        lib.attn_kv8_evict.restype = i
        # (attn_heads_t's are handed over as their packed bytes.)
        rp, hp = ctypes.POINTER(_RopeStruct), ctypes.c_char_p
        lib.attn_rope_phase.argtypes = [ctypes.POINTER(ctypes.c_double), i,
                                        ctypes.POINTER(ctypes.c_ulonglong)]
        lib.attn_rope_phase.restype = i
        lib.attn_qk_rope.argtypes = [rp, hp, hp, hp, vp, vp, i, f, vp, vp, vp,
                                     vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.attn_qk_rope.restype = i
        lib.attn_qk_rope_bwd.argtypes = [rp, vp, vp, vp, hp, hp, vp, vp, i, f,
                                         vp, vp, hp, hp, hp, vp, vp, i, i, i,
                                         i, i, vp, sz, vp]
        lib.attn_qk_rope_bwd.restype = i
        lib.attn_qk_rope_bwd_workspace_bytes.argtypes = [i]
        lib.attn_qk_rope_bwd_workspace_bytes.restype = sz
        lib.attn_prefix_fwd.argtypes = [ctypes.POINTER(_Prefix), vp, vp, vp, i,
                                        i, vp, f, i, i, vp, sz, vp]
        lib.attn_prefix_fwd.restype = i
        lib.attn_selftest_prefix_timeout.argtypes = [
            *lib.attn_prefix_fwd.argtypes[:-1], i, i, ctypes.c_ulonglong, vp]
        lib.attn_selftest_prefix_timeout.restype = i
        lib.attn_prefix_workspace_bytes.argtypes = [i] * 7
        lib.attn_prefix_workspace_bytes.restype = sz
        _lib = lib
        return lib


def attn_fwd(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale, causal,
             input_pos, dtype, stream) -> int:
    """Raw C-ABI call; pointers and the stream are integers (0 = NULL)."""
    return int(load_library().attn_fwd(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(dtype),
        stream or None))


def attn_fwd_window(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale, causal,
                    input_pos, window, dtype, stream) -> int:
    """Raw C-ABI call with a causal sliding window of ``window`` keys."""
    return int(load_library().attn_fwd_window(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(window),
        int(dtype), stream or None))


def attn_fwd_fp8(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale, q_descale,
                 k_descale, v_descale, causal, input_pos, window, num_splits,
                 workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI call with E4M3 inputs and a bfloat16 O."""
    return int(load_library().attn_fwd_fp8(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), float(q_descale), float(k_descale),
        float(v_descale), int(causal), int(input_pos), int(window),
        int(num_splits), workspace or None, int(workspace_bytes),
        stream or None))


def attn_fwd_splitkv_window(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale,
                            causal, input_pos, window, dtype, num_splits,
                            workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI call of the split-KV forward with a sliding window."""
    return int(load_library().attn_fwd_splitkv_window(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(window),
        int(dtype), int(num_splits), workspace or None, int(workspace_bytes),
        stream or None))


def attn_fwd_splitkv(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale, causal,
                     input_pos, dtype, num_splits, workspace, workspace_bytes,
                     stream) -> int:
    """Raw C-ABI call of the split-KV forward; pointers are integers."""
    return int(load_library().attn_fwd_splitkv(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(dtype),
        int(num_splits), workspace or None, int(workspace_bytes),
        stream or None))


def attn_fwd_splitkv_noalloc(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D, scale,
                             causal, input_pos, dtype, num_splits,
                             stream) -> int:
    """Raw C-ABI call of the split-KV forward that uses the library's fixed
    scratch array instead of a workspace (for callers that cannot allocate
    device memory); pointers are integers."""
    return int(load_library().attn_fwd_splitkv_noalloc(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(dtype),
        int(num_splits), stream or None))


def attn_bwd(Q, K, V, O, LSE, dO, dQ, dK, dV, B, Hq, Hkv, Sq, Skv, D, scale,
             causal, input_pos, window, dtype, workspace, workspace_bytes,
             stream) -> int:
    """Raw C-ABI call of the backward pass; pointers are integers."""
    return int(load_library().attn_bwd(
        Q or None, K or None, V or None, O or None, LSE or None, dO or None,
        dQ or None, dK or None, dV or None, B, Hq, Hkv, Sq, Skv, D,
        float(scale), int(causal), int(input_pos), int(window), int(dtype),
        workspace or None, int(workspace_bytes), stream or None))


def attn_bwd_workspace_bytes(B, Hq, Sq) -> int:
    return int(load_library().attn_bwd_workspace_bytes(B, Hq, Sq))


def attn_noalloc_scratch_bytes() -> int:
    return int(load_library().attn_noalloc_scratch_bytes())


def attn_splitkv_plan(B, Hq, Hkv, Sq, Skv, D, causal, input_pos, dtype,
                      num_splits=0):
    """(num_splits, workspace_bytes) attn_fwd_splitkv accepts."""
    ns = ctypes.c_int(int(num_splits))
    ws = ctypes.c_size_t(0)
    st = int(load_library().attn_splitkv_plan(
        B, Hq, Hkv, Sq, Skv, D, int(causal), int(input_pos), int(dtype),
        ctypes.byref(ns), ctypes.byref(ws)))
    if st != ATTN_OK:
        raise AttnError("attn_splitkv_plan: " + attn_status_string(st), st)
    return ns.value, ws.value


def attn_status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def attn_device_status():
    """(status, code): synchronises the device and clears the status word."""
    code = ctypes.c_uint(0)
    st = int(load_library().attn_device_status(ctypes.byref(code)))
    return st, int(code.value)


def attn_stream_status(stream=0):
    """(status, code) of the device status word, read after the work on
    ``stream`` (an integer handle, 0 = the legacy default stream) and
    cleared of the bits it reports."""
    code = ctypes.c_uint(0)
    st = int(load_library().attn_stream_status(stream or None,
                                                ctypes.byref(code)))
    return st, int(code.value)


def attn_selftest_wait_timeout(Q, K, V, O, LSE, B, Hq, Hkv, Sq, Skv, D,
                               scale, causal, input_pos, dtype, timeout_ns,
                               stream) -> int:
    """Raw C-ABI call of the bounded-wait self-test launch (a forward whose
    first CTA withholds its first K tile; waits give up after
    ``timeout_ns``)."""
    return int(load_library().attn_selftest_wait_timeout(
        Q or None, K or None, V or None, O or None, LSE or None, B, Hq, Hkv,
        Sq, Skv, D, float(scale), int(causal), int(input_pos), int(dtype),
        int(timeout_ns), stream or None))


def attn_tile_config(B, Hq, Hkv, Sq, Skv, D, causal, input_pos, dtype):
    """Tile configuration attn_fwd would launch, as a dict (host only)."""
    out = [ctypes.c_int(0) for _ in range(5)]
    st = int(load_library().attn_tile_config(
        B, Hq, Hkv, Sq, Skv, D, int(causal), int(input_pos), int(dtype),
        *[ctypes.byref(o) for o in out]))
    if st != ATTN_OK:
        raise AttnError("attn_tile_config: " + attn_status_string(st), st)
    keys = ("block_m", "block_n", "stages", "grid", "smem_bytes")
    return {k: o.value for k, o in zip(keys, out)}


def attn_dispatch(B, Hq, Hkv, Sq, Skv, D, causal, input_pos, dtype,
                  window=0, num_splits=0):
    """The forward dispatch-table entry for these arguments, as a dict
    (host only)."""
    d = _Dispatch()
    st = int(load_library().attn_dispatch(
        B, Hq, Hkv, Sq, Skv, D, int(causal), int(input_pos), int(window),
        int(dtype), int(num_splits), ctypes.byref(d)))
    if st != ATTN_OK:
        raise AttnError("attn_dispatch: " + attn_status_string(st), st)
    out = {n: getattr(d, n) for n, _ in _Dispatch._fields_}
    out["name"] = d.name.decode()
    return out


def attn_unit_plan(B, Hq, Hkv, Sq, Skv, D, causal, input_pos, grid,
                   window=0):
    """How a one-pass forward call assigns its units to `grid` CTAs (host
    only): dict with planned, work_max, work_rounds (half K/V steps) and,
    when planned, cta_units (one list of unit indices per CTA)."""
    lib = load_library()
    planned = ctypes.c_int(0)
    wmax, wrounds = ctypes.c_longlong(0), ctypes.c_longlong(0)
    d = attn_dispatch(B, Hq, Hkv, Sq, Skv, D, causal, input_pos, ATTN_BF16,
                      window=window)
    n = d["units"]
    g = max(1, min(n, grid))
    order = (ctypes.c_int * max(1, n))()
    start = (ctypes.c_int * (g + 1))()
    st = int(lib.attn_unit_plan(
        B, Hq, Hkv, Sq, Skv, D, int(causal), int(input_pos), int(window),
        int(grid), ctypes.byref(planned), ctypes.byref(wmax),
        ctypes.byref(wrounds), order, start))
    if st != ATTN_OK:
        raise AttnError("attn_unit_plan: " + attn_status_string(st), st)
    out = {"planned": planned.value, "work_max": wmax.value,
           "work_rounds": wrounds.value, "units": n}
    if planned.value:
        out["cta_units"] = [list(order[start[c]:start[c + 1]])
                            for c in range(g)]
    return out


def attn_kv8_append(cache, K, V, Sq, new_lens, dtype, stream) -> int:
    """Raw C-ABI call; ``cache`` is a ``KV8Cache``, pointers are integers."""
    return int(load_library().attn_kv8_append(
        cache.struct, K or None, V or None, Sq, new_lens or None, int(dtype),
        stream or None))


def attn_kv8_fwd(cache, Q, O, LSE, weights, Hq, Sq, new_lens, scale, causal,
                 dtype, workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI call; ``cache`` is a ``KV8Cache``, pointers are integers."""
    return int(load_library().attn_kv8_fwd(
        cache.struct, Q or None, O or None, LSE or None, weights or None, Hq,
        Sq, new_lens or None, float(scale), int(causal), int(dtype),
        workspace or None, int(workspace_bytes), stream or None))


def attn_kv8_workspace_bytes(B, Hq, Hkv, Sq, capacity, D, weights) -> int:
    return int(load_library().attn_kv8_workspace_bytes(
        B, Hq, Hkv, Sq, capacity, D, int(bool(weights))))


def attn_kv8_evict(src, dst, weights, dst_weights, keep, recent, indices,
                   stream) -> int:
    """Raw C-ABI call; ``src`` and ``dst`` are ``KV8Cache``s."""
    return int(load_library().attn_kv8_evict(
        src.struct, dst.struct, weights or None, dst_weights or None, keep,
        recent, indices or None, stream or None))


def attn_rope_phase(freq):
    """Phases (a list of integers, units of 2^-64 of a turn per position) of
    frequencies in radians per position (host only)."""
    n = len(freq)
    out = (ctypes.c_ulonglong * max(n, 1))()
    st = int(load_library().attn_rope_phase(
        (ctypes.c_double * max(n, 1))(*[float(x) for x in freq]), n, out))
    if st != ATTN_OK:
        raise AttnError("attn_rope_phase: " + attn_status_string(st), st)
    return list(out[:n])


def attn_qk_rope(rope, q, k, v, q_weight, k_weight, weight_f32, eps,
                 positions, lens, new_lens, offset, q_out, k_out, v_out, B, S,
                 Hq, Hkv, capacity, dtype, stream) -> int:
    """Raw C-ABI call; ``rope`` is a ``Rope``, q, k, v are (pointer, stride_b,
    stride_s, stride_h) or None, other pointers integers."""
    return int(load_library().attn_qk_rope(
        rope.struct, *[_heads(*x) if x else None for x in (q, k, v)],
        q_weight or None, k_weight or None, int(weight_f32), float(eps),
        positions or None, lens or None, new_lens or None, offset or None,
        q_out or None, k_out or None, v_out or None, B, S, Hq, Hkv, capacity,
        int(dtype), stream or None))


def attn_qk_rope_bwd(rope, dq_out, dk_out, dv_out, q, k, q_weight, k_weight,
                     weight_f32, eps, positions, offset, dq, dk, dv,
                     dq_weight, dk_weight, B, S, Hq, Hkv, dtype, workspace,
                     workspace_bytes, stream) -> int:
    """Raw C-ABI call; arguments like those of ``attn_qk_rope``."""
    view = [_heads(*x) if x else None for x in (q, k, dq, dk, dv)]
    return int(load_library().attn_qk_rope_bwd(
        rope.struct, dq_out or None, dk_out or None, dv_out or None,
        view[0], view[1], q_weight or None, k_weight or None, int(weight_f32),
        float(eps), positions or None, offset or None, *view[2:],
        dq_weight or None, dk_weight or None, B, S, Hq, Hkv, int(dtype),
        workspace or None, int(workspace_bytes), stream or None))


def attn_qk_rope_bwd_workspace_bytes(D) -> int:
    return int(load_library().attn_qk_rope_bwd_workspace_bytes(D))


def attn_prefix_fwd(cache, Q, O, LSE, Hq, Sq, new_lens, scale, causal, dtype,
                    workspace, workspace_bytes, stream) -> int:
    """Raw C-ABI call; ``cache`` is a ``PrefixCache``, pointers are
    integers."""
    return int(load_library().attn_prefix_fwd(
        cache.struct, Q or None, O or None, LSE or None, Hq, Sq,
        new_lens or None, float(scale), int(causal), int(dtype),
        workspace or None, int(workspace_bytes), stream or None))


def attn_selftest_prefix_timeout(cache, Q, O, LSE, Hq, Sq, new_lens, scale,
                                 causal, dtype, workspace, workspace_bytes,
                                 block, query_rows, timeout_ns,
                                 stream) -> int:
    """Raw C-ABI call of the bounded-wait self-test of ``attn_prefix_fwd``
    (thread block ``block`` waits in vain for a key tile, or with ``query_rows``
    for query rows; waits give up after ``timeout_ns``)."""
    return int(load_library().attn_selftest_prefix_timeout(
        cache.struct, Q or None, O or None, LSE or None, Hq, Sq,
        new_lens or None, float(scale), int(causal), int(dtype),
        workspace or None, int(workspace_bytes), int(block), int(query_rows),
        int(timeout_ns), stream or None))


def attn_prefix_workspace_bytes(B, Hq, Hkv, Sq, prefix_capacity, capacity,
                                D) -> int:
    return int(load_library().attn_prefix_workspace_bytes(
        B, Hq, Hkv, Sq, prefix_capacity, capacity, D))


def attn_version() -> int:
    return int(load_library().attn_version())


def _dtype_code(t):
    import torch
    if t.dtype == torch.float16:
        return ATTN_F16
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise AttnError("dtype must be float16 or bfloat16, got %s" % t.dtype,
                    ATTN_ERR_INVALID_ARG)


def fwd(q, k, v, scale=None, causal=True, input_pos=0, out=None, lse=None,
        need_lse=True, stream=None, window=0):
    """Attention forward on CUDA tensors.

    q [B, Hq, Sq, D], k and v [B, Hkv, Skv, D] (contiguous, same dtype,
    float16 or bfloat16).  ``scale`` defaults to 1/sqrt(D).  Returns
    (O, LSE) with LSE float32 [B, Hq, Sq] (None if ``need_lse`` is False).
    ``window`` > 0 (causal only): the query at position p sees keys
    p - window + 1 .. p.  The kernel is enqueued on ``stream`` (default:
    torch's current stream).
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4:
            raise AttnError("%s must be 4-D [B, H, S, D]" % name,
                            ATTN_ERR_INVALID_ARG)
        if not t.is_cuda:
            raise AttnError("%s must be a CUDA tensor" % name,
                            ATTN_ERR_INVALID_ARG)
        if not t.is_contiguous():
            raise AttnError("%s must be contiguous" % name,
                            ATTN_ERR_INVALID_ARG)
    if not (q.dtype == k.dtype == v.dtype):
        raise AttnError("q, k, v must share a dtype", ATTN_ERR_INVALID_ARG)
    dt = _dtype_code(q)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape):
        raise AttnError("inconsistent q/k/v shapes", ATTN_ERR_INVALID_ARG)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if need_lse and lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device):
        if window:
            st = attn_fwd_window(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                lse.data_ptr() if need_lse else 0, B, Hq, Hkv, Sq, Skv, D,
                scale, causal, input_pos, window, dt, stream.cuda_stream)
        else:
            st = attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          out.data_ptr(), lse.data_ptr() if need_lse else 0,
                          B, Hq, Hkv, Sq, Skv, D, scale, causal, input_pos, dt,
                          stream.cuda_stream)
    if st != ATTN_OK:
        raise AttnError("attn_fwd: " + attn_status_string(st), st)
    return out, (lse if need_lse else None)


def fwd_splitkv(q, k, v, scale=None, causal=True, input_pos=0, num_splits=0,
                workspace=None, out=None, lse=None, need_lse=True,
                stream=None, window=0):
    """Split-KV attention forward (few query rows over a long key range).

    Same tensors and result as ``fwd`` (``window`` included).
    ``num_splits`` <= 0 lets the library choose; ``workspace`` (a CUDA
    tensor of at least the planned size, 256-byte aligned) is allocated
    with torch when not given.
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise AttnError("q, k, v must be 4-D [B, H, S, D]",
                        ATTN_ERR_INVALID_ARG)
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError("q, k, v must be contiguous CUDA tensors",
                            ATTN_ERR_INVALID_ARG)
    dt = _dtype_code(q)
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        splits, ws_bytes = attn_splitkv_plan(B, Hq, Hkv, Sq, Skv, D, causal,
                                             input_pos, dt, num_splits)
        if workspace is None:
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8,
                                    device=q.device)
        if out is None:
            out = torch.empty_like(q)
        if need_lse and lse is None:
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32,
                              device=q.device)
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        ws_args = (splits, workspace.data_ptr(),
                   workspace.numel() * workspace.element_size(),
                   stream.cuda_stream)
        if window:
            st = attn_fwd_splitkv_window(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                lse.data_ptr() if need_lse else 0, B, Hq, Hkv, Sq, Skv, D,
                scale, causal, input_pos, window, dt, *ws_args)
        else:
            st = attn_fwd_splitkv(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                lse.data_ptr() if need_lse else 0, B, Hq, Hkv, Sq, Skv, D,
                scale, causal, input_pos, dt, *ws_args)
    if st != ATTN_OK:
        raise AttnError("attn_fwd_splitkv: " + attn_status_string(st), st)
    return out, (lse if need_lse else None)


def fwd_fp8(q, k, v, scale=None, q_descale=1.0, k_descale=1.0,
            v_descale=1.0, causal=True, input_pos=0, window=0, num_splits=0,
            workspace=None, out=None, lse=None, need_lse=True, stream=None):
    """Attention forward on E4M3 CUDA tensors (torch.float8_e4m3fn, or
    uint8 holding the codes): q [B, Hq, Sq, 128], k and v [B, Hkv, Skv,
    128].  The real inputs are the codes times the per-tensor descale
    factors.  Returns (O bfloat16, LSE float32 or None).  ``num_splits``
    0: one pass; > 0 (or -1 to let the library choose): split-KV with a
    ``workspace`` allocated with torch when not given.
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4 or not t.is_cuda or not t.is_contiguous():
            raise AttnError("%s must be a contiguous 4-D CUDA tensor" % name,
                            ATTN_ERR_INVALID_ARG)
        if t.element_size() != 1 or t.dtype not in (
                getattr(torch, "float8_e4m3fn", None), torch.uint8):
            raise AttnError("%s must hold E4M3 codes (float8_e4m3fn or "
                            "uint8), got %s" % (name, t.dtype),
                            ATTN_ERR_INVALID_ARG)
    B, Hq, Sq, D = q.shape
    Bk, Hkv, Skv, Dk = k.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape):
        raise AttnError("inconsistent q/k/v shapes", ATTN_ERR_INVALID_ARG)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        splits, ws_bytes = 0, 0
        if num_splits:
            splits, ws_bytes = attn_splitkv_plan(
                B, Hq, Hkv, Sq, Skv, D, causal, input_pos, ATTN_E4M3,
                max(num_splits, 0))
            if workspace is None:
                workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8,
                                        device=q.device)
        if out is None:
            out = torch.empty((B, Hq, Sq, D), dtype=torch.bfloat16,
                              device=q.device)
        if need_lse and lse is None:
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32,
                              device=q.device)
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        ws_ptr = workspace.data_ptr() if workspace is not None else 0
        ws_len = (workspace.numel() * workspace.element_size()
                  if workspace is not None else 0)
        st = attn_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          out.data_ptr(), lse.data_ptr() if need_lse else 0,
                          B, Hq, Hkv, Sq, Skv, D, scale, q_descale, k_descale,
                          v_descale, causal, input_pos, window, splits,
                          ws_ptr, ws_len, stream.cuda_stream)
    if st != ATTN_OK:
        raise AttnError("attn_fwd_fp8: " + attn_status_string(st), st)
    return out, (lse if need_lse else None)


def bwd(q, k, v, o, lse, do, scale=None, causal=True, input_pos=0, window=0,
        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward pass on CUDA tensors: (dQ, dK, dV) for upstream gradient
    ``do``, given the forward's ``o`` and ``lse`` for the same arguments."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do),
                    ("lse", lse)):
        if not t.is_cuda or not t.is_contiguous():
            raise AttnError("%s must be a contiguous CUDA tensor" % name,
                            ATTN_ERR_INVALID_ARG)
    dt = _dtype_code(q)
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(q.device):
        if dq is None:
            dq = torch.empty_like(q)
        if dk is None:
            dk = torch.empty_like(k)
        if dv is None:
            dv = torch.empty_like(v)
        if workspace is None:
            workspace = torch.empty(max(attn_bwd_workspace_bytes(B, Hq, Sq), 1),
                                    dtype=torch.uint8, device=q.device)
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        st = attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                      lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
                      dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Sq, Skv, D,
                      scale, causal, input_pos, window, dt,
                      workspace.data_ptr(),
                      workspace.numel() * workspace.element_size(),
                      stream.cuda_stream)
    if st != ATTN_OK:
        raise AttnError("attn_bwd: " + attn_status_string(st), st)
    return dq, dk, dv


class KV8Cache:
    """Handle of a KV cache held in 8 bits (``attn_kv8_t``): E4M3 codes with
    one fp32 scale for each ``block`` tokens of a (batch, K/V head).

    k, v [B, Hkv, capacity, D] (torch.float8_e4m3fn, or uint8 holding the
    codes), k_scale, v_scale float32 [B, Hkv, ceil(capacity / block)], lens
    int32 [B]: the tokens of each sequence, the current step's new ones
    included.  All contiguous, on one CUDA device; the tensors stay the
    caller's and are kept alive by the handle.  Advance ``lens`` first, then
    ``kv8_append`` the new tokens, then ``kv8_fwd``; one ``lens`` tensor may
    serve the caches of all layers.
    """

    def __init__(self, k, v, k_scale, v_scale, lens, block=64):
        import torch
        if k.dim() != 4:
            raise AttnError("k must be 4-D [B, Hkv, capacity, D]",
                            ATTN_ERR_INVALID_ARG)
        B, Hkv, capacity, D = k.shape
        if block not in (16, 32, 64, 128):
            raise AttnError("block must be 16, 32, 64 or 128, got %r"
                            % (block,), ATTN_ERR_UNSUPPORTED)
        nblk = -(-capacity // block)
        codes = (getattr(torch, "float8_e4m3fn", None), torch.uint8)
        for name, t, shape, dtypes in (
                ("k", k, (B, Hkv, capacity, D), codes),
                ("v", v, (B, Hkv, capacity, D), codes),
                ("k_scale", k_scale, (B, Hkv, nblk), (torch.float32,)),
                ("v_scale", v_scale, (B, Hkv, nblk), (torch.float32,)),
                ("lens", lens, (B,), (torch.int32,))):
            if tuple(t.shape) != shape or t.dtype not in dtypes:
                raise AttnError("%s must be %s of %s, got %s of %s" % (
                    name, list(shape), dtypes[0], list(t.shape), t.dtype),
                    ATTN_ERR_INVALID_ARG)
            if not t.is_cuda or t.device != k.device or \
                    not t.is_contiguous():
                raise AttnError("%s must be a contiguous CUDA tensor on k's "
                                "device" % name, ATTN_ERR_INVALID_ARG)
        self.k, self.v = k, v
        self.k_scale, self.v_scale, self.lens = k_scale, v_scale, lens
        self.B, self.Hkv, self.capacity, self.D = B, Hkv, capacity, D
        self.block, self.device = block, k.device
        # What every call needs, looked up once: a decoding step of a small
        # model waits for the host.
        self.dtypes = {torch.float16: ATTN_F16, torch.bfloat16: ATTN_BF16}
        self.int32, self.float32 = torch.int32, torch.float32
        self.lib, self.index = load_library(), k.device.index
        # (torch.cuda.current_device without its check for a first use.)
        self.current_device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.struct = ctypes.pointer(_KV8(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), lens.data_ptr(), B, Hkv, capacity, D, block))

    @classmethod
    def empty(cls, B, Hkv, capacity, D, block=64, lens=None, device="cuda"):
        """A cache of new, uninitialised memory; ``lens`` (zeros unless
        given) may be shared with other caches."""
        import torch
        k, v = (torch.empty((B, Hkv, capacity, D), dtype=torch.uint8,
                            device=device).view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.empty((B, Hkv, -(-capacity // block)),
                              dtype=torch.float32, device=device)
                  for _ in range(2))
        if lens is None:
            lens = torch.zeros(B, dtype=torch.int32, device=device)
        return cls(k, v, ks, vs, lens, block)


def _check_tensor(name, t, shape, dtype):
    """A contiguous tensor of this shape and type.  (Whether it is memory of
    the cache's device is checked behind the C ABI, pointer by pointer.)"""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if t.shape != shape or t.dtype != dtype:
        raise AttnError("%s must be %s of %s, got %s of %s" % (
            name, list(shape), dtype, list(t.shape), t.dtype),
            ATTN_ERR_INVALID_ARG)
    raise AttnError("%s must be contiguous" % name, ATTN_ERR_INVALID_ARG)


def _kv8_dtype(cache, name, t):
    """Code of a 4-D float16 or bfloat16 tensor's element type."""
    dt = cache.dtypes.get(t.dtype)
    if dt is None:
        raise AttnError("%s must be float16 or bfloat16, got %s"
                        % (name, t.dtype), ATTN_ERR_INVALID_ARG)
    if t.dim() != 4:
        raise AttnError("%s must be 4-D [B, H, Sq, D]" % name,
                        ATTN_ERR_INVALID_ARG)
    return dt


def _kv8_call(name, f, cache, stream, *args):
    """Calls a C entry point with ``cache``'s device current, on ``stream``
    or torch's current stream there.  (Switching devices is skipped where
    none is needed, and the stream's handle is taken without building a
    Stream object.)"""
    handle = (cache.raw_stream(cache.index) if stream is None
              else stream.cuda_stream)
    if cache.current_device() == cache.index:
        st = f(cache.struct, *args, handle)
    else:
        import torch
        with torch.cuda.device(cache.index):
            st = f(cache.struct, *args, handle)
    if st != ATTN_OK:
        raise AttnError("%s: %s" % (name, attn_status_string(st)), st)


def _kv8_memory(cache, stream):
    """Context in which a call on ``stream`` allocates: memory of that
    stream's own, so that it is neither still in use by work of the current
    stream nor handed out again there before the call has run."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream)


def kv8_append(cache, k, v, new_lens=None, stream=None):
    """Quantise the K and V of new tokens into an 8-bit cache.

    k, v [B, Hkv, Sq, D] (contiguous, float16 or bfloat16) hold the last
    tokens of each sequence, positions lens - Sq .. lens - 1, or with
    ``new_lens`` (int32 [B]) lens - new_lens .. lens - 1 in the first
    new_lens rows.  ``cache.lens`` already counts them and is not changed.
    """
    dt = _kv8_dtype(cache, "k", k)
    dtype, Sq = k.dtype, k.shape[2]
    shape = (cache.B, cache.Hkv, Sq, cache.D)
    _check_tensor("k", k, shape, dtype)
    _check_tensor("v", v, shape, dtype)
    if new_lens is not None:
        _check_tensor("new_lens", new_lens, (cache.B,), cache.int32)
        new_lens = new_lens.data_ptr()
    _kv8_call("attn_kv8_append", cache.lib.attn_kv8_append, cache, stream,
              k.data_ptr(), v.data_ptr(), Sq, new_lens, dt)


def kv8_workspace(cache, Hq, Sq, weights=False):
    """A workspace tensor for ``kv8_fwd`` calls of Hq heads and Sq rows
    (``weights``: calls that accumulate attention weights; with 16 or fewer
    query rows per K/V head it then holds 4 bytes per row and token of the
    capacity)."""
    import torch
    with torch.cuda.device(cache.device):
        n = attn_kv8_workspace_bytes(cache.B, Hq, cache.Hkv, Sq,
                                     cache.capacity, cache.D, weights)
        return torch.empty(max(n, 1), dtype=torch.uint8, device=cache.device)


def kv8_fwd(cache, q, scale=None, causal=True, new_lens=None, weights=None,
            out=None, lse=None, need_lse=True, workspace=None, stream=None):
    """Attention of q [B, Hq, Sq, D] (contiguous, float16 or bfloat16) over
    an 8-bit cache.  Returns (O, LSE) like ``fwd``.

    Row i of a sequence with n new rows (Sq, or ``new_lens[b]`` of them) sits
    at position lens - n + i and sees the tokens up to it (``causal``), or
    all lens tokens.  Rows that see nothing get O = 0 and LSE = -inf; rows at
    or behind new_lens are left as they are in ``out`` and ``lse``.
    ``weights`` (float32 [B, Hkv, capacity]): the attention weight each token
    receives, summed over rows and the group's heads, is added to it.
    ``workspace``: from ``kv8_workspace``, allocated when not given.  What a
    call on ``stream`` allocates is that stream's memory.  As in ``fwd``,
    ``need_lse=False`` writes no LSE, also where ``lse`` is given.
    """
    dt = _kv8_dtype(cache, "q", q)
    dtype, B, shape = q.dtype, cache.B, q.shape
    _, Hq, Sq, D = shape
    if shape[0] != B or D != cache.D or not q.is_contiguous():
        _check_tensor("q", q, (B, Hq, Sq, cache.D), dtype)
    if out is None:
        import torch
        with _kv8_memory(cache, stream):
            out = torch.empty_like(q)
    else:
        _check_tensor("out", out, shape, dtype)
    if not need_lse:
        lse = None
    elif lse is None:
        import torch
        with _kv8_memory(cache, stream):
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32,
                              device=cache.device)
    else:
        _check_tensor("lse", lse, (B, Hq, Sq), cache.float32)
    if workspace is None:
        with _kv8_memory(cache, stream):
            workspace = kv8_workspace(cache, Hq, Sq, weights is not None)
    elif not workspace.is_contiguous():
        raise AttnError("workspace must be contiguous", ATTN_ERR_INVALID_ARG)
    if new_lens is not None:
        _check_tensor("new_lens", new_lens, (B,), cache.int32)
        new_lens = new_lens.data_ptr()
    if weights is not None:
        _check_tensor("weights", weights, (B, cache.Hkv, cache.capacity),
                      cache.float32)
        weights = weights.data_ptr()
    if scale is None:
        scale = cache.D ** -0.5
    _kv8_call("attn_kv8_fwd", cache.lib.attn_kv8_fwd, cache, stream,
              q.data_ptr(), out.data_ptr(),
              lse.data_ptr() if lse is not None else None, weights, Hq, Sq,
              new_lens, scale, bool(causal), dt, workspace.data_ptr(),
              workspace.nbytes)
    return out, lse


def kv8_evict(cache, weights, keep, recent=0, out=None, out_weights=None,
              indices=None, stream=None):
    """Keep ``keep`` tokens of every longer sequence and head: the
    ``recent`` last ones and those of largest ``weights`` (float32 [B, Hkv,
    capacity]), in their order, as the first tokens of ``out``.

    ``out``: another ``KV8Cache`` of the same heads and block, of its own
    memory, lens included; None: in place (the result shares ``cache``'s
    buffers and has a lens tensor of its own; ``cache.lens`` keeps its
    values).  ``out_weights`` (float32 [B, Hkv, out.capacity]) receives the
    kept tokens' weights, then zeros; in place it defaults to ``weights``
    itself.  Returns (out, out_weights, indices): indices int32 [B, Hkv,
    keep] are the kept tokens' old places, -1 behind the last.  What a call
    on ``stream`` allocates is that stream's memory.
    """
    import torch
    dev = cache.device
    keep, recent = int(keep), int(recent)
    if keep < 1:
        raise AttnError("keep must be at least 1", ATTN_ERR_INVALID_ARG)
    _check_tensor("weights", weights, (cache.B, cache.Hkv, cache.capacity),
                  torch.float32)
    if out is None:
        with _kv8_memory(cache, stream):
            lens = torch.empty_like(cache.lens)
        out = KV8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale, lens,
                       cache.block)
        if out_weights is None:
            out_weights = weights
    elif out.device != dev:
        raise AttnError("out must be on the cache's device",
                        ATTN_ERR_INVALID_ARG)
    shape = (cache.B, cache.Hkv, out.capacity)
    if out_weights is None:
        with _kv8_memory(cache, stream):
            out_weights = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _check_tensor("out_weights", out_weights, shape, torch.float32)
    shape = (cache.B, cache.Hkv, keep)
    if indices is None:
        with _kv8_memory(cache, stream):
            indices = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _check_tensor("indices", indices, shape, torch.int32)
    _kv8_call("attn_kv8_evict", cache.lib.attn_kv8_evict, cache, stream,
              out.struct,
              weights.data_ptr(), out_weights.data_ptr(), keep, recent,
              indices.data_ptr())
    return out, out_weights, indices


class _Handle:
    """Handle whose tensors' addresses are handed over in ``struct``: they are
    changed in place (``cache.lens += 1``); another tensor in the place of one
    would not be the one that calls read, and is refused."""
    held = ()

    def __setattr__(self, name, value):
        if name in self.held and getattr(self, name, value) is not value:
            raise AttnError("%s is changed in place, or a handle made of "
                            "another tensor" % name, ATTN_ERR_INVALID_ARG)
        object.__setattr__(self, name, value)


class Rope(_Handle):
    """Handle of a rotation of heads by position (``attn_rope_t``).

    ``freq``: the rot / 2 pairs' frequencies in radians per position (any
    sequence or tensor of numbers; float64 keeps far positions exact); pair i
    is elements (i, i + rot / 2) of a head's D, or (2i, 2i + 1) with
    ``interleaved``.  ``axes``: the axis of each pair, 0 up (all 0 unless
    given), for positions on several axes (time, height, width).
    """
    held = ("phase", "axis")

    def __init__(self, freq, D, axes=None, interleaved=False, device="cuda"):
        import torch
        freq = [float(x) for x in freq]
        axes = [0] * len(freq) if axes is None else [int(a) for a in axes]
        if D not in (64, 128) or (2 * len(freq)) % 8:
            raise AttnError("D must be 64 or 128 and the rotated elements a "
                            "multiple of 8, got %r and %d"
                            % (D, 2 * len(freq)), ATTN_ERR_UNSUPPORTED)
        if 2 * len(freq) > D or len(axes) != len(freq) or \
                not all(0 <= a < 255 for a in axes):
            raise AttnError("at most D / 2 frequencies, and as many axes "
                            "below 255", ATTN_ERR_INVALID_ARG)
        phase = attn_rope_phase(freq)
        dev = torch.device(device)
        if dev.type != "cuda":
            raise AttnError("device must be a CUDA device",
                            ATTN_ERR_INVALID_ARG)
        signed = [x - (1 << 64) if x >> 63 else x for x in phase]
        self.phase = torch.tensor(signed, dtype=torch.int64, device=dev)
        self.axis = torch.tensor(axes, dtype=torch.uint8, device=dev)
        self.D, self.rot, self.weight_shape = D, 2 * len(freq), (D,)
        self.axes = self.most_axes = max(axes, default=0) + 1
        self.interleaved = bool(interleaved)
        self.device = self.phase.device
        # What every call needs, looked up once.
        self.dtypes = {torch.float16: ATTN_F16, torch.bfloat16: ATTN_BF16}
        self.int32, self.float32 = torch.int32, torch.float32
        self.lib, self.index = load_library(), self.device.index
        self.current_device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.struct = ctypes.pointer(_RopeStruct(
            self.phase.data_ptr() or None, self.axis.data_ptr() or None, D,
            self.rot, self.axes, self.interleaved))

    @classmethod
    def make(cls, D, base=10000.0, rot=None, sections=None, interleaved=False,
             device="cuda"):
        """Frequencies base^(-2i / rot) of rot (D unless given) elements;
        ``sections``: pairs of each axis in turn, rot / 2 in all (positions
        may be given for all of them, also where the last have no pairs)."""
        rot = D if rot is None else rot
        if rot < 0 or rot % 8:
            raise AttnError("the rotated elements must be a multiple of 8, "
                            "got %r" % (rot,), ATTN_ERR_UNSUPPORTED)
        axes = None
        if sections is not None:
            axes = [a for a, n in enumerate(sections) for _ in range(n)]
        rope = cls([base ** (-2.0 * i / rot) for i in range(rot // 2)], D,
                   axes, interleaved, device)
        if sections is not None:
            rope.most_axes = max(rope.axes, len(sections))
        return rope


def _heads_view(name, t, shape, dtype):
    """attn_heads_t of a [B, S, H, D] tensor of any strides but the last."""
    if t.dtype is not dtype or t.shape != shape:
        raise AttnError("%s must be %s of %s, got %s of %s" % (
            name, list(shape), dtype, list(t.shape), t.dtype),
            ATTN_ERR_INVALID_ARG)
    b, s, h, d = t.stride()
    if d != 1:
        raise AttnError("%s's last dimension must be contiguous" % name,
                        ATTN_ERR_INVALID_ARG)
    return _heads(t.data_ptr(), b, s, h)


def _rope_weights(rope, q_weight, k_weight, dtype):
    """(pointer, pointer, whether float32) of the norms' weights."""
    wt = None
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if w.shape != rope.weight_shape or not w.is_contiguous() or \
                (w.dtype is not dtype and w.dtype is not rope.float32):
            raise AttnError("weights must be contiguous [%d] of %s or float32"
                            % (rope.D, dtype), ATTN_ERR_INVALID_ARG)
        if wt is not None and w.dtype is not wt:
            raise AttnError("both weights must be of one type",
                            ATTN_ERR_INVALID_ARG)
        wt = w.dtype
    return (None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(),
            wt is rope.float32)


def _rope_positions(rope, positions, B, S):
    if positions is None:
        return None
    if rope.axes > 1 or positions.dim() == 3:
        n = rope.axes  # (axes behind the last with pairs are not read)
        if positions.dim() == 3 and positions.shape[0] == rope.most_axes:
            n = rope.most_axes
        _check_tensor("positions", positions, (n, B, S), rope.int32)
    else:
        _check_tensor("positions", positions, (B, S), rope.int32)
    return positions.data_ptr()


def _counts(rope, name, t, n):
    """Pointer of an int32 [n] tensor, or None."""
    if t is None:
        return None
    if t.dtype is not rope.int32 or t.shape != (n,) or not t.is_contiguous():
        _check_tensor(name, t, (n,), rope.int32)
    return t.data_ptr()


def _rope_dtype(rope, name, t):
    dt = rope.dtypes.get(t.dtype)
    if dt is None or t.dim() != 4:
        raise AttnError("%s must be 4-D, float16 or bfloat16, got %s of %s"
                        % (name, list(t.shape), t.dtype),
                        ATTN_ERR_INVALID_ARG)
    return dt


def qk_rope(rope, q, k, v=None, q_weight=None, k_weight=None, eps=1e-6,
            positions=None, lens=None, new_lens=None, offset=None, q_out=None,
            k_out=None, v_out=None, stream=None):
    """Norm of queries and keys per head, their rotation by position, and the
    layout that attention reads, in one pass.

    q [B, S, Hq, D], k and v [B, S, Hkv, D] (float16 or bfloat16, any strides
    that are multiples of 8 with a contiguous last dimension: projections'
    outputs, or parts of a packed one).  Returns (q, k, v) as [B, H, S, D];
    v is copied, or None.  ``q_weight``, ``k_weight`` ([D], float32 or q's
    type): weights of the norm x / sqrt(mean(x^2) + eps) * weight; None: not
    normed.  ``positions`` int32 [axes, B, S] (or [B, S]); None: counted, from
    ``offset`` (int32 [1]) up.  ``new_lens`` (int32 [B]): rows of each
    sequence; the outputs behind them are left as they are.

    ``lens`` (int32 [B]): k_out and v_out [B, Hkv, capacity, D] are a cache,
    whose last new_lens (or S) of lens tokens the rows are; without
    ``positions`` they count from there.
    """
    dt = _rope_dtype(rope, "q", q)
    dtype, D = q.dtype, rope.D
    B, S, Hq, _ = q.shape
    Hkv = k.shape[2] if k.dim() == 4 else 0
    shape = (B, S, Hkv, D)
    hq = _heads_view("q", q, (B, S, Hq, D), dtype)
    hk = _heads_view("k", k, shape, dtype)
    hv = None if v is None else _heads_view("v", v, shape, dtype)
    wq, wk, f32 = _rope_weights(rope, q_weight, k_weight, dtype)
    if q_out is None or k_out is None or (v_out is None and v is not None):
        if lens is not None and (k_out is None or
                                 (v_out is None and v is not None)):
            raise AttnError("k_out and v_out must be given with lens",
                            ATTN_ERR_INVALID_ARG)
        import torch
        with _kv8_memory(rope, stream):
            if q_out is None:
                q_out = torch.empty((B, Hq, S, D), dtype=dtype,
                                    device=rope.device)
            if k_out is None:
                k_out = torch.empty((B, Hkv, S, D), dtype=dtype,
                                    device=rope.device)
            if v_out is None and v is not None:
                v_out = torch.empty_like(k_out)
    cap = k_out.shape[2] if k_out.dim() == 4 else 0
    shape = (B, Hkv, cap, D)
    _check_tensor("q_out", q_out, (B, Hq, S, D), dtype)
    _check_tensor("k_out", k_out, shape, dtype)
    if v is None:
        to_v = None
    else:
        _check_tensor("v_out", v_out, shape, dtype)
        to_v = v_out.data_ptr()
    _kv8_call("attn_qk_rope", rope.lib.attn_qk_rope, rope, stream, hq, hk, hv,
              wq, wk, f32, eps, _rope_positions(rope, positions, B, S),
              _counts(rope, "lens", lens, B),
              _counts(rope, "new_lens", new_lens, B),
              _counts(rope, "offset", offset, 1), q_out.data_ptr(),
              k_out.data_ptr(), to_v, B, S, Hq, Hkv, cap, dt)
    return q_out, k_out, v_out


def qk_rope_bwd_workspace(rope):
    """A workspace tensor for ``qk_rope_bwd`` calls of any size."""
    import torch
    with torch.cuda.device(rope.device):
        return torch.empty(attn_qk_rope_bwd_workspace_bytes(rope.D),
                           dtype=torch.uint8, device=rope.device)


def qk_rope_bwd(rope, dq, dk, q=None, k=None, dv=None, q_weight=None,
                k_weight=None, eps=1e-6, positions=None, offset=None,
                dq_out=None, dk_out=None, dv_out=None, dq_weight=None,
                dk_weight=None, workspace=None, stream=None):
    """Backward pass of ``qk_rope`` (without ``lens`` and ``new_lens``).

    dq, dk, dv [B, H, S, D] (contiguous): the gradients of its outputs, as
    ``bwd`` returns them; q, k: its inputs (needed where they were normed).
    Returns (dq, dk, dv, dq_weight, dk_weight): the inputs' gradients [B, S,
    H, D] (``dq_out`` ... may be given, of any strides that qk_rope takes,
    parts of one packed tensor among them) and the weights', float32 [D] or
    None.  ``workspace``: from ``qk_rope_bwd_workspace``, allocated when not
    given.
    """
    dt = _rope_dtype(rope, "dq", dq)
    dtype, D = dq.dtype, rope.D
    B, Hq, S, _ = dq.shape
    Hkv = dk.shape[1] if dk.dim() == 4 else 0
    _check_tensor("dq", dq, (B, Hq, S, D), dtype)
    shape = (B, Hkv, S, D)
    _check_tensor("dk", dk, shape, dtype)
    if dv is not None:
        _check_tensor("dv", dv, shape, dtype)
    wq, wk, f32 = _rope_weights(rope, q_weight, k_weight, dtype)
    if (q is None and wq is not None) or (k is None and wk is not None):
        raise AttnError("what was normed must be given", ATTN_ERR_INVALID_ARG)
    q_shape, k_shape = (B, S, Hq, D), (B, S, Hkv, D)
    hq = None if wq is None else _heads_view("q", q, q_shape, dtype)
    hk = None if wk is None else _heads_view("k", k, k_shape, dtype)
    dw = [None if wq is None else dq_weight, None if wk is None else dk_weight]
    if dq_out is None or dk_out is None or (dv is not None and dv_out is None) \
            or (dw[0] is None and wq) or (dw[1] is None and wk) or \
            (workspace is None and (wq or wk)):
        import torch
        with _kv8_memory(rope, stream):
            if dq_out is None:
                dq_out = torch.empty(q_shape, dtype=dtype, device=rope.device)
            if dk_out is None:
                dk_out = torch.empty(k_shape, dtype=dtype, device=rope.device)
            if dv is not None and dv_out is None:
                dv_out = torch.empty(k_shape, dtype=dtype, device=rope.device)
            for i, w in enumerate((wq, wk)):
                if w and dw[i] is None:
                    dw[i] = torch.empty(D, dtype=torch.float32,
                                        device=rope.device)
            if workspace is None and (wq or wk):
                workspace = qk_rope_bwd_workspace(rope)
    for w in dw:
        if w is not None:
            _check_tensor("weights' gradients", w, (D,), rope.float32)
    if workspace is not None and not workspace.is_contiguous():
        raise AttnError("workspace must be contiguous", ATTN_ERR_INVALID_ARG)
    if dv is None:
        dv_out = from_v = to_v = None
    else:
        from_v = dv.data_ptr()
        to_v = _heads_view("dv_out", dv_out, k_shape, dtype)
    _kv8_call("attn_qk_rope_bwd", rope.lib.attn_qk_rope_bwd, rope, stream,
              dq.data_ptr(), dk.data_ptr(), from_v, hq, hk, wq, wk, f32, eps,
              _rope_positions(rope, positions, B, S),
              _counts(rope, "offset", offset, 1),
              _heads_view("dq_out", dq_out, q_shape, dtype),
              _heads_view("dk_out", dk_out, k_shape, dtype), to_v,
              None if dw[0] is None else dw[0].data_ptr(),
              None if dw[1] is None else dw[1].data_ptr(), B, S, Hq, Hkv, dt,
              None if workspace is None else workspace.data_ptr(),
              0 if workspace is None else workspace.nbytes)
    return dq_out, dk_out, dv_out, dw[0], dw[1]


class PrefixCache(_Handle):
    """Handle of the keys and values of a batch whose sequences share a prefix
    (``attn_prefix_cache_t``).

    prefix_k, prefix_v [1, Hkv, prefix_capacity, D]: the prefix's, of which
    prefix_len (int32 [1]) tokens are used; k, v [B, Hkv, capacity, D]: each
    sequence's own behind it, of which lens (int32 [B]) are used, the current
    step's new ones included.  All contiguous, float16 or bfloat16, on one CUDA
    device; the tensors stay the caller's and are kept alive by the handle.
    Advance ``lens`` first (in place), then write the new tokens (``qk_rope``
    with lens=cache.lens, offset=cache.prefix_len, k_out=cache.k,
    v_out=cache.v), then ``prefix_fwd``.
    """
    held = ("prefix_k", "prefix_v", "prefix_len", "k", "v", "lens")

    def __init__(self, prefix_k, prefix_v, prefix_len, k, v, lens):
        import torch
        if k.dim() != 4 or prefix_k.dim() != 4:
            raise AttnError("k must be 4-D [B, Hkv, capacity, D] and prefix_k "
                            "[1, Hkv, prefix_capacity, D]",
                            ATTN_ERR_INVALID_ARG)
        B, Hkv, capacity, D = k.shape
        P = prefix_k.shape[2]
        types = (torch.float16, torch.bfloat16)
        if k.dtype not in types:
            raise AttnError("k must be float16 or bfloat16, got %s" % k.dtype,
                            ATTN_ERR_INVALID_ARG)
        for name, t, shape, dtype in (
                ("prefix_k", prefix_k, (1, Hkv, P, D), k.dtype),
                ("prefix_v", prefix_v, (1, Hkv, P, D), k.dtype),
                ("prefix_len", prefix_len, (1,), torch.int32),
                ("k", k, (B, Hkv, capacity, D), k.dtype),
                ("v", v, (B, Hkv, capacity, D), k.dtype),
                ("lens", lens, (B,), torch.int32)):
            _check_tensor(name, t, shape, dtype)
            if not t.is_cuda or t.device != k.device:
                raise AttnError("%s must be a CUDA tensor on k's device"
                                % name, ATTN_ERR_INVALID_ARG)
        self.prefix_k, self.prefix_v = prefix_k, prefix_v
        self.prefix_len, self.k, self.v, self.lens = prefix_len, k, v, lens
        self.B, self.Hkv, self.capacity, self.D = B, Hkv, capacity, D
        self.prefix_capacity = P
        self.device, self.dtype = k.device, k.dtype
        # What every call needs, looked up once.
        self.dtypes = {k.dtype: ATTN_F16 if k.dtype == torch.float16
                       else ATTN_BF16}
        self.int32, self.float32 = torch.int32, torch.float32
        self.lib, self.index = load_library(), k.device.index
        self.current_device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.struct = ctypes.pointer(_Prefix(
            prefix_k.data_ptr(), prefix_v.data_ptr(), prefix_len.data_ptr(),
            k.data_ptr(), v.data_ptr(), lens.data_ptr(), B, Hkv, P, capacity,
            D))

    @classmethod
    def empty(cls, prefix_k, prefix_v, B, capacity, prefix_len=None,
              lens=None):
        """Caches of new, uninitialised memory for B sequences behind a prefix
        (all of prefix_k's tokens unless ``prefix_len`` is given); ``lens``:
        zeros unless given."""
        import torch
        _, Hkv, P, D = prefix_k.shape
        dev = prefix_k.device
        k, v = (torch.empty((B, Hkv, capacity, D), dtype=prefix_k.dtype,
                            device=dev) for _ in range(2))
        if prefix_len is None:
            prefix_len = torch.tensor([P], dtype=torch.int32, device=dev)
        if lens is None:
            lens = torch.zeros(B, dtype=torch.int32, device=dev)
        return cls(prefix_k, prefix_v, prefix_len, k, v, lens)


def prefix_workspace(cache, Hq, Sq):
    """A workspace tensor for ``prefix_fwd`` calls of Hq heads and Sq rows."""
    import torch
    with torch.cuda.device(cache.device):
        n = attn_prefix_workspace_bytes(cache.B, Hq, cache.Hkv, Sq,
                                        cache.prefix_capacity, cache.capacity,
                                        cache.D)
        return torch.empty(max(n, 1), dtype=torch.uint8, device=cache.device)


def prefix_fwd(cache, q, scale=None, causal=True, new_lens=None, out=None,
               lse=None, need_lse=True, workspace=None, stream=None):
    """Attention of q [B, Hq, Sq, D] (contiguous, the cache's type) over a
    shared prefix and each sequence's own tokens behind it.  Returns (O, LSE)
    like ``fwd``.

    Row i of a sequence with n new rows (Sq, or ``new_lens[b]`` of them) is its
    own token lens - n + i: it sees the prefix and its own tokens up to it
    (``causal``), or all of them.  Rows that see nothing get O = 0 and LSE =
    -inf; rows at or behind new_lens are left as they are in ``out`` and
    ``lse``.  ``workspace``: from ``prefix_workspace``, allocated when not
    given.  What a call on ``stream`` allocates is that stream's memory.
    """
    dt = _kv8_dtype(cache, "q", q)
    dtype, B, shape = q.dtype, cache.B, q.shape
    _, Hq, Sq, D = shape
    if shape[0] != B or D != cache.D or not q.is_contiguous():
        _check_tensor("q", q, (B, Hq, Sq, cache.D), dtype)
    if out is None:
        import torch
        with _kv8_memory(cache, stream):
            out = torch.empty_like(q)
    else:
        _check_tensor("out", out, shape, dtype)
    if not need_lse:
        lse = None
    elif lse is None:
        import torch
        with _kv8_memory(cache, stream):
            lse = torch.empty((B, Hq, Sq), dtype=torch.float32,
                              device=cache.device)
    else:
        _check_tensor("lse", lse, (B, Hq, Sq), cache.float32)
    if workspace is None:
        with _kv8_memory(cache, stream):
            workspace = prefix_workspace(cache, Hq, Sq)
    elif not workspace.is_contiguous():
        raise AttnError("workspace must be contiguous", ATTN_ERR_INVALID_ARG)
    if new_lens is not None:
        _check_tensor("new_lens", new_lens, (B,), cache.int32)
        new_lens = new_lens.data_ptr()
    if scale is None:
        scale = cache.D ** -0.5
    _kv8_call("attn_prefix_fwd", cache.lib.attn_prefix_fwd, cache, stream,
              q.data_ptr(), out.data_ptr(),
              lse.data_ptr() if lse is not None else None, Hq, Sq, new_lens,
              scale, bool(causal), dt, workspace.data_ptr(),
              workspace.nbytes)
    return out, lse
