"""Python binding of libgdn.so: gated-delta verify, ReplaySSM commit and
chunked prefill on MI355X (gfx950), and the serving operators beside them
(linear attention with a decay per head, paged attention with a cache in the
rows' type or in 4 bits, position rotation, token scores, sampled
verification).

Argument marshalling only (with checks of the tensors for the latter): every
step of the path runs in the HIP kernels behind the C ABI declared in
``include/gdn.h``.  torch provides device memory and streams.  There is no fallback: if the built library is missing,
importing this package raises.

Names follow the C ABI: ``verify``, ``commit``, ``prefill_chunked``,
``records_bytes``, ``prefill_workspace_bytes``, ``decay_step``,
``decay_prefill``, ``paged_attention``, ``kv_append``, ``token_scores``,
``rope_append``, ``rope_append_mxfp``, ``paged_attention_mxfp``,
``draft_verify``, ...
"""
from __future__ import annotations

import ctypes
import os
from array import array

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_LIBRARY names another build of the same library (the CPU tests load
# a sanitizer build of the host code this way).
LIB_PATH = os.environ.get("GDN_LIBRARY") or os.path.join(_HERE, "_build",
                                                         "libgdn.so")

GDN_OK, GDN_EINVAL, GDN_EUNSUPPORTED, GDN_EWORKSPACE, GDN_EHIP = 0, -1, -2, -3, -4
GDN_BF16, GDN_F32 = 0, 1
GDN_FLAG_L2NORM_QK = 1
GDN_FLAG_PREFILL_ONE_CHAIN = 2
GDN_FLAG_TOKENWISE = 4
GDN_FLAG_HEAD_DECAY = 8
GDN_FLAG_KEEP_STATE = 16
GDN_FLAG_ROPE_PAIRS = 32
GDN_MAX_LANES = 256
GDN_MAX_T = 64
GDN_MAX_TOP = 32

EXPORTED = ("gdn_records_bytes", "gdn_verify", "gdn_commit",
            "gdn_commit_verify", "gdn_verify_tree", "gdn_commit_path",
            "gdn_kda_records_bytes", "gdn_kda_verify", "gdn_kda_commit",
            "gdn_state_snapshot", "gdn_state_restore",
            "gdn_prefill_workspace_bytes", "gdn_prefill_chunked",
            "gdn_prefill_chunked_noalloc", "gdn_decay_step",
            "gdn_decay_prefill_workspace_bytes", "gdn_decay_prefill",
            "gdn_paged_attention_workspace_bytes", "gdn_paged_attention",
            "gdn_kv_append", "gdn_token_scores_workspace_bytes",
            "gdn_token_scores", "gdn_rope_append", "gdn_rope_append_mxfp",
            "gdn_paged_attention_mxfp_workspace_bytes",
            "gdn_paged_attention_mxfp", "gdn_draft_verify_workspace_bytes",
            "gdn_draft_verify", "gdn_strerror", "gdn_last_error")
PREFILL_SCRATCH_BYTES = 64 << 20


class GdnError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s: %s (%d): %s" % (
            what, _strerror(status), status, lib.gdn_last_error().decode()))
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_lanes", ctypes.c_int32),
                ("h_v", ctypes.c_int32), ("h_k", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("t_max", ctypes.c_int32)]

    @classmethod
    def of(cls, n_layers, n_lanes, h_v, h_k, d_k, d_v, t_max):
        return cls(n_layers, n_lanes, h_v, h_k, d_k, d_v, t_max)


class KvDims(ctypes.Structure):
    _fields_ = [("n_lanes", ctypes.c_int32), ("t_max", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]

    @classmethod
    def of(cls, n_lanes, t_max, h_q, h_kv, d, page_size, n_pages, max_pages):
        return cls(n_lanes, t_max, h_q, h_kv, d, page_size, n_pages, max_pages)


def _load_library():
    # torch ships its own HIP runtime (libamdhip64.so.7).  Load it first so
    # that libgdn.so binds to the same runtime instance as the streams and
    # device memory it is handed; a second runtime in the process would not
    # see torch's device state.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libgdn.so is not built (%s); run commit_gated_delta_amd/build.py "
            "or __graft_entry__.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    ip = ctypes.POINTER(ctypes.c_int32)
    dp = ctypes.POINTER(Dims)
    f = ctypes.c_float
    lib.gdn_records_bytes.argtypes = [dp]
    lib.gdn_records_bytes.restype = sz
    lib.gdn_verify.argtypes = [dp, ip, vp, vp, vp, ctypes.c_int, vp, vp, vp,
                               vp, vp, vp, f, ctypes.c_int, vp]
    lib.gdn_verify.restype = ctypes.c_int
    lib.gdn_commit.argtypes = [dp, ip, ip, vp, vp, vp]
    lib.gdn_commit.restype = ctypes.c_int
    lib.gdn_commit_verify.argtypes = [dp, ip, ip, vp, ip, vp, vp, vp,
                                      ctypes.c_int, vp, vp, vp, vp, vp, vp, f,
                                      ctypes.c_int, vp]
    lib.gdn_commit_verify.restype = ctypes.c_int
    lib.gdn_kda_records_bytes.argtypes = [dp]
    lib.gdn_kda_records_bytes.restype = sz
    lib.gdn_kda_verify.argtypes = lib.gdn_verify.argtypes
    lib.gdn_kda_verify.restype = ctypes.c_int
    lib.gdn_kda_commit.argtypes = lib.gdn_commit.argtypes
    lib.gdn_kda_commit.restype = ctypes.c_int
    lib.gdn_verify_tree.argtypes = [dp, ip, ip, vp, vp, vp, ctypes.c_int, vp,
                                    vp, vp, vp, vp, vp, f, ctypes.c_int, vp]
    lib.gdn_verify_tree.restype = ctypes.c_int
    lib.gdn_commit_path.argtypes = [dp, ip, ip, ip, ip, vp, vp, vp]
    lib.gdn_commit_path.restype = ctypes.c_int
    for fn in (lib.gdn_state_snapshot, lib.gdn_state_restore):
        fn.argtypes = [dp, i32, ip, vp, vp, vp]
        fn.restype = ctypes.c_int
    lib.gdn_prefill_workspace_bytes.argtypes = [i32] * 7
    lib.gdn_prefill_workspace_bytes.restype = sz
    lib.gdn_prefill_chunked.argtypes = [i32] * 8 + [vp] * 3 + [ctypes.c_int] + [
        vp] * 7 + [sz, f, ctypes.c_int, vp]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked_noalloc.argtypes = [i32] * 8 + [vp] * 3 + [
        ctypes.c_int] + [vp] * 6 + [f, ctypes.c_int, vp]
    lib.gdn_prefill_chunked_noalloc.restype = ctypes.c_int
    kp = ctypes.POINTER(KvDims)
    lib.gdn_decay_step.argtypes = [dp, ip, vp, vp, vp, ctypes.c_int, vp, vp,
                                   vp, f, ctypes.c_int, vp]
    lib.gdn_decay_step.restype = ctypes.c_int
    lib.gdn_decay_prefill_workspace_bytes.argtypes = [i32, ip] + [i32] * 4
    lib.gdn_decay_prefill_workspace_bytes.restype = sz
    lib.gdn_decay_prefill.argtypes = [i32, ip] + [i32] * 4 + [vp] * 3 + [
        ctypes.c_int] + [vp] * 5 + [sz, f, ctypes.c_int, vp]
    lib.gdn_decay_prefill.restype = ctypes.c_int
    lib.gdn_paged_attention_workspace_bytes.argtypes = [kp]
    lib.gdn_paged_attention_workspace_bytes.restype = sz
    lib.gdn_paged_attention.argtypes = [kp, ip] + [vp] * 3 + [
        ctypes.c_int] + [vp] * 4 + [sz, f, vp]
    lib.gdn_paged_attention.restype = ctypes.c_int
    lib.gdn_kv_append.argtypes = [kp, ip, vp, vp, ctypes.c_int] + [vp] * 5
    lib.gdn_kv_append.restype = ctypes.c_int
    lib.gdn_token_scores_workspace_bytes.argtypes = [i32] * 3
    lib.gdn_token_scores_workspace_bytes.restype = sz
    lib.gdn_token_scores.argtypes = [i32, i32, ctypes.c_int64, vp,
                                     ctypes.c_int, vp, i32, f] + [
                                         vp] * 5 + [sz, vp]
    lib.gdn_token_scores.restype = ctypes.c_int
    i64 = ctypes.c_int64
    rows = [kp, vp, vp, i64, vp, i64, vp, i64, ctypes.c_int, vp, i32, vp, vp]
    lib.gdn_rope_append.argtypes = rows + [vp] * 4 + [ctypes.c_int, vp]
    lib.gdn_rope_append.restype = ctypes.c_int
    lib.gdn_rope_append_mxfp.argtypes = rows + [vp] * 8 + [ctypes.c_int, vp]
    lib.gdn_rope_append_mxfp.restype = ctypes.c_int
    lib.gdn_paged_attention_mxfp_workspace_bytes.argtypes = [kp]
    lib.gdn_paged_attention_mxfp_workspace_bytes.restype = sz
    lib.gdn_paged_attention_mxfp.argtypes = [kp, vp, vp, ctypes.c_int] + [
        vp] * 8 + [sz, f, vp]
    lib.gdn_paged_attention_mxfp.restype = ctypes.c_int
    lib.gdn_draft_verify_workspace_bytes.argtypes = [i32] * 3
    lib.gdn_draft_verify_workspace_bytes.restype = sz
    lib.gdn_draft_verify.argtypes = [i32, i32, vp, i32, vp, i64, vp, i64,
                                     ctypes.c_int] + [vp] * 7 + [sz, vp]
    lib.gdn_draft_verify.restype = ctypes.c_int
    lib.gdn_strerror.argtypes = [ctypes.c_int]
    lib.gdn_strerror.restype = ctypes.c_char_p
    lib.gdn_last_error.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    return lib


lib = _load_library()


def _strerror(status):
    return lib.gdn_strerror(int(status)).decode()


def _check(status, what):
    if status != GDN_OK:
        raise GdnError(status, what)


def _ptr(t):
    """Device (or host) address of a tensor, or None."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _int_array(values, n):
    vals = [int(x) for x in values]
    if len(vals) != n:
        raise ValueError("expected %d per-lane values, got %d" % (n, len(vals)))
    return (ctypes.c_int32 * n)(*vals)


def _dtype_code(t):
    import torch
    if t is None:       # the C ABI reports the null pointer
        return GDN_BF16
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


def _stream(stream):
    """hipStream_t handle: torch's current stream by default, a
    torch.cuda.Stream, or a raw integer handle (0 = the null stream)."""
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def records_bytes(dims: Dims) -> int:
    return int(lib.gdn_records_bytes(ctypes.byref(dims)))


def _verify_flags(l2norm, tokenwise):
    return ((GDN_FLAG_L2NORM_QK if l2norm else 0) |
            (GDN_FLAG_TOKENWISE if tokenwise else 0))


def verify(dims: Dims, t_lane, q, k, v, beta, g, S, o, records,
           dbg_states=None, scale=1.0, l2norm=True, stream=None,
           raw_status=False, tokenwise=False):
    """gdn_verify on torch tensors (layouts in include/gdn.h;
    tokenwise=True sets GDN_FLAG_TOKENWISE)."""
    st = lib.gdn_verify(ctypes.byref(dims), _int_array(t_lane, dims.n_lanes),
                        _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(beta),
                        _ptr(g), _ptr(S), _ptr(o), _ptr(records),
                        _ptr(dbg_states), float(scale),
                        _verify_flags(l2norm, tokenwise), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_verify")


def commit(dims: Dims, m_lane, t_lane, records, S, stream=None,
           raw_status=False):
    """gdn_commit on torch tensors."""
    st = lib.gdn_commit(ctypes.byref(dims), _int_array(m_lane, dims.n_lanes),
                        _int_array(t_lane, dims.n_lanes), _ptr(records),
                        _ptr(S), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_commit")


def commit_verify(dims: Dims, m_prev, t_prev, records_prev, t_lane, q, k, v,
                  beta, g, S, o, records, dbg_states=None, scale=1.0,
                  l2norm=True, stream=None, raw_status=False, tokenwise=False):
    """gdn_commit_verify on torch tensors: commit(m_prev) of the previous
    window's records, then verify of the new window, in one launch."""
    st = lib.gdn_commit_verify(
        ctypes.byref(dims), _int_array(m_prev, dims.n_lanes),
        _int_array(t_prev, dims.n_lanes), _ptr(records_prev),
        _int_array(t_lane, dims.n_lanes), _ptr(q), _ptr(k), _ptr(v),
        _dtype_code(q), _ptr(beta), _ptr(g), _ptr(S), _ptr(o), _ptr(records),
        _ptr(dbg_states), float(scale), _verify_flags(l2norm, tokenwise),
        _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_commit_verify")


def kda_records_bytes(dims: Dims) -> int:
    return int(lib.gdn_kda_records_bytes(ctypes.byref(dims)))


def kda_verify(dims: Dims, t_lane, q, k, v, beta, g, S, o, records,
               dbg_states=None, scale=1.0, l2norm=True, stream=None,
               raw_status=False, tokenwise=False):
    """gdn_kda_verify; g is [NL][N][T][Hv][d_k] (per-channel log-decay)."""
    st = lib.gdn_kda_verify(ctypes.byref(dims), _int_array(t_lane, dims.n_lanes),
                            _ptr(q), _ptr(k), _ptr(v), _dtype_code(q),
                            _ptr(beta), _ptr(g), _ptr(S), _ptr(o),
                            _ptr(records), _ptr(dbg_states), float(scale),
                            _verify_flags(l2norm, tokenwise),
                            _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_kda_verify")


def kda_commit(dims: Dims, m_lane, t_lane, records, S, stream=None,
               raw_status=False):
    st = lib.gdn_kda_commit(ctypes.byref(dims), _int_array(m_lane, dims.n_lanes),
                            _int_array(t_lane, dims.n_lanes), _ptr(records),
                            _ptr(S), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_kda_commit")


def _table(rows, n, t_max, fill):
    """int32 [n][t_max] from per-lane sequences (padded with ``fill``)."""
    import numpy as np
    a = np.full((n, t_max), fill, dtype=np.int32)
    if len(rows) != n:
        raise ValueError("expected %d per-lane rows, got %d" % (n, len(rows)))
    for i, r in enumerate(rows):
        r = [int(x) for x in r]
        a[i, :len(r)] = r
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def verify_tree(dims: Dims, t_lane, parent, q, k, v, beta, g, S, o, records,
                dbg_states=None, scale=1.0, l2norm=True, stream=None,
                raw_status=False, tokenwise=False):
    """gdn_verify_tree; parent is [n_lanes][<= t_max] (-1: from S0)."""
    keep, pp = _table(parent, dims.n_lanes, dims.t_max, -1)
    st = lib.gdn_verify_tree(
        ctypes.byref(dims), _int_array(t_lane, dims.n_lanes), pp, _ptr(q),
        _ptr(k), _ptr(v), _dtype_code(q), _ptr(beta), _ptr(g), _ptr(S),
        _ptr(o), _ptr(records), _ptr(dbg_states), float(scale),
        _verify_flags(l2norm, tokenwise), _stream(stream))
    del keep
    if raw_status:
        return st
    _check(st, "gdn_verify_tree")


def commit_path(dims: Dims, paths, t_lane, parent, records, S, stream=None,
                raw_status=False):
    """gdn_commit_path; paths[n] lists the accepted nodes of lane n, root
    first (empty: nothing accepted)."""
    keep_p, pp = _table(paths, dims.n_lanes, dims.t_max, 0)
    keep_t, tp = _table(parent, dims.n_lanes, dims.t_max, -1)
    m = [len(p) for p in paths]
    st = lib.gdn_commit_path(ctypes.byref(dims), _int_array(m, dims.n_lanes),
                             pp, _int_array(t_lane, dims.n_lanes), tp,
                             _ptr(records), _ptr(S), _stream(stream))
    del keep_p, keep_t
    if raw_status:
        return st
    _check(st, "gdn_commit_path")


def _lane_list(lanes):
    vals = [int(x) for x in lanes]
    return len(vals), (ctypes.c_int32 * max(len(vals), 1))(*vals)


def state_snapshot(dims: Dims, lanes, S, snapshot, stream=None,
                   raw_status=False):
    """gdn_state_snapshot: snapshot[j] = S[:, lanes[j]] (device or pinned
    host tensor)."""
    n, arr = _lane_list(lanes)
    st = lib.gdn_state_snapshot(ctypes.byref(dims), n, arr, _ptr(S),
                                _ptr(snapshot), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_state_snapshot")


def state_restore(dims: Dims, lanes, snapshot, S, stream=None,
                  raw_status=False):
    """gdn_state_restore: S[:, lanes[j]] = snapshot[j]."""
    n, arr = _lane_list(lanes)
    st = lib.gdn_state_restore(ctypes.byref(dims), n, arr, _ptr(snapshot),
                               _ptr(S), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_state_restore")


def prefill_workspace_bytes(n_seqs, seq_len, h_v, h_k, d_k, d_v,
                            chunk=64) -> int:
    return int(lib.gdn_prefill_workspace_bytes(n_seqs, seq_len, h_v, h_k, d_k,
                                               d_v, chunk))


def _prefill_flags(l2norm, segments):
    return ((GDN_FLAG_L2NORM_QK if l2norm else 0) |
            (0 if segments else GDN_FLAG_PREFILL_ONE_CHAIN))


def prefill_chunked(n_seqs, seq_len, h_v, h_k, d_k, d_v, q, k, v, beta, g,
                    S_init, S_final, o, checkpoints, workspace,
                    ckpt_interval=8192, scale=1.0, l2norm=True, stream=None,
                    raw_status=False, chunk=64, segments=True):
    """gdn_prefill_chunked on torch tensors (segments=False sets
    GDN_FLAG_PREFILL_ONE_CHAIN)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_prefill_chunked(
        n_seqs, seq_len, h_v, h_k, d_k, d_v, chunk, ckpt_interval, _ptr(q),
        _ptr(k), _ptr(v), _dtype_code(q), _ptr(beta), _ptr(g), _ptr(S_init),
        _ptr(S_final), _ptr(o), _ptr(checkpoints), _ptr(workspace), ws_bytes,
        float(scale), _prefill_flags(l2norm, segments), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_prefill_chunked")


def prefill_chunked_noalloc(n_seqs, seq_len, h_v, h_k, d_k, d_v, q, k, v,
                            beta, g, S_init, S_final, o, checkpoints,
                            ckpt_interval=8192, scale=1.0, l2norm=True,
                            stream=None, raw_status=False, chunk=64,
                            segments=True):
    """gdn_prefill_chunked_noalloc: the prefill with the library's fixed
    scratch array as its workspace (no allocation; calls that overlap on
    one GPU race)."""
    st = lib.gdn_prefill_chunked_noalloc(
        n_seqs, seq_len, h_v, h_k, d_k, d_v, chunk, ckpt_interval, _ptr(q),
        _ptr(k), _ptr(v), _dtype_code(q), _ptr(beta), _ptr(g), _ptr(S_init),
        _ptr(S_final), _ptr(o), _ptr(checkpoints), float(scale),
        _prefill_flags(l2norm, segments), _stream(stream))
    if raw_status:
        return st
    _check(st, "gdn_prefill_chunked_noalloc")


# The entry points below also check the tensors they are given: the kernels
# index them by the sizes alone, so a wrong element type, a view that is not
# contiguous, too few elements or another device than the current one is
# refused here.  They are called once per layer and token, so the checks and
# the stream look-up are kept to about 2 us.
import torch  # noqa: E402  (loaded with the library already)

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _tensor(t, name, dtype, numel, device):
    if (t.dtype is dtype and t.get_device() == device and t.is_contiguous()
            and t.numel() >= numel):
        return t.data_ptr()
    raise ValueError(
        "%s: expected a contiguous tensor of %s with %d elements on the "
        "current device (cuda:%d), got %s %s on %s%s" % (
            name, dtype, numel, device, t.dtype, tuple(t.shape), t.device,
            "" if t.is_contiguous() else ", not contiguous"))


def _optional(t, name, dtype, numel, device):
    return None if t is None else _tensor(t, name, dtype, numel, device)


def _workspace(t, device):
    """Address and size in bytes of a workspace (a uint8 tensor or None)."""
    if t is None:
        return None, 0
    return _tensor(t, "workspace", _U8, 0, device), t.numel()


def _code(dtype):
    try:
        return _CODES[dtype]
    except KeyError:
        raise TypeError("expected bfloat16 or float32, got %s" % dtype) from None


def _lanes(t_lane, n):
    if len(t_lane) != n:
        raise ValueError("expected %d per-lane values, got %d"
                         % (n, len(t_lane)))
    return (ctypes.c_int32 * n)(*t_lane)


def _stream_on(stream, device):
    """As _stream, without making a Stream object for the current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if isinstance(stream, int):
        return stream
    if stream.device_index != device:
        raise ValueError("the stream is on cuda:%d, the current device is "
                         "cuda:%d" % (stream.device_index, device))
    return stream.cuda_stream


def decay_step(dims: Dims, t_lane, q, k, v, g, S, o, scale=1.0,
               head_decay=False, keep_state=False, stream=None,
               raw_status=False):
    """gdn_decay_step on torch tensors.  keep_state=True is the verify of a
    window, o=None (q may be None then) with t_lane = m its commit."""
    kind, lanes = k.dtype, _lanes(t_lane, dims.n_lanes)
    code, dev = _code(kind), torch.cuda.current_device()
    h_v, states = dims.h_v, dims.n_layers * dims.n_lanes
    rows = states * dims.t_max
    nk, nv = rows * dims.h_k * dims.d_k, rows * h_v * dims.d_v
    st = lib.gdn_decay_step(
        ctypes.byref(dims), lanes, _optional(q, "q", kind, nk, dev),
        _tensor(k, "k", kind, nk, dev), _tensor(v, "v", kind, nv, dev), code,
        _tensor(g, "g", _F32,
                dims.n_layers * h_v if head_decay else rows * h_v, dev),
        _tensor(S, "S", _F32, states * h_v * dims.d_k * dims.d_v, dev),
        _optional(o, "o", _F32, nv, dev), scale,
        (GDN_FLAG_HEAD_DECAY if head_decay else 0) |
        (GDN_FLAG_KEEP_STATE if keep_state else 0), _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_decay_step")


def decay_prefill_workspace_bytes(seq_len, h_v, h_k, d_k, d_v) -> int:
    n = len(seq_len)
    return int(lib.gdn_decay_prefill_workspace_bytes(
        n, _lanes(seq_len, n), h_v, h_k, d_k, d_v))


def decay_prefill(seq_len, h_v, h_k, d_k, d_v, q, k, v, g, S_init, S_final, o,
                  workspace, scale=1.0, head_decay=False, stream=None,
                  raw_status=False):
    """gdn_decay_prefill on torch tensors; seq_len lists the lengths of the
    packed sequences."""
    n, tokens, kind = len(seq_len), sum(seq_len), k.dtype
    code, dev = _code(kind), torch.cuda.current_device()
    nk, nv, ns = tokens * h_k * d_k, tokens * h_v * d_v, n * h_v * d_k * d_v
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib.gdn_decay_prefill(
        n, _lanes(seq_len, n), h_v, h_k, d_k, d_v,
        _optional(q, "q", kind, nk, dev), _tensor(k, "k", kind, nk, dev),
        _tensor(v, "v", kind, nv, dev), code,
        _tensor(g, "g", _F32, h_v if head_decay else tokens * h_v, dev),
        _optional(S_init, "S_init", _F32, ns, dev),
        _optional(S_final, "S_final", _F32, ns, dev),
        _optional(o, "o", _F32, nv, dev), ws, ws_bytes, scale,
        GDN_FLAG_HEAD_DECAY if head_decay else 0, _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_decay_prefill")


def paged_attention_workspace_bytes(dims: KvDims) -> int:
    return int(lib.gdn_paged_attention_workspace_bytes(ctypes.byref(dims)))


def paged_attention(dims: KvDims, t_lane, q, k_cache, v_cache, page_table,
                    kv_len, o, workspace, scale=1.0, stream=None,
                    raw_status=False):
    """gdn_paged_attention on torch tensors."""
    n, d, kind = dims.n_lanes, dims.d, q.dtype
    lanes, code, dev = _lanes(t_lane, n), _code(kind), torch.cuda.current_device()
    nq = n * dims.t_max * dims.h_q * d
    nc = dims.n_pages * dims.h_kv * dims.page_size * d
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib.gdn_paged_attention(
        ctypes.byref(dims), lanes, _tensor(q, "q", kind, nq, dev),
        _tensor(k_cache, "k_cache", kind, nc, dev),
        _tensor(v_cache, "v_cache", kind, nc, dev), code,
        _tensor(page_table, "page_table", _I32, n * dims.max_pages, dev),
        _tensor(kv_len, "kv_len", _I32, n, dev),
        _tensor(o, "o", _F32, nq, dev), ws, ws_bytes, scale,
        _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_paged_attention")


def kv_append(dims: KvDims, t_lane, k, v, k_cache, v_cache, page_table,
              kv_len, stream=None, raw_status=False):
    """gdn_kv_append on torch tensors."""
    n, kind, row = dims.n_lanes, k.dtype, dims.h_kv * dims.d
    lanes, code, dev = _lanes(t_lane, n), _code(kind), torch.cuda.current_device()
    nr, nc = n * dims.t_max * row, dims.n_pages * dims.page_size * row
    st = lib.gdn_kv_append(
        ctypes.byref(dims), lanes, _tensor(k, "k", kind, nr, dev),
        _tensor(v, "v", kind, nr, dev), code,
        _tensor(k_cache, "k_cache", kind, nc, dev),
        _tensor(v_cache, "v_cache", kind, nc, dev),
        _tensor(page_table, "page_table", _I32, n * dims.max_pages, dev),
        _tensor(kv_len, "kv_len", _I32, n, dev), _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_kv_append")


def token_scores_workspace_bytes(n_rows, vocab, n_top) -> int:
    return int(lib.gdn_token_scores_workspace_bytes(n_rows, vocab, n_top))


def token_scores(logits, tokens, n_top, logprob, entropy, top_ids,
                 top_logprobs, workspace, inv_temperature=1.0, stream=None,
                 raw_status=False):
    """gdn_token_scores on torch tensors.  logits is [n_rows, vocab] with
    contiguous rows (their stride may be larger than vocab)."""
    code, dev = _code(logits.dtype), torch.cuda.current_device()
    rows, vocab = logits.shape
    stride, unit = logits.stride()
    if logits.get_device() != dev or (vocab > 1 and unit != 1) or (
            rows > 1 and stride < vocab):
        raise ValueError("logits: expected a tensor [n_rows, vocab] with "
                         "contiguous rows on the current device (cuda:%d), "
                         "got strides %s on %s" % (dev, logits.stride(),
                                                   logits.device))
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib.gdn_token_scores(
        rows, vocab, stride if rows > 1 else vocab, logits.data_ptr(), code,
        _optional(tokens, "tokens", _I32, rows, dev), n_top, inv_temperature,
        _optional(logprob, "logprob", _F32, rows, dev),
        _optional(entropy, "entropy", _F32, rows, dev),
        _optional(top_ids, "top_ids", _I32, rows * n_top, dev),
        _optional(top_logprobs, "top_logprobs", _F32, rows * n_top, dev),
        ws, ws_bytes, _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_token_scores")


def _lane_ints(t_lane, n):
    """The lanes' values as an int32 array (``buffer_info`` has its address;
    made in a third of the time of a ctypes array)."""
    a = array("i", t_lane)
    if len(a) != n:
        raise ValueError("expected %d per-lane values, got %d" % (n, len(a)))
    return a


def _rows(t, name, dtype, n, t_max, h, d, device):
    """Address and token stride of rows [n, t_max, h, d], each token's h rows
    contiguous and the tokens equally far apart (a part of a projection's
    output, say)."""
    if (t.dtype is dtype and t.get_device() == device
            and t.shape == (n, t_max, h, d)):
        s0, s1, s2, s3 = t.stride()
        step = s1 if t_max > 1 else s0 if n > 1 else h * d
        if (s3 == 1 and (s2 == d or h == 1) and step >= h * d
                and (n == 1 or s0 == t_max * step)):
            return t.data_ptr(), step
    raise ValueError(
        "%s: expected %s rows [%d, %d, %d, %d] with contiguous heads and "
        "equally spaced tokens on the current device (cuda:%d), got %s %s, "
        "strides %s on %s" % (name, dtype, n, t_max, h, d, device, t.dtype,
                              tuple(t.shape), t.stride(), t.device))


def _rope_args(dims, lanes, q, k, v, inv_freq, rot_dim, q_out, positions,
               dev):
    """The arguments that both writers begin with."""
    n, tm, hq, hk, d = dims.n_lanes, dims.t_max, dims.h_q, dims.h_kv, dims.d
    kind = k.dtype
    qp, qs = (None, 0) if q is None else _rows(q, "q", kind, n, tm, hq, d, dev)
    kp, ks = _rows(k, "k", kind, n, tm, hk, d, dev)
    vp, vs = _rows(v, "v", kind, n, tm, hk, d, dev)
    return (ctypes.byref(dims), lanes.buffer_info()[0], qp, qs, kp, ks, vp, vs,
            _code(kind),
            _optional(inv_freq, "inv_freq", _F32, rot_dim // 2, dev), rot_dim,
            _optional(positions, "positions", _I32, n * tm, dev),
            _optional(q_out, "q_out", kind, n * tm * hq * d, dev))


def rope_append(dims: KvDims, t_lane, q, k, v, inv_freq, rot_dim, q_out,
                k_cache, v_cache, page_table, kv_len, positions=None,
                interleaved=False, stream=None, raw_status=False):
    """gdn_rope_append on torch tensors.  q, k, v may be views of one
    projection's output; interleaved=True sets GDN_FLAG_ROPE_PAIRS."""
    n, kind, dev = dims.n_lanes, k.dtype, torch.cuda.current_device()
    lanes = _lane_ints(t_lane, n)
    nc = dims.n_pages * dims.page_size * dims.h_kv * dims.d
    st = lib.gdn_rope_append(
        *_rope_args(dims, lanes, q, k, v, inv_freq, rot_dim, q_out,
                    positions, dev),
        _tensor(k_cache, "k_cache", kind, nc, dev),
        _tensor(v_cache, "v_cache", kind, nc, dev),
        _tensor(page_table, "page_table", _I32, n * dims.max_pages, dev),
        _tensor(kv_len, "kv_len", _I32, n, dev),
        GDN_FLAG_ROPE_PAIRS if interleaved else 0, _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_rope_append")


def _fp4_cache(dims, k_codes, k_scales, v_codes, v_scales, dev):
    rows = dims.n_pages * dims.page_size * dims.h_kv
    nc, ns = rows * (dims.d // 2), rows * (dims.d // 32)
    return (_tensor(k_codes, "k_codes", _U8, nc, dev),
            _tensor(k_scales, "k_scales", _U8, ns, dev),
            _tensor(v_codes, "v_codes", _U8, nc, dev),
            _tensor(v_scales, "v_scales", _U8, ns, dev))


def rope_append_mxfp(dims: KvDims, t_lane, q, k, v, inv_freq, rot_dim, q_out,
                     k_codes, k_scales, v_codes, v_scales, page_table, kv_len,
                     k_held=None, v_held=None, positions=None,
                     interleaved=False, stream=None, raw_status=False):
    """gdn_rope_append_mxfp on torch tensors."""
    n, dev = dims.n_lanes, torch.cuda.current_device()
    lanes = _lane_ints(t_lane, n)
    nr = n * dims.t_max * dims.h_kv * dims.d
    st = lib.gdn_rope_append_mxfp(
        *_rope_args(dims, lanes, q, k, v, inv_freq, rot_dim, q_out,
                    positions, dev),
        *_fp4_cache(dims, k_codes, k_scales, v_codes, v_scales, dev),
        _tensor(page_table, "page_table", _I32, n * dims.max_pages, dev),
        _tensor(kv_len, "kv_len", _I32, n, dev),
        _optional(k_held, "k_held", torch.bfloat16, nr, dev),
        _optional(v_held, "v_held", torch.bfloat16, nr, dev),
        GDN_FLAG_ROPE_PAIRS if interleaved else 0, _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_rope_append_mxfp")


def paged_attention_mxfp_workspace_bytes(dims: KvDims) -> int:
    return int(lib.gdn_paged_attention_mxfp_workspace_bytes(ctypes.byref(dims)))


def paged_attention_mxfp(dims: KvDims, t_lane, q, k_codes, k_scales, v_codes,
                         v_scales, page_table, kv_len, o, workspace, scale=1.0,
                         stream=None, raw_status=False):
    """gdn_paged_attention_mxfp on torch tensors."""
    n, kind = dims.n_lanes, q.dtype
    lanes, code, dev = _lane_ints(t_lane, n), _code(kind), torch.cuda.current_device()
    nq = n * dims.t_max * dims.h_q * dims.d
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib.gdn_paged_attention_mxfp(
        ctypes.byref(dims), lanes.buffer_info()[0], _tensor(q, "q", kind, nq, dev), code,
        *_fp4_cache(dims, k_codes, k_scales, v_codes, v_scales, dev),
        _tensor(page_table, "page_table", _I32, n * dims.max_pages, dev),
        _tensor(kv_len, "kv_len", _I32, n, dev),
        _tensor(o, "o", _F32, nq, dev), ws, ws_bytes, scale,
        _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_paged_attention_mxfp")


def _logit_rows(t, name, dtype, n, rows, vocab, device):
    """Address and row stride of logits [n, rows, vocab] with contiguous,
    equally spaced rows."""
    if (t.dtype is dtype and t.get_device() == device
            and t.shape == (n, rows, vocab)):
        s0, s1, s2 = t.stride()
        step = s1 if rows > 1 else s0 if n > 1 else vocab
        if (s2 == 1 or vocab == 1) and step >= vocab and (
                n == 1 or rows == 0 or s0 == rows * step):
            return t.data_ptr(), step
    raise ValueError(
        "%s: expected %s logits [%d, %d, %d] with contiguous, equally spaced "
        "rows on the current device (cuda:%d), got %s %s, strides %s on %s" % (
            name, dtype, n, rows, vocab, device, t.dtype, tuple(t.shape),
            t.stride(), t.device))


def draft_verify_workspace_bytes(n_lanes, t_max, vocab) -> int:
    return int(lib.gdn_draft_verify_workspace_bytes(n_lanes, t_max, vocab))


def draft_verify(t_lane, logits, draft_logits, tokens, uniforms,
                 inv_temperature, m_lane, next_token, workspace, accept=None,
                 stream=None, raw_status=False):
    """gdn_draft_verify on torch tensors: logits [n_lanes, t_max, vocab],
    draft_logits [n_lanes, t_max - 1, vocab] or None."""
    n, tm, vocab = logits.shape
    kind = logits.dtype
    lanes, code, dev = _lane_ints(t_lane, n), _code(kind), torch.cuda.current_device()
    lp, ls = _logit_rows(logits, "logits", kind, n, tm, vocab, dev)
    dp, ds = (None, 0) if draft_logits is None or tm == 1 else _logit_rows(
        draft_logits, "draft_logits", kind, n, tm - 1, vocab, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    st = lib.gdn_draft_verify(
        n, tm, lanes.buffer_info()[0], vocab, lp, ls, dp, ds, code,
        _tensor(tokens, "tokens", _I32, n * tm, dev),
        _tensor(uniforms, "uniforms", _F32, n * tm, dev),
        _tensor(inv_temperature, "inv_temperature", _F32, n, dev),
        _tensor(m_lane, "m_lane", _I32, n, dev),
        _tensor(next_token, "next_token", _I32, n, dev),
        _optional(accept, "accept", _F32, n * tm, dev), ws, ws_bytes,
        _stream_on(stream, dev))
    if raw_status:
        return st
    _check(st, "gdn_draft_verify")
