"""Python binding of the C ABI in include/dsa.h (argument marshalling only).

Every function here forwards to the same-named entry point of
``libdsa_b200.so``; tensors are passed as raw device pointers.  Nothing is
computed in Python and there is no fallback: if the library is missing or a
call fails, a ``DsaError`` is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa_b200.so")

DSA_OK = 0
DSA_ERR_INVALID_ARG = -1
DSA_ERR_UNSUPPORTED = -2
DSA_ERR_CUDA = -3
DSA_ERR_WORKSPACE = -4
DSA_ERR_TIMEOUT = -5
DSA_ERR_DEVICE_CHECK = -6

OP_INDEXER_SCORES = 0
OP_TOPK = 1
OP_INDEXER_TOPK = 2
OP_SPARSE_MLA_DECODE = 3
OP_SPARSE_MLA_PREFILL = 4
OP_FORWARD = 5
OP_INDEX_KL_SPARSE = 6
OP_INDEX_KL_DENSE = 7
OP_MASKED_MHA = 8

# Bytes of the status word at the start of a workspace.
WS_STATUS_BYTES = 256

ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_YARN = 0, 1, 2, 3
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2

# Entry points declared in include/dsa.h.
ENTRY_POINTS = (
    "dsa_workspace_size", "dsa_indexer_scores", "dsa_topk", "dsa_indexer_topk",
    "dsa_sparse_mla_decode", "dsa_sparse_mla_prefill", "dsa_forward", "dsa_forward_paged",
    "dsa_indexer_topk_static", "dsa_project_workspace_size", "dsa_indexer_project",
    "dsa_index_kl", "dsa_masked_mha_prefill", "dsa_sparse_mla_decode_fp8",
    "dsa_table_workspace_size", "dsa_build_tables", "dsa_rope", "dsa_rope_backward",
    "dsa_latent_append", "dsa_latent_append_fp8", "dsa_shared_prefix_workspace_size",
    "dsa_mla_shared_prefix", "dsa_check_status", "dsa_last_error",
)


class DsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("%s (status %d)" % (msg, code))
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [("nq", ctypes.c_int32), ("h_idx", ctypes.c_int32), ("d_idx", ctypes.c_int32),
                ("h", ctypes.c_int32), ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("max_n", ctypes.c_int32),
                ("q_per_seq", ctypes.c_int32), ("scale", ctypes.c_float)]


class ProjectParams(ctypes.Structure):
    _fields_ = [("nt", ctypes.c_int32), ("hidden", ctypes.c_int32), ("q_lora_rank", ctypes.c_int32),
                ("h_idx", ctypes.c_int32), ("d_idx", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("ln_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


class KV(ctypes.Structure):
    _fields_ = [("q_seq", ctypes.c_void_p), ("q_n", ctypes.c_void_p),
                ("seq_row0", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("cache_rows", ctypes.c_int64)]


class TableParams(ctypes.Structure):
    _fields_ = [("nseq", ctypes.c_int32), ("nt", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_free", ctypes.c_int32), ("sees_self", ctypes.c_int32),
                ("cache_rows", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("rope_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("orig_max_pos", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("mscale", ctypes.c_double)]


class RopeParams(ctypes.Structure):
    _fields_ = [("nt", ctypes.c_int32), ("h", ctypes.c_int32), ("x_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("begin", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64)]


_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None
_P = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """Load libdsa_b200.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise DsaError(DSA_ERR_CUDA, "libdsa_b200.so not built (run "
                               "python -m long_context_decode_indexer_b200.build)")
            L = ctypes.CDLL(LIB_PATH)
            pp, kp = ctypes.POINTER(Params), ctypes.POINTER(KV)
            L.dsa_workspace_size.argtypes = [pp, kp, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
            L.dsa_indexer_scores.argtypes = [pp, kp, _P, _P, _P, _P, _P, ctypes.c_int64, _P,
                                             ctypes.c_size_t, _P]
            L.dsa_topk.argtypes = [pp, _P, ctypes.c_int64, _P, _P, _P, _P, ctypes.c_size_t, _P]
            L.dsa_indexer_topk.argtypes = [pp, kp, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
            for name in ("dsa_sparse_mla_decode", "dsa_sparse_mla_prefill"):
                getattr(L, name).argtypes = [pp, kp, _P, _P, ctypes.c_int64, _P, _P, _P, _P,
                                             ctypes.c_size_t, _P]
            for name in ("dsa_forward", "dsa_forward_paged"):
                getattr(L, name).argtypes = [pp, kp, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P,
                                             _P, _P, _P, ctypes.c_size_t, _P]
            L.dsa_indexer_topk_static.argtypes = [pp, kp, _P, _P, _P, _P, _P, _P, _P, _P]
            jp = ctypes.POINTER(ProjectParams)
            L.dsa_project_workspace_size.argtypes = [jp, ctypes.POINTER(ctypes.c_size_t)]
            L.dsa_indexer_project.argtypes = [jp, kp] + [_P] * 17 + [ctypes.c_size_t, _P]
            L.dsa_index_kl.argtypes = [pp, kp, _P, _P, ctypes.c_int64, _P, ctypes.c_int64, _P, _P, _P,
                                       _P, ctypes.c_size_t, _P]
            L.dsa_masked_mha_prefill.argtypes = [pp, kp, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
            L.dsa_sparse_mla_decode_fp8.argtypes = [pp, kp, _P, _P, ctypes.c_int64, _P, _P, _P, _P, _P,
                                                    ctypes.c_size_t, _P]
            tp, rs, rp = (ctypes.POINTER(t) for t in (TableParams, RopeSpec, RopeParams))
            i32, i64, size_p = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
            L.dsa_table_workspace_size.argtypes = [tp, size_p]
            L.dsa_build_tables.argtypes = [tp] + [_P] * 14 + [ctypes.c_size_t, _P]
            L.dsa_rope.argtypes = [rs, rp, _P, _P, _P, _P]
            L.dsa_rope_backward.argtypes = [rs, rp, _P, _P, _P, _P]
            L.dsa_latent_append.argtypes = [rs, i32, _P, i64, _P, i64, _P, _P, _P, i64, i64, _P,
                                            ctypes.c_size_t, _P]
            L.dsa_latent_append_fp8.argtypes = [rs, i32, _P, i64, _P, i64, _P, _P, _P, i64, _P, i64, _P,
                                                ctypes.c_size_t, _P]
            L.dsa_shared_prefix_workspace_size.argtypes = [pp, kp, i32, size_p]
            L.dsa_mla_shared_prefix.argtypes = [pp, kp, i32, _P, _P, _P, _P, i64, _P, _P, _P,
                                                ctypes.c_size_t, _P]
            L.dsa_check_status.argtypes = [_P, _P]
            L.dsa_last_error.restype = ctypes.c_char_p
            for name in ENTRY_POINTS[:-1]:
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def last_error() -> str:
    return lib().dsa_last_error().decode()


def _check(rc: int, what: str):
    if rc != DSA_OK:
        raise DsaError(rc, "%s: %s" % (what, last_error()))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def make_params(*, nq, h_idx, d_idx, h, topk, max_n, q_per_seq=1, scale, d_qk=576, d_v=512) -> Params:
    return Params(int(nq), int(h_idx), int(d_idx), int(h), int(d_qk), int(d_v), int(topk),
                  int(max_n), int(q_per_seq), float(scale))


def make_kv(*, q_seq, q_n, seq_row0=None, page_table=None, page_size=0, cache_rows) -> KV:
    max_pages = int(page_table.shape[1]) if page_table is not None else 0
    return KV(_ptr(q_seq), _ptr(q_n), _ptr(seq_row0), _ptr(page_table), max_pages,
              int(page_size) if page_table is not None else 0, int(cache_rows))


def workspace_size(p: Params, kv: Optional[KV], op: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dsa_workspace_size(ctypes.byref(p), ctypes.byref(kv) if kv is not None else None,
                                    int(op), ctypes.byref(out)), "dsa_workspace_size")
    return int(out.value)


def indexer_scores(p, kv, q_idx, w, kidx_cache, k_scale, scores, ld_scores, ws, stream=None):
    _check(lib().dsa_indexer_scores(ctypes.byref(p), ctypes.byref(kv), _ptr(q_idx), _ptr(w),
                                    _ptr(kidx_cache), _ptr(k_scale), _ptr(scores), int(ld_scores),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_indexer_scores")


def topk(p, scores, ld_scores, q_n, idx, nsel, ws, stream=None):
    _check(lib().dsa_topk(ctypes.byref(p), _ptr(scores), int(ld_scores), _ptr(q_n), _ptr(idx),
                          _ptr(nsel), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_topk")


def indexer_topk(p, kv, q_idx, w, kidx_cache, k_scale, idx, nsel, ws, stream=None):
    _check(lib().dsa_indexer_topk(ctypes.byref(p), ctypes.byref(kv), _ptr(q_idx), _ptr(w),
                                  _ptr(kidx_cache), _ptr(k_scale), _ptr(idx), _ptr(nsel), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_indexer_topk")


def indexer_topk_static(p, kv, q_idx, w, kidx_cache, k_scale, idx, nsel, status, stream=None):
    """dsa_indexer_topk with the library's fixed scratch array (no workspace)."""
    _check(lib().dsa_indexer_topk_static(ctypes.byref(p), ctypes.byref(kv), _ptr(q_idx), _ptr(w),
                                         _ptr(kidx_cache), _ptr(k_scale), _ptr(idx), _ptr(nsel),
                                         _ptr(status), _stream(stream)),
           "dsa_indexer_topk_static")


def sparse_mla_decode(p, kv, q, kv_cache, kv_row_stride, idx, out, lse, ws, stream=None):
    _check(lib().dsa_sparse_mla_decode(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(kv_cache),
                                       int(kv_row_stride), _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_sparse_mla_decode")


def sparse_mla_decode_fp8(p, kv, q, kv8_cache, kv8_row_bytes, kv_scale, idx, out, lse, ws, stream=None):
    """Sparse attention over an FP8 latent cache (e4m3 codes, power-of-two row scales)."""
    _check(lib().dsa_sparse_mla_decode_fp8(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(kv8_cache),
                                           int(kv8_row_bytes), _ptr(kv_scale), _ptr(idx), _ptr(out),
                                           _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(stream)),
           "dsa_sparse_mla_decode_fp8")


def sparse_mla_prefill(p, kv, q, kv_cache, kv_row_stride, idx, out, lse, ws, stream=None):
    _check(lib().dsa_sparse_mla_prefill(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(kv_cache),
                                        int(kv_row_stride), _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_sparse_mla_prefill")


def index_kl(p, kv, q, kv_cache, kv_row_stride, index_scores, ld_scores, idx, kl, p_out, ws,
             stream=None):
    """Indexer distillation loss per query; idx None selects the dense stage
    (every visible position), else the sparse stage over idx's entries."""
    _check(lib().dsa_index_kl(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(kv_cache),
                              int(kv_row_stride), _ptr(index_scores), int(ld_scores), _ptr(idx),
                              _ptr(kl), _ptr(p_out), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)),
           "dsa_index_kl")


def masked_mha_prefill(p, kv, q, k, v, idx, out, lse, ws, stream=None):
    """Dense MHA under the index set's mask (idx None: causal only)."""
    _check(lib().dsa_masked_mha_prefill(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_masked_mha_prefill")


def forward(p, kv, q_idx, w, kidx_cache, k_scale, q, kv_cache, kv_row_stride, out, lse, idx_out,
            ws, stream=None, paged=False):
    fn = lib().dsa_forward_paged if paged else lib().dsa_forward
    _check(fn(ctypes.byref(p), ctypes.byref(kv), _ptr(q_idx), _ptr(w), _ptr(kidx_cache),
              _ptr(k_scale), _ptr(q), _ptr(kv_cache), int(kv_row_stride), _ptr(out), _ptr(lse),
              _ptr(idx_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_forward_paged" if paged else "dsa_forward")


def make_project_params(*, nt, hidden, q_lora_rank, h_idx, d_idx, rope_dim=64, ln_eps=1e-6,
                        rope_theta=10000.0) -> ProjectParams:
    return ProjectParams(int(nt), int(hidden), int(q_lora_rank), int(h_idx), int(d_idx),
                         int(rope_dim), float(ln_eps), float(rope_theta))


def project_workspace_size(pp: ProjectParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dsa_project_workspace_size(ctypes.byref(pp), ctypes.byref(out)),
           "dsa_project_workspace_size")
    return int(out.value)


def indexer_project(pp, kv, x, q_lora, w_qb, w_k, w_proj, ln_gamma, ln_beta, positions, q_idx,
                    q_scale, w, kidx_cache, k_scale, ws, q_f32=None, k_f32=None, w_f32=None,
                    stream=None):
    _check(lib().dsa_indexer_project(
        ctypes.byref(pp), ctypes.byref(kv), _ptr(x), _ptr(q_lora), _ptr(w_qb), _ptr(w_k),
        _ptr(w_proj), _ptr(ln_gamma), _ptr(ln_beta), _ptr(positions), _ptr(q_idx), _ptr(q_scale),
        _ptr(w), _ptr(kidx_cache), _ptr(k_scale), _ptr(q_f32), _ptr(k_f32), _ptr(w_f32), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)), "dsa_indexer_project")


def make_table_params(*, nseq, nt, page_size, max_pages, n_free, cache_rows, sees_self=1) -> TableParams:
    return TableParams(int(nseq), int(nt), int(page_size), int(max_pages), int(n_free), int(sees_self),
                       int(cache_rows))


def table_workspace_size(tp: TableParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dsa_table_workspace_size(ctypes.byref(tp), ctypes.byref(out)), "dsa_table_workspace_size")
    return int(out.value)


def _device(what, t) -> int:
    """The GPU that tensor `t` of call `what` is on."""
    dev = t.get_device()
    if dev < 0:
        raise DsaError(DSA_ERR_INVALID_ARG, "%s: tensors must be on a CUDA device" % what)
    return dev


def _launch(fn, what, dev, stream, *args):
    """Call `fn` with GPU `dev` current, on the caller's stream or that
    device's current one."""
    torch = _torch()
    if stream is None:  # the raw handle: a Stream object costs a microsecond a call
        st = torch._C._cuda_getCurrentRawStream(dev)
    else:
        st = stream if isinstance(stream, int) else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc:
        _check(rc, what)


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


@functools.lru_cache(maxsize=None)
def _types(kind):
    """Element types the bindings take for `kind` (a name, or a dtype of the
    rotation); integers of the same size stand for the bits of a 16- or 8-bit
    float."""
    t = _torch()
    kind = {DTYPE_BF16: "bf16", DTYPE_FP16: "fp16", DTYPE_FP32: "fp32"}.get(kind, kind)
    if isinstance(kind, int):
        raise DsaError(DSA_ERR_INVALID_ARG, "unknown dtype %d" % kind)
    return {"i32": frozenset((t.int32, t.uint32)), "fp32": frozenset((t.float32,)),
            "bf16": frozenset((t.bfloat16, t.int16, t.uint16)), "fp16": frozenset((t.float16, t.int16, t.uint16)),
            "e4m3": frozenset((t.float8_e4m3fn, t.uint8, t.int8))}[kind]


def _refuse(what, need, t, dev):
    raise DsaError(DSA_ERR_INVALID_ARG, "%s: need %s on GPU %d; got %s %s of strides %s on %s"
                   % (what, need, dev, t.dtype, tuple(t.shape), tuple(t.stride()), t.device))


def _bytes(ws, dev) -> int:
    if ws.get_device() != dev:
        raise DsaError(DSA_ERR_WORKSPACE, "ws must be on GPU %d" % dev)
    return ws.numel() * ws.element_size()


def _dense(what, t, dev, kind, *shape):
    """The address of a contiguous tensor of this shape (or an address as it
    is); anything else the call would misread is refused."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev or t.dtype not in _types(kind) or t.shape != shape or not t.is_contiguous():
        _refuse(what, "contiguous %s of shape %s" % (kind, shape), t, dev)
    return t.data_ptr()


def _list(what, t, dev, n, kinds):
    """The address of n adjacent 4-byte elements (or an address)."""
    try:
        if t.get_device() == dev and t.dtype in kinds and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t
        raise
    _refuse(what, "%d adjacent %s" % (n, "/".join(sorted(str(k) for k in kinds))), t, dev)


def _joined(shape, strides, dims):
    """How many steps the first `dims` dimensions are together, and how far
    apart they lie (0 for one); None where they are not evenly spaced."""
    n, step = 1, 0
    for k in range(dims - 1, -1, -1):
        if shape[k] == 1:
            continue
        if n == 1:
            step = strides[k]
        elif strides[k] != n * step:
            return None
        n *= shape[k]
    return n, step


def _heads(what, t, dev, kind, nt, heads, d, ts, hs):
    """The address of the rows [nt, heads, d] whose tokens are `ts` and heads
    `hs` elements apart.  `t` is that view itself (tokens in one dimension or
    several, perhaps more of them), the same with heads and elements joined,
    [.., heads * d], or a flat buffer."""
    if t.get_device() == dev and t.dtype in _types(kind):
        shape = t.shape
        if nt == 0 or shape == (nt, heads, d) and hs == d and ts == heads * d and t.is_contiguous():
            return t.data_ptr()   # the usual call
        strides = t.stride()
        ends = len(shape) > 0 and (strides[-1] == 1 or shape[-1] == 1)
        dims = -1     # of the tokens
        if ends and shape[-2:] == (heads, d) and (heads == 1 or strides[-2] == hs):
            dims = len(shape) - 2
        elif ends and shape[-1] == heads * d and (heads == 1 or hs == d):
            dims = len(shape) - 1
        if dims >= 0:
            tokens = _joined(shape, strides, dims)
            if tokens and (tokens[0] == nt or dims == 1 and tokens[0] > nt) and (nt == 1 or tokens[1] == ts):
                return t.data_ptr()
        if ends and len(shape) == 1 and shape[0] >= (nt - 1) * ts + (heads - 1) * hs + d:
            return t.data_ptr()
    _refuse(what, "%s rows [%d, %d, %d] of strides (%d, %d, 1)" % (("bf16", "fp16", "fp32")[kind], nt, heads, d, ts, hs), t, dev)


def build_tables(tp, seq_len, new_len, fork_src, free_pages, free_head, page_table, q_start, q_seq,
                 positions, q_n, slots, kv_len, free_head_out, ws, stream=None):
    """Page tables and slot maps of one step from the requests' lengths."""
    n, nt, dev, i32 = tp.nseq, tp.nt, _device("dsa_build_tables", q_start), _types("i32")
    _launch(lib().dsa_build_tables, "dsa_build_tables", dev, stream, ctypes.byref(tp),
            _list("seq_len", seq_len, dev, n, i32), _list("new_len", new_len, dev, n, i32),
            _list("fork_src", fork_src, dev, n, i32), _list("free_pages", free_pages, dev, tp.n_free, i32),
            _list("free_head", free_head, dev, 1, i32), _dense("page_table", page_table, dev, "i32", n, tp.max_pages),
            _list("q_start", q_start, dev, n + 1, i32), _list("q_seq", q_seq, dev, nt, i32),
            _list("positions", positions, dev, nt, i32), _list("q_n", q_n, dev, nt, i32),
            _list("slots", slots, dev, nt, i32), _list("kv_len", kv_len, dev, n, i32),
            _list("free_head_out", free_head_out, dev, 1, i32), ws.data_ptr(), _bytes(ws, dev))


def make_rope_spec(*, rope_dim=64, layout=ROPE_INTERLEAVED, theta=10000.0, scaling=ROPE_SCALE_NONE, factor=1.0,
                   orig_max_pos=0, beta_fast=32.0, beta_slow=1.0, mscale=1.0) -> RopeSpec:
    return RopeSpec(int(rope_dim), int(layout), int(scaling), int(orig_max_pos), float(theta), float(factor),
                    float(beta_fast), float(beta_slow), float(mscale))


def make_rope_params(*, nt, h, d, dtype, x_heads=None, begin=0, x_strides=None, y_strides=None) -> RopeParams:
    """x_strides / y_strides: (token, head) strides in elements, densely
    packed when not given."""
    x_heads = h if x_heads is None else x_heads
    x_strides = (x_heads * d, d) if x_strides is None else x_strides
    y_strides = (h * d, d) if y_strides is None else y_strides
    return RopeParams(int(nt), int(h), int(x_heads), int(d), int(begin), int(dtype), int(x_strides[0]),
                      int(x_strides[1]), int(y_strides[0]), int(y_strides[1]))


def _rope(fn, what, rs, rp, src, positions, dst, stream, backward):
    dev, kind, nt, h, d = _device(what, positions), rp.dtype, rp.nt, rp.h, rp.d
    x, y = (dst, src) if backward else (src, dst)
    xp = _heads("dx" if backward else "x", x, dev, kind, nt, rp.x_heads, d, rp.x_token_stride, rp.x_head_stride)
    yp = _heads("dy" if backward else "y", y, dev, kind, nt, h, d, rp.y_token_stride, rp.y_head_stride)
    _launch(fn, what, dev, stream, ctypes.byref(rs), ctypes.byref(rp), yp if backward else xp,
            _list("positions", positions, dev, nt, _types("i32")), xp if backward else yp)


def rope(rs, rp, x, positions, y, stream=None):
    """Rotary positions: y = x with its rotated range turned (y may be x).
    x and y are [nt, x_heads, d] and [nt, h, d] with rp's strides."""
    _rope(lib().dsa_rope, "dsa_rope", rs, rp, x, positions, y, stream, False)


def rope_backward(rs, rp, dy, positions, dx, stream=None):
    """Gradient of rope (summed over the heads of a shared x)."""
    _rope(lib().dsa_rope_backward, "dsa_rope_backward", rs, rp, dy, positions, dx, stream, True)


def _part(what, t, dev, nt, width):
    """The address of [nt, width] bf16 rows, each one's elements adjacent."""
    if t.get_device() != dev or t.dtype not in _types("bf16") or t.shape != (nt, width) or (nt > 0 and t.stride(1) != 1):
        _refuse(what, "bf16 rows [%d, %d], each one's elements adjacent," % (nt, width), t, dev)
    return t.data_ptr()


def _cache(what, t, dev, kind):
    """The address and row stride of a latent cache [rows, >= 576]."""
    if t.get_device() == dev and t.dtype in _types(kind) and t.dim() == 2 and t.shape[1] >= 576:
        stride, inner = t.stride()
        if inner == 1:
            return t.data_ptr(), stride
    _refuse(what, "%s rows [rows, >= 576], each one's elements adjacent," % kind, t, dev)


def _cache_rows(what, t, dev, kind, rows, row_stride):
    """The address of a latent cache of `rows` rows, `row_stride` elements
    apart: [.., >= 576] (rows, or pages of rows one behind the other), or a
    flat buffer (or an address)."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() == dev and t.dtype in _types(kind):
        shape, strides = t.shape, t.stride()
        if len(shape) == 1:
            if strides[0] == 1 and shape[0] >= (rows - 1) * row_stride + 576:
                return t.data_ptr()
        elif len(shape) > 1 and shape[-1] >= 576 and strides[-1] == 1:
            n = _joined(shape, strides, len(shape) - 1)
            if n and n[0] >= rows and (n[0] == 1 or n[1] == row_stride):
                return t.data_ptr()
    _refuse(what, "%s, %d rows of >= 576 elements, %d apart," % (kind, rows, row_stride), t, dev)


def latent_append(rs, c_kv, k_pe, positions, slots, kv_cache, ws, stream=None):
    """Append [c_kv | rope(k_pe)] rows to the bf16 latent cache [rows, >= 576]."""
    nt, dev, i32 = slots.shape[0], _device("dsa_latent_append", slots), _types("i32")
    cache, stride = _cache("kv_cache", kv_cache, dev, "bf16")
    _launch(lib().dsa_latent_append, "dsa_latent_append", dev, stream, ctypes.byref(rs), nt,
            _part("c_kv", c_kv, dev, nt, 512), c_kv.stride(0), _part("k_pe", k_pe, dev, nt, 64), k_pe.stride(0),
            _list("positions", positions, dev, nt, i32), _list("slots", slots, dev, nt, i32), cache, stride,
            kv_cache.shape[0], ws.data_ptr(), _bytes(ws, dev))


def latent_append_fp8(rs, c_kv, k_pe, positions, slots, kv8_cache, kv_scale, ws, stream=None):
    """The same into the FP8 latent cache [rows, >= 576] (e4m3 codes, power-of-two row scales)."""
    nt, dev, i32 = slots.shape[0], _device("dsa_latent_append_fp8", slots), _types("i32")
    rows = kv8_cache.shape[0]
    cache, stride = _cache("kv8_cache", kv8_cache, dev, "e4m3")
    _launch(lib().dsa_latent_append_fp8, "dsa_latent_append_fp8", dev, stream, ctypes.byref(rs), nt,
            _part("c_kv", c_kv, dev, nt, 512), c_kv.stride(0), _part("k_pe", k_pe, dev, nt, 64), k_pe.stride(0),
            _list("positions", positions, dev, nt, i32), _list("slots", slots, dev, nt, i32), cache, stride,
            _list("kv_scale", kv_scale, dev, rows, _types("fp32")), rows, ws.data_ptr(), _bytes(ws, dev))


def shared_prefix_workspace_size(p: Params, kv: KV, ngroups: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dsa_shared_prefix_workspace_size(ctypes.byref(p), ctypes.byref(kv), int(ngroups),
                                                  ctypes.byref(out)), "dsa_shared_prefix_workspace_size")
    return int(out.value)


def mla_shared_prefix(p, kv, ngroups, group_q0, group_n, q, kv_cache, kv_row_stride, out, lse, ws, stream=None):
    """Dense MLA attention of queries in groups that share a prefix, each
    prefix read once for the whole group."""
    nq, h, dev, i32 = p.nq, p.h, _device("dsa_mla_shared_prefix", group_q0), _types("i32")
    _launch(lib().dsa_mla_shared_prefix, "dsa_mla_shared_prefix", dev, stream, ctypes.byref(p), ctypes.byref(kv),
            ngroups, _list("group_q0", group_q0, dev, ngroups + 1, i32), _list("group_n", group_n, dev, ngroups, i32),
            _dense("q", q, dev, "bf16", nq, h, 576),
            _cache_rows("kv_cache", kv_cache, dev, "bf16", kv.cache_rows, kv_row_stride), kv_row_stride,
            _dense("out", out, dev, "bf16", nq, h, 512), _dense("lse", lse, dev, "fp32", nq, h), ws.data_ptr(),
            _bytes(ws, dev))


def check_status(ws, stream=None) -> int:
    """Synchronise the stream and return (then clear) the device status word."""
    return int(lib().dsa_check_status(_ptr(ws), _stream(stream)))
