"""ctypes binding of libfastar.so: one Python function per C entry point, same name.

Argument marshalling only: tensors become (pointer, strides), the current CUDA
stream is passed through, and a non-zero return code raises FastarError.  All
computation happens in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfastar.so")

F32, BF16 = 0, 1
OK, EINVAL, EUNSUPPORTED, ECAPACITY, EWORKSPACE, ECUDA = 0, -1, -2, -3, -4, -5
DEV_BAD_LEN, DEV_BAD_BUCKET, DEV_BAD_INDEX = 1, 2, 4
DEV_TIMEOUT, DEV_NONFINITE = 8, 16
OP_MATCH, OP_SORT, OP_SPARSE_ATTN, OP_ANNCA, OP_MATCH_ANN, OP_CROSS_ATTN, OP_MATCH_PQ = 1, 2, 3, 4, 5, 6, 7
OP_KV4_ATTN, OP_PAGED_ATTN = 8, 9
MAX_B, MAX_R, MAX_P = 256, 8, 1024

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float
_S = ctypes.c_size_t

# name -> argtypes (restype int unless listed in _RESTYPES)
_SIGS = {
    "fastar_version": [],
    "fastar_kernel_launches": [],
    "fastar_last_cuda_error": [],
    "fastar_status_string": [_I],
    "fastar_workspace_bytes": [_I, _I, _L, _L, _I, _I, _I, _L, _I],
    "fastar_bucket_assign": [_P, _I, _I, _L, _I, _L, _L, _P, _I, _I, _P, _P, _P, _P],
    "fastar_bucket_assign_qk": [_P, _P, _I, _I, _L, _I, _L, _L, _P, _I, _I, _P, _P, _P, _P, _P],
    "fastar_tempcache_match": [_P, _P, _I, _I, _L, _I, _L, _L, _P, _P, _P, _L, _F, _P, _P, _P, _P, _P, _P, _P,
                               _S, _P],
    "fastar_tempcache_match_ann": [_P, _P, _I, _I, _L, _I, _L, _L, _I, _I, _P, _P, _P, _P, _P, _L, _P, _P, _F, _P,
                                   _P, _P, _P, _P, _P, _S, _P],
    "fastar_cache_compact": [_I, _I, _L, _I, _L, _P, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                             _P, _P, _P, _P],
    "fastar_cache_compact_merge": [_I, _I, _L, _I, _L, _P, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "fastar_cache_compact_sorted": [_I, _I, _L, _I, _L, _P, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P],
    "fastar_bucket_sort": [_P, _I, _L, _I, _I, _P, _P, _P, _P, _P],
    "fastar_pq_encode": [_P, _I, _I, _L, _I, _L, _L, _P, _I, _I, _P, _P],
    "fastar_tempcache_match_pq": [_P, _P, _I, _I, _L, _I, _L, _L, _P, _P, _P, _P, _L, _P, _I, _I, _F, _P, _P, _P,
                                  _P, _P, _P, _S, _P],
    "fastar_pq_gather_codes": [_I, _L, _L, _I, _P, _P, _P, _P, _P, _P, _P, _P],
    "fastar_sparse_attn": [_P, _I, _I, _L, _I, _L, _L, _I, _I, _P, _P, _P, _P, _L, _P, _P, _F, _P, _L, _L, _P, _P,
                           _P, _S, _P],
    "fastar_sparse_attn_grouped": [_P, _I, _I, _L, _I, _L, _L, _I, _I, _P, _P, _P, _P, _L, _P, _P, _P, _F, _P, _L,
                                   _L, _P, _P, _P, _S, _P],
    "fastar_sparse_attn_presorted": [_P, _I, _I, _L, _I, _L, _L, _I, _I, _P, _P, _P, _P, _L, _P, _P, _P, _P, _F,
                                     _P, _L, _L, _P, _P, _P, _S, _P],
    "fastar_annca_select": [_P, _I, _I, _I, _L, _I, _L, _L, _P, _I, _P, _P, _L, _F, _I, _I, _I, _P, _P, _P, _P, _P,
                            _P, _P, _P, _P, _P, _P, _S, _P],
    "fastar_annca_select_noalloc": [_P, _I, _I, _I, _L, _I, _L, _L, _P, _I, _P, _P, _L, _F, _I, _I, _P, _P, _P, _P],
    "fastar_cross_attn_subset": [_P, _I, _I, _I, _L, _I, _L, _L, _P, _P, _L, _P, _P, _F, _P, _L, _L, _P, _P, _S,
                                 _P],
    "fastar_cross_attn_kept": [_P, _I, _I, _I, _L, _I, _L, _L, _P, _P, _L, _P, _F, _P, _L, _L, _P, _P],
    "fastar_dense_attn": [_P, _I, _I, _L, _I, _L, _L, _P, _P, _L, _L, _L, _F, _P, _L, _L, _P, _P],
    "fastar_dense_attn_grouped": [_P, _I, _I, _L, _I, _L, _L, _P, _P, _L, _L, _L, _P, _L, _F, _P, _L, _L, _P, _P],
    "fastar_dense_append": [_I, _I, _L, _I, _P, _P, _L, _L, _P, _P, _L, _L, _P],
    "fastar_gemm": [_P, _L, _P, _L, _P, _P, _L, _P, _P, _P, _L, _I, _L, _L, _L, _I, _P, _P],
    "fastar_layernorm_mod": [_P, _L, _L, _I, _F, _P, _P, _P, _P, _P, _P, _P, _L, _P],
    "fastar_rmsnorm_rope": [_P, _L, _L, _I, _I, _F, _P, _I, _I, _P, _I, _I, _F, _P],
    "fastar_sinusoidal_embedding": [_P, _I, _I, _P, _L, _P],
    "fastar_qk_norm_rope": [_I, _L, _I, _I, _P, _L, _L, _P, _L, _L, _I, _P, _L, _L, _P, _L, _L, _P, _P, _F, _I, _I,
                            _I, _P, _I, _P, _I, _I, _F, _P],
    "fastar_kv4_append": [_I, _I, _L, _I, _P, _L, _L, _P, _L, _L, _P, _P, _P, _P, _P, _P, _P, _L, _P, _P, _P],
    "fastar_kv4_read": [_I, _I, _L, _I, _P, _P, _P, _L, _L, _P, _L, _L, _P],
    "fastar_kv4_attn": [_P, _I, _I, _I, _L, _I, _L, _L, _P, _P, _P, _P, _P, _P, _L, _P, _L, _F, _P, _L, _L, _P, _P,
                        _P, _S, _P],
    "fastar_paged_append": [_I, _I, _L, _P, _I, _I, _P, _L, _L, _P, _L, _L, _I, _P, _L, _L, _P, _L, _L, _P, _P, _F, _I,
                            _I, _I, _P, _I, _I, _F, _P, _P, _L, _I, _L, _L, _L, _P, _L, _P, _P, _P, _P],
    "fastar_paged_attn": [_P, _I, _I, _L, _P, _L, _I, _I, _I, _L, _L, _P, _P, _L, _I, _L, _L, _L, _P, _L, _P, _L, _L,
                          _L, _F, _P, _L, _L, _P, _P, _P, _S, _P],
    "fastar_packed_call": [_I, _P, _I],
}
_RESTYPES = {"fastar_status_string": ctypes.c_char_p, "fastar_workspace_bytes": ctypes.c_size_t,
             "fastar_kernel_launches": ctypes.c_longlong, "fastar_last_cuda_error": ctypes.c_char_p}

_lib: Optional[ctypes.CDLL] = None


class FastarError(RuntimeError):
    def __init__(self, name: str, code: int, detail: str | None = None):
        msg = f"{name} returned {code}: {status_string(code)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.code = code
        self.detail = detail


def open_library(path: str) -> ctypes.CDLL:
    """Opens a libfastar build and declares every symbol; raises if it is missing."""
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m kv_cache_tempcache_gb300.build_lib`")
    lib = ctypes.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _RESTYPES.get(name, ctypes.c_int)
    return lib


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """The process-wide libfastar handle (opened on first use)."""
    global _lib
    if _lib is None:
        _lib = open_library(path)
    return _lib


def symbols():
    return list(_SIGS)


def status_string(code: int) -> str:
    return load().fastar_status_string(int(code)).decode()


def version() -> int:
    return load().fastar_version()


def kernel_launches() -> int:
    return int(load().fastar_kernel_launches())


def workspace_bytes(op, H, n, M=0, d=128, B=1, r=1, P=0, F=0) -> int:
    return int(load().fastar_workspace_bytes(op, H, n, M, d, B, r, P, F))


# ---- marshalling helpers -------------------------------------------------------------------

def dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t}")


def ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Device address of a tensor the library addresses as dense (None -> NULL)."""
    if t is None:
        return None
    if not t.is_contiguous() and t.dim() == 3 and t.stride(2) == 1:
        return t.data_ptr()          # a strided token view; strides are passed separately
    if not t.is_contiguous():
        raise ValueError("index/metadata/output buffers must be contiguous")
    return t.data_ptr()


def stream_handle(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def tok_strides(t: torch.Tensor):
    """(head_stride, token_stride) of a [H, N, d] view with a contiguous last dim."""
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError("token tensors must be [H, N, d] views with a contiguous last dimension")
    return t.stride(0), t.stride(1)


def _call(name, *args):
    lib = load()
    rc = getattr(lib, name)(*args)
    if rc != OK:
        detail = lib.fastar_last_cuda_error().decode() if rc == ECUDA else None
        raise FastarError(name, rc, detail)


# ---- entry points --------------------------------------------------------------------------

def fastar_bucket_assign(x, centroids, r, ids, scores=None, norms=None, stream=None):
    H, n, d = x.shape
    hs, ts = tok_strides(x)
    _call("fastar_bucket_assign", ptr(x), dtype_code(x.dtype), H, n, d, hs, ts, ptr(centroids),
          centroids.shape[1], r, ptr(ids), ptr(scores), ptr(norms), stream_handle(stream))


def fastar_bucket_assign_qk(q, k_cur, centroids, r, q_ids, k_ids, k_norms=None, stream=None, q_norms=None):
    H, n, d = q.shape
    hs, ts = tok_strides(q)
    if tok_strides(k_cur) != (hs, ts):
        raise ValueError("q and k_cur must share strides")
    _call("fastar_bucket_assign_qk", ptr(q), ptr(k_cur), dtype_code(q.dtype), H, n, d, hs, ts, ptr(centroids),
          centroids.shape[1], r, ptr(q_ids), ptr(k_ids), ptr(k_norms), ptr(q_norms), stream_handle(stream))


def fastar_tempcache_match(q, k_cur, cache_k, cache_knorm, cache_len, tau, top1, s1, s2, evict, dev_status,
                           workspace, stream=None, owner=None):
    H, nq, d = q.shape
    hs, ts = tok_strides(q)
    if tok_strides(k_cur) != (hs, ts):
        raise ValueError("q and k_cur must share strides")
    _call("fastar_tempcache_match", ptr(q), ptr(k_cur), dtype_code(q.dtype), H, nq, d, hs, ts, ptr(cache_k),
          ptr(cache_knorm), ptr(cache_len), cache_k.shape[1], float(tau), ptr(top1), ptr(s1), ptr(s2), ptr(evict),
          ptr(owner), ptr(dev_status), ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), stream_handle(stream))


def fastar_tempcache_match_ann(q, k_cur, r, B, qperm, qoff, cache_k, cache_knorm, cache_len, kperm, koff, tau,
                               top1, s1, evict, dev_status, workspace, stream=None, owner=None):
    H, nq, d = q.shape
    hs, ts = tok_strides(q)
    if tok_strides(k_cur) != (hs, ts):
        raise ValueError("q and k_cur must share strides")
    _call("fastar_tempcache_match_ann", ptr(q), ptr(k_cur), dtype_code(q.dtype), H, nq, d, hs, ts, int(r), int(B),
          ptr(qperm), ptr(qoff), ptr(cache_k), ptr(cache_knorm), ptr(cache_len), cache_k.shape[1], ptr(kperm),
          ptr(koff), float(tau), ptr(top1), ptr(s1), ptr(evict), ptr(owner), ptr(dev_status), ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), stream_handle(stream))


def fastar_cache_compact(k_cur, v_cur, kcur_norm, kcur_bucket, k_in, v_in, knorm_in, kb_in, len_in, evict,
                         k_out, v_out, knorm_out, kb_out, len_out, index_map, dev_status, stream=None):
    H, nq, d = k_cur.shape
    hs, ts = tok_strides(k_cur)
    if tok_strides(v_cur) != (hs, ts):
        raise ValueError("k_cur and v_cur must share strides")
    _call("fastar_cache_compact", dtype_code(k_cur.dtype), H, nq, d, k_in.shape[1], ptr(k_cur), ptr(v_cur), hs,
          ts, ptr(kcur_norm), ptr(kcur_bucket), ptr(k_in), ptr(v_in), ptr(knorm_in), ptr(kb_in), ptr(len_in),
          ptr(evict), ptr(k_out), ptr(v_out), ptr(knorm_out), ptr(kb_out), ptr(len_out), ptr(index_map),
          ptr(dev_status), stream_handle(stream))


def fastar_cache_compact_sorted(k_cur, v_cur, kcur_norm, kcur_bucket, k_in, v_in, knorm_in, kb_in, len_in, evict,
                                k_out, v_out, knorm_out, kb_out, len_out, index_map, B, kperm, koff, kpos, k_sorted,
                                v_sorted, dev_status, stream=None, qb=None, qperm=None, qoff=None):
    """qb [H, nq, r] int32 (optional): also sort the step's (query, slot) pairs by bucket
    into qperm [H, nq*r] and qoff [H, B+1] in the same launch as the key sort."""
    H, nq, d = k_cur.shape
    hs, ts = tok_strides(k_cur)
    if tok_strides(v_cur) != (hs, ts):
        raise ValueError("k_cur and v_cur must share strides")
    _call("fastar_cache_compact_sorted", dtype_code(k_cur.dtype), H, nq, d, k_in.shape[1], ptr(k_cur), ptr(v_cur),
          hs, ts, ptr(kcur_norm), ptr(kcur_bucket), ptr(k_in), ptr(v_in), ptr(knorm_in), ptr(kb_in), ptr(len_in),
          ptr(evict), ptr(k_out), ptr(v_out), ptr(knorm_out), ptr(kb_out), ptr(len_out), ptr(index_map), int(B),
          ptr(kperm), ptr(koff), ptr(kpos), ptr(k_sorted), ptr(v_sorted), ptr(qb),
          int(qb.shape[2]) if qb is not None else 0, ptr(qperm), ptr(qoff), ptr(dev_status), stream_handle(stream))


def fastar_cache_compact_merge(k_cur, v_cur, kcur_norm, kcur_bucket, k_in, v_in, knorm_in, kb_in, g_in, len_in,
                               evict, top1, owner, k_out, v_out, knorm_out, kb_out, g_out, len_out, index_map,
                               dev_status, stream=None):
    H, nq, d = k_cur.shape
    hs, ts = tok_strides(k_cur)
    if tok_strides(v_cur) != (hs, ts):
        raise ValueError("k_cur and v_cur must share strides")
    _call("fastar_cache_compact_merge", dtype_code(k_cur.dtype), H, nq, d, k_in.shape[1], ptr(k_cur), ptr(v_cur),
          hs, ts, ptr(kcur_norm), ptr(kcur_bucket), ptr(k_in), ptr(v_in), ptr(knorm_in), ptr(kb_in), ptr(g_in),
          ptr(len_in), ptr(evict), ptr(top1), ptr(owner), ptr(k_out), ptr(v_out), ptr(knorm_out), ptr(kb_out),
          ptr(g_out), ptr(len_out), ptr(index_map), ptr(dev_status), stream_handle(stream))


def fastar_pq_encode(x, codebooks, codes, stream=None):
    """codebooks [H, m, Kc, d/m]; codes [H, n, m] uint8."""
    H, n, d = x.shape
    hs, ts = tok_strides(x)
    _call("fastar_pq_encode", ptr(x), dtype_code(x.dtype), H, n, d, hs, ts, ptr(codebooks), codebooks.shape[1],
          codebooks.shape[2], ptr(codes), stream_handle(stream))


def fastar_tempcache_match_pq(q, k_cur, cache_k, cache_knorm, cache_codes, cache_len, codebooks, tau, top1, s1,
                              evict, dev_status, workspace, stream=None, owner=None):
    H, nq, d = q.shape
    hs, ts = tok_strides(q)
    if tok_strides(k_cur) != (hs, ts):
        raise ValueError("q and k_cur must share strides")
    _call("fastar_tempcache_match_pq", ptr(q), ptr(k_cur), dtype_code(q.dtype), H, nq, d, hs, ts, ptr(cache_k),
          ptr(cache_knorm), ptr(cache_codes), ptr(cache_len), cache_k.shape[1], ptr(codebooks), codebooks.shape[1],
          codebooks.shape[2], float(tau), ptr(top1), ptr(s1), ptr(evict), ptr(owner), ptr(dev_status),
          ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
          stream_handle(stream))


def fastar_pq_gather_codes(codes_in, len_in, codes_cur, index_map, len_out, codes_out, dev_status=None,
                           stream=None):
    H, M, m = codes_in.shape
    _call("fastar_pq_gather_codes", H, codes_cur.shape[1], M, m, ptr(codes_in), ptr(len_in), ptr(codes_cur),
          ptr(index_map), ptr(len_out), ptr(codes_out), ptr(dev_status), stream_handle(stream))


def fastar_bucket_sort(ids, B, perm, offsets, n_valid=None, dev_status=None, stream=None):
    H, n, r = ids.shape
    _call("fastar_bucket_sort", ptr(ids), H, n, r, B, ptr(n_valid), ptr(perm), ptr(offsets), ptr(dev_status),
          stream_handle(stream))


def fastar_sparse_attn(q, r, B, qperm, qoff, k, v, kperm, koff, scale, out, lse, dev_status, workspace,
                       stream=None):
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    oh, ot = tok_strides(out)
    _call("fastar_sparse_attn", ptr(q), dtype_code(q.dtype), H, nq, d, qh, qt, r, B, ptr(qperm), ptr(qoff), ptr(k),
          ptr(v), k.shape[1], ptr(kperm), ptr(koff), float(scale), ptr(out), oh, ot, ptr(lse), ptr(dev_status),
          ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
          stream_handle(stream))


def fastar_sparse_attn_presorted(q, r, B, qperm, qoff, k, v, kperm, koff, k_sorted, v_sorted, scale, out, lse,
                                 dev_status, workspace, stream=None):
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    oh, ot = tok_strides(out)
    _call("fastar_sparse_attn_presorted", ptr(q), dtype_code(q.dtype), H, nq, d, qh, qt, r, B, ptr(qperm),
          ptr(qoff), ptr(k), ptr(v), k.shape[1], ptr(kperm), ptr(koff), ptr(k_sorted), ptr(v_sorted), float(scale),
          ptr(out), oh, ot, ptr(lse), ptr(dev_status), ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), stream_handle(stream))


def fastar_sparse_attn_grouped(q, r, B, qperm, qoff, k, v, kperm, koff, group_count, scale, out, lse, dev_status,
                               workspace, stream=None):
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    oh, ot = tok_strides(out)
    _call("fastar_sparse_attn_grouped", ptr(q), dtype_code(q.dtype), H, nq, d, qh, qt, r, B, ptr(qperm), ptr(qoff),
          ptr(k), ptr(v), k.shape[1], ptr(kperm), ptr(koff), ptr(group_count), float(scale), ptr(out), oh, ot,
          ptr(lse), ptr(dev_status), ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), stream_handle(stream))


def fastar_annca_select(q, F, qb, kp, pb, tau_ca, topk, gate, keep, kidx, kcnt, score=None, workspace=None,
                        stream=None, B=0, qperm=None, qoff=None, vp=None, kp_kept=None, vp_kept=None, q_norms=None):
    """kp_kept / vp_kept [H, F, P, d] (optional, with vp): the kept rows copied by the
    ranking launch, fastar_cross_attn_kept's input.  q_norms [H, F * tpf] (optional): the
    queries' norms as fastar_bucket_assign_qk writes them."""
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    tpf = nq // F
    _call("fastar_annca_select", ptr(q), dtype_code(q.dtype), H, F, tpf, d, qh, qt, ptr(qb), qb.shape[2], ptr(kp),
          ptr(pb), kp.shape[1], float(tau_ca), int(topk), int(gate), int(B), ptr(qperm), ptr(qoff), ptr(q_norms),
          ptr(keep),
          ptr(kidx), ptr(kcnt), ptr(score), ptr(vp), ptr(kp_kept), ptr(vp_kept),
          ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
          stream_handle(stream))


def fastar_annca_select_noalloc(q, F, qb, kp, pb, tau_ca, topk, gate, keep, kidx, kcnt, stream=None):
    """fastar_annca_select for callers that cannot allocate: the scores go to the
    library's fixed scratch array (no workspace, no score output)."""
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    tpf = nq // F
    _call("fastar_annca_select_noalloc", ptr(q), dtype_code(q.dtype), H, F, tpf, d, qh, qt, ptr(qb), qb.shape[2],
          ptr(kp), ptr(pb), kp.shape[1], float(tau_ca), int(topk), int(gate), ptr(keep), ptr(kidx), ptr(kcnt),
          stream_handle(stream))


def fastar_cross_attn_subset(q, F, kp, vp, kidx, kcnt, scale, out, lse=None, stream=None, workspace=None):
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    oh, ot = tok_strides(out)
    _call("fastar_cross_attn_subset", ptr(q), dtype_code(q.dtype), H, F, nq // F, d, qh, qt, ptr(kp), ptr(vp),
          kp.shape[1], ptr(kidx), ptr(kcnt), float(scale), ptr(out), oh, ot, ptr(lse), ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), stream_handle(stream))


def fastar_cross_attn_kept(q, F, kp_kept, vp_kept, kcnt, scale, out, lse=None, stream=None):
    """Cross-attention over the kept-row planes [H, F, P, d] fastar_annca_select wrote."""
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    oh, ot = tok_strides(out)
    _call("fastar_cross_attn_kept", ptr(q), dtype_code(q.dtype), H, F, nq // F, d, qh, qt, ptr(kp_kept),
          ptr(vp_kept), kp_kept.shape[2], ptr(kcnt), float(scale), ptr(out), oh, ot, ptr(lse), stream_handle(stream))


def fastar_dense_attn(q, k, v, nk, scale, out, lse=None, stream=None):
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    kh, kt = tok_strides(k)
    oh, ot = tok_strides(out)
    _call("fastar_dense_attn", ptr(q), dtype_code(q.dtype), H, nq, d, qh, qt, ptr(k), ptr(v), int(nk), kh, kt,
          float(scale), ptr(out), oh, ot, ptr(lse), stream_handle(stream))


def fastar_dense_attn_grouped(q, k, v, nk, group_count, scale, out, lse=None, stream=None):
    """group_count: [H, >= nk] int32 (row stride = its second dimension)."""
    H, nq, d = q.shape
    qh, qt = tok_strides(q)
    kh, kt = tok_strides(k)
    oh, ot = tok_strides(out)
    _call("fastar_dense_attn_grouped", ptr(q), dtype_code(q.dtype), H, nq, d, qh, qt, ptr(k), ptr(v), int(nk), kh,
          kt, ptr(group_count), group_count.shape[1], float(scale), ptr(out), oh, ot, ptr(lse),
          stream_handle(stream))


ACT_NONE, ACT_GELU_TANH, ACT_SILU = 0, 1, 2


def fastar_gemm(A, W, C, bias=None, R=None, gate_a=None, gate_b=None, act=ACT_NONE, dev_status=None, stream=None):
    """C = R + gate * act(A @ W^T + bias); A [M, K], W [N, K], C/R [M, N] (2-D row views)."""
    M, K = A.shape
    N = W.shape[0]
    for t in (A, W, C) + ((R,) if R is not None else ()):
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("GEMM operands must be 2-D row-major views")
    _call("fastar_gemm", A.data_ptr(), A.stride(0), W.data_ptr(), W.stride(0), ptr(bias),
          None if R is None else R.data_ptr(), 0 if R is None else R.stride(0), ptr(gate_a), ptr(gate_b),
          C.data_ptr(), C.stride(0), dtype_code(C.dtype), M, N, K, int(act), ptr(dev_status), stream_handle(stream))


def fastar_layernorm_mod(x, out, eps=1e-6, weight=None, bias=None, shift_a=None, shift_b=None, scale_a=None,
                         scale_b=None, stream=None):
    """out = LN(x) [* weight + bias] * (1 + scale) + shift over the rows of x [n, C]."""
    n, C = x.shape
    _call("fastar_layernorm_mod", x.data_ptr(), x.stride(0), n, C, float(eps), ptr(weight), ptr(bias), ptr(shift_a),
          ptr(shift_b), ptr(scale_a), ptr(scale_b), out.data_ptr(), out.stride(0), stream_handle(stream))


def fastar_rmsnorm_rope(x, d, weight=None, rope=False, t0=0, grid=(1, 1), eps=1e-6, theta=10000.0, stream=None,
                        t0_dev=None):
    """In place on x [n, C]: RMS norm (weight given) then rotary positions (rope); the
    chunk's first frame is t0 + t0_dev[0] (t0_dev: optional device int32)."""
    n, C = x.shape
    _call("fastar_rmsnorm_rope", x.data_ptr(), x.stride(0), n, C, int(d), float(eps), ptr(weight), int(bool(rope)),
          int(t0), ptr(t0_dev), int(grid[0]), int(grid[1]), float(theta), stream_handle(stream))


def fastar_sinusoidal_embedding(t, out, stream=None):
    nb, dim = out.shape
    _call("fastar_sinusoidal_embedding", ptr(t), nb, dim, out.data_ptr(), out.stride(0), stream_handle(stream))


# ---- the 4-bit cache, the norm and rotation before it, the paged cache -------------------------

# Every check below refuses what a kernel would misread.  They run on each call of a step that
# may be a few microseconds of device time, so a call asks for everything in one expression, without
# helpers (a Python call is 0.1 us), and only what fails it is looked at again, tensor by tensor,
# for the message.  The stride of a dimension of one element says nothing (torch may give any):
# a call passes the dense one.

_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_device = getattr(torch._C, "_cuda_getDevice", None)                  # not in builds without CUDA
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _packer(call, name):
    """(call, pack, n) for fastar_packed_call: the arguments of `name` as 64-bit words.  One ctypes
    argument instead of up to thirty, 2 us less a call."""
    args = _SIGS[name]
    return call, struct.Struct("=" + "".join("d" if a is _F else "q" for a in args)).pack, len(args)


_CALL_ROPE, _PACK_ROPE, _N_ROPE = _packer(0, "fastar_qk_norm_rope")
_CALL_APPEND, _PACK_APPEND, _N_APPEND = _packer(1, "fastar_kv4_append")
_CALL_READ, _PACK_READ, _N_READ = _packer(2, "fastar_kv4_read")
_CALL_ATTN, _PACK_ATTN, _N_ATTN = _packer(3, "fastar_kv4_attn")
_CALL_PAPPEND, _PACK_PAPPEND, _N_PAPPEND = _packer(4, "fastar_paged_append")
_CALL_PATTN, _PACK_PATTN, _N_PATTN = _packer(5, "fastar_paged_attn")


def _refuse(rows, dense):
    """Raises for the first tensor that is not as expected.  rows: (name, [H, n, d] view, dtype,
    shape); dense: (name, contiguous tensor or None, dtype, shape)."""
    for name, t, dtype, shape in rows + dense:
        if t is None:
            continue
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    for name, t, _, _ in rows:
        if t is not None and t.stride(2) != 1:
            raise ValueError(f"{name}: token tensors must be [H, N, d] views with a contiguous last dimension")
    for name, t, _, _ in dense:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("tensors must be on the current CUDA device, all of them")


def _dims3(name, t):
    s = t.shape
    if len(s) != 3:
        raise ValueError(f"{name} must have three dimensions, not {len(s)}")
    return s


def _raise_dtype(dt):
    raise TypeError(f"unsupported dtype {dt}")


def _raise(name, rc):
    raise FastarError(name, rc, load().fastar_last_cuda_error().decode() if rc == ECUDA else None)


def fastar_qk_norm_rope(q, k, q_out, k_out, wq=None, wk=None, eps=1e-6, axes=(0, 0, 0), pos=None, t0=0, t0_dev=None,
                        grid=(1, 1), theta=10000.0, stream=None):
    """RMS norm of every head (weights given) and rotary positions of three axes: q [Hq, n, d]
    -> q_out, k [Hk, n, d] -> k_out (k and k_out None: q alone).  axes: the channels that turn
    with the frame, the row and the column; pos [n, 3] int32, or the grid's positions."""
    Hq, n, d = qs = _dims3("q", q)
    dt, dev = q.dtype, q.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    ks = (0 if k is None else k.shape[0], n, d)
    if not (
            dev >= 0 and dev == _device()
            and (q_st := q.stride())[2] == 1
            and q_out.dtype is dt and q_out.shape == qs and (qo_st := q_out.stride())[2] == 1
            and q_out.get_device() == dev
            and (k is None or k.dtype is dt and k.shape == ks and (k_st := k.stride())[2] == 1 and k.get_device() == dev
                 and k_out.dtype is dt and k_out.shape == ks and (ko_st := k_out.stride())[2] == 1
                 and k_out.get_device() == dev)
            and (wq is None or wq.dtype is _F32 and wq.shape == (d,) and wq.is_contiguous() and wq.get_device() == dev)
            and (wk is None or wk.dtype is _F32 and wk.shape == (d,) and wk.is_contiguous() and wk.get_device() == dev)
            and (pos is None or pos.dtype is _I32 and pos.shape == (n, 3) and pos.is_contiguous()
                 and pos.get_device() == dev)
            and (t0_dev is None or t0_dev.dtype is _I32 and t0_dev.shape == (1,) and t0_dev.get_device() == dev)):
        _refuse([("q", q, dt, qs), ("q_out", q_out, dt, qs), ("k", k, dt, ks), ("k_out", k_out, dt, ks)],
                [("wq", wq, _F32, (d,)), ("wk", wk, _F32, (d,)), ("pos", pos, _I32, (n, 3)),
                 ("t0_dev", t0_dev, _I32, (1,))])
    Hk = ks[0]
    if k is None:
        k_st = ko_st = (0, 0)
    rc = (_lib or load()).fastar_packed_call(_CALL_ROPE, _PACK_ROPE(
        code, n, d, Hq, q.data_ptr(), q_st[0] if Hq > 1 else n * d, q_st[1] if n > 1 else d,
        q_out.data_ptr(), qo_st[0] if Hq > 1 else n * d, qo_st[1] if n > 1 else d,
        Hk, 0 if k is None else k.data_ptr(), k_st[0] if Hk > 1 else n * d, k_st[1] if n > 1 else d,
        0 if k is None else k_out.data_ptr(), ko_st[0] if Hk > 1 else n * d, ko_st[1] if n > 1 else d,
        0 if wq is None else wq.data_ptr(), 0 if wk is None else wk.data_ptr(), eps, axes[0], axes[1], axes[2],
        0 if pos is None else pos.data_ptr(), t0, 0 if t0_dev is None else t0_dev.data_ptr(), grid[0], grid[1], theta,
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_ROPE)
    if rc:
        _raise("fastar_qk_norm_rope", rc)


def fastar_kv4_append(k, v, k_codes, k_scales, v_codes, v_scales, at=None, len_out=None, dev_status=None, k_exp=None,
                      v_exp=None, stream=None):
    """Rows k, v [H, n, d] into the 4-bit cache (codes [H, cap, d / 2], scales [H, cap, d / 16],
    uint8) from row at[h] on (int32 [H]; None: 0); len_out[h] = at[h] + n."""
    H, n, d = rs = _dims3("k", k)
    dt, dev = k.dtype, k.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    cap = _dims3("k_codes", k_codes)[1]
    cs, ss, hs = (H, cap, d // 2), (H, cap, d // 16), (H,)
    if not (
            dev >= 0 and dev == _device()
            and (k_st := k.stride())[2] == 1
            and v.dtype is dt and v.shape == rs and (v_st := v.stride())[2] == 1 and v.get_device() == dev
            and k_codes.dtype is _U8 and k_codes.shape == cs and k_codes.is_contiguous() and k_codes.get_device() == dev
            and k_scales.dtype is _U8 and k_scales.shape == ss and k_scales.is_contiguous()
            and k_scales.get_device() == dev
            and v_codes.dtype is _U8 and v_codes.shape == cs and v_codes.is_contiguous() and v_codes.get_device() == dev
            and v_scales.dtype is _U8 and v_scales.shape == ss and v_scales.is_contiguous()
            and v_scales.get_device() == dev
            and (at is None or at.dtype is _I32 and at.shape == hs and at.is_contiguous() and at.get_device() == dev)
            and (len_out is None or len_out.dtype is _I32 and len_out.shape == hs and len_out.is_contiguous()
                 and len_out.get_device() == dev)
            and (dev_status is None or dev_status.dtype is _I32 and dev_status.shape == (1,)
                 and dev_status.get_device() == dev)
            and (k_exp is None or k_exp.dtype is _I32 and k_exp.shape == hs and k_exp.is_contiguous()
                 and k_exp.get_device() == dev)
            and (v_exp is None or v_exp.dtype is _I32 and v_exp.shape == hs and v_exp.is_contiguous()
                 and v_exp.get_device() == dev)):
        _refuse([("k", k, dt, rs), ("v", v, dt, rs)],
                [("k_codes", k_codes, _U8, cs), ("k_scales", k_scales, _U8, ss), ("v_codes", v_codes, _U8, cs),
                 ("v_scales", v_scales, _U8, ss), ("at", at, _I32, hs), ("len_out", len_out, _I32, hs),
                 ("dev_status", dev_status, _I32, (1,)), ("k_exp", k_exp, _I32, hs), ("v_exp", v_exp, _I32, hs)])
    rc = (_lib or load()).fastar_packed_call(_CALL_APPEND, _PACK_APPEND(
        code, H, n, d, k.data_ptr(), k_st[0] if H > 1 else n * d, k_st[1] if n > 1 else d,
        v.data_ptr(), v_st[0] if H > 1 else n * d, v_st[1] if n > 1 else d,
        0 if k_exp is None else k_exp.data_ptr(), 0 if v_exp is None else v_exp.data_ptr(),
        0 if at is None else at.data_ptr(), k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
        v_scales.data_ptr(), cap, 0 if len_out is None else len_out.data_ptr(),
        0 if dev_status is None else dev_status.data_ptr(),
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_APPEND)
    if rc:
        _raise("fastar_kv4_append", rc)


def fastar_kv4_read(codes, scales, first, out, exps=None, stream=None):
    """The values of rows first .. first + n of a 4-bit cache -> out [H, n, d]."""
    H, n, d = rs = _dims3("out", out)
    dt, dev = out.dtype, out.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    cap = _dims3("codes", codes)[1]
    cs, ss = (H, cap, d // 2), (H, cap, d // 16)
    if not (
            dev >= 0 and dev == _device()
            and (o_st := out.stride())[2] == 1
            and codes.dtype is _U8 and codes.shape == cs and codes.is_contiguous() and codes.get_device() == dev
            and scales.dtype is _U8 and scales.shape == ss and scales.is_contiguous() and scales.get_device() == dev
            and (exps is None or exps.dtype is _I32 and exps.shape == (H,) and exps.is_contiguous()
                 and exps.get_device() == dev)):
        _refuse([("out", out, dt, rs)],
                [("codes", codes, _U8, cs), ("scales", scales, _U8, ss), ("exps", exps, _I32, (H,))])
    rc = (_lib or load()).fastar_packed_call(_CALL_READ, _PACK_READ(
        code, H, n, d, codes.data_ptr(), scales.data_ptr(), 0 if exps is None else exps.data_ptr(), cap, first,
        out.data_ptr(), o_st[0] if H > 1 else n * d, o_st[1] if n > 1 else d,
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_READ)
    if rc:
        _raise("fastar_kv4_read", rc)


def fastar_kv4_attn(q, k_codes, k_scales, v_codes, v_scales, lens, scale, out, lse=None, block=0, k_exp=None,
                    v_exp=None, dev_status=None, workspace=None, stream=None):
    """Attention of q [Hq, nq, d] over the first lens[h] rows of a 4-bit cache of Hkv heads
    (Hq a multiple of Hkv); block > 0: the tokens are the cache's last nq rows and see no block
    of that many tokens later than their own.  workspace: workspace_bytes(OP_KV4_ATTN, Hq, nq,
    cap, d, Hkv) bytes (None: the keys are not split)."""
    Hq, nq, d = rs = _dims3("q", q)
    dt, dev = q.dtype, q.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    Hkv, cap, _ = _dims3("k_codes", k_codes)
    cs, ss, hs = (Hkv, cap, d // 2), (Hkv, cap, d // 16), (Hkv,)
    if not (
            dev >= 0 and dev == _device()
            and (q_st := q.stride())[2] == 1
            and out.dtype is dt and out.shape == rs and (o_st := out.stride())[2] == 1 and out.get_device() == dev
            and k_codes.dtype is _U8 and k_codes.is_contiguous() and k_codes.shape == cs and k_codes.get_device() == dev
            and k_scales.dtype is _U8 and k_scales.shape == ss and k_scales.is_contiguous()
            and k_scales.get_device() == dev
            and v_codes.dtype is _U8 and v_codes.shape == cs and v_codes.is_contiguous() and v_codes.get_device() == dev
            and v_scales.dtype is _U8 and v_scales.shape == ss and v_scales.is_contiguous()
            and v_scales.get_device() == dev
            and lens.dtype is _I32 and lens.shape == hs and lens.is_contiguous() and lens.get_device() == dev
            and (lse is None or lse.dtype is _F32 and lse.shape == (Hq, nq) and lse.is_contiguous()
                 and lse.get_device() == dev)
            and (dev_status is None or dev_status.dtype is _I32 and dev_status.shape == (1,)
                 and dev_status.get_device() == dev)
            and (k_exp is None or k_exp.dtype is _I32 and k_exp.shape == hs and k_exp.is_contiguous()
                 and k_exp.get_device() == dev)
            and (v_exp is None or v_exp.dtype is _I32 and v_exp.shape == hs and v_exp.is_contiguous()
                 and v_exp.get_device() == dev)
            and (workspace is None or workspace.is_contiguous() and workspace.get_device() == dev)):
        dense = [("k_codes", k_codes, _U8, cs), ("k_scales", k_scales, _U8, ss), ("v_codes", v_codes, _U8, cs),
                 ("v_scales", v_scales, _U8, ss), ("lens", lens, _I32, hs), ("lse", lse, _F32, (Hq, nq)),
                 ("dev_status", dev_status, _I32, (1,)), ("k_exp", k_exp, _I32, hs), ("v_exp", v_exp, _I32, hs)]
        if workspace is not None:
            dense.append(("workspace", workspace, workspace.dtype, workspace.shape))
        _refuse([("q", q, dt, rs), ("out", out, dt, rs)], dense)
    rc = (_lib or load()).fastar_packed_call(_CALL_ATTN, _PACK_ATTN(
        q.data_ptr(), code, Hq, Hkv, nq, d, q_st[0] if Hq > 1 else nq * d, q_st[1] if nq > 1 else d,
        k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
        0 if k_exp is None else k_exp.data_ptr(), 0 if v_exp is None else v_exp.data_ptr(), cap, lens.data_ptr(), block,
        scale, out.data_ptr(), o_st[0] if Hq > 1 else nq * d, o_st[1] if nq > 1 else d,
        0 if lse is None else lse.data_ptr(), 0 if dev_status is None else dev_status.data_ptr(),
        0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_ATTN)
    if rc:
        _raise("fastar_kv4_attn", rc)


def _refuse_paged(rows, dense, k_pool, v_pool, dt, Hk, d, table, at, cu):
    """As _refuse, for the calls over a paged cache (which take a vector in any shape of its size)."""
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t.dtype is not dt:
            raise ValueError(f"{name} must be {dt}, not {t.dtype}")
        if t.dim() != 4 or t.shape[1] != Hk or t.shape[3] != d:
            raise ValueError(f"{name} must have the shape [pages, {Hk}, page, {d}], not {tuple(t.shape)}")
        if t.stride(3) != 1:
            raise ValueError(f"{name} must have a contiguous last dimension")
    if k_pool.shape != v_pool.shape or k_pool.stride() != v_pool.stride():
        raise ValueError("k_pool and v_pool must share shape and strides")
    if table.dim() != 2:
        raise ValueError(f"table must have two dimensions, not {table.dim()}")
    B = table.shape[0]
    _refuse(rows, [("table", table, _I32, table.shape), ("at", at, _I32, (B,)), ("cu", cu, _I32, (B + 1,))] + dense)


def fastar_paged_append(k, v, k_pool, v_pool, table, at, len_out=None, q=None, q_out=None, cu=None, wq=None, wk=None,
                        eps=1e-6, axes=(0, 0, 0), pos=None, grid=(1, 1), theta=10000.0, dev_status=None, stream=None):
    """Rows k, v [Hk, T, d] of the sequences' tokens into the pages of k_pool, v_pool [pages, Hk, page, d]
    (any strides, the same for both) that table [B, max_pages] (int32) names, behind at[b] earlier rows
    (int32 [B]); cu [B + 1] (int32): where each sequence's tokens begin (None: T / B tokens each).  k is
    normed (wk given) and turned by its row's position on the grid, or pos [T, 3]; q [Hq, T, d] likewise into
    q_out.  len_out[b] = at[b] + its tokens."""
    ks = k.shape
    Hk, T, d = ks if len(ks) == 3 else _dims3("k", k)
    dt, dev = k.dtype, k.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    Hq = 0 if q is None else _dims3("q", q)[0]
    qs = (Hq, T, d)
    p_sh, p_st, t_sh = k_pool.shape, k_pool.stride(), table.shape
    B = t_sh[0] if len(t_sh) == 2 else -1
    if not (
            dev >= 0 and dev == _device()
            and (k_st := k.stride())[2] == 1
            and v.dtype is dt and v.shape == ks and (v_st := v.stride())[2] == 1 and v.get_device() == dev
            and len(p_sh) == 4 and p_sh[1] == Hk and p_sh[3] == d and p_st[3] == 1 and k_pool.dtype is dt
            and k_pool.get_device() == dev
            and v_pool.dtype is dt and v_pool.shape == p_sh and v_pool.stride() == p_st and v_pool.get_device() == dev
            and table.dtype is _I32 and B >= 0 and table.is_contiguous() and table.get_device() == dev
            and at.dtype is _I32 and at.numel() == B and at.is_contiguous() and at.get_device() == dev
            and (q is None or q.dtype is dt and q.shape == qs and (q_st := q.stride())[2] == 1 and q.get_device() == dev
                 and q_out.dtype is dt and q_out.shape == qs and (qo_st := q_out.stride())[2] == 1
                 and q_out.get_device() == dev)
            and (cu is None or cu.dtype is _I32 and cu.numel() == B + 1 and cu.is_contiguous() and cu.get_device() == dev)
            and (len_out is None or len_out.dtype is _I32 and len_out.numel() == B and len_out.is_contiguous()
                 and len_out.get_device() == dev)
            and (wq is None or wq.dtype is _F32 and wq.numel() == d and wq.is_contiguous() and wq.get_device() == dev)
            and (wk is None or wk.dtype is _F32 and wk.numel() == d and wk.is_contiguous() and wk.get_device() == dev)
            and (pos is None or pos.dtype is _I32 and pos.shape == (T, 3) and pos.is_contiguous()
                 and pos.get_device() == dev)
            and (dev_status is None or dev_status.dtype is _I32 and dev_status.numel() == 1
                 and dev_status.get_device() == dev)):
        _refuse_paged([("k", k, dt, ks), ("v", v, dt, ks), ("q", q, dt, qs), ("q_out", q_out, dt, qs)],
                      [("len_out", len_out, _I32, table.shape[:1]), ("wq", wq, _F32, (d,)), ("wk", wk, _F32, (d,)),
                       ("pos", pos, _I32, (T, 3)), ("dev_status", dev_status, _I32, (1,))],
                      k_pool, v_pool, dt, Hk, d, table, at, cu)
    if q is None:
        q_st = qo_st = (0, 0)
    rc = (_lib or load()).fastar_packed_call(_CALL_PAPPEND, _PACK_PAPPEND(
        code, B, T, 0 if cu is None else cu.data_ptr(), d, Hq, 0 if q is None else q.data_ptr(),
        q_st[0] if Hq > 1 else T * d, q_st[1] if T > 1 else d, 0 if q is None else q_out.data_ptr(),
        qo_st[0] if Hq > 1 else T * d, qo_st[1] if T > 1 else d, Hk, k.data_ptr(), k_st[0] if Hk > 1 else T * d,
        k_st[1] if T > 1 else d, v.data_ptr(), v_st[0] if Hk > 1 else T * d, v_st[1] if T > 1 else d,
        0 if wq is None else wq.data_ptr(), 0 if wk is None else wk.data_ptr(), eps, axes[0], axes[1], axes[2],
        0 if pos is None else pos.data_ptr(), grid[0], grid[1], theta, k_pool.data_ptr(), v_pool.data_ptr(), p_sh[0],
        p_sh[2], p_st[0] if p_sh[0] > 1 else d, p_st[1] if Hk > 1 else d, p_st[2], table.data_ptr(), t_sh[1],
        at.data_ptr(), 0 if len_out is None else len_out.data_ptr(), 0 if dev_status is None else dev_status.data_ptr(),
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_PAPPEND)
    if rc:
        _raise("fastar_paged_append", rc)


def fastar_paged_attn(q, k_pool, v_pool, table, at, scale, out, lse=None, cu=None, max_q=None, block=0, window=0,
                      sinks=0, dev_status=None, workspace=None, stream=None):
    """Attention of the sequences' tokens q [Hq, T, d] over the pages of k_pool, v_pool [pages, Hkv, page, d]
    that table [B, max_pages] names, the tokens' own rows (behind at[b] earlier ones) among them.  block: 0,
    or the tokens of a block that sees no later one (1: causal); window > 0: only the last `window` rows before
    the token's end, and the first `sinks`.  cu [B + 1] as in fastar_paged_append; max_q: the most tokens
    of a sequence (None: T, with cu None T / B).  It picks the kernel: give it with cu, since single tokens of many
    sequences are several times slower as sequences of T tokens.  workspace: workspace_bytes(OP_PAGED_ATTN, Hq, T,
    max_pages * page, d, Hkv, r=max_q, P=B) bytes (None: the keys are not split)."""
    qs = q.shape
    Hq, T, d = qs if len(qs) == 3 else _dims3("q", q)
    dt, dev = q.dtype, q.get_device()
    code = _CODES[dt] if dt in _CODES else _raise_dtype(dt)
    p_sh, p_st, t_sh = k_pool.shape, k_pool.stride(), table.shape
    B = t_sh[0] if len(t_sh) == 2 else -1
    if not (
            dev >= 0 and dev == _device()
            and (q_st := q.stride())[2] == 1
            and out.dtype is dt and out.shape == qs and (o_st := out.stride())[2] == 1 and out.get_device() == dev
            and len(p_sh) == 4 and p_sh[3] == d and p_st[3] == 1 and k_pool.dtype is dt and k_pool.get_device() == dev
            and v_pool.dtype is dt and v_pool.shape == p_sh and v_pool.stride() == p_st and v_pool.get_device() == dev
            and table.dtype is _I32 and B >= 0 and table.is_contiguous() and table.get_device() == dev
            and at.dtype is _I32 and at.numel() == B and at.is_contiguous() and at.get_device() == dev
            and (cu is None or cu.dtype is _I32 and cu.numel() == B + 1 and cu.is_contiguous() and cu.get_device() == dev)
            and (lse is None or lse.dtype is _F32 and lse.shape == (Hq, T) and lse.is_contiguous()
                 and lse.get_device() == dev)
            and (dev_status is None or dev_status.dtype is _I32 and dev_status.numel() == 1
                 and dev_status.get_device() == dev)
            and (workspace is None or workspace.is_contiguous() and workspace.get_device() == dev)):
        dense = [("lse", lse, _F32, (Hq, T)), ("dev_status", dev_status, _I32, (1,))]
        if workspace is not None:
            dense.append(("workspace", workspace, workspace.dtype, workspace.shape))
        _refuse_paged([("q", q, dt, qs), ("out", out, dt, qs)], dense, k_pool, v_pool, dt,
                      k_pool.shape[1] if k_pool.dim() == 4 else 0, d, table, at, cu)
    if max_q is None:
        max_q = T if cu is not None else T // max(B, 1)
    rc = (_lib or load()).fastar_packed_call(_CALL_PATTN, _PACK_PATTN(
        q.data_ptr(), code, B, T, 0 if cu is None else cu.data_ptr(), max_q, Hq, p_sh[1], d,
        q_st[0] if Hq > 1 else T * d, q_st[1] if T > 1 else d, k_pool.data_ptr(), v_pool.data_ptr(), p_sh[0], p_sh[2],
        p_st[0] if p_sh[0] > 1 else d, p_st[1] if p_sh[1] > 1 else d, p_st[2], table.data_ptr(), t_sh[1],
        at.data_ptr(), block, window, sinks, scale, out.data_ptr(), o_st[0] if Hq > 1 else T * d,
        o_st[1] if T > 1 else d, 0 if lse is None else lse.data_ptr(), 0 if dev_status is None else dev_status.data_ptr(),
        0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        _current_stream(dev) if stream is None else stream.cuda_stream), _N_PATTN)
    if rc:
        _raise("fastar_paged_attn", rc)


def fastar_dense_append(k_cur, v_cur, k_cache, v_cache, at, stream=None):
    H, nq, d = k_cur.shape
    hs, ts = tok_strides(k_cur)
    _call("fastar_dense_append", dtype_code(k_cur.dtype), H, nq, d, ptr(k_cur), ptr(v_cur), hs, ts, ptr(k_cache),
          ptr(v_cache), k_cache.shape[1], int(at), stream_handle(stream))
