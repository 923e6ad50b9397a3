"""Thin Python binding of libmsa (include/msa.h) over ctypes.

Argument marshalling only: every function takes torch tensors that already live
on the GPU, checks dtype/contiguity/device, passes raw pointers and the current
HIP stream to the C entry point of the same name, and raises MsaError on a
non-OK status.  All computation happens in the library's HIP kernels.  bf16
tensors may be torch.bfloat16 or torch.int16/uint16 views of the bit patterns.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MSA_SANITIZED=1 loads the build whose host code carries AddressSanitizer and UBSan checks
LIB_PATH = os.path.join(_PKG, "libmsa_san.so" if os.environ.get("MSA_SANITIZED") == "1" else "libmsa.so")

MSA_OK, MSA_ERR_NULL, MSA_ERR_SHAPE, MSA_ERR_UNSUPPORTED, MSA_ERR_WORKSPACE, MSA_ERR_HIP = range(6)
HEADS, HEAD_DIM, BLOCK_TOKENS, TILE_BLOCKS, MAX_TOPK = 8, 128, 64, 16, 256
ROW4_BYTES = 544            # of a row of the paged local cache held in 4 bits


class MsaError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__("%s failed: status %d (%s): %s" % (fn, status, _status_string(status), message))
        self.status = status


_P, _I32, _I64, _F32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "msa_abi_version": ([], ctypes.c_int),
    "msa_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "msa_last_error": ([], ctypes.c_char_p),
    "msa_group_offsets_host": ([_P, _I64, _P, _P], ctypes.c_int),
    "msa_block_offsets_host": ([_P, _I32, _P, _P, _P], ctypes.c_int),
    "msa_route_tiles": ([_I64], _I64),
    "msa_pool_blocks": ([_I32, _P, _P, _P, _I64, _P, _P, _I32, _I64, _P, _P, _P, _P, _P], ctypes.c_int),
    "msa_pack_route_keys": ([_I32, _P, _I64, _P, _P, _P], ctypes.c_int),
    "msa_block_doc_map": ([_P, _I32, _I64, _P, _P], ctypes.c_int),
    "msa_route_scores": ([_I32, _P, _I32, _I32, _P, _P, _I64, _P, _I32, _I32, _P, _P], ctypes.c_int),
    "msa_topk_docs_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "msa_topk_docs": ([_I32, _I32, _P, _I32, _I32, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "msa_route_topk_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "msa_route_topk": ([_I32, _P, _I32, _I32, _P, _P, _I64, _P, _I32, _I32, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "msa_route_topk_noalloc_max_scratch": ([], _SZ),
    "msa_route_topk_noalloc": ([_I32, _P, _I32, _I32, _P, _P, _I64, _P, _I32, _I32, _P, _P, _P, _P], ctypes.c_int),
    "msa_gather_ctx": ([_I32, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _I64, _I32, _P, _P, _P, _P], ctypes.c_int),
    "msa_sparse_decode_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "msa_sparse_decode": ([_I32, _I32, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _I32, _F32, _P, _P, _SZ, _P],
                          ctypes.c_int),
    "msa_encode_blocks": ([_I32, _I32, _P, _I64, _P, _P, _P, _P, _F32, _F32, _P, _P, _I32, _I64, _P, _P, _P, _P, _P],
                          ctypes.c_int),
    "msa_sparse_prefill": ([_I32, _I32, _I32, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _I32, _F32, _P, _P],
                           ctypes.c_int),
    "msa_paged_append": ([_I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _F32, _F32, _P,
                          _P, _P, _P], ctypes.c_int),
    "msa_paged_attend_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "msa_paged_attend": ([_I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _P,
                          _P, _F32, _I32, _P, _P, _SZ, _P], ctypes.c_int),
    "msa_paged_append4": ([_I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _F32, _F32, _P,
                           _P, _P, _P], ctypes.c_int),
    "msa_paged_attend4_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "msa_paged_attend4": ([_I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _P,
                           _P, _F32, _I32, _P, _P, _SZ, _P], ctypes.c_int),
    "msa_paged_read4": ([_I32, _I32, _I32, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libmsa.so; raises if it has not been built (there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmsa.so is missing at %s: build it with __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _status_string(status: int) -> str:
    try:
        return lib().msa_status_string(status).decode()
    except Exception:  # pragma: no cover - only while reporting another error
        return "?"


def _check(fn: str, status: int):
    if status != MSA_OK:
        raise MsaError(fn, status, lib().msa_last_error().decode(errors="replace"))


def _ptr(t, dtypes, name, allow_none=False, allow_pinned=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if not t.is_cuda and not (allow_pinned and t.is_pinned()):
        raise ValueError("%s must be a GPU tensor%s" % (name, " or pinned host memory" if allow_pinned else ""))
    return ctypes.c_void_p(t.data_ptr())


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I64T = (torch.int64,)
_I32T = (torch.int32,)
_F32T = (torch.float32,)
_ANY = (torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.float32, torch.bfloat16)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ host helpers

def msa_abi_version() -> int:
    return lib().msa_abi_version()


def msa_group_offsets_host(doc_ids):
    """CPU int64 per-token doc ids -> CPU int64 doc_tok_off [n_docs + 1]."""
    ids = torch.as_tensor(doc_ids, dtype=torch.int64).contiguous()
    out = torch.empty(ids.numel() + 1, dtype=torch.int64)
    n = ctypes.c_int32(0)
    _check("msa_group_offsets_host",
           lib().msa_group_offsets_host(ctypes.c_void_p(ids.data_ptr()), ids.numel(),
                                        ctypes.c_void_p(out.data_ptr()), ctypes.byref(n)))
    return out[: n.value + 1].clone()


def msa_block_offsets_host(doc_tok_off):
    """CPU int64 doc_tok_off -> (CPU int64 doc_blk_off, n_blk, max_doc_blocks)."""
    tok = torch.as_tensor(doc_tok_off, dtype=torch.int64).contiguous()
    n_docs = tok.numel() - 1
    out = torch.empty(n_docs + 1, dtype=torch.int64)
    n_blk, mx = ctypes.c_int64(0), ctypes.c_int32(0)
    _check("msa_block_offsets_host",
           lib().msa_block_offsets_host(ctypes.c_void_p(tok.data_ptr()), n_docs, ctypes.c_void_p(out.data_ptr()),
                                        ctypes.byref(n_blk), ctypes.byref(mx)))
    return out, int(n_blk.value), int(mx.value)


def msa_route_tiles(n_blk: int) -> int:
    return int(lib().msa_route_tiles(n_blk))


# ----------------------------------------------------------------------- entry points

def msa_pool_blocks(k, v, kr, doc_tok_off, doc_blk_off, n_blk, kbar, vbar, krbar_route, krbar_norm=None,
                    stream=None):
    L, n_tok = k.shape[0], k.shape[1]
    n_docs = doc_tok_off.numel() - 1
    _check("msa_pool_blocks", lib().msa_pool_blocks(
        L, _ptr(k, _BF16, "k"), _ptr(v, _BF16, "v"), _ptr(kr, _BF16, "kr"), n_tok,
        _ptr(doc_tok_off, _I64T, "doc_tok_off"), _ptr(doc_blk_off, _I64T, "doc_blk_off"), n_docs, n_blk,
        _ptr(kbar, _BF16, "kbar"), _ptr(vbar, _BF16, "vbar"), _ptr(krbar_route, _BF16, "krbar_route"),
        _ptr(krbar_norm, _F32T, "krbar_norm", allow_none=True), _stream(stream)))


def msa_pack_route_keys(krbar_rows, n_blk, krbar_route, krbar_norm=None, stream=None):
    L = krbar_rows.shape[0]
    _check("msa_pack_route_keys", lib().msa_pack_route_keys(
        L, _ptr(krbar_rows, _BF16, "krbar_rows"), n_blk, _ptr(krbar_route, _BF16, "krbar_route"),
        _ptr(krbar_norm, _F32T, "krbar_norm", allow_none=True), _stream(stream)))


def msa_block_doc_map(doc_blk_off, n_blk, blk_doc, stream=None):
    n_docs = doc_blk_off.numel() - 1
    _check("msa_block_doc_map", lib().msa_block_doc_map(
        _ptr(doc_blk_off, _I64T, "doc_blk_off"), n_docs, n_blk, _ptr(blk_doc, _I32T, "blk_doc"), _stream(stream)))


def _norms(krbar_norm, n_layers, n_blk):
    """The optional key norms of the scan: None, or at least [n_layers][tiles][8][16] fp32."""
    if krbar_norm is None:
        return None
    need = n_layers * msa_route_tiles(n_blk) * 128
    if krbar_norm.numel() < need:
        raise ValueError("krbar_norm has %d elements, the scan needs %d" % (krbar_norm.numel(), need))
    return _ptr(krbar_norm, _F32T, "krbar_norm")


def msa_route_scores(qr, krbar_route, n_blk, blk_doc, n_docs, doc_scores, accumulate=False, stream=None,
                     krbar_norm=None):
    L, B, T = qr.shape[0], qr.shape[1], qr.shape[2]
    _check("msa_route_scores", lib().msa_route_scores(
        L, _ptr(qr, _BF16, "qr"), B, T, _ptr(krbar_route, _BF16, "krbar_route"),
        _norms(krbar_norm, L, n_blk), n_blk, _ptr(blk_doc, _I32T, "blk_doc"), n_docs,
        1 if accumulate else 0, _ptr(doc_scores, _F32T, "doc_scores"), _stream(stream)))


def msa_topk_docs_workspace_size(n_layers, B, n_docs, k) -> int:
    return int(lib().msa_topk_docs_workspace_size(n_layers, B, n_docs, k))


def msa_topk_docs(doc_scores, k, topk_ids, topk_scores, workspace, stream=None):
    L, B, n_docs = doc_scores.shape
    _check("msa_topk_docs", lib().msa_topk_docs(
        L, B, _ptr(doc_scores, _F32T, "doc_scores"), n_docs, k, _ptr(topk_ids, _I32T, "topk_ids"),
        _ptr(topk_scores, _F32T, "topk_scores", allow_none=True), _ptr(workspace, _ANY, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_route_topk_workspace_size(n_layers, B, n_docs, k) -> int:
    return int(lib().msa_route_topk_workspace_size(n_layers, B, n_docs, k))


def msa_route_topk(qr, krbar_route, n_blk, blk_doc, n_docs, k, topk_ids, topk_scores, workspace, doc_scores=None,
                   stream=None, krbar_norm=None):
    L, B, T = qr.shape[0], qr.shape[1], qr.shape[2]
    _check("msa_route_topk", lib().msa_route_topk(
        L, _ptr(qr, _BF16, "qr"), B, T, _ptr(krbar_route, _BF16, "krbar_route"),
        _norms(krbar_norm, L, n_blk), n_blk, _ptr(blk_doc, _I32T, "blk_doc"), n_docs, k,
        _ptr(topk_ids, _I32T, "topk_ids"), _ptr(topk_scores, _F32T, "topk_scores", allow_none=True),
        _ptr(doc_scores, _F32T, "doc_scores", allow_none=True), _ptr(workspace, _ANY, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_route_topk_noalloc_max_scratch() -> int:
    return int(lib().msa_route_topk_noalloc_max_scratch())


def msa_route_topk_noalloc(qr, krbar_route, n_blk, blk_doc, n_docs, k, topk_ids, topk_scores, doc_scores=None,
                           stream=None, krbar_norm=None):
    """msa_route_topk without a workspace: the library's fixed per-GPU scratch is used."""
    L, B, T = qr.shape[0], qr.shape[1], qr.shape[2]
    _check("msa_route_topk_noalloc", lib().msa_route_topk_noalloc(
        L, _ptr(qr, _BF16, "qr"), B, T, _ptr(krbar_route, _BF16, "krbar_route"),
        _norms(krbar_norm, L, n_blk), n_blk, _ptr(blk_doc, _I32T, "blk_doc"), n_docs, k,
        _ptr(topk_ids, _I32T, "topk_ids"), _ptr(topk_scores, _F32T, "topk_scores", allow_none=True),
        _ptr(doc_scores, _F32T, "doc_scores", allow_none=True), _stream(stream)))


def msa_gather_ctx(topk_ids, doc_blk_off, max_doc_blocks, kbar, vbar, ctx_k, ctx_v, ctx_len, stream=None):
    """kbar/vbar may live in HBM or in pinned host memory (read over the host link)."""
    L, B, k = topk_ids.shape
    n_docs = doc_blk_off.numel() - 1
    n_blk = kbar.shape[1]
    max_ctx = ctx_k.shape[2]
    _check("msa_gather_ctx", lib().msa_gather_ctx(
        L, B, _ptr(topk_ids, _I32T, "topk_ids"), k, _ptr(doc_blk_off, _I64T, "doc_blk_off"), n_docs,
        max_doc_blocks, _ptr(kbar, _BF16, "kbar", allow_pinned=True), _ptr(vbar, _BF16, "vbar", allow_pinned=True),
        n_blk, max_ctx,
        _ptr(ctx_k, _BF16, "ctx_k"), _ptr(ctx_v, _BF16, "ctx_v"), _ptr(ctx_len, _I32T, "ctx_len"),
        _stream(stream)))


def msa_sparse_decode_workspace_size(n_layers, B, Hq, max_ctx, max_loc) -> int:
    return int(lib().msa_sparse_decode_workspace_size(n_layers, B, Hq, max_ctx, max_loc))


def msa_sparse_decode(q, ctx_k, ctx_v, ctx_len, loc_k, loc_v, loc_len, scale, out, workspace, stream=None):
    L, B, Hq = q.shape[0], q.shape[1], q.shape[2]
    max_ctx = ctx_k.shape[2]
    max_loc = 0 if loc_k is None else loc_k.shape[2]
    _check("msa_sparse_decode", lib().msa_sparse_decode(
        L, B, Hq, _ptr(q, _BF16, "q"), _ptr(ctx_k, _BF16, "ctx_k"), _ptr(ctx_v, _BF16, "ctx_v"),
        _ptr(ctx_len, _I32T, "ctx_len"), max_ctx,
        _ptr(loc_k, _BF16, "loc_k", allow_none=True), _ptr(loc_v, _BF16, "loc_v", allow_none=True),
        _ptr(loc_len, _I32T, "loc_len", allow_none=True), max_loc, float(scale),
        _ptr(out, _F32T, "out"), _ptr(workspace, _ANY, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def msa_sparse_prefill(q, ctx_k, ctx_v, ctx_len, loc_k, loc_v, loc_len, scale, out, stream=None):
    """q [L][B][T][Hq][128] bf16; contexts as for msa_sparse_decode; out [L][B][T][Hq][128] fp32."""
    L, B, T, Hq = q.shape[0], q.shape[1], q.shape[2], q.shape[3]
    _check("msa_sparse_prefill", lib().msa_sparse_prefill(
        L, B, T, Hq, _ptr(q, _BF16, "q"), _ptr(ctx_k, _BF16, "ctx_k"), _ptr(ctx_v, _BF16, "ctx_v"),
        _ptr(ctx_len, _I32T, "ctx_len"), ctx_k.shape[2], _ptr(loc_k, _BF16, "loc_k"), _ptr(loc_v, _BF16, "loc_v"),
        _ptr(loc_len, _I32T, "loc_len"), loc_k.shape[2], float(scale), _ptr(out, _F32T, "out"), _stream(stream)))


def msa_encode_blocks(x, w_k, w_v, w_kr, w_norm, eps, theta, doc_tok_off, doc_blk_off, n_blk, kbar, vbar,
                      krbar_route, krbar_norm=None, stream=None):
    """x [L][n_tok][H]; W_* [L][1024][H] (output-major); w_norm [L][128]; outputs as msa_pool_blocks."""
    L, n_tok, H = x.shape
    n_docs = doc_tok_off.numel() - 1
    _check("msa_encode_blocks", lib().msa_encode_blocks(
        L, H, _ptr(x, _BF16, "x"), n_tok, _ptr(w_k, _BF16, "w_k"), _ptr(w_v, _BF16, "w_v"),
        _ptr(w_kr, _BF16, "w_kr"), _ptr(w_norm, _BF16, "w_norm"), float(eps), float(theta),
        _ptr(doc_tok_off, _I64T, "doc_tok_off"), _ptr(doc_blk_off, _I64T, "doc_blk_off"), n_docs, n_blk,
        _ptr(kbar, _BF16, "kbar"), _ptr(vbar, _BF16, "vbar"), _ptr(krbar_route, _BF16, "krbar_route"),
        _ptr(krbar_norm, _F32T, "krbar_norm", allow_none=True), _stream(stream)))


# ------------------------------------------------------------------ paged local cache

_F32_BF16 = (torch.float32,) + _BF16


# A decode step makes these calls with a dozen tensors around kernels of a few microseconds: each tensor is
# looked at once, and neither a stream object nor a device guard is made where the device is the current one.

def _dims(t, n, name):
    """The sizes of a required n-dimensional tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != n:
        raise ValueError("%s has %d dimensions, expected %d" % (name, t.dim(), n))
    return t.shape


def _on(dev, t, dtypes, shape, name, have=None):
    """Address of a contiguous tensor of this shape (None: any; `have`: its shape, where it is known) on GPU
    `dev` (the kernels take the sizes from other arguments); None for none."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if ((shape is None or (have or t.shape) == shape) and t.dtype in dtypes and t.is_contiguous()
                and t.get_device() == dev and dev >= 0):
            return t.data_ptr()
    _refuse(dev, t, dtypes, shape, name)


def _refuse(dev, t, dtypes, shape, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    raise ValueError("%s is on cuda:%d, the other tensors on cuda:%d" % (name, t.get_device(), dev))


def _required(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError("%s is required" % name)


def _call(fn, dev, stream, args):
    """The entry point on the tensors' device, on `stream` or that device's current one."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index != dev:
        raise ValueError("stream on %s, tensors on cuda:%d" % (stream.device, dev))
    else:
        s = stream.cuda_stream
    f = getattr(lib(), fn)
    if torch.cuda.current_device() == dev:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != MSA_OK:
        _check(fn, status)


def msa_paged_append(k_new, v_new, q, q_off, kv_len, page_table, k_pages, v_pages, q_out, eps, theta, pos_off=None,
                     w_k=None, w_q=None, stream=None):
    """k_new, v_new [L][n_q][8][128], q and q_out [L][n_q][Hq][128] (q may be None, q_out may be q);
    q_off [B+1], kv_len [B] (new tokens included), page_table [B][max_pages], pos_off [B] int32;
    k_pages, v_pages [L][n_pages][page_tokens][8][128]; w_k, w_q [L][128] or None (no norm)."""
    k_shape = _dims(k_new, 4, "k_new")
    L, n_q = k_shape[0], k_shape[1]
    p_shape = _dims(k_pages, 5, "k_pages")
    n_pages, page_tokens = p_shape[1], p_shape[2]
    B, max_pages = _dims(page_table, 2, "page_table")
    _required(v_new=v_new, q_off=q_off, kv_len=kv_len, v_pages=v_pages)
    if q is None:
        Hq, q_out, w_q, q_shape = 0, None, None, None
    else:
        q_shape = _dims(q, 4, "q")
        Hq = q_shape[2]
        _required(q_out=q_out)
    dev = k_new.get_device()
    new, pages, heads = (L, n_q, HEADS, HEAD_DIM), (L, n_pages, page_tokens, HEADS, HEAD_DIM), (L, n_q, Hq, HEAD_DIM)
    _call("msa_paged_append", dev, stream, (
        L, B, n_q, Hq, _on(dev, k_new, _BF16, new, "k_new", k_shape), _on(dev, v_new, _BF16, new, "v_new"),
        _on(dev, q, _BF16, heads, "q", q_shape), _on(dev, q_off, _I32T, (B + 1,), "q_off"),
        _on(dev, kv_len, _I32T, (B,), "kv_len"), _on(dev, pos_off, _I32T, (B,), "pos_off"),
        _on(dev, page_table, _I32T, None, "page_table"), max_pages, page_tokens, n_pages,
        _on(dev, w_k, _BF16, (L, HEAD_DIM), "w_k"), _on(dev, w_q, _BF16, (L, HEAD_DIM), "w_q"), float(eps),
        float(theta), _on(dev, k_pages, _BF16, pages, "k_pages", p_shape), _on(dev, v_pages, _BF16, pages, "v_pages"),
        _on(dev, q_out, _BF16, heads, "q_out")))


def msa_paged_attend_workspace_size(n_layers, B, n_groups, n_q, Hq) -> int:
    return int(lib().msa_paged_attend_workspace_size(n_layers, B, n_groups, n_q, Hq))


def msa_paged_attend(q, q_off, kv_len, page_table, k_pages, v_pages, scale, out, workspace, grp_off=None, ctx_k=None,
                     ctx_v=None, ctx_len=None, pre_len=None, stream=None):
    """q [L][n_q][Hq][128]; the cache as for msa_paged_append; grp_off [n_groups+1], ascending from 0 to
    B, n_groups <= B (None: every sequence its own group), ctx_k, ctx_v [L][n_groups][max_ctx][8][128]
    and ctx_len [L][n_groups] (None: no memory context), pre_len [n_groups] or None; out
    [L][n_q][Hq][128], fp32 or bf16."""
    q_shape = _dims(q, 4, "q")
    L, n_q, Hq = q_shape[0], q_shape[1], q_shape[2]
    p_shape = _dims(k_pages, 5, "k_pages")
    n_pages, page_tokens = p_shape[1], p_shape[2]
    B, max_pages = _dims(page_table, 2, "page_table")
    o_shape = _dims(out, 4, "out")
    _required(q_off=q_off, kv_len=kv_len, v_pages=v_pages, workspace=workspace)
    n_groups = B if grp_off is None else _dims(grp_off, 1, "grp_off")[0] - 1
    if ctx_k is None:
        max_ctx, ctx_v, ctx_len = 0, None, None
    else:
        max_ctx = _dims(ctx_k, 5, "ctx_k")[2]
        _required(ctx_v=ctx_v, ctx_len=ctx_len)
    dev = q.get_device()
    heads, pages = (L, n_q, Hq, HEAD_DIM), (L, n_pages, page_tokens, HEADS, HEAD_DIM)
    ctx = (L, n_groups, max_ctx, HEADS, HEAD_DIM)
    _call("msa_paged_attend", dev, stream, (
        L, B, n_groups, n_q, Hq, _on(dev, q, _BF16, heads, "q", q_shape), _on(dev, q_off, _I32T, (B + 1,), "q_off"),
        _on(dev, grp_off, _I32T, None, "grp_off"), _on(dev, ctx_k, _BF16, ctx, "ctx_k"),
        _on(dev, ctx_v, _BF16, ctx, "ctx_v"), _on(dev, ctx_len, _I32T, (L, n_groups), "ctx_len"), max_ctx,
        _on(dev, k_pages, _BF16, pages, "k_pages", p_shape), _on(dev, v_pages, _BF16, pages, "v_pages"), n_pages,
        page_tokens,
        _on(dev, page_table, _I32T, None, "page_table"), max_pages, _on(dev, kv_len, _I32T, (B,), "kv_len"),
        _on(dev, pre_len, _I32T, (n_groups,), "pre_len"), float(scale), 0 if out.dtype == torch.float32 else 1,
        _on(dev, out, _F32_BF16, heads, "out", o_shape), _on(dev, workspace, _ANY, None, "workspace"),
        workspace.numel() * workspace.element_size()))


# ------------------------------------------------------------------ paged local cache held in 4 bits

_U8 = (torch.uint8,)


def _pages4(k_pages):
    """Shape, pages and tokens a page of [L][n_pages][page_tokens * 544]."""
    p_shape = _dims(k_pages, 3, "k_pages")
    if p_shape[2] % ROW4_BYTES:
        raise ValueError("k_pages has pages of %d bytes, expected a multiple of %d" % (p_shape[2], ROW4_BYTES))
    return p_shape, p_shape[1], p_shape[2] // ROW4_BYTES


def msa_paged_append4(k_new, v_new, q, q_off, kv_len, page_table, k_pages, v_pages, q_out, eps, theta, pos_off=None,
                      w_k=None, w_q=None, stream=None):
    """msa_paged_append into pages in 4 bits: k_pages, v_pages [L][n_pages][page_tokens * ROW4_BYTES] uint8;
    theta 0 for no rotation; the other arguments as there."""
    k_shape = _dims(k_new, 4, "k_new")
    L, n_q = k_shape[0], k_shape[1]
    p_shape, n_pages, page_tokens = _pages4(k_pages)
    B, max_pages = _dims(page_table, 2, "page_table")
    _required(v_new=v_new, q_off=q_off, kv_len=kv_len, v_pages=v_pages)
    if q is None:
        Hq, q_out, w_q, q_shape = 0, None, None, None
    else:
        q_shape = _dims(q, 4, "q")
        Hq = q_shape[2]
        _required(q_out=q_out)
    dev = k_new.get_device()
    new, pages, heads = (L, n_q, HEADS, HEAD_DIM), (L, n_pages, p_shape[2]), (L, n_q, Hq, HEAD_DIM)
    _call("msa_paged_append4", dev, stream, (
        L, B, n_q, Hq, _on(dev, k_new, _BF16, new, "k_new", k_shape), _on(dev, v_new, _BF16, new, "v_new"),
        _on(dev, q, _BF16, heads, "q", q_shape), _on(dev, q_off, _I32T, (B + 1,), "q_off"),
        _on(dev, kv_len, _I32T, (B,), "kv_len"), _on(dev, pos_off, _I32T, (B,), "pos_off"),
        _on(dev, page_table, _I32T, None, "page_table"), max_pages, page_tokens, n_pages,
        _on(dev, w_k, _BF16, (L, HEAD_DIM), "w_k"), _on(dev, w_q, _BF16, (L, HEAD_DIM), "w_q"), float(eps),
        float(theta), _on(dev, k_pages, _U8, pages, "k_pages", p_shape), _on(dev, v_pages, _U8, pages, "v_pages"),
        _on(dev, q_out, _BF16, heads, "q_out")))


def msa_paged_read4(k_pages, v_pages, row_off, page_table, k_out, v_out, row0=None, stream=None):
    """k_pages, v_pages as for msa_paged_append4; row_off [B+1], page_table [B][max_pages], row0 [B] int32 (None:
    from row 0 on); k_out, v_out [L][n_rows][8][128] bf16."""
    p_shape, n_pages, page_tokens = _pages4(k_pages)
    B, max_pages = _dims(page_table, 2, "page_table")
    o_shape = _dims(k_out, 4, "k_out")
    _required(v_pages=v_pages, row_off=row_off, v_out=v_out)
    L, n_rows = p_shape[0], o_shape[1]
    dev = k_pages.get_device()
    rows = (L, n_rows, HEADS, HEAD_DIM)
    _call("msa_paged_read4", dev, stream, (
        L, B, n_rows, _on(dev, row_off, _I32T, (B + 1,), "row_off"), _on(dev, row0, _I32T, (B,), "row0"),
        _on(dev, page_table, _I32T, None, "page_table"), max_pages, page_tokens, n_pages,
        _on(dev, k_pages, _U8, None, "k_pages"), _on(dev, v_pages, _U8, p_shape, "v_pages"),
        _on(dev, k_out, _BF16, rows, "k_out", o_shape), _on(dev, v_out, _BF16, rows, "v_out")))


def msa_paged_attend4_workspace_size(n_layers, B, n_groups, n_q, Hq) -> int:
    return int(lib().msa_paged_attend4_workspace_size(n_layers, B, n_groups, n_q, Hq))


def msa_paged_attend4(q, q_off, kv_len, page_table, k_pages, v_pages, scale, out, workspace, grp_off=None, ctx_k=None,
                      ctx_v=None, ctx_len=None, pre_len=None, stream=None):
    """msa_paged_attend over pages in 4 bits (k_pages, v_pages as for msa_paged_append4); the other arguments as
    there."""
    q_shape = _dims(q, 4, "q")
    L, n_q, Hq = q_shape[0], q_shape[1], q_shape[2]
    p_shape, n_pages, page_tokens = _pages4(k_pages)
    B, max_pages = _dims(page_table, 2, "page_table")
    o_shape = _dims(out, 4, "out")
    _required(q_off=q_off, kv_len=kv_len, v_pages=v_pages, workspace=workspace)
    n_groups = B if grp_off is None else _dims(grp_off, 1, "grp_off")[0] - 1
    if ctx_k is None:
        max_ctx, ctx_v, ctx_len = 0, None, None
    else:
        max_ctx = _dims(ctx_k, 5, "ctx_k")[2]
        _required(ctx_v=ctx_v, ctx_len=ctx_len)
    dev = q.get_device()
    heads, pages, ctx = (L, n_q, Hq, HEAD_DIM), (L, n_pages, p_shape[2]), (L, n_groups, max_ctx, HEADS, HEAD_DIM)
    _call("msa_paged_attend4", dev, stream, (
        L, B, n_groups, n_q, Hq, _on(dev, q, _BF16, heads, "q", q_shape), _on(dev, q_off, _I32T, (B + 1,), "q_off"),
        _on(dev, grp_off, _I32T, None, "grp_off"), _on(dev, ctx_k, _BF16, ctx, "ctx_k"),
        _on(dev, ctx_v, _BF16, ctx, "ctx_v"), _on(dev, ctx_len, _I32T, (L, n_groups), "ctx_len"), max_ctx,
        _on(dev, k_pages, _U8, pages, "k_pages", p_shape), _on(dev, v_pages, _U8, pages, "v_pages"), n_pages, page_tokens,
        _on(dev, page_table, _I32T, None, "page_table"), max_pages, _on(dev, kv_len, _I32T, (B,), "kv_len"),
        _on(dev, pre_len, _I32T, (n_groups,), "pre_len"), float(scale), 0 if out.dtype == torch.float32 else 1,
        _on(dev, out, _F32_BF16, heads, "out", o_shape), _on(dev, workspace, _ANY, None, "workspace"),
        workspace.numel() * workspace.element_size()))
