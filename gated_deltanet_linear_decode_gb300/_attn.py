"""Bindings of include/gdn_attn.h and include/gdn_norm.h (include/gdn_pages.h is in _pages): the paged key-value cache of the
full-attention layers between the gated DeltaNet ones, the attention of new tokens over it, and the
norms around a block.  Argument marshalling only, as in the package's __init__."""
from __future__ import annotations

import ctypes
import math

import torch

from . import GDN_BF16, GDN_FLAG_TEST_STALL, GdnError, _dt, _need, gdn_status_string, library

__all__ = [
    "GdnAttnDims", "GdnKvCache", "GdnNormDims", "KvCache", "make_attn_dims", "make_norm_dims", "gdn_kv_extend",
    "gdn_kv_truncate", "gdn_kv_append", "gdn_attn_decode_workspace_bytes", "gdn_attn_decode",
    "gdn_attn_chunk_workspace_bytes", "gdn_attn_chunk", "gdn_norm_residual",
    "GDN_KV_REFUSED", "GDN_KV_BAD_INDEX", "EXPORTED_SYMBOLS_ATTN",
]

GDN_KV_REFUSED, GDN_KV_BAD_INDEX = 32, 64   # dev_status bits

EXPORTED_SYMBOLS_ATTN = ("gdn_kv_extend", "gdn_kv_truncate", "gdn_kv_append", "gdn_attn_decode_workspace_bytes",
                         "gdn_attn_decode", "gdn_attn_chunk_workspace_bytes", "gdn_attn_chunk", "gdn_norm_residual")

_I32 = torch.int32
_F32 = torch.float32


class GdnAttnDims(ctypes.Structure):
    _fields_ = [("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("act_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class GdnKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class GdnNormDims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
                ("act_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32)]


_fns = None


def _fn(name: str):
    """The C entry point (its signature set on first use)."""
    global _fns
    if _fns is None:
        lib = library()
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D, C, N = ctypes.POINTER(GdnAttnDims), ctypes.POINTER(GdnKvCache), ctypes.POINTER(GdnNormDims)
        sig = {
            "gdn_kv_extend": (ctypes.c_int, [I32] * 5 + [P] * 14),
            "gdn_kv_truncate": (ctypes.c_int, [I32] * 4 + [P] * 11),
            "gdn_kv_append": (ctypes.c_int, [D, C, I32, P, I64, P, I64, P, I64] + [P] * 6 + [I32, P, P, P]),
            "gdn_attn_decode_workspace_bytes": (SZ, [D, I32, I32]),
            "gdn_attn_decode": (ctypes.c_int, [D, C, I32, I32, I32, P, I64, P, I64, P, P, P, P, SZ, P, P]),
            "gdn_attn_chunk_workspace_bytes": (SZ, [D, I32, I32]),
            "gdn_attn_chunk": (ctypes.c_int, [D, C, I32, I32, I32, P, I64, P, I64, P, P, P, P, P, SZ, P, P]),
            "gdn_norm_residual": (ctypes.c_int, [N, I32, P, I64, P, I64, I32, P, P, P, P, P, P, P]),
        }
        for n, (res, args) in sig.items():
            f = getattr(lib, n)
            f.restype, f.argtypes = res, args
        _fns = {n: getattr(lib, n) for n in sig}
    return _fns[name]


def _done(fn: str, status: int) -> None:
    if status != 0:
        raise GdnError(fn, status, gdn_status_string(status))


# A decode step makes a handful of these calls a layer, each a few microseconds on the device, so the checks
# are kept to one expression a tensor; what fails it goes to _need for the message.
_BF16 = torch.bfloat16


def _p(t, dtype, shape):
    """The pointer of a dense tensor of this type and shape."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    _need(t, dtype, shape)
    raise ValueError("bad tensor")


def _opt(t, dtype, shape):
    return None if t is None else _p(t, dtype, shape)


def _rows(t, dtype, T: int, n: int):
    """Pointer and pitch of a [T][n] tensor whose rows are dense (a column slice of a wider one will do)."""
    if t is None:
        raise ValueError("missing tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.dtype is not dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    if t.shape != (T, n):
        raise ValueError(f"expected shape {(T, n)}, got {tuple(t.shape)}")
    ld, one = t.stride()
    if one != 1 and n > 1:
        raise ValueError("rows must be contiguous")
    return t.data_ptr(), ld if T > 1 else n   # one row's pitch is of no account


def _stream(stream):
    """The CUDA stream to launch on: the given one, or torch's current one (its handle alone; building the stream
    object costs 3 us)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _act(dims):
    return _BF16 if dims.act_dtype == GDN_BF16 else _F32


def make_attn_dims(Hq: int, Hkv: int, head_dim: int, act_dtype=torch.bfloat16, out_dtype=torch.float32,
                   rope_dim: int = 0, scale: float | None = None, eps: float = 1e-6,
                   test_stall: bool = False) -> GdnAttnDims:
    """Head counts, head size and types of a full-attention layer; scale defaults to 1/sqrt(head_dim);
    test_stall selects GDN_FLAG_TEST_STALL (the give-up path of the kernel's waits)."""
    return GdnAttnDims(Hq, Hkv, head_dim, rope_dim, 1.0 / math.sqrt(head_dim) if scale is None else scale, eps,
                       _dt(act_dtype), _dt(out_dtype), GDN_FLAG_TEST_STALL if test_stall else 0)


def make_norm_dims(H: int, act_dtype=torch.bfloat16, res_dtype=torch.bfloat16, alpha: float = 1.0,
                   eps: float = 1e-6) -> GdnNormDims:
    """Row width, types and residual scale of gdn_norm_residual."""
    return GdnNormDims(H, eps, alpha, _dt(act_dtype), _dt(res_dtype))


class KvCache:
    """A layer's paged cache: k and v as [page][token][head][channel] views with the same strides, the
    channels contiguous (either order of tokens and heads in memory, or both halves in one buffer)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t in (k, v):
            if not t.is_cuda:
                raise ValueError("tensors must live on a CUDA device")
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError("a cache half is [page][token][head][channel] with contiguous channels")
        if k.dtype != v.dtype or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must have the same type, shape and strides")
        _dt(k.dtype)
        self.k, self.v = k, v
        self.dtype, self.page_size, self.heads, self.head_dim = k.dtype, k.shape[1], k.shape[2], k.shape[3]
        self.struct = GdnKvCache(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[1], *k.stride()[:3])


def _cache(dims: GdnAttnDims, cache: KvCache):
    if cache.dtype != _act(dims):
        raise TypeError(f"expected a cache of {_act(dims)}, got {cache.dtype}")
    if cache.heads != dims.H_kv or cache.head_dim != dims.head_dim:
        raise ValueError(f"expected a cache of {dims.H_kv} heads of {dims.head_dim}, got {cache.heads} of {cache.head_dim}")
    return cache.struct


def gdn_kv_extend(page_size: int, n_new, seq_len, n_pages, block_table, free_list, free_count, slot_map, positions,
                  cu_seqlens, seq_len_out=None, n_pages_out=None, free_count_out=None, dev_status=None,
                  stream=None) -> None:
    """Room for n_new[b] more tokens in every sequence: pages from the free stack into block_table
    [B][max_pages], slot and position of every new token, cu_seqlens [B+1].  The lengths, held pages and
    free count are updated in place unless *_out are given."""
    B, P = block_table.shape
    T, N, nb = slot_map.shape[0], free_list.shape[0], (B,)
    sl, np_, fc = _p(seq_len, _I32, nb), _p(n_pages, _I32, nb), _p(free_count, _I32, (1,))
    _done("gdn_kv_extend", _fn("gdn_kv_extend")(
        page_size, N, B, P, T, _p(n_new, _I32, nb), sl, np_, _p(block_table, _I32, (B, P)), _p(free_list, _I32, (N,)),
        fc, sl if seq_len_out is None else _p(seq_len_out, _I32, nb),
        np_ if n_pages_out is None else _p(n_pages_out, _I32, nb),
        fc if free_count_out is None else _p(free_count_out, _I32, (1,)), _p(slot_map, _I32, (T,)),
        _p(positions, _I32, (T,)), _p(cu_seqlens, _I32, (B + 1,)), _opt(dev_status, _I32, nb), _stream(stream)))


def gdn_kv_truncate(page_size: int, new_len, seq_len, n_pages, block_table, free_list, free_count, seq_len_out=None,
                    n_pages_out=None, free_count_out=None, dev_status=None, stream=None) -> None:
    """Shorten every sequence to new_len[b] tokens (0: finished) and put the pages past them back on the
    free stack; in place unless *_out are given."""
    B, P = block_table.shape
    N, nb = free_list.shape[0], (B,)
    sl, np_, fc = _p(seq_len, _I32, nb), _p(n_pages, _I32, nb), _p(free_count, _I32, (1,))
    _done("gdn_kv_truncate", _fn("gdn_kv_truncate")(
        page_size, N, B, P, _p(new_len, _I32, nb), sl, np_, _p(block_table, _I32, (B, P)), _p(free_list, _I32, (N,)), fc,
        sl if seq_len_out is None else _p(seq_len_out, _I32, nb),
        np_ if n_pages_out is None else _p(n_pages_out, _I32, nb),
        fc if free_count_out is None else _p(free_count_out, _I32, (1,)), _opt(dev_status, _I32, nb), _stream(stream)))


def gdn_kv_append(dims: GdnAttnDims, cache: KvCache, q, k, v, positions, slot_map, q_out, q_norm_w=None,
                  k_norm_w=None, rope_cos=None, rope_sin=None, dev_status=None, stream=None) -> None:
    """Norm and rotate the q and k heads of T tokens (rows of a fused projection, column slices allowed),
    store k and v in the cache at slot_map, q in q_out."""
    T, D, a, r = positions.shape[0], dims.head_dim, _act(dims), dims.rope_dim
    nq, nk = dims.H_q * D, dims.H_kv * D
    c = _cache(dims, cache)
    (xq, ldq), (xk, ldk), (xv, ldv) = _rows(q, a, T, nq), _rows(k, a, T, nk), _rows(v, a, T, nk)
    cos = sin = None
    n_pos = 0
    if r:
        if rope_cos is None:
            raise ValueError("missing tensor")
        n_pos = rope_cos.shape[0]
        cos, sin = _p(rope_cos, _F32, (n_pos, r // 2)), _p(rope_sin, _F32, (n_pos, r // 2))
    _done("gdn_kv_append", _fn("gdn_kv_append")(
        dims, c, T, xq, ldq, xk, ldk, xv, ldv, _p(positions, _I32, (T,)), _p(slot_map, _I32, (T,)),
        _opt(q_norm_w, _F32, (D,)), _opt(k_norm_w, _F32, (D,)), cos, sin, n_pos, _p(q_out, a, (T, nq)),
        _opt(dev_status, _I32, (1,)), _stream(stream)))


def gdn_attn_decode_workspace_bytes(dims: GdnAttnDims, B: int, K: int) -> int:
    return int(_fn("gdn_attn_decode_workspace_bytes")(dims, B, K))


def gdn_attn_decode(dims: GdnAttnDims, cache: KvCache, K: int, q, block_table, seq_len, out, gate=None,
                    workspace=None, dev_status=None, stream=None) -> None:
    """Attention of the last K tokens of each of B sequences (rows b*K + p of q, gate and out) over the
    cache; workspace: gdn_attn_decode_workspace_bytes() bytes, zeroed once before its first use."""
    B, P = block_table.shape
    T, n, a = B * K, dims.H_q * dims.head_dim, _act(dims)
    c = _cache(dims, cache)
    xq, ldq = _rows(q, a, T, n)
    xg, ldg = (None, 0) if gate is None else _rows(gate, a, T, n)
    ws, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _done("gdn_attn_decode", _fn("gdn_attn_decode")(
        dims, c, B, K, P, xq, ldq, xg, ldg, _p(block_table, _I32, (B, P)), _p(seq_len, _I32, (B,)),
        _p(out, _BF16 if dims.out_dtype == GDN_BF16 else _F32, (T, n)), ws, ws_bytes, _opt(dev_status, _I32, (B,)),
        _stream(stream)))


def gdn_attn_chunk_workspace_bytes(dims: GdnAttnDims, B: int = 1, T: int = 1) -> int:
    return int(_fn("gdn_attn_chunk_workspace_bytes")(dims, B, T))


def gdn_attn_chunk(dims: GdnAttnDims, cache: KvCache, q, cu_seqlens, block_table, seq_len, out, gate=None,
                   workspace=None, dev_status=None, stream=None) -> None:
    """Attention of the last cu_seqlens[b+1] - cu_seqlens[b] tokens of each sequence (packed rows of q, gate and
    out, any number of them) over the cache; workspace: gdn_attn_chunk_workspace_bytes() bytes, zeroed once before
    its first use."""
    B, P = block_table.shape
    T, n, a = q.shape[0], dims.H_q * dims.head_dim, _act(dims)
    c = _cache(dims, cache)
    xq, ldq = _rows(q, a, T, n)
    xg, ldg = (None, 0) if gate is None else _rows(gate, a, T, n)
    ws, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _done("gdn_attn_chunk", _fn("gdn_attn_chunk")(
        dims, c, B, T, P, xq, ldq, xg, ldg, _p(cu_seqlens, _I32, (B + 1,)), _p(block_table, _I32, (B, P)),
        _p(seq_len, _I32, (B,)), _p(out, _BF16 if dims.out_dtype == GDN_BF16 else _F32, (T, n)), ws, ws_bytes,
        _opt(dev_status, _I32, (B,)), _stream(stream)))


def gdn_norm_residual(dims: GdnNormDims, h, h_out=None, y=None, gate=None, post_w=None, chan_scale=None, pre_w=None,
                      x=None, stream=None) -> None:
    """h_out = h + alpha * chan_scale * sigmoid(gate) * RMSNorm(y) post_w and x = RMSNorm(h_out) pre_w, every
    part but h optional; gate [T][1] or [T][H]; h_out may be h."""
    T, H, a = h.shape[0], dims.H, _act(dims)
    r, th, w = _BF16 if dims.res_dtype == GDN_BF16 else _F32, (T, H), (H,)
    xy, ldy = (None, 0) if y is None else _rows(y, a, T, H)
    cols = 0 if gate is None else gate.shape[1]
    xg, ldg = (None, 0) if gate is None else _rows(gate, a, T, cols)
    _done("gdn_norm_residual", _fn("gdn_norm_residual")(
        dims, T, xy, ldy, xg, ldg, cols, _p(h, r, th), _opt(post_w, _F32, w), _opt(chan_scale, _F32, w),
        _opt(pre_w, _F32, w), _opt(h_out, r, th), _opt(x, a, th), _stream(stream)))
