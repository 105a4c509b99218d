"""Bindings of include/gdn_pages.h: pages of the key-value cache that sequences share -- forks, releases, compaction -- and
the copies of pages that these ask for.  Argument marshalling only, as in the package's __init__."""
from __future__ import annotations

import ctypes

from . import library
from ._attn import _I32, GdnAttnDims, GdnKvCache, KvCache, _cache, _done, _opt, _p, _stream

__all__ = ["gdn_kv_fork", "gdn_kv_release", "gdn_kv_compact", "gdn_kv_copy_pages", "EXPORTED_SYMBOLS_PAGES"]

EXPORTED_SYMBOLS_PAGES = ("gdn_kv_fork", "gdn_kv_release", "gdn_kv_compact", "gdn_kv_copy_pages")

_fns = None


def _fn(name: str):
    """The C entry point (its signature set on first use)."""
    global _fns
    if _fns is None:
        lib = library()
        P, I32 = ctypes.c_void_p, ctypes.c_int32
        sig = {
            "gdn_kv_fork": [I32] * 5 + [P] * 12,
            "gdn_kv_release": [I32] * 4 + [P] * 11,
            "gdn_kv_compact": [I32] * 3 + [P] * 7 + [I32] + [P] * 5,
            "gdn_kv_copy_pages": [ctypes.POINTER(GdnAttnDims), ctypes.POINTER(GdnKvCache), I32, P, P, P, P],
        }
        for n, args in sig.items():
            f = getattr(lib, n)
            f.restype, f.argtypes = ctypes.c_int, args
        _fns = {n: getattr(lib, n) for n in sig}
    return _fns[name]


def gdn_kv_fork(page_size: int, src, dst, length, seq_len, n_pages, block_table, page_refs, free_list, free_count, copy_src,
                copy_dst, dev_status=None, stream=None) -> None:
    """The empty sequence dst[i] gets the first length[i] tokens of sequence src[i]: full pages shared, a last one that is
    not full from the free stack with a pair copy_src[i] -> copy_dst[i] (-1: none).  seq_len, n_pages, block_table,
    page_refs and free_count are updated in place."""
    B, P = block_table.shape
    N, M, nb = free_list.shape[0], src.shape[0], (B,)
    _done("gdn_kv_fork", _fn("gdn_kv_fork")(
        page_size, N, B, P, M, _p(src, _I32, (M,)), _p(dst, _I32, (M,)), _p(length, _I32, (M,)), _p(seq_len, _I32, nb),
        _p(n_pages, _I32, nb), _p(block_table, _I32, (B, P)), _p(page_refs, _I32, (N,)), _p(free_list, _I32, (N,)),
        _p(free_count, _I32, (1,)), _p(copy_src, _I32, (M,)), _p(copy_dst, _I32, (M,)), _opt(dev_status, _I32, (M,)),
        _stream(stream)))


def gdn_kv_release(page_size: int, new_len, seq_len, n_pages, block_table, page_refs, free_list, free_count, copy_src,
                   copy_dst, dev_status=None, stream=None) -> None:
    """Shorten every sequence to new_len[b] tokens (0: finished) where pages may be shared: those that nobody holds any
    more go back to the free stack; a kept page that is not full but shared is replaced by one from the stack, with a
    pair copy_src[b] -> copy_dst[b] (-1: none).  All the books are updated in place."""
    B, P = block_table.shape
    N, nb = free_list.shape[0], (B,)
    _done("gdn_kv_release", _fn("gdn_kv_release")(
        page_size, N, B, P, _p(new_len, _I32, nb), _p(seq_len, _I32, nb), _p(n_pages, _I32, nb),
        _p(block_table, _I32, (B, P)), _p(page_refs, _I32, (N,)), _p(free_list, _I32, (N,)), _p(free_count, _I32, (1,)),
        _p(copy_src, _I32, nb), _p(copy_dst, _I32, nb), _opt(dev_status, _I32, nb), _stream(stream)))


def gdn_kv_compact(n_pages, block_table, page_refs, free_list, free_count, page_map, copy_src, copy_dst, n_copy,
                   block_table_out=None, dev_status=None, stream=None) -> None:
    """Move the pages that sequences hold to the lowest indices: the tables in place unless block_table_out is given,
    page_refs, the free stack and page_map formed anew, the n_copy[0] moves in copy_src and copy_dst (then -1; at least
    half as many entries as the cache has pages)."""
    B, P = block_table.shape
    N, C, one = free_list.shape[0], copy_src.shape[0], (1,)
    t = _p(block_table, _I32, (B, P))
    _done("gdn_kv_compact", _fn("gdn_kv_compact")(
        N, B, P, _p(n_pages, _I32, (B,)), t, t if block_table_out is None else _p(block_table_out, _I32, (B, P)),
        _p(page_refs, _I32, (N,)), _p(free_list, _I32, (N,)), _p(free_count, _I32, one), _p(page_map, _I32, (N,)), C,
        _p(copy_src, _I32, (C,)), _p(copy_dst, _I32, (C,)), _p(n_copy, _I32, one), _opt(dev_status, _I32, (B,)),
        _stream(stream)))


def gdn_kv_copy_pages(dims: GdnAttnDims, cache: KvCache, copy_src, copy_dst, dev_status=None, stream=None) -> None:
    """Copy page copy_src[i] of a layer's cache to page copy_dst[i], keys and values; pairs of -1 are skipped."""
    n = copy_src.shape[0]
    _done("gdn_kv_copy_pages", _fn("gdn_kv_copy_pages")(
        dims, _cache(dims, cache), n, _p(copy_src, _I32, (n,)), _p(copy_dst, _I32, (n,)), _opt(dev_status, _I32, (1,)),
        _stream(stream)))
