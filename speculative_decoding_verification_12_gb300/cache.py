"""The cache side of a verify step: spec_append, spec_attention and the page bookkeeping calls.

The same thin binding as the package's verify calls, over include/spec_cache.h: checks of the
tensors, then one call into libspecverify.so.  Caches are torch tensors [pages, slots, heads,
head_dim] of any strides whose last is 1, so a [pages, heads, slots, head_dim] cache is passed
as its transpose(1, 2).
"""
from __future__ import annotations

import ctypes as C

import torch

from . import SV_BF16, SV_OK, SvError, lib

SV_F16 = 2
_DTYPES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16}
_I32 = torch.int32


class SvKvCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64), ("num_pages", C.c_int32), ("page_size", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32), ("dtype", C.c_int), ("max_pages", C.c_int32),
                ("block_table", C.c_void_p)]


_calls = None


def _lib():
    global _calls
    if _calls is None:
        l = lib()
        P, I, L, F, Z = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
        for name, args in (
                ("spec_append", [P, P, P, L, L, L, I, P, P, F, P, I, I, F, P, P, P, I, I, I, SvKvCache, P, L, P, P]),
                ("spec_attention", [P, L, I, P, P, P, I, I, I, SvKvCache, F, I, I, P, P, P, Z, P]),
                ("spec_page_reserve", [P, P, I, P, I, P, I, I, P, Z, P]),
                ("spec_page_fork", [P, P, P, I, P, I, P, I, P, I, I, P, P, P, Z, P]),
                ("spec_page_release", [P, I, P, I, P, I, I, I, I, P, P]),
                ("spec_page_compact", [I, P, I, P, I, P, P, I, P, Z, P]),
                ("spec_page_copy", [P, P, L, L, I, L, I, P, P, I, P, P])):
            f = getattr(l, name)
            f.restype, f.argtypes = C.c_int, args
        l.sv_attention_workspace_bytes.restype = Z
        l.sv_attention_workspace_bytes.argtypes = [I]
        l.sv_page_workspace_bytes.restype = Z
        l.sv_page_workspace_bytes.argtypes = [I, I]
        _calls = l
    return _calls


def sv_attention_workspace_bytes(head_dim: int) -> int:
    return int(_lib().sv_attention_workspace_bytes(head_dim))


def sv_page_workspace_bytes(B: int, num_pages: int) -> int:
    return int(_lib().sv_page_workspace_bytes(B, num_pages))


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _fail(name, what):
    raise ValueError(f"{name} must be {what}")


def _p(t, name, dtype=None, numel=None):
    """Pointer of a contiguous CUDA tensor (None: NULL), checked."""
    if t is None:
        return None
    if not t.is_cuda:
        _fail(name, "a CUDA tensor")
    if not t.is_contiguous():
        _fail(name, "contiguous")
    if dtype is not None and t.dtype != dtype:
        _fail(name, f"{dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        _fail(name, f"{numel} elements, got {t.numel()}")
    return t.data_ptr()


def _rows(t, name, dtype, R, heads, D):
    """Pointer and row stride of a [rows, heads, D] tensor whose rows are contiguous inside."""
    if not t.is_cuda:
        _fail(name, "a CUDA tensor")
    if t.dtype != dtype:
        _fail(name, f"{dtype}, got {t.dtype}")
    if t.shape != (R, heads, D):
        _fail(name, f"[{R}, {heads}, {D}], got {list(t.shape)}")
    s = t.stride()
    if (s[2] != 1 and D != 1) or (s[1] != D and heads != 1):
        _fail(name, "contiguous within a row")
    return t.data_ptr(), (s[0] if R > 1 else max(s[0], heads * D))


def _cache(k, v, table, B):
    if not (k.is_cuda and v.is_cuda and table.is_cuda):
        _fail("k_cache, v_cache and block_table", "CUDA tensors")
    if k.dtype not in _DTYPES or v.dtype != k.dtype:
        _fail("k_cache and v_cache", "both bfloat16 or both float16")
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
        _fail("k_cache and v_cache", "[pages, slots, heads, head_dim], of one shape and strides")
    if table.dtype != _I32 or table.dim() != 2 or table.shape[0] != B or not table.is_contiguous():
        _fail("block_table", f"contiguous int32 [{B}, max_pages]")
    s, n = k.stride(), k.shape
    if s[3] != 1:
        _fail("k_cache and v_cache", "contiguous in head_dim")
    return SvKvCache(k.data_ptr(), v.data_ptr(), s[0], s[1], s[2], n[0], n[1], n[2], n[3], _DTYPES[k.dtype],
                     table.shape[1], table.data_ptr())


def _done(st, name):
    if st != SV_OK:
        raise SvError(st, name)


def spec_append(q, k, v, q_weight, k_weight, eps: float, inv_freq, k_cache, v_cache, block_table, kv_seq_len,
                num_drafts, row_offsets, k_max: int, out_q, workspace, interleaved: bool = False,
                rope_scale: float = 1.0, stream=None) -> None:
    """Norm and rotation of the new tokens' queries (to out_q) and keys, and the append of keys and
    values to the cache (see include/spec_cache.h).

    q, out_q [R, Hq, D], k, v [R, Hk, D]: rows of any stride; q_weight, k_weight [D] or None (no
    norm); inv_freq fp32 [rotary_dim / 2] or None (no rotation); k_cache, v_cache [pages,
    page_size, Hk, D]; block_table [B, max_pages], kv_seq_len (the new tokens counted),
    num_drafts [B], row_offsets [B+1] or None: int32; workspace: 256 bytes at least, zeroed once.
    """
    B = num_drafts.numel()
    cache = _cache(k_cache, v_cache, block_table, B)
    dt, D, Hk = k_cache.dtype, cache.head_dim, cache.num_heads
    R, Hq = q.shape[0], q.shape[1]
    pq, sq = _rows(q, "q", dt, R, Hq, D)
    pk, sk = _rows(k, "k", dt, R, Hk, D)
    pv, sv = _rows(v, "v", dt, R, Hk, D)
    po, so = _rows(out_q, "out_q", dt, R, Hq, D)
    if workspace.numel() * workspace.element_size() < 256:
        _fail("workspace", "256 bytes at least")
    _done(_lib().spec_append(pq, pk, pv, sq, sk, sv, Hq, _p(q_weight, "q_weight", dt, D),
                             _p(k_weight, "k_weight", dt, D), eps, _p(inv_freq, "inv_freq", torch.float32),
                             0 if inv_freq is None else 2 * inv_freq.numel(), 1 if interleaved else 0, rope_scale,
                             _p(num_drafts, "num_drafts", _I32), _p(row_offsets, "row_offsets", _I32, B + 1),
                             _p(kv_seq_len, "kv_seq_len", _I32, B), B, k_max, R, cache, po, so,
                             _p(workspace, "workspace"), _stream(stream)), "spec_append")


def spec_attention(q, k_cache, v_cache, block_table, kv_seq_len, num_drafts, row_offsets, k_max: int, scale: float,
                   window: int, sinks: int, out, out_lse, workspace, stream=None) -> None:
    """The new tokens' rows attend over the paged cache: causal, the last `window` tokens (0: all)
    and the first `sinks` (see include/spec_cache.h).

    q [R, Hq, D], rows of any stride; out [R, Hq, D]; out_lse fp32 [R, Hq] or None; workspace of
    sv_attention_workspace_bytes(D) bytes, its first 256 zeroed once; the rest as spec_append.
    """
    B = num_drafts.numel()
    cache = _cache(k_cache, v_cache, block_table, B)
    dt, D = k_cache.dtype, cache.head_dim
    R, Hq = q.shape[0], q.shape[1]
    pq, sq = _rows(q, "q", dt, R, Hq, D)
    _done(_lib().spec_attention(pq, sq, Hq, _p(num_drafts, "num_drafts", _I32),
                                _p(row_offsets, "row_offsets", _I32, B + 1), _p(kv_seq_len, "kv_seq_len", _I32, B),
                                B, k_max, R, cache, scale, window, sinks, _p(out, "out", dt, R * Hq * D),
                                _p(out_lse, "out_lse", torch.float32, R * Hq), _p(workspace, "workspace"),
                                workspace.numel() * workspace.element_size(), _stream(stream)), "spec_attention")


def _pages(kv_seq_len, block_table, ref_count):
    if block_table.dim() != 2:
        _fail("block_table", "[B, max_pages]")
    B, M = block_table.shape
    return (_p(kv_seq_len, "kv_seq_len", _I32, B), B, _p(block_table, "block_table", _I32), M,
            _p(ref_count, "ref_count", _I32), ref_count.numel())


def spec_page_reserve(num_drafts, kv_seq_len, block_table, ref_count, page_size: int, workspace,
                      stream=None) -> None:
    """kv_seq_len[b] += num_drafts[b] + 1 (-1 drafts: an idle request), with pages to hold them."""
    ln, B, tab, M, ref, N = _pages(kv_seq_len, block_table, ref_count)
    _done(_lib().spec_page_reserve(_p(num_drafts, "num_drafts", _I32, B), ln, B, tab, M, ref, N, page_size,
                                   _p(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "spec_page_reserve")


def spec_page_fork(parents, children, fork_len, kv_seq_len, block_table, ref_count, page_size: int, copy_src,
                   copy_dst, workspace, stream=None) -> None:
    """Empty requests children[f] continue from the first fork_len[f] tokens of parents[f] (None:
    from all), sharing full pages; (copy_src[f], copy_dst[f]) is the page to copy, or -1s."""
    ln, B, tab, M, ref, N = _pages(kv_seq_len, block_table, ref_count)
    F = parents.numel()
    _done(_lib().spec_page_fork(_p(parents, "parents", _I32), _p(children, "children", _I32, F),
                                _p(fork_len, "fork_len", _I32, F), F, ln, B, tab, M, ref, N, page_size,
                                _p(copy_src, "copy_src", _I32, F), _p(copy_dst, "copy_dst", _I32, F),
                                _p(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "spec_page_fork")


def spec_page_release(kv_seq_len, block_table, ref_count, page_size: int, window: int, sinks: int, workspace,
                      stream=None) -> None:
    """Gives back the pages past each length and, with a window, those that no later row sees."""
    ln, B, tab, M, ref, N = _pages(kv_seq_len, block_table, ref_count)
    _done(_lib().spec_page_release(ln, B, tab, M, ref, N, page_size, window, sinks, _p(workspace, "workspace"),
                                   _stream(stream)), "spec_page_release")


def spec_page_compact(block_table, ref_count, copy_src, copy_dst, workspace, stream=None) -> None:
    """Moves used pages down into free ones below the number of pages in use; copy_src, copy_dst
    [capacity] receive the pairs to copy, then -1s."""
    _, B, tab, M, ref, N = _pages(None, block_table, ref_count)
    cap = copy_src.numel()
    _done(_lib().spec_page_compact(B, tab, M, ref, N, _p(copy_src, "copy_src", _I32),
                                   _p(copy_dst, "copy_dst", _I32, cap), cap, _p(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
          "spec_page_compact")


def spec_page_copy(k_cache, v_cache, copy_src, copy_dst, workspace, stream=None) -> None:
    """Copies the pages of the pairs in caches [pages, ...] or [layers, pages, ., ., .] (v_cache
    may be None); a page's elements have to be contiguous, in any order of its dimensions."""
    layered = k_cache.dim() == 5
    s, n = k_cache.stride(), k_cache.shape
    if not k_cache.is_cuda or k_cache.dim() not in (2, 3, 4, 5):
        _fail("k_cache", "a CUDA tensor [pages, ...] or [layers, pages, slots, heads, head_dim]")
    if v_cache is not None and (v_cache.shape != n or v_cache.stride() != s or v_cache.dtype != k_cache.dtype
                                or not v_cache.is_cuda):
        _fail("v_cache", "like k_cache")
    first, size, want = (2 if layered else 1), k_cache.element_size(), 1
    for st, m in sorted((s[i], n[i]) for i in range(first, len(n)) if n[i] != 1):
        if st != want:
            _fail("k_cache", "contiguous within a page")
        want *= m
    pairs = copy_src.numel()
    _done(_lib().spec_page_copy(k_cache.data_ptr(), None if v_cache is None else v_cache.data_ptr(), want * size,
                                s[first - 1] * size, n[0] if layered else 1, s[0] * size if layered else 0,
                                n[first - 1], _p(copy_src, "copy_src", _I32), _p(copy_dst, "copy_dst", _I32, pairs),
                                pairs, _p(workspace, "workspace"), _stream(stream)), "spec_page_copy")
