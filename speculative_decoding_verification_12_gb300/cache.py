"""The cache side of a verify step: spec_append, spec_attention, their forms for a cache in 8 bits, the page
bookkeeping calls, and spec_logits.

The same thin binding as the package's verify calls, over include/spec_cache.h and include/spec_logits.h: checks of the
tensors, then one call into libspecverify.so.  The checks are compiled (csrc/binding.cpp), since
several of these kernels run for less time than Python needs to look at a dozen tensors.  Caches
are torch tensors [pages, slots, heads, head_dim] of any strides whose last is 1, so a [pages,
heads, slots, head_dim] cache is passed as its transpose(1, 2).
"""
from __future__ import annotations

import ctypes as C

import torch

from . import SV_OK, SvError, lib

SV_F16 = 2


class SvKvCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64), ("num_pages", C.c_int32), ("page_size", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32), ("dtype", C.c_int), ("max_pages", C.c_int32),
                ("block_table", C.c_void_p)]


class SvKvCache8(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("page_stride", C.c_int64), ("token_stride", C.c_int64), ("head_stride", C.c_int64),
                ("scale_page_stride", C.c_int64), ("scale_block_stride", C.c_int64), ("scale_head_stride", C.c_int64),
                ("num_pages", C.c_int32), ("page_size", C.c_int32), ("scale_tokens", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32), ("max_pages", C.c_int32),
                ("block_table", C.c_void_p)]


class SvLogitRules(C.Structure):
    _fields_ = [("repetition", C.c_void_p), ("presence", C.c_void_p), ("frequency", C.c_void_p),
                ("prior_offsets", C.c_void_p), ("prior_tokens", C.c_void_p), ("prior_counts", C.c_void_p),
                ("prior_len", C.c_int32), ("bias_len", C.c_int32), ("bias_offsets", C.c_void_p),
                ("bias_tokens", C.c_void_p), ("bias_values", C.c_void_p), ("masks", C.c_void_p),
                ("mask_rows", C.c_void_p), ("num_masks", C.c_int32), ("mask_words", C.c_int32)]


_calls = None


def _lib():
    global _calls
    if _calls is None:
        l = lib()
        P, I, L, F, Z = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
        for name, args in (
                ("spec_append", [P, P, P, L, L, L, I, P, P, F, P, I, I, F, P, P, P, I, I, I, SvKvCache, P, L, P, P]),
                ("spec_attention", [P, L, I, P, P, P, I, I, I, SvKvCache, F, I, I, P, P, P, Z, P]),
                ("spec_append8", [P, P, P, I, L, L, L, I, P, P, F, P, I, I, F, P, P, P, I, I, I, SvKvCache8, P, L, P, P]),
                ("spec_attention8", [P, I, L, I, P, P, P, I, I, I, SvKvCache8, F, I, I, P, P, P, Z, P]),
                ("spec_logits", [P, I, P, P, P, I, I, I, I, SvLogitRules, P, P, P]),
                ("spec_page_reserve", [P, P, I, P, I, P, I, I, P, Z, P]),
                ("spec_cache_rollback", [P, P, P, I, P, P]),
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


# the entry points that the compiled binding calls, in its order
ENTRIES = ("spec_append", "spec_attention", "spec_page_reserve", "spec_page_fork", "spec_page_release",
           "spec_page_compact", "spec_page_copy", "spec_rollback", "spec_cache_rollback", "spec_append8",
           "spec_attention8", "spec_logits")
_native = None


def _load():
    """The compiled binding, handed the loaded library's entry points."""
    global _native
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("the compiled binding is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')") from e
    l = _lib()
    _binding.init(*(C.cast(getattr(l, name), C.c_void_p).value for name in ENTRIES), torch._C._cuda_getCurrentRawStream)
    _native = _binding
    return _binding


def binding():
    """The compiled binding, or None where it was not built."""
    try:
        return _native or _load()
    except RuntimeError:
        return None


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
    st = (_native or _load()).append(q, k, v, q_weight, k_weight, eps, inv_freq, k_cache, v_cache, block_table,
                                     kv_seq_len, num_drafts, row_offsets, k_max, out_q, workspace, interleaved,
                                     rope_scale, stream)
    if st != SV_OK:
        raise SvError(st, "spec_append")


def spec_attention(q, k_cache, v_cache, block_table, kv_seq_len, num_drafts, row_offsets, k_max: int, scale: float,
                   window: int, sinks: int, out, out_lse, workspace, stream=None) -> None:
    """The new tokens' rows attend over the paged cache: causal, the last `window` tokens (0: all)
    and the first `sinks` (see include/spec_cache.h).

    q [R, Hq, D], rows of any stride; out [R, Hq, D]; out_lse fp32 [R, Hq] or None; workspace of
    sv_attention_workspace_bytes(D) bytes, its first 256 zeroed once; the rest as spec_append.
    """
    st = (_native or _load()).attention(q, k_cache, v_cache, block_table, kv_seq_len, num_drafts, row_offsets, k_max,
                                        scale, window, sinks, out, out_lse, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_attention")


def spec_append8(q, k, v, q_weight, k_weight, eps: float, inv_freq, k_cache, v_cache, k_scale, v_scale, block_table,
                 kv_seq_len, num_drafts, row_offsets, k_max: int, out_q, workspace, interleaved: bool = False,
                 rope_scale: float = 1.0, stream=None) -> None:
    """spec_append to a cache in 8 bits: k_cache, v_cache float8_e4m3fn [pages, page_size, Hk, D],
    k_scale, v_scale fp32 [pages, blocks, Hk], a scale for each page_size / blocks tokens of a head (see
    include/spec_cache.h); the rest as spec_append, with q, k, v bfloat16 or float16.
    """
    st = (_native or _load()).append8(q, k, v, q_weight, k_weight, eps, inv_freq, k_cache, v_cache, k_scale, v_scale,
                                      block_table, kv_seq_len, num_drafts, row_offsets, k_max, out_q, workspace,
                                      interleaved, rope_scale, stream)
    if st != SV_OK:
        raise SvError(st, "spec_append8")


def spec_attention8(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_seq_len, num_drafts, row_offsets, k_max: int,
                    scale: float, window: int, sinks: int, out, out_lse, workspace, stream=None) -> None:
    """spec_attention over a cache in 8 bits, as spec_append8 fills it (see include/spec_cache.h)."""
    st = (_native or _load()).attention8(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_seq_len, num_drafts,
                                         row_offsets, k_max, scale, window, sinks, out, out_lse, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_attention8")


def spec_logits(logits, draft_tokens, num_drafts, row_offsets, k_max: int, repetition, presence, frequency, prior, bias,
                mask, mask_rows, out, workspace, stream=None) -> None:
    """Penalties for repeated tokens, biases and grammar masks on a verify step's logits (see
    include/spec_logits.h).

    logits, out [R, V] bf16 or fp32 (out may be logits); draft_tokens [R-B], num_drafts [B], row_offsets
    [B+1] or None: int32, as in spec_verify; repetition, presence, frequency fp32 [B] or None; prior None or
    (offsets [B+1], tokens [H], counts [H]) int32; bias None or (offsets [B+1], tokens [N] int32, values
    [N] fp32); mask int32 [masks, words], a bit per token, and mask_rows int32 [R] (-1: none), or None
    both; workspace: 256 bytes at least, zeroed once.
    """
    st = (_native or _load()).logits(logits, draft_tokens, num_drafts, row_offsets, k_max, repetition, presence,
                                     frequency, *(prior or (None,) * 3), *(bias or (None,) * 3), mask, mask_rows, out,
                                     workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_logits")


def spec_page_reserve(num_drafts, kv_seq_len, block_table, ref_count, page_size: int, workspace,
                      stream=None) -> None:
    """kv_seq_len[b] += num_drafts[b] + 1 (-1 drafts: an idle request), with pages to hold them."""
    st = (_native or _load()).reserve(num_drafts, kv_seq_len, block_table, ref_count, page_size, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_page_reserve")


def spec_cache_rollback(kv_seq_len, accept_len, num_drafts, workspace, stream=None) -> None:
    """kv_seq_len[b] <- kv_seq_len[b] - num_drafts[b] + accept_len[b] (-1 drafts: an idle request, unchanged)."""
    st = (_native or _load()).commit(kv_seq_len, accept_len, num_drafts, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_cache_rollback")


def spec_page_fork(parents, children, fork_len, kv_seq_len, block_table, ref_count, page_size: int, copy_src,
                   copy_dst, workspace, stream=None) -> None:
    """Empty requests children[f] continue from the first fork_len[f] tokens of parents[f] (None:
    from all), sharing full pages; (copy_src[f], copy_dst[f]) is the page to copy, or -1s."""
    st = (_native or _load()).fork(parents, children, fork_len, kv_seq_len, block_table, ref_count, page_size,
                                   copy_src, copy_dst, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_page_fork")


def spec_page_release(kv_seq_len, block_table, ref_count, page_size: int, window: int, sinks: int, workspace,
                      stream=None) -> None:
    """Gives back the pages past each length and, with a window, those that no later row sees."""
    st = (_native or _load()).release(kv_seq_len, block_table, ref_count, page_size, window, sinks, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_page_release")


def spec_page_compact(block_table, ref_count, copy_src, copy_dst, workspace, stream=None) -> None:
    """Moves used pages down into free ones below the number of pages in use; copy_src, copy_dst
    [capacity] receive the pairs to copy, then -1s."""
    st = (_native or _load()).compact(block_table, ref_count, copy_src, copy_dst, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_page_compact")


def spec_page_copy(k_cache, v_cache, copy_src, copy_dst, workspace, stream=None) -> None:
    """Copies the pages of the pairs in caches [pages, ...] or [layers, pages, ., ., .] (v_cache
    may be None); a page's elements have to be contiguous, in any order of its dimensions."""
    st = (_native or _load()).copy(k_cache, v_cache, copy_src, copy_dst, workspace, stream)
    if st != SV_OK:
        raise SvError(st, "spec_page_copy")


class PagedCache:
    """The paged KV cache of `slots` requests over `layers` layers, resident on a CUDA device, with
    one method per step of the header's sequence.  Plumbing only, like batch.DeviceBatch: it holds
    the tensors and the workspace, and every method is one or two of the calls above.

    k, v [layers, pages, page_size, heads, head_dim]; kv_seq_len [slots], block_table [slots,
    max_pages], ref_count [pages]: the state that spec_page_* work on.  All requests start empty.

    With dtype float8_e4m3fn the cache is in 8 bits: k_scale, v_scale [layers, pages, page_size /
    scale_tokens, heads] fp32 hold a scale for each scale_tokens tokens and head, each page's scales behind its numbers
    in the same allocation, so that a page and its scales are shared, moved and copied as one.
    append and attend then take queries of either 16-bit type.

    The cache is ready when the constructor returns (it waits for its fills), so that every method may
    be given any stream.  One cache's calls share its state and workspace: order those of different
    streams as for any tensors, by events or synchronisation.
    """

    def __init__(self, layers: int, slots: int, pages: int, page_size: int, max_pages: int, heads: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", scale_tokens: int = 16):
        shape = (layers, pages, page_size, heads, head_dim)
        self.k_scale = self.v_scale = None
        if dtype == torch.float8_e4m3fn:
            scale_tokens = min(scale_tokens, page_size)
            if scale_tokens < 1 or page_size % scale_tokens:
                raise ValueError("scale_tokens must divide page_size")
            blocks, size = page_size // scale_tokens, page_size * heads * head_dim
            if size % 16:
                raise ValueError("a page's keys must be a multiple of 16 bytes")
            # pages as bytes: their numbers, then their scales, in multiples of 16.  (Pages so begin anywhere in 128 bytes, which
            # attention feels where little else bounds it: 256 requests of one row over 4096 keys of 4 heads of 128 take 239 us,
            # 172 with pages that begin at multiples of 128; of 8 heads 328 and 323.  Appending does not feel it.)
            held = (layers, pages, size + (4 * blocks * heads + 15) // 16 * 16, 1, 1)
            self._pages = tuple(torch.zeros(held, dtype=torch.uint8, device=device) for _ in range(2))
            self.k, self.v = (x[:, :, :size, 0, 0].view(dtype).unflatten(2, shape[2:]) for x in self._pages)
            self.k_scale, self.v_scale = (
                x[:, :, :, 0, 0].view(torch.float32)[:, :, size // 4:size // 4 + blocks * heads].unflatten(2, (blocks, heads))
                for x in self._pages)
        else:
            self._pages = None
            self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        ints = dict(dtype=torch.int32, device=device)
        self.kv_seq_len = torch.zeros(slots, **ints)
        self.block_table = torch.full((slots, max_pages), -1, **ints)
        self.ref_count = torch.zeros(pages, **ints)
        self.page_size = page_size
        # pages to copy, kept: a tensor of one call would belong to the current stream alone
        self._pairs = torch.empty((2, max(slots, pages)), **ints)
        need = max(sv_attention_workspace_bytes(head_dim), sv_page_workspace_bytes(slots, pages))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.workspace[:256].zero_()
        if self.k.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.k.device).synchronize()

    def reserve(self, num_drafts, stream=None) -> None:
        """Room for num_drafts[b] + 1 new tokens of every request (-1: idle)."""
        spec_page_reserve(num_drafts, self.kv_seq_len, self.block_table, self.ref_count, self.page_size,
                          self.workspace, stream)

    def append(self, layer: int, q, k, v, q_weight, k_weight, eps, inv_freq, num_drafts, row_offsets, k_max, out_q,
               interleaved=False, rope_scale=1.0, stream=None) -> None:
        if self.k_scale is not None:
            spec_append8(q, k, v, q_weight, k_weight, eps, inv_freq, self.k[layer], self.v[layer], self.k_scale[layer],
                         self.v_scale[layer], self.block_table, self.kv_seq_len, num_drafts, row_offsets, k_max, out_q,
                         self.workspace, interleaved, rope_scale, stream)
            return
        spec_append(q, k, v, q_weight, k_weight, eps, inv_freq, self.k[layer], self.v[layer], self.block_table,
                    self.kv_seq_len, num_drafts, row_offsets, k_max, out_q, self.workspace, interleaved, rope_scale,
                    stream)

    def attend(self, layer: int, q, num_drafts, row_offsets, k_max, scale, out, window=0, sinks=0, out_lse=None,
               stream=None) -> None:
        if self.k_scale is not None:
            spec_attention8(q, self.k[layer], self.v[layer], self.k_scale[layer], self.v_scale[layer], self.block_table,
                            self.kv_seq_len, num_drafts, row_offsets, k_max, scale, window, sinks, out, out_lse,
                            self.workspace, stream)
            return
        spec_attention(q, self.k[layer], self.v[layer], self.block_table, self.kv_seq_len, num_drafts, row_offsets,
                       k_max, scale, window, sinks, out, out_lse, self.workspace, stream)

    def commit(self, accept_len, num_drafts, window=0, sinks=0, stream=None) -> None:
        """Rolls every request back to its accepted drafts (idle ones, -1 drafts, stay) and gives the
        pages past them back."""
        spec_cache_rollback(self.kv_seq_len, accept_len, num_drafts, self.workspace, stream)
        self.release(window, sinks, stream)

    def release(self, window=0, sinks=0, stream=None) -> None:
        spec_page_release(self.kv_seq_len, self.block_table, self.ref_count, self.page_size, window, sinks,
                          self.workspace, stream)

    def fork(self, parents, children, fork_len=None, stream=None) -> None:
        """Empty slots children[f] continue from (the first fork_len[f] tokens of) parents[f]."""
        src, dst = self._pairs[:, :parents.numel()]
        spec_page_fork(parents, children, fork_len, self.kv_seq_len, self.block_table, self.ref_count, self.page_size,
                       src, dst, self.workspace, stream)
        spec_page_copy(*(self._pages or (self.k, self.v)), src, dst, self.workspace, stream)

    def compact(self, capacity: int, stream=None) -> None:
        """Moves up to `capacity` used pages down into the free ones below them."""
        src, dst = self._pairs[:, :capacity]
        spec_page_compact(self.block_table, self.ref_count, src, dst, self.workspace, stream)
        spec_page_copy(*(self._pages or (self.k, self.v)), src, dst, self.workspace, stream)
