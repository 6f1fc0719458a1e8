"""Binding of the paged 4-bit K/V cache: the cache's arrays, attention over it and what keeps it.

    cache = KVCache.empty(pages=4096, page_size=64, kv_heads=8, head_dim=128, group=64)
    kv_append(cache, k, v, page_table, lens, cu_tokens)            # k, v: [tokens, kv_heads, head_dim]
    o, lse = kv_attention(cache, q, page_table, lens, cu_tokens)   # q, o: [tokens, heads, head_dim]

As everywhere in the package this is argument marshalling: quantizing, attention and the moves are
kernels behind the C ABI (include/qmm.h, whose comments hold each call's contract).  Page tables
[seqs, pages], lengths [seqs] and offsets [seqs + 1] are int32 tensors on the cache's device, read in
stream order, so captured graphs can be replayed with other contents.  ``KVSequences`` is the host's
side of a serving loop: which page belongs to whom, with fork and free.
"""
from __future__ import annotations

import ctypes

import torch

import bit_quantized_gemm_qmm_b200 as _q

_ARRAYS = ("k_packed", "k_scales", "k_biases", "v_packed", "v_scales", "v_biases")


class KVCache:
    """The six arrays of a paged cache (packed [pages, kv_heads, page_size, head_dim/8] int32, scales
    and biases [..., head_dim/group] fp16, for K and for V) and their format.  The tensors are the
    caller's and are kept alive by the cache."""

    def __init__(self, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, group: int):
        arrays = (k_packed, k_scales, k_biases, v_packed, v_scales, v_biases)
        if not all(t.is_cuda and t.device == k_packed.device for t in arrays):
            raise ValueError("the cache's arrays must be on one CUDA device")
        if k_packed.dim() != 4:
            raise ValueError("k_packed must be [pages, kv_heads, page_size, head_dim/8]")
        pages, heads, page, words = k_packed.shape
        dim = words * 8
        if group <= 0 or dim % group:
            raise ValueError(f"head_dim={dim} is not a multiple of group={group}")
        for name, t in zip(_ARRAYS, arrays):
            want = (pages, heads, page, words if name.endswith("packed") else dim // group)
            kind = torch.int32 if name.endswith("packed") else torch.float16
            if tuple(t.shape) != want or t.dtype is not kind or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {kind} {list(want)}, got {t.dtype} {list(t.shape)}")
            setattr(self, name, t)
        self.pages, self.kv_heads, self.page_size, self.head_dim, self.group = pages, heads, page, dim, group
        self.device, self.scale = k_packed.device, dim ** -0.5
        self._index = k_packed.get_device()
        self._desc = _q.CacheDesc(*(t.data_ptr() for t in arrays), pages, page, heads, dim, group, 4, 0)
        self._addr = ctypes.addressof(self._desc)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, group: int = 64, device="cuda") -> "KVCache":
        """A cache over newly allocated arrays; positions hold nothing until they are appended."""
        if group <= 0 or head_dim % group or head_dim % 8:
            raise ValueError(f"head_dim={head_dim} is not a multiple of group={group}")
        shape = (pages, kv_heads, page_size)
        one = [torch.zeros((*shape, head_dim // 8), dtype=torch.int32, device=device),
               torch.zeros((*shape, head_dim // group), dtype=torch.float16, device=device),
               torch.zeros((*shape, head_dim // group), dtype=torch.float16, device=device)]
        return cls(*one, *(torch.zeros_like(t) for t in one), group=group)

    def arrays(self) -> list[torch.Tensor]:
        return [getattr(self, name) for name in _ARRAYS]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.arrays())


_call = None
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _calls():
    """The C hand-off module, bound to the loaded library's functions.  It checks the tensors (device,
    dtype, shape, strides) and passes them on with the device's current stream."""
    global _call
    if _call is None:
        L = _q.lib()
        try:
            from . import _qmm_call
        except ImportError as e:
            raise _q.QmmUnavailable(f"the _qmm_call module is missing ({e}); run __graft_entry__.build()") from e
        if not hasattr(_qmm_call, "bind_kv"):
            raise _q.QmmUnavailable("the K/V cache needs a torch with DLPack's exchange functions (1.3)")
        _qmm_call.bind_kv(*(ctypes.cast(getattr(L, "qmm_kv_" + n), ctypes.c_void_p).value
                            for n in ("append", "gather", "copy_pages", "compact", "attention")), torch.Tensor)
        _call = _qmm_call
    return _call


def _run(cache: KVCache, fn, *args) -> None:
    """One hand-off, on the cache's device; a status other than OK is raised."""
    if cache._index == _device():
        st = fn(cache._addr, cache._index, *args)
    else:  # the library launches on the calling thread's current device
        with torch.cuda.device(cache._index):
            st = fn(cache._addr, cache._index, *args)
    if st:
        _q._check(st)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
              cu_tokens: torch.Tensor) -> None:
    """Quantizes new tokens' K and V rows ([tokens, kv_heads, head_dim], any token and head strides)
    into the cache.  lens counts each sequence's tokens with the new ones, which are its last; rows
    cu_tokens[b]..cu_tokens[b+1]-1 are sequence b's."""
    _run(cache, _calls().kv_append, k, v, page_table, lens, cu_tokens)


def kv_gather(cache: KVCache, page_table: torch.Tensor, starts: torch.Tensor, cu_tokens: torch.Tensor, tokens: int,
              dtype: torch.dtype = torch.float16, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Cache rows as dense (k, v) [tokens, kv_heads, head_dim]: rows cu_tokens[b] + i are positions
    starts[b] + i of sequence b.  Rows of no sequence are left as they are."""
    if out is None:
        k = torch.empty(tokens, cache.kv_heads, cache.head_dim, dtype=dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        if k.shape[0] != tokens or k.dtype is not dtype:
            raise ValueError("out must be two [tokens, kv_heads, head_dim] tensors of dtype")
    _run(cache, _calls().kv_gather, k, v, page_table, starts, cu_tokens)
    return k, v


def kv_copy_pages(cache: KVCache, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Page dst[i] becomes a copy of page src[i] (all heads, K and V).  No page may be one pair's
    source and another's target; of pairs with one target the last counts."""
    _run(cache, _calls().kv_copy_pages, src, dst)


def kv_compact(cache: KVCache, page_table: torch.Tensor, starts: torch.Tensor, keep: torch.Tensor,
               cu_keep: torch.Tensor) -> None:
    """Moves accepted draft rows together: entries cu_keep[b]..cu_keep[b+1]-1 of keep, rising, are
    offsets from starts[b] of the rows of sequence b that become rows starts[b], starts[b] + 1, ..."""
    _run(cache, _calls().kv_compact, page_table, starts, keep, cu_keep)


def kv_attention(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, cu_tokens: torch.Tensor,
                 scale: float | None = None, window: int = 0, tree: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """(o, lse) = attention of q [tokens, heads, head_dim] over the cache, the new tokens included
    (kv_append comes first).  scale: head_dim ** -0.5 by default.  window > 0: a token sees the last
    `window` positions up to its own.  tree: int64 [tokens], bit j of a token's mask set where it sees
    its sequence's new token j (and every position before the new ones).  o has q's dtype; lse is fp32
    [tokens, heads], -inf where a row sees nothing.  Rows of no sequence are left as they are."""
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if lse is None:
        n, heads = q.shape[:2]
        lse = torch.empty(n, heads, dtype=torch.float32, device=cache.device)
    _run(cache, _calls().kv_attention, q, page_table, lens, cu_tokens, out, lse, tree, window,
         cache.scale if scale is None else scale)
    return out, lse


class KVSequences:
    """Which pages of a cache belong to which sequence: the host's bookkeeping of a serving loop, with
    page tables and lengths on the device for the calls.

    Sequences are named by the numbers that ``add`` and ``fork`` return.  Forked sequences share their
    full pages; a partly filled last page is copied when the fork is made.  Pages go back to the pool
    when the last sequence that holds them lets go.  One cache, so one layer: a model has an object a layer.
    Each step lists its sequences' pages anew on the host (0.4 ms for 32 sequences of 8,192 positions in pages
    of 64); a loop that is bound by that keeps its own tables and makes the calls itself.

        s = KVSequences(cache)
        a = s.add()
        o = s.step([a], q, k, v, [len(q)])            # a prompt: append, then attend
        b = s.fork(a)
        o = s.step([a, b], q, k, v, [5, 5], tree)     # a draft each
        s.accept([a, b], [[0, 2], [0, 1, 4]])         # what the model agreed with
        s.free(a)
    """

    def __init__(self, cache: KVCache):
        self.cache = cache
        self._free = list(range(cache.pages - 1, -1, -1))  # taken from the end: low pages first
        self._held = [0] * cache.pages
        self._pages: dict[int, list[int]] = {}
        self._lens: dict[int, int] = {}
        self._drafts: dict[int, int] = {}
        self._next = 0

    def add(self) -> int:
        """A new, empty sequence."""
        name, self._next = self._next, self._next + 1
        self._pages[name], self._lens[name] = [], 0
        return name

    def length(self, seq: int) -> int:
        return self._lens[seq]

    def pages(self, seq: int) -> list[int]:
        return list(self._pages[seq])

    def free_pages(self) -> int:
        return len(self._free)

    def _take(self, n: int) -> list[int]:
        if n > len(self._free):
            raise RuntimeError(f"the cache is full: {n} pages needed, {len(self._free)} free")
        got = [self._free.pop() for _ in range(n)]
        for p in got:
            self._held[p] = 1
        return got

    def _drop(self, pages: list[int]) -> None:
        for p in reversed(pages):
            self._held[p] -= 1
            if self._held[p] == 0:
                self._free.append(p)

    def fork(self, seq: int) -> int:
        """A sequence that begins as a copy of `seq`: full pages shared, the last one copied."""
        pages, n = self._pages[seq], self._lens[seq]
        full = n // self.cache.page_size
        own = self._copies(pages[full:full + 1] if n % self.cache.page_size else [])
        name = self.add()
        for p in pages[:full]:
            self._held[p] += 1
        self._pages[name], self._lens[name] = pages[:full] + own, n
        return name

    def free(self, seq: int) -> None:
        """Ends a sequence; its pages that no other sequence holds are free again."""
        self._drop(self._pages.pop(seq))
        del self._lens[seq]
        self._drafts.pop(seq, None)

    def _device(self, *lists):
        """Lists of integers as int32 vectors on the device, in one copy."""
        host = torch.tensor([x for values in lists for x in values], dtype=torch.int32).pin_memory()
        return host.to(self.cache.device, non_blocking=True).split([len(values) for values in lists])

    def _copies(self, pages: list[int]) -> list[int]:
        """New pages that are copies of some; none where the copying is refused."""
        own = self._take(len(pages))
        try:
            if own:
                kv_copy_pages(self.cache, *self._device(pages, own))
        except Exception:
            self._drop(own)
            raise
        return own

    def _table(self, seqs: list[int]):
        """The sequences' page table as one list, and its columns."""
        cols = max((len(self._pages[s]) for s in seqs), default=0)
        return [p for s in seqs for p in self._pages[s] + [-1] * (cols - len(self._pages[s]))], cols

    def tables(self, seqs: list[int]):
        """(page_table, lens) of some sequences on the device."""
        flat, cols = self._table(seqs)
        table, lens = self._device(flat, [self._lens[s] for s in seqs])
        return table.reshape(len(seqs), cols), lens

    def _own(self, seqs: list[int], ranges: list[tuple[int, int]]) -> None:
        """Gives each sequence copies of its own of those pages numbered ranges[i][0] up to ranges[i][1] that
        others hold too: rows are about to be written there.  All or, where the pool is too small, none."""
        shared = [(s, i) for s, (lo, hi) in zip(seqs, ranges) for i in range(lo, min(hi, len(self._pages[s])))
                  if self._held[self._pages[s][i]] > 1]
        if not shared:
            return
        was = [self._pages[s][i] for s, i in shared]
        for (s, i), p in zip(shared, self._copies(was)):
            self._pages[s][i] = p
        self._drop(was)

    def truncate(self, seq: int, length: int) -> None:
        """Forgets a sequence's tokens from `length` on."""
        if not 0 <= length <= self._lens[seq]:
            raise ValueError(f"length={length} of a sequence of {self._lens[seq]} tokens")
        page = self.cache.page_size
        need = -(-length // page)
        if length % page:  # appending goes on in the last page
            self._own([seq], [(need - 1, need)])
        self._drop(self._pages[seq][need:])
        del self._pages[seq][need:]
        self._lens[seq] = length
        self._drafts[seq] = 0

    def step(self, seqs: list[int], q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, new: list[int],
             tree: torch.Tensor | None = None, window: int = 0, scale: float | None = None) -> torch.Tensor:
        """Appends new[i] tokens to sequence seqs[i] (rows of q, k and v in that order) and returns
        their attention [tokens, heads, head_dim]."""
        if len(set(seqs)) != len(seqs) or len(new) != len(seqs) or sum(new) != q.shape[0] or min(new, default=0) < 0:
            raise ValueError("seqs must be different sequences, new their counts of the rows")
        for t in (q, k, v):
            if t.dim() != 3 or t.shape[0] != q.shape[0] or t.shape[2] != self.cache.head_dim or t.dtype is not q.dtype:
                raise ValueError("q, k and v must be [tokens, heads, head_dim] of one dtype")
        page = self.cache.page_size
        need = [-(-(self._lens[s] + n) // page) - len(self._pages[s]) for s, n in zip(seqs, new)]
        got = self._take(sum(need))
        was = [(s, len(self._pages[s]), self._lens[s], self._drafts.get(s, 0)) for s in seqs]
        for s, n, m in zip(seqs, new, need):
            self._pages[s] += got[:m]
            del got[:m]
            self._lens[s] += n
            self._drafts[s] = n
        try:
            flat, cols = self._table(seqs)
            table, lens, cu = self._device(flat, [self._lens[s] for s in seqs], [sum(new[:i]) for i in range(len(new) + 1)])
            table = table.reshape(len(seqs), cols)
            kv_append(self.cache, k, v, table, lens, cu)
            return kv_attention(self.cache, q, table, lens, cu, scale=scale, window=window, tree=tree)[0]
        except Exception:  # a refused call leaves the sequences as they were
            for s, pages, n, draft in was:
                self._drop(self._pages[s][pages:])
                del self._pages[s][pages:]
                self._lens[s], self._drafts[s] = n, draft
            raise

    def accept(self, seqs: list[int], keep: list[list[int]]) -> None:
        """Keeps some of the tokens of each sequence's last step (their numbers in it, rising) and
        forgets the others."""
        if len(set(seqs)) != len(seqs):
            raise ValueError("seqs must be different sequences")
        starts = []
        for s, mine in zip(seqs, keep, strict=True):
            n = self._drafts.get(s, 0)
            if any(not 0 <= j < n for j in mine) or any(a >= b for a, b in zip(mine, mine[1:])):
                raise ValueError(f"keep={mine}: rising numbers below {n} expected")
            starts.append(self._lens[s] - n)
        page = self.cache.page_size
        self._own(seqs, [(start // page, -(-(start + len(mine)) // page)) for start, mine in zip(starts, keep)])
        moves = [i for i, mine in enumerate(keep) if mine != list(range(len(mine)))]
        if moves:
            names, kept = [seqs[i] for i in moves], [keep[i] for i in moves]
            flat, cols = self._table(names)
            table, first, rows, cu = self._device(flat, [starts[i] for i in moves], [j for mine in kept for j in mine],
                                                  [sum(len(m) for m in kept[:i]) for i in range(len(kept) + 1)])
            kv_compact(self.cache, table.reshape(len(names), cols), first, rows, cu)
        for s, start, mine in zip(seqs, starts, keep):
            self.truncate(s, start + len(mine))
