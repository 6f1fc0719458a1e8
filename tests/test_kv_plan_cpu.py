"""The K/V cache operators' index arithmetic (csrc/qmm_kv_plan.h, plain C++), on the CPU: attention's
units are dealt out once each, partial sums land in slots of their own that the join reads again, and
the positions of a block's tiles are those that its rows see and that the page table can name.  Also
what the C ABI refuses, which needs no GPU, and the host's bookkeeping of pages."""
import ctypes
import random
import shutil
import subprocess

import pytest
import torch

import bit_quantized_gemm_qmm_b200 as q
from bit_quantized_gemm_qmm_b200 import _build, kv

HARNESS = r"""
#include <vector>
#include "qmm_kv_plan.h"
using namespace qmm_impl;
// Walks the blocks as the kernels do.  Returns 0, or the number of the first check that fails.
extern "C" int walk(int seqs, const int* cu, const int* lens, int tokens, int capacity, int kv_heads, int gh, int rows,
                    int window, int tree, int blocks, int unit, int warps, int start) {
    std::vector<AttnSeq> s;
    std::vector<int> item0, unit0;  // items and units in front of each sequence
    int units = 0, items = 0;
    for (int b = 0; b < seqs; ++b) {
        if (cu[b + 1] < cu[b]) return 0;  // nothing is done
        s.push_back(attn_seq(cu[b], cu[b + 1], lens[b], tokens, capacity, gh, rows, unit, window));
        const AttnSeq& q = s.back();
        if (q.row0 < 0 || q.n < 0 || q.row0 + q.n > tokens || q.keys < 0 || q.keys > capacity) return 1;
        if (q.lo < 0 || q.lo % kAttnSub || q.lo > q.keys || q.units < 1) return 2;
        item0.push_back(items), unit0.push_back(units);
        units += attn_seq_units(q, kv_heads);
        items += attn_seq_items(q, kv_heads);
    }
    const AttnPlan p = attn_plan(units, items, blocks, start, warps);
    if (p.per < 1) return 3;
    std::vector<int> taken(units, 0), slots(2 * blocks, -1);  // slot -> item
    struct Shared { int c0, c1; };
    std::vector<Shared> shared(items, Shared{-1, -1});
    int order = 0;
    for (int b = 0; b < seqs; ++b) order += attn_seq_weight(p, s[b], kv_heads);
    if (p.pieces && order > blocks) return 4;
    if (!p.pieces && (order != p.total || (int64_t)blocks * p.per < order)) return 5;
    for (int i = 0; i < blocks; ++i) {
        int x = p.pieces ? i : i * p.per;
        const int end = p.pieces ? x + 1 : x + p.per < order ? x + p.per : order;
        if (x >= order) continue;
        int b = 0, before = 0;
        while (x < end) {
            const int weight = attn_seq_weight(p, s[b], kv_heads);
            if (x >= before + weight) { before += weight; if (++b >= seqs) return 6; continue; }
            const AttnShare h = attn_share(p, s[b], x, end, before);
            if (h.places < 1) return 23;
            if (h.item < 0 || h.item >= s[b].rt * kv_heads || h.u0 < 0 || h.n < 0 || h.u0 + h.n > s[b].units) return 7;
            if (h.n == 0) { x += h.places; continue; }
            if (i < h.c0 || i > h.c1 || h.c1 >= blocks) return 8;
            if ((h.n == s[b].units) != (h.c0 == h.c1)) return 9;
            if ((h.u0 == 0) != (i == h.c0)) return 24;
            for (int u = 0; u < h.n; ++u) ++taken[unit0[b] + h.item * s[b].units + h.u0 + u];
            const int id = item0[b] + h.item;
            if (h.n != s[b].units) {
                const int slot = attn_slot(i, h.c0);
                if (slot < 0 || slot >= 2 * blocks || slots[slot] != -1) return 10;
                slots[slot] = id;
                if (shared[id].c0 >= 0 && (shared[id].c0 != h.c0 || shared[id].c1 != h.c1)) return 11;
                shared[id] = Shared{h.c0, h.c1};
            }
            // tiles of the run
            const int rt = h.item % s[b].rt, r0 = rt * rows, nr = s[b].n * gh - r0 < rows ? s[b].n * gh - r0 : rows;
            if (nr < 1) return 12;
            int lo, hi;
            attn_range(s[b], r0, r0 + nr, gh, window, tree, &lo, &hi);
            if (lo < 0 || hi < 0 || hi > s[b].keys) return 13;
            if (window > 0 && lo < s[b].lo) return 14;
            const int t0 = s[b].lo + unit * h.u0;
            std::vector<int> by(h.n, 0);  // units some warp takes
            for (int w = 0; unit == kAttnUnit && w < warps; ++w) {
                int j0, j1;
                attn_warp_units(t0, h.n, w, warps, lo, hi, &j0, &j1);
                if (j0 < 0) return 15;
                for (int j = j0; j < j1; ++j) {
                    if (w + warps * j >= h.n) return 16;
                    ++by[w + warps * j];
                }
            }
            for (int u = 0; u < h.n; ++u) {
                const int t = t0 + unit * u;
                const bool any = t < hi && t + unit > lo && t < s[b].keys;
                if (unit == kAttnUnit && by[u] != (any ? 1 : 0)) return 17;
                if (t < 0 || t % kAttnSub) return 18;
            }
            x += h.places;
        }
    }
    for (int u = 0; u < units; ++u) if (taken[u] != 1) return 19;
    // the join: an item's blocks c0..c1 read the slots that they wrote, and no two items share a counter
    std::vector<int> counter(blocks, -1), read(2 * blocks, 0);
    for (int id = 0; id < items; ++id) {
        if (shared[id].c0 < 0) continue;
        if (counter[shared[id].c0] != -1) return 20;
        counter[shared[id].c0] = id;
        for (int i = shared[id].c0; i <= shared[id].c1; ++i) {
            const int slot = attn_slot(i, shared[id].c0);
            if (slots[slot] != id) return 21;
            read[slot] = 1;
        }
    }
    for (int k = 0; k < 2 * blocks; ++k) if ((slots[k] != -1) != (read[k] != 0)) return 22;
    return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_plan")
    (d / "walk.cpp").write_text(HARNESS)
    subprocess.check_call([shutil.which("g++"), "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I" + _build.CSRC,
                           str(d / "walk.cpp"), "-o", str(d / "walk.so")])
    return ctypes.CDLL(str(d / "walk.so")).walk


def test_every_unit_once_and_every_slot_its_own(walk):
    rng = random.Random(5)
    for turn in range(400):
        seqs = rng.choice([1, 2, 5, 40])
        page_cap = 16 * rng.randrange(0, 60)
        new = [rng.choice([0, 1, 1, 1, 3, 17, 70]) for _ in range(seqs)]
        lens = [rng.choice([0, 1, n, n + 1, n + rng.randrange(0, 900), rng.randrange(0, 30)]) for n in new]
        cu = [sum(new[:i]) for i in range(seqs + 1)]
        tokens = sum(new) + rng.choice([0, 0, 3])
        if turn % 5 == 0:  # whatever device memory may hold
            cu = [c + rng.choice([0, 0, -9, 2 ** 30, -2 ** 31]) if rng.random() < 0.3 else c for c in cu]
            cu = [max(-2 ** 31, min(2 ** 31 - 1, c)) for c in cu]
            lens = [rng.choice([n, -5, -2 ** 31, page_cap + 7]) for n in lens]
        window = rng.choice([0, 0, 1, 15, 16, 100, 2 ** 29])
        tree = 0 if window else rng.choice([0, 1])
        arr = lambda v: (ctypes.c_int * len(v))(*v)  # noqa: E731
        args = (seqs, arr(cu), arr(lens), tokens, page_cap, rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 8]),
                rng.choice([8, 16, 32, 64]), window, tree, rng.choice([1, 2, 7, 148, 296]), *rng.choice([(32, 4, 20), (32, 6, 20), (128, 1, 2), (32, 6, 0)]))
        got = walk(*args)
        assert got == 0, (got, seqs, cu, lens, args[3:])


# ------------------------------------------------------------------------------ what the ABI refuses
@pytest.fixture(scope="module")
def L():
    _build.build()
    return q.lib()


def cache(**kw):
    a = dict(k_packed=16, k_scales=16, k_biases=16, v_packed=16, v_scales=16, v_biases=16, pages=4, page_size=64,
             kv_heads=2, head_dim=128, group=64, bits=4, reserved=0)
    a.update(kw)
    return q.CacheDesc(**a)


def seqs(**kw):
    a = dict(page_table=16, cu_tokens=16, seqs=2, table_stride=3, max_pages=3)
    a.update(kw)
    return q.SeqsDesc(**a)


def calls(L, c, s, tokens=2, dtype=0, k=16, stride=256, at=16):
    r = ctypes.byref
    return [L.qmm_kv_append(r(c), k, stride, 128, k, stride, 128, r(s), at, tokens, dtype, None),
            L.qmm_kv_gather(r(c), r(s), at, tokens, k, stride, 128, k, stride, 128, dtype, None),
            L.qmm_kv_attention(r(c), k, stride, 128, k, stride, 128, None, r(s), at, tokens, 2, 1.0, 0, None, dtype, None)]


BAD_CACHE = [(dict(bits=8), 2), (dict(head_dim=96, group=32), 2), (dict(head_dim=512), 2), (dict(group=16), 2),
             (dict(head_dim=64, group=128), 1), (dict(page_size=8), 2), (dict(page_size=24), 2), (dict(page_size=2048), 2),
             (dict(page_size=0), 2), (dict(kv_heads=0), 2), (dict(kv_heads=257), 2), (dict(pages=0), 1), (dict(pages=-1), 1),
             (dict(pages=2 ** 31), 1), (dict(pages=2 ** 29), 2), (dict(k_packed=0), 1), (dict(v_biases=0), 1), (dict(k_scales=24), 1)]
BAD_SEQS = [(dict(seqs=-1), 1), (dict(seqs=65537), 2), (dict(max_pages=-1), 1), (dict(table_stride=2), 1),
            (dict(page_table=0), 1), (dict(cu_tokens=0), 1), (dict(page_table=18), 1), (dict(cu_tokens=17), 1),
            (dict(max_pages=2 ** 25, table_stride=2 ** 25), 2)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_refuses_caches(L, kw, status):
    c = cache(**kw)
    assert calls(L, c, seqs()) == [status] * 3
    assert L.qmm_kv_copy_pages(ctypes.byref(c), 16, 16, 1, None) == status
    assert L.qmm_kv_compact(ctypes.byref(c), ctypes.byref(seqs()), 16, 16, 1, None) == status
    assert L.qmm_last_error()


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_refuses_sequences(L, kw, status):
    s = seqs(**kw)
    assert calls(L, cache(), s) == [status] * 3
    assert L.qmm_kv_compact(ctypes.byref(cache()), ctypes.byref(s), 16, 16, 1, None) == status


def test_refuses_other_arguments(L):
    r = ctypes.byref
    c, s = cache(), seqs()
    assert calls(L, c, s, dtype=7) == [1] * 3
    assert calls(L, c, s, tokens=-1) == [1] * 3
    assert calls(L, c, s, tokens=2 ** 20 + 1) == [2] * 3
    assert calls(L, c, s, k=0) == [1] * 3
    assert calls(L, c, s, k=17) == [1] * 3
    assert calls(L, c, s, at=0) == [1] * 3
    assert calls(L, c, s, at=18) == [1] * 3
    att = lambda o=16, ostr=256, lse=None, heads=2, window=0, tree=None: L.qmm_kv_attention(  # noqa: E731
        r(c), 16, 256, 128, o, ostr, 128, lse, r(s), 16, 2, heads, 1.0, window, tree, 0, None)
    assert att(heads=3) == 1 and att(heads=0) == 2 and att(heads=258) == 2 and att(heads=-2) == 2
    assert att(window=-1) == 1 and att(window=4, tree=16) == 2
    assert att(o=0) == 1 and att(o=12) == 1 and att(ostr=258) == 1 and att(lse=18) == 1 and att(tree=20) == 1
    gather = lambda k=16, stride=256: L.qmm_kv_gather(r(c), r(s), 16, 2, k, stride, 128, 16, 256, 128, 0, None)  # noqa: E731
    assert gather(k=24) == 1 and gather(stride=260) == 1
    # output rows that overlap: broadcast tokens, tokens closer than their heads take
    assert gather(stride=0) == 1 and gather(stride=128) == 1 and gather(stride=248) == 1 and gather(stride=-248) == 1
    assert att(ostr=0) == 1 and att(ostr=252) == 1 and att(ostr=-252) == 1
    assert L.qmm_kv_copy_pages(r(c), 16, 16, -1, None) == 1 and L.qmm_kv_copy_pages(r(c), 16, 16, 2 ** 16 + 1, None) == 2
    assert L.qmm_kv_copy_pages(r(c), 0, 16, 1, None) == 1 and L.qmm_kv_copy_pages(r(c), 16, 18, 1, None) == 1
    assert L.qmm_kv_compact(r(c), r(s), 16, 0, 1, None) == 1 and L.qmm_kv_compact(r(c), r(s), 16, 18, 1, None) == 1
    null = ctypes.POINTER(q.CacheDesc)()
    assert L.qmm_kv_copy_pages(null, 16, 16, 1, None) == 1
    assert L.qmm_kv_compact(r(c), ctypes.POINTER(q.SeqsDesc)(), 16, 16, 1, None) == 1
    # nothing to do: no pointer is looked at
    none = seqs(seqs=0, page_table=0, cu_tokens=0)
    assert calls(L, c, none, k=0, at=0) == [0] * 3 and calls(L, c, s, tokens=0, k=0, at=0) == [0] * 3
    assert L.qmm_kv_copy_pages(r(c), 0, 0, 0, None) == 0 and L.qmm_kv_compact(r(c), r(s), 0, 0, 0, None) == 0


def test_call_module_refuses(L):
    """The C hand-off looks at every tensor before it calls: types, counts of arguments, devices."""
    m = kv._calls()
    c = cache()
    a, t = ctypes.addressof(c), torch.zeros(2, 2, 128, dtype=torch.float16)
    for f, n in ((m.kv_append, 7), (m.kv_gather, 7), (m.kv_copy_pages, 4), (m.kv_compact, 6), (m.kv_attention, 11)):
        for args in ([0] * (n - 1), [a, 0] + [t] * (n - 3), [a, 0] + [3] * (n - 2), ["a", 0] + [t] * (n - 2),
                     [a, "0"] + [t] * (n - 2), [a, 0] + [None] * (n - 2)):
            with pytest.raises(TypeError):
                f(*args)
        with pytest.raises(ValueError, match="CUDA device"):
            f(a, 0, *[t] * (n - 2))
        with pytest.raises(ValueError, match="null"):
            f(0, 0, *[t] * (n - 2))
    with pytest.raises((ValueError, TypeError)):
        m.bind_kv(0, 0, 0, 0, 0, torch.Tensor)
    with pytest.raises(TypeError):
        m.bind_kv(1, 1, 1, 1, 1, 1)


def test_cache_refuses_cpu_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        q.KVCache(z(2, 1, 16, 8, dtype=torch.int32), *[z(2, 1, 16, 1, dtype=torch.float16)] * 2,
                  z(2, 1, 16, 8, dtype=torch.int32), *[z(2, 1, 16, 1, dtype=torch.float16)] * 2, group=64)


# ------------------------------------------------------------------------------ the host's bookkeeping
class Pages:
    """A cache on the host, as far as the bookkeeping looks at it: rows are numbers."""

    def __init__(self, pages, page_size):
        self.pages, self.page_size, self.kv_heads, self.head_dim, self.device, self._index = pages, page_size, 1, 64, "cpu", -1
        self.rows = [[None] * page_size for _ in range(pages)]


@pytest.fixture
def book(monkeypatch):
    c = Pages(40, 4)

    def copy(cache, src, dst):
        assert not set(src.tolist()) & set(dst.tolist()) and len(set(dst.tolist())) == len(dst)
        for a, b in zip(src.tolist(), dst.tolist()):
            cache.rows[b] = list(cache.rows[a])

    def append(cache, k, v, table, lens, cu):
        for b in range(table.shape[0]):
            r0, r1 = cu[b].item(), cu[b + 1].item()
            for i in range(r0, r1):
                p = lens[b].item() - (r1 - r0) + i - r0
                cache.rows[table[b, p // cache.page_size].item()][p % cache.page_size] = k[i, 0, 0].item()

    def compact(cache, table, starts, keep, cu):
        for b in range(table.shape[0]):
            at = lambda p: (table[b, p // cache.page_size].item(), p % cache.page_size)  # noqa: B023,E731
            mine = keep[cu[b]:cu[b + 1]].tolist()
            got = [cache.rows[at(starts[b].item() + j)[0]][at(starts[b].item() + j)[1]] for j in mine]
            for i, x in enumerate(got):
                pg, r = at(starts[b].item() + i)
                cache.rows[pg][r] = x

    monkeypatch.setattr(kv, "kv_copy_pages", copy)
    monkeypatch.setattr(kv, "kv_append", append)
    monkeypatch.setattr(kv, "kv_compact", compact)
    monkeypatch.setattr(kv, "kv_attention", lambda cache, x, *a, **k: (x, None))
    monkeypatch.setattr(kv.KVSequences, "_device", lambda self, *lists: tuple(torch.tensor(v, dtype=torch.int32) for v in lists))
    return c, kv.KVSequences(c)


def test_bookkeeping_against_plain_lists(book):
    """Random steps, forks, accepts, cuts and ends: every sequence reads back its own rows."""
    c, s = book
    rng = random.Random(11)
    rows, drafts, stamp = {}, {}, 0

    def held(name):
        return [c.rows[s.pages(name)[p // 4]][p % 4] for p in range(s.length(name))]

    for turn in range(600):
        do = rng.choice(["add", "step", "step", "step", "fork", "accept", "accept", "cut", "free"])
        names = list(rows)
        some = rng.sample(names, rng.randrange(0, len(names) + 1)) if names else []
        try:
            if do == "add" and len(rows) < 6:
                n = s.add()
                rows[n], drafts[n] = [], 0
            elif do == "step" and some:
                new = [rng.randrange(0, 9) for _ in some]
                k = torch.arange(stamp, stamp + sum(new), dtype=torch.float32)[:, None, None].repeat(1, 1, 64)
                s.step(some, k, k, k, new)
                for n, m in zip(some, new):
                    rows[n] = rows[n] + list(range(stamp, stamp + m))
                    drafts[n] = m
                    stamp += m
            elif do == "fork" and names and len(rows) < 6:
                f = s.fork(names[0])
                rows[f], drafts[f] = list(rows[names[0]]), 0
            elif do == "accept" and some:
                keep = [sorted(rng.sample(range(drafts[n]), rng.randrange(0, drafts[n] + 1))) for n in some]
                s.accept(some, keep)
                for n, mine in zip(some, keep):
                    base = len(rows[n]) - drafts[n]
                    rows[n], drafts[n] = rows[n][:base] + [rows[n][base + j] for j in mine], 0
            elif do == "cut" and names:
                at = rng.randrange(0, len(rows[names[-1]]) + 1)
                s.truncate(names[-1], at)
                rows[names[-1]], drafts[names[-1]] = rows[names[-1]][:at], 0
            elif do == "free" and names and rng.random() < 0.5:
                n = rng.choice(names)
                s.free(n)
                del rows[n], drafts[n]
        except RuntimeError as e:
            assert "full" in str(e)
            for n in list(rows):  # make room
                if rng.random() < 0.6:
                    s.free(n)
                    del rows[n], drafts[n]
        for n in rows:
            assert held(n) == rows[n], (turn, do, n)
    for n in list(rows):
        s.free(n)
    assert s.free_pages() == 40


def test_bookkeeping_refusals(book):
    c, s = book
    a = s.add()
    k = torch.zeros(5, 1, 64)
    with pytest.raises(ValueError):
        s.step([a, a], k, k, k, [2, 3])
    with pytest.raises(ValueError):
        s.step([a], k, k, k, [4])
    with pytest.raises(KeyError):
        s.step([a + 1], k, k, k, [5])
    with pytest.raises(RuntimeError, match="full"):
        big = torch.zeros(200, 1, 64)
        s.step([a], big, big, big, [200])
    assert s.length(a) == 0 and s.free_pages() == 40
    s.step([a], k, k, k, [5])
    for keep in ([0, 0], [1, 0], [5], [-1]):
        with pytest.raises(ValueError):
            s.accept([a], [keep])
    with pytest.raises(ValueError):
        s.truncate(a, 6)
    with pytest.raises(ValueError):
        s.accept([a], [])
    assert s.length(a) == 5


@pytest.mark.parametrize("call", ["kv_append", "kv_attention"])
def test_refused_step_changes_nothing(book, monkeypatch, call):
    """A step whose calls refuse their arguments (a tree with a window, say) leaves lengths, pages and drafts."""
    c, s = book
    a, b = s.add(), s.add()
    k = torch.zeros(9, 1, 64)
    s.step([a, b], k, k, k, [6, 3])
    pages = [s.pages(a), s.pages(b)]

    def refuse(*args, **kwargs):
        raise ValueError("refused")

    with monkeypatch.context() as m:
        m.setattr(kv, call, refuse)
        with pytest.raises(ValueError, match="refused"):
            s.step([b, a], k, k, k, [2, 7])
    assert (s.length(a), s.length(b)) == (6, 3) and [s.pages(a), s.pages(b)] == pages and s.free_pages() == 37
    s.accept([a, b], [[0, 5], [2]])
    assert (s.length(a), s.length(b)) == (2, 1) and s.free_pages() == 38
