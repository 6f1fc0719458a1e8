// qmm_kv_plan.h -- index arithmetic of the paged K/V cache operators, shared by host and device
// (plain C++, so it is also tested on the CPU): which rows of the token axis a sequence has,
// which cache positions they see, and how attention's work is cut over its blocks.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define QMM_HD __host__ __device__ __forceinline__
#else
#define QMM_HD inline
#endif

namespace qmm_impl {

constexpr int kAttnSub = 16;              // positions whose page is looked up once (pages are multiples of it)
constexpr int kAttnUnit = 2 * kAttnSub;   // unit of work of the warps' kernel: what a warp takes at a time
constexpr int kAttnTcUnit = 128;          // unit of work of the tensor-core kernel: what a block takes at a time

// One sequence of an attention call.
struct AttnSeq {
    int row0;    // its first row of the token axis
    int n;       // its new tokens (query rows)
    int start;   // cache position of the first of them (negative where the length is too short)
    int keys;    // positions that exist: its length, at most what its page table can name
    int lo;      // first position that a query sees, rounded down to a multiple of kAttnSub
    int units;   // units of positions [lo, keys) (one at least, so that empty rows are written)
    int rt;      // tiles of `rows` query rows (new tokens x heads of a K/V head)
    bool falls;  // its offsets fall: the sums over sequences have no bound then, and nothing is done
};

QMM_HD int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// c0, c1: the sequence's entries of the offsets; every value is taken as it comes from device
// memory, so nothing derived from them may leave [0, tokens] and [0, capacity].
QMM_HD AttnSeq attn_seq(int c0, int c1, int len, int tokens, int capacity, int group_heads, int rows, int unit,
                         int window) {
    AttnSeq s;
    s.row0 = clamp_int(c0, 0, tokens);
    s.n = clamp_int(c1, 0, tokens) - s.row0;
    s.falls = c1 < c0;
    if (s.n < 0) s.n = 0;
    if (len < 0) len = 0;
    s.start = len - s.n;
    s.keys = len < capacity ? len : capacity;
    s.lo = 0;
    if (window > 0 && s.start >= window) {  // the first query sees positions from start - window + 1
        s.lo = s.start - window + 1;
        if (s.lo > s.keys) s.lo = s.keys;
        s.lo -= s.lo % kAttnSub;
    }
    s.units = (s.keys - s.lo + unit - 1) / unit;
    if (s.units < 1) s.units = 1;
    s.rt = int((int64_t(s.n) * group_heads + rows - 1) / rows);
    return s;
}

// All units of a sequence: items (K/V head, row tile), row tiles next to one another, each of
// s.units units of positions.  The host bounds the sum over all sequences (of offsets
// that do not fall) below 2^29, and there are at most 2^26 items.
QMM_HD int attn_seq_items(const AttnSeq& s, int kv_heads) { return kv_heads * s.rt; }
QMM_HD int attn_seq_units(const AttnSeq& s, int kv_heads) { return attn_seq_items(s, kv_heads) * s.units; }

QMM_HD int ceil_div_int(int a, int b) { return (a - 1) / b + 1; }  // a >= 1

// How the work is dealt out over `blocks` blocks.  To begin an item costs a block about as much as `start`
// units (its query rows, its sums and their join), so an item weighs its units and that.
// Even shares: block i takes places [i * per, (i + 1) * per) of all items' weights, laid end to end, each
// item's start before its units.  Pieces, where items are few: each item is cut into pieces of `per` units
// (the last one shorter), one a block, so that no block changes items; the pieces are as small as keeps
// their number within the blocks, and give each of a block's warps a unit at least.
struct AttnPlan {
    int total, per, pieces, start;  // weight of all; weight a block (units, in pieces); 1: pieces; an item's start
};
QMM_HD AttnPlan attn_plan(int units, int items, int blocks, int start, int warps) {
    AttnPlan p;
    p.start = start;
    p.total = units + items * p.start;
    p.pieces = 0;
    p.per = p.total < 1 ? 1 : ceil_div_int(p.total, blocks);
    if (units > 0 && items < blocks) {
        int piece = ceil_div_int(units, blocks - items);
        if (piece < warps) piece = warps;
        if (piece <= p.per + p.start / 2) p.pieces = 1, p.per = piece;
    }
    return p;
}

// Weight of a sequence in the order of the blocks: what find_seq adds up.
QMM_HD int attn_seq_weight(const AttnPlan& p, const AttnSeq& s, int kv_heads) {
    return attn_seq_items(s, kv_heads) * (p.pieces ? ceil_div_int(s.units, p.per) : s.units + p.start);
}

// A block's share of an item.  x: the place in the order of the blocks (the block itself, or a place in the
// weights), `before` the weight of the sequences in front.
struct AttnShare {
    int item, u0, n;  // item of the sequence, first unit, units (0: of its start alone)
    int c0, c1;       // the blocks that have units of the item
    int places;       // from x to the end of the share
};
QMM_HD AttnShare attn_share(const AttnPlan& p, const AttnSeq& s, int x, int x_end, int before) {
    AttnShare h;
    const int in = x - before;
    if (p.pieces) {
        const int np = ceil_div_int(s.units, p.per);
        h.item = in / np;
        h.u0 = (in - h.item * np) * p.per;
        h.n = s.units - h.u0 < p.per ? s.units - h.u0 : p.per;
        h.c0 = before + h.item * np;
        h.c1 = h.c0 + np - 1;
        h.places = 1;
    } else {
        const int w = s.units + p.start;
        h.item = in / w;
        const int at = in - h.item * w, end = w - at < x_end - x ? w : at + (x_end - x);
        h.u0 = at > p.start ? at - p.start : 0;
        h.n = end > p.start ? end - p.start - h.u0 : 0;
        const int first = x - at + p.start;  // place of the item's first unit
        h.c0 = first / p.per;
        h.c1 = (first + s.units - 1) / p.per;
        h.places = end - at;
    }
    return h;
}

// Positions [lo, hi) that rows [r0, r1) (row = token * group_heads + head) of a sequence can see.
QMM_HD void attn_range(const AttnSeq& s, int r0, int r1, int group_heads, int window, bool tree, int* lo, int* hi) {
    const int first = s.start + r0 / group_heads, last = s.start + (r1 - 1) / group_heads;
    *hi = tree || last + 1 > s.keys ? s.keys : last + 1 < 0 ? 0 : last + 1;
    *lo = window > 0 && first >= window ? first - window + 1 : 0;
}

// Of n units from position t0 of an item (t0 = its lo + kAttnUnit * first unit), a block's warp w takes
// units w, w + warps, ...: those numbered [j0, j1) of them hold positions in [lo, hi).
QMM_HD void attn_warp_units(int t0, int n, int w, int warps, int lo, int hi, int* j0, int* j1) {
    const int t = t0 + kAttnUnit * w, step = kAttnUnit * warps;
    *j0 = lo > t + kAttnUnit - 1 ? (lo - (t + kAttnUnit - 1) + step - 1) / step : 0;
    int last = hi > t ? (hi - t + step - 1) / step : 0;
    const int mine = n > w ? (n - w + warps - 1) / warps : 0;
    *j1 = last < mine ? last : mine;
}

// A block writes the sums of an item it does not take whole to one of two slots: 2 i + 1 if the item's
// first unit is its own, else 2 i (there are no others: items between are whole).
QMM_HD int attn_slot(int block, int c0) { return 2 * block + (block == c0 ? 1 : 0); }

}  // namespace qmm_impl
