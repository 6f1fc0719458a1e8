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

constexpr int kAttnTile = 16;                        // positions a warp takes at a time
constexpr int kAttnWarps = 4;                        // warps a block
constexpr int kAttnUnit = kAttnTile * kAttnWarps;    // positions a block takes at a time

// One sequence of an attention call.
struct AttnSeq {
    int row0;    // its first row of the token axis
    int n;       // its new tokens (query rows)
    int start;   // cache position of the first of them (negative where the length is too short)
    int keys;    // positions that exist: its length, at most what its page table can name
    int lo;      // first position that a query sees, rounded down to a tile
    int units;   // units of positions [lo, keys) (one at least, so that empty rows are written)
    int rt;      // tiles of `rows` query rows (new tokens x heads of a K/V head)
};

QMM_HD int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// c0, c1: the sequence's entries of the offsets; every value is taken as it comes from device
// memory, so nothing derived from them may leave [0, tokens] and [0, capacity].
QMM_HD AttnSeq attn_seq(int c0, int c1, int len, int tokens, int capacity, int group_heads, int rows, int window) {
    AttnSeq s;
    s.row0 = clamp_int(c0, 0, tokens);
    s.n = clamp_int(c1, 0, tokens) - s.row0;
    if (s.n < 0) s.n = 0;
    if (len < 0) len = 0;
    s.start = len - s.n;
    s.keys = len < capacity ? len : capacity;
    s.lo = 0;
    if (window > 0 && s.start >= window) {  // the first query sees positions from start - window + 1
        s.lo = s.start - window + 1;
        if (s.lo > s.keys) s.lo = s.keys;
        s.lo -= s.lo % kAttnTile;
    }
    s.units = (s.keys - s.lo + kAttnUnit - 1) / kAttnUnit;
    if (s.units < 1) s.units = 1;
    s.rt = int((int64_t(s.n) * group_heads + rows - 1) / rows);
    return s;
}

// All units of a sequence: items (K/V head, row tile), row tiles next to one another, each of
// s.units units of positions.
QMM_HD int64_t attn_seq_units(const AttnSeq& s, int kv_heads) { return int64_t(kv_heads) * s.rt * s.units; }

// Blocks take even, contiguous shares of all units, none of them empty: of `shares` blocks, block i
// takes [attn_share(i), attn_share(i + 1)).
QMM_HD int64_t attn_shares(int64_t total, int64_t blocks) { return total < blocks ? total : blocks; }
QMM_HD int64_t attn_share(int64_t i, int64_t total, int64_t shares) { return i * total / shares; }
// The block that takes unit x.
QMM_HD int attn_owner(int64_t x, int64_t total, int64_t shares) { return int(((x + 1) * shares - 1) / total); }

// Positions [lo, hi) that rows [r0, r1) (row = token * group_heads + head) of a sequence can see.
QMM_HD void attn_range(const AttnSeq& s, int r0, int r1, int group_heads, int window, bool tree, int* lo, int* hi) {
    const int first = s.start + r0 / group_heads, last = s.start + (r1 - 1) / group_heads;
    *hi = tree || last + 1 > s.keys ? s.keys : last + 1 < 0 ? 0 : last + 1;
    *lo = window > 0 && first >= window ? first - window + 1 : 0;
}

// A block writes the partial sums of an item it does not take whole to one of two slots: the
// first item of its share to slot 2i, its last to 2i + 1 (there are no others: those between
// are whole).
QMM_HD int attn_slot(int block, bool first_item) { return 2 * block + (first_item ? 0 : 1); }

}  // namespace qmm_impl
