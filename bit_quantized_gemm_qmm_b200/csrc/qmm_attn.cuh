// qmm_attn.cuh -- what the two kernels of qmm_kv_attention share: the plan of a block's work, rows of
// the output, the join of items that several blocks share.
#pragma once

#include <climits>

#include "qmm_common.cuh"
#include "qmm_internal.h"
#include "qmm_kv_plan.h"

namespace qmm_impl {

constexpr float kNoRef = -3.402823466e38f;  // reference of a query that has seen nothing yet: below every score
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float half_lo(uint32_t v) { return __half2float(__ushort_as_half(uint16_t(v))); }
__device__ __forceinline__ float half_hi(uint32_t v) { return __half2float(__ushort_as_half(uint16_t(v >> 16))); }

// Score sums are in units of 2^-24 (codes are subnormal) times the row's power of two.  Sums of Q over a group
// are raised by 2^17, and with them K's scales: up to 2^15 in fp16, so that three terms of 11 bits are all
// normal numbers (without it the second would be subnormal, and the sum good to 2^-18 only).
constexpr float kSumUp = 131072.f;

// Natural log of l * 2^ref.  l may be far from one: its power of two is added exactly.
__device__ __forceinline__ float lse_of(float ref, float l) {
    if (l == 0.f) return -INFINITY;
    if (!(l < INFINITY)) return l;
    const uint32_t u = __float_as_uint(l);
    return (ref + float(int(u >> 23) - 127) + lg2(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u))) * 0.693147180559945309f;
}

// Four values of an output row: sum / l, rounded once; with the first of them the row's lse.
// A row that saw nothing (l = 0) is zeros and -infinity.
__device__ __forceinline__ void store_row4(const AttnArgs& a, int row, int head, int d, float4 v, float l, float ref) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    uint2 out;
    if (a.is_bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        out = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
        out = make_uint2(f32x2_to_f16x2(v.x, v.y), f32x2_to_f16x2(v.z, v.w));
    }
    *reinterpret_cast<uint2*>(a.o + int64_t(row) * a.o_ts + int64_t(head) * a.o_hs + d) = out;
    if (d == 0 && a.lse != nullptr)
        a.lse[int64_t(row) * (a.kv_heads * a.group_heads) + head] = lse_of(ref, l);
}

// How a kernel cuts the work: query rows a tile, positions a unit, warps that take units of their own, and what
// an item's start costs in units.
struct AttnCut {
    int rows, unit, warps, start;
};

__device__ __forceinline__ AttnSeq load_seq(const AttnArgs& a, int b, AttnCut cut) {
    return attn_seq(a.cu[b], a.cu[b + 1], a.lens[b], a.tokens, a.capacity, a.group_heads, cut.rows, cut.unit, a.window);
}

// Units and items of all sequences; false if offsets fall.
__device__ __forceinline__ bool all_work(const AttnArgs& a, AttnCut cut, int lane, int* units, int* items) {
    int u = 0, n = 0;
    bool falls = false;
    for (int b = lane; b < a.seqs; b += 32) {
        const AttnSeq s = load_seq(a, b, cut);
        falls |= s.falls;
        u += attn_seq_units(s, a.kv_heads);
        n += attn_seq_items(s, a.kv_heads);
    }
    *units = __reduce_add_sync(kFull, u);
    *items = __reduce_add_sync(kFull, n);
    return !__any_sync(kFull, falls);
}

// The sequence in which place x of the running sum of the sequences' weights falls (seqs if past the
// end); *before = the sum of those in front of it.
__device__ __forceinline__ int find_seq(const AttnArgs& a, const AttnPlan& p, AttnCut cut, int x, int lane, int* before) {
    int base = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        const int b = b0 + lane;
        const int w = b < a.seqs ? attn_seq_weight(p, load_seq(a, b, cut), a.kv_heads) : 0;
        int inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += u;
        }
        const unsigned past = __ballot_sync(kFull, base + inc > x);
        if (past) {
            const int l = __ffs(past) - 1;
            *before = base + __shfl_sync(kFull, inc - w, l);
            return b0 + l;
        }
        base += __shfl_sync(kFull, inc, 31);
    }
    return a.seqs;
}

// One block's share of one item.  Kept in shared memory: it is looked at once an item.
struct Run {
    int row0, start, keys, units;  // of the sequence (AttnSeq)
    int b, h;          // sequence, K/V head
    int u0, n;         // first unit of the item, units
    int row_lo, rows;  // first query row (of the sequence) and how many
    int lo, hi;        // positions that some row sees
    int full_lo, full_hi;  // positions [full_lo, full_hi) that every row sees
    int t0;            // position of the first unit
    int places;        // from x to the end of this share
    int c0, c1;        // the blocks that share the item
    int x, before;     // place in the order of the blocks; weight of the sequences in front of b
};
static_assert(sizeof(Run) <= 96, "Run does not fit its place");


// The next run with units at or behind place x of the order of the blocks, in or after sequence b: written
// by `writer` to *r.  False if the block's share has none (then r->n is 0); *bad if the table cannot name
// all of the sequence's positions.
__device__ __forceinline__ bool plan_run(const AttnArgs& a, const AttnPlan& pl, AttnCut cut, int x, int x_end, int b,
                                         int before, bool writer, Run* r, bool* bad) {
    AttnSeq s;
    AttnShare sh;
    sh.n = 0;
    if (x < x_end) s = load_seq(a, b, cut);
    while (x < x_end) {
        const int weight = attn_seq_weight(pl, s, a.kv_heads);
        if (x >= before + weight) {
            before += weight;
            s = load_seq(a, ++b, cut);
            continue;
        }
        sh = attn_share(pl, s, x, x_end, before);
        if (sh.n > 0) break;
        x += sh.places;  // only the start of an item: its units are the next block's
    }
    if (sh.n == 0) {
        if (writer) r->n = 0;
        return false;
    }
    const int h = sh.item / s.rt, row_lo = (sh.item - h * s.rt) * cut.rows, nrows = s.n * a.group_heads;
    const int rows = nrows - row_lo < cut.rows ? nrows - row_lo : cut.rows;
    const int first = s.start + row_lo / a.group_heads, last = s.start + (row_lo + rows - 1) / a.group_heads;
    int lo, hi;
    attn_range(s, row_lo, row_lo + rows, a.group_heads, a.window, a.tree != nullptr, &lo, &hi);
    if (writer) {
        r->row0 = s.row0, r->start = s.start, r->keys = s.keys, r->units = s.units;
        r->b = b, r->h = h, r->u0 = sh.u0, r->n = sh.n;
        r->row_lo = row_lo, r->rows = rows, r->lo = lo, r->hi = hi;
        const int all = a.tree ? s.start : first + 1;
        r->full_hi = all < s.keys ? all : s.keys;
        r->full_lo = a.window > 0 && last >= a.window ? last - a.window + 1 : 0;
        r->t0 = s.lo + cut.unit * sh.u0;
        r->c0 = sh.c0, r->c1 = sh.c1, r->x = x, r->places = sh.places, r->before = before;
    }
    *bad |= s.start + s.n > a.capacity;
    return true;
}

// The block's place in the work: its first run and the end of its share.  0: it has none; 1: go on;
// -1: the offsets fall, and nothing is done.
__device__ __forceinline__ int plan_block(const AttnArgs& a, AttnCut cut, int lane, bool writer, AttnPlan* pl, int* x_end,
                                          Run* r, bool* bad) {
    int units, items, before = 0;
    if (!all_work(a, cut, lane, &units, &items)) return -1;
    *pl = attn_plan(units, items, gridDim.x, cut.start, cut.warps);
    const int x = pl->pieces ? int(blockIdx.x) : int(blockIdx.x) * pl->per;
    *x_end = pl->pieces ? x + 1 : x + pl->per < pl->total ? x + pl->per : pl->total;
    const int b = find_seq(a, *pl, cut, x, lane, &before);
    return b < a.seqs && plan_run(a, *pl, cut, x, *x_end, b, before, writer, r, bad) ? 1 : 0;
}

// Joins the sums of an item that several blocks share (all of a block's threads call it, with its own sums
// written to its slot).  Eight neighbouring blocks' sums are added by the last of them to arrive, eight such
// results by the last of those, and so on: always in block order, and each step reads its slots in one
// round (55 blocks of a 128k-position sequence: 2 steps; one block adding all of them took 7 rounds).  A
// slot is [ROWS][D] sums, the rows' references and their l; a step's result goes to its first block's.
template <int D, int ROWS>
__device__ __forceinline__ void join_item(const AttnArgs& a, const Run* cur, int tid, int threads, int* flag) {
    const int c0 = cur->c0, n = cur->c1 - c0 + 1;
    int me = int(blockIdx.x) - c0;
    auto slot_of = [&](int i) { return a.part + int64_t(attn_slot(c0 + i, c0)) * (ROWS * (D + 2)); };
    for (int span = 1, level = 0;; span *= 8, ++level) {
        me -= me % (8 * span);  // the first of the eight
        const int left = (n - me + span - 1) / span, members = left < 8 ? left : 8;
        if (members > 1) {
            __threadfence();
            __syncthreads();
            if (tid == 0)  // wraps to 0
                *flag = atomicInc(a.count + level * kArrivalBlocks + c0 + me, unsigned(members - 1)) == unsigned(members - 1);
            __syncthreads();
            if (!*flag) return;
            __threadfence();
        }
        const bool last = 8 * span >= n;
        if (members > 1 || last) {
            for (int i = tid; i < cur->rows * (D / 4); i += threads) {
                const int row = i / (D / 4), d = i % (D / 4) * 4;
                float4 v[8];
                float rf[8], ll[8], top = kNoRef;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const bool on = k < members;
                    const float* from = slot_of(on ? me + k * span : me);
                    rf[k] = on ? __ldcg(from + ROWS * D + row) : kNoRef;
                    ll[k] = on ? __ldcg(from + ROWS * D + ROWS + row) : 0.f;
                    v[k] = on ? __ldcg(reinterpret_cast<const float4*>(from + row * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, rf[k]);
                float lsum = 0.f;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = ex2(rf[k] - top);
                    sum.x = fmaf(f, v[k].x, sum.x), sum.y = fmaf(f, v[k].y, sum.y);
                    sum.z = fmaf(f, v[k].z, sum.z), sum.w = fmaf(f, v[k].w, sum.w);
                    lsum = fmaf(f, ll[k], lsum);
                }
                if (last) {
                    const int qr = cur->row_lo + row, tok = qr / a.group_heads;
                    store_row4(a, cur->row0 + tok, cur->h * a.group_heads + qr - tok * a.group_heads, d, sum, lsum, top);
                } else {
                    __stcg(reinterpret_cast<float4*>(slot_of(me) + row * D + d), sum);
                }
            }
        }
        if (last) return;
        if (members > 1) {  // the rows' constants, once nobody reads the old ones
            __syncthreads();
            for (int row = tid; row < cur->rows; row += threads) {
                float rf[8], top = kNoRef, lsum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) rf[k] = k < members ? __ldcg(slot_of(me + k * span) + ROWS * D + row) : kNoRef;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, rf[k]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < members) lsum = fmaf(ex2(rf[k] - top), __ldcg(slot_of(me + k * span) + ROWS * D + ROWS + row), lsum);
                __stcg(slot_of(me) + ROWS * D + row, top);
                __stcg(slot_of(me) + ROWS * D + ROWS + row, lsum);
            }
        }
    }
}

// per_sm blocks for each of the device's SMs; allows the kernel its shared memory, once per device and kernel.
// regs: registers a thread that the kernel must have been built with (it shares them out anew), or 0.
cudaError_t attn_blocks(void (*fn)(const AttnArgs), int smem, int per_sm, int regs, int* out);
// Launches a kernel over the resident blocks, with its workspace.
cudaError_t launch_attn_blocks(AttnArgs a, void (*fn)(const AttnArgs), int threads, int smem, int slot, int rows, int unit,
                               int per_sm, int regs, cudaStream_t stream);
// The tensor-core kernel (qmm_attn_tc.cu).  query_rows: about how many a sequence and K/V head have.
bool attn_tc_supported(int head_dim);
cudaError_t launch_attn_tc(const AttnArgs& a, int query_rows, int head_dim, int group, cudaStream_t stream);
cudaError_t attn_tc_read_and_clear_errors(unsigned* out);

}  // namespace qmm_impl
