// qmm_attn.cu -- attention over a paged 4-bit K/V cache (qmm_kv_attention).
//
//   x[r, t] = scale * sum_d q[r, d] * (s_t q_td + b_t)      (affine K row t, group scales s, b)
//   o[r]    = sum_t softmax(x[r])_t * (s'_t q'_t + b'_t)     (affine V row t)
//
// Rows r of one tile are the (new token, query head) pairs that share a K/V head, so every
// cache byte is read once for all of them.  The codes enter the MMA as they are: a nibble in
// the low bits of an fp16 is the subnormal q * 2^-24 (one AND a pair, exact), one place up it
// is q * 2^-20, and the factor 16 between them is put into Q (for K) or into the output rows
// (for V).  Both products run with the codes as the 16-row operand and 8 query rows as the
// 8-column one (mma.sync m16n8k16):
//   - K: ldmatrix gives lane (g, c) word c of row g, whose nibble pairs are two k indices; the
//     group's fp32 sums are scaled by s afterwards, b enters as b * sum(Q over the group).
//   - V: ldmatrix.trans on the 16-bit units (four codes) of the rows gives lane (g, c) the unit
//     g of rows 2c and 2c + 1 in one register, whose nibble pairs are two positions (k) of one
//     d (row).  V's codes are centred (q - 8, one packed add a pair), and each group's P * s is
//     rounded once to fp16: with centred codes that rounding weighs in with the spread of V and
//     not with its distance from the bias.  b + 8s enters through fp32 sums of P * (b + 8s).
// The scores' layout (position by query) is the transpose of the second product's operand;
// movmatrix turns the packed P * s round.
//
// Softmax: each warp keeps a reference per query, not the maximum: x - ref goes through ex2 and
// the sums are rescaled only when some P * s reaches 2 (one OR over the packed values: the sign
// of a large or NaN fp16 is bit 14) or x - ref reaches 60.  The reference is then put so that
// the largest P * s of the tile is 2^-4.
//
// Work: units of 64 positions of one (sequence, K/V head, row tile) are dealt out evenly over
// the resident blocks (qmm_kv_plan.h), whatever the lengths; a warp streams 16-position tiles of
// its block's share through its own cp.async ring.  Items that several blocks share are summed
// by a second small kernel in block order, so results do not depend on timing.
#include <climits>
#include <mutex>
#include <type_traits>
#include <unordered_map>

#include "qmm_common.cuh"
#include "qmm_internal.h"
#include "qmm_kv_plan.h"
#include "sm100.cuh"

namespace qmm_impl {
namespace {

__device__ unsigned g_attn_errors;  // bit 1: a page or position outside the cache

constexpr float kNoRef = -1e30f;  // reference of a query that has seen nothing yet
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
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t saddr, uint32_t (&d)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(saddr));
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t hadd2_bits(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float half_lo(uint32_t v) { return __half2float(__ushort_as_half(uint16_t(v))); }
__device__ __forceinline__ float half_hi(uint32_t v) { return __half2float(__ushort_as_half(uint16_t(v >> 16))); }

// NG fp16 values of one row from shared memory, as floats.
template <int NG>
__device__ __forceinline__ void lds_halves(uint32_t addr, float (&f)[NG]) {
    if constexpr (NG == 1) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
        f[0] = half_lo(v);
    } else if constexpr (NG == 2) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
        f[0] = half_lo(v), f[1] = half_hi(v);
    } else {
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            uint32_t v, w;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v), "=r"(w) : "r"(addr + 8 * i));
            f[4 * i] = half_lo(v), f[4 * i + 1] = half_hi(v), f[4 * i + 2] = half_lo(w), f[4 * i + 3] = half_hi(w);
        }
    }
}

// Shared-memory layout of an instance: per warp a ring of tiles (reused for the warp's partial
// sums at the end of an item), then Q as MMA fragments and the rows' constants.
template <int D, int GRP, int NT>
struct AttnFmt {
    static constexpr int NG = D / GRP;
    static constexpr int CH = D / 32;              // 16-byte pieces (32 codes) of a row
    static constexpr int ROWS = 8 * NT;
    static constexpr int CODES = kAttnTile * D / 2;  // bytes of a tile's K (or V) codes
    static constexpr int SB = kAttnTile * NG * 2;    // bytes of a tile's K scales (or biases, V's)
    static constexpr int TILE = 2 * CODES + 4 * SB;
    static constexpr int RING = D == 256 ? 3 : 4;
    static constexpr int OROW = D + 4;             // floats between rows of the partial sums
    static constexpr int MERGE = ROWS * OROW * 4 + ROWS * 8;
    static constexpr int WARP = RING * TILE > MERGE ? RING * TILE : (MERGE + 127) / 128 * 128;
    static constexpr int QF = ROWS * D * 2;        // Q fragments
    static constexpr int OFF_Q = kAttnWarps * WARP;
    static constexpr int OFF_F = OFF_Q + QF;       // float per row: factor of the code sums
    static constexpr int OFF_QB = OFF_F + ROWS * 4;       // float per row and group: factor of b
    static constexpr int OFF_LIM = OFF_QB + ROWS * NG * 4;  // int per row: last position seen
    static constexpr int OFF_BITS = (OFF_LIM + ROWS * 4 + 7) / 8 * 8;  // 64-bit mask per row
    static constexpr int SMEM = OFF_BITS + ROWS * 8;
    static constexpr int SLOT = ROWS * (D + 2);    // floats of one partial-sum slot
};

__device__ __forceinline__ AttnSeq load_seq(const AttnArgs& a, int b, int rows) {
    return attn_seq(a.cu[b], a.cu[b + 1], a.lens[b], a.tokens, a.capacity, a.group_heads, rows, a.window);
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
        a.lse[int64_t(row) * (a.kv_heads * a.group_heads) + head] =
            l == 0.f ? -INFINITY : (ref + lg2(l)) * 0.693147180559945309f;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ int64_t all_units(const AttnArgs& a, int rows, int lane) {
    int64_t sum = 0;
    for (int b = lane; b < a.seqs; b += 32) sum += attn_seq_units(load_seq(a, b, rows), a.kv_heads);
    return warp_sum64(sum);
}

// The sequence in which position x of the running sum of `weight` falls; *before = the sum of
// those in front of it.
template <class F>
__device__ __forceinline__ int find_seq(int seqs, int64_t x, int lane, int64_t* before, F weight) {
    int64_t base = 0;
    for (int b0 = 0; b0 < seqs; b0 += 32) {
        const int b = b0 + lane;
        const int64_t w = b < seqs ? weight(b) : 0;
        int64_t inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(kFull, inc, o);
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
    *before = base;
    return seqs;
}

// One block's share of one item, and what its warps need of it.
struct Run {
    int b, h, rt;      // sequence, K/V head, row tile
    int u0, n;         // first unit of the item, units
    int row_lo, rows;  // first query row (of the sequence) and how many
    int lo, hi;        // positions that some row sees
    int full_lo, full_hi;  // positions [full_lo, full_hi) that every row sees
};

template <int D, int GRP, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, NT == 1 && D <= 128 ? 4 : D == 256 && NT == 2 ? 2 : NT == 4 ? 2 : 3)
    attn_kernel(const __grid_constant__ AttnArgs a) {
    using F = AttnFmt<D, GRP, NT>;
    constexpr int NG = F::NG, CH = F::CH, R = F::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t ring = sbase + w * F::WARP;

    grid_dependency_wait();
    grid_dependents_launch();

    const int64_t total = all_units(a, R, lane);
    const int64_t shares = attn_shares(total, gridDim.x);
    if (blockIdx.x >= shares) return;
    int64_t x = attn_share(blockIdx.x, total, shares);
    const int64_t x_end = attn_share(int64_t(blockIdx.x) + 1, total, shares);
    int64_t before;
    int b = find_seq(a.seqs, x, lane, &before, [&](int i) { return attn_seq_units(load_seq(a, i, R), a.kv_heads); });

    // per-lane constants of the tile copies: codes (16-byte piece i of a tile goes to row i / CH,
    // piece i % CH, xor-swizzled so that eight rows' equal pieces fall into different banks)
    auto swz = [](int row, int ch) { return row * (D / 2) + ((ch ^ ((row * (D / 2) >> 7) & (CH - 1))) << 4); };
    constexpr int CPT = kAttnTile * CH / 32;  // 16-byte pieces of codes a lane copies, K and V each
    constexpr int SPT = (8 * NG + 31) / 32;   // of scales and biases
    bool first_item = true;
    bool bad = false;

    while (x < x_end) {
        // ---- the item and this block's part of it
        const AttnSeq s = load_seq(a, b, R);
        const int64_t wb = attn_seq_units(s, a.kv_heads);
        if (x >= before + wb) {
            before += wb;
            ++b;
            continue;
        }
        Run r;
        const int64_t in = x - before;
        const int item = int(in / s.units);
        r.u0 = int(in - int64_t(item) * s.units);
        r.n = int(x_end - x < s.units - r.u0 ? x_end - x : s.units - r.u0);
        r.b = b;
        r.h = item / s.rt;
        r.rt = item - r.h * s.rt;
        r.row_lo = r.rt * R;
        const int nrows = s.n * a.group_heads;
        r.rows = nrows - r.row_lo < R ? nrows - r.row_lo : R;
        attn_range(s, r.row_lo, r.row_lo + r.rows, a.group_heads, a.window, a.tree != nullptr, &r.lo, &r.hi);
        {
            const int first = s.start + r.row_lo / a.group_heads;
            const int last = s.start + (r.row_lo + r.rows - 1) / a.group_heads;
            r.full_hi = a.tree ? s.start : first + 1;
            if (r.full_hi > s.keys) r.full_hi = s.keys;
            r.full_lo = a.window > 0 && last >= a.window ? last - a.window + 1 : 0;
        }
        if (s.start + s.n > a.capacity) bad = true;  // the table cannot name all of its positions
        const bool whole = r.n == s.units;

        // ---- Q: fragments in shared memory, scaled by a power of two per row
        for (int i = tid; i < R * (D / 8); i += 32 * kAttnWarps) {
            const int row = i / (D / 8), p8 = i % (D / 8);  // eight values from 8 * p8
            float v[8];
            const int qr = r.row_lo + row, tok = qr / a.group_heads, hg = qr - tok * a.group_heads;
            if (row < r.rows) {
                const uint16_t* src = a.q + int64_t(s.row0 + tok) * a.q_ts + int64_t(r.h * a.group_heads + hg) * a.q_hs + p8 * 8;
                uint32_t raw[4];
                if (a.q_vec) {
                    const uint4 u = *reinterpret_cast<const uint4*>(src);
                    raw[0] = u.x, raw[1] = u.y, raw[2] = u.z, raw[3] = u.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) raw[j] = uint32_t(src[2 * j]) | uint32_t(src[2 * j + 1]) << 16;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = a.is_bf16 ? bf16lo_to_f32(raw[j]) : half_lo(raw[j]);
                    v[2 * j + 1] = a.is_bf16 ? bf16hi_to_f32(raw[j]) : half_hi(raw[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.f;
            }
            float mx = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[j])), sum += v[j];
#pragma unroll
            for (int o = 1; o < D / 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
#pragma unroll
            for (int o = 1; o < GRP / 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
            // exponent e with max * 2^e in [2^14, 2^15); rows of zeros, infinities or NaN: 0
            int e = 0;
            if (mx > 0.f && mx < INFINITY) e = 14 + 127 - int(__float_as_uint(mx) >> 23);
            if (e > 126) e = 126;  // subnormal rows
            const float up = exp2i(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= up;
            // nibbles 0, 2 of a pair's place are codes * 2^-24, nibbles 1, 3 codes * 2^-20
            uint4 f;
            f.x = f32x2_to_f16x2(v[0], v[4]);
            f.y = f32x2_to_f16x2(v[2], v[6]);
            f.z = f32x2_to_f16x2(v[1] * 0.0625f, v[5] * 0.0625f);
            f.w = f32x2_to_f16x2(v[3] * 0.0625f, v[7] * 0.0625f);
            const int nt = row >> 3, ch = p8 >> 2, ln = (row & 7) * 4 + (p8 & 3);
            sts_v4(sbase + F::OFF_Q + ((nt * CH + ch) * 32 + ln) * 16, f);
            if (p8 % (GRP / 8) == 0)
                *reinterpret_cast<float*>(smem + F::OFF_QB + (row * NG + p8 / (GRP / 8)) * 4) = sum * a.scale_log2;
            if (p8 == 0) {
                // 2^24 * 2^-e in two exact steps (e may be as low as -113)
                *reinterpret_cast<float*>(smem + F::OFF_F + row * 4) = a.scale_log2 * 16777216.f * exp2i(-e);
                *reinterpret_cast<int*>(smem + F::OFF_LIM + row * 4) = row < r.rows ? s.start + tok : INT_MAX;
                *reinterpret_cast<int64_t*>(smem + F::OFF_BITS + row * 8) =
                    a.tree != nullptr && row < r.rows ? a.tree[s.row0 + tok] : -1;
            }
        }
        __syncthreads();

        float qf[NT][2], qb[NT][2][NG];
        uint4 qreg[NT == 1 ? CH : 1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = nt * 8 + 2 * c + k;
                qf[nt][k] = *reinterpret_cast<const float*>(smem + F::OFF_F + row * 4);
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    qb[nt][k][j] = *reinterpret_cast<const float*>(smem + F::OFF_QB + (row * NG + j) * 4);
            }
        if constexpr (NT == 1) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) qreg[ch] = lds_v4(sbase + F::OFF_Q + (ch * 32 + lane) * 16);
        }

        // ---- this warp's tiles: positions t0 + 64 j, j in [j0, j1)
        const int t0 = s.lo + kAttnUnit * r.u0 + kAttnTile * w;
        int j0 = r.lo > t0 + kAttnTile - 1 ? (r.lo - (t0 + kAttnTile - 1) + kAttnUnit - 1) / kAttnUnit : 0;
        int j1 = r.hi > t0 ? (r.hi - t0 + kAttnUnit - 1) / kAttnUnit : 0;
        if (j1 > r.n) j1 = r.n;
        const int32_t* table = a.table + int64_t(b) * a.table_stride;
        auto page_of = [&](int j) { return j < j1 ? table[(t0 + kAttnUnit * j) / a.page] : -1; };
        int idb = j0, ids = page_of(j0 + lane), ids_next = page_of(j0 + 32 + lane);
        uint32_t live = 0;  // bit per ring slot: the tile there was copied

        auto issue = [&](int j, int slot) {
            if (j < j1) {
                if (j - idb == 32) {
                    idb = j;
                    ids = ids_next;
                    ids_next = page_of(j + 32 + lane);
                }
                const int page = __shfl_sync(kFull, ids, j - idb);
                if (page >= 0 && page < a.pages) {
                    live |= 1u << slot;
                    const int t = t0 + kAttnUnit * j;
                    const int64_t row = (int64_t(page) * a.kv_heads + r.h) * a.page + t % a.page;
                    const uint32_t dst = ring + slot * F::TILE;
                    const uint8_t* ksrc = a.kc + row * (D / 2) + lane * 16;
                    const uint8_t* vsrc = a.vc + row * (D / 2) + lane * 16;
#pragma unroll
                    for (int i = 0; i < CPT; ++i) {
                        const int piece = i * 32 + lane;
                        const uint32_t o = swz(piece / CH, piece % CH);
                        cp_async_16(dst + o, ksrc + i * 512);
                        cp_async_16(dst + F::CODES + o, vsrc + i * 512);
                    }
#pragma unroll
                    for (int i = 0; i < SPT; ++i) {
                        const int piece = i * 32 + lane;
                        if (8 * NG % 32 == 0 || piece < 8 * NG) {
                            const int arr = piece / (2 * NG), at = piece % (2 * NG);
                            const uint8_t* base = reinterpret_cast<const uint8_t*>(
                                arr == 0 ? a.ks : arr == 1 ? a.kb : arr == 2 ? a.vs : a.vb);
                            cp_async_16(dst + 2 * F::CODES + piece * 16, base + row * (NG * 2) + at * 16);
                        }
                    }
                } else {
                    live &= ~(1u << slot);
                    bad = true;
                }
            }
            sm100::cp_async_commit();
        };

        // sums, relative to the queries' references
        float ref[NT][2], l[NT][2], bs[NT][2][NG], o[NT][CH][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ref[nt][k] = kNoRef, l[nt][k] = 0.f;
#pragma unroll
                for (int j = 0; j < NG; ++j) bs[nt][k][j] = 0.f;
            }
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][ch][m][i] = 0.f;
        }

        auto tile = [&](int t, uint32_t st, auto masked_c) {
            constexpr bool MASKED = decltype(masked_c)::value;
            // which of this lane's (position, query) pairs are seen
            uint32_t see = 0xFFFFFFFFu;
            bool in0 = true, in1 = true;
            if constexpr (MASKED) {
                in0 = t + g < s.keys, in1 = t + g + 8 < s.keys;
                see = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = nt * 8 + 2 * c + (i & 1), p = t + g + (i >> 1) * 8;
                        bool ok;
                        if (a.tree != nullptr) {
                            const int64_t bits = *reinterpret_cast<const int64_t*>(smem + F::OFF_BITS + row * 8);
                            const int d = p - s.start;
                            ok = d < 0 || (d < 64 && ((bits >> d) & 1));
                        } else {
                            const int lim = *reinterpret_cast<const int*>(smem + F::OFF_LIM + row * 4);
                            ok = p <= lim && (a.window <= 0 || lim == INT_MAX || p > lim - a.window);
                        }
                        if (ok && p < s.keys) see |= 1u << (nt * 4 + i);
                    }
            }
            // ---- scores: code sums per group, scaled
            float acc[NT][4];
            float bias[NT][4];
            {
                float ks0[NG], ks1[NG], kb0[NG], kb1[NG];
                const uint32_t sb = st + 2 * F::CODES + g * (2 * NG);
                lds_halves<NG>(sb, ks0);
                lds_halves<NG>(sb + 16 * NG, ks1);
                lds_halves<NG>(sb + F::SB, kb0);
                lds_halves<NG>(sb + F::SB + 16 * NG, kb1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bias[nt][i] = 0.f;
#pragma unroll
                        for (int j = 0; j < NG; ++j)
                            bias[nt][i] = fmaf(i < 2 ? kb0[j] : kb1[j], qb[nt][i & 1][j], bias[nt][i]);
                        acc[nt][i] = 0.f;
                    }
                float part[NT][4];
                uint32_t kw[4];
                const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    if (ch % 2 == 0) ldsm_x4(st + swz(krow, ch + (lane >> 4)), kw);
                    const uint32_t w0 = kw[2 * (ch & 1)], w1 = kw[2 * (ch & 1) + 1];
                    const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
                    const uint32_t e0 = w0 & 0x000F000Fu, e1 = w1 & 0x000F000Fu, e2 = h0 & 0x000F000Fu, e3 = h1 & 0x000F000Fu;
                    const uint32_t f0 = w0 & 0x00F000F0u, f1 = w1 & 0x00F000F0u, f2 = h0 & 0x00F000F0u, f3 = h1 & 0x00F000F0u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 q = NT == 1 ? qreg[NT == 1 ? ch : 0] : lds_v4(sbase + F::OFF_Q + ((nt * CH + ch) * 32 + lane) * 16);
                        if (ch * 32 % GRP == 0) mma_16816_z(part[nt], e0, e1, e2, e3, q.x, q.y);
                        else mma_16816(part[nt], e0, e1, e2, e3, q.x, q.y);
                        mma_16816(part[nt], f0, f1, f2, f3, q.z, q.w);
                    }
                    if ((ch + 1) * 32 % GRP == 0) {
                        const int j = ch * 32 / GRP;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[nt][i] = fmaf(i < 2 ? ks0[j] : ks1[j], part[nt][i], acc[nt][i]);
                    }
                }
            }
            // ---- probabilities, V's scales applied, packed for the second product
            float vs0[NG], vs1[NG], vb0[NG], vb1[NG];
            {
                const uint32_t sb = st + 2 * F::CODES + 2 * F::SB + g * (2 * NG);
                lds_halves<NG>(sb, vs0);
                lds_halves<NG>(sb + 16 * NG, vs1);
                lds_halves<NG>(sb + F::SB, vb0);
                lds_halves<NG>(sb + F::SB + 16 * NG, vb1);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    if constexpr (MASKED) {
                        if (!in0) vs0[j] = vb0[j] = 0.f;
                        if (!in1) vs1[j] = vb1[j] = 0.f;
                    }
                    vb0[j] = fmaf(8.f, vs0[j], vb0[j]);
                    vb1[j] = fmaf(8.f, vs1[j], vb1[j]);
                }
            }
            float p[NT][4];
            uint32_t pk[NT][NG][2];
            auto probabilities = [&]() -> bool {
                uint32_t any = 0;
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float xv = fmaf(qf[nt][i & 1], acc[nt][i], bias[nt][i] - ref[nt][i & 1]);
                        if (MASKED && !((see >> (nt * 4 + i)) & 1)) xv = -INFINITY;
                        top = fmaxf(top, xv);
                        p[nt][i] = ex2(xv);
                    }
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        float m0 = p[nt][0] * vs0[j], m1 = p[nt][1] * vs0[j], m2 = p[nt][2] * vs1[j], m3 = p[nt][3] * vs1[j];
                        if constexpr (MASKED) {
                            if (!((see >> (nt * 4)) & 1)) m0 = 0.f;
                            if (!((see >> (nt * 4 + 1)) & 1)) m1 = 0.f;
                            if (!((see >> (nt * 4 + 2)) & 1)) m2 = 0.f;
                            if (!((see >> (nt * 4 + 3)) & 1)) m3 = 0.f;
                        }
                        pk[nt][j][0] = f32x2_to_f16x2(m0, m1);
                        pk[nt][j][1] = f32x2_to_f16x2(m2, m3);
                        any |= pk[nt][j][0] | pk[nt][j][1];
                    }
                }
                return (any & 0x40004000u) != 0 || top > 60.f;
            };
            if (__any_sync(kFull, probabilities())) {
                // new references from this tile: the largest P * s becomes 2^-4 (and P at most 2^20)
                float sg0 = 0.f, sg1 = 0.f;
#pragma unroll
                for (int j = 0; j < NG; ++j) sg0 = fmaxf(sg0, fabsf(vs0[j])), sg1 = fmaxf(sg1, fabsf(vs1[j]));
                const float l0 = lg2(sg0), l1 = lg2(sg1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float m = -INFINITY;
#pragma unroll
                        for (int i = k; i < 4; i += 2) {
                            const float sc = fmaf(qf[nt][k], acc[nt][i], bias[nt][i]);
                            const float v = fmaxf(sc + (i < 2 ? l0 : l1) + 4.f, sc - 20.f);
                            if (!MASKED || ((see >> (nt * 4 + i)) & 1)) m = fmaxf(m, v);
                        }
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
                        const float nr = fmaxf(ref[nt][k], m);
                        const float f = ex2(ref[nt][k] - nr);
                        ref[nt][k] = nr;
                        l[nt][k] *= f;
#pragma unroll
                        for (int j = 0; j < NG; ++j) bs[nt][k][j] *= f;
#pragma unroll
                        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                            for (int mm = 0; mm < 2; ++mm) o[nt][ch][mm][k] *= f, o[nt][ch][mm][k + 2] *= f;
                    }
                probabilities();
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                l[nt][0] += p[nt][0] + p[nt][2];
                l[nt][1] += p[nt][1] + p[nt][3];
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    if constexpr (MASKED) {
                        bs[nt][0][j] += ((see >> (nt * 4)) & 1) ? p[nt][0] * vb0[j] : 0.f;
                        bs[nt][1][j] += ((see >> (nt * 4 + 1)) & 1) ? p[nt][1] * vb0[j] : 0.f;
                        bs[nt][0][j] += ((see >> (nt * 4 + 2)) & 1) ? p[nt][2] * vb1[j] : 0.f;
                        bs[nt][1][j] += ((see >> (nt * 4 + 3)) & 1) ? p[nt][3] * vb1[j] : 0.f;
                    } else {
                        bs[nt][0][j] = fmaf(p[nt][2], vb1[j], fmaf(p[nt][0], vb0[j], bs[nt][0][j]));
                        bs[nt][1][j] = fmaf(p[nt][3], vb1[j], fmaf(p[nt][1], vb0[j], bs[nt][1][j]));
                    }
                    pk[nt][j][0] = movmatrix_trans(pk[nt][j][0]);
                    pk[nt][j][1] = movmatrix_trans(pk[nt][j][1]);
                }
            }
            // ---- sums over V: rows d = 32 ch + 4 g + {m, m + 2}
            uint32_t vw[4];
            const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                if (ch % 2 == 0) ldsm_x4_trans(st + F::CODES + swz(vrow, ch + (lane >> 4)), vw);
                const uint32_t w0 = vw[2 * (ch & 1)], w1 = vw[2 * (ch & 1) + 1];
                const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
                constexpr uint32_t m8 = 0x80088008u, m80 = 0x80808080u;  // -8 * 2^-24, -8 * 2^-20
                const uint32_t e0 = hadd2_bits(w0 & 0x000F000Fu, m8), e1 = hadd2_bits(h0 & 0x000F000Fu, m8);
                const uint32_t e2 = hadd2_bits(w1 & 0x000F000Fu, m8), e3 = hadd2_bits(h1 & 0x000F000Fu, m8);
                const uint32_t f0 = hadd2_bits(w0 & 0x00F000F0u, m80), f1 = hadd2_bits(h0 & 0x00F000F0u, m80);
                const uint32_t f2 = hadd2_bits(w1 & 0x00F000F0u, m80), f3 = hadd2_bits(h1 & 0x00F000F0u, m80);
                const int j = ch * 32 / GRP;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(o[nt][ch][0], e0, e1, e2, e3, pk[nt][j][0], pk[nt][j][1]);
                    mma_16816(o[nt][ch][1], f0, f1, f2, f3, pk[nt][j][0], pk[nt][j][1]);
                }
            }
        };

        // ---- stream the tiles
#pragma unroll
        for (int i = 0; i < F::RING - 1; ++i) issue(j0 + i, i);
        int slot = 0;
        for (int j = j0; j < j1; ++j) {
            sm100::cp_async_wait<F::RING - 2>();
            __syncwarp();
            issue(j + F::RING - 1, slot == 0 ? F::RING - 1 : slot - 1);
            const int t = t0 + kAttnUnit * j;
            if ((live >> slot) & 1) {
                if (t >= r.full_lo && t + kAttnTile <= r.full_hi) tile(t, ring + slot * F::TILE, std::false_type{});
                else tile(t, ring + slot * F::TILE, std::true_type{});
            }
            slot = slot == F::RING - 1 ? 0 : slot + 1;
        }
        sm100::cp_async_wait<0>();
        __syncwarp();

        // ---- the warp's sums to shared memory (its own, drained ring)
        float* mo = reinterpret_cast<float*>(smem + w * F::WARP);
        float* ml = mo + R * F::OROW;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[nt][k] += __shfl_xor_sync(kFull, l[nt][k], off);
#pragma unroll
                    for (int j = 0; j < NG; ++j) bs[nt][k][j] += __shfl_xor_sync(kFull, bs[nt][k][j], off);
                }
                const int row = nt * 8 + 2 * c + k;
                if (g == 0) ml[row] = ref[nt][k], ml[R + row] = l[nt][k];
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    const float bb = bs[nt][k][ch * 32 / GRP];
                    float4 v;
                    v.x = fmaf(o[nt][ch][0][k], 16777216.f, bb);
                    v.y = fmaf(o[nt][ch][1][k], 1048576.f, bb);
                    v.z = fmaf(o[nt][ch][0][k + 2], 16777216.f, bb);
                    v.w = fmaf(o[nt][ch][1][k + 2], 1048576.f, bb);
                    *reinterpret_cast<float4*>(mo + row * F::OROW + 32 * ch + 4 * g) = v;
                }
            }
        __syncthreads();
        // ---- the block's sums: to the output, or to this block's slot of the workspace
        float* slot_o = a.part + int64_t(attn_slot(blockIdx.x, first_item)) * F::SLOT;
        for (int i = tid; i < r.rows * (D / 4); i += 32 * kAttnWarps) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float rf[kAttnWarps], top = kNoRef;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                rf[k] = reinterpret_cast<const float*>(smem + k * F::WARP)[R * F::OROW + row];
                top = fmaxf(top, rf[k]);
            }
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float lsum = 0.f;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                const float* from = reinterpret_cast<const float*>(smem + k * F::WARP);
                const float f = ex2(rf[k] - top);
                const float4 v = *reinterpret_cast<const float4*>(from + row * F::OROW + d);
                sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
                sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
                lsum = fmaf(f, from[R * F::OROW + R + row], lsum);
            }
            if (whole) {
                const int qr = r.row_lo + row, tok = qr / a.group_heads;
                const int head = r.h * a.group_heads + qr - tok * a.group_heads;
                store_row4(a, s.row0 + tok, head, d, sum, lsum, top);
            } else {
                *reinterpret_cast<float4*>(slot_o + row * D + d) = sum;
                if (d == 0) slot_o[R * D + row] = top, slot_o[R * D + R + row] = lsum;
            }
        }
        __syncthreads();
        x += r.n;
        first_item = false;
    }
    if (bad && lane == 0) atomicOr(&g_attn_errors, 2u);
}

// Sums the items that several blocks shared: one block a (item, row), its warps over the
// partial sums in block order.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs a, int blocks) {
    constexpr int V = D / 128 > 0 ? D / 128 : 1;  // float4 a lane (lanes past D / 4 idle at D = 64)
    constexpr int SLOT = ROWS * (D + 2);
    __shared__ float4 so[8][D / 4];
    __shared__ float sl[8];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t total = all_units(a, ROWS, lane);
    int64_t before;
    // block = (item, row): the sequence from the rows in front of it
    const int64_t at = blockIdx.x;
    const int b = find_seq(a.seqs, at, lane, &before, [&](int i) { return int64_t(load_seq(a, i, ROWS).rt) * a.kv_heads * ROWS; });
    if (b >= a.seqs) return;
    const AttnSeq s = load_seq(a, b, ROWS);
    const int item = int((at - before) / ROWS), row = int((at - before) % ROWS);
    const int h = item / s.rt, rt = item - h * s.rt;
    const int qr = rt * ROWS + row;
    if (qr >= s.n * a.group_heads) return;
    int64_t units_before;
    // units in front of the sequence: the same search, by units
    {
        int64_t sum = 0;
        for (int i = lane; i < b; i += 32) sum += attn_seq_units(load_seq(a, i, ROWS), a.kv_heads);
        units_before = warp_sum64(sum);
    }
    const int64_t x0 = units_before + int64_t(item) * s.units;
    const int64_t shares = attn_shares(total, blocks);
    const int c0 = attn_owner(x0, total, shares), c1 = attn_owner(x0 + s.units - 1, total, shares);
    if (c0 == c1) return;  // written by its block
    // the first block's share may begin before the item
    auto slot_of = [&](int i) {
        return a.part + int64_t(attn_slot(i, attn_share(i, total, shares) >= x0)) * SLOT;
    };
    float top = kNoRef;
    for (int i = c0 + lane; i <= c1; i += 32) top = fmaxf(top, slot_of(i)[ROWS * D + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float4 sum[V];
    float lsum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = c0 + w; i <= c1; i += 8) {
        const float* from = slot_of(i);
        const float f = ex2(from[ROWS * D + row] - top);
        lsum = fmaf(f, from[ROWS * D + ROWS + row], lsum);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k * 32 + lane < D / 4) {
                const float4 v = *reinterpret_cast<const float4*>(from + row * D + (k * 32 + lane) * 4);
                sum[k].x = fmaf(f, v.x, sum[k].x), sum[k].y = fmaf(f, v.y, sum[k].y);
                sum[k].z = fmaf(f, v.z, sum[k].z), sum[k].w = fmaf(f, v.w, sum[k].w);
            }
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k * 32 + lane < D / 4) so[w][k * 32 + lane] = sum[k];
    if (lane == 0) sl[w] = lsum;
    __syncthreads();
    if (threadIdx.x < D / 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v.x += so[k][threadIdx.x].x, v.y += so[k][threadIdx.x].y;
            v.z += so[k][threadIdx.x].z, v.w += so[k][threadIdx.x].w;
            ls += sl[k];
        }
        const int tok = qr / a.group_heads, head = h * a.group_heads + qr - tok * a.group_heads;
        store_row4(a, s.row0 + tok, head, threadIdx.x * 4, v, ls, top);
    }
}

using AttnFn = void (*)(const AttnArgs);
using JoinFn = void (*)(const AttnArgs, int);
struct AttnInst {
    AttnFn fn;
    JoinFn join;
    int smem, slot, rows;
};

template <int D, int GRP, int NT>
AttnInst inst() {
    using F = AttnFmt<D, GRP, NT>;
    static_assert(F::SMEM <= 227 * 1024, "larger than a block's shared memory");
    return AttnInst{attn_kernel<D, GRP, NT>, attn_join_kernel<D, F::ROWS>, F::SMEM, F::SLOT, F::ROWS};
}
template <int D, int GRP>
AttnInst inst_nt(int nt) {
    if constexpr (D == 256) return nt == 1 ? inst<D, GRP, 1>() : inst<D, GRP, 2>();
    else return nt == 1 ? inst<D, GRP, 1>() : nt == 2 ? inst<D, GRP, 2>() : inst<D, GRP, 4>();
}
AttnInst instance(int d, int grp, int nt) {
    if (d == 64) return grp == 32 ? inst_nt<64, 32>(nt) : inst_nt<64, 64>(nt);
    if (d == 128) return grp == 32 ? inst_nt<128, 32>(nt) : grp == 64 ? inst_nt<128, 64>(nt) : inst_nt<128, 128>(nt);
    return grp == 32 ? inst_nt<256, 32>(nt) : grp == 64 ? inst_nt<256, 64>(nt) : inst_nt<256, 128>(nt);
}

// SMs x resident blocks of an instance, once per device and instance.
cudaError_t attn_resident(const AttnInst& k, int* out) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = reinterpret_cast<uint64_t>(k.fn) * 64 + uint64_t(dev);
    std::lock_guard<std::mutex> lk(mu);
    auto it = cache.find(key);
    if (it != cache.end()) {
        *out = it->second;
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return e;
    int per = 0, sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k.fn, 32 * kAttnWarps, size_t(k.smem));
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (per < 1) return cudaErrorInvalidConfiguration;
    *out = per * sms;
    cache.emplace(key, *out);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& in, int head_dim, int group, cudaStream_t stream) {
    AttnArgs a = in;
    // query rows of a tile: as many 8-row columns as the average sequence has rows for, so that the
    // cache is streamed once wherever the rows fit
    const int64_t rows = (int64_t(a.tokens) + a.seqs - 1) / a.seqs * a.group_heads;
    const int nt = rows <= 8 ? 1 : rows <= 16 || head_dim == 256 ? 2 : 4;
    const AttnInst k = instance(head_dim, group, nt);
    int blocks = 0;
    cudaError_t e = attn_resident(k, &blocks);
    if (e != cudaSuccess) return e;
    // never more blocks than units there can be
    const int64_t tiles = int64_t(a.tokens) * a.group_heads / k.rows + a.seqs;
    const int64_t per_item = (int64_t(a.capacity) + kAttnUnit - 1) / kAttnUnit;
    const int64_t units = tiles * a.kv_heads * (per_item > 0 ? per_item : 1);
    if (units < blocks) blocks = int(units);
    void* ws = nullptr;
    e = split_workspace(stream, size_t(2) * blocks * k.slot * sizeof(float), &ws);
    if (e != cudaSuccess) return e;
    a.part = static_cast<float*>(ws);

    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(32 * kAttnWarps);
    cfg.dynamicSmemBytes = size_t(k.smem);
    e = cudaLaunchKernelEx(&cfg, k.fn, static_cast<const AttnArgs>(a));
    if (e != cudaSuccess || blocks == 1 || per_item <= 1) return e;  // nothing can be shared
    cfg.gridDim = dim3(unsigned(tiles * a.kv_heads * k.rows));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k.join, static_cast<const AttnArgs>(a), blocks);
}

cudaError_t attn_read_and_clear_errors(unsigned* out) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_errors, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_attn_errors, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace qmm_impl
