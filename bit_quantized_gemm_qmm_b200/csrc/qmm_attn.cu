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
//     group's fp32 sums are scaled by s afterwards.  b * sum(Q over the group) is one more MMA: b as
//     it is, the sum as three fp16 terms.
//   - V: ldmatrix.trans on the 16-bit units (four codes) of the rows gives lane (g, c) the unit
//     g of rows 2c and 2c + 1 in one register, whose nibble pairs are two positions (k) of one
//     d (row).  Each group's P * s is rounded once to fp16.  V's codes are centred (q - 8), so that
//     this rounding weighs in with the spread of V and not with its distance from the bias: 8 times
//     the sum of the rounded P * s is taken off at the end (one more MMA a group, of a constant),
//     or, with many columns, each pair of codes by a packed add.  b + 8s enters through fp32 sums
//     of P * (b + 8s).
// The scores' layout (position by query) is the transpose of the second product's operand;
// movmatrix turns the packed P * s round.
//
// Softmax: each warp keeps a reference per query, not the maximum: x - ref goes through ex2 and
// the sums are rescaled only when some P * s reaches 2^15 or x - ref reaches 60.  The reference is then
// put so that the largest P * s of the tile is 2^10: fp16 rounds by 2^-11 down to 2^-24 of that, whatever the
// weight of a position and however small a group's V beside the others' (with the largest at 2^-4 all that
// lay 2^-20 below it was lost; the wider range costs 1 us of 69 where 32 sequences of up to 16,384 decode).
//
// Work: units of 32 positions of one (sequence, K/V head, row tile) are dealt out evenly over
// the resident blocks (qmm_kv_plan.h), whatever the lengths; a block's warps take them in turn, each
// through its own cp.async ring.  Items that several blocks share are summed by the last of them to
// arrive, in an order that does not depend on timing.
//
// Bound by the stream of codes and, nearly as much, by the instructions that take them apart: 32 sequences of
// up to 16,384 positions (313 MB) take 70 us, 4.5 TB/s (issue slots 55% busy, ALU 50%); what is missing is the items'
// starts and shares that do not end together.  One token over 1,024 positions takes 9 us: the plan, the first tiles
// and the join, one after another.
#include <mutex>
#include <type_traits>
#include <unordered_map>

#include "qmm_attn.cuh"
#include "sm100.cuh"

namespace qmm_impl {
namespace {

__device__ unsigned g_attn_errors;  // bit 1: a page or position outside the cache

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
// Of three, in one instruction: the largest, and the largest magnitude (NaN are passed over).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

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

// Shared-memory layout of an instance: per warp a ring of tiles of kAttnUnit positions (its first slots
// hold the warp's partial sums at the end of an item), then Q as MMA fragments and the rows' constants.
template <int D, int GRP, int NT>
struct AttnFmt {
    static constexpr int W = 4, BLOCKS = D == 256 || NT > 1 ? 2 : 3;  // warps a block, blocks an SM
    static constexpr int NG = D / GRP;
    static constexpr int CH = D / 32;                 // 16-byte pieces (32 codes) of a row
    static constexpr int ROWS = 8 * NT;
    static constexpr int CODES = kAttnUnit * D / 2;   // bytes of a tile's K (or V) codes
    static constexpr int SB = kAttnUnit * NG * 2;     // bytes of a tile's K scales (or biases, V's)
    static constexpr int TILE = 2 * CODES + 4 * SB;
    static constexpr int OROW = D + 4;                // floats between rows of the partial sums
    static constexpr int MERGE = ROWS * OROW * 4 + ROWS * 8;
    static constexpr int MS = (MERGE + TILE - 1) / TILE;  // ring slots under the partial sums
    static constexpr int QF = ROWS * D * 2;           // Q fragments
    static constexpr int CONSTS = ROWS * (4 + 4 + 8 + 8 * NG) + 16 + 3 * 96;
    // the ring: four tiles, or as many as leave room for the SM's other blocks
    static constexpr int ROOM = (BLOCKS == 2 ? 113 : 75) * 1024 - QF - CONSTS;
    static constexpr int FIT = ROOM / (W * TILE);
    static constexpr int RING = FIT > 4 ? 4 : FIT;
    static_assert(RING >= 2 && RING >= MS, "ring too small");
    static constexpr int WARP = RING * TILE;
    static constexpr int OFF_Q = W * WARP;
    static constexpr int OFF_F = OFF_Q + QF;          // float per row: factor of the sums
    static constexpr int OFF_LIM = OFF_F + ROWS * 4;  // int per row: last position seen
    static constexpr int OFF_BITS = OFF_LIM + ROWS * 4;   // 64-bit mask per row
    static constexpr int OFF_QB = OFF_BITS + ROWS * 8;    // sum of Q over a group as three fp16 (and a zero), per row and group
    static constexpr int OFF_LAST = OFF_QB + ROWS * NG * 8;
    static constexpr int OFF_RUN = OFF_LAST + 16;     // this run and the next two
    static constexpr int SMEM = OFF_RUN + 3 * 96;
    static constexpr int SLOT = ROWS * (D + 2);       // floats of one partial-sum slot
    static constexpr int SUBS = NT == 1 && D * NG <= 256 ? 2 : 1;  // 16-position halves of a tile taken together
    static constexpr bool SUMS = NT == 1 && NG <= 4;       // V's codes centred by sums of P * s, not one by one
};

template <int D, int GRP, int NT>
__global__ void __launch_bounds__(32 * AttnFmt<D, GRP, NT>::W, AttnFmt<D, GRP, NT>::BLOCKS) attn_kernel(const __grid_constant__ AttnArgs a) {
    using F = AttnFmt<D, GRP, NT>;
    constexpr int NG = F::NG, CH = F::CH, R = F::ROWS, W = F::W, SUBS = F::SUBS, THREADS = 32 * W;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t sbase = smem_addr(smem);
    const uint32_t ring = sbase + w * F::WARP;

    grid_dependency_wait();
    grid_dependents_launch();

    // start: measured on 32 sequences of 100 to 16,384 positions, by the spread of the blocks' ends
    constexpr AttnCut cut{R, kAttnUnit, W, 20};
    AttnPlan pl;
    int x_end;
    Run* cur = reinterpret_cast<Run*>(smem + F::OFF_RUN);
    Run *next = cur + 1, *then = cur + 2;  // one warp plans a run, two ahead
    bool bad = false;
    {
        const int got = plan_block(a, cut, lane, tid == 0, &pl, &x_end, cur, &bad);
        if (got < 0 && blockIdx.x == 0 && tid == 0) atomicOr(&g_attn_errors, 2u);
        if (got <= 0) return;
        __syncthreads();
    }
    auto plan_after = [&](const Run* r, Run* to) {
        if (r->n == 0) {
            if (lane == 0) to->n = 0;
        } else {
            plan_run(a, pl, cut, r->x + r->places, x_end, r->b, r->before, lane == 0, to, &bad);
        }
    };

    // ---- tile copies.  Codes: 16-byte piece p of a tile goes to row p / CH, piece p % CH, xor-swizzled
    // so that eight rows' equal pieces fall into different banks.  A lane's pieces of 16 rows lie at
    // fixed distances, in the cache and in the tile.
    auto swz = [](int row, int ch) { return row * (D / 2) + ((ch ^ ((row * (D / 2) >> 7) & (CH - 1))) << 4); };
    constexpr int CPT = CH / 2;                 // pieces of codes a lane copies of a half tile, K and V each
    constexpr int SPT = NG >= 2 ? NG / 2 : 1;   // pieces of scales and biases a lane copies of a tile
    uint32_t cdst[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) cdst[i] = ring + swz((i * 32 + lane) / CH, (i * 32 + lane) % CH);
    const bool s_on = 16 * NG >= 32 || lane < 16 * NG;
    const int s_sub = (lane % (4 * NG)) / (2 * NG);
    const uint8_t* ssrc[SPT];
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
        const int p = i * 32 + (s_on ? lane : 0), arr = p / (4 * NG);
        ssrc[i] = reinterpret_cast<const uint8_t*>(arr == 0 ? a.ks : arr == 1 ? a.kb : arr == 2 ? a.vs : a.vb) + p % (2 * NG) * 16;
    }
    const uint8_t* const ksrc = a.kc + lane * 16;
    const uint8_t* const vsrc = a.vc + lane * 16;

    int t0 = 0, j0 = 0, j1 = 0;      // this warp's tiles of the run: positions t0 + 32 W j, j in [j0, j1)
    int idb = 0, ids = -1, ids_next = -1;  // lane 2 k + s: index (in 16 rows) of half s of tile idb + k; -1 none, -2 bad
    // index (in 16 rows) of this lane's half of the tiles from j on, of a run's tiles as above
    auto rows16 = [&](const Run* r, int from, int j, int end) {
        const int t = from + kAttnUnit * W * (j + (lane >> 1)) + kAttnSub * (lane & 1);
        if (t >= r->hi || j + (lane >> 1) >= end) return -1;
        const int col = t / a.page, page = a.table[int64_t(r->b) * a.table_stride + col];
        return page < 0 || page >= a.pages ? -2 : int((int64_t(page) * a.kv_heads + r->h) * (a.page / kAttnSub)) + (t - col * a.page) / kAttnSub;
    };
    int n_t0, n_j0, n_j1, n_ids;  // the next run's, looked up while the current one's first tiles come
    auto prepare = [&](const Run* r) {
        attn_warp_units(r->t0, r->n, w, W, r->lo, r->hi, &n_j0, &n_j1);
        n_t0 = r->t0 + kAttnUnit * w;
        n_ids = rows16(r, n_t0, n_j0, n_j1);
    };
    auto begin = [&](const Run* r) {
        t0 = n_t0, j0 = n_j0, j1 = n_j1, ids = n_ids;
        idb = j0;
        ids_next = rows16(r, t0, j0 + 16, j1);
    };
    uint32_t live = 0;  // two bits a ring slot: its halves were copied
    auto issue = [&](const Run* r, int j, int slot) {
        if (j < j1) {
            if (j - idb == 16) {
                idb = j;
                ids = ids_next;
                ids_next = rows16(r, t0, j + 16, j1);
            }
            const int r0 = __shfl_sync(kFull, ids, 2 * (j - idb)), r1 = __shfl_sync(kFull, ids, 2 * (j - idb) + 1);
            bad |= r0 == -2 || r1 == -2;
            live = (live & ~(3u << (2 * slot))) | ((r0 >= 0 ? 1u : 0u) | (r1 >= 0 ? 2u : 0u)) << (2 * slot);
            // halves that are not there copy the pool's first rows, and are masked
            const int64_t at0 = r0 < 0 ? 0 : r0, at1 = r1 < 0 ? 0 : r1;
            const uint32_t off = slot * F::TILE;
            const uint8_t* const k0 = ksrc + at0 * (kAttnSub * D / 2);
            const uint8_t* const k1 = ksrc + at1 * (kAttnSub * D / 2);
            const uint8_t* const v0 = vsrc + at0 * (kAttnSub * D / 2);
            const uint8_t* const v1 = vsrc + at1 * (kAttnSub * D / 2);
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                cp_async_16(cdst[i] + off, k0 + i * 512);
                cp_async_16(cdst[i] + off + F::CODES / 2, k1 + i * 512);
                cp_async_16(cdst[i] + off + F::CODES, v0 + i * 512);
                cp_async_16(cdst[i] + off + F::CODES + F::CODES / 2, v1 + i * 512);
            }
            const int64_t sat = (s_sub ? at1 : at0) * (kAttnSub * NG * 2);
#pragma unroll
            for (int i = 0; i < SPT; ++i) {
                const uint32_t dst = ring + off + 2 * F::CODES + (i * 32 + lane) * 16;
                if constexpr (16 * NG >= 32) cp_async_16(dst, ssrc[i] + sat);
                else if (s_on) cp_async_16(dst, ssrc[i] + sat);
            }
        }
        sm100::cp_async_commit();
    };

    // eight values of Q, for thread-item i of a run's rows
    auto load_q = [&](const Run* r, int i) {
        const int row = i / (D / 8), p8 = i % (D / 8);
        if (row >= r->rows) return make_uint4(0u, 0u, 0u, 0u);
        const int qr = r->row_lo + row, tok = qr / a.group_heads, hg = qr - tok * a.group_heads;
        const uint16_t* src = a.q + int64_t(r->row0 + tok) * a.q_ts + int64_t(r->h * a.group_heads + hg) * a.q_hs + p8 * 8;
        if (a.q_vec) return *reinterpret_cast<const uint4*>(src);
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = uint32_t(src[2 * j]) | uint32_t(src[2 * j + 1]) << 16;
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    uint4 q_first = load_q(cur, tid);  // on its way while the tiles' pages are looked up
    prepare(cur);
    begin(cur);
#pragma unroll
    for (int i = 0; i < F::RING - F::MS; ++i) issue(cur, j0 + i, F::MS + i);
    if (w == 0) plan_after(cur, next);
    while (true) {
        // ---- Q: fragments in shared memory, scaled by a power of two per row
        for (int i = tid; i < R * (D / 8); i += THREADS) {
            const int row = i / (D / 8), p8 = i % (D / 8);  // eight values from 8 * p8
            float v[8];
            {
                const uint4 u = i == tid ? q_first : load_q(cur, i);
                const uint32_t raw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = a.is_bf16 ? bf16lo_to_f32(raw[j]) : half_lo(raw[j]);
                    v[2 * j + 1] = a.is_bf16 ? bf16hi_to_f32(raw[j]) : half_hi(raw[j]);
                }
            }
            const int tok = (cur->row_lo + row) / a.group_heads;
            float mx = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[j]));
#pragma unroll
            for (int o = 1; o < D / 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
            // exponent e with max * 2^e in [2^14, 2^15); rows of zeros, infinities or NaN: 0
            int e = 0;
            if (mx > 0.f && mx < INFINITY) e = 14 + 127 - int(__float_as_uint(mx) >> 23);
            if (e > 126) e = 126;  // subnormal rows
            const float up = exp2i(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= up, sum += v[j];
#pragma unroll
            for (int o = 1; o < GRP / 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
            // nibbles 0, 2 of a pair's place are codes * 2^-24, nibbles 1, 3 codes * 2^-20
            uint4 f;
            f.x = f32x2_to_f16x2(v[0], v[4]);
            f.y = f32x2_to_f16x2(v[2], v[6]);
            f.z = f32x2_to_f16x2(v[1] * 0.0625f, v[5] * 0.0625f);
            f.w = f32x2_to_f16x2(v[3] * 0.0625f, v[7] * 0.0625f);
            const int nt = row >> 3, ch = p8 >> 2, ln = (row & 7) * 4 + (p8 & 3);
            sts_v4(sbase + F::OFF_Q + ((nt * CH + ch) * 32 + ln) * 16, f);
            if (p8 % (GRP / 8) == 0) {
                // the group's sum in the same units, as three fp16 terms
                const float s0 = sum * (0x1p-24f * kSumUp), h0 = __half2float(__float2half_rn(s0));
                const float s1 = s0 - h0, h1 = __half2float(__float2half_rn(s1));
                uint32_t* qb = reinterpret_cast<uint32_t*>(smem + F::OFF_QB + (row * NG + p8 / (GRP / 8)) * 8);
                qb[0] = f32x2_to_f16x2(h0, h1);
                qb[1] = f32x2_to_f16x2(s1 - h1, 0.f);
            }
            if (p8 == 0) {
                // 2^24 / kSumUp * 2^-e in two steps (e may be as low as -113)
                *reinterpret_cast<float*>(smem + F::OFF_F + row * 4) = a.scale_log2 * (16777216.f / kSumUp) * exp2i(-e);
                *reinterpret_cast<int*>(smem + F::OFF_LIM + row * 4) = row < cur->rows ? cur->start + tok : INT_MAX;
                *reinterpret_cast<int64_t*>(smem + F::OFF_BITS + row * 8) =
                    a.tree != nullptr && row < cur->rows ? a.tree[cur->row0 + tok] : -1;
            }
        }
        __syncthreads();
        // the slots that the last item's sums were in
#pragma unroll
        for (int i = F::RING - F::MS; i < F::RING - 1; ++i) issue(cur, j0 + i, (F::MS + i) % F::RING);
        const bool more = next->n > 0;
        if (more) prepare(next);

        // constants of the queries: in registers for one column of them, else from shared memory each time
        constexpr int QBM = (NG + 3) / 4;  // MMAs for the biases: four groups each
        auto q_frag = [&](int nt, int ch) { return lds_v4(sbase + F::OFF_Q + ((nt * CH + ch) * 32 + lane) * 16); };
        auto q_factor = [&](int nt) { return lds_f2(sbase + F::OFF_F + (nt * 8 + 2 * c) * 4); };
        auto q_bias = [&](int nt, int m) {
            const uint2 v = lds_u2(sbase + F::OFF_QB + ((nt * 8 + g) * NG + m * 4 + (NG < 4 ? c % NG : c)) * 8);
            return m * 4 + c < NG ? v : make_uint2(0u, 0u);
        };
        uint4 qreg[NT == 1 ? CH : 1];
        float2 qfreg = make_float2(0.f, 0.f);
        uint2 qbreg[NT == 1 ? QBM : 1];
        if constexpr (NT == 1) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) qreg[ch] = q_frag(0, ch);
            qfreg = q_factor(0);
#pragma unroll
            for (int m = 0; m < QBM; ++m) qbreg[m] = q_bias(0, m);
        }

        // sums, relative to the queries' references
        float ref[NT][2], l[NT][2], bs[NT][2][NG], o[NT][CH][2][4], os[F::SUMS ? NT : 1][F::SUMS ? NG : 1][4];
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
            if constexpr (F::SUMS) {
#pragma unroll
                for (int j = 0; j < NG; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) os[nt][j][i] = 0.f;
            }
        }

        // SUBS halves of a tile from its half h0 on; `there`: bit per half of the tile that was copied
        // COLS of the NT columns of query rows are in use
        auto part = [&](int t, uint32_t st, int h0, uint32_t there, auto masked_c, auto cols_c) {
            constexpr bool MASKED = decltype(masked_c)::value;
            constexpr int COLS = decltype(cols_c)::value;
            const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix: this lane's row and piece
            const int kch = lane >> 4;
            // which of this lane's (position, query) pairs are seen
            uint32_t see[SUBS];
            bool in[SUBS][2];
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                see[u] = 0xFFFFFFFFu;
                in[u][0] = in[u][1] = true;
                if constexpr (MASKED) {
                    see[u] = 0;
                    const bool ok = (there >> (h0 + u)) & 1;
                    const int tu = t + kAttnSub * (h0 + u) + g;
                    in[u][0] = ok && tu < cur->keys, in[u][1] = ok && tu + 8 < cur->keys;
#pragma unroll
                    for (int nt = 0; nt < COLS; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = nt * 8 + 2 * c + (i & 1), p = tu + (i >> 1) * 8;
                            bool on;
                            if (a.tree != nullptr) {
                                const int64_t bits = *reinterpret_cast<const int64_t*>(smem + F::OFF_BITS + row * 8);
                                const int d = p - cur->start;
                                on = d < 0 || (d < 64 && ((bits >> d) & 1));
                            } else {
                                const int lim = *reinterpret_cast<const int*>(smem + F::OFF_LIM + row * 4);
                                on = p <= lim && (a.window <= 0 || lim == INT_MAX || p > lim - a.window);
                            }
                            if (on && in[u][i >> 1]) see[u] |= 1u << (nt * 4 + i);
                        }
                }
            }
            // ---- scores.  acc = sum over groups of b * sum(Q) (one MMA) + s * code sums
            float acc[SUBS][COLS][4], ks[SUBS][2][NG];
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                const uint32_t sb = st + 2 * F::CODES + (kAttnSub * (h0 + u) + g) * (2 * NG);
                lds_halves<NG>(sb, ks[u][0]);
                lds_halves<NG>(sb + 16 * NG, ks[u][1]);
#pragma unroll
                for (int j = 0; j < NG; ++j) ks[u][0][j] *= kSumUp, ks[u][1][j] *= kSumUp;
#pragma unroll
                for (int m = 0; m < QBM; ++m) {
                    const uint32_t at = sb + F::SB + (m * 4 + (NG < 4 ? c % NG : c)) * 2;
                    uint16_t b0, b1;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b0) : "r"(at));
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b1) : "r"(at + 16 * NG));
                    const uint32_t p0 = b0 * 0x10001u, p1 = b1 * 0x10001u;
#pragma unroll
                    for (int nt = 0; nt < COLS; ++nt) {
                        const uint2 qb = NT == 1 ? qbreg[NT == 1 ? m : 0] : q_bias(nt, m);
                        if (m == 0) mma_16816_z(acc[u][nt], p0, p1, p0, p1, qb.x, qb.y);
                        else mma_16816(acc[u][nt], p0, p1, p0, p1, qb.x, qb.y);
                    }
                }
            }
            {
                float sums[SUBS][COLS][4], low[MASKED ? SUBS : 1][MASKED ? COLS : 1][4];
                uint32_t kw[SUBS][4];
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
                    for (int u = 0; u < SUBS; ++u) {
                        if (ch % 2 == 0) ldsm_x4(st + swz(kAttnSub * (h0 + u) + krow, ch + kch), kw[u]);
                        const uint32_t w0 = kw[u][2 * (ch & 1)], w1 = kw[u][2 * (ch & 1) + 1];
                        const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
                        // The MMA aligns products by the exponents' fields, where a subnormal's is 2^-14 whatever its
                        // value: beside q's largest, products below 2^-15 (codes in place) or 2^-19 (one place up) are cut
                        // off.  Where few positions may be seen all codes go one place up, the shifted ones summed apart
                        constexpr uint32_t me = MASKED ? 0x00F000F0u : 0x000F000Fu;
                        constexpr int up = MASKED ? 4 : 0;
                        const uint32_t e0 = (w0 << up) & me, e1 = (w1 << up) & me, e2 = (y0 << up) & me, e3 = (y1 << up) & me;
                        const uint32_t f0 = w0 & 0x00F000F0u, f1 = w1 & 0x00F000F0u, f2 = y0 & 0x00F000F0u, f3 = y1 & 0x00F000F0u;
#pragma unroll
                        for (int nt = 0; nt < COLS; ++nt) {
                            const uint4 q = NT == 1 ? qreg[NT == 1 ? ch : 0] : q_frag(nt, ch);
                            if constexpr (MASKED) {
                                if (ch * 32 % GRP == 0) mma_16816_z(low[u][nt], e0, e1, e2, e3, q.x, q.y), mma_16816_z(sums[u][nt], f0, f1, f2, f3, q.z, q.w);
                                else mma_16816(low[u][nt], e0, e1, e2, e3, q.x, q.y), mma_16816(sums[u][nt], f0, f1, f2, f3, q.z, q.w);
                            } else {
                                if (ch * 32 % GRP == 0) mma_16816_z(sums[u][nt], e0, e1, e2, e3, q.x, q.y);
                                else mma_16816(sums[u][nt], e0, e1, e2, e3, q.x, q.y);
                                mma_16816(sums[u][nt], f0, f1, f2, f3, q.z, q.w);
                            }
                        }
                        if ((ch + 1) * 32 % GRP == 0) {
#pragma unroll
                            for (int nt = 0; nt < COLS; ++nt)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if constexpr (MASKED) sums[u][nt][i] = fmaf(low[u][nt][i], 0.0625f, sums[u][nt][i]);
                                    acc[u][nt][i] = fmaf(ks[u][i >> 1][ch * 32 / GRP], sums[u][nt][i], acc[u][nt][i]);
                                }
                        }
                    }
                }
            }
            // ---- probabilities, V's scales applied, packed for the second product
            float vs[SUBS][2][NG], vb[SUBS][2][NG];
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                const uint32_t sb = st + 2 * F::CODES + 2 * F::SB + (kAttnSub * (h0 + u) + g) * (2 * NG);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    lds_halves<NG>(sb + k * 16 * NG, vs[u][k]);
                    lds_halves<NG>(sb + F::SB + k * 16 * NG, vb[u][k]);
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        if (MASKED && !in[u][k]) vs[u][k][j] = vb[u][k][j] = 0.f;
                        vb[u][k][j] = fmaf(8.f, vs[u][k][j], vb[u][k][j]);
                    }
                }
            }
            float p[SUBS][COLS][4];
            uint32_t pk[SUBS][COLS][NG][2];
            auto probabilities = [&]() -> bool {
                float most = 0.f;
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < SUBS; ++u)
#pragma unroll
                    for (int nt = 0; nt < COLS; ++nt) {
                        const float2 qf = NT == 1 ? qfreg : q_factor(nt);
                        float xs[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // rounded before ref comes off: scores past 2^24 would leave a product's lost bits otherwise
                            float xv = __fmul_rn(i & 1 ? qf.y : qf.x, acc[u][nt][i]) - ref[nt][i & 1];
                            if (MASKED && !((see[u] >> (nt * 4 + i)) & 1)) xv = -INFINITY;
                            xs[i] = xv;
                            p[u][nt][i] = ex2(xv);
                        }
                        top = max3(max3(top, xs[0], xs[1]), xs[2], xs[3]);
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            float m[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                m[i] = p[u][nt][i] * vs[u][i >> 1][j];
                                if (MASKED && !((see[u] >> (nt * 4 + i)) & 1)) m[i] = 0.f;
                            }
                            pk[u][nt][j][0] = f32x2_to_f16x2(m[0], m[1]);
                            pk[u][nt][j][1] = f32x2_to_f16x2(m[2], m[3]);
                            most = max3_abs(max3_abs(most, m[0], m[1]), m[2], m[3]);
                        }
                    }
                return most >= 32768.f || top > 60.f;
            };
            if (__any_sync(kFull, probabilities())) {
                // New references from these positions: the largest P * s becomes 2^10, or P is 1 where s alone is
                // larger (and at most 2^34: s is 2^-24 at least, or nothing).  The reference is rounded towards
                // the score, so that scores far past 2^24 leave P between 1 and what it should be
                float lg[SUBS][2];
#pragma unroll
                for (int u = 0; u < SUBS; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float m = 0.f;
#pragma unroll
                        for (int j = 0; j < NG; ++j) m = fmaxf(m, fabsf(vs[u][k][j]) < INFINITY ? fabsf(vs[u][k][j]) : 0.f);
                        lg[u][k] = fminf(fmaxf(lg2(m) - 10.f, -34.f), 0.f);
                    }
#pragma unroll
                for (int nt = 0; nt < COLS; ++nt) {
                    const float2 qf = NT == 1 ? qfreg : q_factor(nt);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float m = -INFINITY;
#pragma unroll
                        for (int u = 0; u < SUBS; ++u)
#pragma unroll
                            for (int i = k; i < 4; i += 2) {
                                const float sc = __fmul_rn(k ? qf.y : qf.x, acc[u][nt][i]);
                                const float v = __fadd_ru(sc, lg[u][i >> 1]);
                                if (!MASKED || ((see[u] >> (nt * 4 + i)) & 1)) m = fmaxf(m, v);
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
                        if constexpr (F::SUMS) {
#pragma unroll
                            for (int j = 0; j < NG; ++j) os[nt][j][k] *= f, os[nt][j][k + 2] *= f;
                        }
                    }
                }
                probabilities();
            }
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int nt = 0; nt < COLS; ++nt) {
                    l[nt][0] += p[u][nt][0] + p[u][nt][2];
                    l[nt][1] += p[u][nt][1] + p[u][nt][3];
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (MASKED) bs[nt][i & 1][j] += ((see[u] >> (nt * 4 + i)) & 1) ? p[u][nt][i] * vb[u][i >> 1][j] : 0.f;
                            else bs[nt][i & 1][j] = fmaf(p[u][nt][i], vb[u][i >> 1][j], bs[nt][i & 1][j]);
                        }
                        pk[u][nt][j][0] = movmatrix_trans(pk[u][nt][j][0]);
                        pk[u][nt][j][1] = movmatrix_trans(pk[u][nt][j][1]);
                        if constexpr (F::SUMS)  // 8 * 2^-24 in every row: the sum of P * s, for the centre of the codes
                            mma_16816(os[nt][j], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, pk[u][nt][j][0], pk[u][nt][j][1]);
                    }
                }
            // ---- sums over V: rows d = 32 ch + 4 g + {m, m + 2}
            uint32_t vw[SUBS][4];
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const int j = ch * 32 / GRP;
#pragma unroll
                for (int u = 0; u < SUBS; ++u) {
                    if (ch % 2 == 0) ldsm_x4_trans(st + F::CODES + swz(kAttnSub * (h0 + u) + krow, ch + kch), vw[u]);
                    const uint32_t w0 = vw[u][2 * (ch & 1)], w1 = vw[u][2 * (ch & 1) + 1];
                    const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
                    uint32_t e0 = w0 & 0x000F000Fu, e1 = y0 & 0x000F000Fu, e2 = w1 & 0x000F000Fu, e3 = y1 & 0x000F000Fu;
                    uint32_t f0 = w0 & 0x00F000F0u, f1 = y0 & 0x00F000F0u, f2 = w1 & 0x00F000F0u, f3 = y1 & 0x00F000F0u;
                    if constexpr (!F::SUMS) {
                        constexpr uint32_t m8 = 0x80088008u, m80 = 0x80808080u;  // -8 * 2^-24, -8 * 2^-20
                        e0 = hadd2_bits(e0, m8), e1 = hadd2_bits(e1, m8), e2 = hadd2_bits(e2, m8), e3 = hadd2_bits(e3, m8);
                        f0 = hadd2_bits(f0, m80), f1 = hadd2_bits(f1, m80), f2 = hadd2_bits(f2, m80), f3 = hadd2_bits(f3, m80);
                    }
#pragma unroll
                    for (int nt = 0; nt < COLS; ++nt) {
                        mma_16816(o[nt][ch][0], e0, e1, e2, e3, pk[u][nt][j][0], pk[u][nt][j][1]);
                        mma_16816(o[nt][ch][1], f0, f1, f2, f3, pk[u][nt][j][0], pk[u][nt][j][1]);
                    }
                }
            }
        };

        // ---- stream the tiles
        int slot = F::MS % F::RING;
        const int full_lo = cur->full_lo, full_hi = cur->full_hi, cols = (cur->rows + 7) / 8;
        for (int j = j0; j < j1; ++j) {
            sm100::cp_async_wait<F::RING - 2>();
            __syncwarp();
            issue(cur, j + F::RING - 1, slot == 0 ? F::RING - 1 : slot - 1);
            const int t = t0 + kAttnUnit * W * j;
            const uint32_t there = (live >> (2 * slot)) & 3u, st = ring + slot * F::TILE;
            auto tile = [&](auto cols_c) {
                if (there == 3 && t >= full_lo && t + kAttnUnit <= full_hi) {
#pragma unroll
                    for (int h0 = 0; h0 < 2; h0 += SUBS) part(t, st, h0, there, std::false_type{}, cols_c);
                } else if (there) {
#pragma unroll 1
                    for (int h0 = 0; h0 < 2; h0 += SUBS) part(t, st, h0, there, std::true_type{}, cols_c);
                }
            };
            if (NT >= 4 && cols == 4) tile(std::integral_constant<int, NT >= 4 ? 4 : 1>{});
            else if (NT >= 3 && cols == 3) tile(std::integral_constant<int, NT >= 3 ? 3 : 1>{});
            else if (NT >= 2 && cols == 2) tile(std::integral_constant<int, NT >= 2 ? 2 : 1>{});
            else tile(std::integral_constant<int, 1>{});
            slot = slot == F::RING - 1 ? 0 : slot + 1;
        }
        sm100::cp_async_wait<0>();
        __syncwarp();

        // ---- the next item's first tiles are fetched while this one's sums are put together
        if (more) {
            q_first = load_q(next, tid);
            begin(next);
#pragma unroll
            for (int i = 0; i < F::RING - F::MS; ++i) issue(next, j0 + i, F::MS + i);
        }
        if (w == W - 1) plan_after(next, then);
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
                    float bb = bs[nt][k][ch * 32 / GRP];
                    if constexpr (F::SUMS) bb = fmaf(os[nt][ch * 32 / GRP][k], -16777216.f, bb);
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
        const bool whole = cur->n == cur->units;
        float* slot_o = a.part + int64_t(attn_slot(blockIdx.x, cur->c0)) * F::SLOT;
        for (int i = tid; i < cur->rows * (D / 4); i += THREADS) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float rf[W], top = kNoRef;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                rf[k] = reinterpret_cast<const float*>(smem + k * F::WARP)[R * F::OROW + row];
                top = fmaxf(top, rf[k]);
            }
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float lsum = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float* from = reinterpret_cast<const float*>(smem + k * F::WARP);
                const float f = ex2(rf[k] - top);
                const float4 v = *reinterpret_cast<const float4*>(from + row * F::OROW + d);
                sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
                sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
                lsum = fmaf(f, from[R * F::OROW + R + row], lsum);
            }
            if (whole) {
                const int qr = cur->row_lo + row, tok = qr / a.group_heads;
                store_row4(a, cur->row0 + tok, cur->h * a.group_heads + qr - tok * a.group_heads, d, sum, lsum, top);
            } else {
                __stcg(reinterpret_cast<float4*>(slot_o + row * D + d), sum);
                if (d == 0) __stcg(slot_o + R * D + row, top), __stcg(slot_o + R * D + R + row, lsum);
            }
        }
        if (!whole) join_item<D, R>(a, cur, tid, THREADS, reinterpret_cast<int*>(smem + F::OFF_LAST));
        if (!more) break;
        __syncthreads();  // the sums' ring slots and Q are free
        Run* const was = cur;
        cur = next, next = then, then = was;
    }
    if (__any_sync(kFull, bad) && lane == 0) atomicOr(&g_attn_errors, 2u);
}

using AttnFn = void (*)(const AttnArgs);
struct AttnInst {
    AttnFn fn;
    int smem, slot, rows, threads, blocks;
};

template <int D, int GRP, int NT>
AttnInst inst() {
    using F = AttnFmt<D, GRP, NT>;
    static_assert(F::SMEM <= (F::BLOCKS == 2 ? 114 : 76) * 1024, "the blocks do not fit an SM");
    return AttnInst{attn_kernel<D, GRP, NT>, F::SMEM, F::SLOT, F::ROWS, 32 * F::W, F::BLOCKS};
}
template <int D, int GRP>
AttnInst inst_nt(int nt) {
    if constexpr (D == 256) return nt == 1 ? inst<D, GRP, 1>() : inst<D, GRP, 2>();
    else return nt == 1 ? inst<D, GRP, 1>() : nt == 2 ? inst<D, GRP, 2>() : nt == 3 ? inst<D, GRP, 3>() : inst<D, GRP, 4>();
}
AttnInst instance(int d, int grp, int nt) {
    if (d == 64) return grp == 32 ? inst_nt<64, 32>(nt) : inst_nt<64, 64>(nt);
    if (d == 128) return grp == 32 ? inst_nt<128, 32>(nt) : grp == 64 ? inst_nt<128, 64>(nt) : inst_nt<128, 128>(nt);
    return grp == 32 ? inst_nt<256, 32>(nt) : grp == 64 ? inst_nt<256, 64>(nt) : inst_nt<256, 128>(nt);
}

}  // namespace

cudaError_t attn_blocks(void (*fn)(const AttnArgs), int smem, int per_sm, int regs, int* out) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = reinterpret_cast<uint64_t>(fn) * 64 + uint64_t(dev);
    std::lock_guard<std::mutex> lk(mu);
    auto it = cache.find(key);
    if (it != cache.end()) {
        *out = it->second;
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (regs) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, fn);
        if (e != cudaSuccess) return e;
        if (at.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    *out = per_sm * sms;
    cache.emplace(key, *out);
    return cudaSuccess;
}

cudaError_t launch_attn_blocks(AttnArgs a, void (*fn)(const AttnArgs), int threads, int smem, int slot, int rows, int unit,
                               int per_sm, int regs, cudaStream_t stream) {
    int blocks = 0;
    cudaError_t e = attn_blocks(fn, smem, per_sm, regs, &blocks);
    if (e != cudaSuccess) return e;
    // never more blocks than units there can be
    const int64_t tiles = int64_t(a.tokens) * a.group_heads / rows + a.seqs;
    const int64_t per_item = (int64_t(a.capacity) + unit - 1) / unit;
    const int64_t units = tiles * a.kv_heads * (per_item > 0 ? per_item : 1);
    if (units >= int64_t(1) << 29) return cudaErrorNotSupported;  // with the items' starts, below 2^31
    if (units < blocks) blocks = int(units);
    if (blocks > kArrivalBlocks) blocks = kArrivalBlocks;
    void* ws = nullptr;
    e = split_workspace(stream, size_t(2) * blocks * slot * sizeof(float), &ws);
    if (e != cudaSuccess) return e;
    a.part = static_cast<float*>(ws);
    e = arrival_counters(stream, &a.count);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    return cudaLaunchKernelEx(&cfg, fn, static_cast<const AttnArgs>(a));
}

cudaError_t launch_attn(const AttnArgs& a, int head_dim, int group, cudaStream_t stream) {
    // Query rows of a tile: what the sequences have, so that the cache is streamed once wherever they fit.  Only
    // the average is known here; where there are several sequences, some are taken to have half as many again.  That
    // is too many where they are all alike, or their longest is not much longer: 8 sequences of 6 tokens of 4 heads
    // (24 rows each, taken for 36) run in the tensor-core kernel in 44 us over 4,096 positions and 103 over 16,384,
    // in three columns of the warps' kernel in 35 and 76; of up to 6 tokens in 28 and 57 against 25 and 49.
    // It saves 8 of 8 tokens, whose fourth column spills: 45 and 105 us against 58 and 160.
    const int64_t mean = (int64_t(a.tokens) + a.seqs - 1) / a.seqs;
    const int64_t rows = (a.seqs > 1 ? mean + mean / 2 : mean) * a.group_heads;
    // The warps' kernel up to 32 rows (as counted above) of 128, up to 512 of 64, whose two passes over the codes
    // cost half (128 tokens of 4 heads over 8k positions: 56 us against 70; 16 sequences of 64 tokens over 2k in
    // groups of 32: 85 against 82).  Heads of 256 have only the former
    const int most_rows = head_dim == 64 ? 512 : 32;
    if (rows > most_rows && attn_tc_supported(head_dim)) return launch_attn_tc(a, int(rows < 65536 ? rows : 65536), head_dim, group, stream);
    const int64_t cols = (rows + 7) / 8, most = head_dim == 256 ? 2 : 4;
    const AttnInst k = instance(head_dim, group, int(cols < most ? cols : most));
    return launch_attn_blocks(a, k.fn, k.threads, k.smem, k.slot, k.rows, kAttnUnit, k.blocks, 0, stream);
}

cudaError_t attn_read_and_clear_errors(unsigned* out) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_errors, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_attn_errors, &zero, sizeof(zero));
    if (e != cudaSuccess) return e;
    unsigned t = 0;
    e = attn_tc_read_and_clear_errors(&t);
    *out = v | t;
    return e;
}

}  // namespace qmm_impl
