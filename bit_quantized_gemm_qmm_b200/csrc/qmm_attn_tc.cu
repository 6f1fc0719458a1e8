// qmm_attn_tc.cu -- attention over the paged 4-bit K/V cache for many query rows (tcgen05).
//
// The same operation as qmm_attn.cu, for tiles of up to 64 query rows against 128 positions at a
// time: drafts of several tokens, chunks of a prompt.  Positions are the MMA's 128 rows and query rows
// its columns, so that what belongs to a position (page, codes, scales, validity) is one thread's own, and
// few query rows still give every thread work.  One warpgroup converts, one does the softmax:
//
//   1. K: a converting thread writes its row's codes to shared memory as fp16 (a nibble in place is the
//      subnormal q * 2^-24, one place up q * 2^-20; the factor 16 is in Q), and its biases as 16 more
//      columns against three fp16 terms of each group's sum of Q.  tcgen05.mma sums each group into
//      columns of its own in tensor memory, and the biases into more.
//   2. V: the row as RN_fp16(s q + b) (what qmm_dequantize gives); where that passes fp16's range, 2^-5 times it,
//      and the position's P 2^5 times.
//   3. A softmax thread reads its position's sums: x = f * (bias + sum over groups of s * sum) - ref, all
//      fp32 (the product rounded before ref comes off, so that the largest x lies between 0 and 8 however large
//      the scores are), P = 2^x, and keeps its share of the rows' sums l in registers; P goes to shared memory as
//      fp16 (for fp16 outputs as two terms, so that V's rounding is the only one before the output's).
//   4. O^T += V^T P: V's rows as they are stored are the transposed (MN-major) operand, and so is P.
//
// References are moved only when some x passes 15 (fp16 holds P up to 2^16): then so that the largest x of the
// tile is 8 (redux over the warps' lanes), with O rescaled in tensor memory; fp16 is exact to 2^-11 down to 2^-22
// of the largest P (100,000 positions of 2^-23.4 each lost a third of their part with it at 1).
// K of the next tile is converted and its scores are under way while this tile's softmax runs; two blocks an SM fill
// what waits are left.
// 1,024 tokens of 32 heads over 8,191 positions of 128: 412 us, 0.31 PFLOP/s; bound by the two warpgroups'
// waits for each other (issue slots 44% busy, tensor pipe 16%), not by the MMAs.
// Every wait on a barrier is bounded; a block whose wait runs out goes through its barriers and says so.
// Work and joins are those of qmm_attn.cu, in units of 128 positions.
#include <climits>

#include "qmm_attn.cuh"
#include "sm100.cuh"

namespace qmm_impl {
namespace {

using namespace sm100;

__device__ unsigned g_tc_attn_errors;  // bit 0: a wait ran out; bit 1: a page or position outside the cache

constexpr int kPos = kAttnTcUnit;          // positions a tile
constexpr int kTcThreads = 2 * kPos;       // a warpgroup for the softmax, one for the conversions
constexpr float kMaxX = 15.f, kAimX = 8.f;  // where references move, and what the largest x is then
constexpr int kRegsS = 152, kRegsC = 104;  // registers a thread of the two, of 128 each at the launch: their sum is 256

template <int D, int GRP, int N>
struct TcAttnFmt {
    static constexpr int NG = D / GRP;
    static constexpr int WORDS = D / 8;                // 32-bit words of codes a row: 16-byte pieces as fp16
    static constexpr int CH = 8;                       // query rows read from tensor memory at a time
    // whether the two warpgroups share their registers out anew
    static constexpr bool SPLIT = N > 32;
    // Whether all of K's codes go into their operand one place up (2^-20): products are aligned by the exponents'
    // fields, where a subnormal's is 2^-14, so that beside q's largest those below 2^-15 (codes in place) or 2^-19
    // are cut off.  fp16's 11 bits of q need it (lse of rows that see one position 1.3e-6 off, or 2e-7; 1% more time
    // for the shifts), and run with 32 rows alone; bf16's 8 do not
    static constexpr bool HIGH = N <= 32;
    static constexpr int PANELS = D / 64;              // 128-byte wide panels of a row of D fp16
    static constexpr int PANEL = kPos * 128;           // bytes of a panel of K or V
    // V first: where D = 64, V's MMA reads a second panel behind it, whose rows of O^T nobody looks at
    static constexpr int OFF_V = 0;
    static constexpr int OFF_K = PANELS * PANEL;
    static constexpr int OFF_P = 2 * PANELS * PANEL;   // P; with N <= 32 its second term in the rows' other halves
    static constexpr int OFF_Q = OFF_P + PANEL;
    static constexpr int QPANEL = N * 128;
    static constexpr int OFF_KB = OFF_Q + PANELS * QPANEL;  // biases: 16 columns, [2][kPos] 16-byte pieces
    static constexpr int OFF_QB = OFF_KB + kPos * 32;
    static constexpr int OFF_F = OFF_QB + N * 32;      // per row: factor of the sums; minus the reference
    static constexpr int OFF_NREF = OFF_F + N * 4;
    static constexpr int OFF_LIM = OFF_F + N * 8;
    static constexpr int OFF_BITS = OFF_LIM + N * 4;
    static constexpr int OFF_OUT = OFF_BITS + N * 8;   // per row: where its output is, in elements
    static constexpr int OFF_RED = OFF_OUT + N * 8;    // per warp and row
    static constexpr int OFF_POS = OFF_RED + 4 * N * 4;    // per position, for two tiles: K's scales, what is the matter
    static constexpr int OFF_BAR = OFF_POS + 2 * kPos * (NG + 1) * 4;
    static constexpr int OFF_RUN = OFF_BAR + 64;       // this run and the next
    static constexpr int OFF_NAN = OFF_RUN + 2 * 96;   // per group, bit per row: it sees a V that is not finite
    static constexpr int USED = OFF_NAN + NG * 8;
    static constexpr int SMEM = (USED > 80 * 1024 ? USED : 80 * 1024) + 1024;  // two blocks an SM at most; alignment
    // tensor memory columns: group sums, biases, O^T
    static constexpr int COL_B = NG * N, COL_O = COL_B + N;
    static constexpr int COLS = COL_O + N <= 64 ? 64 : COL_O + N <= 128 ? 128 : 256;
    static_assert(COL_O + N <= 256, "two blocks' columns do not fit tensor memory");
    static constexpr int SLOT = N * (D + 2);
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return smem_desc_sw128(addr, sbo) & ~(uint64_t(0x3FFF) << 16) | uint64_t((lbo >> 4) & 0x3FFF) << 16;
}
// D[tmem] (+)= A[smem] * B[smem], fp16 in, fp32 sums
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[8]) { tmem_ld_32x32b_x8(taddr, v); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) { tmem_st_32x32b_x8(taddr, v); }
// Pairs of fp32 in one register pair: two results an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ uint64_t bits2(uint32_t a, uint32_t b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Barriers of one warpgroup (1: conversions, 2: softmax).
__device__ __forceinline__ void group_sync(int id) {
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_or(int id, bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred.aligned q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(uint32_t(v))
        : "memory");
    return r != 0;
}
template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// What is the matter with a position (OFF_POS): it is not there; its V is past fp16, and kept 2^-5 times what it
// is; its V is zeroed, because not finite, in group j (kOdd << j).
constexpr uint32_t kAbsent = 1, kFar = 2, kOdd = 4;
constexpr int kFarShift = 5;  // 15 |s| + |b| is below 2^20

template <int D, int GRP, int N>
__global__ void __launch_bounds__(kTcThreads, 2) attn_tc_kernel(const __grid_constant__ AttnArgs a) {
    using F = TcAttnFmt<D, GRP, N>;
    constexpr int NG = F::NG, WORDS = F::WORDS, CH = F::CH, HR = N > 32 ? 32 : N;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + (1024 - (smem_addr(raw_smem) & 1023)) % 1024;  // swizzle atoms
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int me = tid & (kPos - 1);     // this thread's position of a tile
    const bool softmax = tid < kPos;
    // full: scores of a tile are in tensor memory, K's place is free, and OFF_POS is written; free: the scores
    // have been read; both: V and P are in place; done: O is up to date, V's and P's places are free
    const uint32_t bar_full = sbase + F::OFF_BAR, bar_free = bar_full + 8, bar_both = bar_full + 16, bar_done = bar_full + 24;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(smem + F::OFF_BAR + 32);
    int* const flag = reinterpret_cast<int*>(smem + F::OFF_BAR + 36);

    grid_dependency_wait();

    constexpr AttnCut cut{N, kPos, 1, 2};
    AttnPlan pl;
    int x_end;
    Run* cur = reinterpret_cast<Run*>(smem + F::OFF_RUN);
    Run* next = cur + 1;
    bool bad = false;
    {
        const int got = plan_block(a, cut, lane, tid == 0, &pl, &x_end, cur, &bad);
        if (got < 0 && blockIdx.x == 0 && tid == 0) atomicOr(&g_tc_attn_errors, 2u);
        if (got <= 0) return;
    }
    if (tid == 0) {
        mbar_init(bar_full, kPos + 1);
        mbar_init(bar_free, kPos);
        mbar_init(bar_both, kTcThreads);
        mbar_init(bar_done, 1);
        fence_mbar_init();
    }
    if (w == 0) {
        tmem_alloc(smem_addr(tmem_at), F::COLS);
        tmem_relinquish();
    }
    // columns of the bias operands that no group uses are zeros
    for (int i = tid; i < kPos * 8; i += kTcThreads) reinterpret_cast<uint32_t*>(smem + F::OFF_KB)[i] = 0;
    for (int i = tid; i < N * 8; i += kTcThreads) reinterpret_cast<uint32_t*>(smem + F::OFF_QB)[i] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now: a following kernel's blocks may take tensor memory as soon as they are resident
    grid_dependents_launch();
    const uint32_t tmem = *tmem_at;
    const uint32_t tmem_row = tmem + (uint32_t((w & 3) * 32) << 16);  // this warp's lanes
    constexpr uint32_t idesc = idesc_f16_f32(128, N);
    constexpr uint32_t idesc_t = idesc | 1u << 15 | 1u << 16;   // both operands MN-major
    uint32_t tile = 0;  // tiles so far: the barriers' phases
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t of) {  // until tile number `of` of the block has passed
        if (dead || mbar_try_wait(bar, of & 1)) return;
        const long long deadline = clock64() + 4000000000ll;  // about two seconds
        while (!mbar_try_wait(bar, of & 1))
            if (clock64() > deadline) {
                dead = true;
                break;
            }
    };
    // first unit at or behind u that some row sees a position of; n if none
    auto seek = [&](const Run* r, int u) {
        if (r->lo > r->t0 + kPos * (u + 1) - 1) u = (r->lo - r->t0) / kPos;
        return r->t0 + kPos * u < r->hi && u < r->n ? u : r->n;
    };
    // panel-swizzled place of 16-byte piece p of row r
    auto place = [](int row, int p, int panel_bytes) { return (p >> 3) * panel_bytes + row * 128 + (((p & 7) ^ (row & 7)) << 4); };
    uint32_t own[8];  // 16-byte pieces of this thread's position
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] = sbase + place(me, i, 0);
    auto put = [&](int off, int p, uint4 v) { sts_v4(own[p & 7] + off + (p >> 3) * F::PANEL, v); };

    // ---- Q of the current run: K-major panels, scaled by a power of two per row (as in qmm_attn.cu)
    auto stage_q = [&]() {
        if (tid < 2 * NG) reinterpret_cast<uint32_t*>(smem + F::OFF_NAN)[tid] = 0;
        auto load = [&](int i) {
            const int qr = cur->row_lo + i / WORDS, tok = qr / a.group_heads, hg = qr - tok * a.group_heads;
            if (i / WORDS >= cur->rows) return make_uint4(0u, 0u, 0u, 0u);
            const uint16_t* src = a.q + int64_t(cur->row0 + tok) * a.q_ts + int64_t(cur->h * a.group_heads + hg) * a.q_hs + i % WORDS * 8;
            if (a.q_vec) return *reinterpret_cast<const uint4*>(src);
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = uint32_t(src[2 * j]) | uint32_t(src[2 * j + 1]) << 16;
            return make_uint4(u[0], u[1], u[2], u[3]);
        };
        uint4 raw = load(tid);
#pragma unroll 1
        for (int i = tid; i < N * WORDS; i += kTcThreads) {
            const int row = i / WORDS, p8 = i % WORDS;
            const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
            raw = load(i + kTcThreads);  // zeros past the last row
            float v[8];
            float mx = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = a.is_bf16 ? bf16lo_to_f32(rw[j]) : half_lo(rw[j]);
                v[2 * j + 1] = a.is_bf16 ? bf16hi_to_f32(rw[j]) : half_hi(rw[j]);
                mx = fmaxf(mx, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
            }
#pragma unroll
            for (int o = 1; o < WORDS; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
            int e = 0;
            if (mx > 0.f && mx < INFINITY) e = 14 + 127 - int(__float_as_uint(mx) >> 23);
            if (e > 126) e = 126;
            const float up = exp2i(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= up, sum += v[j];
#pragma unroll
            for (int o = 1; o < GRP / 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
            // the order of a code word's pairs: 0 4, 1 5 (codes * 2^-20), 2 6, 3 7 (codes * 2^-20)
            uint4 f;
            f.x = f32x2_to_f16x2(v[0], v[4]);
            constexpr float k1 = F::HIGH ? 1.f : 0.0625f;
            f.y = f32x2_to_f16x2(v[1] * k1, v[5] * k1);
            f.z = f32x2_to_f16x2(v[2], v[6]);
            f.w = f32x2_to_f16x2(v[3] * k1, v[7] * k1);
            sts_v4(sbase + F::OFF_Q + place(row, p8, F::QPANEL), f);
            if (p8 % (GRP / 8) == 0) {
                const float s0 = sum * (0x1p-24f * kSumUp), h0 = __half2float(__float2half_rn(s0));
                const float s1 = s0 - h0, h1 = __half2float(__float2half_rn(s1));
                const float h[3] = {h0, h1, s1 - h1};
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int c = 3 * (p8 / (GRP / 8)) + k;
                    *reinterpret_cast<__half*>(smem + F::OFF_QB + (c >> 3) * (N * 16) + (row >> 3) * 128 + (row & 7) * 16 + (c & 7) * 2) =
                        __float2half_rn(h[k]);
                }
            }
            if (p8 == 0) {
                const int qr = cur->row_lo + row, tok = qr / a.group_heads, head = cur->h * a.group_heads + qr - tok * a.group_heads;
                *reinterpret_cast<int64_t*>(smem + F::OFF_OUT + row * 8) = int64_t(cur->row0 + tok) * a.o_ts + int64_t(head) * a.o_hs;
                *reinterpret_cast<float*>(smem + F::OFF_F + row * 4) = a.scale_log2 * (16777216.f / kSumUp) * exp2i(-e);
                *reinterpret_cast<float*>(smem + F::OFF_NREF + row * 4) = -kNoRef;
                *reinterpret_cast<int*>(smem + F::OFF_LIM + row * 4) = row < cur->rows ? cur->start + tok : INT_MAX;
                *reinterpret_cast<int64_t*>(smem + F::OFF_BITS + row * 8) =
                    a.tree != nullptr && row < cur->rows ? a.tree[cur->row0 + tok] : -1;
            }
        }
        fence_async_smem();
    };

    if (!softmax) {
        // ================================================= conversions: K and V of a position a thread
        if constexpr (F::SPLIT) regs_down<kRegsC>();
        uint4 kr[WORDS / 4], vr[WORDS / 4];
        uint16_t ksr[NG], kbr[NG], vsr[NG], vbr[NG];
        int page = -1, in_page = 0;
        int64_t row = -1;  // of the cache, for the tile that is fetched; -1: not there
        auto look = [&](const Run* r, int u) {  // the page, a tile ahead of the rows
            const int t = r->t0 + kPos * u + me;
            const int col = t / a.page;
            in_page = t - col * a.page;
            page = u < r->n && t < r->hi ? a.table[int64_t(r->b) * a.table_stride + col] : -1;
        };
        auto fetch_k = [&](const Run* r, int u) {
            const int t = r->t0 + kPos * u + me;
            const bool in = u < r->n && t < r->hi, there = in && page >= 0 && page < a.pages;
            bad |= in && !there;
            row = there ? (int64_t(page) * a.kv_heads + r->h) * a.page + in_page : -1;
            if (there) {
                const uint4* k = reinterpret_cast<const uint4*>(a.kc + row * (D / 2));
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i) kr[i] = __ldg(k + i);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    ksr[j] = __ldg(a.ks + row * NG + j), kbr[j] = __ldg(a.kb + row * NG + j);
                    vsr[j] = __ldg(a.vs + row * NG + j), vbr[j] = __ldg(a.vb + row * NG + j);
                }
            }
        };
        auto fetch_v = [&]() {  // of the row that fetch_k found
            if (row >= 0) {
                const uint4* v = reinterpret_cast<const uint4*>(a.vc + row * (D / 2));
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i) vr[i] = __ldg(v + i);
            }
        };
        // V^T P of tile number `of`: the first of its run overwrites O
        auto sums = [&](uint32_t of, bool add) {
            if (tid == kPos + 32) {
                wait(bar_both, of);
                tc_fence_after();
                for (int term = 0; term < (N > 32 || a.is_bf16 ? 1 : 2); ++term)
#pragma unroll
                    for (int k = 0; k < kPos / 16; ++k)
                        umma_f16_ss(tmem + F::COL_O, desc_sw128(sbase + F::OFF_V + k * 2048, F::PANEL, 1024),
                                    desc_sw128(sbase + F::OFF_P + term * 64 + k * 2048, F::PANEL, 1024), idesc_t,
                                    add || term || k);
                umma_commit(bar_done);
            }
            __syncwarp();
        };
        int u = seek(cur, 0);
        look(cur, u);
        fetch_k(cur, u);
        fetch_v();
        look(cur, seek(cur, u + 1));
        while (true) {
            stage_q();
            __syncthreads();
            uint32_t in_run = 0;  // tiles of this run so far
            while (u < cur->n) {
                const bool there = row >= 0;
                const bool masked = !(cur->t0 + kPos * u >= cur->full_lo && cur->t0 + kPos * (u + 1) <= cur->full_hi);
                const int u_next = seek(cur, u + 1);
                // V's constants: rows that are not there are zeros.  Where a tile is masked, a group that is not finite
                // is zeros too; the softmax notes which query rows see it, and those become NaN at the end
                uint32_t vsb[NG], state = there ? 0u : kAbsent;
                bool odd = false;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    vsb[j] = there ? uint32_t(vsr[j]) | uint32_t(vbr[j]) << 16 : 0u;
                    // 15 s + b, the value furthest from b, is infinite or NaN (so it is if s or b are)
                    odd |= (hfma2(vsb[j], 0x4B804B80u, vsb[j] >> 16) & 0x7C00u) == 0x7C00u;
                }
                if (odd) {
                    // Finite constants whose values pass fp16's range: V counts 2^-5 times, its probability 2^5 times (its
                    // other groups may lose what lies below 2^-16)
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        const bool inf = (((vsb[j] & 0x7C007C00u) + 0x04000400u) & 0x80008000u) != 0;  // an exponent of ones
                        if (!inf && (hfma2(vsb[j], 0x4B804B80u, vsb[j] >> 16) & 0x7C00u) == 0x7C00u) state |= kFar;
                        if (masked && inf) vsb[j] = 0, state |= kOdd << j;
                    }
                    if (state & kFar)
#pragma unroll
                        for (int j = 0; j < NG; ++j) vsb[j] = hfma2(vsb[j], 0x28002800u, 0x80008000u);  // 2^-5; -0 added
                }
                // ---- K, and the scores' MMAs
                if (tile) wait(bar_full, tile - 1);
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    const uint4 q = kr[i >> 2];
                    const uint32_t c = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w, y = c >> 8;
                    if constexpr (F::HIGH) put(F::OFF_K, i, make_uint4((c << 4) & 0x00F000F0u, c & 0x00F000F0u, (c >> 4) & 0x00F000F0u, y & 0x00F000F0u));
                    else put(F::OFF_K, i, make_uint4(c & 0x000F000Fu, c & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u));
                }
                {  // each group's bias three times, in columns 3 j, 3 j + 1, 3 j + 2
                    uint32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 3 * NG; ++k) c[k >> 1] |= there ? uint32_t(kbr[k / 3]) << (16 * (k & 1)) : 0u;
                    sts_v4(sbase + F::OFF_KB + me * 16, make_uint4(c[0], c[1], c[2], c[3]));
                    if (3 * NG > 8) sts_v4(sbase + F::OFF_KB + kPos * 16 + me * 16, make_uint4(c[4], c[5], c[6], c[7]));
                }
                uint32_t* const pos = reinterpret_cast<uint32_t*>(smem + F::OFF_POS) + (tile & 1) * kPos * (NG + 1) + me;
                pos[NG * kPos] = state;
#pragma unroll
                for (int j = 0; j < NG; ++j) pos[j * kPos] = __float_as_uint(__half2float(__ushort_as_half(ksr[j])) * (F::HIGH ? kSumUp / 16 : kSumUp));
                fence_async_smem();
                mbar_arrive(bar_full);
                group_sync(1);
                if (tid == kPos) {
                    if (tile) wait(bar_free, tile - 1);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t o = (k & 3) * 32;
                        umma_f16_ss(tmem + (k * 16 / GRP) * N, smem_desc_sw128(sbase + F::OFF_K + (k >> 2) * F::PANEL + o, 1024),
                                    smem_desc_sw128(sbase + F::OFF_Q + (k >> 2) * F::QPANEL + o, 1024), idesc, k * 16 % GRP != 0);
                    }
                    umma_f16_ss(tmem + F::COL_B, smem_desc_noswz(sbase + F::OFF_KB, kPos * 16, 128),
                                smem_desc_noswz(sbase + F::OFF_QB, N * 16, 128), idesc, 0);
                    umma_commit(bar_full);
                }
                __syncwarp();
                if (u_next < cur->n) {
                    fetch_k(cur, u_next);
                    look(cur, seek(cur, u_next + 1));
                }
                // ---- the last tile's sums (whose V is in the way), then V
                if (in_run) sums(tile - 1, in_run > 1);
                if (tile) wait(bar_done, tile - 1);
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    const uint4 q = vr[i >> 2];
                    const uint32_t c = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w, y = c >> 8;
                    const uint32_t sb = vsb[i * 8 / GRP], s = __byte_perm(sb, 0, 0x1010), b = __byte_perm(sb, 0, 0x3232);
                    // 1024 + q and 1024 + 16 q, to q, to s q + b
                    uint4 o;
                    o.x = hfma2(hfma2((c & 0x000F000Fu) | kMagic1024x2, kOnes, kMinus1024x2), s, b);
                    o.y = hfma2(hfma2((c & 0x00F000F0u) | kMagic1024x2, 0x2C002C00u, 0xD400D400u), s, b);
                    o.z = hfma2(hfma2((y & 0x000F000Fu) | kMagic1024x2, kOnes, kMinus1024x2), s, b);
                    o.w = hfma2(hfma2((y & 0x00F000F0u) | kMagic1024x2, 0x2C002C00u, 0xD400D400u), s, b);
                    put(F::OFF_V, i, o);
                }
                fence_async_smem();
                mbar_arrive(bar_both);
                if (u_next < cur->n) fetch_v();
                ++tile, ++in_run;
                u = u_next;
            }
            if (in_run) sums(tile - 1, in_run > 1);
            // ---- the next run's first rows are on their way while the softmax warps put this one together
            const bool more = plan_run(a, pl, cut, cur->x + cur->places, x_end, cur->b, cur->before, tid == kPos, next, &bad);
            group_sync(1);
            if (more) {
                u = seek(next, 0);
                look(next, u);
                fetch_k(next, u);
                fetch_v();
                look(next, seek(next, u + 1));
            }
            __syncthreads();  // the run's sums are written
            if (cur->n != cur->units) join_item<D, N>(a, cur, tid, kTcThreads, flag);
            if (!more) break;
            __syncthreads();  // Q, the rows' constants and red are free
            Run* const was = cur;
            cur = next;
            next = was;
        }
    } else {
        // ================================================= softmax: the scores of a position a thread
        if constexpr (F::SPLIT) regs_up<kRegsS>();
        float* const red = reinterpret_cast<float*>(smem + F::OFF_RED);
        float* const nref = reinterpret_cast<float*>(smem + F::OFF_NREF);
        while (true) {
            stage_q();
            __syncthreads();
            uint64_t l[N / 2];  // pairs of rows
#pragma unroll
            for (int r = 0; r < N / 2; ++r) l[r] = pair(0.f, 0.f);
            bool any_tile = false;
            int u = seek(cur, 0);
            while (u < cur->n) {
                const int t = cur->t0 + kPos * u + me;
                const bool masked = !(cur->t0 + kPos * u >= cur->full_lo && cur->t0 + kPos * (u + 1) <= cur->full_hi);
                wait(bar_full, tile);
                tc_fence_after();
                const uint32_t* const pos = reinterpret_cast<const uint32_t*>(smem + F::OFF_POS) + (tile & 1) * kPos * (NG + 1) + me;
                const uint32_t state = pos[NG * kPos];
                uint64_t ks[NG];
#pragma unroll
                for (int j = 0; j < NG; ++j) ks[j] = bits2(pos[j * kPos], pos[j * kPos]);
                // half of the rows at a time where there are 64
#pragma unroll
                for (int h0 = 0; h0 < N; h0 += HR) {
                    uint32_t see = state & kAbsent ? 0u : 0xFFFFFFFFu;  // rows of this half that see the position
                    if (masked && see) {
                        const int d = t - cur->start;
                        see = 0;
                        if (t < cur->keys) {
#pragma unroll 1
                            for (int r = 0; r < HR; r += 4) {
                                uint32_t on = 0;
                                if (a.tree != nullptr) {
                                    const uint4 b0 = lds_v4(sbase + F::OFF_BITS + (h0 + r) * 8), b1 = lds_v4(sbase + F::OFF_BITS + (h0 + r) * 8 + 16);
                                    const uint32_t lo[4] = {b0.x, b0.z, b1.x, b1.z}, hi[4] = {b0.y, b0.w, b1.y, b1.w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        on |= (d < 0 ? 1u : d < 64 ? (d < 32 ? lo[k] >> d : hi[k] >> (d - 32)) & 1u : 0u) << k;
                                } else {
                                    const uint4 l4 = lds_v4(sbase + F::OFF_LIM + (h0 + r) * 4);
                                    const int lim[4] = {int(l4.x), int(l4.y), int(l4.z), int(l4.w)};
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        on |= uint32_t(t <= lim[k] && (a.window <= 0 || lim[k] == INT_MAX || t > lim[k] - a.window)) << k;
                                }
                                see |= on << r;
                            }
#pragma unroll 1
                            for (int j = 0; j < NG && state >= kOdd << j; ++j)
                                if (state & (kOdd << j)) atomicOr(reinterpret_cast<uint32_t*>(smem + F::OFF_NAN) + 2 * j + h0 / 32, see);
                        }
                    }
                    const bool all = see == 0xFFFFFFFFu && !(state & kFar);
                    const float up = state & kFar ? float(kFarShift) : 0.f;
                    // the sums of rows [r0, r0 + CH) of this half, as a ring of two: one is read while the other is used
                    uint32_t sb[2][CH], sg[2][NG][CH];
                    auto read = [&](int at, int r0) {
                        tmem_ld(tmem_row + F::COL_B + h0 + r0, sb[at]);
#pragma unroll
                        for (int j = 0; j < NG; ++j) tmem_ld(tmem_row + j * N + h0 + r0, sg[at][j]);
                    };
                    float p[HR];
                    for (bool moved = false;; moved = true) {
                        float top = -INFINITY;
                        read(0, 0);
#pragma unroll
                        for (int r0 = 0; r0 < HR; r0 += CH) {
                            const int at = r0 / CH & 1;
                            tc_wait_ld();
                            if (r0 + CH < HR) read(at ^ 1, r0 + CH);
#pragma unroll
                            for (int k = 0; k < CH; k += 4) {
                                const uint4 f4 = lds_v4(sbase + F::OFF_F + (h0 + r0 + k) * 4), n4 = lds_v4(sbase + F::OFF_NREF + (h0 + r0 + k) * 4);
                                const uint64_t f[2] = {bits2(f4.x, f4.y), bits2(f4.z, f4.w)}, n[2] = {bits2(n4.x, n4.y), bits2(n4.z, n4.w)};
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int i = k + 2 * h;
                                    uint64_t x = bits2(sb[at][i], sb[at][i + 1]);
#pragma unroll
                                    for (int j = 0; j < NG; ++j) x = fma2(ks[j], bits2(sg[at][j][i], sg[at][j][i + 1]), x);
                                    // rounded, as for the references, before those come off.  One by one: a packed
                                    // product and a packed sum are made one operation by the assembler
                                    const float2 y = unpair(mul2(f[h], x)), m = unpair(n[h]);
                                    p[r0 + i] = __fadd_rn(y.x, m.x), p[r0 + i + 1] = __fadd_rn(y.y, m.y);
                                }
                            }
                        }
                        if (!all) {
#pragma unroll
                            for (int r = 0; r < HR; ++r) p[r] = (see >> r) & 1 ? p[r] + up : -INFINITY;
                        }
#pragma unroll
                        for (int r = 0; r < HR; ++r) top = fmaxf(top, p[r]);
                        if (moved || !group_or(2, top > kMaxX)) break;
                        // new references: the largest x of each row becomes 0.  x - ref has lost x where there was no
                        // reference yet, so the scores are taken from the sums again
                        if (any_tile) wait(bar_done, tile - 1);  // O is rescaled
                        tc_fence_after();
#pragma unroll 1
                        for (int r0 = 0; r0 < HR; r0 += CH) {
                            read(0, r0);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < CH; ++k) {
                                float x = __uint_as_float(sb[0][k]);
#pragma unroll
                                for (int j = 0; j < NG; ++j) x = fmaf(unpair(ks[j]).x, __uint_as_float(sg[0][j][k]), x);
                                x = __fadd_rn(__fmul_rn(x, reinterpret_cast<const float*>(smem + F::OFF_F)[h0 + r0 + k]), up);
                                const float m = warp_max((see >> (r0 + k)) & 1 ? x : -INFINITY);
                                if (lane == 0) red[w * N + h0 + r0 + k] = m;
                            }
                        }
                        group_sync(2);
                        if (tid < HR) {  // the factor of what there is, in red's first row
                            const int r = h0 + tid;
                            const float was = -nref[r];
                            // rounded up: x stays below kAimX however large the scores are
                            const float now = fmaxf(was, __fadd_ru(fmaxf(fmaxf(red[r], red[N + r]), fmaxf(red[2 * N + r], red[3 * N + r])), -kAimX));
                            red[r] = ex2(was - now);
                            nref[r] = -now;
                        }
                        group_sync(2);
#pragma unroll
                        for (int r = 0; r < HR; r += 4) {
                            const uint4 f = lds_v4(sbase + F::OFF_RED + (h0 + r) * 4);
                            l[(h0 + r) / 2] = mul2(l[(h0 + r) / 2], bits2(f.x, f.y));
                            l[(h0 + r) / 2 + 1] = mul2(l[(h0 + r) / 2 + 1], bits2(f.z, f.w));
                        }
                        if (any_tile) {
#pragma unroll 1
                            for (int r0 = 0; r0 < HR; r0 += CH) {
                                uint32_t o[CH];
                                tmem_ld(tmem_row + F::COL_O + h0 + r0, o);
                                tc_wait_ld();
#pragma unroll
                                for (int k = 0; k < CH; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * red[h0 + r0 + k]);
                                tmem_st(tmem_row + F::COL_O + h0 + r0, o);
                                tc_wait_st();
                            }
                        }
                        group_sync(2);
                    }
                    if (h0 + HR == N) {
                        tc_fence_before();
                        mbar_arrive(bar_free);
                    }
                    // (l's share of a P kept 2^5 times what it is)
                    const float lw = state & kFar ? 1.f / (1 << kFarShift) : 1.f;
                    if (any_tile && h0 == 0) wait(bar_done, tile - 1);  // P's place is free
#pragma unroll
                    for (int r0 = 0; r0 < HR; r0 += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float p0 = ex2(p[r0 + 2 * k]), p1 = ex2(p[r0 + 2 * k + 1]);
                            l[(h0 + r0) / 2 + k] = fma2(pair(p0, p1), pair(lw, lw), l[(h0 + r0) / 2 + k]);
                            h[k] = f32x2_to_f16x2(p0, p1);
                            p[r0 + 2 * k] = p0, p[r0 + 2 * k + 1] = p1;
                        }
                        sts_v4(own[(h0 + r0) / 8] + F::OFF_P, make_uint4(h[0], h[1], h[2], h[3]));
                        if (N <= 32 && !a.is_bf16) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) h[k] = f32x2_to_f16x2(p[r0 + 2 * k] - half_lo(h[k]), p[r0 + 2 * k + 1] - half_hi(h[k]));
                            sts_v4(own[(4 + r0 / 8) & 7] + F::OFF_P, make_uint4(h[0], h[1], h[2], h[3]));
                        }
                    }
                }
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(bar_both);
                any_tile = true;
                ++tile;
                u = seek(cur, u + 1);
            }
#pragma unroll
            for (int r = 0; r < N; ++r) {
                float v = r & 1 ? unpair(l[r / 2]).y : unpair(l[r / 2]).x;
#pragma unroll
                for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
                if (lane == 0) red[w * N + r] = v;
            }
            group_sync(2);
            if (any_tile) wait(bar_done, tile - 1);
            tc_fence_after();
            const bool whole = cur->n == cur->units;
            float* const slot = a.part + int64_t(attn_slot(blockIdx.x, cur->c0)) * F::SLOT;
            float* const inv = reinterpret_cast<float*>(smem + F::OFF_F);  // the factors are done with
            if (tid < cur->rows) {
                const float ls = (red[tid] + red[N + tid]) + (red[2 * N + tid] + red[3 * N + tid]);
                inv[tid] = ls == 0.f ? 0.f : 1.f / ls;
                if (!whole) {
                    __stcg(slot + N * D + tid, -nref[tid]);
                    __stcg(slot + N * D + N + tid, ls);
                } else if (a.lse != nullptr) {
                    const int qr = cur->row_lo + tid, tok = qr / a.group_heads;
                    a.lse[int64_t(cur->row0 + tok) * (a.kv_heads * a.group_heads) + cur->h * a.group_heads + qr - tok * a.group_heads] =
                        lse_of(-nref[tid], ls);
                }
            }
            group_sync(2);
            // this thread's d: the codes' order within a word
            const int o8 = me & 7, d = (me & ~7) + (o8 >> 1) + (o8 & 1) * 4;
            const uint32_t* const nan = reinterpret_cast<const uint32_t*>(smem + F::OFF_NAN) + (me < D ? me / GRP * 2 : 0);
            const bool some = (nan[0] | nan[1]) != 0;
#pragma unroll 1
            for (int r0 = 0; r0 < N; r0 += CH) {
                if (r0 >= cur->rows) break;
                uint32_t o[CH];
                tmem_ld(tmem_row + F::COL_O + r0, o);
                tc_wait_ld();
                if (some) {
                    const uint32_t odd = nan[r0 >> 5] >> (r0 & 31);
#pragma unroll
                    for (int k = 0; k < CH; ++k) o[k] = (odd >> k) & 1 ? 0x7FFFFFFFu : o[k];
                }
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int r = r0 + k;
                    if (r >= cur->rows || me >= D) continue;
                    const float v = any_tile ? __uint_as_float(o[k]) : 0.f;
                    if (whole) {
                        const float out = v * inv[r];
                        a.o[*reinterpret_cast<const int64_t*>(smem + F::OFF_OUT + r * 8) + d] =
                            a.is_bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(out)) : __half_as_ushort(__float2half_rn(out));
                    } else {
                        __stcg(slot + r * D + d, v);
                    }
                }
            }
            tc_fence_before();
            if (!whole) __threadfence();
            __syncthreads();  // the run's sums are written
            if (!whole) join_item<D, N>(a, cur, tid, kTcThreads, flag);
            if (next->n == 0) break;  // planned by the other warpgroup
            __syncthreads();  // Q, the rows' constants and red are free
            Run* const was = cur;
            cur = next;
            next = was;
        }
    }
    __syncthreads();
    if (w == 0) tmem_dealloc(tmem, F::COLS);
    if (dead) atomicOr(&g_tc_attn_errors, 1u);
    if (__any_sync(kFull, bad) && lane == 0) atomicOr(&g_tc_attn_errors, 2u);
}

using TcAttnFn = void (*)(const AttnArgs);
struct TcAttnInst {
    TcAttnFn fn;
    int smem, slot, rows;
};
template <int D, int GRP, int N>
TcAttnInst inst() {
    using F = TcAttnFmt<D, GRP, N>;
    return TcAttnInst{attn_tc_kernel<D, GRP, N>, F::SMEM, F::SLOT, N};
}
// Rows at a time: 32 take half as long to start and to finish, 64 convert the cache half as often.  64 where P
// goes in one term, the groups' columns leave room, and a sequence has more than 256 rows (32 tokens of 4 heads
// of 128 over 2k positions: 45 us with 64, 27 with 32; 64 tokens over 8k: 64 and 63; 256 tokens: 140 and 171).
template <int D, int GRP>
TcAttnInst inst_n(bool wide) {
    if constexpr (D / GRP > 2) return inst<D, GRP, 32>();
    else return wide ? inst<D, GRP, 64>() : inst<D, GRP, 32>();
}
TcAttnInst instance(int d, int grp, bool wide) {
    if (d == 64) return grp == 32 ? inst_n<64, 32>(wide) : inst_n<64, 64>(wide);
    return grp == 32 ? inst_n<128, 32>(wide) : grp == 64 ? inst_n<128, 64>(wide) : inst_n<128, 128>(wide);
}

}  // namespace

bool attn_tc_supported(int head_dim) { return head_dim == 64 || head_dim == 128; }

cudaError_t launch_attn_tc(const AttnArgs& a, int query_rows, int head_dim, int group, cudaStream_t stream) {
    const TcAttnInst k = instance(head_dim, group, a.is_bf16 && query_rows > 256);
    return launch_attn_blocks(a, k.fn, kTcThreads, k.smem, k.slot, k.rows, kAttnTcUnit, 2, k.rows > 32 ? 128 : 0, stream);
}

cudaError_t attn_tc_read_and_clear_errors(unsigned* out) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_attn_errors, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_tc_attn_errors, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace qmm_impl
