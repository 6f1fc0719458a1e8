// qmm_attn_tc.cu -- attention over the paged 4-bit K/V cache for many query rows (tcgen05).
//
// The same operation as qmm_attn.cu, for tiles of up to 64 query rows against 128 positions at a
// time: drafts of several tokens, chunks of a prompt.  Positions are the MMA's 128 rows and query rows
// its columns, so that each of the block's 128 threads owns one position: what belongs to a position
// (page, codes, scales, validity) is its thread's own, and few query rows still give every thread work.
//
//   1. K: the thread writes its row's codes to shared memory as fp16 (a nibble in place is the
//      subnormal q * 2^-24, one place up q * 2^-20; the factor 16 is in Q), and its biases as 16 more
//      columns against three fp16 terms of each group's sum of Q.  tcgen05.mma sums each group into
//      columns of its own in tensor memory, and the biases into more.
//   2. V: while that runs, the row as RN_fp16(s q + b) (what qmm_dequantize gives).
//   3. The thread reads its position's sums: x = f * (bias + sum over groups of s * sum) - ref, all
//      fp32, P = 2^x, and keeps its share of the rows' sums l in registers; P goes to shared memory as
//      fp16 (for fp16 outputs as two terms, so that V's rounding is the only one before the output's).
//   4. O^T += V^T P: V's rows as they are stored are the transposed (MN-major) operand, and so is P.
//
// References are moved only when some x passes 14 (fp16 holds P up to 2^15): then by the largest x of
// the tile (redux over the warps' lanes), with O rescaled in tensor memory.  K and P share their
// shared memory (K is read before P is written).  Two blocks an SM, so that one block's
// conversions run beside the other's MMAs; the raw rows of the next tile are loaded ahead into registers.
// Work and joins are those of qmm_attn.cu, in units of 128 positions.
#include <climits>

#include "qmm_attn.cuh"
#include "sm100.cuh"

namespace qmm_impl {
namespace {

using namespace sm100;

__device__ unsigned g_tc_attn_errors;  // bit 0: a wait ran out; bit 1: a page or position outside the cache

constexpr int kPos = kAttnTcUnit;  // positions a tile, and threads a block
constexpr float kMaxX = 14.f;

template <int D, int GRP, int N>
struct TcAttnFmt {
    static constexpr int NG = D / GRP;
    static constexpr int WORDS = D / 8;                // 32-bit words of codes a row: 16-byte pieces as fp16
    static constexpr int PANELS = D / 64;              // 128-byte wide panels of a row of D fp16
    static constexpr int PANEL = kPos * 128;           // bytes of a panel of K or V
    // V first: where D = 64, V's MMA reads a second panel behind it, whose rows of O^T nobody looks at
    static constexpr int OFF_V = 0;
    static constexpr int OFF_K = PANELS * PANEL;       // K, then P (two terms)
    static constexpr int OFF_KB = OFF_K + 2 * PANEL;   // biases: 16 columns, [2][kPos] 16-byte pieces
    static constexpr int OFF_Q = OFF_KB + kPos * 32;
    static constexpr int QPANEL = N * 128;
    static constexpr int OFF_QB = OFF_Q + PANELS * QPANEL;
    static constexpr int OFF_F = OFF_QB + N * 32;      // per row: factor of the sums, reference
    static constexpr int OFF_LIM = OFF_F + N * 8;
    static constexpr int OFF_BITS = OFF_LIM + N * 4;
    static constexpr int OFF_RED = OFF_BITS + N * 8;   // per warp and row
    static constexpr int OFF_BAR = OFF_RED + 4 * N * 4;
    static constexpr int OFF_RUN = OFF_BAR + 32;       // this run and the next
    static constexpr int USED = OFF_RUN + 2 * 96;
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

template <int D, int GRP, int N>
__global__ void __launch_bounds__(kPos, 2) attn_tc_kernel(const __grid_constant__ AttnArgs a) {
    using F = TcAttnFmt<D, GRP, N>;
    constexpr int NG = F::NG, WORDS = F::WORDS;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + (1024 - (smem_addr(raw_smem) & 1023)) % 1024;  // swizzle atoms
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const uint32_t bar_s = sbase + F::OFF_BAR, bar_o = bar_s + 8;
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(smem + F::OFF_BAR + 16);
    int* const flag = reinterpret_cast<int*>(smem + F::OFF_BAR + 20);

    grid_dependency_wait();

    constexpr AttnCut cut{N, kPos, 1};
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
        mbar_init(bar_s, 1);
        mbar_init(bar_o, 1);
        fence_mbar_init();
    }
    if (w == 0) {
        tmem_alloc(smem_addr(tmem_at), F::COLS);
        tmem_relinquish();
    }
    // columns of the bias operands that no group uses are zeros
    for (int i = tid; i < kPos * 8; i += kPos) reinterpret_cast<uint32_t*>(smem + F::OFF_KB)[i] = 0;
    for (int i = tid; i < N * 8; i += kPos) reinterpret_cast<uint32_t*>(smem + F::OFF_QB)[i] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // only now: a following kernel's blocks may take tensor memory as soon as they are resident
    grid_dependents_launch();
    const uint32_t tmem = *tmem_at;
    const uint32_t tmem_row = tmem + (uint32_t(w * 32) << 16);  // this warp's lanes
    constexpr uint32_t idesc = idesc_f16_f32(128, N);
    constexpr uint32_t idesc_t = idesc | 1u << 15 | 1u << 16;   // both operands MN-major
    uint32_t par_s = 0, par_o = 0;
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t& parity) {
        if (!dead && !mbar_wait(bar, parity, clock64() + 4000000000ll)) dead = true;  // about two seconds
        parity ^= 1;
    };

    // ---- this thread's position of the next tile: raw rows in registers
    uint4 kr[WORDS / 4], vr[WORDS / 4];
    uint16_t ksr[NG], kbr[NG], vsr[NG], vbr[NG];
    bool there = false;
    auto fetch = [&](const Run* r, int u) {  // unit u of the run
        const int t = r->t0 + kPos * u + tid;
        there = false;
        if (u < r->n && t < r->hi && t >= 0) {
            const int col = t / a.page, page = a.table[int64_t(r->b) * a.table_stride + col];
            there = page >= 0 && page < a.pages;
            bad |= !there;
            if (there) {
                const int64_t row = (int64_t(page) * a.kv_heads + r->h) * a.page + (t - col * a.page);
                const uint4* k = reinterpret_cast<const uint4*>(a.kc + row * (D / 2));
                const uint4* v = reinterpret_cast<const uint4*>(a.vc + row * (D / 2));
#pragma unroll
                for (int i = 0; i < WORDS / 4; ++i) kr[i] = __ldg(k + i), vr[i] = __ldg(v + i);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    ksr[j] = __ldg(a.ks + row * NG + j), kbr[j] = __ldg(a.kb + row * NG + j);
                    vsr[j] = __ldg(a.vs + row * NG + j), vbr[j] = __ldg(a.vb + row * NG + j);
                }
            }
        }
    };
    // first unit at or behind u that some row sees a position of; n if none
    auto seek = [&](const Run* r, int u) {
        if (r->lo > r->t0 + kPos * (u + 1) - 1) u = (r->lo - r->t0) / kPos;
        return r->t0 + kPos * u < r->hi ? u : r->n;
    };
    // panel-swizzled place of 16-byte piece p of row r
    auto place = [](int row, int p, int panel_bytes) { return (p >> 3) * panel_bytes + row * 128 + (((p & 7) ^ (row & 7)) << 4); };

    int u = seek(cur, 0);
    fetch(cur, u);
    while (true) {
        // ---- Q: K-major panels, scaled by a power of two per row (as in qmm_attn.cu)
        for (int i = tid; i < N * WORDS; i += kPos) {
            const int row = i / WORDS, p8 = i % WORDS;
            const int qr = cur->row_lo + row, tok = qr / a.group_heads, hg = qr - tok * a.group_heads;
            uint32_t rw[4] = {0, 0, 0, 0};
            if (row < cur->rows) {
                const uint16_t* src = a.q + int64_t(cur->row0 + tok) * a.q_ts + int64_t(cur->h * a.group_heads + hg) * a.q_hs + p8 * 8;
                if (a.q_vec) {
                    const uint4 x = *reinterpret_cast<const uint4*>(src);
                    rw[0] = x.x, rw[1] = x.y, rw[2] = x.z, rw[3] = x.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) rw[j] = uint32_t(src[2 * j]) | uint32_t(src[2 * j + 1]) << 16;
                }
            }
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
            f.y = f32x2_to_f16x2(v[1] * 0.0625f, v[5] * 0.0625f);
            f.z = f32x2_to_f16x2(v[2], v[6]);
            f.w = f32x2_to_f16x2(v[3] * 0.0625f, v[7] * 0.0625f);
            sts_v4(sbase + F::OFF_Q + place(row, p8, F::QPANEL), f);
            if (p8 % (GRP / 8) == 0) {
                const float s0 = sum * 0x1p-24f, h0 = __half2float(__float2half_rn(s0));
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
                *reinterpret_cast<float2*>(smem + F::OFF_F + row * 8) = make_float2(a.scale_log2 * 16777216.f * exp2i(-e), kNoRef);
                *reinterpret_cast<int*>(smem + F::OFF_LIM + row * 4) = row < cur->rows ? cur->start + tok : INT_MAX;
                *reinterpret_cast<int64_t*>(smem + F::OFF_BITS + row * 8) =
                    a.tree != nullptr && row < cur->rows ? a.tree[cur->row0 + tok] : -1;
            }
        }
        float l[N];
#pragma unroll
        for (int r = 0; r < N; ++r) l[r] = 0.f;
        bool any_tile = false;

        while (u < cur->n) {
            const int t = cur->t0 + kPos * u + tid;
            const bool mine = there;
            const bool masked = !(cur->t0 + kPos * u >= cur->full_lo && cur->t0 + kPos * (u + 1) <= cur->full_hi);
            float ks[NG];
            // ---- K to shared memory (P of the last tile was there)
            if (any_tile) wait(bar_o, par_o);
#pragma unroll
            for (int j = 0; j < NG; ++j) ks[j] = __half2float(__ushort_as_half(ksr[j]));
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint4 q = kr[i >> 2];
                const uint32_t c = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w, y = c >> 8;
                sts_v4(sbase + F::OFF_K + place(tid, i, F::PANEL),
                       make_uint4(c & 0x000F000Fu, c & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u));
            }
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int c = 3 * j + k;
                    *reinterpret_cast<uint16_t*>(smem + F::OFF_KB + (c >> 3) * (kPos * 16) + tid * 16 + (c & 7) * 2) = mine ? kbr[j] : 0;
                }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = (k & 3) * 32;
                    umma_f16_ss(tmem + (k * 16 / GRP) * N, smem_desc_sw128(sbase + F::OFF_K + (k >> 2) * F::PANEL + o, 1024),
                                smem_desc_sw128(sbase + F::OFF_Q + (k >> 2) * F::QPANEL + o, 1024), idesc, k * 16 % GRP != 0);
                }
                umma_f16_ss(tmem + F::COL_B, smem_desc_noswz(sbase + F::OFF_KB, kPos * 16, 128),
                            smem_desc_noswz(sbase + F::OFF_QB, N * 16, 128), idesc, 0);
                umma_commit(bar_s);
            }
            // ---- V to shared memory, dequantized; rows that are not there are zeros.  Where a tile is masked,
            // a row that is not finite is zeros too, and rows that see it become NaN through their score
            bool odd = false;
#pragma unroll
            for (int j = 0; j < NG; ++j) odd |= (vsr[j] & 0x7C00) == 0x7C00 || (vbr[j] & 0x7C00) == 0x7C00;
            const bool zero = !mine || (masked && odd);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint4 q = vr[i >> 2];
                const uint32_t c = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w, y = c >> 8;
                const uint32_t s = vsr[i * 8 / GRP] * 0x10001u, b = vbr[i * 8 / GRP] * 0x10001u;
                // 1024 + q and 1024 + 16 q, to q, to s q + b
                uint4 o;
                o.x = hfma2(hfma2((c & 0x000F000Fu) | kMagic1024x2, kOnes, kMinus1024x2), s, b);
                o.y = hfma2(hfma2((c & 0x00F000F0u) | kMagic1024x2, 0x2C002C00u, 0xD400D400u), s, b);
                o.z = hfma2(hfma2((y & 0x000F000Fu) | kMagic1024x2, kOnes, kMinus1024x2), s, b);
                o.w = hfma2(hfma2((y & 0x00F000F0u) | kMagic1024x2, 0x2C002C00u, 0xD400D400u), s, b);
                if (zero) o = make_uint4(0, 0, 0, 0);
                sts_v4(sbase + F::OFF_V + place(tid, i, F::PANEL), o);
            }
            // ---- the next tile's rows are on their way from here on
            const int u_next = seek(cur, u + 1);
            if (u_next < cur->n) fetch(cur, u_next);
            // ---- probabilities
            wait(bar_s, par_s);
            tc_fence_after();
            float p[N];
            while (true) {
                float top = -INFINITY;
#pragma unroll
                for (int r0 = 0; r0 < N; r0 += 16) {
                    uint32_t sb[16], sg[NG][16];
                    tmem_ld16(tmem_row + F::COL_B + r0, sb);
#pragma unroll
                    for (int j = 0; j < NG; ++j) tmem_ld16(tmem_row + j * N + r0, sg[j]);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 c = *reinterpret_cast<const float2*>(smem + F::OFF_F + (r0 + k) * 8);
                        float x = __uint_as_float(sb[k]);
#pragma unroll
                        for (int j = 0; j < NG; ++j) x = fmaf(ks[j], __uint_as_float(sg[j][k]), x);
                        p[r0 + k] = fmaf(c.x, x, -c.y);
                    }
                }
                if (masked) {
                    const bool in = mine && t < cur->keys;
                    const int d = t - cur->start;
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        bool on;
                        if (a.tree != nullptr) {
                            const int64_t bits = *reinterpret_cast<const int64_t*>(smem + F::OFF_BITS + r * 8);
                            on = d < 0 || (d < 64 && ((bits >> d) & 1));
                        } else {
                            const int lim = *reinterpret_cast<const int*>(smem + F::OFF_LIM + r * 4);
                            on = t <= lim && (a.window <= 0 || lim == INT_MAX || t > lim - a.window);
                        }
                        p[r] = on && in ? (odd ? NAN : p[r]) : -INFINITY;
                    }
                } else if (!mine) {  // a page outside the pool
#pragma unroll
                    for (int r = 0; r < N; ++r) p[r] = -INFINITY;
                }
#pragma unroll
                for (int r = 0; r < N; ++r) top = fmaxf(top, p[r]);
                if (!__syncthreads_or(top > kMaxX)) break;
                // new references: the largest x of each row becomes 0.  Sums again without a reference
                float* const red = reinterpret_cast<float*>(smem + F::OFF_RED);
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    // x - ref loses x where ref is kNoRef: the score itself is f * sums
                    p[r] = p[r] == -INFINITY ? -INFINITY : 0.f;
                }
#pragma unroll
                for (int r0 = 0; r0 < N; r0 += 16) {
                    uint32_t sb[16], sg[NG][16];
                    tmem_ld16(tmem_row + F::COL_B + r0, sb);
#pragma unroll
                    for (int j = 0; j < NG; ++j) tmem_ld16(tmem_row + j * N + r0, sg[j]);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float x = __uint_as_float(sb[k]);
#pragma unroll
                        for (int j = 0; j < NG; ++j) x = fmaf(ks[j], __uint_as_float(sg[j][k]), x);
                        x *= reinterpret_cast<const float2*>(smem + F::OFF_F)[r0 + k].x;
                        const float m = warp_max(x + p[r0 + k]);
                        if (lane == 0) red[w * N + r0 + k] = m;
                    }
                }
                __syncthreads();
                float* const fr = reinterpret_cast<float*>(smem + F::OFF_F);
                float f[N];
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    const float was = fr[2 * r + 1];
                    const float m = fmaxf(fmaxf(red[r], red[N + r]), fmaxf(red[2 * N + r], red[3 * N + r]));
                    f[r] = ex2(was - fmaxf(was, m));
                    l[r] *= f[r];
                }
                __syncthreads();
                if (tid < N) {
                    const float m = fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid]));
                    fr[2 * tid + 1] = fmaxf(fr[2 * tid + 1], m);
                }
                if (any_tile) {  // its sums are complete: waited for above
#pragma unroll
                    for (int r0 = 0; r0 < N; r0 += 16) {
                        uint32_t o[16];
                        tmem_ld16(tmem_row + F::COL_O + r0, o);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[r0 + k]);
                        tmem_st_32x32b_x16(tmem_row + F::COL_O + r0, o);
                    }
                    tc_wait_st();
                }
                __syncthreads();
            }
#pragma unroll
            for (int r0 = 0; r0 < N; r0 += 8) {
                uint4 hi, lo;
                uint32_t* const h = reinterpret_cast<uint32_t*>(&hi);
                uint32_t* const q = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float p0 = ex2(p[r0 + 2 * k]), p1 = ex2(p[r0 + 2 * k + 1]);
                    l[r0 + 2 * k] += p0, l[r0 + 2 * k + 1] += p1;
                    h[k] = f32x2_to_f16x2(p0, p1);
                    q[k] = f32x2_to_f16x2(p0 - half_lo(h[k]), p1 - half_hi(h[k]));
                }
                sts_v4(sbase + F::OFF_K + place(tid, r0 / 8, F::PANEL), hi);
                if (!a.is_bf16) sts_v4(sbase + F::OFF_K + F::PANEL + place(tid, r0 / 8, F::PANEL), lo);
            }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                for (int term = 0; term < (a.is_bf16 ? 1 : 2); ++term)
#pragma unroll
                    for (int k = 0; k < kPos / 16; ++k)
                        umma_f16_ss(tmem + F::COL_O, desc_sw128(sbase + F::OFF_V + k * 2048, F::PANEL, 1024),
                                    desc_sw128(sbase + F::OFF_K + term * F::PANEL + k * 2048, F::PANEL, 1024), idesc_t,
                                    any_tile || term || k);
                umma_commit(bar_o);
            }
            any_tile = true;
            u = u_next;
        }
        if (any_tile) wait(bar_o, par_o);
        tc_fence_after();

        // ---- the next item's first rows are on their way while this one is put together
        const int x = pl.pieces ? x_end : cur->x + cur->n;
        const bool more = x < x_end;
        if (more) {
            bad |= plan_run(a, pl, cut, x, x_end, cur->b, cur->before, false, tid == 0, next);
        }
        float* const red = reinterpret_cast<float*>(smem + F::OFF_RED);
#pragma unroll
        for (int r = 0; r < N; ++r) {
            float v = l[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == 0) red[w * N + r] = v;
        }
        __syncthreads();
        if (more) {
            u = seek(next, 0);
            fetch(next, u);
        }
        const bool whole = cur->n == cur->units;
        float* const slot = a.part + int64_t(attn_slot(blockIdx.x, cur->first)) * F::SLOT;
        // this thread's d: the codes' order within a word
        const int pos = tid & 7, d = (tid & ~7) + (pos >> 1) + (pos & 1) * 4;
        const float* const fr = reinterpret_cast<const float*>(smem + F::OFF_F);
#pragma unroll
        for (int r0 = 0; r0 < N; r0 += 16) {
            if (r0 >= cur->rows) break;
            uint32_t o[16];
            tmem_ld16(tmem_row + F::COL_O + r0, o);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int r = r0 + k;
                if (r >= cur->rows || tid >= D) continue;
                const float ls = (red[r] + red[N + r]) + (red[2 * N + r] + red[3 * N + r]);
                const float v = any_tile ? __uint_as_float(o[k]) : 0.f;
                if (whole) {
                    const int qr = cur->row_lo + r, tok = qr / a.group_heads;
                    const int head = cur->h * a.group_heads + qr - tok * a.group_heads;
                    const float out = ls == 0.f ? 0.f : v / ls;
                    uint16_t* dst = a.o + int64_t(cur->row0 + tok) * a.o_ts + int64_t(head) * a.o_hs + d;
                    *dst = a.is_bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(out)) : __half_as_ushort(__float2half_rn(out));
                    if (tid == 0 && a.lse != nullptr)
                        a.lse[int64_t(cur->row0 + tok) * (a.kv_heads * a.group_heads) + head] =
                            ls == 0.f ? -INFINITY : (fr[2 * r + 1] + lg2(ls)) * 0.693147180559945309f;
                } else {
                    __stcg(slot + r * D + d, v);
                    if (tid == 0) __stcg(slot + N * D + r, fr[2 * r + 1]), __stcg(slot + N * D + N + r, ls);
                }
            }
        }
        tc_fence_before();
        if (!whole) join_item<D, N>(a, pl, cur, tid, kPos, flag);
        if (!more) break;
        __syncthreads();  // Q, the rows' constants and red are free
        Run* const was = cur;
        cur = next;
        next = was;
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
template <int D, int GRP>
TcAttnInst inst_n(int n) {
    if constexpr (D / GRP > 2) return n == 16 ? inst<D, GRP, 16>() : inst<D, GRP, 32>();
    else return n == 16 ? inst<D, GRP, 16>() : n == 32 ? inst<D, GRP, 32>() : inst<D, GRP, 64>();
}
TcAttnInst instance(int d, int grp, int n) {
    if (d == 64) return grp == 32 ? inst_n<64, 32>(n) : inst_n<64, 64>(n);
    return grp == 32 ? inst_n<128, 32>(n) : grp == 64 ? inst_n<128, 64>(n) : inst_n<128, 128>(n);
}

}  // namespace

bool attn_tc_supported(int head_dim) { return head_dim == 64 || head_dim == 128; }

cudaError_t launch_attn_tc(const AttnArgs& in, int head_dim, int group, int64_t rows, cudaStream_t stream) {
    AttnArgs a = in;
    const TcAttnInst k = instance(head_dim, group, rows <= 16 ? 16 : rows <= 32 ? 32 : 64);
    return launch_attn_blocks(a, k.fn, kPos, k.smem, k.slot, k.rows, kAttnTcUnit, stream);
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
