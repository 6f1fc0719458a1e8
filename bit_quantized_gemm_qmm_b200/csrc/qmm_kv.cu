// qmm_kv.cu -- the paged 4-bit K/V cache around attention: appending rows (quantize), reading
// them back (dequantize), copying pages and moving accepted draft rows together.
//
// All four move each byte once and do next to no arithmetic: they are bound by memory (large
// calls) or by the latency of a launch and two dependent loads, offsets and page table, before
// the first row can be addressed (small calls).  Every position is checked against the sequence's
// page table and every page against the pool; what fails is skipped and sets the error bit.
#include "qmm_common.cuh"
#include "qmm_internal.h"
#include "qmm_kv_plan.h"

namespace qmm_impl {
namespace {

__device__ unsigned g_kv_errors;  // bit 1: a page or position outside the cache

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;

__device__ __forceinline__ void flag_bad(bool bad) {
    if (bad) atomicOr(&g_kv_errors, 2u);
}

// The sequence that row `tok` of the token axis belongs to: the last one whose offset is <= tok.
// One round trip for up to 32 sequences: the warp's lanes look at 32 offsets each step, for the
// smallest row of the warp; the few lanes of later rows walk on from there.  seqs if none.
__device__ __forceinline__ int seq_of(const int32_t* cu, int seqs, int tok) {
    const int lane = threadIdx.x & 31;
    const int first = __reduce_min_sync(kFull, tok);
    int b = 0;  // offsets 1..seqs that are <= first
    for (int i = lane; i - lane < seqs; i += 32) {
        const unsigned le = __ballot_sync(kFull, i < seqs && cu[i + 1] <= first);
        b += __popc(le);
        if (le != kFull) break;
    }
    while (b < seqs && cu[b + 1] <= tok) ++b;
    return b;
}

// Row index (of [pages, kv_heads, page]) of a sequence's position for head h, or -1.
__device__ __forceinline__ int64_t cache_row(const KvArgs& a, int b, int pos, int h) {
    if (pos < 0 || pos >= a.capacity) return -1;
    const int col = pos / a.page;
    const int page = a.table[int64_t(b) * a.table_stride + col];
    if (page < 0 || page >= a.pages) return -1;
    return (int64_t(page) * a.kv_heads + h) * a.page + (pos - col * a.page);
}

// A thread's NW words (eight values each) of the token axis: token, head and place in the row.  Row counts
// stay below 2^28 (2^20 tokens, 256 heads), so only the number of the words needs 64 bits.
struct Words {
    int tok, h, at;  // at: first of the values
    bool on;
};
template <int NW>
__device__ __forceinline__ Words my_words(const KvArgs& a) {
    const int lg = (a.dim == 64 ? 3 : a.dim == 128 ? 4 : 5) - (NW - 1);
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int row = int(i >> lg);
    Words w;
    w.on = row < a.tokens * a.kv_heads;
    w.at = (int(i) & ((1 << lg) - 1)) * (8 * NW);
    w.tok = w.on ? row / a.kv_heads : a.tokens - 1;
    w.h = w.on ? row - w.tok * a.kv_heads : 0;
    return w;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// ---------------------------------------------------------------- append
// One thread the same one or two words of K and of V; a group's range is found by the lanes that share it.
// Two words halve what a thread spends on finding its rows; one is faster while the threads do not fill the
// GPU (8 heads of 128: 64 tokens 4.0 us against 5.5, 512 tokens 4.4 against 5.8, 8,191 tokens 23.4 against 20.9,
// which is 2.1 TB/s of rows in and codes out: issue slots are 65% busy, 24 instructions a value, DRAM 18%).
// The steps are the scheme of qmm_quant.cu, rounded the same way, so the bits are those of qmm_quantize (its
// scan keeps the first of equal extremes, which decides the sign of a zero: so does this one).  A group
// with an infinity or NaN, or whose scale or bias leaves fp16, is stored so that it reads as NaN.
struct Quantized {
    uint32_t w[2];
    uint16_t s, b;
};
template <bool BF>
__device__ __forceinline__ float value_of(uint32_t h) {
    return BF ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(uint16_t(h)));
}
template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (BF) asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int GRP, bool BF, int NW>
__device__ __forceinline__ Quantized quantize_words(const uint32_t (&raw)[4 * NW]) {
    constexpr int LANES = GRP / (8 * NW);  // that share a group
    const int lane = threadIdx.x & 31;
    // the range in 16 bits (its ends are values): least of v in the low half, least of -v in the high half
    constexpr uint32_t exps = BF ? 0x7F807F80u : 0x7C007C00u, one = BF ? 0x00800080u : 0x04000400u;
    uint32_t odd = 0, up = raw[0], down = raw[0] ^ 0x80008000u;
#pragma unroll
    for (int j = 0; j < 4 * NW; ++j) {
        odd |= (raw[j] & exps) + one;  // an exponent of ones carries into its sign's place
        up = min2<BF>(up, raw[j]), down = min2<BF>(down, raw[j] ^ 0x80008000u);
    }
    uint32_t ends = min2<BF>(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) ends = min2<BF>(ends, __shfl_xor_sync(kFull, ends, o));
    float lo = value_of<BF>(ends & 0xFFFF);
    const float hi = -value_of<BF>(ends >> 16);
    const unsigned group_lanes = ((1u << LANES) - 1u) << (lane & ~(LANES - 1));
    bool bad = (__ballot_sync(kFull, (odd & 0x80008000u) != 0) & group_lanes) != 0;
    if (__any_sync(kFull, lo == 0.f)) {
        // a zero's sign: the first of the group's zeros in order
        float z = 1.f;
#pragma unroll
        for (int j = 4 * NW - 1; j >= 0; --j) {
            const float v1 = value_of<BF>(raw[j] >> 16), v0 = value_of<BF>(raw[j] & 0xFFFF);
            z = v1 == 0.f ? v1 : z;
            z = v0 == 0.f ? v0 : z;
        }
        const unsigned with = __ballot_sync(kFull, z == 0.f) & group_lanes;
        z = __shfl_sync(kFull, z, with ? __ffs(with) - 1 : lane);
        if (lo == 0.f) lo = z;
    }
    Quantized r;
    r.s = __half_as_ushort(__float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
    r.b = __half_as_ushort(__float2half_rn(lo));
    bad |= (r.s & 0x7C00) == 0x7C00 || (r.b & 0x7C00) == 0x7C00;
    if (bad) r.s = r.b = 0x7FFF;
    const float s = __half2float(__ushort_as_half(r.s)), bf = __half2float(__ushort_as_half(r.b));
    r.w[0] = r.w[1] = 0;
    if (!bad && s != 0.f) {
        // rint(RN(d / s)) from t = d * RN(1 / s), which is within 2^-22 of d / s in relative terms: it has the
        // same nearest whole number unless it lies within 2^-12 of a half.  No code leaves [0, 15] where the
        // bias is off by less than 0.4 s (fp16's half step, 2^-11 of it or 2^-25) and the scale is a normal fp16
        // number, whose own rounding moves the last code by 15 * 2^-11 at most (a subnormal one is off by up to
        // 2^-25 whatever its size: at 2 * 2^-24 the last code may be 18).  Elsewhere the divisions themselves
        // decide, and their codes are clamped.
        const float inv = __frcp_rn(s);
        constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
        const uint64_t nb = pack2(-bf, -bf), inv2 = pack2(inv, inv), whole = pack2(kWhole, kWhole), nwhole = pack2(-kWhole, -kWhole);
        const uint64_t ninv2 = pack2(-inv, -inv);
        float off = s < 0x1p-14f || fabsf(bf) * 0x1p-11f > 0.4f * s ? 1.f : 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            uint32_t word = 0;
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const uint32_t h = raw[4 * k + j];
                const uint64_t v = BF ? pack2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u))
                                      : pack2(value_of<false>(h & 0xFFFF), value_of<false>(h >> 16));
                const uint64_t d = add_f32x2(v, nb), w = fma_f32x2(d, inv2, whole);
                const float2 e = unpack2(fma_f32x2(d, ninv2, add_f32x2(w, nwhole)));  // whole number - t
                const float2 q = unpack2(w);
                off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
                word = word * 16 + __float_as_uint(q.y);
                word = word * 16 + __float_as_uint(q.x);
            }
            // each addend was 0x4B400000 + code: the constants' sum, 0x4B400000 * 0x11111111, comes off again
            r.w[k] = word - 0x4B400000u * 0x11111111u;
        }
        if (off > 0.5f - 0.000244140625f) {
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                r.w[k] = 0;
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    const uint32_t two = j < 2 ? raw[4 * k] : j < 4 ? raw[4 * k + 1] : j < 6 ? raw[4 * k + 2] : raw[4 * k + 3];
                    const float x = value_of<BF>((two >> (16 * (j & 1))) & 0xFFFF);
                    r.w[k] |= uint32_t(clamp_int(__float2int_rn(__fdiv_rn(__fsub_rn(x, bf), s)), 0, 15)) << (4 * j);
                }
            }
        }
    }
    return r;
}

template <int GRP, bool BF, int NW>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ KvArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const Words w = my_words<NW>(a);
    const uint16_t* src[2] = {a.k + int64_t(w.tok) * a.k_ts + int64_t(w.h) * a.k_hs + w.at,
                              a.v + int64_t(w.tok) * a.v_ts + int64_t(w.h) * a.v_hs + w.at};
    uint32_t raw[2][4 * NW];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (a.vec) {
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const uint4 u = ldg_stream_v4(src[k] + 8 * j);
                raw[k][4 * j] = u.x, raw[k][4 * j + 1] = u.y, raw[k][4 * j + 2] = u.z, raw[k][4 * j + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4 * NW; ++j) raw[k][j] = uint32_t(src[k][2 * j]) | uint32_t(src[k][2 * j + 1]) << 16;
        }
    }
    const int b = seq_of(a.cu, a.seqs, w.tok);
    int64_t at = -1;
    if (w.on && b < a.seqs && a.cu[b] <= w.tok) {  // rows in front of the first or behind the last sequence are left
        const AttnSeq s = attn_seq(a.cu[b], a.cu[b + 1], a.at[b], a.tokens, a.capacity, 1, 1, kAttnUnit, 0);
        at = cache_row(a, b, s.start + (w.tok - s.row0), w.h);
        flag_bad(at < 0);
    }
    const Quantized k = quantize_words<GRP, BF, NW>(raw[0]), v = quantize_words<GRP, BF, NW>(raw[1]);
    if (at < 0) return;
    const int64_t val = at * a.dim + w.at;
    if constexpr (NW == 2) {
        *reinterpret_cast<uint2*>(a.kc + val / 8) = make_uint2(k.w[0], k.w[1]);
        *reinterpret_cast<uint2*>(a.vc + val / 8) = make_uint2(v.w[0], v.w[1]);
    } else {
        a.kc[val / 8] = k.w[0];
        a.vc[val / 8] = v.w[0];
    }
    if (w.at % GRP == 0) {
        const int64_t gi = val / GRP;
        a.ks[gi] = k.s, a.kb[gi] = k.b;
        a.vs[gi] = v.s, a.vb[gi] = v.b;
    }
}

// ---------------------------------------------------------------- gather
// One thread a word of K and of V: RNE_out(RN_fp32(s * q + b)), the values qmm_dequantize gives.
// 1.2 MB take 2.6 us, a launch and the loads that depend on one another; 27 MB 8.6 us.
__device__ __forceinline__ uint4 dequantize_word(uint32_t word, uint16_t sh, uint16_t bh, int is_bf16) {
    const float s = __half2float(__ushort_as_half(sh)), b = __half2float(__ushort_as_half(bh));
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = __fmaf_rn(s, float((word >> (8 * j)) & 15), b);
        const float y = __fmaf_rn(s, float((word >> (8 * j + 4)) & 15), b);
        if (is_bf16) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
            out[j] = *reinterpret_cast<const uint32_t*>(&t);
        } else {
            out[j] = f32x2_to_f16x2(x, y);
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ KvArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const Words w = my_words<1>(a);
    const int b = seq_of(a.cu, a.seqs, w.tok);
    if (!w.on || b >= a.seqs) return;
    const int c0 = clamp_int(a.cu[b], 0, a.tokens);
    if (w.tok < c0) return;
    const int64_t at = cache_row(a, b, a.at[b] + (w.tok - c0), w.h);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (at >= 0) {
        const int64_t val = at * a.dim + w.at;
        const int64_t gi = a.group == 32 ? val >> 5 : a.group == 64 ? val >> 6 : val >> 7;
        const uint32_t kw = a.kc[val >> 3], vw = a.vc[val >> 3];
        const uint16_t ks = a.ks[gi], kb = a.kb[gi], vs = a.vs[gi], vb = a.vb[gi];
        k = dequantize_word(kw, ks, kb, a.is_bf16);
        v = dequantize_word(vw, vs, vb, a.is_bf16);
    }
    flag_bad(at < 0);
    *reinterpret_cast<uint4*>(a.k_out + int64_t(w.tok) * a.k_ts + int64_t(w.h) * a.k_hs + w.at) = k;
    *reinterpret_cast<uint4*>(a.v_out + int64_t(w.tok) * a.v_ts + int64_t(w.h) * a.v_hs + w.at) = v;
}

// ---------------------------------------------------------------- copy pages
// One pair of pages by gridDim.y blocks, each an even part of the six arrays' 16-byte pieces (a
// page is contiguous in each), at most kCopy a thread: all of them are loaded before the pairs are
// looked through.  A pair whose target is a later pair's too is left to that one; a pair whose source
// is another pair's target has no defined answer and is skipped as an error.  1,500 pages (221 MB moved) take
// 38 us, 5.8 TB/s; 4 pages 2.5 us.
constexpr int kCopy = 9;
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ KvArgs a, const int32_t* src,
                                                        const int32_t* dst, int pairs) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int i = blockIdx.x;
    const int from = src[i], to = dst[i];
    bool bad = from < 0 || from >= a.pages || to < 0 || to >= a.pages;
    const int rows = a.kv_heads * a.page;
    const int cp = rows * (a.dim / 32), sp = rows * (a.dim / a.group) / 8;  // 16-byte pieces of a page
    const int all = 2 * cp + 4 * sp;
    const int p0 = int(int64_t(all) * blockIdx.y / gridDim.y), p1 = int(int64_t(all) * (blockIdx.y + 1) / gridDim.y);
    // where piece p of page `page` is
    auto at = [&](int p, int page) {
        const bool codes = p < 2 * cp;
        const int n = codes ? cp : sp, q = codes ? p : p - 2 * cp;
        const int k = (q >= n) + (q >= 2 * n) + (q >= 3 * n);
        uint32_t* const c = k ? a.vc : a.kc;
        uint16_t* const s = k == 0 ? a.ks : k == 1 ? a.kb : k == 2 ? a.vs : a.vb;
        return reinterpret_cast<uint4*>(codes ? static_cast<void*>(c) : static_cast<void*>(s)) + int64_t(page) * n + (q - k * n);
    };
    uint4 v[kCopy];
    if (!bad) {
#pragma unroll
        for (int j = 0; j < kCopy; ++j) {
            const int p = p0 + j * kThreads + threadIdx.x;
            if (p < p1) v[j] = *at(p, from);
        }
    }
    bool later = false, torn = false;
    for (int j = threadIdx.x; j < pairs; j += kThreads) {
        const int d = dst[j];
        later |= j > i && d == to;
        torn |= j != i && d == from;
    }
    later = __syncthreads_or(later);
    torn = __syncthreads_or(torn);
    bad |= torn && from != to;
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_bad(bad);
    if (bad || later || from == to) return;
#pragma unroll
    for (int j = 0; j < kCopy; ++j) {
        const int p = p0 + j * kThreads + threadIdx.x;
        if (p < p1) *at(p, to) = v[j];
    }
}

// ---------------------------------------------------------------- compact
// One block a (sequence, head): up to kKeep rows are read, then written, so rows may move over one
// another; further ones (in rising order, so they lie behind all that is written) follow.
// 8 drafts of 6 take 3.5 us, 256 of 64 5.6 us: offsets, page table, rows, one after another.
constexpr int kKeep = 64;
__global__ void __launch_bounds__(128) compact_kernel(const __grid_constant__ KvArgs a, const int32_t* keep, int kept) {
    extern __shared__ uint4 codes[];  // K's, then V's: [kKeep][dim / 32] pieces each; then the constants
    __shared__ int64_t from[kKeep], to[kKeep];
    const int b = blockIdx.x, h = blockIdx.y, t = threadIdx.x;
    grid_dependency_wait();
    grid_dependents_launch();
    const int k0 = clamp_int(a.cu[b], 0, kept), k1 = clamp_int(a.cu[b + 1], 0, kept), first = a.at[b];
    const int vec = a.dim / 32, ng = a.dim / a.group;
    uint4* const vcodes = codes + kKeep * vec;
    uint16_t* const consts = reinterpret_cast<uint16_t*>(vcodes + kKeep * vec);
    const int cs = kKeep * ng;
    for (int j0 = k0; j0 < k1; j0 += kKeep) {
        const int n = k1 - j0 < kKeep ? k1 - j0 : kKeep;
        if (t < n) {
            const int mine = keep[j0 + t];
            const int64_t f = mine < 0 ? -1 : cache_row(a, b, first + mine, h);
            const int64_t d = cache_row(a, b, first + (j0 - k0) + t, h);
            flag_bad(f < 0 || d < 0);
            from[t] = f < 0 || d < 0 || f == d ? -1 : f;
            to[t] = d;
        }
        __syncthreads();
        for (int i = t; i < n * vec; i += 128) {
            const int r = i / vec, p = i - r * vec;
            if (from[r] < 0) continue;
            codes[i] = reinterpret_cast<const uint4*>(a.kc)[from[r] * vec + p];
            vcodes[i] = reinterpret_cast<const uint4*>(a.vc)[from[r] * vec + p];
        }
        for (int i = t; i < n * ng; i += 128) {
            const int r = i / ng, p = i - r * ng;
            if (from[r] < 0) continue;
            const int64_t at = from[r] * ng + p;
            consts[i] = a.ks[at], consts[cs + i] = a.kb[at];
            consts[2 * cs + i] = a.vs[at], consts[3 * cs + i] = a.vb[at];
        }
        __syncthreads();
        for (int i = t; i < n * vec; i += 128) {
            const int r = i / vec, p = i - r * vec;
            if (from[r] < 0) continue;
            reinterpret_cast<uint4*>(a.kc)[to[r] * vec + p] = codes[i];
            reinterpret_cast<uint4*>(a.vc)[to[r] * vec + p] = vcodes[i];
        }
        for (int i = t; i < n * ng; i += 128) {
            const int r = i / ng, p = i - r * ng;
            if (from[r] < 0) continue;
            const int64_t at = to[r] * ng + p;
            a.ks[at] = consts[i], a.kb[at] = consts[cs + i];
            a.vs[at] = consts[2 * cs + i], a.vb[at] = consts[3 * cs + i];
        }
        __syncthreads();
    }
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = stream;
    return cfg;
}

unsigned word_blocks(const KvArgs& a, int words) {
    return unsigned((int64_t(a.tokens) * a.kv_heads * (a.dim / (8 * words)) + kThreads - 1) / kThreads);
}

}  // namespace

template <int NW>
cudaError_t append_words(const KvArgs& a, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(word_blocks(a, NW)), kThreads, stream, &attr);
    auto fn = a.is_bf16 ? (a.group == 32 ? append_kernel<32, true, NW> : a.group == 64 ? append_kernel<64, true, NW> : append_kernel<128, true, NW>)
                        : (a.group == 32 ? append_kernel<32, false, NW> : a.group == 64 ? append_kernel<64, false, NW> : append_kernel<128, false, NW>);
    return cudaLaunchKernelEx(&cfg, fn, a);
}

cudaError_t launch_kv_append(const KvArgs& a, cudaStream_t stream) {
    return word_blocks(a, 1) > 148 * 8 ? append_words<2>(a, stream) : append_words<1>(a, stream);
}

cudaError_t launch_kv_gather(const KvArgs& a, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(word_blocks(a, 1)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, gather_kernel, a);
}

cudaError_t launch_kv_copy_pages(const KvArgs& a, const int32_t* src, const int32_t* dst, int pairs, cudaStream_t stream) {
    // at most kCopy pieces a thread, in more blocks a pair while the pairs alone do not fill the SMs
    const int64_t rows = int64_t(a.kv_heads) * a.page;
    const int64_t pieces = rows * (a.dim / 16) + rows * (a.dim / a.group) / 2;
    int64_t parts = (pieces + kCopy * kThreads - 1) / (kCopy * kThreads);
    const int64_t fill = (148 * 4 + pairs - 1) / pairs, most = (pieces + kThreads - 1) / kThreads;
    if (parts < fill) parts = fill < most ? fill : most;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(unsigned(pairs), unsigned(parts)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, copy_kernel, a, src, dst, pairs);
}

cudaError_t launch_kv_compact(const KvArgs& a, const int32_t* keep, int kept, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(dim3(unsigned(a.seqs), unsigned(a.kv_heads)), 128, stream, &attr);
    cfg.dynamicSmemBytes = size_t(kKeep) * (a.dim + 8 * (a.dim / a.group));
    return cudaLaunchKernelEx(&cfg, compact_kernel, a, keep, kept);
}

cudaError_t kv_read_and_clear_errors(unsigned* out) {
    unsigned v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_errors, sizeof(v));
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_kv_errors, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace qmm_impl
