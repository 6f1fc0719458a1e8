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

// ---------------------------------------------------------------- append
// One thread a word (eight values); a group's range is found by its GRP / 8 lanes.  Each step is
// the scheme of qmm_quant.cu, rounded the same way, so the bits are those of qmm_quantize (its scan
// keeps the first of equal extremes, which decides the sign of a zero: so does this one).  A group
// with an infinity or NaN, or whose scale or bias leaves fp16, is stored so that it reads as NaN.
template <int GRP>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ KvArgs a) {
    const int per = a.dim / 8;
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t row = i / per;
    const int p8 = int(i - row * per), lane = threadIdx.x & 31;
    const bool is_v = blockIdx.y != 0;
    const bool on = row < int64_t(a.tokens) * a.kv_heads;
    const int tok = on ? int(row / a.kv_heads) : a.tokens - 1, h = on ? int(row - int64_t(tok) * a.kv_heads) : 0;
    grid_dependency_wait();
    grid_dependents_launch();
    float v[8];
    {
        const uint16_t* src = is_v ? a.v + int64_t(tok) * a.v_ts + int64_t(h) * a.v_hs
                                   : a.k + int64_t(tok) * a.k_ts + int64_t(h) * a.k_hs;
        src += p8 * 8;
        uint32_t raw[4];
        if (a.vec) {
            const uint4 u = ldg_stream_v4(src);
            raw[0] = u.x, raw[1] = u.y, raw[2] = u.z, raw[3] = u.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[j] = uint32_t(src[2 * j]) | uint32_t(src[2 * j + 1]) << 16;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = a.is_bf16 ? bf16lo_to_f32(raw[j]) : __half2float(__ushort_as_half(uint16_t(raw[j])));
            v[2 * j + 1] = a.is_bf16 ? bf16hi_to_f32(raw[j]) : __half2float(__ushort_as_half(uint16_t(raw[j] >> 16)));
        }
    }
    const int b = seq_of(a.cu, a.seqs, tok);
    int64_t at = -1;
    bool bad = false;
    if (on && b < a.seqs && a.cu[b] <= tok) {  // rows in front of the first or behind the last sequence are left
        const AttnSeq s = attn_seq(a.cu[b], a.cu[b + 1], a.at[b], a.tokens, a.capacity, 1, 1, 0);
        at = cache_row(a, b, s.start + (tok - s.row0), h);
        bad = at < 0;
    }
    float lo = v[0], hi = v[0];
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (v[j] < lo) lo = v[j];
        if (v[j] > hi) hi = v[j];
        odd |= !(fabsf(v[j]) < INFINITY);
    }
#pragma unroll
    for (int o = 1; o < GRP / 8; o <<= 1) {
        const float lo2 = __shfl_xor_sync(kFull, lo, o), hi2 = __shfl_xor_sync(kFull, hi, o);
        const bool later = lane & o;  // the lanes before this one keep their value on a tie
        if (later ? !(lo < lo2) : lo2 < lo) lo = lo2;
        if (later ? !(hi > hi2) : hi2 > hi) hi = hi2;
    }
    const unsigned group_lanes = ((1u << (GRP / 8)) - 1u) << (lane & ~(GRP / 8 - 1));
    odd = (__ballot_sync(kFull, odd) & group_lanes) != 0;
    uint16_t sh = __half_as_ushort(__float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
    uint16_t bh = __half_as_ushort(__float2half_rn(lo));
    odd |= (sh & 0x7C00) == 0x7C00 || (bh & 0x7C00) == 0x7C00;
    if (odd) sh = bh = 0x7FFF;
    const float s = __half2float(__ushort_as_half(sh)), bf = __half2float(__ushort_as_half(bh));
    uint32_t word = 0;
    if (!odd && s != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int q = __float2int_rn(__fdiv_rn(__fsub_rn(v[j], bf), s));
            word |= uint32_t(clamp_int(q, 0, 15)) << (4 * j);
        }
    }
    flag_bad(bad);
    if (at < 0) return;
    (is_v ? a.vc : a.kc)[at * per + p8] = word;
    if (p8 % (GRP / 8) == 0) {
        const int64_t gi = at * (a.dim / GRP) + p8 / (GRP / 8);
        (is_v ? a.vs : a.ks)[gi] = sh;
        (is_v ? a.vb : a.kb)[gi] = bh;
    }
}

// ---------------------------------------------------------------- gather
// One thread a word: RNE_out(RN_fp32(s * q + b)), the values qmm_dequantize gives.
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ KvArgs a) {
    const int per = a.dim / 8;
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t row = i / per;
    const int p8 = int(i - row * per);
    const bool is_v = blockIdx.y != 0;
    const bool on = row < int64_t(a.tokens) * a.kv_heads;
    const int tok = on ? int(row / a.kv_heads) : a.tokens - 1, h = on ? int(row - int64_t(tok) * a.kv_heads) : 0;
    grid_dependency_wait();
    grid_dependents_launch();
    const int b = seq_of(a.cu, a.seqs, tok);
    if (!on || b >= a.seqs) return;
    const int c0 = clamp_int(a.cu[b], 0, a.tokens);
    if (tok < c0) return;
    const int64_t at = cache_row(a, b, a.at[b] + (tok - c0), h);
    uint32_t out[4] = {0, 0, 0, 0};
    if (at >= 0) {
        const uint32_t word = (is_v ? a.vc : a.kc)[at * per + p8];
        const int64_t gi = at * (a.dim / a.group) + p8 / (a.group / 8);
        const float s = __half2float(__ushort_as_half((is_v ? a.vs : a.ks)[gi]));
        const float bb = __half2float(__ushort_as_half((is_v ? a.vb : a.kb)[gi]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = __fmaf_rn(s, float((word >> (8 * j)) & 15), bb);
            const float y = __fmaf_rn(s, float((word >> (8 * j + 4)) & 15), bb);
            if (a.is_bf16) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
                out[j] = *reinterpret_cast<const uint32_t*>(&t);
            } else {
                out[j] = f32x2_to_f16x2(x, y);
            }
        }
    }
    flag_bad(at < 0);
    uint16_t* dst = is_v ? a.v_out + int64_t(tok) * a.v_ts + int64_t(h) * a.v_hs
                         : a.k_out + int64_t(tok) * a.k_ts + int64_t(h) * a.k_hs;
    *reinterpret_cast<uint4*>(dst + p8 * 8) = make_uint4(out[0], out[1], out[2], out[3]);
}

// ---------------------------------------------------------------- copy pages
// One pair of pages by gridDim.y blocks, each an even part of the six arrays' 16-byte pieces (a
// page is contiguous in each).  A pair whose target is a later pair's too is left to that one; a
// pair whose source is another pair's target has no defined answer and is skipped as an error.
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ KvArgs a, const int32_t* src,
                                                        const int32_t* dst, int pairs) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int i = blockIdx.x;
    const int from = src[i], to = dst[i];
    bool later = false, torn = false;
    for (int j = threadIdx.x; j < pairs; j += kThreads) {
        const int d = dst[j];
        later |= j > i && d == to;
        torn |= j != i && d == from;
    }
    later = __syncthreads_or(later);
    torn = __syncthreads_or(torn);
    const bool bad = from < 0 || from >= a.pages || to < 0 || to >= a.pages || (torn && from != to);
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_bad(bad);
    if (bad || later || from == to) return;
    const int64_t rows = int64_t(a.kv_heads) * a.page;
    const int64_t cp = rows * a.dim / 32, sp = rows * (a.dim / a.group) / 8;  // 16-byte pieces of a page
    const int64_t all = 2 * cp + 4 * sp;
    const int64_t p0 = all * blockIdx.y / gridDim.y, p1 = all * (blockIdx.y + 1) / gridDim.y;
    uint16_t* const arr[6] = {reinterpret_cast<uint16_t*>(a.kc), reinterpret_cast<uint16_t*>(a.vc), a.ks, a.kb, a.vs, a.vb};
    int64_t base = 0;
#pragma unroll
    for (int k = 0; k < 6; ++k) {
        const int64_t n = k < 2 ? cp : sp;
        const int64_t lo = p0 > base ? p0 - base : 0, hi = p1 - base < n ? p1 - base : n;
        const uint4* s = reinterpret_cast<const uint4*>(arr[k]) + int64_t(from) * n;
        uint4* d = reinterpret_cast<uint4*>(arr[k]) + int64_t(to) * n;
        int64_t p = lo + threadIdx.x;
        for (; p + 3 * kThreads < hi; p += 4 * kThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = s[p + j * kThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[p + j * kThreads] = v[j];
        }
        for (; p < hi; p += kThreads) d[p] = s[p];
        base += n;
    }
}

// ---------------------------------------------------------------- compact
// One block a (sequence, head): up to kKeep rows are read, then written, so rows may move over one
// another; further ones (in rising order, so they lie behind all that is written) follow.
constexpr int kKeep = 64;
__global__ void __launch_bounds__(128) compact_kernel(const __grid_constant__ KvArgs a, const int32_t* keep, int kept) {
    __shared__ uint4 codes[2 * kKeep * 8];
    __shared__ uint16_t consts[4 * kKeep * 8];
    __shared__ int64_t from[kKeep], to[kKeep];
    const int b = blockIdx.x, h = blockIdx.y, t = threadIdx.x;
    grid_dependency_wait();
    grid_dependents_launch();
    const int k0 = clamp_int(a.cu[b], 0, kept), k1 = clamp_int(a.cu[b + 1], 0, kept), first = a.at[b];
    const int vec = a.dim / 32, ng = a.dim / a.group;
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
            codes[kKeep * 8 + i] = reinterpret_cast<const uint4*>(a.vc)[from[r] * vec + p];
        }
        for (int i = t; i < n * ng; i += 128) {
            const int r = i / ng, p = i - r * ng;
            if (from[r] < 0) continue;
            const int64_t at = from[r] * ng + p;
            consts[i] = a.ks[at], consts[kKeep * 8 + i] = a.kb[at];
            consts[2 * kKeep * 8 + i] = a.vs[at], consts[3 * kKeep * 8 + i] = a.vb[at];
        }
        __syncthreads();
        for (int i = t; i < n * vec; i += 128) {
            const int r = i / vec, p = i - r * vec;
            if (from[r] < 0) continue;
            reinterpret_cast<uint4*>(a.kc)[to[r] * vec + p] = codes[i];
            reinterpret_cast<uint4*>(a.vc)[to[r] * vec + p] = codes[kKeep * 8 + i];
        }
        for (int i = t; i < n * ng; i += 128) {
            const int r = i / ng, p = i - r * ng;
            if (from[r] < 0) continue;
            const int64_t at = to[r] * ng + p;
            a.ks[at] = consts[i], a.kb[at] = consts[kKeep * 8 + i];
            a.vs[at] = consts[2 * kKeep * 8 + i], a.vb[at] = consts[3 * kKeep * 8 + i];
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

unsigned word_blocks(const KvArgs& a) {
    return unsigned((int64_t(a.tokens) * a.kv_heads * (a.dim / 8) + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(word_blocks(a), 2), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, a.group == 32 ? append_kernel<32> : a.group == 64 ? append_kernel<64> : append_kernel<128>, a);
}

cudaError_t launch_kv_gather(const KvArgs& a, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(word_blocks(a), 2), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, gather_kernel, a);
}

cudaError_t launch_kv_copy_pages(const KvArgs& a, const int32_t* src, const int32_t* dst, int pairs, cudaStream_t stream) {
    // about 16 pieces a thread, in more blocks a pair while the pairs alone do not fill the SMs
    const int64_t rows = int64_t(a.kv_heads) * a.page;
    const int64_t pieces = rows * (a.dim / 16) + rows * (a.dim / a.group) / 2;
    int64_t parts = (pieces + 16 * kThreads - 1) / (16 * kThreads);
    const int64_t fill = (148 * 4 + pairs - 1) / pairs;
    if (parts < fill) parts = fill;
    const int64_t most = (pieces + kThreads - 1) / kThreads;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    if (parts > 65535) parts = 65535;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(unsigned(pairs), unsigned(parts)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, copy_kernel, a, src, dst, pairs);
}

cudaError_t launch_kv_compact(const KvArgs& a, const int32_t* keep, int kept, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(unsigned(a.seqs), unsigned(a.kv_heads)), 128, stream, &attr);
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
