// qmm_kv_api.cu -- the C ABI of the paged 4-bit K/V cache: argument checks and launches.  The
// contracts are in include/qmm.h; everything that the host can see is checked before a launch, what
// only the device can see (lengths, offsets, pages) by the kernels.
#include <cstring>

#include "qmm_internal.h"

namespace qmm_impl {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxSeqs = 65536;
constexpr int64_t kMaxPairs = 65536;  // every block looks through all of them
constexpr int kMaxHeads = 256;

qmm_status check_cache(const qmm_kv_cache* c) {
    if (!c) return fail(QMM_ERR_INVALID_ARG, "cache is null");
    if (c->bits != 4) return fail(QMM_ERR_UNSUPPORTED, "cache bits=%d (supported: 4)", c->bits);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(QMM_ERR_UNSUPPORTED, "head_dim=%d (supported: 64, 128, 256)", c->head_dim);
    if (c->group != 32 && c->group != 64 && c->group != 128)
        return fail(QMM_ERR_UNSUPPORTED, "group=%d (supported: 32, 64, 128)", c->group);
    if (c->head_dim % c->group)
        return fail(QMM_ERR_INVALID_ARG, "head_dim=%d is not a multiple of group=%d", c->head_dim, c->group);
    if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16)
        return fail(QMM_ERR_UNSUPPORTED, "page_size=%d (a multiple of 16 up to 1024)", c->page_size);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
        return fail(QMM_ERR_UNSUPPORTED, "kv_heads=%d (1..%d)", c->kv_heads, kMaxHeads);
    if (c->pages < 1 || c->pages > INT32_MAX)
        return fail(QMM_ERR_INVALID_ARG, "pages=%lld", (long long)c->pages);
    if (c->pages * c->kv_heads > (int64_t(1) << 31) / (c->page_size / 16) - 1)
        return fail(QMM_ERR_UNSUPPORTED, "pages * kv_heads * page_size: more than 2^35 rows");
    const void* p[6] = {c->k_packed, c->k_scales, c->k_biases, c->v_packed, c->v_scales, c->v_biases};
    for (const void* q : p)
        if (!q || !aligned(q, 16)) return fail(QMM_ERR_INVALID_ARG, "the cache's arrays must be 16-byte aligned pointers");
    return QMM_OK;
}

// Sequences, and the sizes their arrays go with.  *none: nothing to do.
qmm_status check_seqs(const qmm_kv_cache* c, const qmm_kv_seqs* s, const int32_t* at, int64_t tokens, bool* none) {
    *none = false;
    if (!s) return fail(QMM_ERR_INVALID_ARG, "seqs is null");
    if (s->seqs < 0 || s->max_pages < 0 || tokens < 0)
        return fail(QMM_ERR_INVALID_ARG, "negative size: seqs=%lld max_pages=%lld tokens=%lld", (long long)s->seqs,
                    (long long)s->max_pages, (long long)tokens);
    if (s->seqs > kMaxSeqs) return fail(QMM_ERR_UNSUPPORTED, "seqs=%lld > %lld", (long long)s->seqs, (long long)kMaxSeqs);
    if (tokens > kMaxTokens) return fail(QMM_ERR_UNSUPPORTED, "tokens=%lld > %lld", (long long)tokens, (long long)kMaxTokens);
    if (s->max_pages > (int64_t(1) << 30) / c->page_size)
        return fail(QMM_ERR_UNSUPPORTED, "max_pages=%lld: more than 2^30 positions", (long long)s->max_pages);
    if (s->table_stride < s->max_pages) return fail(QMM_ERR_INVALID_ARG, "table_stride < max_pages");
    if (s->seqs == 0 || tokens == 0) {
        *none = true;
        return QMM_OK;
    }
    if (!at || !s->cu_tokens || (!s->page_table && s->max_pages > 0))
        return fail(QMM_ERR_INVALID_ARG, "null page table, lengths or offsets");
    if (!aligned(at, 4) || !aligned(s->cu_tokens, 4) || !aligned(s->page_table, 4))
        return fail(QMM_ERR_INVALID_ARG, "page table, lengths and offsets must be 4-byte aligned");
    return QMM_OK;
}

KvArgs kv_args(const qmm_kv_cache* c, const qmm_kv_seqs* s, const int32_t* at, int64_t tokens) {
    KvArgs a;
    std::memset(&a, 0, sizeof(a));
    a.kc = c->k_packed, a.vc = c->v_packed;
    a.ks = c->k_scales, a.kb = c->k_biases, a.vs = c->v_scales, a.vb = c->v_biases;
    a.pages = c->pages;
    a.page = c->page_size;
    a.dim = c->head_dim;
    a.group = c->group;
    a.kv_heads = c->kv_heads;
    a.tokens = int(tokens);
    if (s) {
        a.table = s->page_table;
        a.at = at;
        a.cu = s->cu_tokens;
        a.table_stride = s->table_stride;
        a.capacity = int(s->max_pages * c->page_size);
        a.seqs = int(s->seqs);
    }
    return a;
}

// Whether [tokens, heads] output rows of dim values do not overlap.  The rows of one index lie within the
// other's step, so every layout that comes from slicing or transposing a dense tensor passes.
bool rows_apart(int64_t tokens, int64_t heads, int64_t token_stride, int64_t head_stride, int64_t dim) {
    const __int128 ts = token_stride < 0 ? -__int128(token_stride) : token_stride;
    const __int128 hs = head_stride < 0 ? -__int128(head_stride) : head_stride;
    if (tokens <= 1) return heads <= 1 || hs >= dim;
    if (heads <= 1) return ts >= dim;
    return (hs >= dim && ts >= (heads - 1) * hs + dim) || (ts >= dim && hs >= (tokens - 1) * ts + dim);
}

qmm_status check_dtype(qmm_dtype d) {
    return d == QMM_F16 || d == QMM_BF16 ? QMM_OK : fail(QMM_ERR_INVALID_ARG, "dtype=%d", int(d));
}

}  // namespace
}  // namespace qmm_impl

using namespace qmm_impl;

extern "C" {

qmm_status qmm_kv_append(const qmm_kv_cache* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                         const void* v, int64_t v_token_stride, int64_t v_head_stride, const qmm_kv_seqs* seqs,
                         const int32_t* lens, int64_t tokens, qmm_dtype dtype, void* stream) {
    bool none;
    qmm_status s;
    if ((s = check_cache(cache)) != QMM_OK || (s = check_dtype(dtype)) != QMM_OK) return s;
    if ((s = check_seqs(cache, seqs, lens, tokens, &none)) != QMM_OK || none) return s;
    if (!k || !v || !aligned(k, 2) || !aligned(v, 2)) return fail(QMM_ERR_INVALID_ARG, "k and v must be 2-byte aligned pointers");
    KvArgs a = kv_args(cache, seqs, lens, tokens);
    a.k = static_cast<const uint16_t*>(k), a.v = static_cast<const uint16_t*>(v);
    a.k_ts = k_token_stride, a.k_hs = k_head_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    a.is_bf16 = dtype == QMM_BF16;
    a.vec = aligned(k, 16) && aligned(v, 16) && (k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8 == 0;
    return launch_result(launch_kv_append(a, static_cast<cudaStream_t>(stream)), "qmm_kv_append launch");
}

qmm_status qmm_kv_gather(const qmm_kv_cache* cache, const qmm_kv_seqs* seqs, const int32_t* starts, int64_t tokens,
                         void* k, int64_t k_token_stride, int64_t k_head_stride, void* v, int64_t v_token_stride,
                         int64_t v_head_stride, qmm_dtype dtype, void* stream) {
    bool none;
    qmm_status s;
    if ((s = check_cache(cache)) != QMM_OK || (s = check_dtype(dtype)) != QMM_OK) return s;
    if ((s = check_seqs(cache, seqs, starts, tokens, &none)) != QMM_OK || none) return s;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) ||
        (k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8 != 0)
        return fail(QMM_ERR_INVALID_ARG, "k and v must be 16-byte aligned, their strides multiples of 8 elements");
    if (!rows_apart(tokens, cache->kv_heads, k_token_stride, k_head_stride, cache->head_dim) ||
        !rows_apart(tokens, cache->kv_heads, v_token_stride, v_head_stride, cache->head_dim))
        return fail(QMM_ERR_INVALID_ARG, "rows of k or v overlap");
    KvArgs a = kv_args(cache, seqs, starts, tokens);
    a.k_out = static_cast<uint16_t*>(k), a.v_out = static_cast<uint16_t*>(v);
    a.k_ts = k_token_stride, a.k_hs = k_head_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    a.is_bf16 = dtype == QMM_BF16;
    return launch_result(launch_kv_gather(a, static_cast<cudaStream_t>(stream)), "qmm_kv_gather launch");
}

qmm_status qmm_kv_copy_pages(const qmm_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t pairs,
                             void* stream) {
    qmm_status s = check_cache(cache);
    if (s != QMM_OK) return s;
    if (pairs < 0) return fail(QMM_ERR_INVALID_ARG, "negative pairs=%lld", (long long)pairs);
    if (pairs > kMaxPairs) return fail(QMM_ERR_UNSUPPORTED, "pairs=%lld > %lld", (long long)pairs, (long long)kMaxPairs);
    if (pairs == 0) return QMM_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4))
        return fail(QMM_ERR_INVALID_ARG, "src and dst must be 4-byte aligned pointers");
    return launch_result(launch_kv_copy_pages(kv_args(cache, nullptr, nullptr, 0), src, dst, int(pairs),
                                              static_cast<cudaStream_t>(stream)),
                         "qmm_kv_copy_pages launch");
}

qmm_status qmm_kv_compact(const qmm_kv_cache* cache, const qmm_kv_seqs* seqs, const int32_t* starts, const int32_t* keep,
                          int64_t kept, void* stream) {
    bool none;
    qmm_status s;
    if ((s = check_cache(cache)) != QMM_OK) return s;
    if ((s = check_seqs(cache, seqs, starts, kept, &none)) != QMM_OK || none) return s;
    if (!keep || !aligned(keep, 4)) return fail(QMM_ERR_INVALID_ARG, "keep must be a 4-byte aligned pointer");
    return launch_result(launch_kv_compact(kv_args(cache, seqs, starts, 0), keep, int(kept),
                                           static_cast<cudaStream_t>(stream)),
                         "qmm_kv_compact launch");
}

qmm_status qmm_kv_attention(const qmm_kv_cache* cache, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            void* o, int64_t o_token_stride, int64_t o_head_stride, float* lse, const qmm_kv_seqs* seqs,
                            const int32_t* lens, int64_t tokens, int heads, float scale, int64_t window,
                            const int64_t* tree, qmm_dtype dtype, void* stream) {
    bool none;
    qmm_status s;
    if ((s = check_cache(cache)) != QMM_OK || (s = check_dtype(dtype)) != QMM_OK) return s;
    if (heads < 1 || heads > kMaxHeads) return fail(QMM_ERR_UNSUPPORTED, "heads=%d (1..%d)", heads, kMaxHeads);
    if (heads % cache->kv_heads)
        return fail(QMM_ERR_INVALID_ARG, "heads=%d is not a multiple of kv_heads=%d", heads, cache->kv_heads);
    if (window < 0) return fail(QMM_ERR_INVALID_ARG, "negative window=%lld", (long long)window);
    if (window > 0 && tree) return fail(QMM_ERR_UNSUPPORTED, "window and tree cannot be combined");
    if ((s = check_seqs(cache, seqs, lens, tokens, &none)) != QMM_OK || none) return s;
    if (!q || !aligned(q, 2)) return fail(QMM_ERR_INVALID_ARG, "q must be a 2-byte aligned pointer");
    if (!o || !aligned(o, 8) || (o_token_stride | o_head_stride) % 4 != 0)
        return fail(QMM_ERR_INVALID_ARG, "o must be 8-byte aligned, its strides multiples of 4 elements");
    if (!rows_apart(tokens, heads, o_token_stride, o_head_stride, cache->head_dim))
        return fail(QMM_ERR_INVALID_ARG, "rows of o overlap");
    if (!aligned(lse, 4) || !aligned(tree, 8)) return fail(QMM_ERR_INVALID_ARG, "lse must be 4-byte and tree 8-byte aligned");
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.kc = reinterpret_cast<const uint8_t*>(cache->k_packed), a.vc = reinterpret_cast<const uint8_t*>(cache->v_packed);
    a.ks = cache->k_scales, a.kb = cache->k_biases, a.vs = cache->v_scales, a.vb = cache->v_biases;
    a.q = static_cast<const uint16_t*>(q);
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = o_token_stride, a.o_hs = o_head_stride;
    a.table = seqs->page_table;
    a.table_stride = seqs->table_stride;
    a.lens = lens;
    a.cu = seqs->cu_tokens;
    a.tree = tree;
    a.pages = cache->pages;
    a.page = cache->page_size;
    a.capacity = int(seqs->max_pages * cache->page_size);
    a.seqs = int(seqs->seqs);
    a.tokens = int(tokens);
    a.kv_heads = cache->kv_heads;
    a.group_heads = heads / cache->kv_heads;
    a.window = window < (int64_t(1) << 30) ? int(window) : 0;  // no sequence is longer
    a.scale_log2 = scale * 1.44269504088896341f;
    a.is_bf16 = dtype == QMM_BF16;
    a.q_vec = aligned(q, 16) && (q_token_stride | q_head_stride) % 8 == 0;
    try {  // the workspaces are kept in host containers
        return launch_result(launch_attn(a, cache->head_dim, cache->group, static_cast<cudaStream_t>(stream)),
                             "qmm_kv_attention launch");
    } catch (...) {
        return fail(QMM_ERR_CUDA, "qmm_kv_attention: out of host memory");
    }
}

}  // extern "C"
