// C ABI of the exact-token cache (declared in include/skv.h): argument checks, workspace plan and
// launches. Nothing here allocates, throws or synchronises.
#include <cmath>

#include "token_cache.cuh"

using namespace skv;

namespace {

constexpr size_t kTicketOffset = 64;   // the append's CTA count, inside the workspace header
// The attention's counters have a place of their own for the most units of any call, so that calls of
// different shapes can share a workspace: no call's partials lie where another's counters are.
constexpr size_t kPartOffset = kWsHeader + (static_cast<size_t>(kMaxPagedUnits) + 2 * kMaxPagedCtas) * 4;
static_assert(kPartOffset % 256 == 0, "partials start on 256 bytes");
constexpr int64_t kMaxCacheTokens = int64_t{1} << 30;   // per sequence: positions are int32

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t group_bytes(int dtype, int format, int d) {
    const size_t elem = format == SKV_CACHE_E4M3 ? 1 : dtype == SKV_BF16 ? 2 : 4;
    return 2 * kGroupTokens * d * elem + (format == SKV_CACHE_E4M3 ? 2 * kGroupTokens : 0);
}

// What every entry point of the cache asks of its geometry.
skv_status check_cache(int dtype, int format, int B, int Hkv, int d, int max_pages) {
    if (B < 1 || B > SKV_MAX_SEQS || Hkv < 1 || max_pages < 1) return SKV_ERR_INVALID_ARG;
    if (format != SKV_CACHE_RAW && format != SKV_CACHE_E4M3) return SKV_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || (dtype != SKV_BF16 && dtype != SKV_F32)) return SKV_ERR_UNSUPPORTED;
    if (Hkv > 65535 || static_cast<int64_t>(max_pages) * SKV_CACHE_PAGE_TOKENS > kMaxCacheTokens)
        return SKV_ERR_UNSUPPORTED;
    return SKV_OK;
}

// Groups are counted in 32 bits (2^31 of the smallest, 2,080 bytes, are 4 TB).
skv_status check_pool(const skv_token_cache *c, int Hkv) {
    if (!c || !c->pages || !aligned(c->pages, 16) || c->num_pages < 0) return SKV_ERR_INVALID_ARG;
    return c->num_pages > INT32_MAX / (static_cast<int64_t>(Hkv) * kPageGroups) ? SKV_ERR_UNSUPPORTED : SKV_OK;
}

// Vectors are read 16 bytes at a time. A dimension of one element has no stride that matters.
bool stride_ok(int64_t stride, int64_t n, int64_t elem) { return stride >= 0 && (n <= 1 || stride * elem % 16 == 0); }

bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

skv_status plan_paged(int dtype, int B, int R, int Hq, int Hkv, int d, int max_pages, PagedArgs *a, size_t *total) {
    const skv_status st = check_cache(dtype, SKV_CACHE_RAW, B, Hkv, d, max_pages);
    if (st != SKV_OK) return st;
    if (R < 1 || Hq < 1) return SKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return SKV_ERR_UNSUPPORTED;
    const int64_t rows = static_cast<int64_t>(R) * (Hq / Hkv);
    if (rows > (1 << 20)) return SKV_ERR_UNSUPPORTED;
    a->B = B;
    a->R = R;
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->G = Hq / Hkv;
    a->inv_G = 1.0f / static_cast<float>(a->G);
    a->d = d;
    a->dtype = dtype;
    a->rows = static_cast<int>(rows);
    a->pass_rows = paged_pass_rows(dtype, a->rows);
    a->passes = (a->rows + a->pass_rows - 1) / a->pass_rows;
    const int64_t per_seq = static_cast<int64_t>(Hkv) * a->passes;
    if (per_seq * B > kMaxPagedUnits) return SKV_ERR_UNSUPPORTED;
    // the weight (rounds of at least 4 groups, and a cost) of one sequence's units is counted in int32
    if (per_seq * (static_cast<int64_t>(max_pages) * kPageGroups / 4 + 16) > INT32_MAX) return SKV_ERR_UNSUPPORTED;
    *total = kPartOffset + align256(static_cast<size_t>(kMaxPagedCtas) * 2 * a->pass_rows * d * 4) +
             align256(static_cast<size_t>(kMaxPagedCtas) * 2 * a->pass_rows * 4);
    return SKV_OK;
}

}  // namespace

extern "C" {

size_t skv_cache_page_bytes(skv_dtype dtype, skv_cache_format format, int Hkv, int d) {
    if (check_cache(dtype, format, 1, Hkv, d, 1) != SKV_OK) return 0;
    return group_bytes(dtype, format, d) * kPageGroups * Hkv;
}

skv_status skv_cache_append(const void *k, const void *v, skv_dtype dtype, int64_t k_token_stride,
                            int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, int B, int Hkv, int d,
                            int n_tokens, const int32_t *cu_new, skv_cache_format format, const skv_token_cache *cache,
                            const int32_t *page_table, int max_pages, const int32_t *lens, int32_t *new_lens,
                            void *workspace, size_t ws_bytes, void *stream) {
    skv_status st = check_cache(dtype, format, B, Hkv, d, max_pages);
    if (st != SKV_OK) return st;
    if (n_tokens < 0 || (!cu_new && n_tokens % B != 0)) return SKV_ERR_INVALID_ARG;
    if ((n_tokens > 0 && (!k || !v)) || !page_table || !lens || !new_lens) return SKV_ERR_INVALID_ARG;
    if ((st = check_pool(cache, Hkv)) != SKV_OK) return st;
    const int64_t elem = dtype == SKV_BF16 ? 2 : 4;
    if (!stride_ok(k_token_stride, n_tokens, elem) || !stride_ok(k_head_stride, Hkv, elem) ||
        !stride_ok(v_token_stride, n_tokens, elem) || !stride_ok(v_head_stride, Hkv, elem))
        return SKV_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(new_lens, 4))
        return SKV_ERR_INVALID_ARG;
    // new_lens may be lens itself, and nothing in between; nor may it lie in what is read beside it
    const size_t n4 = static_cast<size_t>(B) * 4;
    if ((new_lens != lens && overlap(new_lens, n4, lens, n4)) || (cu_new && overlap(new_lens, n4, cu_new, n4 + 4)) ||
        overlap(new_lens, n4, page_table, n4 * max_pages))
        return SKV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(n_tokens) * Hkv > INT32_MAX) return SKV_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < kWsHeader) return SKV_ERR_WORKSPACE;
    AppendArgs a{};
    a.k = k;
    a.v = v;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.B = B;
    a.Hkv = Hkv;
    a.d = d;
    a.dtype = dtype;
    a.format = format;
    a.n_tokens = n_tokens;
    a.per_seq = n_tokens / B;
    a.cu = cu_new;
    a.pages = static_cast<uint8_t *>(cache->pages);
    a.num_pages = cache->num_pages;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.lens = lens;
    a.new_lens = new_lens;
    a.flags = static_cast<uint32_t *>(workspace);
    a.ticket = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + kTicketOffset);
    return launch_cache_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}

skv_status skv_cache_read(const skv_token_cache *cache, skv_dtype dtype, skv_cache_format format, int B, int Hkv, int d,
                          const int32_t *first_host, const int32_t *T_host, const int32_t *page_table, int max_pages,
                          void *k, void *v, void *workspace, size_t ws_bytes, void *stream) {
    skv_status st = check_cache(dtype, format, B, Hkv, d, max_pages);
    if (st != SKV_OK) return st;
    if (!first_host || !T_host || !page_table || !aligned(page_table, 4)) return SKV_ERR_INVALID_ARG;
    if ((st = check_pool(cache, Hkv)) != SKV_OK) return st;
    ReadTable t;
    int64_t rows = 0, items = 0;
    for (int b = 0; b < B; ++b) {
        const int64_t first = first_host[b], T = T_host[b];
        if (first < 0 || T < 0 || first + T > static_cast<int64_t>(max_pages) * SKV_CACHE_PAGE_TOKENS)
            return SKV_ERR_INVALID_ARG;
        t.rows[b] = ReadRow{rows, static_cast<int32_t>(first), static_cast<int32_t>(T), static_cast<int32_t>(items), 0};
        rows += T * Hkv;
        if (T > 0) items += ((first + T + kGroupTokens - 1) / kGroupTokens - first / kGroupTokens) * Hkv;
        if (items > INT32_MAX) return SKV_ERR_UNSUPPORTED;
    }
    const size_t bytes = static_cast<size_t>(rows) * d * (dtype == SKV_BF16 ? 2 : 4);
    if (rows > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16) || overlap(k, bytes, v, bytes))) return SKV_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < kWsHeader) return SKV_ERR_WORKSPACE;
    ReadArgs a{};
    a.B = B;
    a.Hkv = Hkv;
    a.d = d;
    a.dtype = dtype;
    a.format = format;
    a.items = static_cast<int>(items);
    a.pages = static_cast<const uint8_t *>(cache->pages);
    a.num_pages = cache->num_pages;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.k = k;
    a.v = v;
    a.flags = static_cast<uint32_t *>(workspace);
    return launch_cache_read(a, t, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}

size_t skv_paged_attn_workspace_bytes(int B, int R, int Hq, int Hkv, int d, int max_pages) {
    PagedArgs a{};
    size_t bf16 = 0, f32 = 0;   // one size for both types
    if (plan_paged(SKV_BF16, B, R, Hq, Hkv, d, max_pages, &a, &bf16) != SKV_OK ||
        plan_paged(SKV_F32, B, R, Hq, Hkv, d, max_pages, &a, &f32) != SKV_OK)
        return 0;
    return bf16 > f32 ? bf16 : f32;
}

skv_status skv_paged_attn(const void *q, skv_dtype dtype, int64_t q_seq_stride, int64_t q_row_stride,
                          int64_t q_head_stride, int B, int R, int Hq, int Hkv, int d, skv_cache_format format,
                          const skv_token_cache *cache, const int32_t *page_table, int max_pages, const int32_t *lens,
                          void *out, float *lse, void *workspace, size_t ws_bytes,
                          const skv_paged_attn_options *options, void *stream) {
    PagedArgs a{};
    size_t total = 0;
    if (format != SKV_CACHE_RAW && format != SKV_CACHE_E4M3) return SKV_ERR_INVALID_ARG;
    skv_status st = plan_paged(dtype, B, R, Hq, Hkv, d, max_pages, &a, &total);
    if (st != SKV_OK) return st;
    if (!q || !page_table || !lens || !out || !lse) return SKV_ERR_INVALID_ARG;
    if ((st = check_pool(cache, Hkv)) != SKV_OK) return st;
    const int64_t elem = dtype == SKV_BF16 ? 2 : 4;
    if (!stride_ok(q_seq_stride, B, elem) || !stride_ok(q_row_stride, R, elem) || !stride_ok(q_head_stride, Hq, elem))
        return SKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(lens, 4))
        return SKV_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(B) * R * Hq;
    if (overlap(out, n * d * elem, lse, n * 4)) return SKV_ERR_INVALID_ARG;
    a.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    if (options) {
        for (int i = 0; i < 4; ++i)
            if (options->reserved[i] != 0) return SKV_ERR_INVALID_ARG;
        if (!std::isfinite(options->scale) || !std::isfinite(options->softcap) || options->softcap < 0.f ||
            options->window < 0)
            return SKV_ERR_INVALID_ARG;
        if (!options->prior_out != !options->prior_lse) return SKV_ERR_INVALID_ARG;
        if (!aligned(options->first, 4) || !aligned(options->slopes, 4) || !aligned(options->prior_out, 16) ||
            !aligned(options->prior_lse, 4))
            return SKV_ERR_INVALID_ARG;
        // the outputs may replace the prior's; its partitions are read by several threads, so that they may not
        if (options->prior_out && ((options->prior_out != out && overlap(options->prior_out, n * d * elem, out, n * d * elem)) ||
                                   overlap(options->prior_lse, n * 4, lse, n * 4) ||
                                   overlap(options->prior_lse, n * 4, out, n * d * elem)))
            return SKV_ERR_INVALID_ARG;
        if (options->scale != 0.f) a.scale = options->scale;
        a.softcap = options->softcap;
        a.window = options->window;
        a.first = options->first;
        a.slopes = options->slopes;
        a.prior_out = options->prior_out;
        a.prior_lse = options->prior_lse;
    }
    if (!workspace || !aligned(workspace, 256) || ws_bytes < total) return SKV_ERR_WORKSPACE;
    a.q = q;
    a.q_b = q_seq_stride;
    a.q_r = q_row_stride;
    a.q_h = q_head_stride;
    a.format = format;
    a.pages = static_cast<const uint8_t *>(cache->pages);
    a.num_pages = cache->num_pages;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.lens = lens;
    a.out = out;
    a.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.flags = reinterpret_cast<uint32_t *>(ws);
    a.counters = reinterpret_cast<int32_t *>(ws + kWsHeader);
    uint8_t *part = ws + kPartOffset;
    a.part_o = reinterpret_cast<float *>(part);
    a.part_l = reinterpret_cast<float *>(part + align256(static_cast<size_t>(kMaxPagedCtas) * 2 * a.pass_rows * d * 4));
    return launch_paged_attn(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SKV_OK : SKV_ERR_CUDA;
}

}  // extern "C"
