// The serving operators' C ABI: argument checks on the host, then the launchers (as abi.cpp does for the
// products).  What the device holds (lengths, tables, slots, token numbers) cannot be checked here; the kernels
// check every index they form from it.
#include <hip/hip_runtime.h>

#include "serve_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_dtype(int t) { return t == LB_F32 || t == LB_BF16 || t == LB_F16; }
bool is_page(int64_t p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
bool is_head_dim(int64_t d) { return d == 64 || d == 128 || d == 256; }

constexpr int64_t kMax = INT32_MAX;
constexpr int64_t kMaxExperts = 1024, kMaxPairs = (int64_t)1 << 30; // (places of tiles are numbered in 32 bits)
constexpr const char *kTiles = "the step has 2^23 tiles, or parts of tiles, or more";

// The cache's shape; LB_OK or the failure.
lb_status check_cache(const char *fn, int64_t pages, int64_t heads, int64_t P, int64_t D)
{
    if (!is_page(P))
        return lb::abi_fail(LB_ESHAPE, fn, "page_tokens must be a power of two from 16 to 1024");
    if (!is_head_dim(D))
        return lb::abi_fail(LB_ESHAPE, fn, "head_dim must be 64, 128 or 256");
    if (heads < 1 || heads > 65536)
        return lb::abi_fail(LB_ESHAPE, fn, "kv_heads must be from 1 to 65536");
    if (pages < 0 || pages > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "negative number of pages, or over 2^31-1");
    if (heads * lb::kv_record_bytes(P, D) >= (int64_t)1 << 32)
        return lb::abi_fail(LB_ESHAPE, fn, "a page of 4 GiB or more");
    return LB_OK;
}

// Rows [T][heads][D] with a token stride in elements.
lb_status check_rows(const char *fn, const void *p, int64_t stride, int64_t width, int dtype)
{
    if (!p)
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (stride < width)
        return lb::abi_fail(LB_ESHAPE, fn, "a row stride is shorter than the row");
    if (!aligned(p, 16) || (stride * lb::dtype_bytes(dtype)) % 16)
        return lb::abi_fail(LB_EALIGN, fn, "rows need 16-byte alignment, their strides too");
    return LB_OK;
}

} // namespace

extern "C" {

int64_t lowbit_kv_cache_bytes(int64_t pages, int64_t kv_heads, int64_t page_tokens, int64_t head_dim)
{
    if (check_cache("lowbit_kv_cache_bytes", pages, kv_heads, page_tokens, head_dim) != LB_OK)
        return -1;
    return pages * kv_heads * lb::kv_record_bytes(page_tokens, head_dim); // below 2^63, a page being below 2^32
}

lb_status lowbit_kv_plan(const int32_t *new_lens, int64_t B, int64_t page_tokens, const int32_t *kv_lens, int32_t *kv_lens_out,
                         int32_t *block_table, int64_t table_stride, const int32_t *free_pages, int64_t free_capacity,
                         const int32_t *free_count, int32_t *free_count_out, int32_t *cu_q, int32_t *cu_pages, int64_t *slots,
                         int32_t *positions, int64_t max_tokens, int32_t *status, hipStream_t s)
{
    const char *fn = "lowbit_kv_plan";
    // the kernels bisect over the requests with 32-bit sums of two numbers of them
    if (B < 0 || B > (1 << 30) || table_stride < 0 || table_stride > kMax || free_capacity < 0 || free_capacity > kMax || max_tokens < 0 ||
        max_tokens > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "negative size, over 2^30 requests, or another size over 2^31-1");
    if (!is_page(page_tokens))
        return lb::abi_fail(LB_ESHAPE, fn, "page_tokens must be a power of two from 16 to 1024");
    if (B == 0)
        return LB_OK;
    if (!new_lens || !kv_lens || !kv_lens_out || !free_count || !free_count_out || !cu_q || !cu_pages || !status ||
        (!block_table && table_stride) || (!free_pages && free_capacity) || ((!slots || !positions) && max_tokens))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(new_lens, 4) || !aligned(kv_lens, 4) || !aligned(kv_lens_out, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
        !aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(cu_q, 4) || !aligned(cu_pages, 4) || !aligned(positions, 4) ||
        !aligned(status, 4) || !aligned(slots, 8))
        return lb::abi_fail(LB_EALIGN, fn, "slots need 8-byte alignment, everything else 4-byte alignment");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::PlanArgs a = {};
    a.new_lens = new_lens, a.kv_lens = kv_lens, a.free_pages = free_pages, a.free_count = free_count;
    a.kv_lens_out = kv_lens_out, a.block_table = block_table, a.free_count_out = free_count_out, a.cu_q = cu_q;
    a.cu_pages = cu_pages, a.positions = positions, a.status = status, a.slots = slots;
    a.B = B, a.page_tokens = page_tokens, a.table_stride = table_stride, a.free_capacity = free_capacity, a.max_tokens = max_tokens;
    return lb::abi_hip(fn, lb::launch_kv_plan(a, s));
}

lb_status lowbit_kv_release(const int32_t *done, int64_t B, int64_t page_tokens, int32_t *kv_lens, const int32_t *block_table,
                            int64_t table_stride, int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int32_t *status,
                            hipStream_t s)
{
    const char *fn = "lowbit_kv_release";
    // one workgroup of 256 a request: the launch's threads are numbered in 32 bits
    if (B < 0 || B >= (1 << 24) || table_stride < 0 || table_stride > kMax || free_capacity < 0 || free_capacity > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "negative size, 2^24 requests or more, or another size over 2^31-1");
    if (!is_page(page_tokens))
        return lb::abi_fail(LB_ESHAPE, fn, "page_tokens must be a power of two from 16 to 1024");
    if (B == 0)
        return LB_OK;
    if (!done || !kv_lens || !free_count || !status || (!block_table && table_stride) || (!free_pages && free_capacity))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(done, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) ||
        !aligned(status, 4))
        return lb::abi_fail(LB_EALIGN, fn, "4-byte alignment is needed");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::ReleaseArgs a = {};
    a.done = done, a.block_table = block_table, a.kv_lens = kv_lens, a.free_pages = free_pages, a.free_count = free_count;
    a.status = status, a.B = B, a.page_tokens = page_tokens, a.table_stride = table_stride, a.free_capacity = free_capacity;
    return lb::abi_hip(fn, lb::launch_kv_release(a, s));
}

static lb_status rows_common(const char *fn, int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t T,
                             int64_t kv_heads, int64_t head_dim, const int64_t *slots, const void *cache, int64_t pages,
                             int64_t page_tokens, bool append, hipStream_t s)
{
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown row type");
    lb_status st = check_cache(fn, pages, kv_heads, page_tokens, head_dim);
    if (st != LB_OK)
        return st;
    // a launch's threads are numbered in 32 bits, head_dim / 8 of them a row and head
    if (T < 0 || T > kMax || (T + 31) * kv_heads * (head_dim / 8) >= (int64_t)1 << 32)
        return lb::abi_fail(LB_ESHAPE, fn, "negative T, or T * kv_heads * head_dim of 2^35 or more");
    if (T == 0)
        return LB_OK;
    if (!slots || (!cache && pages))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    st = check_rows(fn, k, k_stride, kv_heads * head_dim, dtype);
    if (st == LB_OK)
        st = check_rows(fn, v, v_stride, kv_heads * head_dim, dtype);
    if (st != LB_OK)
        return st;
    if (!aligned(cache, 16) || !aligned(slots, 8))
        return lb::abi_fail(LB_EALIGN, fn, "the cache needs 16-byte alignment, slots 8-byte alignment");
    st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::RowsArgs a = {};
    a.k = const_cast<void *>(k), a.v = const_cast<void *>(v), a.k_stride = k_stride, a.v_stride = v_stride;
    a.T = T, a.kv_heads = kv_heads, a.head_dim = head_dim, a.slots = slots;
    a.cache = static_cast<uint8_t *>(const_cast<void *>(cache)), a.pages = pages, a.page_tokens = page_tokens;
    return lb::abi_hip(fn, append ? lb::launch_kv_append(dtype, a, s) : lb::launch_kv_read(dtype, a, s));
}

lb_status lowbit_kv_append(int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t T, int64_t kv_heads,
                           int64_t head_dim, const int64_t *slots, void *cache, int64_t pages, int64_t page_tokens, hipStream_t s)
{
    return rows_common("lowbit_kv_append", dtype, k, k_stride, v, v_stride, T, kv_heads, head_dim, slots, cache, pages, page_tokens,
                       true, s);
}

lb_status lowbit_kv_read(int dtype, const void *cache, int64_t pages, int64_t page_tokens, int64_t T, int64_t kv_heads, int64_t head_dim,
                         const int64_t *slots, void *k, int64_t k_stride, void *v, int64_t v_stride, hipStream_t s)
{
    return rows_common("lowbit_kv_read", dtype, k, k_stride, v, v_stride, T, kv_heads, head_dim, slots, cache, pages, page_tokens, false,
                       s);
}

lb_status lowbit_kv_append_rotary(int dtype, const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride, int64_t T, int64_t q_heads, int64_t kv_heads,
                                  int64_t head_dim, const int32_t *positions, const float *inv_freq, int64_t rotary_dim, int style,
                                  float factor, const int64_t *slots, void *cache, int64_t pages, int64_t page_tokens, hipStream_t s)
{
    const char *fn = "lowbit_kv_append_rotary";
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown row type");
    if (style != LB_ROTARY_HALVES && style != LB_ROTARY_PAIRS)
        return lb::abi_fail(LB_EINVAL, fn, "unknown style of rotation");
    lb_status st = check_cache(fn, pages, kv_heads, page_tokens, head_dim);
    if (st != LB_OK)
        return st;
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16)
        return lb::abi_fail(LB_ESHAPE, fn, "rotary_dim must be a multiple of 16, from 16 to head_dim");
    if (q_heads < 0 || q_heads > 65536)
        return lb::abi_fail(LB_ESHAPE, fn, "q_heads must be from 0 to 65536");
    // a launch's threads are numbered in 32 bits, head_dim / 8 of them a row and head; a grid has 65535 runs of heads at most
    const int64_t heads = q_heads + kv_heads;
    if (heads > 65535)
        return lb::abi_fail(LB_ESHAPE, fn, "over 65535 heads in all");
    if (T < 0 || T > kMax || (T + 31) * heads * (head_dim / 8) >= (int64_t)1 << 32)
        return lb::abi_fail(LB_ESHAPE, fn, "negative T, or T * (q_heads + kv_heads) * head_dim of 2^35 or more");
    if (T == 0)
        return LB_OK;
    if (!positions || !inv_freq || !slots || (!cache && pages))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    st = check_rows(fn, k, k_stride, kv_heads * head_dim, dtype);
    if (st == LB_OK)
        st = check_rows(fn, v, v_stride, kv_heads * head_dim, dtype);
    if (st == LB_OK && q_heads)
        st = check_rows(fn, q, q_stride, q_heads * head_dim, dtype);
    if (st == LB_OK && q_heads)
        st = check_rows(fn, q_out, q_out_stride, q_heads * head_dim, dtype);
    if (st != LB_OK)
        return st;
    if (q_heads && q_out == q && q_stride != q_out_stride)
        return lb::abi_fail(LB_ESHAPE, fn, "in place, both strides of the queries have to be the same");
    if (!aligned(cache, 16) || !aligned(slots, 8) || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return lb::abi_fail(LB_EALIGN, fn, "the cache needs 16-byte alignment, slots 8-byte, positions and inv_freq 4-byte alignment");
    st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::RotaryArgs a = {};
    a.q = q, a.k = k, a.v = v, a.q_out = q_out, a.q_stride = q_stride, a.q_out_stride = q_out_stride, a.k_stride = k_stride;
    a.v_stride = v_stride, a.T = T, a.q_heads = q_heads, a.kv_heads = kv_heads, a.head_dim = head_dim, a.rotary_dim = rotary_dim;
    a.positions = positions, a.inv_freq = inv_freq, a.factor = factor, a.pairs = style == LB_ROTARY_PAIRS, a.slots = slots;
    a.cache = static_cast<uint8_t *>(cache), a.pages = pages, a.page_tokens = page_tokens;
    return lb::abi_hip(fn, lb::launch_kv_append_rotary(dtype, a, s));
}

// Sizes of an attention call; the ones the workspace depends on.
static lb_status attn_sizes(const char *fn, lb::AttnArgs &a, int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                            int64_t max_q, int64_t max_kv, int64_t window)
{
    if (T < 0 || B < 0 || q_heads < 1 || max_q < 0 || max_kv < 0 || window < 0)
        return lb::abi_fail(LB_ESHAPE, fn, "negative size, or no query heads");
    if (!is_head_dim(head_dim))
        return lb::abi_fail(LB_ESHAPE, fn, "head_dim must be 64, 128 or 256");
    if (kv_heads < 1 || kv_heads > 65536 || q_heads > 65536 || q_heads % kv_heads)
        return lb::abi_fail(LB_ESHAPE, fn, "q_heads must be a multiple of kv_heads, and both at most 65536");
    if (T > kMax || B > kMax || max_kv >= kMax - 4096 || max_q > kMax || window > kMax || T * q_heads > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "a size over 2^31-1 (T * q_heads too)");
    a.T = T, a.B = B, a.q_heads = q_heads, a.kv_heads = kv_heads, a.head_dim = head_dim;
    // a request has no more new tokens than the step, and a window longer than the cache is none
    a.max_q = max_q < T ? max_q : T, a.max_kv = max_kv, a.window = window >= max_kv ? 0 : window;
    return LB_OK;
}

int64_t lowbit_kv_attention_workspace(int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_q,
                                      int64_t max_kv, int64_t window)
{
    const char *fn = "lowbit_kv_attention_workspace";
    lb::AttnArgs a = {};
    if (attn_sizes(fn, a, T, B, q_heads, kv_heads, head_dim, max_q, max_kv, window) != LB_OK)
        return -1;
    const int64_t need = T && B ? lb::kv_attention_workspace(a) : 0;
    if (need < 0)
        (void)lb::abi_fail(LB_ESHAPE, fn, kTiles);
    return need;
}

lb_status lowbit_kv_attention(int dtype, const void *q, int64_t q_stride, int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads,
                              int64_t head_dim, const int32_t *cu_q, const int32_t *kv_lens, const int32_t *block_table,
                              int64_t table_stride, const void *cache, int64_t pages, int64_t page_tokens, int64_t max_q,
                              int64_t max_kv, float scale, int64_t window, void *out, int64_t out_stride, void *workspace,
                              int64_t workspace_bytes, hipStream_t s)
{
    const char *fn = "lowbit_kv_attention";
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown row type");
    lb::AttnArgs a = {};
    lb_status st = check_cache(fn, pages, kv_heads, page_tokens, head_dim);
    if (st == LB_OK)
        st = attn_sizes(fn, a, T, B, q_heads, kv_heads, head_dim, max_q, max_kv, window);
    if (st != LB_OK)
        return st;
    if (T && B && !lb::kv_attention_fits(dtype, a))
        return lb::abi_fail(LB_ESHAPE, fn, kTiles);
    if (table_stride < 0 || table_stride > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "negative table stride, or over 2^31-1");
    if (max_kv > 0 && pages == 0)
        return lb::abi_fail(LB_ESHAPE, fn, "a cache without pages holds no tokens (max_kv must be 0)");
    if (T == 0 || B == 0)
        return LB_OK;
    if (!cu_q || !kv_lens || (!block_table && table_stride) || (!cache && pages))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    st = check_rows(fn, q, q_stride, q_heads * head_dim, dtype);
    if (st == LB_OK)
        st = check_rows(fn, out, out_stride, q_heads * head_dim, dtype);
    if (st != LB_OK)
        return st;
    if (!aligned(cache, 16) || !aligned(workspace, 16) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4))
        return lb::abi_fail(LB_EALIGN, fn, "the cache and the workspace need 16-byte alignment, the tables 4-byte alignment");
    const int64_t need = lb::kv_attention_workspace(a);
    if (need > 0 && !workspace)
        return lb::abi_fail(LB_EINVAL, fn, "null pointer (lowbit_kv_attention_workspace gives the workspace's size)");
    if (workspace_bytes < need)
        return lb::abi_fail(LB_ESHAPE, fn, "the workspace is smaller than lowbit_kv_attention_workspace says");
    st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    a.q = q, a.out = out, a.q_stride = q_stride, a.out_stride = out_stride, a.cu_q = cu_q, a.kv_lens = kv_lens;
    a.block_table = block_table, a.table_stride = table_stride, a.cache = static_cast<const uint8_t *>(cache), a.pages = pages;
    a.page_tokens = page_tokens, a.scale = scale, a.workspace = workspace;
    return lb::abi_hip(fn, lb::launch_kv_attention(dtype, a, s));
}

lb_status lowbit_route(int dtype, const void *logits, int64_t stride, int64_t T, int64_t E, int score, const float *bias, int64_t groups,
                       int64_t groups_kept, int64_t group_best, int64_t top_k, int renormalise, float factor, const int32_t *count,
                       int32_t *experts, float *weights, hipStream_t s)
{
    const char *fn = "lowbit_route";
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown logit type");
    if (score != LB_SCORE_SOFTMAX && score != LB_SCORE_SIGMOID)
        return lb::abi_fail(LB_EINVAL, fn, "unknown score");
    if (T < 0 || T >= (1 << 26) || E < 1 || E > kMaxExperts)
        return lb::abi_fail(LB_ESHAPE, fn, "T must be from 0 to 2^26 - 1, E from 1 to 1024");
    if (groups < 1 || groups > 64 || E % groups || groups_kept < 1 || groups_kept > groups || group_best < 1 || group_best > 2)
        return lb::abi_fail(LB_ESHAPE, fn, "groups must be a divisor of E up to 64, groups_kept from 1 to groups, group_best 1 or 2");
    if (top_k < 1 || top_k > 64 || top_k > E / groups * groups_kept)
        return lb::abi_fail(LB_ESHAPE, fn, "top_k must be from 1 to 64, and at most the experts of the groups kept");
    if (lb::route_blocks(T, E, groups) >= (1 << 24)) // a launch's threads are numbered in 32 bits
        return lb::abi_fail(LB_ESHAPE, fn, "over 2^26 - 4 tokens with more than 256 experts or 32 groups");
    if (stride < E)
        return lb::abi_fail(LB_ESHAPE, fn, "a row stride is shorter than the row");
    if (T == 0)
        return LB_OK;
    if (!logits || !experts || !weights)
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(logits, lb::dtype_bytes(dtype)) || !aligned(bias, 4) || !aligned(count, 4) || !aligned(experts, 4) || !aligned(weights, 4))
        return lb::abi_fail(LB_EALIGN, fn, "a pointer is not aligned to its elements");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::RouteArgs a = {};
    a.logits = logits, a.stride = stride, a.T = T, a.E = E, a.groups = groups, a.kept = groups_kept, a.best = group_best, a.top_k = top_k;
    a.sigmoid = score == LB_SCORE_SIGMOID, a.renormalise = renormalise != 0, a.bias = bias, a.factor = factor, a.count = count;
    a.experts = experts, a.weights = weights;
    return lb::abi_hip(fn, lb::launch_route(dtype, a, s));
}

int64_t lowbit_experts_weight_bytes(int fmt, int64_t E, int64_t N, int64_t K)
{
    const int64_t one = lowbit_weight_bytes(fmt, N, K);
    if (one < 0 || one >= (int64_t)1 << 32 || E < 0 || E > kMaxExperts)
        return -1;
    return E * ((one + 15) / 16 * 16);
}

int64_t lowbit_experts_plan_bytes(int64_t pairs, int64_t E)
{
    if (pairs < 0 || pairs > kMaxPairs || E < 1 || E > kMaxExperts)
        return -1;
    const int64_t tiles = lb::experts_max_tiles(pairs, E);
    return (4 * lb::experts_pairs_at(tiles, tiles, lb::experts_tile_rows(pairs, E)) + 15) / 16 * 16;
}

lb_status lowbit_experts_plan(const int32_t *experts, int64_t pairs, int64_t E, void *plan, hipStream_t s)
{
    const char *fn = "lowbit_experts_plan";
    if (pairs < 0 || pairs > kMaxPairs || E < 1 || E > kMaxExperts)
        return lb::abi_fail(LB_ESHAPE, fn, "pairs must be from 0 to 2^30, E from 1 to 1024");
    if (pairs == 0)
        return LB_OK;
    if (!experts || !plan)
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(experts, 4) || !aligned(plan, 16))
        return lb::abi_fail(LB_EALIGN, fn, "the plan needs 16-byte alignment, experts 4-byte alignment");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    return lb::abi_hip(fn, lb::launch_experts_plan(experts, pairs, E, static_cast<int32_t *>(plan), s));
}

lb_status lowbit_experts_matmul(int fmt, const void *W, int64_t E, int64_t N, int64_t K, const int8_t *xq, const void *xscale,
                                const int32_t *experts, int64_t pairs, int64_t pairs_per_row, const void *plan, float *y, hipStream_t s)
{
    const char *fn = "lowbit_experts_matmul";
    if (fmt < LB_Q1_0 || fmt > LB_Q4_0)
        return lb::abi_fail(LB_EINVAL, fn, "unknown weight format");
    if (fmt != LB_Q1_0 && fmt != LB_Q2_0_G64 && fmt != LB_Q4_0)
        return lb::abi_fail(LB_EUNSUPPORTED, fn, "experts are Q1_0, Q2_0_g64 or Q4_0");
    if (N < 0 || K < 1 || pairs < 0 || pairs_per_row < 1 || E < 1 || E > kMaxExperts || N > kMax || pairs > kMaxPairs || pairs_per_row > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "a size below its least (K, E and pairs_per_row: 1), E over 1024, pairs over 2^30, or another over 2^31 - 1");
    if (K % (fmt == LB_Q2_0_G64 ? 64 : 128) || K > (fmt == LB_Q4_0 ? 16384 : 32768))
        return lb::abi_fail(LB_ESHAPE, fn, "K must be a multiple of 128 (64 for Q2_0_g64), at most 32768 (16384 for Q4_0)");
    if (lowbit_weight_bytes(fmt, N, K) >= (int64_t)1 << 32)
        return lb::abi_fail(LB_ESHAPE, fn, "an expert's tensor of 4 GiB or more");
    if (((pairs + pairs_per_row - 1) / pairs_per_row) * K >= (int64_t)1 << 32)
        return lb::abi_fail(LB_ESHAPE, fn, "activations of 4 GiB or more");
    if (N == 0 || pairs == 0)
        return LB_OK;
    if (!W || !xq || !xscale || !y || (!plan && !experts))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(W, 16) || !aligned(xq, 16) || !aligned(plan, 16) || !aligned(xscale, 4) || !aligned(experts, 4) || !aligned(y, 4))
        return lb::abi_fail(LB_EALIGN, fn, "W, xq and the plan need 16-byte alignment, everything else 4-byte alignment");
    lb::ExpertsArgs a = {};
    a.W = static_cast<const uint8_t *>(W), a.expert_bytes = lowbit_experts_weight_bytes(fmt, 1, N, K);
    a.E = (int32_t)E, a.N = (int32_t)N, a.K = (int32_t)K, a.pairs = (int32_t)pairs, a.per_row = (int32_t)pairs_per_row;
    a.xq = xq, a.xs = static_cast<const uint16_t *>(xscale), a.experts = experts, a.plan = static_cast<const int32_t *>(plan);
    a.max_tiles = lb::experts_max_tiles(pairs, E), a.y = y;
    const int64_t rows = plan ? lb::experts_tile_rows(pairs, E) : 1;
    // a launch's threads are numbered in 32 bits
    const int64_t blocks = plan ? a.max_tiles * ((N + 63) / 64) + 7 : lb::experts_pair_blocks(fmt, a);
    if (blocks >= (int64_t)1 << (rows > 16 ? 23 : 24))
        return lb::abi_fail(LB_ESHAPE, fn, "over 2^32 threads");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    return lb::abi_hip(fn, rows > 16 ? lb::launch_experts_gemm(fmt, a, s) : rows > 1 ? lb::launch_experts_tile(fmt, a, s) : lb::launch_experts_pairs(fmt, a, s));
}

lb_status lowbit_experts_combine(int dtype, const float *y, const int32_t *experts, const float *weights, int64_t T, int64_t top_k, int64_t E,
                                 int64_t N, void *out, int64_t out_stride, hipStream_t s)
{
    const char *fn = "lowbit_experts_combine";
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown row type");
    if (T < 0 || T > kMax || top_k < 1 || top_k > 1024 || E < 1 || E > kMaxExperts || N < 0 || N > kMax)
        return lb::abi_fail(LB_ESHAPE, fn, "negative size, top_k or E not from 1 to 1024, or another size over 2^31 - 1");
    if (T * ((N + 255) / 256) >= (1 << 24))
        return lb::abi_fail(LB_ESHAPE, fn, "2^32 outputs or more");
    if (out_stride < N)
        return lb::abi_fail(LB_ESHAPE, fn, "a row stride is shorter than the row");
    if (T == 0 || N == 0)
        return LB_OK;
    if (!y || !experts || !weights || !out)
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!aligned(y, 4) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(out, lb::dtype_bytes(dtype)))
        return lb::abi_fail(LB_EALIGN, fn, "a pointer is not aligned to its elements");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::CombineArgs a = {};
    a.y = y, a.experts = experts, a.weights = weights, a.T = T, a.top_k = top_k, a.E = E, a.N = N, a.out = out, a.out_stride = out_stride;
    return lb::abi_hip(fn, lb::launch_experts_combine(dtype, a, s));
}

lb_status lowbit_logits_process(int dtype, const void *logits, int64_t in_stride, int64_t B, int64_t V, const int32_t *tokens,
                                int64_t tok_stride, const int32_t *prompt_lens, const int32_t *total_lens, const float *repetition,
                                const float *presence, const float *frequency, const int32_t *bias_tokens, const float *bias_values,
                                int64_t bias_stride, const int32_t *bias_lens, const uint32_t *mask, int64_t mask_stride, void *out,
                                int64_t out_stride, hipStream_t s)
{
    const char *fn = "lowbit_logits_process";
    if (!is_dtype(dtype))
        return lb::abi_fail(LB_EINVAL, fn, "unknown logit type");
    if (B < 0 || V < 0 || B > kMax || V > kMax || tok_stride < 0 || tok_stride > kMax || bias_stride < 0)
        return lb::abi_fail(LB_ESHAPE, fn, "negative size, or over 2^31-1");
    if (bias_stride > 16384)
        return lb::abi_fail(LB_ESHAPE, fn, "over 16384 biases a row");
    if (B * ((V + 1023) / 1024) >= (1 << 22))
        return lb::abi_fail(LB_ESHAPE, fn, "over 2^32 logits");
    if (B == 0 || V == 0)
        return LB_OK;
    if (!logits || !out || (tokens && !total_lens) || (bias_tokens && (!bias_values || !bias_lens)))
        return lb::abi_fail(LB_EINVAL, fn, "null pointer");
    if (!tokens && (repetition || presence || frequency))
        return lb::abi_fail(LB_EINVAL, fn, "penalties need the tokens of the history");
    if (in_stride < V || out_stride < V || (mask && mask_stride < (V + 31) / 32))
        return lb::abi_fail(LB_ESHAPE, fn, "a stride is shorter than the row");
    if (out == logits && in_stride != out_stride)
        return lb::abi_fail(LB_ESHAPE, fn, "in place, both strides have to be the same");
    const int64_t e = lb::dtype_bytes(dtype);
    if (!aligned(logits, e) || !aligned(out, e) || !aligned(tokens, 4) || !aligned(prompt_lens, 4) || !aligned(total_lens, 4) ||
        !aligned(repetition, 4) || !aligned(presence, 4) || !aligned(frequency, 4) || !aligned(bias_tokens, 4) ||
        !aligned(bias_values, 4) || !aligned(bias_lens, 4) || !aligned(mask, 4))
        return lb::abi_fail(LB_EALIGN, fn, "a pointer is not aligned to its elements");
    lb_status st = lb::abi_check_device(fn);
    if (st != LB_OK)
        return st;
    lb::LogitsArgs a = {};
    a.logits = logits, a.out = out, a.in_stride = in_stride, a.out_stride = out_stride, a.B = B, a.V = V;
    a.tokens = tokens, a.tok_stride = tok_stride, a.prompt_lens = prompt_lens, a.total_lens = total_lens;
    a.repetition = repetition, a.presence = presence, a.frequency = frequency;
    a.bias_tokens = bias_tokens, a.bias_lens = bias_lens, a.bias_values = bias_values, a.bias_stride = bias_stride;
    a.mask = mask, a.mask_stride = mask_stride;
    return lb::abi_hip(fn, lb::launch_logits_process(dtype, a, s));
}

} // extern "C"
