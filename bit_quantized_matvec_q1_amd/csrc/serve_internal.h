// Shared by the serving operators' translation units: the paged 4-bit cache's record layout and the 16- and
// 32-bit row types.
#pragma once

#include "lowbit_internal.h"

namespace lb {

// One record per page and kv head, P tokens of head size D, nb = D / 32 blocks a row (include/lowbit.h):
//   K codes [P][4][nb][4 bytes] | V codes [P/4][16][4][nb bytes] | K scales [P/4][nb][4] | V scales [P/4][nb][4]
// The orders are those in which the attention's matrix instructions take their operands: a lane of the
// 16x16x32 product holds 8 consecutive elements of each 32-block of one key (the four lane groups g hold the
// four quarters of every block, so a lane's share of a key is D/8 contiguous bytes), and for the values one
// column c = element mod 16 of four consecutive tokens, which are 4 nb contiguous bytes.
inline __host__ __device__ int64_t kv_record_bytes(int64_t P, int64_t D) { return P * D * 9 / 8; }
inline __host__ __device__ int kv_k_byte(int D, int o, int g, int b) { return o * (D / 2) + g * (D / 8) + b * 4; }
inline __host__ __device__ int kv_v_byte(int P, int D, int o, int c)
{
    return P * D / 2 + ((o >> 2) * 16 + c) * (D / 8) + (o & 3) * (D / 32);
}
// byte offset of a scale (K: which = 0, V: which = 1)
inline __host__ __device__ int kv_scale_byte(int P, int D, int which, int o, int b)
{
    return P * D + which * (P * (D / 32) * 2) + ((o >> 2) * (D / 32) * 4 + b * 4 + (o & 3)) * 2;
}

inline int64_t dtype_bytes(int t) { return t == LB_F32 ? 4 : 2; }

// E values of a row as fp32, and back (one rounding to nearest even), by 16-byte accesses where E * size allows
template <int DT> struct RowType;
template <> struct RowType<LB_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};
template <> struct RowType<LB_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ T put(float v)
    {
        const uint32_t u = __float_as_uint(v);
        if ((u & 0x7fffffffu) > 0x7f800000u)
            return (uint16_t)((u >> 16) | 0x40u); // a NaN stays one
        return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
    }
};
template <> struct RowType<LB_F16> {
    using T = _Float16;
    static __device__ __forceinline__ float get(T v) { return (float)v; }
    static __device__ __forceinline__ T put(float v) { return (_Float16)v; }
};

template <int DT, int E> struct alignas(E * (DT == LB_F32 ? 4 : 2) >= 16 ? 16 : E * (DT == LB_F32 ? 4 : 2)) RowVec {
    typename RowType<DT>::T v[E];
};

// --- launchers (arguments checked by the ABI layer) ---

struct PlanArgs {
    const int32_t *new_lens, *kv_lens, *free_pages, *free_count;
    int32_t *kv_lens_out, *block_table, *free_count_out, *cu_q, *cu_pages, *positions, *status;
    int64_t *slots;
    int64_t B, page_tokens, table_stride, free_capacity, max_tokens;
};
hipError_t launch_kv_plan(const PlanArgs &a, hipStream_t s);

struct ReleaseArgs {
    const int32_t *done, *block_table;
    int32_t *kv_lens, *free_pages, *free_count, *status;
    int64_t B, page_tokens, table_stride, free_capacity;
};
hipError_t launch_kv_release(const ReleaseArgs &a, hipStream_t s);

struct RowsArgs { // append (k, v read) and read (k, v written)
    void *k, *v;
    int64_t k_stride, v_stride, T, kv_heads, head_dim;
    const int64_t *slots;
    uint8_t *cache;
    int64_t pages, page_tokens;
};
hipError_t launch_kv_append(int dtype, const RowsArgs &a, hipStream_t s);
hipError_t launch_kv_read(int dtype, const RowsArgs &a, hipStream_t s);

struct RotaryArgs {
    const void *q, *k, *v; // q, q_out unused where q_heads is 0
    void *q_out;
    int64_t q_stride, q_out_stride, k_stride, v_stride, T, q_heads, kv_heads, head_dim, rotary_dim;
    const int32_t *positions;
    const float *inv_freq;
    float factor;
    bool pairs;
    const int64_t *slots;
    uint8_t *cache;
    int64_t pages, page_tokens;
};
hipError_t launch_kv_append_rotary(int dtype, const RotaryArgs &a, hipStream_t s);

struct AttnArgs {
    const void *q;
    void *out;
    int64_t q_stride, out_stride, T, B, q_heads, kv_heads, head_dim;
    const int32_t *cu_q, *kv_lens, *block_table;
    int64_t table_stride;
    const uint8_t *cache;
    int64_t pages, page_tokens, max_q, max_kv, window;
    float scale;
    void *workspace;
};
int64_t kv_attention_workspace(const AttnArgs &a);
bool kv_attention_fits(int dtype, const AttnArgs &a);
hipError_t launch_kv_attention(int dtype, const AttnArgs &a, hipStream_t s);

struct RouteArgs {
    const void *logits;
    int64_t stride, T, E, groups, kept, best, top_k;
    bool sigmoid, renormalise;
    const float *bias;
    float factor;
    const int32_t *count;
    int32_t *experts;
    float *weights;
};
int64_t route_blocks(int64_t T, int64_t E, int64_t groups); // workgroups (of 256) of launch_route
hipError_t launch_route(int dtype, const RouteArgs &a, hipStream_t s);

// The routed pairs by expert (include/lowbit.h, lowbit_experts_plan), in tiles of R = experts_tile_rows() places, of one
// expert each.  int32 words, for `tiles` = experts_max_tiles():
//   [0] tiles in use, [1] routed pairs, [2], [3] unused; {expert, rows} [tiles]; pairs [tiles][R]
// A tile may have no rows (those past the last in use, and others); places behind a tile's rows hold -1.  A tile's entry and
// its pairs are at addresses of the tile's number alone, so that neither waits for the other.
inline __host__ __device__ int64_t experts_tile_at(int64_t tile) { return 4 + 2 * tile; }
inline __host__ __device__ int64_t experts_pairs_at(int64_t tiles, int64_t tile, int64_t rows) { return 4 + (2 * tiles + 3) / 4 * 4 + tile * rows; }
int64_t experts_tile_rows(int64_t pairs, int64_t E);
int64_t experts_max_tiles(int64_t pairs, int64_t E);

struct ExpertsArgs {
    const uint8_t *W;
    int64_t expert_bytes; // from one expert's tensor to the next
    int32_t E, N, K, pairs, per_row;
    const int8_t *xq;
    const uint16_t *xs;
    const int32_t *experts, *plan; // plan null: every pair by itself
    int64_t max_tiles;             // of the plan
    float *y;
};
hipError_t launch_experts_plan(const int32_t *experts, int64_t pairs, int64_t E, int32_t *plan, hipStream_t s);
int64_t experts_pair_blocks(int fmt, const ExpertsArgs &a); // workgroups of launch_experts_pairs
hipError_t launch_experts_pairs(int fmt, const ExpertsArgs &a, hipStream_t s);
hipError_t launch_experts_tile(int fmt, const ExpertsArgs &a, hipStream_t s);
hipError_t launch_experts_gemm(int fmt, const ExpertsArgs &a, hipStream_t s);
struct CombineArgs {
    const float *y;
    const int32_t *experts;
    const float *weights;
    int64_t T, top_k, E, N, out_stride;
    void *out;
};
hipError_t launch_experts_combine(int dtype, const CombineArgs &a, hipStream_t s);

struct LogitsArgs {
    const void *logits;
    void *out;
    int64_t in_stride, out_stride, B, V;
    const int32_t *tokens, *prompt_lens, *total_lens;
    int64_t tok_stride;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_tokens, *bias_lens;
    const float *bias_values;
    int64_t bias_stride;
    const uint32_t *mask;
    int64_t mask_stride;
};
hipError_t launch_logits_process(int dtype, const LogitsArgs &a, hipStream_t s);

} // namespace lb
