// Shared by the attention kernels over the 4-bit cache (kvattn.hip, kvattn_prompt.hip): the launch's geometry, the
// tiles of query rows, queries as binary16, and codes as binary16.
#pragma once

#include "serve_internal.h"

namespace lb {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int ATT_ROWS = 16;     // query rows a tile
constexpr int PROMPT_ROWS = 128; // of a prompt's, or twice as many
constexpr int ATT_STEP = 32;  // tokens a step
constexpr int ATT_WAVES = 4;
// Rows of a request up to which the 16-row tiles are taken: 16 requests of 2000 tokens, 20 / 64 / 96 rows each: 39 /
// 54 / 88 us with them, 61 / 67 / 70 us with a prompt's; 64 requests of 500: 32 / 53 / 74 against 36 / 43 / 45 us.
constexpr int PROMPT_FROM = 64;
constexpr float REF_BELOW = 7.0f, REF_MOST = 15.0f; // of a row's reference, log2

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// Four bytes of codes -> eight binary16 numbers, exact.
__device__ __forceinline__ f16x8 codes8(uint32_t w)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Byte b's two codes.
__device__ __forceinline__ f16x2 codes2(uint32_t w, int b)
{
    switch (b & 3) {
    case 0:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    }
}

template <int N> struct Words {
    uint32_t w[N];
};
// ONCE: nothing else reads the bytes, and they need not stay in the caches.
template <int N, bool ONCE> __device__ __forceinline__ Words<N> load_words(const uint8_t *p)
{
    Words<N> r;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 *at = reinterpret_cast<const u32x4 *>(p + 4 * i);
            const u32x4 t = ONCE ? __builtin_nontemporal_load(at) : *at;
            r.w[i] = t.x, r.w[i + 1] = t.y, r.w[i + 2] = t.z, r.w[i + 3] = t.w;
        }
    } else {
        const u32x2 *at = reinterpret_cast<const u32x2 *>(p);
        const u32x2 t = ONCE ? __builtin_nontemporal_load(at) : *at;
        r.w[0] = t.x, r.w[1] = t.y;
    }
    return r;
}
__device__ __forceinline__ float half_of(uint32_t w, int hi) { return half_bits_to_float((uint16_t)(hi ? w >> 16 : w)); }

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// An upper bound of the log2 of a binary16 magnitude's bits, by less than 1 from its normal range on.
__device__ __forceinline__ float log2_above(uint32_t bits) { return (float)((int)(bits >> 10) - 14); }
// The same for every number, down to -64 for 0: far below the least number's -23, and a weight of 2^64 times as much
// still is far from fp32's end.
__device__ __forceinline__ float log2_above_all(uint32_t bits)
{
    const int e = (int)(bits >> 10);
    return (float)(e ? e - 14 : bits ? 8 - __clz((int)bits) : -64);
}

// Column c of four consecutive tokens (nb bytes each, byte b holding elements 32 b + c and 32 b + 16 + c) as
// pairs of tokens: byte b of word [pair][half][b / 4] has element 32 b + 16 half + c of tokens 2 pair, 2 pair + 1.
template <int D> struct Pairs {
    static constexpr int W = D > 128 ? 2 : 1;
    uint32_t w[2][2][W];
};
template <int D> __device__ __forceinline__ Pairs<D> pair_tokens(const Words<D / 32> &v)
{
    Pairs<D> r;
    constexpr uint32_t LO = 0x0f0f0f0fu, HI = 0xf0f0f0f0u;
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
        for (int i = 0; i < Pairs<D>::W; i++) {
            uint32_t x, y; // the two tokens' bytes
            if constexpr (D == 64)
                x = v.w[p], y = v.w[p] >> 16; // both in one word
            else
                x = v.w[2 * p * Pairs<D>::W + i], y = v.w[(2 * p + 1) * Pairs<D>::W + i];
            r.w[p][0][i] = (x & LO) | ((y << 4) & HI);
            r.w[p][1][i] = ((x >> 4) & LO) | (y & HI);
        }
    return r;
}

struct Geo { // of a launch
    int G, nsplit, chunk, shift;
    int tile, rows; // rows of a tile, and of those the ones that a request may fill
    enum { PACKED, WIDE, PROMPT } kind;
    bool by_request; // a request has at most one tile: the tile's slot is the request
    int64_t slots;
    uint32_t tiles; // slots times kv heads
};

struct Tile {
    int b, row0, rows, n, pos0;  // request, first row, the request's rows, its new tokens, first token's position
    int lo, hi;                  // tokens any row of the tile sees
    bool over;                   // the request is longer than max_kv: its rows become NaN
};

// The tile of a slot.  Slots are handed out so that request b's begin at floor(cu[b] * G / 16) + b, which leaves
// it at least ceil(n_b * G / 16) of them: no sum over the requests' tiles is needed.
__device__ __forceinline__ Tile tile_of(const AttnArgs &a, const Geo &g, int64_t slot, int rows_per_tile)
{
    Tile t;
    int tile = 0;
    if (g.by_request) {
        t.b = (int)slot;
    } else {
        int lo = 0, hi = (int)a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)a.cu_q[mid] * g.G / rows_per_tile + mid <= slot)
                lo = mid;
            else
                hi = mid;
        }
        t.b = lo;
        tile = (int)(slot - ((int64_t)a.cu_q[lo] * g.G / rows_per_tile + lo));
    }
    const int q0 = a.cu_q[t.b], q1 = a.cu_q[t.b + 1];
    t.n = max(0, min(q1, (int)a.T) - q0);
    if (q0 < 0 || tile < 0) // no offsets of a step, or a slot of the rows before the first request's
        t.n = tile = 0;
    t.rows = (int)min((int64_t)t.n * g.G, (int64_t)INT32_MAX);
    t.row0 = tile * rows_per_tile;
    const int len = max(a.kv_lens[t.b], 0);
    t.over = len > a.max_kv || len > a.table_stride << g.shift;
    t.pos0 = len - t.n;
    t.lo = t.hi = 0;
    if (t.row0 < t.rows && !t.over) {
        const int first = t.pos0 + t.row0 / g.G, last = t.pos0 + min(t.rows - 1, t.row0 + rows_per_tile - 1) / g.G;
        t.hi = max(0, last + 1);
        t.lo = a.window > 0 ? (int)max((int64_t)0, first - a.window + 1) & ~(ATT_STEP - 1) : 0;
    }
    return t;
}

// sum and maximum over the four lane groups that hold one row's tokens
__device__ __forceinline__ float groups_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float groups_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Queries are held as binary16 numbers times 2^e, the row's largest from 2^14 up to 2^15: what is far below it keeps
// its bits down to 2^-29 of it, and is off by half the least step, 2^-39 of it, from there on.  (A small element can
// meet a block of keys as much larger.)
constexpr int QUERY_TOP = 15;
// The exponent e for a row whose largest magnitude is am.
__device__ __forceinline__ int row_exponent(float am)
{
    int e = 0;
    if (am > 0.0f && am < INFINITY) { // not finite: the row stays as it is, and its result is not finite either
        (void)frexpf(am, &e);
        e -= QUERY_TOP;
    }
    return e;
}
// What takes a row's scores to powers of two, e its exponent.  Never 0: a masked score of -inf has to stay one (with
// 2^-100, which a scale of 0 and the smallest queries get, every score that is not is 0 for the exponential).
__device__ __forceinline__ float score_scale(float scale, int e)
{
    const float s = ldexpf(fabsf(scale) * 1.44269504088896341f, e);
    return s < 0x1p-100f ? 0x1p-100f : s;
}
template <bool SPLIT> __device__ __forceinline__ void query_halves(const float (&x)[8], int e, bool negate, f16x8 &hi, f16x8 &lo)
{
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float y = ldexpf(negate ? -x[j] : x[j], -e);
        const _Float16 h = (_Float16)y;
        hi[j] = h;
        if constexpr (SPLIT)
            lo[j] = (_Float16)(y - (float)h); // the rest: 22 bits in all
    }
}
template <int DT> __device__ __forceinline__ float load_eight(const typename RowType<DT>::T *q, float (&x)[8])
{
    const RowVec<DT, 8> v = *reinterpret_cast<const RowVec<DT, 8> *>(q);
    float am = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        x[j] = RowType<DT>::get(v.v[j]);
        am = fmaxf(am, fabsf(x[j]));
    }
    return am;
}
// Parts of tiles that are joined later: ROWS sums of weighted values, and COLS references and sums of weights.
template <int D, int ROWS, int COLS> struct PartialOf {
    float acc[ROWS][D];
    float ref[COLS], sum[COLS];
};

// Tiles of PROMPT_ROWS rows or twice as many (kvattn_prompt.hip); binary16 and bfloat16 rows.
hipError_t launch_attn_prompt(int dtype, const AttnArgs &a, const Geo &g, hipStream_t s);

} // namespace lb
