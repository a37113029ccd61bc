// The 4-bit cache's rows, for the kernels that write and read them: codes, scales, and a row's place.
#pragma once

#include "serve_internal.h"

namespace lb {

constexpr uint32_t F16_NAN = 0x7e00u;

// maximum over quads of lanes of bit patterns of magnitudes: a NaN's pattern is above an infinity's, and that above
// every number's
__device__ __forceinline__ uint32_t quad_umax(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false)); // quad_perm [1,0,3,2]
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false)); // quad_perm [2,3,0,1]
}

// The block's scale from its magnitude's bit pattern: saturated at the largest binary16, NaN if a value is not
// finite (the block then reads back as NaN rather than as some number).  The format takes the product with fp32(1/6)
// for amax / 6: one rounding like a quotient's, without a division, and for 6 times a binary16 it rounds to that
// binary16, so that fp32 rows read back and appended again keep their values (scales below binary16's normal range
// may not: there the largest code need not be 6).
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax)
{
    if (amax >= 0x7f800000u)
        return F16_NAN;
    return __half_as_ushort(__float2half_rn(fminf(__uint_as_float(amax) * (1.0f / 6.0f), 65504.0f)));
}

__device__ __forceinline__ uint32_t e2m1_code(float x, float d)
{
    const float a = fabsf(x);
    uint32_t c = (uint32_t)(a > d * 0.25f) + (uint32_t)(a >= d * 0.75f) + (uint32_t)(a > d * 1.25f) + (uint32_t)(a >= d * 1.75f) +
                 (uint32_t)(a > d * 2.5f) + (uint32_t)(a >= d * 3.5f) + (uint32_t)(a > d * 5.0f);
    return c | (x < 0.0f ? 8u : 0u);
}

__device__ __forceinline__ float e2m1_value(uint32_t c)
{
    const uint32_t m = c & 7u; // 0 .5 1 1.5 2 3 4 6
    const float v = m < 2u ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

struct Slot {
    uint8_t *rec; // the record of (page, head), null if the slot is none
    int o;        // token within the page
};
// slot s of a cache of `pages` pages of 2^shift tokens
__device__ __forceinline__ Slot slot_of(uint8_t *cache, int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t s, int head, int shift)
{
    if (s < 0 || s >= pages << shift)
        return {nullptr, 0};
    return {cache + ((s >> shift) * kv_heads + head) * kv_record_bytes((int64_t)1 << shift, head_dim), (int)(s & ((1 << shift) - 1))};
}
__device__ __forceinline__ Slot slot_of(const RowsArgs &a, int64_t t, int head, int shift)
{
    return slot_of(a.cache, a.pages, a.kv_heads, a.head_dim, a.slots[t], head, shift);
}

// Eight values' codes, element i in nibble i, for the scale d (0 and NaN: none).
template <int DT> __device__ __forceinline__ uint32_t eight_codes(const float (&x)[8], float d)
{
    if (!(d > 0.0f))
        return 0;
    uint32_t w = 0;
    if constexpr (DT == LB_F32) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            w |= e2m1_code(x[i], d) << (4 * i);
    } else {
        // 16-bit values: x has at most 11 bits and d * border 14, so x / d is either a border or over 2^-15 of itself
        // away from it, and a quotient right to 2^-23, and exact where it is a short number, rounds as the true one
        // does, to the nearest and ties to even, by the conversion.  (fp32 values can lie closer to a border than
        // their quotient's rounding, hence the comparisons.)  Past 6 it saturates.
        const float r = __builtin_amdgcn_rcpf(d);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float t = x[i] * r;
            y[i] = fmaf(fmaf(-t, d, x[i]), r, t); // also makes a -0 a 0
        }
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
    }
    return w;
}

// log2 of a power of two
inline int log2_of(int64_t p)
{
    int s = 0;
    while (((int64_t)1 << s) < p)
        s++;
    return s;
}

// Orders a wave's LDS writes before its lanes' reads of them (and those before the next writes).
__device__ __forceinline__ void row_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One row's key and value into the record of its slot, by the D / 8 lanes of the row (all of them in one wave, 256 / (D / 8)
// rows a workgroup of 256): lane `at` of the row has elements 8 at .. 8 at + 7 of both, a quarter of a block.  The key's
// four bytes of codes lie together in the record.  The value's go through LDS (`lds`, a dword a thread): there a row's
// bytes are in the record's order (column c = element mod 16, then block), each made of two lanes' codes, and every lane
// takes four of them.  Lanes of a row without a slot (s.rec null) come along and write nothing; `values` puts the others'
// elements into its two arguments (there, where they are used: loaded under a branch of their own before this one, they cost
// 16384 bf16 tokens of 8 heads of 128 17.2 us instead of 15.5, and fp32 ones of a decode step 3.4 instead of 3.2).
template <int DT, int D, typename Values> __device__ __forceinline__ void write_row(const Slot &s, int shift, Values &&values, uint32_t *lds)
{
    constexpr int LR = D / 8, NB = D / 32;
    const int P = 1 << shift, at = threadIdx.x % LR, b = at >> 2, g = at & 3;
    uint32_t wv = 0;
    if (s.rec) { // whole rows: the quads' maxima stay within them
        float xk[8], xv[8];
        values(xk, xv);
        uint32_t ak = 0, av = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            ak = max(ak, __float_as_uint(xk[i]) & 0x7fffffffu);
            av = max(av, __float_as_uint(xv[i]) & 0x7fffffffu);
        }
        const uint32_t dk = scale_bits(quad_umax(ak)), dv = scale_bits(quad_umax(av));
        *reinterpret_cast<uint32_t *>(s.rec + kv_k_byte(D, s.o, g, b)) = eight_codes<DT>(xk, half_bits_to_float((uint16_t)dk));
        wv = eight_codes<DT>(xv, half_bits_to_float((uint16_t)dv));
        if (g < 2) // one lane of a block writes the key's scale, another the value's
            *reinterpret_cast<uint16_t *>(s.rec + kv_scale_byte(P, D, g, s.o, b)) = (uint16_t)(g ? dv : dk);
    }
    // columns 8 (g & 1) + 0, 2, 4, 6 in the lanes with the lower codes (g < 2), and 1, 3, 5, 7 in the others
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)wv, 0x4E, 0xF, 0xF, false); // quad_perm [2,3,0,1]
    const uint32_t bytes = g < 2 ? (wv & 0x0f0f0f0fu) | ((other & 0x0f0f0f0fu) << 4) : ((other >> 4) & 0x0f0f0f0fu) | (wv & 0xf0f0f0f0u);
    uint8_t *mine = reinterpret_cast<uint8_t *>(lds) + threadIdx.x / LR * (D / 2);
    row_fence(); // a wave's LDS accesses run in their order: only the compiler has to keep it
#pragma unroll
    for (int j = 0; j < 4; j++)
        mine[(8 * (g & 1) + 2 * j + (g >> 1)) * NB + b] = (uint8_t)(bytes >> (8 * j));
    row_fence();
    if (!s.rec)
        return;
    const uint32_t out = lds[threadIdx.x]; // bytes 4 at .. 4 at + 3 of the row
    if constexpr (NB == 2) { // two columns
        *reinterpret_cast<uint16_t *>(s.rec + kv_v_byte(P, D, s.o, 2 * at)) = (uint16_t)out;
        *reinterpret_cast<uint16_t *>(s.rec + kv_v_byte(P, D, s.o, 2 * at + 1)) = (uint16_t)(out >> 16);
    } else {
        *reinterpret_cast<uint32_t *>(s.rec + kv_v_byte(P, D, s.o, at * 4 / NB) + at * 4 % NB) = out;
    }
}

} // namespace lb
