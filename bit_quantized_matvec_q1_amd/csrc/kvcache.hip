// Rows into the paged 4-bit cache, and back.  32 consecutive values of a head share the scale
// d = fp16_rne(amax * fp32(1/6)), and each value becomes the E2M1 number nearest to x / d, ties to the even code.  The
// borders between neighbouring E2M1 numbers are .25 .75 1.25 1.75 2.5 3.5 5, and d times one
// of them has 11 + 3 significant bits: the comparisons |x| against d * border are exact in fp32, without a
// division, for every input type, and so is the code.
//
// Both directions are bound by HBM (2 to 4 bytes a value in or out, 9/16 byte in the cache).  16384 tokens of 8 heads
// of 128: 16-bit rows appended in 18.6 us (86 MB, 4.6 TB/s), fp32 rows in 35.6 us (153 MB, 4.3 TB/s: seven comparisons
// a value in place of a conversion); read back as fp32 in 34 us (153 MB, 4.5 TB/s), as bfloat16 in 26 us (86 MB, 3.3
// TB/s: there the single bytes of values, eight loads a lane, show).  A large copy reaches 4.7 to 5.0 here.
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
__device__ __forceinline__ Slot slot_of(const RowsArgs &a, int64_t t, int head, int shift)
{
    const int64_t s = a.slots[t];
    if (s < 0 || s >= a.pages << shift)
        return {nullptr, 0};
    return {a.cache + ((s >> shift) * a.kv_heads + head) * kv_record_bytes((int64_t)1 << shift, a.head_dim), (int)(s & ((1 << shift) - 1))};
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

// A workgroup takes 2048 / D tokens of one head, as the four tokens of a quad share the lines of its value codes and
// scales: written from different workgroups, and so from different L2s, each line would go out in parts.  A lane has
// a quarter of a block, 8 consecutive elements, of a row's key and of its value.  The key's four bytes of codes lie
// together in the record.  The value's go through LDS: there a row's bytes are in the record's order (column c =
// element mod 16, then block), each made of two lanes' codes, and every lane takes four of them.
template <int DT, int D> __global__ __launch_bounds__(256) void append_kernel(RowsArgs a, int shift)
{
    using R = RowType<DT>;
    constexpr int LR = D / 8, NB = D / 32; // lanes a row
    __shared__ uint32_t lds[256];
    const uint32_t group = blockIdx.x / (uint32_t)a.kv_heads;
    const int64_t t = (int64_t)group * (256 / LR) + threadIdx.x / LR;
    const int head = (int)(blockIdx.x - group * (uint32_t)a.kv_heads), P = 1 << shift;
    const int at = threadIdx.x % LR, b = at >> 2, g = at & 3;
    const bool row = t < a.T;
    Slot s = {nullptr, 0};
    if (row)
        s = slot_of(a, t, head, shift);
    uint32_t wv = 0;
    if (s.rec) { // whole rows: the quads' maxima stay within them
        auto load = [&](const void *p, int64_t stride, float (&x)[8]) {
            const RowVec<DT, 8> v = *reinterpret_cast<const RowVec<DT, 8> *>(static_cast<const typename R::T *>(p) + t * stride + (int64_t)head * D + 8 * at);
            uint32_t am = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                x[i] = R::get(v.v[i]);
                am = max(am, __float_as_uint(x[i]) & 0x7fffffffu);
            }
            return am;
        };
        float xk[8], xv[8];
        const uint32_t ak = load(a.k, a.k_stride, xk), av = load(a.v, a.v_stride, xv);
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
#pragma unroll
    for (int j = 0; j < 4; j++)
        mine[(8 * (g & 1) + 2 * j + (g >> 1)) * NB + b] = (uint8_t)(bytes >> (8 * j));
    __syncthreads();
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

// A lane gives 8 consecutive elements of a row's key and of its value; a row without a slot is zeros.
template <int DT, int D> __global__ __launch_bounds__(256) void read_kernel(RowsArgs a, int shift)
{
    using R = RowType<DT>;
    constexpr int LR = D / 8, NB = D / 32; // lanes a row
    const uint32_t group = blockIdx.x / (uint32_t)a.kv_heads;
    const int64_t t = (int64_t)group * (256 / LR) + threadIdx.x / LR;
    const int head = (int)(blockIdx.x - group * (uint32_t)a.kv_heads), P = 1 << shift, e0 = (threadIdx.x % LR) * 8, b = e0 >> 5;
    if (t >= a.T)
        return;
    const Slot s = slot_of(a, t, head, shift);
    float xk[8], xv[8];
    if (s.rec) {
        const uint32_t wk = *reinterpret_cast<const uint32_t *>(s.rec + kv_k_byte(D, s.o, (e0 >> 3) & 3, b));
        const float dk = half_bits_to_float(*reinterpret_cast<const uint16_t *>(s.rec + kv_scale_byte(P, D, 0, s.o, b)));
        const float dv = half_bits_to_float(*reinterpret_cast<const uint16_t *>(s.rec + kv_scale_byte(P, D, 1, s.o, b)));
        const int sh = (e0 & 16) ? 4 : 0; // the upper codes of a byte are the block's second half
        const uint8_t *v = s.rec + kv_v_byte(P, D, s.o, e0 & 15) + b;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            xk[i] = e2m1_value(wk >> (4 * i)) * dk;
            xv[i] = e2m1_value((uint32_t)v[i * 4 * NB] >> sh) * dv;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            xk[i] = xv[i] = 0.0f;
    }
    auto put = [&](void *p, int64_t stride, const float (&x)[8]) {
        typename R::T *to = static_cast<typename R::T *>(p) + t * stride + (int64_t)head * D + e0;
        constexpr int W = DT == LB_F32 ? 4 : 8; // 16-byte stores
#pragma unroll
        for (int i = 0; i < 8; i += W) {
            RowVec<DT, W> o;
#pragma unroll
            for (int j = 0; j < W; j++)
                o.v[j] = R::put(x[i + j]);
            *reinterpret_cast<RowVec<DT, W> *>(to + i) = o;
        }
    };
    put(a.k, a.k_stride, xk);
    put(a.v, a.v_stride, xv);
}

static int log2_of(int64_t p)
{
    int s = 0;
    while (((int64_t)1 << s) < p)
        s++;
    return s;
}

template <int DT> static hipError_t rows_d(const RowsArgs &a, bool append, hipStream_t s)
{
    const int shift = log2_of(a.page_tokens);
    const int per = 2048 / (int)a.head_dim; // tokens a workgroup
    const dim3 grid((unsigned)((a.T + per - 1) / per * a.kv_heads));
#define LB_ROWS(d)                                                                                            \
    case d:                                                                                                   \
        if (append)                                                                                           \
            hipLaunchKernelGGL((append_kernel<DT, d>), grid, dim3(256), 0, s, a, shift);                        \
        else                                                                                                  \
            hipLaunchKernelGGL((read_kernel<DT, d>), grid, dim3(256), 0, s, a, shift);                          \
        return hipGetLastError();
    switch (a.head_dim) {
        LB_ROWS(64) LB_ROWS(128) LB_ROWS(256)
    }
#undef LB_ROWS
    return hipErrorInvalidValue;
}

static hipError_t rows(int dtype, const RowsArgs &a, bool append, hipStream_t s)
{
    return dtype == LB_F32 ? rows_d<LB_F32>(a, append, s) : dtype == LB_BF16 ? rows_d<LB_BF16>(a, append, s) : rows_d<LB_F16>(a, append, s);
}

hipError_t launch_kv_append(int dtype, const RowsArgs &a, hipStream_t s) { return rows(dtype, a, true, s); }
hipError_t launch_kv_read(int dtype, const RowsArgs &a, hipStream_t s) { return rows(dtype, a, false, s); }

} // namespace lb
