// Rows into the paged 4-bit cache, and back.  32 consecutive values of a head share the scale
// d = fp16_rne(amax / 6) (the fp32 quotient), and each value becomes the E2M1 number nearest to x / d, ties to
// the even code.  The borders between neighbouring E2M1 numbers are .25 .75 1.25 1.75 2.5 3.5 5, and d times one
// of them has 11 + 3 significant bits: the comparisons |x| against d * border are exact in fp32, without a
// division, for every input type, and so is the code.
//
// Both directions are bound by HBM (2 to 4 bytes a value in or out, 9/16 byte in the cache).
#include "serve_internal.h"

namespace lb {

constexpr uint32_t F16_NAN = 0x7e00u;

// maximum over aligned groups of 4 (quads) or 16 lanes, of bit patterns of magnitudes: a NaN's pattern is above
// an infinity's, and that above every number's
template <int L> __device__ __forceinline__ uint32_t group_umax(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false)); // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false)); // quad_perm [2,3,0,1]
    if (L == 16) {
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false)); // row_half_mirror
        v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false)); // row_mirror
    }
    return v;
}

// The block's scale from its magnitude's bit pattern: saturated at the largest binary16, NaN if a value is not
// finite (the block then reads back as NaN rather than as some number).
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax)
{
    if (amax >= 0x7f800000u)
        return F16_NAN;
    return __half_as_ushort(__float2half_rn(fminf(__uint_as_float(amax) / 6.0f, 65504.0f)));
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

// 16 lanes a row (token and head).  Keys: a lane takes D/16 consecutive elements.  Values: a lane takes the
// column c = lane, elements 16 n + c, whose codes are its D/32 consecutive bytes of the record.
template <int DT, int D> __global__ __launch_bounds__(256) void append_kernel(RowsArgs a, int shift)
{
    using R = RowType<DT>;
    constexpr int E = D / 16, NB = D / 32;
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    if (row >= a.T * a.kv_heads) // whole groups of 16 lanes leave: the DPP maxima stay within a group
        return;
    const int64_t t = row / a.kv_heads;
    const int head = (int)(row - t * a.kv_heads), P = 1 << shift, c = threadIdx.x & 15;
    const Slot s = slot_of(a, t, head, shift);
    if (!s.rec)
        return;
    const typename R::T *k = static_cast<const typename R::T *>(a.k) + t * a.k_stride + (int64_t)head * D;
    const typename R::T *v = static_cast<const typename R::T *>(a.v) + t * a.v_stride + (int64_t)head * D;

    // keys, in runs of 8 elements (a quarter g of a block b, four codes' bytes each in the record); D = 64 has
    // half a run a lane
    constexpr int RUN = E < 8 ? E : 8, LB = 32 / RUN; // lanes a block
    static_assert(LB == 4 || LB == 8, "");
#pragma unroll
    for (int r = 0; r < E / RUN; r++) {
        const int e0 = (r * 16 + c) * RUN; // first element
        const RowVec<DT, RUN> x = *reinterpret_cast<const RowVec<DT, RUN> *>(k + e0);
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < RUN; i++)
            am = max(am, __float_as_uint(R::get(x.v[i])) & 0x7fffffffu);
        am = group_umax<4>(am);
        if (LB == 8)
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x141, 0xF, 0xF, false)); // row_half_mirror
        const uint32_t sb = scale_bits(am);
        const float d = half_bits_to_float((uint16_t)sb);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < RUN; i++)
            w |= (d > 0.0f ? e2m1_code(R::get(x.v[i]), d) : 0u) << (4 * i);
        uint8_t *to = s.rec + kv_k_byte(D, s.o, (e0 >> 3) & 3, e0 >> 5) + (e0 & 7) / 2;
        if constexpr (RUN == 8)
            *reinterpret_cast<uint32_t *>(to) = w;
        else
            *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
        if ((e0 & 31) == 0)
            *reinterpret_cast<uint16_t *>(s.rec + kv_scale_byte(P, D, 0, s.o, e0 >> 5)) = (uint16_t)sb;
    }

    uint64_t w = 0;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const float x0 = R::get(v[32 * b + c]), x1 = R::get(v[32 * b + 16 + c]);
        const uint32_t am = group_umax<16>(max(__float_as_uint(x0) & 0x7fffffffu, __float_as_uint(x1) & 0x7fffffffu));
        const uint32_t sb = scale_bits(am);
        const float d = half_bits_to_float((uint16_t)sb);
        if (d > 0.0f)
            w |= (uint64_t)(e2m1_code(x0, d) | e2m1_code(x1, d) << 4) << (8 * b);
        if (c == 0)
            *reinterpret_cast<uint16_t *>(s.rec + kv_scale_byte(P, D, 1, s.o, b)) = (uint16_t)sb;
    }
    uint8_t *to = s.rec + kv_v_byte(P, D, s.o, c);
    if constexpr (NB == 2)
        *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
    else if constexpr (NB == 4)
        *reinterpret_cast<uint32_t *>(to) = (uint32_t)w;
    else
        *reinterpret_cast<uint64_t *>(to) = w;
}

// A lane gives 8 consecutive elements of a row's key and of its value; a row without a slot is zeros.
template <int DT, int D> __global__ __launch_bounds__(256) void read_kernel(RowsArgs a, int shift)
{
    using R = RowType<DT>;
    constexpr int LR = D / 8, NB = D / 32; // lanes a row
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LR;
    if (row >= a.T * a.kv_heads)
        return;
    const int64_t t = row / a.kv_heads;
    const int head = (int)(row - t * a.kv_heads), P = 1 << shift, e0 = (threadIdx.x % LR) * 8, b = e0 >> 5;
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
    const int64_t rows = a.T * a.kv_heads;
    const int per = append ? 16 : 2048 / (int)a.head_dim; // rows a workgroup
    const dim3 grid((unsigned)((rows + per - 1) / per));
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
