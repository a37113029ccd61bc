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
#include "kvcache_device.h"

namespace lb {

// A workgroup takes 2048 / D tokens of one head, as the four tokens of a quad share the lines of its value codes and
// scales: written from different workgroups, and so from different L2s, each line would go out in parts.
template <int DT, int D> __global__ __launch_bounds__(256) void append_kernel(RowsArgs a, int shift)
{
    using R = RowType<DT>;
    constexpr int LR = D / 8; // lanes a row
    __shared__ uint32_t lds[256];
    const uint32_t group = blockIdx.x / (uint32_t)a.kv_heads;
    const int64_t t = (int64_t)group * (256 / LR) + threadIdx.x / LR;
    const int head = (int)(blockIdx.x - group * (uint32_t)a.kv_heads), at = threadIdx.x % LR;
    Slot s = {nullptr, 0};
    if (t < a.T)
        s = slot_of(a, t, head, shift);
    auto load = [&](const void *p, int64_t stride, float (&x)[8]) {
        const RowVec<DT, 8> v = *reinterpret_cast<const RowVec<DT, 8> *>(static_cast<const typename R::T *>(p) + t * stride + (int64_t)head * D + 8 * at);
#pragma unroll
        for (int i = 0; i < 8; i++)
            x[i] = R::get(v.v[i]);
    };
    write_row<DT, D>(s, shift, [&](float (&xk)[8], float (&xv)[8]) { load(a.k, a.k_stride, xk), load(a.v, a.v_stride, xv); }, lds);
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
