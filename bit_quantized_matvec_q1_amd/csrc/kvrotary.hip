// Queries and keys turned by their positions, and keys and values into the paged 4-bit cache, in one pass over the rows:
//   a_i = position * inv_freq[i],  (x, y) -> factor * (x cos a_i - y sin a_i, y cos a_i + x sin a_i)
// for the pairs (x, y) of the first rotary_dim elements of a head; the turned key is quantised as append_kernel does.
//
// An angle reaches 2^31 (a far position times a frequency of 1), where fp32 has no digits left behind the point, and a key
// a rounding away from a border between two 4-bit codes would change by a whole step.  So angles, sines and products are in
// 64 bits (a position times a frequency has at most 55 significant bits) and the turned value is rounded to fp32 and then to
// the row type: the cache's bytes are those of rotating in 64 bits and then appending.  The hardware's fp64 rate is its fp32
// rate without packing, so this is not what a long prompt waits for; the sines are, if every head computes them again.
// Hence the split: a workgroup takes 2048 / D tokens and a run of heads, computes the tokens' sines and cosines once,
// spread over its threads, through LDS, and keeps each lane's in registers over the heads.
#include "kvcache_device.h"

namespace lb {

template <int DT, int D> __global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int shift, int per)
{
    using R = RowType<DT>;
    constexpr int LR = D / 8, RW = 256 / LR; // lanes a row, rows (tokens) a workgroup
    __shared__ double2 turn[RW * (D / 2)];   // 16 KiB
    __shared__ uint32_t lds[256];
    const int64_t t0 = (int64_t)blockIdx.x * RW, t = t0 + threadIdx.x / LR;
    const int at = threadIdx.x % LR, e = 8 * at, half = (int)a.rotary_dim / 2;
    const int nt = (int)min((int64_t)RW, a.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += 256) {
        const int r = i / half;
        double sn, cs;
        sincos((double)a.positions[t0 + r] * (double)a.inv_freq[i - r * half], &sn, &cs);
        turn[i] = make_double2(cs * (double)a.factor, sn * (double)a.factor);
    }
    __syncthreads();
    const int64_t slot = t < a.T ? a.slots[t] : -1;
    const bool row = slot >= 0 && slot < a.pages << shift; // a row without a slot is left out, its queries too
    const bool turned = row && e < a.rotary_dim;
    // element e + j becomes x * c + other * s, the other one being j ^ 1 here, or element j of the lane's partner chunk
    double c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        c[j] = 1.0, s[j] = 0.0;
        if (turned) {
            const bool first = a.pairs ? (j & 1) == 0 : e < half;
            const double2 v = turn[threadIdx.x / LR * half + (a.pairs ? 4 * at + j / 2 : first ? e + j : e - half + j)];
            c[j] = v.x, s[j] = first ? -v.y : v.y;
        }
    }
    const int partner = e < half ? e + half : e - half; // (halves)

    // 8 elements of the lane's row at p (the head's first element), turned or as they are
    auto load8 = [&](const typename R::T *p, float (&x)[8]) {
        const RowVec<DT, 8> v = *reinterpret_cast<const RowVec<DT, 8> *>(p);
#pragma unroll
        for (int j = 0; j < 8; j++)
            x[j] = R::get(v.v[j]);
    };
    auto turned8 = [&](const typename R::T *p, float (&x)[8]) {
        load8(p + e, x);
        if (!turned)
            return;
        float o[8];
        if (a.pairs) { // uniform
#pragma unroll
            for (int j = 0; j < 8; j++)
                o[j] = x[j ^ 1];
        } else {
            load8(p + partner, o);
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            x[j] = R::get(R::put((float)((double)x[j] * c[j] + (double)o[j] * s[j])));
    };

    const int q_heads = (int)a.q_heads, heads = q_heads + (int)a.kv_heads;
    const int h1 = min((int)(blockIdx.y + 1) * per, heads);
    for (int h = blockIdx.y * per; h < h1; h++) { // uniform
        if (h < q_heads) {
            if (row) {
                float x[8];
                turned8(static_cast<const typename R::T *>(a.q) + t * a.q_stride + (int64_t)h * D, x);
                // (all lanes of the row have read it: they are in one wave, and their partners' elements are used above)
                typename R::T *to = static_cast<typename R::T *>(a.q_out) + t * a.q_out_stride + (int64_t)h * D + e;
                constexpr int W = DT == LB_F32 ? 4 : 8; // 16-byte stores
#pragma unroll
                for (int i = 0; i < 8; i += W) {
                    RowVec<DT, W> o;
#pragma unroll
                    for (int j = 0; j < W; j++)
                        o.v[j] = R::put(x[i + j]);
                    *reinterpret_cast<RowVec<DT, W> *>(to + i) = o;
                }
            }
        } else {
            const int head = h - q_heads;
            float xk[8] = {}, xv[8] = {};
            if (row) {
                turned8(static_cast<const typename R::T *>(a.k) + t * a.k_stride + (int64_t)head * D, xk);
                load8(static_cast<const typename R::T *>(a.v) + t * a.v_stride + (int64_t)head * D + e, xv);
            }
            write_row<DT, D>(slot_of(a.cache, a.pages, a.kv_heads, D, slot, head, shift), shift, xk, xv, lds);
        }
    }
}

template <int DT> static hipError_t rotary_d(const RotaryArgs &a, hipStream_t s)
{
    const int shift = log2_of(a.page_tokens);
    const int64_t groups = (a.T + 2048 / a.head_dim - 1) / (2048 / a.head_dim), heads = a.q_heads + a.kv_heads;
    // heads a workgroup: as many as leave 4096 workgroups (two rounds of eight on each CU), so that sines are computed
    // for few of them again
    int64_t per = groups * heads / 4096;
    per = per < 1 ? 1 : per > heads ? heads : per;
    const dim3 grid((unsigned)groups, (unsigned)((heads + per - 1) / per));
    switch (a.head_dim) {
    case 64:
        hipLaunchKernelGGL((rotary_kernel<DT, 64>), grid, dim3(256), 0, s, a, shift, (int)per);
        return hipGetLastError();
    case 128:
        hipLaunchKernelGGL((rotary_kernel<DT, 128>), grid, dim3(256), 0, s, a, shift, (int)per);
        return hipGetLastError();
    case 256:
        hipLaunchKernelGGL((rotary_kernel<DT, 256>), grid, dim3(256), 0, s, a, shift, (int)per);
        return hipGetLastError();
    }
    return hipErrorInvalidValue;
}

hipError_t launch_kv_append_rotary(int dtype, const RotaryArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? rotary_d<LB_F32>(a, s) : dtype == LB_BF16 ? rotary_d<LB_BF16>(a, s) : rotary_d<LB_F16>(a, s);
}

} // namespace lb
