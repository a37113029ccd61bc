// Queries and keys turned by their positions, and keys and values into the paged 4-bit cache, in one pass over the rows:
//   a_i = position * inv_freq[i],  (x, y) -> factor * (x cos a_i - y sin a_i, y cos a_i + x sin a_i)
// for the pairs (x, y) of the first rotary_dim elements of a head; the turned key is quantised as append_kernel does.
//
// An angle reaches 2^31 (a far position times a frequency of 1), where fp32 has no digits left behind the point, and a key
// a rounding away from a border between two 4-bit codes would change by a whole step.  So angles, sines and products are in
// 64 bits (a position times a frequency has at most 55 significant bits) and the turned value is rounded to fp32 and then to
// the row type: the cache's bytes are those of rotating in 64 bits and then appending.
//
// The rows are what has to move, but 64 bits cost more than their bytes if done carelessly: sines computed again for every
// head, elements converted twice.  Hence the split: a workgroup takes 2048 / D tokens and a run of heads (queries, or keys
// and values), and computes the tokens' sines and cosines once, spread over its threads, through LDS.  A lane of a query has
// four whole pairs, four elements of either half of the turned part, and keeps their sines over the heads; the next heads'
// elements are loaded ahead.  (Keys are written by lanes of eight consecutive elements, which read the other half's again.)
//
// Measured: 16384 bf16 rows of 32 query and 2 x 8 key and value heads of 128: 76 to 84 us, 355 MB, 4.2 to 4.7 TB/s of the 5.1
// that a large copy reaches (120 us with sines by head and the library's functions); 32 fp32 rows 6 us.
#include "kvcache_device.h"

namespace lb {

// Sine and cosine in 64 bits.  Up to 2^30 the angle is brought to [-pi/4, pi/4] by n pi/2, n < 2^30, with pi/2 as a sum of
// two: the first fma is exact (n times 53 bits, less an angle of the same size), the second leaves 2^-53 of the rest.  There
// the Taylor series, whose next terms are below 2^-57.  Beyond, and for what is no number, the library's.
__device__ __forceinline__ void sin_cos(double a, double *sn, double *cs)
{
    if (!(fabs(a) < 1073741824.0)) {
        sincos(a, sn, cs);
        return;
    }
    const double n = rint(a * 0x1.45f306dc9c883p-1);                              // 2 / pi
    const double r = fma(-n, 0x1.1a62633145c07p-54, fma(-n, 0x1.921fb54442d18p0, a)); // pi / 2
    const double z = r * r;
    double s = 1.0 / 355687428096000.0, c = 1.0 / 20922789888000.0; // 17!, 16!
    s = fma(s, z, -1.0 / 1307674368000.0), c = fma(c, z, -1.0 / 87178291200.0);
    s = fma(s, z, 1.0 / 6227020800.0), c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, -1.0 / 39916800.0), c = fma(c, z, -1.0 / 3628800.0);
    s = fma(s, z, 1.0 / 362880.0), c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, -1.0 / 5040.0), c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, 1.0 / 120.0), c = fma(c, z, 1.0 / 24.0);
    s = fma(s, z, -1.0 / 6.0), c = fma(c, z, -0.5);
    s = fma(s * z, r, r), c = fma(c, z, 1.0);
    const int q = (int)n;
    const double u = q & 1 ? c : s, v = q & 1 ? s : c;
    *sn = q & 2 ? -u : u;
    *cs = (q + 1) & 2 ? -v : v;
}

// Two fp32 values to the row type, by the hardware's conversion where it has one of its own.
template <int DT> __device__ __forceinline__ void put2(typename RowType<DT>::T *to, float a, float b)
{
    if constexpr (DT == LB_BF16) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        const b2 v = __builtin_convertvector((f2){a, b}, b2);
        __builtin_memcpy(to, &v, 4);
    } else {
        to[0] = RowType<DT>::put(a), to[1] = RowType<DT>::put(b);
    }
}

template <int DT, int D, int H> __global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int shift, int q_runs, int q_per, int kv_per)
{
    using R = RowType<DT>;
    using T = typename R::T;
    constexpr int LR = D / 8, RW = 256 / LR; // lanes a row, rows (tokens) a workgroup
    __shared__ double2 turn[RW * (D / 2)];   // 16 KiB
    __shared__ uint32_t lds[256];
    const int64_t t0 = (int64_t)blockIdx.x * RW, t = t0 + threadIdx.x / LR;
    const int at = threadIdx.x % LR, rd = (int)a.rotary_dim, half = rd / 2;
    const int nt = (int)min((int64_t)RW, a.T - t0);
    const int64_t slot = t < a.T ? a.slots[t] : -1;
    const bool row = slot >= 0 && slot < a.pages << shift; // a row without a slot is left out, its queries too
    const double2 *mine = turn + threadIdx.x / LR * half;
    auto sines = [&] {
        for (int i = threadIdx.x; i < nt * half; i += 256) {
            const int r = i / half;
            double sn, cs;
            sin_cos((double)a.positions[t0 + r] * (double)a.inv_freq[i - r * half], &sn, &cs);
            turn[i] = make_double2(cs * (double)a.factor, sn * (double)a.factor);
        }
        __syncthreads();
    };

    if ((int)blockIdx.y < q_runs) { // uniform
        const int h0 = blockIdx.y * q_per, h1 = min(h0 + q_per, (int)a.q_heads);
        // lanes below rd / 8 have four pairs of the turned part, the others eight of the elements behind it
        const bool turned = 8 * at < rd, halves = turned && !a.pairs;
        const int e0 = halves ? 4 * at : 8 * at, e1 = halves ? half + 4 * at : 8 * at + 4;
        const T *from = static_cast<const T *>(a.q) + t * a.q_stride;
        T *to = static_cast<T *>(a.q_out) + t * a.q_out_stride;
        using V = RowVec<DT, 4>;
        V v0[H] = {}, v1[H] = {};
        auto load = [&](int h) {
#pragma unroll
            for (int i = 0; i < H; i++) {
                const int hn = min(h + i, h1 - 1);
                v0[i] = *reinterpret_cast<const V *>(from + hn * D + e0), v1[i] = *reinterpret_cast<const V *>(from + hn * D + e1);
            }
        };
        if (row)
            load(h0);
        sines();
        if (!row)
            return;
        double c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const double2 v = mine[turned ? 4 * at + j : 0];
            c[j] = v.x, s[j] = v.y;
        }
        for (int g = h0; g < h1; g += H) {
            V w0[H], w1[H];
#pragma unroll
            for (int i = 0; i < H; i++)
                w0[i] = v0[i], w1[i] = v1[i];
            load(g + H);
#pragma unroll
            for (int i = 0; i < H; i++) {
                const int h = g + i;
                if (h >= h1)
                    break;
                const V x0 = w0[i], x1 = w1[i];
                V o0 = x0, o1 = x1;
                if (turned) {
                    float u[8];
                    if (a.pairs) { // uniform
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const double x = (double)R::get((j < 2 ? x0 : x1).v[2 * j % 4]), y = (double)R::get((j < 2 ? x0 : x1).v[2 * j % 4 + 1]);
                            u[2 * j] = (float)(x * c[j] - y * s[j]), u[2 * j + 1] = (float)(y * c[j] + x * s[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const double x = (double)R::get(x0.v[j]), y = (double)R::get(x1.v[j]);
                            u[j] = (float)(x * c[j] - y * s[j]), u[4 + j] = (float)(y * c[j] + x * s[j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; j += 2)
                        put2<DT>(o0.v + j, u[j], u[j + 1]), put2<DT>(o1.v + j, u[4 + j], u[5 + j]);
                }
                // (in place: a lane reads and writes its own elements only)
                *reinterpret_cast<V *>(to + h * D + e0) = o0, *reinterpret_cast<V *>(to + h * D + e1) = o1;
            }
        }
        return;
    }

    // keys and values: a lane has elements e .. e + 7
    const int e = 8 * at, partner = e >= rd ? e : e < half ? e + half : e - half;
    const bool turned = e < rd, first = e < half;
    const int h0 = ((int)blockIdx.y - q_runs) * kv_per, h1 = min(h0 + kv_per, (int)a.kv_heads);
    const T *kf = static_cast<const T *>(a.k) + t * a.k_stride, *vf = static_cast<const T *>(a.v) + t * a.v_stride + e;
    using V = RowVec<DT, 8>;
    V k0 = {}, k1 = {}, v0 = {};
    auto ahead = [&](int h) {
        if (row)
            k0 = *reinterpret_cast<const V *>(kf + (int64_t)h * D + e), k1 = *reinterpret_cast<const V *>(kf + (int64_t)h * D + partner),
            v0 = *reinterpret_cast<const V *>(vf + (int64_t)h * D);
    };
    ahead(h0);
    sines();
    double c[8], s[8]; // of elements e + j, the sine with the sign that its product has (pairs: four, each twice)
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const double2 v = mine[!turned ? 0 : a.pairs ? 4 * at + j / 2 : first ? e + j : e - half + j];
        c[j] = v.x, s[j] = (a.pairs ? (j & 1) == 0 : first) ? -v.y : v.y;
    }
    for (int h = h0; h < h1; h++) { // uniform
        const V kx = k0, ko = k1, vx = v0;
        ahead(min(h + 1, h1 - 1));
        float xk[8], xv[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            xk[j] = R::get(kx.v[j]), xv[j] = R::get(vx.v[j]);
        if (row && turned) {
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const double x = (double)xk[j] * c[j], y = (double)R::get(a.pairs ? kx.v[j ^ 1] : ko.v[j]) * s[j];
                u[j] = (float)(x + y);
            }
            T w[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                put2<DT>(w + j, u[j], u[j + 1]);
#pragma unroll
            for (int j = 0; j < 8; j++)
                xk[j] = R::get(w[j]);
        }
        auto values = [&](float (&wk)[8], float (&wv)[8]) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                wk[j] = xk[j], wv[j] = xv[j];
        };
        write_row<DT, D>(slot_of(a.cache, a.pages, a.kv_heads, D, slot, h, shift), shift, values, lds);
    }
}

template <int DT> static hipError_t rotary_d(const RotaryArgs &a, hipStream_t s)
{
    const int shift = log2_of(a.page_tokens);
    const int64_t groups = (a.T + 2048 / a.head_dim - 1) / (2048 / a.head_dim), heads = a.q_heads + a.kv_heads;
    // heads a workgroup: as many as leave some 2048 workgroups, eight on each CU, so that sines are computed for few of them
    // again
    int64_t runs = 2048 / groups;
    runs = runs < 1 ? 1 : runs > heads ? heads : runs;
    const int64_t per = (heads + runs - 1) / runs, q_per = per < a.q_heads ? per : a.q_heads, kv_per = per < a.kv_heads ? per : a.kv_heads;
    const int64_t q_runs = a.q_heads ? (a.q_heads + q_per - 1) / q_per : 0, kv_runs = (a.kv_heads + kv_per - 1) / kv_per;
    const dim3 grid((unsigned)groups, (unsigned)(q_runs + kv_runs));
    // Long runs of heads load four heads ahead (16384 rows of 32 + 2 x 8 heads of 128: 8 to 4 % faster), short
    // ones one, which are done sooner (4096 fp16 rows of 40 heads: 23.6 us, 25.0 with four).
#define LB_ROTARY(d)                                                                                          \
    case d:                                                                                                   \
        if (per >= 8)                                                                                         \
            hipLaunchKernelGGL((rotary_kernel<DT, d, 4>), grid, dim3(256), 0, s, a, shift, (int)q_runs, (int)q_per, (int)kv_per);  \
        else                                                                                                  \
            hipLaunchKernelGGL((rotary_kernel<DT, d, 1>), grid, dim3(256), 0, s, a, shift, (int)q_runs, (int)q_per, (int)kv_per);  \
        return hipGetLastError();
    switch (a.head_dim) {
        LB_ROTARY(64) LB_ROTARY(128) LB_ROTARY(256)
    }
#undef LB_ROTARY
    return hipErrorInvalidValue;
}

hipError_t launch_kv_append_rotary(int dtype, const RotaryArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? rotary_d<LB_F32>(a, s) : dtype == LB_BF16 ? rotary_d<LB_BF16>(a, s) : rotary_d<LB_F16>(a, s);
}

} // namespace lb
