// A row's logits before sampling: penalties for the tokens of its history, biases, and a grammar's mask.
//   seen in prompt or output:  l = l > 0 ? l / r : l * r
//   n times in the output:     l = l - f * n, and l - p if n > 0
//   biases of the token:       l + (their sum, added up in list order)
//   masked:                    -inf
// in fp32, in this order, each step rounded once; the result is rounded once to the row type.
//
// Bound by HBM: every logit is read and written once.  A workgroup takes a stretch of a row's vocabulary, holds
// its logits in registers (loaded before anything else) and counts the history's tokens that fall into the
// stretch in LDS, by integer atomics, whose order does not matter.  Every stretch reads the whole history (from
// L2, after the first), so the stretches are as long as the number of rows lets them be.  96 fp32 rows of 151669, 6000
// tokens of history, 64 biases, a mask: 33 us (118 MB, 3.6 TB/s; a plain copy of the rows 24 us); the rest is the
// histories' reads and the counts' round through LDS, five barriers and three passes over 64 KB.  Other stretches
// and sizes of workgroups took 33 to 42 us, a bitmap of the touched logits 34.  One row of 128256: 4.4 us.
#include "serve_internal.h"

namespace lb {

constexpr uint32_t SEEN = 0x80000000u; // in the prompt; the lower bits count the output

// WG threads, V4 groups of four consecutive logits a thread: a stretch of WG * V4 * 4 logits.
template <int DT, int WG_, int V4> __global__ __launch_bounds__(WG_) void logits_kernel(LogitsArgs a, int stretches)
{
    using R = RowType<DT>;
    using T = typename R::T;
    constexpr int CH = WG_ * V4 * 4;
    __shared__ uint32_t tab[CH];
    const int tid = threadIdx.x;
    const int64_t b = blockIdx.x / stretches, v0 = (int64_t)(blockIdx.x % stretches) * CH;
    const int n = (int)(a.V - v0 < CH ? a.V - v0 : CH); // logits of this stretch
    const T *in = static_cast<const T *>(a.logits) + b * a.in_stride + v0;
    T *out = static_cast<T *>(a.out) + b * a.out_stride + v0;

    // rows start at any element, so the four are loaded as the hardware allows: unaligned
    struct Four {
        T v[4];
    };
    float x[V4][4];
#pragma unroll
    for (int g = 0; g < V4; g++) {
        const int i = (g * WG_ + tid) * 4;
        Four f = {};
        if (i + 3 < n)
            __builtin_memcpy(&f, in + i, sizeof(f));
        else
            for (int j = 0; j < 4; j++)
                if (i + j < n)
                    f.v[j] = in[i + j];
#pragma unroll
        for (int j = 0; j < 4; j++)
            x[g][j] = R::get(f.v[j]);
    }
    uint4 *tab4 = reinterpret_cast<uint4 *>(tab);

    int total = 0, prompt = 0;
    if (a.tokens) {
        total = min((int64_t)max(a.total_lens[b], 0), a.tok_stride);
        prompt = a.prompt_lens ? min(max(a.prompt_lens[b], 0), total) : 0;
    }
    if (total > 0) {
        for (int g = 0; g < V4; g++)
            tab4[g * WG_ + tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        const int32_t *tok = a.tokens + b * a.tok_stride;
        for (int i = tid; i < total; i += WG_) {
            const int64_t t = (int64_t)tok[i] - v0; // a token outside the vocabulary falls into no stretch
            if (t >= 0 && t < n) {
                if (i < prompt)
                    atomicOr(&tab[t], SEEN);
                else
                    atomicAdd(&tab[t], 1u);
            }
        }
        __syncthreads();
        const float rep = a.repetition ? a.repetition[b] : 1.0f;
        const float pres = a.presence ? a.presence[b] : 0.0f, freq = a.frequency ? a.frequency[b] : 0.0f;
#pragma unroll
        for (int g = 0; g < V4; g++) {
            const uint4 c4 = tab4[g * WG_ + tid];
            const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
            if ((c[0] | c[1] | c[2] | c[3]) == 0)
                continue;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (c[j] == 0)
                    continue;
                float l = x[g][j];
                if (a.repetition)
                    l = l > 0.0f ? l / rep : l * rep;
                const uint32_t k = c[j] & ~SEEN;
                if (k) {
                    if (a.frequency)
                        l = l - freq * (float)k;
                    if (a.presence)
                        l = l - pres;
                }
                x[g][j] = l;
            }
        }
    }

    const int nb = a.bias_tokens ? (int)min((int64_t)max(a.bias_lens[b], 0), a.bias_stride) : 0;
    if (nb > 0) {
        // The sum of a token's biases is made by the first of its entries, in list order.  The table holds the
        // first entry's index, and MORE if there are others; each thread remembers which of its entries (at
        // most 64: lists are at most 16384 long) are first ones, as the table then takes their sums.
        constexpr uint32_t MORE = 0x40000000u, NONE = 0x3fffffffu;
        const int32_t *tok = a.bias_tokens + b * a.bias_stride;
        const float *val = a.bias_values + b * a.bias_stride;
        __syncthreads();
        for (int g = 0; g < V4; g++)
            tab4[g * WG_ + tid] = make_uint4(NONE, NONE, NONE, NONE);
        __syncthreads();
        for (int i = tid; i < nb; i += WG_) {
            const int64_t t = (int64_t)tok[i] - v0;
            if (t >= 0 && t < n)
                atomicMin(&tab[t], (uint32_t)i);
        }
        __syncthreads();
        uint64_t first = 0;
        for (int i = tid, e = 0; i < nb; i += WG_, e++) {
            const int64_t t = (int64_t)tok[i] - v0;
            if (t >= 0 && t < n) {
                if ((tab[t] & ~MORE) == (uint32_t)i)
                    first |= (uint64_t)1 << e;
                else
                    atomicOr(&tab[t], MORE);
            }
        }
        __syncthreads();
        uint64_t more = 0;
        for (int i = tid, e = 0; i < nb; i += WG_, e++)
            if (first >> e & 1 && tab[tok[i] - v0] & MORE)
                more |= (uint64_t)1 << e;
        __syncthreads();
        // the sums take the entries' places; a bias of -0 stands for "none", which adds nothing either
        for (int g = 0; g < V4; g++)
            tab4[g * WG_ + tid] = make_uint4(0x80000000u, 0x80000000u, 0x80000000u, 0x80000000u);
        __syncthreads();
        for (int i = tid, e = 0; i < nb; i += WG_, e++) {
            if (!(first >> e & 1))
                continue;
            const int t = tok[i];
            float sum = val[i];
            if (more >> e & 1)
                for (int k = i + 1; k < nb; k++)
                    if (tok[k] == t)
                        sum = sum + val[k];
            tab[t - v0] = __float_as_uint(sum);
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < V4; g++) {
            const uint4 c = tab4[g * WG_ + tid];
            x[g][0] += __uint_as_float(c.x);
            x[g][1] += __uint_as_float(c.y);
            x[g][2] += __uint_as_float(c.z);
            x[g][3] += __uint_as_float(c.w);
        }
    }

    const uint32_t *mask = a.mask ? a.mask + b * a.mask_stride + v0 / 32 : nullptr;
#pragma unroll
    for (int g = 0; g < V4; g++) {
        const int i = (g * WG_ + tid) * 4;
        if (i >= n)
            continue;
        const uint32_t allow = mask ? mask[i >> 5] >> (i & 31) : 0xfu; // four logits lie within a word
        Four f;
#pragma unroll
        for (int j = 0; j < 4; j++)
            f.v[j] = R::put(allow >> j & 1u ? x[g][j] : -INFINITY);
        if (i + 3 < n)
            __builtin_memcpy(out + i, &f, sizeof(f));
        else
            for (int j = 0; j < 4; j++)
                if (i + j < n)
                    out[i + j] = f.v[j];
    }
}

template <int DT> static hipError_t launch(const LogitsArgs &a, hipStream_t s)
{
    auto go = [&](auto kernel, int wg, int ch) {
        const int64_t st = (a.V + ch - 1) / ch;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(st * a.B)), dim3(wg), 0, s, a, (int)st);
        return hipGetLastError();
    };
    // the longest stretch that still gives every CU two workgroups
    if (a.B * ((a.V + 16383) / 16384) >= 512)
        return go(logits_kernel<DT, 1024, 4>, 1024, 16384);
    if (a.B * ((a.V + 4095) / 4096) >= 512)
        return go(logits_kernel<DT, 256, 4>, 256, 4096);
    return go(logits_kernel<DT, 256, 1>, 256, 1024);
}

hipError_t launch_logits_process(int dtype, const LogitsArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? launch<LB_F32>(a, s) : dtype == LB_BF16 ? launch<LB_BF16>(a, s) : launch<LB_F16>(a, s);
}

} // namespace lb
