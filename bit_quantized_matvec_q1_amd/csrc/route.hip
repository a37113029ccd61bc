// Routing of tokens to experts.  A token's logits become scores p (a softmax over all experts, or a sigmoid each); the
// experts are ordered by p + bias, first their groups where there are several; the chosen ones' weights are p.
//
// Which experts are chosen is a question of order, and scores of neighbouring ranks can lie closer than fp32's rounding of
// an exponential: computed in 32 bits, a token goes to another expert than the formula's now and then.  So scores, their
// sums and comparisons are in 64 bits (the hardware's fp64 rate is its fp32 rate without packing), and equal values go to
// the lowest index.
//
// A wave takes one token, lane l the experts l, l + 64, ... .  A choice is one maximum over the wave by DPP (an instruction
// and two moves a step), found again by comparing: the first element number with a lane that has it, and of those the
// lowest lane, is the lowest index.
#include "serve_internal.h"

namespace lb {

namespace {

constexpr int WAVES = 4; // tokens a workgroup

template <int CTRL, int ROWS> __device__ __forceinline__ double dpp(double v, double fill)
{
    const uint64_t b = __double_as_longlong(v), f = __double_as_longlong(fill);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)f, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(f >> 32), (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double v, int l) // l uniform
{
    const uint64_t b = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
// over the wave, in every lane; no NaN among them
__device__ __forceinline__ double wave_max(double v)
{
    v = fmax(v, dpp<0xB1, 0xF>(v, v));  // quad_perm [1,0,3,2]
    v = fmax(v, dpp<0x4E, 0xF>(v, v));  // quad_perm [2,3,0,1]
    v = fmax(v, dpp<0x141, 0xF>(v, v)); // row_half_mirror
    v = fmax(v, dpp<0x140, 0xF>(v, v)); // row_mirror
    v = fmax(v, dpp<0x142, 0xA>(v, v)); // row_bcast:15 into rows 1, 3
    v = fmax(v, dpp<0x143, 0xC>(v, v)); // row_bcast:31 into rows 2, 3
    return lane_of(v, 63);
}
__device__ __forceinline__ double wave_sum(double v)
{
    v += dpp<0xB1, 0xF>(v, 0.0);
    v += dpp<0x4E, 0xF>(v, 0.0);
    v += dpp<0x141, 0xF>(v, 0.0);
    v += dpp<0x140, 0xF>(v, 0.0);
    v += dpp<0x142, 0xA>(v, 0.0);
    v += dpp<0x143, 0xC>(v, 0.0);
    return lane_of(v, 63);
}

// An allowed expert's value is at least LEAST, one that is taken or not allowed -inf.
constexpr double LEAST = -1.7976931348623157e308;
__device__ __forceinline__ double value_of(double v) { return v >= LEAST ? v : LEAST; } // a NaN and -inf count least

template <int DT, int NE> __global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteArgs a)
{
    using R = RowType<DT>;
    extern __shared__ double shared[]; // [WAVES][E], where there are groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = (int)a.E, k = (int)a.top_k;
    const int64_t t = (int64_t)blockIdx.x * WAVES + wave;
    const bool grouped = a.groups > 1; // uniform
    const bool live = t < a.T && (!a.count || t < (int64_t)a.count[0]);
    const double NONE = -__builtin_inf();
    double p[NE], sel[NE];

    float x[NE];
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = i * 64 + lane;
        x[i] = -__builtin_inff();
        if (live && e < E) {
            const float v = R::get(static_cast<const typename R::T *>(a.logits)[t * a.stride + e]);
            x[i] = v == v ? v : -__builtin_inff(); // a NaN counts as the least logit
        }
    }
    if (a.sigmoid) { // uniform
#pragma unroll
        for (int i = 0; i < NE; i++)
            p[i] = 1.0 / (1.0 + exp(-(double)x[i]));
    } else {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            m = fmaxf(m, x[i]);
        const double top = wave_max((double)m);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < NE; i++) { // (the largest is 1 also where it is infinite)
            p[i] = i * 64 + lane < E ? ((double)x[i] == top ? 1.0 : exp((double)x[i] - top)) : 0.0;
            z += p[i];
        }
        z = wave_sum(z);
#pragma unroll
        for (int i = 0; i < NE; i++)
            p[i] /= z;
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = i * 64 + lane;
        sel[i] = e < E ? value_of(a.bias ? p[i] + (double)a.bias[e] : p[i]) : NONE;
    }

    if (grouped) {
        double *mine = shared + wave * E;
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (i * 64 + lane < E)
                mine[i * 64 + lane] = sel[i];
        __syncthreads();
        // `each` lanes a group (a power of two), which look through its experts in turn
        const int groups = (int)a.groups, size = E / groups;
        int each = 1;
        while (2 * each * groups <= 64)
            each *= 2;
        const int g = lane / each;
        double m1 = LEAST, m2 = LEAST; // the best two
        if (g < groups)
            for (int e = lane % each; e < size; e += each) {
                const double v = mine[g * size + e];
                m2 = fmax(m2, fmin(m1, v));
                m1 = fmax(m1, v);
            }
        for (int d = 1; d < each; d *= 2) {
            const double o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
            m2 = fmax(fmin(m1, o1), fmax(m2, o2));
            m1 = fmax(m1, o1);
        }
        double gs = value_of(a.best == 2 && size > 1 ? m1 + m2 : m1);
        gs = __shfl(gs, min(lane * each, 63)); // group l in lane l
        gs = lane < groups ? gs : NONE;
        uint64_t kept = 0;
        for (int r = 0; r < (int)a.kept; r++) {
            const uint64_t at = __ballot(gs == wave_max(gs)) & (groups < 64 ? ((uint64_t)1 << groups) - 1 : ~(uint64_t)0);
            const int best = __ffsll((unsigned long long)at) - 1;
            kept |= (uint64_t)1 << best;
            gs = lane == best ? NONE : gs;
        }
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = i * 64 + lane;
            if (e < E && !(kept >> (e / size) & 1))
                sel[i] = NONE;
        }
    }

    double weight = 0.0; // choice j in lane j
    int chosen = -1;
    for (int j = 0; j < k; j++) {
        double m = sel[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            m = fmax(m, sel[i]);
        m = wave_max(m);
        bool found = false;
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const uint64_t at = found ? 0 : __ballot(sel[i] == m);
            if (at) { // uniform
                found = true;
                const int l = __ffsll((unsigned long long)at) - 1;
                const double w = lane_of(p[i], l);
                weight = lane == j ? w : weight;
                chosen = lane == j ? i * 64 + l : chosen;
                sel[i] = lane == l ? NONE : sel[i];
            }
        }
    }
    if (a.renormalise) {
        const double z = wave_sum(lane < k ? weight : 0.0);
        weight = z > 0.0 ? weight / z : 0.0;
    }
    if (t < a.T && lane < k) {
        a.experts[t * k + lane] = live ? chosen : -1;
        a.weights[t * k + lane] = live ? (float)(weight * (double)a.factor) : 0.0f;
    }
}

template <int DT> hipError_t route_d(const RouteArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + WAVES - 1) / WAVES)), block(64 * WAVES);
    const size_t lds = a.groups > 1 ? (size_t)a.E * WAVES * sizeof(double) : 0;
    const int n = (int)((a.E + 63) / 64);
    if (n <= 1)
        hipLaunchKernelGGL((route_kernel<DT, 1>), grid, block, lds, s, a);
    else if (n <= 2)
        hipLaunchKernelGGL((route_kernel<DT, 2>), grid, block, lds, s, a);
    else if (n <= 4)
        hipLaunchKernelGGL((route_kernel<DT, 4>), grid, block, lds, s, a);
    else if (n <= 8)
        hipLaunchKernelGGL((route_kernel<DT, 8>), grid, block, lds, s, a);
    else
        hipLaunchKernelGGL((route_kernel<DT, 16>), grid, block, lds, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_route(int dtype, const RouteArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? route_d<LB_F32>(a, s) : dtype == LB_BF16 ? route_d<LB_BF16>(a, s) : route_d<LB_F16>(a, s);
}

} // namespace lb
