// Routing of tokens to experts.  A token's logits become scores p (a softmax over all experts, or a sigmoid each); the
// experts are ordered by p + bias, first their groups where there are several; the chosen ones' weights are p.
//
// Which experts are chosen is a question of order, and scores of neighbouring ranks can lie closer than fp32's rounding of
// an exponential: computed in 32 bits, a token goes to another expert than the formula's now and then.  So scores, their
// sums and comparisons are in 64 bits (the hardware's fp64 rate is its fp32 rate without packing), and equal values go to
// the lowest index.
//
// A token has LT lanes, 32 or a whole wave, lane l the experts l, l + LT, ... .  A choice is one maximum over the lanes
// (DPP within rows of 16, row swaps across them: an instruction and two moves a step), and a minimum of the indexes of
// those that have it.  What it takes is instructions, and nearly as many for 32 lanes as for 64: so long batches put two
// tokens in a wave, and short ones, where a single token's time counts, one.
//
// Measured: 8191 bf16 tokens of 256 experts in 8 groups, 8 chosen: 13 to 15 us (4.2 MB in).  That is one round of four waves a
// SIMD with 1572 vector instructions each, which keep the vector unit busy for 75 % of the kernel; the rest is its start, the
// logits' way in, and where the four waves wait in their chains of reductions at once.  One fp32 token of 64 experts 3 us, a
// launch.  With the library's exponential and a token a wave the first took 18 us.
#include "serve_internal.h"

namespace lb {

namespace {

constexpr int WAVES = 4; // a workgroup

template <int CTRL> __device__ __forceinline__ double dpp(double v)
{
    const uint64_t b = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
struct Both {
    double a, b;
};
// v of the even and of the odd row of 16 of each two (ROW), or of the lower and upper 32 lanes, in both of them
template <bool ROW> __device__ __forceinline__ Both halves(double v)
{
    const uint64_t x = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
    const auto p = ROW ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false) : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto q = ROW ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false) : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    return {__longlong_as_double((uint64_t)(uint32_t)q[0] << 32 | (uint32_t)p[0]), __longlong_as_double((uint64_t)(uint32_t)q[1] << 32 | (uint32_t)p[1])};
}
// The maximum, as one instruction (fmax makes its operands canonical first, an instruction each; there is no NaN here).
__device__ __forceinline__ double dmax(double a, double b)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// e^a for a <= 0: a = n ln 2 + r, |r| <= ln 2 / 2, with ln 2 as a sum of two, and the Taylor series of e^r, whose next term
// is below 2^-57; 0 below the smallest number.
__device__ __forceinline__ double exp_down(double a)
{
    a = dmax(a, -800.0);
    const double n = rint(a * 0x1.71547652b82fep0);                             // 1 / ln 2
    const double r = fma(-n, 0x1.abc9e3b39803fp-56, fma(-n, 0x1.62e42fefa39efp-1, a)); // ln 2
    double e = 1.0 / 6227020800.0; // 13!
    e = fma(e, r, 1.0 / 479001600.0);
    e = fma(e, r, 1.0 / 39916800.0);
    e = fma(e, r, 1.0 / 3628800.0);
    e = fma(e, r, 1.0 / 362880.0);
    e = fma(e, r, 1.0 / 40320.0);
    e = fma(e, r, 1.0 / 5040.0);
    e = fma(e, r, 1.0 / 720.0);
    e = fma(e, r, 1.0 / 120.0);
    e = fma(e, r, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return ldexp(e, (int)n);
}
// 1 / (1 + e^-x): with e = e^-|x| <= 1, 1 / (1 + e) or e / (1 + e), the reciprocal by Newton's steps
__device__ __forceinline__ double sigmoid(double x)
{
    const double e = exp_down(-fabs(x)), d = 1.0 + e;
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return x >= 0.0 ? r : e * r;
}

// f over a token's LT lanes, in all of them
template <int LT, typename Op> __device__ __forceinline__ double over_lanes(double v, Op &&f)
{
    v = f(v, dpp<0xB1>(v));  // quad_perm [1,0,3,2]
    v = f(v, dpp<0x4E>(v));  // quad_perm [2,3,0,1]
    v = f(v, dpp<0x141>(v)); // row_half_mirror
    v = f(v, dpp<0x140>(v)); // row_mirror
    Both o = halves<true>(v);
    v = f(o.a, o.b);
    if (LT == 64) {
        o = halves<false>(v);
        v = f(o.a, o.b);
    }
    return v;
}
template <int LT> __device__ __forceinline__ double lanes_max(double v) // no NaN among them
{
    return over_lanes<LT>(v, [](double a, double b) { return dmax(a, b); });
}
template <int LT> __device__ __forceinline__ double lanes_sum(double v)
{
    return over_lanes<LT>(v, [](double a, double b) { return a + b; });
}
template <int LT> __device__ __forceinline__ uint32_t lanes_min(uint32_t v)
{
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = min((uint32_t)p[0], (uint32_t)p[1]);
    if (LT == 64) {
        p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = min((uint32_t)p[0], (uint32_t)p[1]);
    }
    return v;
}

// An allowed expert's value is at least LEAST, one that is taken or not allowed -inf.
constexpr double LEAST = -1.7976931348623157e308;
__device__ __forceinline__ double value_of(double v) { return v >= LEAST ? v : LEAST; } // a NaN and -inf count least

template <int DT, int LT, int NE> __global__ __launch_bounds__(64 * WAVES) void route_kernel(RouteArgs a)
{
    using R = RowType<DT>;
    extern __shared__ double shared[]; // [tokens][E] scores, then the values they are ordered by, where there are groups
    constexpr int TOKENS = 64 / LT * WAVES;
    const int lane = threadIdx.x % LT, local = threadIdx.x / LT, E = (int)a.E, k = (int)a.top_k;
    const int64_t t = (int64_t)blockIdx.x * TOKENS + local;
    const bool grouped = a.groups > 1; // uniform
    const bool live = t < a.T && (!a.count || t < (int64_t)a.count[0]);
    const double NONE = -__builtin_inf();
    double p[NE], sel[NE];

    float x[NE];
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = i * LT + lane;
        x[i] = -__builtin_inff();
        if (live && e < E) {
            const float v = R::get(static_cast<const typename R::T *>(a.logits)[t * a.stride + e]);
            x[i] = v == v ? v : -__builtin_inff(); // a NaN counts as the least logit
        }
    }
    if (a.sigmoid) { // uniform
#pragma unroll
        for (int i = 0; i < NE; i++)
            p[i] = sigmoid((double)x[i]);
    } else {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            m = fmaxf(m, x[i]);
        const double top = lanes_max<LT>((double)m);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < NE; i++) { // (the largest is 1 also where it is infinite)
            p[i] = i * LT + lane < E ? ((double)x[i] == top ? 1.0 : exp_down((double)x[i] - top)) : 0.0;
            z += p[i];
        }
        z = 1.0 / lanes_sum<LT>(z);
#pragma unroll
        for (int i = 0; i < NE; i++)
            p[i] *= z;
    }
    double *scores = shared + local * E;
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = i * LT + lane;
        sel[i] = e < E ? value_of(a.bias ? p[i] + (double)a.bias[e] : p[i]) : NONE;
        if (e < E)
            scores[e] = p[i];
    }

    if (grouped) {
        double *mine = shared + (TOKENS + local) * E;
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (i * LT + lane < E)
                mine[i * LT + lane] = sel[i];
        __syncthreads();
        // `each` lanes a group (a power of two), which look through its experts in turn
        const int groups = (int)a.groups, size = E / groups;
        int each = 1;
        while (2 * each * groups <= LT)
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
        gs = __shfl(gs, min(lane * each, LT - 1), LT); // group l in lane l
        gs = lane < groups ? gs : NONE;
        uint64_t kept = 0;
        for (int r = 0; r < (int)a.kept; r++) {
            const double m = lanes_max<LT>(gs);
            const int best = (int)lanes_min<LT>(lane < groups && gs == m ? (uint32_t)lane : 63u);
            kept |= (uint64_t)1 << best;
            gs = lane == best ? NONE : gs;
        }
        // e / size: (e + 1/2) / size is 2^-11 or more from a whole number, and the quotient below 64 off by less than 2^-16
        const float part = 1.0f / (float)size;
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = i * LT + lane, in = (int)(((float)e + 0.5f) * part);
            if (e < E && !(kept >> in & 1))
                sel[i] = NONE;
        }
    }

    uint32_t mine[2] = {0, 0}; // choices `lane` and LT + `lane`
    for (int j = 0; j < k; j++) {
        double m = sel[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            m = dmax(m, sel[i]);
        m = lanes_max<LT>(m);
        uint32_t at = ~0u;
#pragma unroll
        for (int i = NE - 1; i >= 0; i--)
            at = sel[i] == m ? (uint32_t)(i * LT + lane) : at;
        at = lanes_min<LT>(at);
#pragma unroll
        for (int i = 0; i < NE; i++)
            sel[i] = at == (uint32_t)(i * LT + lane) ? NONE : sel[i];
        mine[0] = j == lane ? at : mine[0];
        if (LT == 32)
            mine[1] = j == LT + lane ? at : mine[1];
    }
    __syncthreads(); // the scores are in place
    double w[2] = {0.0, 0.0};
#pragma unroll
    for (int h = 0; h < 64 / LT; h++)
        if (h * LT + lane < k)
            w[h] = scores[min(mine[h], (uint32_t)(E - 1))];
    if (a.renormalise) {
        const double z = lanes_sum<LT>(w[0] + w[1]);
        w[0] = z > 0.0 ? w[0] / z : 0.0, w[1] = z > 0.0 ? w[1] / z : 0.0;
    }
#pragma unroll
    for (int h = 0; h < 64 / LT; h++) {
        const int j = h * LT + lane;
        if (t < a.T && j < k) {
            a.experts[t * k + j] = live ? (int32_t)mine[h] : -1;
            a.weights[t * k + j] = live ? (float)(w[h] * (double)a.factor) : 0.0f;
        }
    }
}

template <int DT, int LT, int NE> hipError_t route_n(const RouteArgs &a, hipStream_t s)
{
    constexpr int TOKENS = 64 / LT * WAVES;
    const size_t lds = (size_t)a.E * TOKENS * sizeof(double) * (a.groups > 1 ? 2 : 1);
    hipLaunchKernelGGL((route_kernel<DT, LT, NE>), dim3((unsigned)((a.T + TOKENS - 1) / TOKENS)), dim3(64 * WAVES), lds, s, a);
    return hipGetLastError();
}

// two tokens a wave from 1024 tokens on, where their experts are at most eight a lane
bool two_a_wave(int64_t T, int64_t E, int64_t groups) { return T >= 1024 && E <= 256 && groups <= 32; }

template <int DT> hipError_t route_d(const RouteArgs &a, hipStream_t s)
{
    if (two_a_wave(a.T, a.E, a.groups))
        return a.E <= 32 ? route_n<DT, 32, 1>(a, s) : a.E <= 64 ? route_n<DT, 32, 2>(a, s) : a.E <= 128 ? route_n<DT, 32, 4>(a, s) : route_n<DT, 32, 8>(a, s);
    return a.E <= 64    ? route_n<DT, 64, 1>(a, s)
           : a.E <= 128 ? route_n<DT, 64, 2>(a, s)
           : a.E <= 256 ? route_n<DT, 64, 4>(a, s)
           : a.E <= 512 ? route_n<DT, 64, 8>(a, s)
                        : route_n<DT, 64, 16>(a, s);
}

} // namespace

int64_t route_blocks(int64_t T, int64_t E, int64_t groups)
{
    const int64_t tokens = two_a_wave(T, E, groups) ? 2 * WAVES : WAVES;
    return (T + tokens - 1) / tokens;
}

hipError_t launch_route(int dtype, const RouteArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? route_d<LB_F32>(a, s) : dtype == LB_BF16 ? route_d<LB_BF16>(a, s) : route_d<LB_F16>(a, s);
}

} // namespace lb
