// The experts' products: every routed pair (token, expert) multiplies one row of activations by one expert's matrix.
//
// The plan sorts the pairs by expert, in tiles of rows that share a read of the weights: of 16 rows (experts_tile.hip), or of
// 128 where an expert has many (the prefill product's tiles, gemm.hip).  A single token's few pairs need none: each is a
// batch-1 product by itself (matvec_tile.h).  The sum over a token's experts is a kernel of its own.
#include "matvec_tile.h"
#include "serve_internal.h"

namespace lb {

namespace {

// ---- the plan -----------------------------------------------------------------------------------
// A workgroup an expert.  Each goes through all pairs for itself, so that one launch without a workspace finds where its
// expert's pairs begin, and then writes them in their order: a wave goes through a run of pairs of its own, whose count it
// knows from the first pass.  Bound by latency: 360 pairs of 128 experts 3.8 us, 4000 of 32 4.6, 24576 of 64 10.8 (a wave's
// two passes over 1536 pairs, four loads of 64 ahead).
//
// Where an expert's tiles begin depends on the tiles of all experts before it.  For few pairs each workgroup counts every
// expert (a histogram in LDS, whose atomics give the same sums in any order), and the table has no gaps.  For many the
// atomics would take most of the time (24576 pairs of 64 experts: 20 us, 11 without them): there only the pairs of lower
// experts are counted, and tile i of expert e is at floor(pairs before / rows a tile) + e + i, with up to one empty tile
// behind each expert's.
constexpr int PLAN_WG = 1024, PLAN_WAVES = PLAN_WG / 64, MAX_E = 1024, FEW_PAIRS = 4096;

template <bool FEW>
__global__ __launch_bounds__(PLAN_WG) void plan_kernel(const int32_t *__restrict__ experts, int pairs, int E, int32_t *__restrict__ plan,
                                                       int tile_rows, int max_tiles)
{
    __shared__ int hist[FEW ? MAX_E : 1];
    __shared__ int mine[PLAN_WAVES], before[PLAN_WAVES], tiles[PLAN_WAVES];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (FEW) {
        for (int i = threadIdx.x; i < E; i += PLAN_WG)
            hist[i] = 0;
        __syncthreads();
    }
    const int64_t run = ((int64_t)pairs + PLAN_WG - 1) / PLAN_WG * 64; // pairs a wave, whole steps of 64
    const int64_t p0 = wave * run, p1 = min(p0 + run, (int64_t)pairs);
    constexpr int U = 4; // loads ahead
    auto load = [&](int64_t p, int (&x)[U]) {
#pragma unroll
        for (int u = 0; u < U; u++)
            x[u] = p + 64 * u + lane < p1 ? experts[p + 64 * u + lane] : -1;
    };
    int own = 0, lower = 0;
    for (int64_t p = p0; p < p1; p += 64 * U) { // uniform in the wave
        int x[U];
        load(p, x);
#pragma unroll
        for (int u = 0; u < U; u++) {
            own += __popcll(__ballot(x[u] == e));
            if (!FEW)
                lower += __popcll(__ballot((unsigned)x[u] < (unsigned)e));
            else if ((unsigned)x[u] < (unsigned)E)
                atomicAdd(&hist[x[u]], 1);
        }
    }
    if (lane == 0)
        mine[wave] = own;
    if (!FEW && lane == 0)
        before[wave] = lower, tiles[wave] = 0;
    __syncthreads();
    if (FEW) { // pairs and tiles of the experts before this one: E <= PLAN_WG, a thread an expert
        int n = 0, nt = 0;
        if ((int)threadIdx.x < e) {
            n = hist[threadIdx.x];
            nt = (n + tile_rows - 1) / tile_rows;
        }
        n = group_sum_i<64>(n);
        nt = group_sum_i<64>(nt);
        if (lane == 63)
            before[wave] = n, tiles[wave] = nt;
        __syncthreads();
    }
    int first = 0, tile = 0, at = 0, rows = 0; // `first`: pairs of the experts before
    for (int w = 0; w < PLAN_WAVES; w++) {
        first += before[w], tile += tiles[w], rows += mine[w];
        at += w < wave ? mine[w] : 0;
    }
    const int own_tiles = (rows + tile_rows - 1) / tile_rows;
    int entries = own_tiles;
    if (!FEW) {
        tile = first / tile_rows + e;
        entries = (first + rows) / tile_rows + e + 1 - tile;
    }
    if (e == E - 1) { // the rest of the table too
        if (threadIdx.x == 0)
            plan[0] = tile + entries, plan[1] = first + rows, plan[2] = plan[3] = 0;
        entries = max_tiles - tile;
    }
    int2 *table = reinterpret_cast<int2 *>(plan + experts_tile_at(tile));
    for (int i = threadIdx.x; i < entries; i += PLAN_WG)
        table[i] = make_int2(e, max(0, min(tile_rows, rows - i * tile_rows)));
    int32_t *places = plan + experts_pairs_at(max_tiles, tile, tile_rows);
    for (int i = rows + threadIdx.x; i < own_tiles * tile_rows; i += PLAN_WG)
        places[i] = -1;
    for (int64_t p = p0; p < p1; p += 64 * U) {
        int x[U];
        load(p, x);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint64_t m = __ballot(x[u] == e);
            if (x[u] == e)
                places[at + __popcll(m & (((uint64_t)1 << lane) - 1))] = (int32_t)(p + 64 * u + lane);
            at += __popcll(m);
        }
    }
}

// ---- pairs by themselves ------------------------------------------------------------------------
// A tile of weight rows of one pair's expert, as a work list's batch-1 product: the results are lowbit_matvec's.  Eight pairs
// of Q2_0_g64 experts of 1536 x 2048 (7.1 MB): 5.0 us, of which some 3 are a launch's.
template <int FMT, int L, int S> __global__ __launch_bounds__(WG) void experts_pair_kernel(ExpertsArgs a, int tiles, int tile_rows)
{
    extern __shared__ uint32_t lds[];
    const int pair = blockIdx.x / tiles, row0 = (int)(blockIdx.x % tiles) * tile_rows;
    const int e = a.experts[pair];
    if ((unsigned)e >= (unsigned)a.E)
        return;
    const int64_t row = pair / a.per_row;
    matvec_tile<FMT, L, S, false, false>(a.W + e * a.expert_bytes, a.N, a.K, 1.0f, a.xq + row * a.K, a.xs + row * (a.K / QK8),
                                         a.y + (int64_t)pair * a.N, nullptr, row0, min(tile_rows, a.N - row0), lds);
}

struct PairLaunch {
    int cfg, tiles, tile_rows;
};
PairLaunch pair_launch(int fmt, const ExpertsArgs &a)
{
    PairLaunch r = {pick_cfg(fmt, a.K / sw_of(fmt)), 0, 0};
    if (r.cfg < 0)
        return r;
    // whole iterations of rows, as few as leave some 2048 workgroups, at most 32 (as launch_matvec)
    const int64_t step = 64 / kCfgs[r.cfg].L * (WG / 64), steps = (a.N + step - 1) / step;
    int64_t per = (steps * a.pairs + 2047) / 2048;
    per = per > 32 ? 32 : per;
    r.tile_rows = (int)(per * step);
    r.tiles = (int)((a.N + r.tile_rows - 1) / r.tile_rows);
    return r;
}

template <int FMT> hipError_t pairs_fmt(const ExpertsArgs &a, hipStream_t s)
{
    const PairLaunch r = pair_launch(FMT, a);
    const size_t lds = (size_t)(a.K / sw_of(FMT)) * rec_of(FMT) * 4;
    switch (r.cfg) {
#define LB_PCASE(i, l, s_)                                                                                    \
    case i:                                                                                                   \
        if constexpr (cfg_allowed(FMT, s_))                                                                   \
            hipLaunchKernelGGL((experts_pair_kernel<FMT, l, s_>), dim3((unsigned)((int64_t)a.pairs * r.tiles)), dim3(WG), lds, s, a,   \
                               r.tiles, r.tile_rows);                                                         \
        break;
        LB_CFGS(LB_PCASE)
#undef LB_PCASE
    default:
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// ---- the sum over a token's experts -------------------------------------------------------------
// out[t] = sum_j weights[t][j] * y[t top_k + j], in fp32 in the order of j, rounded once.  Bound by the reads, top_k rows of
// fp32 (1000 tokens of 4 x 2560: 8.3 us for 46 MB, 5.6 TB/s, what the product left in the caches included).  A thread has V
// columns.
template <int DT, int V> __global__ __launch_bounds__(WG) void combine_kernel(CombineArgs a, int chunks)
{
    using R = RowType<DT>;
    const int64_t t = blockIdx.x / (uint32_t)chunks;
    const int64_t n = ((int64_t)(blockIdx.x % (uint32_t)chunks) * WG + threadIdx.x) * V;
    if (n >= a.N)
        return;
    float acc[V] = {};
    for (int64_t j = 0; j < a.top_k; j++) {
        const int64_t p = t * a.top_k + j;
        if ((uint32_t)a.experts[p] >= (uint32_t)a.E)
            continue; // not routed: its row was not written
        const float w = a.weights[p];
        const RowVec<LB_F32, V> v = *reinterpret_cast<const RowVec<LB_F32, V> *>(a.y + p * a.N + n);
#pragma unroll
        for (int i = 0; i < V; i++)
            acc[i] = fmaf(w, v.v[i], acc[i]);
    }
    RowVec<DT, V> o;
#pragma unroll
    for (int i = 0; i < V; i++)
        o.v[i] = R::put(acc[i]);
    *reinterpret_cast<RowVec<DT, V> *>(static_cast<typename R::T *>(a.out) + t * a.out_stride + n) = o;
}

template <int DT> hipError_t combine_d(const CombineArgs &a, hipStream_t s)
{
    // four columns a thread where rows of the output and of y allow 16- (8-) byte accesses
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.out), size = (uintptr_t)dtype_bytes(DT);
    const bool wide = a.N % 4 == 0 && a.out_stride % 4 == 0 && at % (4 * size) == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    const int64_t per = WG * (wide ? 4 : 1), chunks = (a.N + per - 1) / per;
    if (wide)
        hipLaunchKernelGGL((combine_kernel<DT, 4>), dim3((unsigned)(a.T * chunks)), dim3(WG), 0, s, a, (int)chunks);
    else
        hipLaunchKernelGGL((combine_kernel<DT, 1>), dim3((unsigned)(a.T * chunks)), dim3(WG), 0, s, a, (int)chunks);
    return hipGetLastError();
}

} // namespace

// Rows a tile: 16, and 128 from 64 pairs an expert on.  Measured with 64 experts of 1536 x 2048 and 128 of 2048 x 768 (us with
// tiles of 16 and of 128): 48 pairs an expert Q1_0 56 and 66, 63 and 73, Q2_0 60 and 67, 76 and 79, Q4_0 75 and 76, 93 and 84;
// 64 pairs 69 and 72, 82 and 82, 75 and 72, 97 and 91, 92 and 83, 116 and 94; 80 pairs 85 and 81 to 139 and 103.
int64_t experts_tile_rows(int64_t pairs, int64_t E) { return pairs >= 64 * E ? 128 : 16; }
int64_t experts_max_tiles(int64_t pairs, int64_t E) { return pairs / experts_tile_rows(pairs, E) + (pairs < E ? pairs : E); }

hipError_t launch_experts_plan(const int32_t *experts, int64_t pairs, int64_t E, int32_t *plan, hipStream_t s)
{
    const int rows = (int)experts_tile_rows(pairs, E);
    if (pairs <= FEW_PAIRS)
        hipLaunchKernelGGL(plan_kernel<true>, dim3((unsigned)E), dim3(PLAN_WG), 0, s, experts, (int)pairs, (int)E, plan, rows,
                           (int)experts_max_tiles(pairs, E));
    else
        hipLaunchKernelGGL(plan_kernel<false>, dim3((unsigned)E), dim3(PLAN_WG), 0, s, experts, (int)pairs, (int)E, plan, rows,
                           (int)experts_max_tiles(pairs, E));
    return hipGetLastError();
}

int64_t experts_pair_blocks(int fmt, const ExpertsArgs &a) { return (int64_t)a.pairs * pair_launch(fmt, a).tiles; }

hipError_t launch_experts_pairs(int fmt, const ExpertsArgs &a, hipStream_t s)
{
    return fmt == LB_Q1_0 ? pairs_fmt<LB_Q1_0>(a, s) : fmt == LB_Q2_0_G64 ? pairs_fmt<LB_Q2_0_G64>(a, s) : pairs_fmt<LB_Q4_0>(a, s);
}

hipError_t launch_experts_combine(int dtype, const CombineArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? combine_d<LB_F32>(a, s) : dtype == LB_BF16 ? combine_d<LB_BF16>(a, s) : combine_d<LB_F16>(a, s);
}

} // namespace lb
