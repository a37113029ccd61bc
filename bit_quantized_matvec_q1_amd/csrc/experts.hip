// The experts' products: every routed pair (token, expert) multiplies one row of activations by one expert's matrix.
//
// A decode step's pairs are few a matrix, so the weights are the work: bytes that each expert with a row is read for once.
// The plan sorts the pairs by expert, in tiles of rows that share a read; with many rows an expert (prompts) the tiles are
// those of the prefill product (gemm.hip), with few they are at most four rows and this file's kernel, whose arithmetic is
// the batch-1 product's (matvec_tile.h): nibble dot products in exact integers, scales in fp32.
#include "matvec_tile.h"
#include "serve_internal.h"

namespace lb {

namespace {

constexpr int ROWS = 4; // rows a tile of experts_rows_kernel

// ---- the plan -----------------------------------------------------------------------------------
// A workgroup an expert; each counts all pairs of all experts for itself (a histogram in LDS, whose atomics give the same
// sums in any order), so that one launch without a workspace finds where its expert's pairs begin, and then writes them in
// their order: a wave goes through a run of pairs of its own, whose count it knows from the first pass.
constexpr int PLAN_WG = 1024, PLAN_WAVES = PLAN_WG / 64, MAX_E = 1024;

__global__ __launch_bounds__(PLAN_WG) void plan_kernel(const int32_t *__restrict__ experts, int pairs, int E, int32_t *__restrict__ plan,
                                                       int tile_rows, int64_t tiles_at)
{
    __shared__ int hist[MAX_E];
    __shared__ int mine[PLAN_WAVES], before[PLAN_WAVES], tiles[PLAN_WAVES];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < E; i += PLAN_WG)
        hist[i] = 0;
    __syncthreads();
    const int64_t run = ((int64_t)pairs + PLAN_WG - 1) / PLAN_WG * 64; // pairs a wave, whole steps of 64
    const int64_t p0 = wave * run, p1 = min(p0 + run, (int64_t)pairs);
    int own = 0;
    for (int64_t p = p0 + lane; p - lane < p1; p += 64) { // uniform in the wave
        const int x = p < p1 ? experts[p] : -1;
        if ((unsigned)x < (unsigned)E)
            atomicAdd(&hist[x], 1);
        own += __popcll(__ballot(x == e));
    }
    if (lane == 0)
        mine[wave] = own;
    __syncthreads();
    // pairs and tiles of the experts before this one: E <= PLAN_WG, a thread an expert
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
    int first = 0, tile = 0, at = 0;
    for (int w = 0; w < PLAN_WAVES; w++) {
        first += before[w], tile += tiles[w];
        at += w < wave ? mine[w] : 0;
    }
    const int rows = hist[e], own_tiles = (rows + tile_rows - 1) / tile_rows;
    if (e == E - 1 && threadIdx.x == 0)
        plan[0] = tile + own_tiles, plan[1] = first + rows, plan[2] = plan[3] = 0;
    int4 *table = reinterpret_cast<int4 *>(plan + tiles_at);
    for (int i = threadIdx.x; i < own_tiles; i += PLAN_WG)
        table[tile + i] = make_int4(e, first + i * tile_rows, min(tile_rows, rows - i * tile_rows), 0);
    int32_t *order = plan + 4 + first;
    for (int64_t p = p0 + lane; p - lane < p1; p += 64) {
        const bool is = p < p1 && experts[p] == e;
        const uint64_t m = __ballot(is);
        if (is)
            order[at + __popcll(m & (((uint64_t)1 << lane) - 1))] = (int32_t)p;
        at += __popcll(m);
    }
}

// ---- few rows an expert -------------------------------------------------------------------------
struct RowsConfig {
    int L, S;
};
// lanes a weight row, records a lane; the staged activations of RR rows have to fit 96 registers, so that two waves or more
// are resident on each SIMD, or those of one row 160, as in matvec_tile.h
#define LB_ECFGS(X)                                                                                           \
    X(0, 4, 1) X(1, 4, 2) X(2, 4, 3) X(3, 8, 1) X(4, 8, 2) X(5, 8, 3) X(6, 16, 1) X(7, 16, 2) X(8, 16, 3)     \
    X(9, 32, 1) X(10, 32, 2) X(11, 32, 3) X(12, 64, 1) X(13, 64, 2) X(14, 64, 3) X(15, 64, 4) X(16, 64, 8)
#define LB_ECFG_ENTRY(i, l, s) {l, s},
constexpr RowsConfig kRows[] = {LB_ECFGS(LB_ECFG_ENTRY)};
#undef LB_ECFG_ENTRY
constexpr int kRowsN = sizeof(kRows) / sizeof(kRows[0]);
constexpr bool rows_allowed(int fmt, int S, int RR) { return S * rec_of(fmt) * RR <= (RR > 1 ? 96 : 160); }

// One chunk of weight rows [row0, row0 + nrows) of one expert times RR rows of activations (nr of them real: the others
// repeat the last and are not stored): the pairs order[0 .. nr), or pair `tile` where order is null.  Loads and their clamps are those of matvec_tile.
template <int FMT, int L, int S, int RR>
__device__ __forceinline__ void rows_body(const ExpertsArgs &a, const uint8_t *__restrict__ W, const int32_t *__restrict__ order, int tile, int nr,
                                          int row0, int nrows, uint32_t *__restrict__ lds)
{
    constexpr int REC = F<FMT>::REC, NAB = F<FMT>::NAB, DX = F<FMT>::SW / 4;
    constexpr int GROUPS = 64 / L, STEP = GROUPS * (WG / 64);
    const int ns = a.K / F<FMT>::SW, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane % L, rbase = wave * GROUPS + lane / L;
    const uint8_t *scales = W + (int64_t)a.N * ns * CODE_BYTES;
    const uint32_t rowbytes = (uint32_t)ns * CODE_BYTES, stepb = STEP * rowbytes, last = (uint32_t)(row0 + nrows - 1) * rowbytes;
    uint32_t slo[S];
#pragma unroll
    for (int i = 0; i < S; i++)
        slo[i] = (uint32_t)min(li + i * L, ns - 1) * CODE_BYTES;
    uint32_t onext = (uint32_t)(row0 + min(rbase, nrows - 1)) * rowbytes;
    RowRegs<FMT, S> buf[2];
    auto issue = [&](RowRegs<FMT, S> &r) {
        const uint32_t off = min(onext, last);
#pragma unroll
        for (int i = 0; i < S; i++) {
            const v4u t = *(gv4u *)((gu8 *)W + (off + slo[i]));
            r.code[i] = make_uint4(t.x, t.y, t.z, t.w);
            r.sc[i] = *(gu16 *)((gu8 *)scales + ((off + slo[i]) >> 3));
        }
        onext += stepb;
    };
    int64_t pair[RR];
#pragma unroll
    for (int r = 0; r < RR; r++) {
        pair[r] = order ? min((uint32_t)order[min(r, nr - 1)], (uint32_t)(a.pairs - 1)) : (uint32_t)tile;
        const int64_t row = pair[r] / a.per_row;
        if (r < nr) { // uniform
            const int8_t *xq = a.xq + row * a.K;
            const uint16_t *xs = a.xs + row * (a.K / QK8);
            if (r == 0)
                stage_activation<FMT, 1>(xq, xs, ns, lds, [&] { issue(buf[0]); });
            else
                stage_activation<FMT, 1>(xq, xs, ns, lds + r * ns * REC, [] {});
        }
    }
    __syncthreads();
    uint32_t act[RR][S][REC];
    float cfold[RR][S]; // Q1_0: as in matvec_tile
#pragma unroll
    for (int r = 0; r < RR; r++)
#pragma unroll
        for (int i = 0; i < S; i++) {
            const int sl = li + i * L;
            const uint4 *p = reinterpret_cast<const uint4 *>(lds + (min(r, nr - 1) * ns + min(sl, ns - 1)) * REC);
#pragma unroll
            for (int q = 0; q < REC / 4; q++) {
                const uint4 t = p[q];
                act[r][i][4 * q] = t.x, act[r][i][4 * q + 1] = t.y, act[r][i][4 * q + 2] = t.z, act[r][i][4 * q + 3] = t.w;
            }
            float c = 0.0f;
            if (FMT == LB_Q1_0) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    c = fmaf((j == 0 ? 0.5f : j == 1 ? 1.0f : j == 2 ? 2.0f : 4.0f) * __uint_as_float(act[r][i][32 + j]), (float)(int)act[r][i][36 + j], c);
            }
            cfold[r][i] = c;
        }
    for (int it = 0; it < nrows; it += 2 * STEP) {
#pragma unroll
        for (int b = 0; b < 2; b++) {
            issue(buf[1 - b]);
            __builtin_amdgcn_sched_barrier(0); // the next row's loads go out before this row's arithmetic
            float part[RR];
#pragma unroll
            for (int r = 0; r < RR; r++)
                part[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < S; i++) {
                const float d = half_bits_to_float((uint16_t)buf[b].sc[i]);
                const bool in = li + i * L < ns;
#pragma unroll
                for (int r = 0; r < RR; r++) {
                    const uint32_t *A = act[r][i];
                    float t;
                    if (FMT == LB_Q2_0_G64) {
                        int i0, i1;
                        q2_isums(buf[b].code[i], A, i0, i1);
                        t = fmaf(__uint_as_float(A[DX + 1]), (float)i1, __uint_as_float(A[DX]) * (float)i0);
                    } else if (FMT == LB_Q4_0) {
                        t = __uint_as_float(A[DX]) * (float)q4_isum(buf[b].code[i], A);
                    } else {
                        int C[4];
                        q1_group_sums(buf[b].code[i], A, C);
                        t = cfold[r][i];
#pragma unroll
                        for (int j = 0; j < NAB; j++)
                            t = fmaf(__uint_as_float(A[DX + j]), (float)C[j], t);
                    }
                    const float c = fmaf(d, t, part[r]);
                    part[r] = in ? c : part[r];
                }
            }
            const int rl = it + b * STEP + rbase;
#pragma unroll
            for (int r = 0; r < RR; r++) {
                const float v = group_sum_f<L>(part[r]);
                if (li == L - 1 && rl < nrows && r < nr)
                    a.y[pair[r] * a.N + row0 + rl] = v;
            }
        }
    }
}

// RR: the most rows taken at once (as many as the row's length allows); a tile with more takes several passes, each
// reading the chunk's weights again, from the cache.
template <int FMT, int L, int S, int RR> __global__ __launch_bounds__(WG) void experts_rows_kernel(ExpertsArgs a, int chunks, int chunk_rows)
{
    extern __shared__ uint32_t lds[];
    const int chunk = blockIdx.x % chunks, tile = blockIdx.x / chunks;
    int e, rows;
    const int32_t *order = nullptr;
    if (a.plan) {
        if (tile >= a.plan[0])
            return;
        const int4 t = reinterpret_cast<const int4 *>(a.plan + experts_tiles_at(a.pairs))[tile];
        e = t.x;
        if (t.y < 0 || t.z < 1 || t.z > ROWS || t.y > a.pairs - t.z)
            return; // no plan of these pairs
        rows = t.z;
        order = a.plan + experts_order_at() + t.y;
    } else {
        e = a.experts[tile];
        rows = 1;
    }
    const int row0 = chunk * chunk_rows, nrows = min(chunk_rows, a.N - row0);
    if ((unsigned)e >= (unsigned)a.E || nrows <= 0)
        return;
    const uint8_t *W = a.W + e * a.expert_bytes;
    for (int r = 0; r < rows; r += RR) {
        if (r)
            __syncthreads(); // every wave has its rows of the pass before
        const int nr = min(RR, rows - r);
        if (RR > 2 && nr > 2)
            rows_body<FMT, L, S, RR>(a, W, order ? order + r : nullptr, tile, nr, row0, nrows, lds);
        else if (RR > 1 && nr == 2)
            rows_body<FMT, L, S, 2>(a, W, order ? order + r : nullptr, tile, nr, row0, nrows, lds);
        else
            rows_body<FMT, L, S, 1>(a, W, order ? order + r : nullptr, tile, nr, row0, nrows, lds);
    }
}

struct RowsChoice {
    int cfg, rr;
};
// As many rows at once as a configuration has registers for, then the fewest idle lane slots, then the fewest lanes.  The
// length of a row alone decides, so that a pair's result does not depend on the others, or on the plan.
RowsChoice rows_choice(int fmt, int64_t ns)
{
    for (int rr = ROWS; rr >= 1; rr /= 2) {
        int best = -1;
        for (int c = 0; c < kRowsN; c++) {
            const int64_t slots = (int64_t)kRows[c].L * kRows[c].S;
            if (slots >= ns && rows_allowed(fmt, kRows[c].S, rr) &&
                (best < 0 || slots < (int64_t)kRows[best].L * kRows[best].S ||
                 (slots == (int64_t)kRows[best].L * kRows[best].S && kRows[c].L < kRows[best].L)))
                best = c;
        }
        if (best >= 0)
            return {best, rr};
    }
    return {-1, 0};
}

struct RowsLaunch {
    RowsChoice c;
    int chunks, chunk_rows;
    int64_t blocks;
};
RowsLaunch rows_launch(int fmt, const ExpertsArgs &a)
{
    const int64_t ns = a.K / sw_of(fmt);
    RowsLaunch r = {rows_choice(fmt, ns), 0, 0, 0};
    if (r.c.cfg < 0)
        return r;
    // chunks of whole iterations: enough workgroups to fill the device several times over
    const int step = 64 / kRows[r.c.cfg].L * (WG / 64);
    const int64_t steps = ((int64_t)a.N + step - 1) / step;
    int64_t per = steps * a.max_tiles / 2048;
    per = per < 1 ? 1 : per > 64 ? 64 : per;
    r.chunk_rows = (int)per * step;
    r.chunks = (int)((a.N + r.chunk_rows - 1) / r.chunk_rows);
    r.blocks = a.max_tiles * r.chunks;
    return r;
}

template <int FMT, int RR> hipError_t rows_rr(const ExpertsArgs &a, const RowsLaunch &r, hipStream_t s)
{
    const size_t lds = (size_t)(a.K / sw_of(FMT)) * rec_of(FMT) * 4 * RR;
    switch (r.c.cfg) {
#define LB_ECASE(i, l, s_)                                                                                    \
    case i:                                                                                                   \
        if constexpr (rows_allowed(FMT, s_, RR))                                                              \
            hipLaunchKernelGGL((experts_rows_kernel<FMT, l, s_, RR>), dim3((unsigned)r.blocks), dim3(WG), lds, s, a, r.chunks,  \
                               r.chunk_rows);                                                                 \
        break;
        LB_ECFGS(LB_ECASE)
#undef LB_ECASE
    default:
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}
template <int FMT> hipError_t rows_fmt(const ExpertsArgs &a, hipStream_t s)
{
    const RowsLaunch r = rows_launch(FMT, a);
    if (!a.plan) // a pair a tile
        return r.c.cfg < 0 ? hipErrorInvalidValue : rows_rr<FMT, 1>(a, r, s);
    return r.c.rr == 4 ? rows_rr<FMT, 4>(a, r, s) : r.c.rr == 2 ? rows_rr<FMT, 2>(a, r, s) : r.c.rr == 1 ? rows_rr<FMT, 1>(a, r, s) : hipErrorInvalidValue;
}

// ---- the sum over a token's experts -------------------------------------------------------------
// out[t] = sum_j weights[t][j] * y[t top_k + j], in fp32 in the order of j, rounded once.  Bound by HBM: top_k rows of
// fp32 in.  A thread has V columns.
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

// Tiles of the prefill product from 16 rows an expert on average
int64_t experts_tile_rows(int64_t pairs, int64_t E) { return pairs >= 16 * E ? 128 : ROWS; }
int64_t experts_max_tiles(int64_t pairs, int64_t E) { return pairs / experts_tile_rows(pairs, E) + (pairs < E ? pairs : E); }

hipError_t launch_experts_plan(const int32_t *experts, int64_t pairs, int64_t E, int32_t *plan, hipStream_t s)
{
    hipLaunchKernelGGL(plan_kernel, dim3((unsigned)E), dim3(PLAN_WG), 0, s, experts, (int)pairs, (int)E, plan,
                       (int)experts_tile_rows(pairs, E), experts_tiles_at(pairs));
    return hipGetLastError();
}

int64_t experts_rows_blocks(int fmt, const ExpertsArgs &a) { return rows_launch(fmt, a).blocks; }

hipError_t launch_experts_rows(int fmt, const ExpertsArgs &a, hipStream_t s)
{
    return fmt == LB_Q1_0 ? rows_fmt<LB_Q1_0>(a, s) : fmt == LB_Q2_0_G64 ? rows_fmt<LB_Q2_0_G64>(a, s) : rows_fmt<LB_Q4_0>(a, s);
}

hipError_t launch_experts_combine(int dtype, const CombineArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? combine_d<LB_F32>(a, s) : dtype == LB_BF16 ? combine_d<LB_BF16>(a, s) : combine_d<LB_F16>(a, s);
}

} // namespace lb
