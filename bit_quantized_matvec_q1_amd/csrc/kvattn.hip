// Attention of a step's new tokens over the paged 4-bit cache: for query row i of a request that holds len
// tokens, n of them new, at position pos = len - n + i,
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - max),   pos - window < j <= pos,
// and zeros where no j is left.
//
// One pass over the cache, 32 tokens at a time, on the matrix cores.  A tile has 16 query rows: G = q_heads /
// kv_heads heads of a token share a kv head, so row r of a request is token r / G, head r % G of the group.
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16 per 32-block b of the head: A = 16 keys' codes, B = 16 query rows.
//                 The codes are exact in binary16, the queries are scaled per row by a power of two; the
//                 block's sum is multiplied by the key's block scale in fp32, so nothing of K is rounded.
//   O += P V      A = p_j times v_j's block scale, B = V's codes.  S^T leaves the matrix core with the query row
//                 along the lanes and four consecutive tokens in each lane's registers, which is how the second
//                 product takes its left operand: the weights never leave the registers.  The cache holds V in
//                 quads of four tokens for the right operand.
// Softmax: p is taken against a reference a row, 2^7 below the largest seen when it was set, that only moves when
// some score passes it by 15 (in powers of two), so the usual step has no reduction across lanes and no
// rescaling.  A score counts with its value's scale (s + log2 max_b dv_b): p times the scale then stays below
// binary16's 2^16 whatever the values' range, and the largest are far above its lower end (2^-24), so that what
// is rounded away there is 2^-31 of them: of the block's largest where a block has columns, and with them a reference,
// of its own (packed), of the row's where one reference serves all blocks (wide; there a block of values 2^-12 of
// another's keeps 2^-19 of itself in fp32 rows.  A reference a block would take a product more for every weight).
// fp32 queries and outputs: the queries and p times the scale are split into two binary16 numbers each (22
// bits), and every product is done twice.
//
// Decode is bound by HBM, so the tokens of one (request, kv head) are cut into chunks, one workgroup each, and the
// chunks' results joined by a second launch.  Measured at head size 128, four heads a kv head, one new token a
// request (attention + join): 32 requests of up to 4000 tokens over 5 kv heads, 54 MB of cache, 18.2 + 4.0 us; one of
// 131071 over 8, 151 MB, 29.2 + 6.3 us (5.2 TB/s); 64 of up to 12345 over 8, 537 MB, 102 + 5.1 us (5.3 TB/s, a plain
// read of as much reaches 6.7).  A copy of the kernel that does nothing but its loads, in the same chunks, takes 18.0,
// 27.5 and 95.4 us: the arithmetic is hidden behind them (the vector unit, unpacking and softmax, is at 51 % of its
// cycles, the matrix cores at 12 %).  For the one long request that is the rate at which a plain read of as much goes
// (5.6 TB/s).  For the others the chunks' places count too: of 1120 workgroups launched some 650 have tokens, of 4096
// some 2500, so that the last round is mostly empty.
#include <type_traits>

#include "kvattn_internal.h"

namespace lb {

// Two ways of placing query rows on the 16 columns of S^T:
//   wide    16 rows; a lane scales four tokens' sums of every block, and needs all of their scales.
//   packed  16 / nb rows, each once a block: column b * rows + r has row r's block b and zeros elsewhere, so one
//           chain of products leaves every block's sums in its own column.  A lane multiplies them by its one
//           block's scales, the nb columns of a row are added across the lanes, and the weights are multiplied by
//           one block's value scales too; of O the rows (b, r) count in block b's columns.  Per step and lane 8
//           scores' scalings instead of 8 nb, and 8 of the weights' instead of 8 nb, with a quarter of the scale
//           registers.  For one token of up to 16 / nb heads a kv head (4 at head size 128) the rows fill the
//           columns, which are empty otherwise.
template <int D, bool PACK> struct Shape {
    static constexpr int ROWS = PACK ? 16 / (D / 32) : ATT_ROWS;
    static constexpr int SW = PACK ? 2 : D / 16; // words of scales a lane holds of four tokens
    static __device__ __forceinline__ int word(int b, int i) { return (PACK ? 0 : 2 * b) + i / 2; }
    // the column with row r's reference and sum for element d
    static __device__ __forceinline__ int column(int r, int d) { return PACK ? d / 32 * ROWS + r : r; }
};

// One step's share of the cache in a lane: 16 tokens (sub 0) and 16 more (sub 1).
template <int D, bool PACK> struct Step {
    Words<D / 32> k[2]; // quarter g of every block of key c
    Words<D / 32> v[2]; // column c of the quad g's four tokens
    Words<Shape<D, PACK>::SW> ks[2], vs[2]; // [block][token of the quad g], binary16; packed: the lane's block
};

// A lane's column of queries, elements 32 b + 8 g + j, as binary16 times 2^-e; returns e.
template <int DT, int D, bool PACK, bool SPLIT>
__device__ __forceinline__ int load_query(const typename RowType<DT>::T *q, int c, int g, bool negate, f16x8 (&hi)[D / 32], f16x8 (&lo)[SPLIT ? D / 32 : 1])
{
    constexpr int NB = D / 32;
    if constexpr (PACK) {
        constexpr int ROWS = Shape<D, true>::ROWS;
        float x[8];
        float am = groups_max(load_eight<DT>(q + 32 * (c / ROWS) + 8 * g, x));
#pragma unroll
        for (int d = ROWS; d < 16; d *= 2)
            am = fmaxf(am, __shfl_xor(am, d));
        const int e = row_exponent(am);
        f16x8 h, l;
        query_halves<SPLIT>(x, e, negate, h, l);
#pragma unroll
        for (int b = 0; b < NB; b++) {
            hi[b] = b == c / ROWS ? h : f16x8{};
            if constexpr (SPLIT)
                lo[b] = b == c / ROWS ? l : f16x8{};
        }
        return e;
    } else {
        float x[NB][8], am = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; b++)
            am = fmaxf(am, load_eight<DT>(q + 32 * b + 8 * g, x[b]));
        const int e = row_exponent(groups_max(am));
#pragma unroll
        for (int b = 0; b < NB; b++)
            query_halves<SPLIT>(x[b], e, negate, hi[b], lo[SPLIT ? b : 0]);
        return e;
    }
}

// sum over the lanes of a 16-lane row that are a multiple of N apart
template <int N> __device__ __forceinline__ float sum_columns(float v)
{
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false)); // row_ror:8
    if (N <= 4)
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false)); // row_ror:4
    if (N <= 2)
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xF, 0xF, false)); // row_ror:2
    return v;
}

template <int D, bool PACK> using Partial = PartialOf<D, Shape<D, PACK>::ROWS, 16>; // of a tile and chunk, in the workspace

// Workgroups a CU (waves a SIMD) that the registers have to leave room for.
constexpr int attn_waves(bool split, int D, bool pack)
{
    if (pack)
        return D == 256 ? 2 : D == 128 ? 4 : 5;
    return D == 256 ? 1 : D == 128 ? (split ? 2 : 3) : 4;
}

template <int DT, int D, bool PACK>
__global__ __launch_bounds__(64 * ATT_WAVES, attn_waves(DT == LB_F32, D, PACK)) void attn_kernel(AttnArgs a, Geo geo)
{
    using R = RowType<DT>;
    using S = Shape<D, PACK>;
    constexpr bool SPLIT = DT == LB_F32;
    constexpr int NB = D / 32, NC = D / 16, ROWS = S::ROWS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // All tiles' first chunks, then their second ones: workgroups go round the eight XCDs in order, and with a tile's
    // chunks side by side, eight of them, the first chunks, which every request has, would all land on one (64
    // requests of very different lengths: 137 us, and 101 us so).
    const uint32_t split_u = blockIdx.x / geo.tiles, sh = blockIdx.x - split_u * geo.tiles, slot = sh / (uint32_t)a.kv_heads;
    const int split = (int)split_u, head = (int)(sh - slot * (uint32_t)a.kv_heads);
    const Tile t = tile_of(a, geo, slot, ROWS);
    if (t.row0 >= t.rows)
        return;
    const int start = t.lo + split * geo.chunk;
    if (split > 0 && start >= t.hi)
        return;
    const int end = start + min(t.hi - start, geo.chunk); // start + chunk can pass 2^31
    const int P = 1 << geo.shift;

    // this lane's query row; the rows past the last repeat it, and are not stored
    const int row = min(t.row0 + c % ROWS, t.rows - 1);
    const int tok = row / geo.G, hq = head * geo.G + row % geo.G;
    const int pos = t.pos0 + tok;                                              // last token it sees
    const int from = a.window > 0 ? (int)max((int64_t)0, pos - a.window + 1) : 0; // and the first
    f16x8 qh[NB], ql[SPLIT ? NB : 1];
    const typename R::T *qp = static_cast<const typename R::T *>(a.q) + (int64_t)(a.cu_q[t.b] + tok) * a.q_stride + (int64_t)hq * D;
    const float qscale = score_scale(a.scale, load_query<DT, D, PACK, SPLIT>(qp, c, g, a.scale < 0.0f, qh, ql));

    f32x4 acc[NC];
#pragma unroll
    for (int n = 0; n < NC; n++)
        acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float ref = -INFINITY, sum = 0.0f;

    const int32_t *table = a.block_table + (int64_t)t.b * a.table_stride;
    const int64_t rec = kv_record_bytes(P, D);
    // positions that every row of the tile sees: no comparisons there
    const int all_to = t.pos0 + t.row0 / geo.G, all_from = a.window > 0 ? (int)max((int64_t)0, t.pos0 + (int64_t)(min(t.rows - 1, t.row0 + ROWS - 1) / geo.G) - a.window + 1) : 0;
    const int own = PACK ? c / ROWS : 0; // the first block whose scales this lane holds

    // the pages of a step's two halves; past the end the first's again (its tokens are masked)
    auto pages_of = [&](int t0, int (&page)[2]) {
        const int t1 = t0 < end ? t0 : end - 1;
        page[0] = __builtin_amdgcn_readfirstlane(table[t1 >> geo.shift]);
        page[1] = __builtin_amdgcn_readfirstlane(table[(t1 + 16 < end ? t1 + 16 : t1) >> geo.shift]);
    };
    auto record = [&](int page) {
        return a.cache + ((int64_t)((uint32_t)page < (uint32_t)a.pages ? page : 0) * a.kv_heads + head) * rec;
    };
    // a half past the end lies in the page that pages_of gave for it, whatever it holds there
    Step<D, PACK> s;
    auto load_keys = [&](int t0, const int (&page)[2]) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const uint8_t *r = record(page[u]);
            const int o = (t0 + 16 * u) & (P - 1);
            s.k[u] = load_words<NB, PACK>(r + kv_k_byte(D, o + c, g, 0));
            s.ks[u] = load_words<S::SW, PACK>(r + kv_scale_byte(P, D, 0, o + 4 * g, own));
        }
    };
    auto load_values = [&](int t0, const int (&page)[2]) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const uint8_t *r = record(page[u]);
            const int o = (t0 + 16 * u) & (P - 1);
            s.v[u] = load_words<NB, PACK>(r + kv_v_byte(P, D, o + 4 * g, c));
            s.vs[u] = load_words<S::SW, PACK>(r + kv_scale_byte(P, D, 1, o + 4 * g, own));
        }
    };

    // The next step's keys are loaded once this step's are used up, its values likewise, each into the same
    // registers, and its pages were looked up a step earlier.  Loads past the end give some page of the request's,
    // and are not used.
    constexpr int NEXT = ATT_WAVES * ATT_STEP;
    int page[3][2];
    const int t_first = start + wave * ATT_STEP;
    if (t_first < end) {
        pages_of(t_first, page[0]);
        pages_of(t_first + NEXT, page[1]);
        load_keys(t_first, page[0]);
        load_values(t_first, page[0]);
    }
    for (int t0 = t_first; t0 < end; t0 += NEXT) {
        pages_of(t0 + 2 * NEXT, page[2]);
        const int (&pg)[2] = page[0];
        float sc[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            f32x4 x[PACK ? 1 : NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const f16x8 k = codes8(s.k[u].w[b]);
                f32x4 &to = x[PACK ? 0 : b];
                to = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qh[b], PACK && b ? to : f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
                if constexpr (SPLIT)
                    to = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[b], to, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float v = 0.0f;
#pragma unroll
                for (int b = 0; b < (PACK ? 1 : NB); b++)
                    v = fmaf(half_of(s.ks[u].w[S::word(b, i)], i & 1), x[b][i], v);
                if constexpr (PACK)
                    v = sum_columns<ROWS>(v);
                asm volatile("" : "+v"(v)); // computed here, not where it is used
                sc[u][i] = v;
            }
        }
        // the loads must not move above the last use of the registers they fill: the copies that this costs would
        // wait for them at the step's end
        __builtin_amdgcn_sched_barrier(0);
        load_keys(t0 + NEXT, page[1]);
        Words<S::SW> vs[2] = {s.vs[0], s.vs[1]};
        float most = -INFINITY;
        uint32_t wide = 0; // the lane's largest value scales, two to a word
        const bool inside = (uint32_t)pg[0] < (uint32_t)a.pages && (uint32_t)pg[1] < (uint32_t)a.pages;
        if (!(inside && t0 + ATT_STEP <= end && t0 + ATT_STEP - 1 <= all_to && t0 >= all_from)) {
            // At an edge: what a row does not see gets the score -inf, and no value scale, as that may be NaN.  What
            // it sees of a page that is none is NaN.
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const bool none = (uint32_t)pg[u] >= (uint32_t)a.pages;
                    uint32_t keep = 0;
#pragma unroll
                    for (int i = 2 * h; i < 2 * h + 2; i++) {
                        const int j = t0 + 16 * u + 4 * g + i;
                        const bool see = j <= pos && j >= from && j < end;
                        sc[u][i] = see ? (none ? NAN : sc[u][i]) : -INFINITY;
                        keep |= see ? 0xffffu << (16 * (i & 1)) : 0u;
                    }
#pragma unroll
                    for (int w = h; w < S::SW; w += 2)
                        vs[u].w[w] &= keep;
                }
        }
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                most = fmaxf(most, sc[u][i]);
#pragma unroll
            for (int i = 0; i < S::SW; i++)
                wide = max_u16x2(wide, vs[u].w[i]); // a sign, which no scale has, would only raise it
        }
        // no token of the lane passes the reference if its largest score with its largest value scale does not
        const float bound = fmaf(most, qscale, log2_above(max(wide >> 16, wide & 0xffffu)));
        if (__ballot(bound > ref + REF_MOST)) {
            float m = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                Words<S::SW> d = vs[u];
#pragma unroll
                for (int k = 0; k < S::SW; k++)
                    asm volatile("" : "+v"(d.w[k])); // nothing made of them here is kept for what follows: registers
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    uint32_t w = 0;
#pragma unroll
                    for (int k = i / 2; k < S::SW; k += 2) {
                        const uint32_t x = (i & 1 ? d.w[k] >> 16 : d.w[k]) & 0x7fffu;
                        w = max(w, x < 0x7c00u ? x : 0u); // a block that is not finite has no say over the others
                    }
                    m = fmaxf(m, fmaf(sc[u][i], qscale, log2_above_all(w)));
                }
            }
            const bool past = m > ref + REF_MOST;
            if (__ballot(past)) {
                const float now = fmaxf(ref, groups_max(m) - REF_BELOW);
                const float f = now > -INFINITY ? exp2_raw(ref - now) : 1.0f; // a row with nothing yet has sums of 0
                ref = now;
                sum *= f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float fr = __shfl(f, 4 * g + i); // the accumulators' rows
#pragma unroll
                    for (int n = 0; n < NC; n++)
                        acc[n][i] *= fr;
                }
            }
        }
        const float against = ref > -INFINITY ? ref : 0.0f;
        float p[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                p[u][i] = exp2_raw(fmaf(sc[u][i], qscale, -against));
                sum += p[u][i];
            }
        const Pairs<D> vp[2] = {pair_tokens<D>(s.v[0]), pair_tokens<D>(s.v[1])};
        constexpr int PB = PACK ? 1 : NB;
        f16x8 ph[PB], pl[SPLIT ? PB : 1]; // [first half's tokens, second's]
#pragma unroll
        for (int b = 0; b < PB; b++)
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float w = fmaf(half_of(vs[u].w[S::word(b, i)], i & 1), p[u][i], 0.0f);
                    const _Float16 h = (_Float16)w;
                    ph[b][4 * u + i] = h;
                    if constexpr (SPLIT)
                        pl[b][4 * u + i] = (_Float16)(w - (float)h);
                }
        __builtin_amdgcn_sched_barrier(0);
        load_values(t0 + NEXT, page[1]);
#pragma unroll
        for (int b = 0; b < NB; b++) {
#pragma unroll
            for (int half = 0; half < 2; half++) {
                u32x4 w;
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int pair = 0; pair < 2; pair++)
                        w[2 * u + pair] = __builtin_bit_cast(uint32_t, codes2(vp[u].w[pair][half][b / 4], b));
                const f16x8 v = __builtin_bit_cast(f16x8, w);
                acc[2 * b + half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph[PACK ? 0 : b], v, acc[2 * b + half], 0, 0, 0);
                if constexpr (SPLIT)
                    acc[2 * b + half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl[PACK ? 0 : b], v, acc[2 * b + half], 0, 0, 0);
            }
        }
        page[0][0] = page[1][0], page[0][1] = page[1][1];
        page[1][0] = page[2][0], page[1][1] = page[2][1];
    }

    // the four waves' results together
    __shared__ float s_acc[ATT_WAVES][ROWS][D];
    __shared__ float s_ref[ATT_WAVES][16], s_sum[ATT_WAVES][16];
    sum = groups_sum(sum);
    if (g == 0)
        s_ref[wave][c] = ref, s_sum[wave][c] = sum;
#pragma unroll
    for (int n = 0; n < NC; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int col = 4 * g + i; // the accumulators' rows are the columns of S^T
            if (!PACK || col / ROWS == n / 2)
                s_acc[wave][col % ROWS][16 * n + c] = acc[n][i];
        }
    __syncthreads();
    const bool only = t.hi - t.lo <= geo.chunk; // nothing to join with
    Partial<D, PACK> *part = static_cast<Partial<D, PACK> *>(a.workspace) + ((int64_t)sh * geo.nsplit + split);
    const int real = min(ROWS, t.rows - t.row0); // rows
    for (int e = threadIdx.x; e < real * D; e += 64 * ATT_WAVES) {
        const int r = e / D, d = e % D, col = S::column(r, d);
        float m = s_ref[0][col];
#pragma unroll
        for (int w = 1; w < ATT_WAVES; w++)
            m = fmaxf(m, s_ref[w][col]);
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++) {
            const float f = s_ref[w][col] > -INFINITY ? exp2_raw(s_ref[w][col] - m) : s_sum[w][col]; // 0, or NaN where a score was
            o = fmaf(f, s_acc[w][r][d], o);
            l = fmaf(f, s_sum[w][col], l);
        }
        if (only) {
            const int rr = t.row0 + r;
            typename R::T *op = static_cast<typename R::T *>(a.out) + (int64_t)(a.cu_q[t.b] + rr / geo.G) * a.out_stride + (int64_t)(head * geo.G + rr % geo.G) * D;
            op[d] = R::put(t.over ? NAN : l == 0.0f ? 0.0f : o / l);
        } else {
            part->acc[r][d] = o;
            if (!PACK ? d == 0 : d % 32 == 0)
                part->ref[col] = m, part->sum[col] = l;
        }
    }
}

// Joins the chunks of rows: the 256 threads are D/4 groups of four columns times 1024/D shares.  With many chunks a
// workgroup takes one row, each share its own of the chunks, whose loads do not wait for each other, and the shares
// are added in LDS; with at most as many chunks as shares, each share takes a row of its own.
// TILE: rows of a prompt's tile; 0 for the tiles of attn_kernel.
template <int DT, int D, bool PACK, int TILE> __global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Geo geo)
{
    using R = RowType<DT>;
    using S = Shape<D, PACK>;
    using Part = std::conditional_t<TILE != 0, PartialOf<D, TILE, TILE>, Partial<D, PACK>>;
    constexpr int COLS = D / 4, SHARES = 256 / COLS;
    __shared__ float s_ref[SHARES][COLS], s_l[SHARES][COLS];
    __shared__ f32x4 s_o[SHARES][COLS];
    const bool apart = geo.nsplit > SHARES; // a row's chunks over the shares
    const int groups = apart ? geo.rows : (geo.rows + SHARES - 1) / SHARES;
    const uint32_t sh = blockIdx.x / (uint32_t)groups, slot = sh / (uint32_t)a.kv_heads;
    const int group = threadIdx.x % COLS, share = threadIdx.x / COLS;
    const int r0 = (int)(blockIdx.x - sh * groups), r = apart ? r0 : r0 * SHARES + share;
    const int head = (int)(sh - slot * (uint32_t)a.kv_heads);
    const Tile t = tile_of(a, geo, slot, geo.tile);
    const int rr = t.row0 + r;
    if (rr >= t.rows || r >= geo.rows || t.over || t.hi - t.lo <= geo.chunk) // all of the workgroup, if its shares are added
        return;
    const int n = min((t.hi - t.lo + geo.chunk - 1) / geo.chunk, geo.nsplit);
    const Part *part = static_cast<const Part *>(a.workspace) + (int64_t)sh * geo.nsplit;
    const int first = apart ? share : 0, step = apart ? SHARES : 1, col = S::column(r, 4 * group);
    // the reference first: the sums then need no rescaling
    float m = -INFINITY;
#pragma unroll 4
    for (int i = first; i < n; i += step)
        m = fmaxf(m, part[i].ref[col]);
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
#pragma unroll 4
    for (int i = first; i < n; i += step) {
        const float ref = part[i].ref[col], sum = part[i].sum[col];
        const f32x4 x = *reinterpret_cast<const f32x4 *>(&part[i].acc[r][4 * group]);
        const float f = ref > -INFINITY ? exp2_raw(ref - m) : sum; // 0, or NaN where a score was
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = fmaf(f, x[k], o[k]);
        l = fmaf(f, sum, l);
    }
    if (apart) {
        s_o[share][group] = o;
        s_ref[share][group] = m;
        s_l[share][group] = l;
        __syncthreads();
        if (share > 0)
            return;
        for (int i = 0; i < SHARES; i++)
            m = fmaxf(m, s_ref[i][group]);
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
        for (int i = 0; i < SHARES; i++) {
            const f32x4 x = s_o[i][group];
            const float f = s_ref[i][group] > -INFINITY ? exp2_raw(s_ref[i][group] - m) : s_l[i][group];
#pragma unroll
            for (int k = 0; k < 4; k++)
                o[k] = fmaf(f, x[k], o[k]);
            l = fmaf(f, s_l[i][group], l);
        }
    }
    RowVec<DT, 4> v;
#pragma unroll
    for (int k = 0; k < 4; k++)
        v.v[k] = R::put(l == 0.0f ? 0.0f : o[k] / l);
    typename R::T *op = static_cast<typename R::T *>(a.out) + (int64_t)(a.cu_q[t.b] + rr / geo.G) * a.out_stride + (int64_t)(head * geo.G + rr % geo.G) * D;
    *reinterpret_cast<RowVec<DT, 4> *>(op + 4 * group) = v;
}

static Geo geometry(int dtype, const AttnArgs &a)
{
    Geo g;
    g.G = (int)(a.q_heads / a.kv_heads);
    g.shift = 0;
    while (((int64_t)1 << g.shift) < a.page_tokens)
        g.shift++;
    const int64_t most = (a.max_q > 0 ? a.max_q : 1) * g.G; // rows of a request
    const int packed = (int)(16 / (a.head_dim / 32));
    // fp32 rows need the wide kernel's exact keys and split operands
    g.kind = most <= packed ? Geo::PACKED : most <= PROMPT_FROM || dtype == LB_F32 ? Geo::WIDE : Geo::PROMPT;
    g.tile = g.kind == Geo::PACKED ? packed : g.kind == Geo::WIDE ? ATT_ROWS : PROMPT_ROWS;
    // Larger tiles where every CU gets two of them: of 32 heads over 8 at head size 128, prompts of 2048 / 4096 / 8192
    // tokens (256, 512 and 1024 such tiles) 91 / 215 / 719 us with 128 rows, 94 / 188 / 663 us with 256; 64 requests of
    // 64 after 936 156 and 119; 16 of 256 57 and 58; 8000 with a window of 1000 231 and 233.  They are counted from
    // what the requests may bring, not from the rows of a padded step, so that there really are as many: tiles of 256
    // rows are never split (below), and the parts and their join know 128.
    const int64_t real = a.T < a.B * a.max_q ? a.T : a.B * a.max_q;
    if (g.kind == Geo::PROMPT && a.head_dim <= 128 && real * g.G / (2 * PROMPT_ROWS) * a.kv_heads >= 512)
        g.tile = 2 * PROMPT_ROWS;
    g.by_request = most <= g.tile;
    g.rows = (int)(g.by_request ? most : g.tile);
    g.slots = g.by_request ? a.B : a.T * g.G / g.tile + a.B;
    int64_t span = a.max_kv; // tokens a tile may see
    if (a.window > 0)
        span = span < a.window + g.tile + ATT_STEP ? span : a.window + g.tile + ATT_STEP;
    const int64_t tiles = g.slots * a.kv_heads;
    g.tiles = (uint32_t)(tiles < UINT32_MAX ? tiles : UINT32_MAX); // more are refused
    // Single tokens and the 16-row tiles: chunks such that the workgroups fill the chip in whole rounds of what the
    // registers allow, each one's start (about 3 us; a chunk of 2048 tokens takes 40) being paid once a round; one
    // round, unless the chunks would pass 2048 tokens: lengths may differ.  Several rounds of tiles are not split at
    // all.  The chunks come from max_kv, the longest request: of requests of uneven lengths some workgroups are empty.
    // A prompt's tiles: 768 parts, a round and a half of four-wave workgroups (310 tiles whole 107 us, in 512 / 768 /
    // 1024 parts 126 / 105 / 113 with their join).
    const int64_t fill = g.kind == Geo::PROMPT ? 768 : 256 * attn_waves(dtype == LB_F32, (int)a.head_dim, g.kind == Geo::PACKED);
    constexpr int64_t UNIT = ATT_WAVES * ATT_STEP;
    // a prompt's part is 64 KB to write and read again: none where every CU has a tile
    if (tiles >= (g.kind == Geo::PROMPT ? 256 : 4 * fill)) {
        g.chunk = (int)(span > UNIT ? (span + UNIT - 1) / UNIT * UNIT : UNIT);
        g.nsplit = 1;
        return g;
    }
    const int64_t rounds = g.kind == Geo::PROMPT ? 1 : (span * tiles / fill + 2047) / 2048;
    int64_t chunk = (span * tiles / (fill * (rounds > 1 ? rounds : 1)) + UNIT - 1) / UNIT * UNIT;
    chunk = chunk < UNIT ? UNIT : chunk;
    g.chunk = (int)chunk;
    g.nsplit = (int)(span > 0 ? (span + chunk - 1) / chunk : 1);
    return g;
}

static int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

static int64_t part_bytes(const Geo &g, const AttnArgs &a)
{
    const int64_t part = g.tile * a.head_dim + 2 * (g.kind == Geo::PROMPT ? g.tile : 16);
    return g.nsplit == 1 ? 0 : g.slots * a.kv_heads * g.nsplit * part * 4;
}

// Workgroups of the join: a row each, or as many rows as a workgroup has shares.
static int64_t join_workgroups(const Geo &g, const AttnArgs &a)
{
    const int64_t shares = 1024 / a.head_dim;
    return g.nsplit == 1 ? 0 : g.slots * a.kv_heads * (g.nsplit > shares ? g.rows : (g.rows + shares - 1) / shares);
}

// Up to 512 threads a workgroup, numbered in 32 bits.
bool kv_attention_fits(int dtype, const AttnArgs &a)
{
    const Geo g = geometry(dtype, a);
    return larger(g.slots * a.kv_heads * g.nsplit, join_workgroups(g, a)) < (1 << 23);
}

// Enough for any row type whose launch fits; -1 where none does.
int64_t kv_attention_workspace(const AttnArgs &a)
{
    int64_t need = -1;
    for (int dtype : {LB_F32, LB_F16})
        if (kv_attention_fits(dtype, a))
            need = larger(need, part_bytes(geometry(dtype, a), a));
    return need;
}

template <int DT, int D> static hipError_t run(const AttnArgs &a, const Geo &g, hipStream_t s)
{
    static_assert(sizeof(Partial<D, true>) == (Shape<D, true>::ROWS * D + 32) * 4 && sizeof(Partial<D, false>) == (ATT_ROWS * D + 32) * 4 &&
                      sizeof(PartialOf<D, PROMPT_ROWS, PROMPT_ROWS>) == (PROMPT_ROWS * D + 2 * PROMPT_ROWS) * 4,
                  "the workspace's size");
    const int64_t tiles = g.slots * a.kv_heads;
    const dim3 grid((unsigned)(tiles * g.nsplit)), join((unsigned)join_workgroups(g, a));
    hipError_t e = hipSuccess;
    if (g.kind == Geo::PROMPT) {
        e = launch_attn_prompt(DT, a, g, s);
    } else {
        if (g.kind == Geo::PACKED)
            hipLaunchKernelGGL((attn_kernel<DT, D, true>), grid, dim3(64 * ATT_WAVES), 0, s, a, g);
        else
            hipLaunchKernelGGL((attn_kernel<DT, D, false>), grid, dim3(64 * ATT_WAVES), 0, s, a, g);
        e = hipGetLastError();
    }
    if (e != hipSuccess || g.nsplit == 1)
        return e;
    if (g.kind == Geo::PACKED)
        hipLaunchKernelGGL((attn_join_kernel<DT, D, true, 0>), join, dim3(256), 0, s, a, g);
    else if (g.kind == Geo::WIDE)
        hipLaunchKernelGGL((attn_join_kernel<DT, D, false, 0>), join, dim3(256), 0, s, a, g);
    else if constexpr (DT != LB_F32) // tiles of twice as many rows are never split
        hipLaunchKernelGGL((attn_join_kernel<DT, D, false, PROMPT_ROWS>), join, dim3(256), 0, s, a, g);
    return hipGetLastError();
}

template <int DT> static hipError_t run_d(const AttnArgs &a, hipStream_t s)
{
    const Geo g = geometry(DT, a);
    switch (a.head_dim) {
    case 64:
        return run<DT, 64>(a, g, s);
    case 128:
        return run<DT, 128>(a, g, s);
    case 256:
        return run<DT, 256>(a, g, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_kv_attention(int dtype, const AttnArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? run_d<LB_F32>(a, s) : dtype == LB_BF16 ? run_d<LB_BF16>(a, s) : run_d<LB_F16>(a, s);
}

} // namespace lb
