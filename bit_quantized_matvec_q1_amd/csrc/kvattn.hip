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
// is rounded away there is 2^-31 of them.
// fp32 queries and outputs: the queries and p times the scale are split into two binary16 numbers each (22
// bits), and every product is done twice.
//
// Decode is bound by HBM and by the vector unit (unpacking, softmax), so the tokens of one (request, kv head)
// are cut into chunks, one workgroup each, and the chunks' results joined by a second launch.
#include "serve_internal.h"

namespace lb {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int ATT_ROWS = 16;  // query rows a tile
constexpr int ATT_STEP = 32;  // tokens a step
constexpr int ATT_WAVES = 4;
constexpr float REF_BELOW = 7.0f, REF_MOST = 15.0f; // of a row's reference, log2

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// Four bytes of codes -> eight binary16 numbers, exact.
__device__ __forceinline__ f16x8 codes8(uint32_t w)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Byte b's two codes.
__device__ __forceinline__ f16x2 codes2(uint32_t w, int b)
{
    switch (b & 3) {
    case 0:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default:
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    }
}

template <int N> struct Words {
    uint32_t w[N];
};
template <int N> __device__ __forceinline__ Words<N> load_words(const uint8_t *p)
{
    Words<N> r;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 t = *reinterpret_cast<const u32x4 *>(p + 4 * i);
            r.w[i] = t.x, r.w[i + 1] = t.y, r.w[i + 2] = t.z, r.w[i + 3] = t.w;
        }
    } else {
        const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
        r.w[0] = t.x, r.w[1] = t.y;
    }
    return r;
}
__device__ __forceinline__ float half_of(uint32_t w, int hi) { return half_bits_to_float((uint16_t)(hi ? w >> 16 : w)); }

// Column c of four consecutive tokens (nb bytes each, byte b holding elements 32 b + c and 32 b + 16 + c) as
// pairs of tokens: byte b of word [pair][half][b / 4] has element 32 b + 16 half + c of tokens 2 pair, 2 pair + 1.
template <int D> struct Pairs {
    static constexpr int W = D > 128 ? 2 : 1;
    uint32_t w[2][2][W];
};
template <int D> __device__ __forceinline__ Pairs<D> pair_tokens(const Words<D / 32> &v)
{
    Pairs<D> r;
    constexpr uint32_t LO = 0x0f0f0f0fu, HI = 0xf0f0f0f0u;
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
        for (int i = 0; i < Pairs<D>::W; i++) {
            uint32_t x, y; // the two tokens' bytes
            if constexpr (D == 64)
                x = v.w[p], y = v.w[p] >> 16; // both in one word
            else
                x = v.w[2 * p * Pairs<D>::W + i], y = v.w[(2 * p + 1) * Pairs<D>::W + i];
            r.w[p][0][i] = (x & LO) | ((y << 4) & HI);
            r.w[p][1][i] = ((x >> 4) & LO) | (y & HI);
        }
    return r;
}

// One step's share of the cache in a lane: 16 tokens (sub 0) and 16 more (sub 1).
template <int D> struct Step {
    Words<D / 32> k[2];     // quarter g of every block of key c
    Words<D / 32> v[2];     // column c of the quad g's four tokens
    Words<D / 16> ks[2];    // [block][token of the quad g], binary16
    Words<D / 16> vs[2];
};

struct Geo { // of a launch
    int G, nsplit, chunk, shift;
    bool by_request; // a request has at most one tile: the tile's slot is the request
    int64_t slots;
};

struct Tile {
    int b, row0, rows, n, pos0;  // request, first row, the request's rows, its new tokens, first token's position
    int lo, hi;                  // tokens any row of the tile sees
    bool over;                   // the request is longer than max_kv: its rows become NaN
};

// The tile of a slot.  Slots are handed out so that request b's begin at floor(cu[b] * G / 16) + b, which leaves
// it at least ceil(n_b * G / 16) of them: no sum over the requests' tiles is needed.
__device__ __forceinline__ Tile tile_of(const AttnArgs &a, const Geo &g, int64_t slot, int rows_per_tile)
{
    Tile t;
    int tile = 0;
    if (g.by_request) {
        t.b = (int)slot;
    } else {
        int lo = 0, hi = (int)a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)a.cu_q[mid] * g.G / rows_per_tile + mid <= slot)
                lo = mid;
            else
                hi = mid;
        }
        t.b = lo;
        tile = (int)(slot - ((int64_t)a.cu_q[lo] * g.G / rows_per_tile + lo));
    }
    const int q0 = a.cu_q[t.b], q1 = a.cu_q[t.b + 1];
    t.n = max(0, min(q1, (int)a.T) - q0);
    if (q0 < 0 || tile < 0) // no offsets of a step
        t.n = 0;
    t.rows = (int)min((int64_t)t.n * g.G, (int64_t)INT32_MAX);
    t.row0 = tile * rows_per_tile;
    const int len = max(a.kv_lens[t.b], 0);
    t.over = len > a.max_kv || len > a.table_stride << g.shift;
    t.pos0 = len - t.n;
    t.lo = t.hi = 0;
    if (t.row0 < t.rows && !t.over) {
        const int first = t.pos0 + t.row0 / g.G, last = t.pos0 + min(t.rows - 1, t.row0 + rows_per_tile - 1) / g.G;
        t.hi = max(0, last + 1);
        t.lo = a.window > 0 ? (int)max((int64_t)0, first - a.window + 1) & ~(ATT_STEP - 1) : 0;
    }
    return t;
}

// sum and maximum over the four lane groups that hold one row's tokens
__device__ __forceinline__ float groups_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float groups_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// A query row's elements 32 b + 8 g + j as binary16, times 2^-e with the row's magnitude below 2^e; returns 2^e.
template <int DT, int D, bool SPLIT> __device__ __forceinline__ float load_query(const typename RowType<DT>::T *q, int g, f16x8 (&hi)[D / 32], f16x8 (&lo)[SPLIT ? D / 32 : 1])
{
    using R = RowType<DT>;
    float x[D / 32][8];
    float am = 0.0f;
#pragma unroll
    for (int b = 0; b < D / 32; b++) {
        const RowVec<DT, 8> v = *reinterpret_cast<const RowVec<DT, 8> *>(q + 32 * b + 8 * g);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            x[b][j] = R::get(v.v[j]);
            am = fmaxf(am, fabsf(x[b][j]));
        }
    }
    am = groups_max(am);
    int e = 0;
    if (am > 0.0f && am < INFINITY) { // not finite: the row stays as it is, and its result is not finite either
        (void)frexpf(am, &e);
        e = min(e, 127);
    }
#pragma unroll
    for (int b = 0; b < D / 32; b++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float y = ldexpf(x[b][j], -e);
            const _Float16 h = (_Float16)y;
            hi[b][j] = h;
            if constexpr (SPLIT)
                lo[b][j] = (_Float16)(y - (float)h); // the rest: 22 bits in all
        }
    return ldexpf(1.0f, e);
}

template <int D> struct Partial { // of a tile and chunk, in the workspace
    float acc[ATT_ROWS][D];
    float ref[ATT_ROWS], sum[ATT_ROWS];
};

template <int DT, int D> __global__ __launch_bounds__(64 * ATT_WAVES, 2) void attn_kernel(AttnArgs a, Geo geo)
{
    using R = RowType<DT>;
    constexpr bool SPLIT = DT == LB_F32;
    constexpr int NB = D / 32, NC = D / 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int64_t id = blockIdx.x;
    const int split = (int)(id % geo.nsplit);
    const int64_t sh = id / geo.nsplit;
    const int head = (int)(sh % a.kv_heads);
    const int64_t slot = sh / a.kv_heads;
    const Tile t = tile_of(a, geo, slot, ATT_ROWS);
    if (t.row0 >= t.rows)
        return;
    const int start = t.lo + split * geo.chunk;
    if (split > 0 && start >= t.hi)
        return;
    const int end = min(t.hi, start + geo.chunk);
    const int P = 1 << geo.shift;

    // this lane's query row; the rows past the last repeat it, and are not stored
    const int row = min(t.row0 + c, t.rows - 1);
    const int tok = row / geo.G, hq = head * geo.G + row % geo.G;
    const int pos = t.pos0 + tok;                                              // last token it sees
    const int from = a.window > 0 ? (int)max((int64_t)0, pos - a.window + 1) : 0; // and the first
    f16x8 qh[NB], ql[SPLIT ? NB : 1];
    const typename R::T *qp = static_cast<const typename R::T *>(a.q) + (int64_t)(a.cu_q[t.b] + tok) * a.q_stride + (int64_t)hq * D;
    const float qscale = load_query<DT, D, SPLIT>(qp, g, qh, ql) * (a.scale * 1.44269504088896341f); // scores in powers of two

    f32x4 acc[NC];
#pragma unroll
    for (int n = 0; n < NC; n++)
        acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float ref = -INFINITY, sum = 0.0f;

    const int32_t *table = a.block_table + (int64_t)t.b * a.table_stride;
    const int64_t rec = kv_record_bytes(P, D);
    // positions that every row of the tile sees: no comparisons there
    const int all_to = t.pos0 + t.row0 / geo.G, all_from = a.window > 0 ? (int)max((int64_t)0, t.pos0 + (int64_t)(min(t.rows - 1, t.row0 + ATT_ROWS - 1) / geo.G) - a.window + 1) : 0;

    auto load = [&](int t0, Step<D> &s, int (&bad)[2]) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            // past the end the step's first page is read again; its tokens are masked
            const int at = t0 + 16 * u < end ? t0 + 16 * u : t0;
            int page = __builtin_amdgcn_readfirstlane(table[at >> geo.shift]);
            bad[u] = (uint32_t)page >= (uint32_t)a.pages;
            page = bad[u] ? 0 : page;
            const uint8_t *r = a.cache + ((int64_t)page * a.kv_heads + head) * rec;
            const int o = at & (P - 1);
            s.k[u] = load_words<NB>(r + kv_k_byte(D, o + c, g, 0));
            s.ks[u] = load_words<NB * 2>(r + kv_scale_byte(P, D, 0, o + 4 * g, 0));
            s.v[u] = load_words<NB>(r + kv_v_byte(P, D, o + 4 * g, c));
            s.vs[u] = load_words<NB * 2>(r + kv_scale_byte(P, D, 1, o + 4 * g, 0));
        }
    };

    for (int t0 = start + wave * ATT_STEP; t0 < end; t0 += ATT_WAVES * ATT_STEP) {
        Step<D> s;
        int bad[2];
        load(t0, s, bad);
        float sc[2][4], key[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            f32x4 x[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const f16x8 k = codes8(s.k[u].w[b]);
                x[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qh[b], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
                if constexpr (SPLIT)
                    x[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[b], x[b], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float v = 0.0f;
                uint32_t m = 0;
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    v = fmaf(half_of(s.ks[u].w[2 * b + i / 2], i & 1), x[b][i], v);
                    const uint32_t w = s.vs[u].w[2 * b + i / 2];
                    m = max(m, (i & 1 ? w >> 16 : w) & 0x7fffu);
                }
                sc[u][i] = bad[u] ? NAN : v * qscale;
                // the exponent of the largest value scale: an upper bound of its log2
                key[u][i] = sc[u][i] + (float)((int)(m >> 10) - 14);
            }
        }
        const bool whole = t0 + ATT_STEP <= end && t0 + ATT_STEP - 1 <= all_to && t0 >= all_from;
        bool see[2][4];
        bool past = false;
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = t0 + 16 * u + 4 * g + i;
                see[u][i] = whole || (j <= pos && j >= from && j < end);
                past = past || (see[u][i] && key[u][i] > ref + REF_MOST);
            }
        if (__ballot(past)) {
            float m = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    m = see[u][i] ? fmaxf(m, key[u][i]) : m;
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
        const float against = ref > -INFINITY ? ref : 0.0f;
        float p[2][4];
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                p[u][i] = see[u][i] ? exp2_raw(sc[u][i] - against) : 0.0f;
                sum += p[u][i];
            }
        const Pairs<D> vp[2] = {pair_tokens<D>(s.v[0]), pair_tokens<D>(s.v[1])};
#pragma unroll
        for (int b = 0; b < NB; b++) {
            f16x8 ph, pl;
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    // a token that is not seen may hold any scale, NaN too
                    const float w = see[u][i] ? p[u][i] * half_of(s.vs[u].w[2 * b + i / 2], i & 1) : 0.0f;
                    const _Float16 h = (_Float16)w;
                    ph[4 * u + i] = h;
                    if constexpr (SPLIT)
                        pl[4 * u + i] = (_Float16)(w - (float)h);
                }
#pragma unroll
            for (int half = 0; half < 2; half++) {
                f16x8 v;
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int pair = 0; pair < 2; pair++) {
                        const f16x2 h = codes2(vp[u].w[pair][half][b / 4], b);
                        v[4 * u + 2 * pair] = h.x;
                        v[4 * u + 2 * pair + 1] = h.y;
                    }
                acc[2 * b + half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, v, acc[2 * b + half], 0, 0, 0);
                if constexpr (SPLIT)
                    acc[2 * b + half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, v, acc[2 * b + half], 0, 0, 0);
            }
        }
    }

    // the four waves' results together
    __shared__ float s_acc[ATT_WAVES][ATT_ROWS][D];
    __shared__ float s_ref[ATT_WAVES][ATT_ROWS], s_sum[ATT_WAVES][ATT_ROWS];
    sum = groups_sum(sum);
    if (g == 0)
        s_ref[wave][c] = ref, s_sum[wave][c] = sum;
#pragma unroll
    for (int n = 0; n < NC; n++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            s_acc[wave][4 * g + i][16 * n + c] = acc[n][i];
    __syncthreads();
    const bool only = t.hi - t.lo <= geo.chunk; // nothing to join with
    Partial<D> *part = static_cast<Partial<D> *>(a.workspace) + (sh * geo.nsplit + split);
    for (int e = threadIdx.x; e < ATT_ROWS * D; e += 64 * ATT_WAVES) {
        const int r = e / D, d = e % D;
        float m = s_ref[0][r];
#pragma unroll
        for (int w = 1; w < ATT_WAVES; w++)
            m = fmaxf(m, s_ref[w][r]);
        float o = 0.0f, l = 0.0f;
#pragma unroll
        for (int w = 0; w < ATT_WAVES; w++) {
            const float f = s_ref[w][r] > -INFINITY ? exp2_raw(s_ref[w][r] - m) : s_sum[w][r]; // 0, or NaN where a score was
            o = fmaf(f, s_acc[w][r][d], o);
            l = fmaf(f, s_sum[w][r], l);
        }
        if (only) {
            const int rr = t.row0 + r;
            if (rr < t.rows) {
                typename R::T *op = static_cast<typename R::T *>(a.out) + (int64_t)(a.cu_q[t.b] + rr / geo.G) * a.out_stride + (int64_t)(head * geo.G + rr % geo.G) * D;
                op[d] = R::put(t.over ? NAN : l == 0.0f ? 0.0f : o / l);
            }
        } else {
            part->acc[r][d] = o;
            if (d == 0)
                part->ref[r] = m, part->sum[r] = l;
        }
    }
}

// Joins the chunks of a tile: D threads a row.
template <int DT, int D> __global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Geo geo)
{
    using R = RowType<DT>;
    constexpr int RPW = 256 / D; // rows a workgroup
    const int64_t id = blockIdx.x;
    const int64_t sh = id / (ATT_ROWS / RPW);
    const int r = (int)(id % (ATT_ROWS / RPW)) * RPW + threadIdx.x / D, d = threadIdx.x % D;
    const int head = (int)(sh % a.kv_heads);
    const Tile t = tile_of(a, geo, sh / a.kv_heads, ATT_ROWS);
    const int rr = t.row0 + r;
    if (rr >= t.rows || t.hi - t.lo <= geo.chunk)
        return;
    const int n = min((t.hi - t.lo + geo.chunk - 1) / geo.chunk, geo.nsplit);
    const Partial<D> *part = static_cast<const Partial<D> *>(a.workspace) + sh * geo.nsplit;
    float m = -INFINITY;
    for (int i = 0; i < n; i++)
        m = fmaxf(m, part[i].ref[r]);
    float o = 0.0f, l = 0.0f;
    for (int i = 0; i < n; i++) {
        const float f = part[i].ref[r] > -INFINITY ? exp2_raw(part[i].ref[r] - m) : part[i].sum[r];
        o = fmaf(f, part[i].acc[r][d], o);
        l = fmaf(f, part[i].sum[r], l);
    }
    typename R::T *op = static_cast<typename R::T *>(a.out) + (int64_t)(a.cu_q[t.b] + rr / geo.G) * a.out_stride + (int64_t)(head * geo.G + rr % geo.G) * D;
    op[d] = R::put(l == 0.0f ? 0.0f : o / l);
}

static Geo geometry(const AttnArgs &a)
{
    Geo g;
    g.G = (int)(a.q_heads / a.kv_heads);
    g.shift = 0;
    while (((int64_t)1 << g.shift) < a.page_tokens)
        g.shift++;
    g.by_request = a.max_q * g.G <= ATT_ROWS;
    g.slots = g.by_request ? a.B : a.T * g.G / ATT_ROWS + a.B;
    // tokens a tile may see, and the longest chunk that still gives the chip 2048 workgroups (8 a CU)
    int64_t span = a.max_kv;
    if (a.window > 0)
        span = span < a.window + ATT_ROWS + ATT_STEP ? span : a.window + ATT_ROWS + ATT_STEP;
    int64_t chunk = 2048;
    while (g.slots * a.kv_heads * ((span + chunk - 1) / chunk) > 65536 && chunk < span)
        chunk *= 2;
    while (chunk > 128 && g.slots * a.kv_heads * ((span + chunk - 1) / chunk) < 2048)
        chunk /= 2;
    g.chunk = (int)chunk;
    g.nsplit = (int)(span > 0 ? (span + chunk - 1) / chunk : 1);
    return g;
}

int64_t kv_attention_workspace(const AttnArgs &a)
{
    const Geo g = geometry(a);
    if (g.nsplit == 1)
        return 0;
    const int64_t one = ATT_ROWS * (a.head_dim + 2) * 4;
    return g.slots * a.kv_heads * g.nsplit * one;
}

int64_t kv_attention_workgroups(const AttnArgs &a)
{
    const Geo g = geometry(a);
    return g.slots * a.kv_heads * g.nsplit;
}

template <int DT, int D> static hipError_t run(const AttnArgs &a, hipStream_t s)
{
    static_assert(sizeof(Partial<D>) == ATT_ROWS * (D + 2) * 4, "the workspace's size");
    const Geo g = geometry(a);
    const int64_t tiles = g.slots * a.kv_heads;
    hipLaunchKernelGGL((attn_kernel<DT, D>), dim3((unsigned)(tiles * g.nsplit)), dim3(64 * ATT_WAVES), 0, s, a, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || g.nsplit == 1)
        return e;
    hipLaunchKernelGGL((attn_join_kernel<DT, D>), dim3((unsigned)(tiles * (ATT_ROWS * D / 256))), dim3(256), 0, s, a, g);
    return hipGetLastError();
}

template <int DT> static hipError_t run_d(const AttnArgs &a, hipStream_t s)
{
    switch (a.head_dim) {
    case 64:
        return run<DT, 64>(a, s);
    case 128:
        return run<DT, 128>(a, s);
    case 256:
        return run<DT, 256>(a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_kv_attention(int dtype, const AttnArgs &a, hipStream_t s)
{
    return dtype == LB_F32 ? run_d<LB_F32>(a, s) : dtype == LB_BF16 ? run_d<LB_BF16>(a, s) : run_d<LB_F16>(a, s);
}

} // namespace lb
