// Attention of many new tokens over the 4-bit cache (the operator of kvattn.hip, for bfloat16 and binary16 rows).
//
// A workgroup takes 128 or 256 query rows (token, head of the kv head's group) and walks the tokens 64 at a time.  Its
// waves unpack the 64 keys and values once, into binary16 in LDS, and each multiplies them with its own 32 rows:
// S^T = K Q^T and O += P V on v_mfma_f32_32x32x16_f16.  S^T leaves the matrix core with a query row along the lanes
// and runs of four tokens in each lane's registers, which is the order of the second product's left operand; LDS holds
// the operands as the instructions read them, 16 bytes a lane and lanes side by side, so nothing is shuffled and no
// bank is met twice.
//
// Three forms, of about 250 registers a wave, so two waves a SIMD: four waves of 32 rows, two workgroups a CU; eight
// waves of 32 rows, half of them unpacking keys and half values (geometry in kvattn.hip says where); eight waves in
// halves, two of them with the same 32 rows and each with 32 of the 64 tokens (in_halves below).  At head size 256 the
// registers are enough for one wave a SIMD, and there are four waves.
//
// What bounds it: instruction issue.  Per 32 rows and 32 tokens at head size 128 there are 512 cycles of matrix
// instructions, about 280 of the vector unit for the scores (16 exponentials of 8 cycles, and a fused multiply-add,
// a sum, a maximum and half a conversion each), and a share of the unpacking that falls with the rows a workgroup
// has.  One prompt of 8192 tokens, 32 heads over 8: 653 us in an undisturbed stream (842 TFLOP/s, a large library
// matrix product reaches 1132 here), 739 us a pass in the profiler's trace; tiles of 128 rows 719 us, and 16 rows a
// wave, each unpacking for itself, 1500 us.  Counted: the matrix cores are busy for 34 % of the cycles and the vector
// unit for 48 %, the two together leaving under a fifth to waits; raising a wave's priority around its products
// changes nothing.  LDS reads (16 bytes a lane, 16 KB a wave and 32 tokens) are at a quarter of their rate.
// Four prompts' chunks of 777 tokens after up to 1800, 20 heads over 5 (300 tiles, in halves): 87 us, matrix cores
// 13 %, vector unit 31 %: neither bounds it, but the chain of a step in the longest tiles, 1.76 us per 64 tokens.
//
// Precision: a code times its block's scale is rounded to binary16 (scales have 11 bits and the codes 1.5, 3 and 6
// two, so some lose one or two), and so are the weights: 2^-11 relative at most each, against the 2^-8 of a bfloat16
// output, and of the order of a binary16 output's own rounding (on prompts of normal values the keys' rounding gives
// 3.4e-4 of the result's size, the values' and the weights' 1.9e-4 each, the output's 2.0e-4; all of them 4.4e-4).
// Keeping the keys' rest in a second number would take half as many matrix instructions again and half as much LDS.
// The scales are taken times a power of two that brings the largest seen so far to 2^9, for keys and for values; it
// changes, with the tile unpacked again, if a later tile passes it by 2^5.  So only what is below 2^-22 of the largest
// loses more than that (7 * 2^-33 of the largest at most).  Scores are kept against a reference a row as in kvattn.hip,
// without the values' scales: weights end at 2^-31 of the row's largest.
#include "kvattn_internal.h"

namespace lb {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int PR_TOKENS = 64;
constexpr int EXP_MOST = 27, EXP_AIM = 23; // a scale's exponent field plus the shift: 6 times 2^13 still is a binary16

// A thread's share of 64 tokens, as the cache holds them.
template <int D> struct StagedKeys { // key i % 64: quarter i / 64 of every block, and its scales
    static constexpr int NB = D / 32;
    Words<NB> k;
    uint16_t s[NB];
    int page;
    bool in; // before the end
};
template <int D> struct StagedValues { // column i % 16 of two quads of tokens, eight apart, and the scales of half of the blocks
    static constexpr int NB = D / 32;
    Words<NB> v[2], s[2];
    int page;
};

// NW waves of 32 query rows.  With four, every thread unpacks keys and values; with eight, half of the waves do each.
// HALVES: waves w and w + NW / 2 have the same rows, and each one half of every 64 tokens; joined at the end (where the
// longest tiles' own time is what counts: in_halves).
template <int DT, int D, int NW, bool HALVES> __global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_prompt_kernel(AttnArgs a, Geo geo)
{
    using R = RowType<DT>;
    constexpr int NB = D / 32, NK = D / 16, SETS = HALVES ? NW / 2 : NW, ROWS = 32 * SETS;
    constexpr int HALF = PR_TOKENS * D; // binary16 numbers of 64 keys, or values
    __shared__ __align__(16) _Float16 lds[2][2][HALF];
    __shared__ int s_need[2][2], s_nan[2];
    __shared__ float s_ref[HALVES ? SETS : 1][64], s_sum[HALVES ? SETS : 1][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, h = lane >> 5, set = wave % SETS;
    const bool does_k = NW == 4 || wave < NW / 2, does_v = NW == 4 || wave >= NW / 2;
    const uint32_t sh = blockIdx.x / (uint32_t)geo.nsplit, rev = sh / (uint32_t)a.kv_heads;
    const int split = (int)(blockIdx.x - sh * geo.nsplit), head = (int)(sh - rev * (uint32_t)a.kv_heads);
    const int64_t slot = geo.slots - 1 - rev; // the last tokens' tiles see the most keys: they go first
    const Tile t = tile_of(a, geo, slot, ROWS);
    if (t.row0 >= t.rows)
        return;
    const int start = t.lo + split * geo.chunk;
    if (split > 0 && start >= t.hi)
        return;
    const int end = start + min(t.hi - start, geo.chunk), P = 1 << geo.shift; // start + chunk can pass 2^31

    if (tid < 4)
        s_need[tid >> 1][tid & 1] = 0;
    if (tid < 2)
        s_nan[tid] = 0;

    // this lane's query row; the rows past the last repeat it, and are not stored
    const int w0 = t.row0 + set * 32;
    const bool some = w0 < t.rows; // the wave has rows
    const int row = min(w0 + c, t.rows - 1);
    const int tok = row / geo.G, hq = head * geo.G + row % geo.G;
    const int pos = t.pos0 + tok, from = a.window > 0 ? (int)max((int64_t)0, pos - a.window + 1) : 0;
    const int pos_a = t.pos0 + min(w0, t.rows - 1) / geo.G, pos_z = t.pos0 + min(w0 + 31, t.rows - 1) / geo.G;
    const int from_a = a.window > 0 ? (int)max((int64_t)0, pos_a - a.window + 1) : 0;
    const int from_z = a.window > 0 ? (int)max((int64_t)0, pos_z - a.window + 1) : 0;

    f16x8 q[NK];
    float qscale;
    {
        const typename R::T *qp = static_cast<const typename R::T *>(a.q) + (int64_t)(a.cu_q[t.b] + tok) * a.q_stride + (int64_t)hq * D + 8 * h;
        float x[NK][8], am = 0.0f;
#pragma unroll
        for (int k = 0; k < NK; k++)
            am = fmaxf(am, load_eight<DT>(qp + 16 * k, x[k]));
        const int e = row_exponent(fmaxf(am, __shfl_xor(am, 32)));
        f16x8 none;
#pragma unroll
        for (int k = 0; k < NK; k++)
            query_halves<false>(x[k], e, a.scale < 0.0f, q[k], none);
        qscale = score_scale(a.scale, e);
    }

    f32x16 acc[NB];
#pragma unroll
    for (int n = 0; n < NB; n++)
#pragma unroll
        for (int i = 0; i < 16; i++)
            acc[n][i] = 0.0f;
    float ref = -INFINITY, sum = 0.0f;

    const int32_t *table = a.block_table + (int64_t)t.b * a.table_stride;
    const uint32_t rec = (uint32_t)kv_record_bytes(P, D), page_bytes = rec * (uint32_t)a.kv_heads; // below 2^32
    const uint8_t *cache = a.cache + (uint64_t)rec * head;
    // thread -> key: token i % 64, quarter i / 64; values: column, half of the blocks, quads 4s + g and 4s + 2 + g
    // of a half of the tokens (the eight tokens of one operand)
    const int i = tid & 255, kt = i & 63, kg = i >> 6;
    const int vc = i & 15, vb = (i >> 4) & 1, vp = i >> 5;
    const int v16 = (vp >> 1) * 16, vq = (vp & 1) * 4; // its 16 tokens, and the quad's first there

    // the pages are looked up a tile ahead of the loads that need them
    StagedKeys<D> sk;
    StagedValues<D> sv;
    int next_k = 0, next_v = 0;
    auto look_up = [&](int t0) {
        if (does_k)
            next_k = table[min(t0 + kt, end - 1) >> geo.shift];
        if (does_v)
            next_v = table[min(t0 + v16, end - 1) >> geo.shift];
    };
    auto stage_load = [&](int t0) {
        if (does_k) {
            const int j = t0 + kt;
            sk.in = j < end;
            sk.page = next_k;
            const uint8_t *r = cache + (uint64_t)((uint32_t)sk.page < (uint32_t)a.pages ? (uint32_t)sk.page : 0u) * page_bytes;
            const int o = j & (P - 1);
            sk.k = load_words<NB, false>(r + kv_k_byte(D, o, kg, 0));
#pragma unroll
            for (int b = 0; b < NB; b++)
                sk.s[b] = *reinterpret_cast<const uint16_t *>(r + kv_scale_byte(P, D, 0, o, 0) + 8 * b);
        }
        if (does_v) {
            sv.page = next_v;
            const uint8_t *r = cache + (uint64_t)((uint32_t)sv.page < (uint32_t)a.pages ? (uint32_t)sv.page : 0u) * page_bytes;
            const int o = ((t0 + v16) & (P - 1)) + vq;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                sv.v[u] = load_words<NB, false>(r + kv_v_byte(P, D, o + 8 * u, vc));
                sv.s[u] = load_words<NB, false>(r + kv_scale_byte(P, D, 1, o + 8 * u, vb * (NB / 2)));
            }
        }
    };
    // What is not there: keys past the end are 0 (their scores are masked), keys of a page that is none NaN; values
    // of either 0.
    auto settle = [&](int t0) {
        if (does_k) {
            const uint32_t put = !sk.in ? 0u : 0x7e00u;
            if (!sk.in || (uint32_t)sk.page >= (uint32_t)a.pages)
#pragma unroll
                for (int b = 0; b < NB; b++)
                    sk.s[b] = (uint16_t)put;
        }
        if (does_v) {
            const bool none = (uint32_t)sv.page >= (uint32_t)a.pages;
            if (none || t0 + PR_TOKENS > end)
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int w = 0; w < NB; w++) {
                        const int at = t0 + v16 + vq + 8 * u + 2 * (w & 1);
                        sv.s[u].w[w] &= none ? 0u : (at < end ? 0xffffu : 0u) | (at + 1 < end ? 0xffff0000u : 0u);
                    }
        }
    };
    auto key_bits = [&] { // the largest scale's magnitude bits
        uint32_t m = 0;
#pragma unroll
        for (int b = 0; b < NB; b++)
            m = max(m, (uint32_t)sk.s[b] & 0x7fffu);
        return m;
    };
    auto value_bits = [&] {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int w = 0; w < NB; w++)
                m = max_u16x2(m, sv.s[u].w[w] & 0x7fff7fffu);
        return max(m >> 16, m & 0xffffu);
    };
    // Unpacks into LDS with the scales times 2^shift; says in s_need and s_nan what does not fit.
    auto stage_store = [&](int t0, int par, int shift_k, int shift_v) {
        settle(t0);
        if (does_k) {
            uint32_t m = key_bits();
            if (m >= 0x7c00u) { // a NaN has no size, and is multiplied as it is
                m = 0;
#pragma unroll
                for (int b = 0; b < NB; b++)
                    m = max(m, (sk.s[b] & 0x7c00u) == 0x7c00u ? 0u : (uint32_t)sk.s[b]);
            }
            if ((int)(m >> 10) + shift_k > EXP_MOST)
                atomicMax(&s_need[par][0], (int)(m >> 10));
            const _Float16 f = (_Float16)ldexpf(1.0f, shift_k);
            _Float16 *K = lds[par][0];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const _Float16 d1 = __builtin_bit_cast(_Float16, sk.s[b]) * f;
                const f16x2 d = {d1, d1};
                u32x4 out;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    out[e] = __builtin_bit_cast(uint32_t, codes2(sk.k.w[b], e) * d);
                const int chunk = (((kt >> 5) * NK + 2 * b + (kg >> 1)) * 2 + (kg & 1)) * 32 + (kt & 31);
                *reinterpret_cast<u32x4 *>(K + chunk * 8) = out;
            }
        }
        if (does_v) {
            uint32_t m = value_bits();
            if (m >= 0x7c00u) { // not finite: taken out here, and put into the rows that see it afterwards
                atomicMax(&s_nan[par], t0 + 1);
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int w = 0; w < NB; w++) {
                        uint32_t &x = sv.s[u].w[w];
                        x &= ((x & 0x7c00u) == 0x7c00u ? 0u : 0xffffu) | ((x & 0x7c000000u) == 0x7c000000u ? 0u : 0xffff0000u);
                    }
                m = value_bits();
            }
            if ((int)(m >> 10) + shift_v > EXP_MOST)
                atomicMax(&s_need[par][1], (int)(m >> 10));
            const _Float16 f1 = (_Float16)ldexpf(1.0f, shift_v);
            const f16x2 f = {f1, f1};
            _Float16 *V = lds[par][1];
            const Pairs<D> w[2] = {pair_tokens<D>(sv.v[0]), pair_tokens<D>(sv.v[1])};
#pragma unroll
            for (int e = 0; e < NB / 2; e++) {
                f16x2 d[2][2];
#pragma unroll
                for (int u = 0; u < 2; u++)
#pragma unroll
                    for (int p = 0; p < 2; p++)
                        d[u][p] = __builtin_bit_cast(f16x2, sv.s[u].w[2 * e + p]) * f;
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    u32x4 out;
#pragma unroll
                    for (int u = 0; u < 2; u++)
#pragma unroll
                        for (int p = 0; p < 2; p++) {
                            // byte e of the lower or the upper half of the blocks
                            const uint32_t lower = w[u].w[p][half][0], upper = D > 128 ? w[u].w[p][half][Pairs<D>::W - 1] : lower >> (4 * NB);
                            out[2 * u + p] = __builtin_bit_cast(uint32_t, codes2(vb ? upper : lower, e) * d[u][p]);
                        }
                    const int b = vb * (NB / 2) + e;
                    const int chunk = ((((vp >> 2) * NB + b) * 2 + ((vp >> 1) & 1)) * 2 + (vp & 1)) * 32 + 16 * half + vc;
                    *reinterpret_cast<u32x4 *>(V + chunk * 8) = out;
                }
            }
        }
    };

    int shift_k = 0, shift_v = 0;
    __syncthreads();
    if (start < end) { // the first tokens' scales set the shifts
        look_up(start);
        stage_load(start);
        look_up(start + PR_TOKENS);
        settle(start);
        const uint32_t km = does_k ? key_bits() : 0, vm = does_v ? value_bits() : 0;
        atomicMax(&s_need[1][0], km < 0x7c00u ? (int)(km >> 10) : 0);
        atomicMax(&s_need[1][1], vm < 0x7c00u ? (int)(vm >> 10) : 0);
        __syncthreads();
        shift_k = min(15, EXP_AIM - __builtin_amdgcn_readfirstlane(s_need[1][0]));
        shift_v = min(15, EXP_AIM - __builtin_amdgcn_readfirstlane(s_need[1][1]));
    }

    int par = 0;
    for (int t0 = start; t0 < end; t0 += PR_TOKENS, par ^= 1) {
        // While this half of LDS is filled, the slower waves may still read the other one: one barrier a tile.  Past
        // the end the loads give some page of the request's, and are not used.
        stage_store(t0, par, shift_k, shift_v);
        stage_load(t0 + PR_TOKENS);
        look_up(t0 + 2 * PR_TOKENS);
        __syncthreads();
        const int need_k = __builtin_amdgcn_readfirstlane(s_need[par][0]), need_v = __builtin_amdgcn_readfirstlane(s_need[par][1]);
        if (need_k + shift_k > EXP_MOST || need_v + shift_v > EXP_MOST) { // for all waves alike
            const int was = shift_v;
            shift_k = min(shift_k, EXP_AIM - need_k);
            shift_v = min(shift_v, EXP_AIM - need_v);
            const float f = ldexpf(1.0f, shift_v - was);
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    acc[n][e] *= f;
            look_up(t0);
            stage_load(t0);
            __syncthreads(); // every wave has read s_need
            stage_store(t0, par, shift_k, shift_v);
            look_up(t0 + PR_TOKENS);
            stage_load(t0 + PR_TOKENS);
            look_up(t0 + 2 * PR_TOKENS);
            __syncthreads();
        }
        const bool nans = __builtin_amdgcn_readfirstlane(s_nan[par]) == t0 + 1;
        const float qs = qscale * ldexpf(1.0f, -shift_k);
        const f16x8 *K = reinterpret_cast<const f16x8 *>(lds[par][0]), *V = reinterpret_cast<const f16x8 *>(lds[par][1]);
#pragma unroll
        for (int turn = 0; turn < (HALVES ? 1 : 2); turn++) {
            const int sub = HALVES ? wave / SETS : turn;
            const int j0 = t0 + 32 * sub;
            if (!some || j0 >= end || j0 > pos_z || j0 + 31 < from_a)
                continue;
            f32x16 x;
#pragma unroll
            for (int i = 0; i < 16; i++)
                x[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < NK; k++)
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(K[((sub * NK + k) * 2 + h) * 32 + c], q[k], x, 0, 0, 0);
            if (!(j0 + 31 <= pos_a && j0 >= from_z && j0 + 31 < end)) {
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int j = j0 + 8 * (i / 4) + 4 * h + i % 4;
                    x[i] = j <= pos && j >= from && j < end ? x[i] : -INFINITY;
                }
            }
            float most = x[0];
#pragma unroll
            for (int i = 1; i < 16; i++)
                most = fmaxf(most, x[i]);
            // The weights are 2^(score - ref) and stay below 2^15; what the values' shift took comes off at the end.
            most *= qs;
            if (__ballot(most > ref + REF_MOST)) {
                const float m = fmaxf(most, __shfl_xor(most, 32));
                if (__ballot(m > ref + REF_MOST)) {
                    const float now = fmaxf(ref, m - REF_BELOW);
                    const float f = now > -INFINITY ? exp2_raw(ref - now) : 1.0f;
                    ref = now;
                    sum *= f;
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const float fr = __shfl(f, 8 * (i / 4) + 4 * h + i % 4); // the accumulators' rows
#pragma unroll
                        for (int n = 0; n < NB; n++)
                            acc[n][i] *= fr;
                    }
                }
            }
            const float against = ref > -INFINITY ? ref : 0.0f;
            f16x8 p[2];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const float w = exp2_raw(fmaf(x[i], qs, -against));
                sum += w;
                p[i / 8][i % 8] = (_Float16)w;
            }
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
                for (int n = 0; n < NB; n++)
                    acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(p[k], V[(((sub * NB + n) * 2 + k) * 2 + h) * 32 + c], acc[n], 0, 0, 0);
            if (nans) { // value scales that are not finite: NaN in their block's elements of the rows that see them
                for (int j = j0; j < min(j0 + 32, end); j++) {
                    const int page = table[j >> geo.shift];
                    if ((uint32_t)page >= (uint32_t)a.pages)
                        continue;
                    const uint8_t *r = a.cache + ((int64_t)page * a.kv_heads + head) * rec;
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        if ((*reinterpret_cast<const uint16_t *>(r + kv_scale_byte(P, D, 1, j & (P - 1), n)) & 0x7c00u) != 0x7c00u)
                            continue;
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            const int at = t.pos0 + min(w0 + 8 * (i / 4) + 4 * h + i % 4, t.rows - 1) / geo.G;
                            if (j <= at && (a.window == 0 || j > at - a.window))
                                acc[n][i] = NAN;
                        }
                    }
                }
            }
        }
    }
    sum += __shfl_xor(sum, 32);
    if constexpr (HALVES) { // the second half of the waves hands over, through the LDS of the tiles
        static_assert(sizeof(lds) >= SETS * 16 * NB * 64 * sizeof(float), "room for the accumulators");
        float *theirs = reinterpret_cast<float *>(lds) + set * 16 * NB * 64 + lane;
        __syncthreads();
        if (wave >= SETS) {
            s_ref[set][lane] = ref, s_sum[set][lane] = sum;
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
                for (int i = 0; i < 16; i++)
                    theirs[(n * 16 + i) * 64] = acc[n][i];
        }
        __syncthreads();
        if (wave >= SETS)
            return;
        const float ref2 = s_ref[set][lane], sum2 = s_sum[set][lane], m = fmaxf(ref, ref2);
        // a half without a score above -inf has a sum of 0, or NaN where a score was
        const float f = ref > -INFINITY ? exp2_raw(ref - m) : sum, f2 = ref2 > -INFINITY ? exp2_raw(ref2 - m) : sum2;
        ref = m;
        sum = fmaf(f, sum, f2 * sum2);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float fr = __shfl(f, 8 * (i / 4) + 4 * h + i % 4), fr2 = __shfl(f2, 8 * (i / 4) + 4 * h + i % 4);
#pragma unroll
            for (int n = 0; n < NB; n++)
                acc[n][i] = fmaf(fr, acc[n][i], fr2 * theirs[(n * 16 + i) * 64]);
        }
    }
    if (!some)
        return;
    const float back = ldexpf(1.0f, -shift_v);
    const bool only = t.hi - t.lo <= geo.chunk;
    using Part = PartialOf<D, ROWS, ROWS>;
    Part *part = static_cast<Part *>(a.workspace) + (slot * a.kv_heads + head) * geo.nsplit + split;
    const float inv = t.over ? NAN : sum == 0.0f ? 0.0f : back / sum;
    if (!only && h == 0)
        part->ref[set * 32 + c] = ref, part->sum[set * 32 + c] = sum;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int r = 8 * (i / 4) + 4 * h + i % 4, rr = w0 + r;
        const float f = __shfl(inv, r);
        if (rr >= t.rows)
            continue;
        typename R::T *op = static_cast<typename R::T *>(a.out) + (int64_t)(a.cu_q[t.b] + rr / geo.G) * a.out_stride + (int64_t)(head * geo.G + rr % geo.G) * D;
#pragma unroll
        for (int n = 0; n < NB; n++) {
            if (only)
                op[32 * n + c] = R::put(acc[n][i] * f);
            else
                part->acc[set * 32 + r][32 * n + c] = acc[n][i] * back;
        }
    }
}

// Whether tiles of 128 rows take eight waves in halves (one workgroup a CU) or four (two a CU, each nearly as fast as
// one alone).  Per 64 tokens, head size 128: a workgroup of four waves 2.3 us, alone or beside another; one of eight
// 1.76.  So halves pay where one round of 256 workgroups has nearly all of the work, and cost up to half where there are
// two rounds of equal tiles.  Measured, four waves against halves, us at head size 128 (64 behaves alike, a little in
// favour of halves), 32 heads over 8 where nothing else is said:
//   one round, not split:  one prompt of 1024 after 0 / 700 / 3000 others 50 / 72 / 145 against 44 / 59 / 113; 8 requests
//       of 128 after 470 34 against 30; two windows of 300 over 1024 32 against 31.  Of 100 tokens in all 22 against 24;
//       16 of 64 (512 slots of which 256 have rows, in 384 places) 62 against 85: hence the bounds on both.
//   two, uneven requests:  4 of 777 to 2600, 20 / 5 heads 104 against 86; 6 of 330 to 4000 150 against 129; 12 of 160 to
//       6000 (400 slots) 220 against 192; 5 of 380 to 800 47 against 56; 10 of 190 to 1500 (376 slots) 70 against 77
//   two, one prompt:  from its start, 1100 / 1400 / 1700 / 1800 tokens (432 and 456 slots the last) 55 / 64 / 74 / 77
//       against 47 / 60 / 74 / 79; after half and as many others again 81 / 100 against 82 / 110
//   two, equal requests:  4 prompts of 300 33 against 48; 4 of 777 (20 / 5) 53 against 70; a window of 300 38 against 58
//   parts of split tiles:  47 to 90 against 65 to 126; fewer than 256 workgroups (short requests) 19 to 27 against 21 to 29
static bool in_halves(const AttnArgs &a, const Geo &g)
{
    const int64_t tiles = g.slots * a.kv_heads, rows = a.T < a.B * a.max_q ? a.T : a.B * a.max_q;
    const int64_t filled = g.by_request ? tiles : (rows * g.G + g.tile - 1) / g.tile * a.kv_heads;
    const int64_t span = a.window > 0 ? a.window : a.max_kv;
    if (g.nsplit > 1 || span < 256)
        return false;
    if (filled <= 256)
        return tiles <= 320;
    if (4 * rows <= 3 * a.B * a.max_q)
        return filled <= 320 && (span >= 2048 ? tiles <= 400 : span >= 1024 && tiles <= 336);
    return a.B == 1 && a.window == 0 && tiles <= 432 && 5 * a.max_kv <= 6 * a.max_q;
}

template <int DT, int D> static hipError_t run(const AttnArgs &a, const Geo &g, hipStream_t s)
{
    const dim3 grid((unsigned)(g.slots * a.kv_heads * g.nsplit));
    if constexpr (D <= 128) // at 256 the registers are enough for one wave a SIMD
        if (g.tile == 2 * PROMPT_ROWS) {
            hipLaunchKernelGGL((attn_prompt_kernel<DT, D, 8, false>), grid, dim3(512), 0, s, a, g);
            return hipGetLastError();
        }
    if constexpr (D <= 128)
        if (in_halves(a, g)) {
            hipLaunchKernelGGL((attn_prompt_kernel<DT, D, 8, true>), grid, dim3(512), 0, s, a, g);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((attn_prompt_kernel<DT, D, 4, false>), grid, dim3(256), 0, s, a, g);
    return hipGetLastError();
}

template <int DT> static hipError_t run_d(const AttnArgs &a, const Geo &g, hipStream_t s)
{
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

hipError_t launch_attn_prompt(int dtype, const AttnArgs &a, const Geo &g, hipStream_t s)
{
    return dtype == LB_BF16 ? run_d<LB_BF16>(a, g, s) : dtype == LB_F16 ? run_d<LB_F16>(a, g, s) : hipErrorInvalidValue;
}

} // namespace lb
