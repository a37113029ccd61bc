// The experts' products with up to 16 rows of activations a tile, on the int8 matrix cores.
//
// Between a decode step's one or two rows an expert, where nibble dot products on the vector unit keep up with HBM
// (experts.hip), and a prompt's hundreds (gemm.hip) products of 16 x 16 read the weights once for 16 rows: the activations
// are the A operand (from LDS), 16 weight rows the B operand, unpacked in registers as they come from HBM.  Lane (n, q) =
// (lane mod 16, lane / 16) loads whole 16-byte records, record 4 s + q of weight row n.
//  * The order of weights within a block is free, as long as the activations have the same: they are staged in the order in
//    which shifts and masks isolate the weights' bytes, which needs no further arrangement.  Q4_0: nibbles in the upper
//    halves of bytes, 16 w (the factor is in the activation scale); Q2_0_g64: codes w + 1; Q1_0: 2 bit = w + 1.  The sum of
//    the activations that codes carry too much is subtracted by the accumulator's start.
//  * Results are read as fp32 through the bias 1.5 * 2^23 as in gemm.hip: round(d_x * isum), then one multiply-add with the
//    weight scale (one value a lane).  That takes as long as anything else, and 16 x 16 results of which few are wanted
//    would cost it in full.  Hence two ways:
//  * Up to four rows (eight, of Q4_0 and Q2_0_g64, in two turns): the A operand's 16 rows are four rows times four records.
//    Its row (j, r) has row r's activations where quarter j's record is, and zeros elsewhere, so that one product has the
//    sums of four records, each lane those of its own record, as it was loaded; the quarters are added at the end.
//  * More: the A operand's rows are 16 rows of activations.  A q8_0 block's weights have to be spread over the four q then, so
//    four records are transposed between the lanes' quarters, dword by dword (v_permlane32_swap, v_permlane16_swap: four
//    instructions for four records).  A Q2_0_g64 dword belongs to one of its record's two blocks: the 64-deep product is
//    taken twice, with the other block's activations read as zeros.
// A wave has G groups of 16 weight rows, so that what it reads from LDS (activations, scales, accumulator starts) is read
// once for all of them.  lowbit_gemm takes the same kernel for Q4_0 products of few rows, whose tiles need no plan.
//
// Measured (us, the first way against the second alone): 64 experts of 1536 x 2048 with half a pair each Q1_0 7.7 and 12.0,
// Q2_0 8.5 and 14.4, Q4_0 12.1 and 15.4; 360 pairs of 128 experts of 2048 x 768 14.6 and 16.4, 14.6 and 18.4, 22.7 and 24.9 (107
// MB of Q4_0: 4.7 TB/s, bound by loads; two runs of weight rows a workgroup, which starts half as often, take 5 to 50 %
// longer, one group a wave up to 30).  Of Q1_0 and Q2_0, 27 and 54 MB there, it is not the bytes: the vector unit is 58 and 49 %
// busy, and the time grows with the columns (768 to 4608 of them: 15 to 66 us, 14 to 76), so it is their unpacking and their
// activations' way through LDS, and not a workgroup's start.  With many rows the vector unit bounds it (12 to 14 instructions
// for eight weights of a lane and 16 rows, eight of them the rescale).  Two things made that: each row's scales staged through
// LDS by whole lines (read four at a time from memory, their lines came through the caches again for every step, Q4_0 875 ->
// 577 us for 32768 pairs), and results in vector registers.
#include "matvec_tile.h"
#include "serve_internal.h"

namespace lb {

namespace {

constexpr int TR = 16;   // activation rows a tile
constexpr int KC = 1024; // columns staged at a time: 18 or 20 KiB of LDS, 2 to 8 of zeros, and 1 to 9 of weight scales
constexpr uint32_t BIAS = 0x4B400000u; // 1.5 * 2^23 as fp32 bits
constexpr float BIASF = 12582912.0f;

typedef int v4i __attribute__((ext_vector_type(4)));

template <int FMT, int G, bool KS> struct __attribute__((aligned(16))) TileLds {
    static constexpr int BLOCKS = KC / QK8, RECORDS = KC / F<FMT>::SW, WROWS = (KS ? 16 : 64) * G;
    // a weight row's scales of the chunk, 8 bytes apart from the next row's (16 rows' reads of 8 bytes meet 16 pairs of banks)
    static constexpr int SCALES = RECORDS + 4;
    // Few rows: [four records][block][half][row / 4][record][row mod 4] 16 bytes.  Otherwise Q4_0, Q1_0: [block][q][row] 8
    // bytes; Q2_0_g64: [record][q][row] 16 bytes.
    uint32_t x[KC * TR / 4];
    uint32_t zeros[F<FMT>::SW * TR]; // as many bytes as four records have there, so that both are read at the same offsets
    float dx[BLOCKS * TR];   // [block][row]
    int start[FMT == LB_Q4_0 ? 4 : BLOCKS * TR]; // accumulator starts, [block][row]
    uint16_t dw[WROWS * SCALES];
};

__device__ __forceinline__ uint32_t bperm(uint32_t s0, uint32_t s1, uint32_t sel) { return __builtin_amdgcn_perm(s0, s1, sel); }

// A workgroup barrier after this thread's LDS accesses, which leaves its loads from memory in flight (__syncthreads() would
// wait for them); the empty asm statements keep the compiler from moving LDS accesses across it.
__device__ __forceinline__ void chunk_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// d[i] of lane quarter q becomes d[q] of quarter i
__device__ __forceinline__ void transpose_quarters(uint32_t (&d)[4])
{
    auto p = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    d[0] = p[0], d[2] = p[1];
    p = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    d[1] = p[0], d[3] = p[1];
    p = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
    d[0] = p[0], d[1] = p[1];
    p = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
    d[2] = p[0], d[3] = p[1];
}

// Four values a lane, summed over the lanes' quarters: value row_of(q) in quarter q
__device__ __forceinline__ int row_of(int q) { return (q & 1) << 1 | q >> 1; }
__device__ __forceinline__ float sum_quarters(const float (&v)[4])
{
    auto both = [](float a, float b, bool row) {
        const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
        const auto p = row ? __builtin_amdgcn_permlane16_swap(x, y, false, false) : __builtin_amdgcn_permlane32_swap(x, y, false, false);
        return __uint_as_float((uint32_t)p[0]) + __uint_as_float((uint32_t)p[1]);
    };
    return both(both(v[0], v[1], false), both(v[2], v[3], false), true);
}

// Block b (32 columns from column 32 b of the chunk) of activation row r: 32 bytes, in the order in which the weights' bytes
// are isolated, and their scale.
template <int FMT, bool FEW, typename Lds> __device__ __forceinline__ void stage_block(Lds &lds, int b, int r, uint4 lo, uint4 hi, float dx)
{
    constexpr int BPR = F<FMT>::SW / QK8;
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (FEW) {
        const int rec = b / BPR;
        uint32_t *to = lds.x + (((rec >> 2) * BPR + b % BPR) * 2 * TR + (r >> 2 << 2)) * 16 + ((rec & 3) * 4 + (r & 3)) * 4;
#pragma unroll
        for (int m = 0; m < 2; m++) {
            const uint32_t *e = w + 4 * m;
            uint4 o;
            if (FMT == LB_Q2_0_G64) { // weights 16 m + 4 t + i at byte t of dword i
                const uint32_t lo01 = bperm(e[1], e[0], 0x05010400u), hi01 = bperm(e[1], e[0], 0x07030602u);
                const uint32_t lo23 = bperm(e[3], e[2], 0x05010400u), hi23 = bperm(e[3], e[2], 0x07030602u);
                o = make_uint4(bperm(lo23, lo01, 0x05040100u), bperm(lo23, lo01, 0x07060302u), bperm(hi23, hi01, 0x05040100u), bperm(hi23, hi01, 0x07060302u));
            } else { // weights 16 m + 0, 2, 4, 6, then 1, 3, 5, 7, then eight further on
                o = make_uint4(bperm(e[1], e[0], 0x06040200u), bperm(e[1], e[0], 0x07050301u), bperm(e[3], e[2], 0x06040200u), bperm(e[3], e[2], 0x07050301u));
            }
            *reinterpret_cast<uint4 *>(to + m * TR * 16) = o;
        }
    } else if (FMT == LB_Q2_0_G64) { // weights 16 q + 4 t + s at byte t of dword s
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t *e = w + 4 * h;
            const uint32_t lo01 = bperm(e[1], e[0], 0x05010400u), hi01 = bperm(e[1], e[0], 0x07030602u);
            const uint32_t lo23 = bperm(e[3], e[2], 0x05010400u), hi23 = bperm(e[3], e[2], 0x07030602u);
            *reinterpret_cast<uint4 *>(lds.x + (b >> 1) * 256 + ((2 * (b & 1) + h) * TR + r) * 4) =
                make_uint4(bperm(lo23, lo01, 0x05040100u), bperm(lo23, lo01, 0x07060302u), bperm(hi23, hi01, 0x05040100u), bperm(hi23, hi01, 0x07060302u));
        }
    } else { // weights 8 q + 0, 2, 4, 6, then 8 q + 1, 3, 5, 7
#pragma unroll
        for (int q = 0; q < 4; q++)
            *reinterpret_cast<uint2 *>(lds.x + b * 128 + (q * TR + r) * 2) =
                make_uint2(bperm(w[2 * q + 1], w[2 * q], 0x06040200u), bperm(w[2 * q + 1], w[2 * q], 0x07050301u));
    }
    int sq = 0;
    if (FMT != LB_Q4_0) {
#pragma unroll
        for (int k = 0; k < 8; k++)
            sq = __builtin_amdgcn_sdot4((int)w[k], 0x01010101, sq, false);
    }
    lds.dx[b * TR + r] = FMT == LB_Q4_0 ? dx * 0.0625f : dx;
    if (FMT != LB_Q4_0)
        lds.start[b * TR + r] = (int)BIAS - sq;
}

// Place r's pair
__device__ __forceinline__ uint32_t pair_at(const ExpertsArgs &a, const int32_t *pairs, int tile, int r)
{
    return min(pairs ? (uint32_t)pairs[r] : (uint32_t)(TR * tile + r), (uint32_t)(a.pairs - 1));
}

// The main loop, for tiles of up to 4 NG rows.
template <int FMT, int G, bool WHOLE, bool KS, int NG>
__device__ __forceinline__ void tile_rows(const ExpertsArgs &a, TileLds<FMT, G, KS> &lds, const uint8_t *W, int chunk, int rows, uint32_t row16,
                                          const int32_t *pairs, int tile)
{
    using Lds = TileLds<FMT, G, KS>;
    constexpr int BPR = F<FMT>::SW / QK8; // q8_0 blocks a record
    constexpr bool FEW = NG < 4;
    constexpr int ROWS = 4 * NG, STEP4 = F<FMT>::SW * TR; // dwords of four records' activations
    const int ns = a.K / F<FMT>::SW;
    const uint8_t *scales = W + (int64_t)a.N * ns * CODE_BYTES;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
    const int wrow = (KS ? 0 : wave * G * 16) + (lane & 15); // this lane's weight row of the workgroup's, in group 0
    const int n0 = chunk * Lds::WROWS + wrow;
    // staging: a thread has blocks tid / ROWS, and so on by 256 / ROWS, of activation row tid mod ROWS
    constexpr int BSTEP = WG / ROWS, U = (Lds::BLOCKS + BSTEP - 1) / BSTEP;
    const int sr = threadIdx.x % ROWS, sb = threadIdx.x / ROWS;
    const int64_t row = (uint32_t)__shfl((int)row16, sr);

    uint32_t rec0[G]; // first record of the lane's rows
#pragma unroll
    for (int g = 0; g < G; g++)
        rec0[g] = (uint32_t)min(n0 + 16 * g, a.N - 1) * (uint32_t)ns;
    // A step is H times four records of a row.  Q4_0, whose records are soonest computed, takes 128 bytes, whole lines, at
    // once; for the others the registers of a second half cost more than the lines' second visit.
    constexpr int H = FMT == LB_Q4_0 ? 2 : 1;
    struct Regs {
        uint4 code[H][G];
    };
    auto issue = [&](Regs &r, int s) {
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int h = 0; h < H; h++) {
                const v4u c = *(gv4u *)((gu8 *)W + (rec0[g] + (uint32_t)min(4 * (H * s + h) + q, ns - 1)) * (uint32_t)CODE_BYTES);
                r.code[h][g] = make_uint4(c.x, c.y, c.z, c.w);
            }
    };
    // The activations that this lane gives a product: row lane mod 4 of its quarter's record, or zeros.
    const bool live = ((lane & 15) >> 2) == q;
    const uint32_t xat = live ? (uint32_t)(4 * (lane & 15)) : (uint32_t)(lds.zeros - lds.x);
    float acc[FEW ? NG : 1][G][4] = {};
    auto compute_few = [&](const uint4 (&code)[G], int s, int first) { // records 4 s .. 4 s + 3; first: the chunk's first
        const int own = min(4 * s + q, ns - 1) - first; // this quarter's record, of the chunk's
        float dw[G];
#pragma unroll
        for (int g = 0; g < G; g++) {
            dw[g] = half_bits_to_float(lds.dw[(wrow + g * 16) * Lds::SCALES + own]);
            if (!WHOLE)
                dw[g] = 4 * s + q < ns ? dw[g] : 0.0f; // no record: its sums count nothing
        }
        const uint32_t *x = lds.x + (xat + (live ? (uint32_t)((4 * s - first) / 4 * STEP4) : 0u));
#pragma unroll
        for (int b = 0; b < BPR; b++) {
            v4i w[G][2];
#pragma unroll
            for (int g = 0; g < G; g++) {
                const uint32_t v[4] = {code[g].x, code[g].y, code[g].z, code[g].w};
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        uint32_t o;
                        if (FMT == LB_Q2_0_G64) { // codes i, 4 + i, 8 + i, 12 + i
                            o = (v[2 * b + m] >> (2 * i)) & 0x03030303u;
                        } else {
                            const uint32_t d = v[2 * m + (i >> 1)];
                            if (FMT == LB_Q4_0) // even nibbles, odd nibbles
                                o = (i & 1 ? d : d << 4) & 0xF0F0F0F0u;
                            else // the sign of block b, at bit b of each nibble, moved to bit 1
                                o = (i & 1 ? d >> (b + 3) : b ? d >> (b - 1) : d << 1) & 0x02020202u;
                        }
                        w[g][m][i] = (int)o;
                    }
            }
#pragma unroll
            for (int r = 0; r < NG; r++) {
                const v4i x0 = *reinterpret_cast<const v4i *>(x + b * 512 + r * 64), x1 = *reinterpret_cast<const v4i *>(x + b * 512 + 256 + r * 64);
                const int at = (own * BPR + b) * TR + 4 * r;
                const float4 dx = *reinterpret_cast<const float4 *>(lds.dx + at);
                v4i start = {(int)BIAS, (int)BIAS, (int)BIAS, (int)BIAS};
                if (FMT != LB_Q4_0)
                    start = *reinterpret_cast<const v4i *>(lds.start + at);
                const float dxv[4] = {dx.x, dx.y, dx.z, dx.w};
                float c[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    c[i] = -dxv[i] * BIASF; // exact: an 11-bit significand times 3 * 2^22
#pragma unroll
                for (int g = 0; g < G; g++) {
                    v4i D = __builtin_amdgcn_mfma_i32_16x16x64_i8(x0, w[g][0], start, 0, 0, 0);
                    D = __builtin_amdgcn_mfma_i32_16x16x64_i8(x1, w[g][1], D, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        acc[r][g][i] = fmaf(dw[g], fmaf(dxv[i], __int_as_float(D[i]), c[i]), acc[r][g][i]); // round(d_x * isum)
                }
            }
        }
    };

    auto compute_16 = [&](const uint4 (&code)[G], int s, int first) { // the same
        uint32_t d[G][4];
        uint2 sc[G];
#pragma unroll
        for (int g = 0; g < G; g++) {
            sc[g] = *reinterpret_cast<const uint2 *>(lds.dw + (wrow + g * 16) * Lds::SCALES + (4 * s - first));
            d[g][0] = code[g].x, d[g][1] = code[g].y, d[g][2] = code[g].z, d[g][3] = code[g].w;
            transpose_quarters(d[g]);
        }
        auto record = [&](int j) {
            const int rec = 4 * s + j;
            // the record's weights as bytes: Q2_0_g64 16 of them, the others 8 for each of its blocks
            constexpr int WB = FMT == LB_Q1_0 ? 4 : 1, WD = FMT == LB_Q2_0_G64 ? 4 : 2;
            uint32_t w[G][WB][WD];
            float dw[G];
#pragma unroll
            for (int g = 0; g < G; g++) {
                const uint32_t v = d[g][j], h = j < 2 ? sc[g].x : sc[g].y;
                dw[g] = half_bits_to_float((uint16_t)(j & 1 ? h >> 16 : h));
                if (FMT == LB_Q2_0_G64) {
#pragma unroll
                    for (int i = 0; i < WD; i++)
                        w[g][0][i] = (v >> (2 * i)) & 0x03030303u;
                } else if (FMT == LB_Q4_0) {
                    w[g][0][0] = (v << 4) & 0xF0F0F0F0u, w[g][0][1] = v & 0xF0F0F0F0u;
                } else { // the sign of block b, at bit b of each nibble, moved to bit 1
#pragma unroll
                    for (int b = 0; b < WB; b++)
                        w[g][b][0] = (b ? v >> (b - 1) : v << 1) & 0x02020202u, w[g][b][1] = (v >> (b + 3)) & 0x02020202u;
                }
            }
            const int r0 = rec - first;
            float tg[G][4];
#pragma unroll
            for (int b = 0; b < BPR; b++) {
                const int at = (r0 * BPR + b) * TR + 4 * q;
                const float4 dx = *reinterpret_cast<const float4 *>(lds.dx + at);
                v4i start = {(int)BIAS, (int)BIAS, (int)BIAS, (int)BIAS};
                if (FMT != LB_Q4_0)
                    start = *reinterpret_cast<const v4i *>(lds.start + at);
                const float dxv[4] = {dx.x, dx.y, dx.z, dx.w};
                float c[4];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    c[i] = -dxv[i] * BIASF; // exact: an 11-bit significand times 3 * 2^22
                v4i xw = {};
                long xb = 0;
                if (FMT == LB_Q2_0_G64) {
                    const uint32_t *p = (q >> 1) == b ? lds.x + r0 * 256 + lane * 4 : lds.zeros;
                    xw = *reinterpret_cast<const v4i *>(p);
                } else {
                    xb = *reinterpret_cast<const long *>(lds.x + (r0 * BPR + b) * 128 + lane * 2);
                }
#pragma unroll
                for (int g = 0; g < G; g++) {
                    v4i D;
                    if (FMT == LB_Q2_0_G64) {
                        const v4i wv = {(int)w[g][0][0], (int)w[g][0][1], (int)w[g][0][WD - 2], (int)w[g][0][WD - 1]};
                        D = __builtin_amdgcn_mfma_i32_16x16x64_i8(xw, wv, start, 0, 0, 0);
                    } else {
                        const int wb = FMT == LB_Q1_0 ? b : 0;
                        D = __builtin_amdgcn_mfma_i32_16x16x32_i8(xb, (long)((uint64_t)w[g][wb][1] << 32 | w[g][wb][0]), start, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float f = fmaf(dxv[i], __int_as_float(D[i]), c[i]); // round(d_x * isum)
                        tg[g][i] = b ? tg[g][i] + f : f;
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    acc[0][g][i] = fmaf(dw[g], tg[g][i], acc[0][g][i]);
        };
        if (4 * s + 4 <= ns) { // uniform: in one piece, so that one record's loads from LDS go out in another's arithmetic
#pragma unroll
            for (int j = 0; j < 4; j++)
                record(j);
        } else {
#pragma unroll
            for (int j = 0; j < 3; j++)
                if (4 * s + j < ns)
                    record(j);
        }
    };

    const int8_t *xq = a.xq + row * a.K;
    const uint16_t *xs = a.xs + row * (a.K / QK8);

    // and eight scales of a weight row (their lines would be read again for every four records otherwise)
    constexpr int PARTS = Lds::RECORDS / 8, PIECES = Lds::WROWS * PARTS, P = (PIECES + WG - 1) / WG;
    // A chunk's activations and scales are loaded into registers a chunk ahead, the weights a step ahead: what is waited for
    // was asked for long before.
    uint4 lo[U], hi[U], dws[P];
    uint32_t sc[U];
    auto load_chunk = [&](int k0) {
        const int nblk = min(Lds::BLOCKS, (a.K - k0) / QK8);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int b = min(sb + BSTEP * u, nblk - 1);
            lo[u] = *reinterpret_cast<const uint4 *>(xq + k0 + 32 * b);
            hi[u] = *reinterpret_cast<const uint4 *>(xq + k0 + 32 * b + 16);
            sc[u] = xs[k0 / QK8 + b];
        }
#pragma unroll
        for (int u = 0; u < P; u++) {
            const int p = threadIdx.x + u * WG, rec = k0 / F<FMT>::SW + p % PARTS * 8;
            const uint32_t at = (uint32_t)min(chunk * Lds::WROWS + p / PARTS, a.N - 1) * (uint32_t)ns;
            if (WHOLE) { // the eight lie in the row, and on 16 bytes
                const v4u d = *(gv4u *)((gu8 *)scales + (at + (uint32_t)min(rec, ns - 8)) * 2u);
                dws[u] = make_uint4(d.x, d.y, d.z, d.w);
            } else {
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 8; j++)
                    h[j] = *(gu16 *)((gu8 *)scales + (at + (uint32_t)min(rec + j, ns - 1)) * 2u);
                dws[u] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
            }
        }
    };
    const int steps = (ns + 4 * H - 1) / (4 * H);
    constexpr int SPC = Lds::RECORDS / (4 * H); // steps a chunk
    auto stage_chunk = [&](int k0) { // the loaded one, from column k0; then the next one's loads go out
        const int nblk = min(Lds::BLOCKS, (a.K - k0) / QK8);
        if (k0)
            chunk_barrier(); // every wave has read the chunk before
#pragma unroll
        for (int v = 0; v < U; v++)
            if (sb + BSTEP * v < nblk)
                stage_block<FMT, FEW>(lds, sb + BSTEP * v, sr, lo[v], hi[v], half_bits_to_float((uint16_t)sc[v]));
#pragma unroll
        for (int v = 0; v < P; v++) {
            const int p = threadIdx.x + v * WG;
            if (PIECES % WG == 0 || p < PIECES) {
                uint2 *to = reinterpret_cast<uint2 *>(lds.dw + p / PARTS * Lds::SCALES + p % PARTS * 8);
                to[0] = make_uint2(dws[v].x, dws[v].y), to[1] = make_uint2(dws[v].z, dws[v].w);
            }
        }
        if (k0 + KC < a.K) // uniform
            load_chunk(k0 + KC);
        chunk_barrier();
    };
    auto step = [&](const Regs &r, int s, int first) {
#pragma unroll
        for (int h = 0; h < H; h++)
            if (h == 0 || 4 * (H * s + h) < ns) { // uniform
                if constexpr (FEW)
                    compute_few(r.code[h], H * s + h, first);
                else
                    compute_16(r.code[h], H * s + h, first);
            }
    };
    Regs buf[2];
    load_chunk(0);
    for (int i = threadIdx.x; i < STEP4; i += WG) // (a barrier follows)
        lds.zeros[i] = 0;
    if constexpr (KS) {
        // the waves have the same weight rows and a step of every chunk each, and add up what they have at the end
        const int mine = min(wave, SPC - 1), chunks_k = (steps + SPC - 1) / SPC;
        issue(buf[0], min(mine, steps - 1));
        for (int c = 0; c < chunks_k; c += 2) {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                if (c + u >= chunks_k) // uniform
                    break;
                stage_chunk((c + u) * KC);
                issue(buf[1 - u], min((c + u + 1) * SPC + mine, steps - 1));
                __builtin_amdgcn_sched_barrier(0); // these loads go out before this step's arithmetic
                if (wave < SPC && (c + u) * SPC + wave < steps) // uniform in the wave
                    step(buf[u], (c + u) * SPC + wave, (c + u) * Lds::RECORDS);
            }
        }
        chunk_barrier();
    } else {
        issue(buf[0], 0);
        for (int s = 0; s < steps; s += 2) {
#pragma unroll
            for (int u = 0; u < 2; u++) {
                if (s + u >= steps) // uniform
                    break;
                if (u % SPC == 0 && (s + u) % SPC == 0) // uniform: the next chunk
                    stage_chunk((s + u) / SPC * KC);
                issue(buf[1 - u], min(s + u + 1, steps - 1));
                __builtin_amdgcn_sched_barrier(0); // these loads go out before this step's arithmetic
                step(buf[u], s + u, (s + u) / SPC * Lds::RECORDS);
            }
        }
    }
    // FEW: the four quarters' sums, row row_of(q) of each four in quarter q; otherwise quarter q has rows 4 q to 4 q + 3
    float sum[NG][G];
#pragma unroll
    for (int r = 0; r < NG; r++)
#pragma unroll
        for (int g = 0; g < G; g++)
            sum[r][g] = FEW ? sum_quarters(acc[FEW ? r : 0][g]) : acc[0][g][r];
    if constexpr (KS) { // and the waves'
        float *sums = reinterpret_cast<float *>(lds.x); // [wave][four rows][group][lane]
        static_assert(sizeof(lds.x) >= 4 * (WG / 64) * NG * G * 64, "the waves' sums");
#pragma unroll
        for (int r = 0; r < NG; r++)
#pragma unroll
            for (int g = 0; g < G; g++)
                sums[((wave * NG + r) * G + g) * 64 + lane] = sum[r][g];
        __syncthreads();
        if (wave)
            return;
#pragma unroll
        for (int r = 0; r < NG; r++)
#pragma unroll
            for (int g = 0; g < G; g++)
                for (int w = 1; w < WG / 64; w++)
                    sum[r][g] += sums[((w * NG + r) * G + g) * 64 + lane];
    }
#pragma unroll
    for (int r = 0; r < NG; r++) {
        const int at = FEW ? 4 * r + row_of(q) : 4 * q + r;
        const int64_t pair = pair_at(a, pairs, tile, at);
#pragma unroll
        for (int g = 0; g < G; g++)
            if (at < rows && n0 + 16 * g < a.N)
                a.y[pair * a.N + n0 + 16 * g] = sum[r][g];
    }
}

// (Two waves a SIMD at the least: with 256 registers the matrix products' results are in vector registers; with more the
// compiler has them in accumulator registers, which costs a move each.)
template <int FMT, int G, bool WHOLE, bool KS> __global__ __launch_bounds__(WG, 2) void experts_tile_kernel(ExpertsArgs a, int chunks)
{
    __shared__ TileLds<FMT, G, KS> lds;
    const int chunk = blockIdx.x % chunks, tile = blockIdx.x / chunks;
    // without a plan the rows are those of one matrix product, one after another
    const int2 t = a.plan ? *reinterpret_cast<const int2 *>(a.plan + experts_tile_at(tile)) : make_int2(0, a.pairs - TR * tile);
    const int32_t *pairs = a.plan ? a.plan + experts_pairs_at(a.max_tiles, tile, TR) : nullptr;
    // place lane mod 16's activation row (a place without a pair reads some row, and is not stored)
    const uint32_t row16 = pair_at(a, pairs, tile, threadIdx.x % TR) / (uint32_t)a.per_row;
    const int rows = min(t.y, TR);
    if ((unsigned)t.x >= (unsigned)a.E || rows < 1)
        return; // no tile, or no plan of these pairs
    const uint8_t *W = a.W + t.x * a.expert_bytes;
    if (rows <= 4)
        tile_rows<FMT, G, WHOLE, KS, 1>(a, lds, W, chunk, rows, row16, pairs, tile);
    else if (FMT != LB_Q1_0 && rows <= 8) // (Q1_0, whose unpacking is most of a second turn: 64 experts of 1536 x 2048 18.7 and 20.3)
        tile_rows<FMT, G, WHOLE, KS, 2>(a, lds, W, chunk, rows, row16, pairs, tile);
    else
        tile_rows<FMT, G, WHOLE, KS, 4>(a, lds, W, chunk, rows, row16, pairs, tile);
}

template <int FMT, int G, bool KS> hipError_t tile_g(const ExpertsArgs &a, hipStream_t s)
{
    constexpr int WROWS = TileLds<FMT, G, KS>::WROWS;
    const int chunks = (a.N + WROWS - 1) / WROWS;
    const dim3 grid((unsigned)(a.max_tiles * chunks));
    if (a.K / F<FMT>::SW % 8 == 0)
        hipLaunchKernelGGL((experts_tile_kernel<FMT, G, true, KS>), grid, dim3(WG), 0, s, a, chunks);
    else
        hipLaunchKernelGGL((experts_tile_kernel<FMT, G, false, KS>), grid, dim3(WG), 0, s, a, chunks);
    return hipGetLastError();
}
// By the workgroups that 64 weight rows each would make.  Many: two groups of 16 rows a wave, which share what is read from
// LDS.  Under three a CU, one; under one and a half, the waves of a workgroup share its rows instead and divide K, so that
// all CUs have work.  Measured with Q4_0, 16 rows: 4096 x 12288 (64 workgroups) 24 us so with one group, 28 with two, 44
// with K whole; 12288 x 4096 (192) 17, 15, 16; 64 rows of 12288 x 4096 (768) 28 us with one group and K whole, 30 with two
// (Q1_0's chunk of K has work for two waves only, and nothing is gained.)
template <int FMT> hipError_t tile_fmt(const ExpertsArgs &a, hipStream_t s)
{
    const int64_t w = a.max_tiles * ((a.N + 63) / 64);
    if constexpr (FMT != LB_Q1_0) {
        if (w <= 64)
            return tile_g<FMT, 1, true>(a, s);
        if (w <= 384)
            return tile_g<FMT, 2, true>(a, s);
    }
    return w <= 768 ? tile_g<FMT, 1, false>(a, s) : tile_g<FMT, 2, false>(a, s);
}

} // namespace

hipError_t launch_experts_tile(int fmt, const ExpertsArgs &a, hipStream_t s)
{
    return fmt == LB_Q1_0 ? tile_fmt<LB_Q1_0>(a, s) : fmt == LB_Q2_0_G64 ? tile_fmt<LB_Q2_0_G64>(a, s) : tile_fmt<LB_Q4_0>(a, s);
}

} // namespace lb
