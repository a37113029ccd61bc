// Q4_0 weights (32 signed 4-bit weights and a binary16 scale, 18 bytes) x q8_0 activations: the instances of
// matvec_tile.h's kernels for this format, in a translation unit of their own so that they compile beside the others.
// A Q4_0 block is one 16-byte code record, as a Q2_0_g64 or Q1_0 block is, so configurations, tiles and the work lists
// are theirs.
//
// Bound by HBM as they are: 151669 x 4096 (349 MB) takes 51.5 us, 6.8 TB/s of the 7.1 that a plain read reaches; 12288 x
// 4096 (28 MB) 6.7 us and 640 x 2560 3.1 us, of which some 3 us are a launch's.
#include "matvec_tile.h"

namespace lb {

hipError_t launch_q4(int cfg, const uint8_t *W, int64_t N, int64_t K, const int8_t *xq, const uint16_t *xs, float *y, int32_t *sums,
                     int tile_rows, hipStream_t s)
{
    return sums ? launch_single<LB_Q4_0, true>(cfg, W, (int)N, (int)K, 1.0f, xq, xs, y, sums, tile_rows, s)
                : launch_single<LB_Q4_0, false>(cfg, W, (int)N, (int)K, 1.0f, xq, xs, y, sums, tile_rows, s);
}

hipError_t launch_q4_batched(const BatchGroup &g, size_t lds, hipStream_t s) { return launch_batched_fmt<LB_Q4_0>(g, s, lds); }

int q4_blocks_per_cu(int cfg, bool full, bool qin, size_t lds) { return blocks_per_cu_fmt<LB_Q4_0>(cfg, full, qin, lds); }

} // namespace lb
