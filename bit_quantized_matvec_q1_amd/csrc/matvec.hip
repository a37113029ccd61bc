// Batch-1 decode products: the formats that share matvec_tile.h's kernels (Q1_0, Q2_0_g64 and planar ternary here,
// Q4_0 in q4.hip), and the dispatch to those with kernels of their own (Q8_0, base-3).
#include "matvec_tile.h"

namespace lb {

int matvec_config(int fmt, int64_t K)
{
    if (fmt == LB_Q8_0)
        return q8_config(K);
    if (fmt == LB_TERNARY_B3)
        return b3_config(K);
    if (K <= 0 || K % sw_of(fmt))
        return -1;
    return pick_cfg(fmt, K / sw_of(fmt));
}

bool matvec_supported_k(int fmt, int64_t K) { return matvec_config(fmt, K) >= 0; }

bool matvec_config_full(int fmt, int cfg, int64_t K)
{
    if (fmt == LB_Q8_0 || fmt == LB_TERNARY_B3)
        return true; // one kernel per configuration; idle lanes are clamped inside it
    return (int64_t)kCfgs[cfg].L * kCfgs[cfg].S == K / sw_of(fmt);
}

int matvec_config_rows_per_iter(int fmt, int cfg)
{
    if (fmt == LB_Q8_0)
        return q8_rows_per_iter(cfg);
    if (fmt == LB_TERNARY_B3)
        return b3_rows_per_iter(cfg);
    return (64 / kCfgs[cfg].L) * (WG / 64);
}

int matvec_stage_bytes(int fmt, int64_t K)
{
    if (fmt == LB_Q8_0)
        return (int)q8_stage_bytes(K);
    if (fmt == LB_TERNARY_B3)
        return (int)b3_stage_bytes(K);
    return (int)((K / sw_of(fmt)) * rec_of(fmt) * 4);
}

hipError_t launch_matvec(int fmt, const uint8_t *W, int64_t N, int64_t K, float w_scale, const int8_t *xq,
                         const void *xscale, float *y, int32_t *sums, hipStream_t s)
{
    if (fmt == LB_Q8_0)
        return launch_q8(W, N, K, xq, static_cast<const uint16_t *>(xscale), y, sums, s);
    if (fmt == LB_TERNARY_B3)
        return launch_b3(W, N, K, w_scale, xq, static_cast<const float *>(xscale), y, sums, s);
    const int cfg = matvec_config(fmt, K);
    if (cfg < 0)
        return hipErrorInvalidValue;
    // enough workgroups to cover the device when the product allows it, whole iterations per tile
    const int rpi = matvec_config_rows_per_iter(fmt, cfg);
    int64_t tile = (N + 1023) / 1024;
    tile = ((tile + rpi - 1) / rpi) * rpi;
    if (tile < rpi)
        tile = rpi;
    if (tile > 32 * rpi)
        tile = 32 * rpi;
    if (fmt == LB_Q4_0)
        return launch_q4(cfg, W, N, K, xq, static_cast<const uint16_t *>(xscale), y, sums, (int)tile, s);
    const bool emit = sums != nullptr;
    const int n = (int)N, k = (int)K, t = (int)tile;
    switch (fmt) {
    case LB_Q1_0:
        return emit ? launch_single<LB_Q1_0, true>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s)
                    : launch_single<LB_Q1_0, false>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s);
    case LB_Q2_0_G64:
        return emit ? launch_single<LB_Q2_0_G64, true>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s)
                    : launch_single<LB_Q2_0_G64, false>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s);
    case LB_TERNARY_PLANAR:
        return emit ? launch_single<LB_TERNARY_PLANAR, true>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s)
                    : launch_single<LB_TERNARY_PLANAR, false>(cfg, W, n, k, w_scale, xq, xscale, y, sums, t, s);
    }
    return hipErrorInvalidValue;
}

int matvec_batched_blocks_per_cu(int fmt, int cfg, bool full, bool qin, size_t lds_bytes)
{
    switch (fmt) {
    case LB_Q1_0:
        return blocks_per_cu_fmt<LB_Q1_0>(cfg, full, qin, lds_bytes);
    case LB_Q2_0_G64:
        return blocks_per_cu_fmt<LB_Q2_0_G64>(cfg, full, qin, lds_bytes);
    case LB_TERNARY_PLANAR:
        return blocks_per_cu_fmt<LB_TERNARY_PLANAR>(cfg, full, false, lds_bytes);
    case LB_Q4_0:
        return q4_blocks_per_cu(cfg, full, qin, lds_bytes);
    case LB_Q8_0:
        return q8_blocks_per_cu(cfg, lds_bytes);
    case LB_TERNARY_B3:
        return b3_blocks_per_cu(cfg, lds_bytes);
    }
    return 1;
}

hipError_t launch_matvec_batched(const BatchGroup &g, hipStream_t s, size_t lds_bytes)
{
    switch (g.fmt) {
    case LB_Q1_0:
        return launch_batched_fmt<LB_Q1_0>(g, s, lds_bytes);
    case LB_Q2_0_G64:
        return launch_batched_fmt<LB_Q2_0_G64>(g, s, lds_bytes);
    case LB_TERNARY_PLANAR:
        return launch_batched_fmt<LB_TERNARY_PLANAR>(g, s, lds_bytes);
    case LB_Q4_0:
        return launch_q4_batched(g, lds_bytes, s);
    case LB_Q8_0:
        return launch_q8_batched(g, lds_bytes, s);
    case LB_TERNARY_B3:
        return launch_b3_batched(g, lds_bytes, s);
    }
    return hipErrorInvalidValue;
}

} // namespace lb
