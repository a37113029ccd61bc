// Block tables and slot maps of a step, from the requests' lengths: which free pages every request's new
// tokens take, and where in the cache each token goes.  With P tokens a page, request b holding len_b tokens
// and bringing new_b needs ceil((len_b + new_b) / P) - ceil(len_b / P) pages; two running sums over the
// requests (of new tokens, of new pages) give every token its row and every page its place in the free list.
//
// A few KB are moved: the time is launches and dependent loads.  One workgroup computes both sums; where the
// step is small (a decode step, or a few prompts) the same workgroup also writes the tokens' slots, with the
// sums in LDS, so there is one launch.  A larger step's slots are written by a second launch over the whole
// chip, each token finding its request by bisection in the sums.  64 requests of one token: 4.9 us; 512 requests of
// 400 tokens: 3.8 + 6.5 us.
#include "serve_internal.h"

namespace lb {

constexpr int PLAN_WG = 1024;
constexpr int PLAN_SMALL_B = 2048; // requests whose sums are held in LDS (16 KB)

__device__ __forceinline__ int64_t ceil_div_pos(int64_t a, int shift) { return (a + ((int64_t)1 << shift) - 1) >> shift; }

// Last b in [0, n) with cu[b] <= t (cu[0] = 0 <= t < cu[n]): requests without tokens are passed over.  n is at most
// 2^30, so that lo + hi stays below 2^31.
template <class P> __device__ __forceinline__ int find_request(P cu, int n, int t)
{
    int lo = 0, hi = n; // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Token t's slot and position, or the padding's.  old: tokens held before this step; the i-th new page of the
// step is the i-th from the top of the free list.
template <class P>
__device__ __forceinline__ void plan_token(const PlanArgs &a, int shift, P cu, P cup, int64_t count, int64_t t)
{
    int64_t slot = -1;
    int pos = 0;
    if (t < cu[a.B]) {
        const int b = find_request(cu, (int)a.B, (int)t);
        const int old = a.kv_lens_out[b] - a.new_lens[b];
        pos = old + (int)(t - cu[b]);
        const int blk = pos >> shift, have = (int)ceil_div_pos(old, shift);
        const int page = blk < have ? a.block_table[b * a.table_stride + blk] : a.free_pages[count - 1 - (cup[b] + blk - have)];
        slot = (int64_t)page * ((int64_t)1 << shift) + (pos & ((1 << shift) - 1));
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
}

template <class P>
__device__ __forceinline__ void plan_page(const PlanArgs &a, int shift, P cup, int64_t count, int i)
{
    const int b = find_request(cup, (int)a.B, i);
    const int have = (int)ceil_div_pos(a.kv_lens_out[b] - a.new_lens[b], shift);
    a.block_table[b * a.table_stride + have + (i - cup[b])] = a.free_pages[count - 1 - i];
}

template <bool FILL> __global__ __launch_bounds__(PLAN_WG) void plan_kernel(PlanArgs a, int shift)
{
    __shared__ int64_t wsum[PLAN_WG / 64][2];
    __shared__ int s_bad;
    __shared__ int s_cu[FILL ? PLAN_SMALL_B + 1 : 1], s_cup[FILL ? PLAN_SMALL_B + 1 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0)
        s_bad = 0;
    const int64_t count = *a.free_count;
    const int64_t per = (a.B + PLAN_WG - 1) / PLAN_WG;
    const int64_t b0 = tid * per < a.B ? tid * per : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
    int64_t tok = 0, pg = 0;
    bool bad = false;
    for (int64_t b = b0; b < b1; b++) {
        const int64_t old = a.kv_lens[b], add = a.new_lens[b];
        if (old < 0 || add < 0) {
            bad = true;
            continue;
        }
        const int64_t want = ceil_div_pos(old + add, shift);
        // positions are 32-bit: a table that long would name over 2^31 tokens
        bad = bad || want > a.table_stride || old + add > INT32_MAX;
        tok += add;
        pg += want - ceil_div_pos(old, shift);
    }
    int64_t it = tok, ip = pg; // inclusive sums over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t ut = __shfl_up(it, d), up = __shfl_up(ip, d);
        if (lane >= d)
            it += ut, ip += up;
    }
    if (lane == 63)
        wsum[wave][0] = it, wsum[wave][1] = ip;
    __syncthreads();
    if (bad)
        s_bad = 1;
    int64_t bt = it - tok, bp = ip - pg, total_t = 0, total_p = 0;
    for (int w = 0; w < PLAN_WG / 64; w++) {
        if (w < wave)
            bt += wsum[w][0], bp += wsum[w][1];
        total_t += wsum[w][0], total_p += wsum[w][1];
    }
    __syncthreads();
    const int st = (total_p > count ? 1 : 0) | (total_t > a.max_tokens ? 2 : 0) | (s_bad ? 4 : 0) | (count < 0 || count > a.free_capacity ? 8 : 0);
    for (int64_t b = b0; b < b1; b++) {
        const int old = a.kv_lens[b], add = a.new_lens[b];
        const int ct = st ? 0 : (int)bt, cp = st ? 0 : (int)bp;
        a.cu_q[b] = ct;
        a.cu_pages[b] = cp;
        if constexpr (FILL)
            s_cu[b] = ct, s_cup[b] = cp;
        a.kv_lens_out[b] = st ? old : old + add;
        if (!st) {
            bt += add;
            bp += ceil_div_pos((int64_t)old + add, shift) - ceil_div_pos(old, shift);
        }
    }
    if (tid == 0) {
        const int ct = st ? 0 : (int)total_t, cp = st ? 0 : (int)total_p;
        a.cu_q[a.B] = ct;
        a.cu_pages[a.B] = cp;
        if constexpr (FILL)
            s_cu[a.B] = ct, s_cup[a.B] = cp;
        *a.free_count_out = (int)(count - cp);
        a.status[0] = st;
        a.status[1] = (int)(total_p < INT32_MAX ? total_p : INT32_MAX);
        a.status[2] = (int)(total_t < INT32_MAX ? total_t : INT32_MAX);
    }
    if constexpr (FILL) {
        __syncthreads();
        for (int64_t t = tid; t < a.max_tokens; t += PLAN_WG)
            plan_token(a, shift, s_cu, s_cup, count, t);
        for (int i = tid; i < s_cup[a.B]; i += PLAN_WG)
            plan_page(a, shift, s_cup, count, i);
    }
}

// The slots and table entries of a step whose sums plan_kernel<false> has left in cu_q and cu_pages.
__global__ __launch_bounds__(256) void plan_fill_kernel(PlanArgs a, int shift)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int pages = a.cu_pages[a.B];
    const int64_t count = (int64_t)*a.free_count_out + pages; // as it was before the step
    if (t < a.max_tokens)
        plan_token<const int32_t *>(a, shift, a.cu_q, a.cu_pages, count, t);
    if (t < pages) // every new page holds at least one new token, so there are no more of them than tokens
        plan_page<const int32_t *>(a, shift, a.cu_pages, count, (int)t);
}

static int log2_of(int64_t p)
{
    int s = 0;
    while (((int64_t)1 << s) < p)
        s++;
    return s;
}

hipError_t launch_kv_plan(const PlanArgs &a, hipStream_t s)
{
    const int shift = log2_of(a.page_tokens);
    // one launch up to 8192 tokens (eight a thread); beyond that the bisections of one workgroup take longer
    // than a second launch
    if (a.B <= PLAN_SMALL_B && a.max_tokens <= 8192) {
        hipLaunchKernelGGL(plan_kernel<true>, dim3(1), dim3(PLAN_WG), 0, s, a, shift);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_kernel<false>, dim3(1), dim3(PLAN_WG), 0, s, a, shift);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.max_tokens == 0)
        return e;
    hipLaunchKernelGGL(plan_fill_kernel, dim3((unsigned)((a.max_tokens + 255) / 256)), dim3(256), 0, s, a, shift);
    return hipGetLastError();
}

// --- release: the pages of finished requests go back on top of the free list, in request and block order.
// The first launch only reads lengths and count, the second changes them.  64 requests of up to 4000 tokens in pages of
// 16: 4.7 us for both (two launches: 3.7 is one alone); 4096 of up to 500: 18.5 us (24.5 with a workgroup each).

__device__ __forceinline__ int64_t held_pages(const ReleaseArgs &a, int shift, int64_t b)
{
    return a.done[b] && a.kv_lens[b] > 0 ? ceil_div_pos(a.kv_lens[b], shift) : 0;
}

struct Released {
    int64_t before; // pages of the requests before b
    int wrong;      // some length is beyond its table
};

// Every thread of the workgroup gets the result; a barrier has passed since the lengths were read.
__device__ __forceinline__ Released released_before(const ReleaseArgs &a, int shift, int64_t b)
{
    __shared__ int64_t ws[4];
    __shared__ int wr[4];
    int64_t v = 0;
    int wrong = 0;
    for (int64_t i = threadIdx.x; i < a.B; i += 256) {
        const int64_t n = held_pages(a, shift, i);
        wrong |= n > a.table_stride;
        v += i < b ? n : 0;
    }
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d), wrong |= __shfl_xor(wrong, d);
    if ((threadIdx.x & 63) == 0)
        ws[threadIdx.x >> 6] = v, wr[threadIdx.x >> 6] = wrong;
    __syncthreads();
    return {ws[0] + ws[1] + ws[2] + ws[3], wr[0] | wr[1] | wr[2] | wr[3]};
}

// A workgroup a request; beyond RELEASE_WGS requests, each takes a run of them, so that the sums of the requests
// before are read that many times and not once a request.
constexpr int64_t RELEASE_WGS = 1024;
__global__ __launch_bounds__(256) void release_copy_kernel(ReleaseArgs a, int shift, int per)
{
    const int64_t end = (int64_t)(blockIdx.x + 1) * per < a.B ? (int64_t)(blockIdx.x + 1) * per : a.B, count = *a.free_count;
    int64_t b = (int64_t)blockIdx.x * per, n = 0;
    for (; b < end && n == 0; b++) // the first one that gives something back
        n = held_pages(a, shift, b);
    if (n == 0 || count < 0)
        return;
    b--;
    int64_t at = count + released_before(a, shift, b).before;
    for (;;) {
        if (n > a.table_stride) // the release is refused in the end
            return;
        // what lies above the count is nobody's: a release that is refused has lost nothing by this
        for (int64_t i = threadIdx.x; i < n && at + i < a.free_capacity; i += 256)
            a.free_pages[at + i] = a.block_table[b * a.table_stride + i];
        if (++b >= end)
            return;
        at += n;
        n = held_pages(a, shift, b);
    }
}

__global__ __launch_bounds__(256) void release_end_kernel(ReleaseArgs a, int shift)
{
    const int64_t count = *a.free_count;
    const Released r = released_before(a, shift, a.B);
    const int st = (count < 0 || count + r.before > a.free_capacity ? 8 : 0) | (r.wrong ? 4 : 0);
    if (!st)
        for (int64_t i = threadIdx.x; i < a.B; i += 256)
            if (a.done[i])
                a.kv_lens[i] = 0;
    if (threadIdx.x == 0) {
        a.status[0] = st;
        a.status[1] = (int)(r.before < INT32_MAX ? r.before : INT32_MAX);
        if (!st)
            *a.free_count = (int)(count + r.before);
    }
}

hipError_t launch_kv_release(const ReleaseArgs &a, hipStream_t s)
{
    const int shift = log2_of(a.page_tokens);
    const int64_t per = (a.B + RELEASE_WGS - 1) / RELEASE_WGS;
    hipLaunchKernelGGL(release_copy_kernel, dim3((unsigned)((a.B + per - 1) / per)), dim3(256), 0, s, a, shift, (int)per);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(release_end_kernel, dim3(1), dim3(256), 0, s, a, shift);
    return hipGetLastError();
}

} // namespace lb
