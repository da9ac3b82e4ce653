// Page selection of the sparse decode: the pages of each (sequence, key head)
// whose keys can reach the largest logits.
//
// A page's key bounds lo, hi (per dim the smallest and largest key) bound the
// logit of every key in it: q.k <= sum_d max(q_d lo_d, q_d hi_d).  The score
// of a page is the largest such bound over the key head's query heads, in 64
// bits (products of bf16 values are exact in 32, sums of at most 128 of them
// nearly so in 64: pages that differ are told apart, equal pages tie and the
// lower index goes first).  The first n_first and the last n_last pages are
// always taken.
#include <cuda_bf16.h>

#include "paged.h"
#include "saga_device.cuh"

namespace saga {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kPickThreads = 512;

__device__ __forceinline__ int pages_of(const PagedGeom& g, const int32_t* seq_lens, int b, uint32_t* err) {
    int len = seq_lens[b];
    if (len < 0 || len > g.max_pages * g.P) {
        if (threadIdx.x == 0) raise_device_error(err, kErrBounds);
        len = len < 0 ? 0 : g.max_pages * g.P;
    }
    return (len + g.P - 1) / g.P;
}

// One warp per page.
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const PagedSelectArgs a) {
    pdl_wait();
    pdl_trigger();
    const PagedGeom& g = a.g;
    const int row = blockIdx.y, b = row / g.hk, kh = row % g.hk;
    const int lane = threadIdx.x & 31;
    const int page = blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
    const int np = pages_of(g, a.seq_lens, b, a.err);
    if (page >= np || np <= a.n_sel) return;
    const int phys = a.page_table[static_cast<size_t>(b) * g.max_pages + page];
    double best = -static_cast<double>(kInf);
    if (phys >= 0 && phys < g.n_pages) {
        const __nv_bfloat16* box = reinterpret_cast<const __nv_bfloat16*>(a.bounds) + (static_cast<size_t>(phys) * g.hk + kh) * 2 * g.dk;
        for (int h = 0; h < g.Gk; ++h) {
            const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * g.hq + kh * g.Gk + h) * g.dk;
            double s = 0.0;
            for (int d = lane; d < g.dk; d += 32) {
                const float x = __bfloat162float(q[d]);
                s += static_cast<double>(fmaxf(x * __bfloat162float(box[d]), x * __bfloat162float(box[g.dk + d])));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            best = fmax(best, s);
        }
    } else if (lane == 0) {
        raise_device_error(a.err, kErrBounds);
    }
    if (lane == 0) a.scores[static_cast<size_t>(row) * g.max_pages + page] = best;
}

__device__ __forceinline__ unsigned long long double_to_key(double x) {
    unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    if (u == 0x8000000000000000ull) u = 0ull;
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// One CTA per row: the n_sel-th largest key bit by bit, then the pages at or
// above it in order (of the equal ones the lowest indices).
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const PagedSelectArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int warp_n[kPickThreads / 32], warp_e[kPickThreads / 32];
    const PagedGeom& g = a.g;
    const int row = blockIdx.x, b = row / g.hk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int np = pages_of(g, a.seq_lens, b, a.err);
    int32_t* sel = a.sel + static_cast<size_t>(row) * a.n_sel;
    if (np <= a.n_sel) {
        for (int p = threadIdx.x; p < np; p += kPickThreads) sel[p] = p;
        if (threadIdx.x == 0) a.sel_cnt[row] = np;
        return;
    }
    const double* scores = a.scores + static_cast<size_t>(row) * g.max_pages;
    auto key = [&](int p) {
        return p < a.n_first || p >= np - a.n_last ? ~0ull : double_to_key(scores[p]);
    };
    unsigned long long t = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long c = t | (1ull << bit);
        int n = 0;
        for (int p = threadIdx.x; p < np; p += kPickThreads) n += key(p) >= c;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) warp_n[warp] = n;
        __syncthreads();
        n = 0;
        for (int i = 0; i < kPickThreads / 32; ++i) n += warp_n[i];
        __syncthreads();
        if (n >= a.n_sel) t = c;
    }
    int above = 0;
    for (int p = threadIdx.x; p < np; p += kPickThreads) above += key(p) > t;
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0) warp_n[warp] = above;
    __syncthreads();
    above = 0;
    for (int i = 0; i < kPickThreads / 32; ++i) above += warp_n[i];
    __syncthreads();
    const int ties = a.n_sel - above;  // pages equal to the threshold that fit
    int base = 0, base_e = 0;
    for (int p0 = 0; p0 < np; p0 += kPickThreads) {
        const int p = p0 + threadIdx.x;
        const unsigned long long k = p < np ? key(p) : 0ull;
        const bool gt = p < np && k > t, eq = p < np && k == t;
        const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_n[warp] = __popc(bg), warp_e[warp] = __popc(be);
        __syncthreads();
        int ng = base, ne = base_e;
        for (int i = 0; i < warp; ++i) ng += warp_n[i], ne += warp_e[i];
        for (int i = 0; i < kPickThreads / 32; ++i) base += warp_n[i], base_e += warp_e[i];
        __syncthreads();
        ng += __popc(bg & lanemask_lt());
        ne += __popc(be & lanemask_lt());
        if (gt || (eq && ne < ties)) sel[ng + min(ne, ties)] = p;
    }
    if (threadIdx.x == 0) a.sel_cnt[row] = a.n_sel;
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectArgs& a, int sms, cudaStream_t stream) {
    (void)sms;
    const int rows = a.g.b * a.g.hk;
    const int per = kScoreThreads / 32;
    const cudaError_t e = launch_dependent(score_kernel, dim3((a.g.max_pages + per - 1) / per, rows),
                                           dim3(kScoreThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(pick_kernel, dim3(rows), dim3(kPickThreads), 0, stream, a);
}

}  // namespace saga
