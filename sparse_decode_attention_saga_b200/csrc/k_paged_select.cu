// Page selection of the sparse decode: the pages of each (sequence, key head)
// whose keys can reach the largest logits.
//
// A page's key bounds lo, hi (per dim the smallest and largest key) bound the
// logit of every key in it: q.k <= sum_d max(q_d lo_d, q_d hi_d) = q+ . hi +
// q- . lo, with q+ = max(q, 0) and q- = min(q, 0).  The score of a page is the
// largest such bound over the key head's query heads, compared in 64 bits (the
// lower index first where equal).
//
// Scores come from the tensor cores in bf16 with fp32 sums, 16 pages by 8
// query heads a tile, straight from global memory (each bound is used once,
// its fragment is 16 contiguous bytes per lane).  A score is off by less than
// E = 2^-14 max_h sum|q| max|bound| (at most 16 tile products of 17 addends,
// each cut at 2^-23 of the largest).  The row's last CTA then finds the n-th
// largest fp32 score to within E; pages further than 2E above are in, further
// below out, and only those between (a page or two, unless scores tie) are
// scored again in 64 bits.  One launch; bound by the read of the bounds and,
// in small batches, by the chain of the last CTA's steps.
#include <cuda_bf16.h>

#include "paged.h"
#include "saga_device.cuh"

namespace saga {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = kWarps * 16;  // pages scored by a CTA
constexpr int kPer = 16;             // pages a thread holds in registers in the search
constexpr int kRound = kThreads * kPer;
constexpr int kBand = 1024;  // pages scored again in shared memory
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ unsigned long long double_to_key(double x) {
    unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    if (u == 0x8000000000000000ull) u = 0ull;
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Sum over the block of up to three 10-bit counts per thread group packed in
// one word per warp (each warp's below 1024); all threads get the sums.
__device__ __forceinline__ int3 block_sum3(uint32_t packed, uint32_t (&buf)[2][kWarps], int& turn) {
    packed = __reduce_add_sync(kFull, packed);
    if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = packed;
    __syncthreads();
    int3 s = make_int3(0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint32_t v = buf[turn][w];
        s.x += v & 1023u, s.y += (v >> 10) & 1023u, s.z += v >> 20;
    }
    turn ^= 1;  // the other buffer next: one barrier a round
    return s;
}

__device__ __forceinline__ int block_sum(int n, uint32_t (&buf)[2][kWarps], int& turn) {
    n = __reduce_add_sync(kFull, n);
    if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = n;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += buf[turn][w];
    turn ^= 1;
    return s;
}

// Exclusive prefix of n over the block's threads, and the total.
__device__ __forceinline__ int block_prefix(int n, int& total, uint32_t (&buf)[2][kWarps], int& turn) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) buf[turn][warp] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int v = buf[turn][w];
        before += w < warp ? v : 0;
        total += v;
    }
    turn ^= 1;
    return before + incl - n;
}

template <int DK, int NT>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const PagedSelectArgs a) {
    constexpr int CH = DK / 32;  // 16-byte chunks of a bound row per lane
    __shared__ uint32_t sums[2][kWarps];
    __shared__ int band_page[kBand];
    __shared__ unsigned long long band_key[kBand];
    __shared__ int n_band, is_last;
    __shared__ float q_sum;
    pdl_wait();
    pdl_trigger();
    const PagedGeom& g = a.g;
    const int row = blockIdx.y, b = row / g.hk, kh = row % g.hk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    int len = a.seq_lens[b];
    if (len < 0 || len > g.max_pages * g.P) {
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        len = len < 0 ? 0 : g.max_pages * g.P;
    }
    const int np = (len + g.P - 1) / g.P;
    int32_t* sel = a.sel + static_cast<size_t>(row) * a.n_sel;
    if (np <= a.n_sel) {  // every page
        if (blockIdx.x == 0) {
            for (int p = threadIdx.x; p < np; p += kThreads) sel[p] = p;
            if (threadIdx.x == 0) a.sel_cnt[row] = np;
        }
        return;
    }
    const int chunks = (np + kChunk - 1) / kChunk;
    if (static_cast<int>(blockIdx.x) >= chunks) return;
    const int32_t* table = a.page_table + static_cast<size_t>(b) * g.max_pages;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * g.hq + kh * g.Gk) * DK;
    const __nv_bfloat16* boxes = reinterpret_cast<const __nv_bfloat16*>(a.bounds);
    float* scores = a.scores + static_cast<size_t>(row) * g.max_pages;
    const int p0 = blockIdx.x * kChunk + warp * 16;
    if (p0 < np) {
        uint4 lo[2][CH], hi[2][CH];
        bool bad[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int p = p0 + gq + 8 * r;
            const int phys = p < np ? table[p] : -1;
            const bool ok = phys >= 0 && phys < g.n_pages;
            bad[r] = !ok;
            if (!ok && p < np && tq == 0) raise_device_error(a.err, kErrBounds);
            const __nv_bfloat16* box = boxes + (static_cast<size_t>(ok ? phys : 0) * g.hk + kh) * 2 * DK;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                lo[r][c] = make_uint4(0u, 0u, 0u, 0u);
                hi[r][c] = lo[r][c];
                if (ok) {
                    lo[r][c] = __ldg(reinterpret_cast<const uint4*>(box) + tq + 4 * c);
                    hi[r][c] = __ldg(reinterpret_cast<const uint4*>(box + DK) + tq + 4 * c);
                }
            }
        }
        float d[NT][4] = {};
        __nv_bfloat162 big = __float2bfloat162_rn(0.f);
        const __nv_bfloat162 zero = big;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t l0[4] = {lo[0][c].x, lo[0][c].y, lo[0][c].z, lo[0][c].w}, l1[4] = {lo[1][c].x, lo[1][c].y, lo[1][c].z, lo[1][c].w};
            const uint32_t h0[4] = {hi[0][c].x, hi[0][c].y, hi[0][c].z, hi[0][c].w}, h1[4] = {hi[1][c].x, hi[1][c].y, hi[1][c].z, hi[1][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                big = __hmax2(big, __hmax2(__habs2(as_bf162(l0[i])), __habs2(as_bf162(l1[i]))));
                big = __hmax2(big, __hmax2(__habs2(as_bf162(h0[i])), __habs2(as_bf162(h1[i]))));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (8 * nt + gq < g.Gk) v = *(reinterpret_cast<const uint4*>(q + (8 * nt + gq) * DK) + tq + 4 * c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // a k-step of 16 dims: pairs 2s and 2s + 1 of each lane's chunk
                    mma_16816(d[nt], l0[2 * s], l1[2 * s], l0[2 * s + 1], l1[2 * s + 1],
                              as_u32(__hmin2(as_bf162(w[2 * s]), zero)), as_u32(__hmin2(as_bf162(w[2 * s + 1]), zero)));
                    mma_16816(d[nt], h0[2 * s], h1[2 * s], h0[2 * s + 1], h1[2 * s + 1],
                              as_u32(__hmax2(as_bf162(w[2 * s]), zero)), as_u32(__hmax2(as_bf162(w[2 * s + 1]), zero)));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float s = -kInf;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * nt + 2 * tq + i < g.Gk) s = fmaxf(s, d[nt][2 * r + i]);
            s = fmaxf(s, __shfl_xor_sync(kFull, s, 1));
            s = fmaxf(s, __shfl_xor_sync(kFull, s, 2));
            const int p = p0 + gq + 8 * r;
            if (tq == 0 && p < np) scores[p] = bad[r] ? -kInf : s;
        }
        const float m = warp_max(fmaxf(__low2float(big), __high2float(big)));
        if (lane == 0) atomicMax(a.row_max + row, __float_as_uint(m));  // not below 0: ordered as bits
    }
    // ---- the row's last CTA picks
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        is_last = atomicAdd(a.tickets + row, 1u) == static_cast<unsigned>(chunks - 1);
        n_band = 0;
        q_sum = 0.f;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    // sum |q| per head, the largest
    for (int h = warp; h < g.Gk; h += kWarps) {
        float s = 0.f;
#pragma unroll
        for (int i = lane; i < DK; i += 32) s += fabsf(__bfloat162float(q[h * DK + i]));
        s = warp_sum(s);
        if (lane == 0) atomicMax(reinterpret_cast<int*>(&q_sum), __float_as_int(s));
    }
    auto forced = [&](int p) { return p < a.n_first || p >= np - a.n_last; };
    const int want = a.n_sel - a.n_first - a.n_last;  // pages to pick beside the forced ones
    // this thread's pages: 16 in a row per round, their keys in registers (the only round, as a rule)
    const int rounds = (np + kRound - 1) / kRound;
    uint32_t key[kPer];
    auto load_keys = [&](int round) {
        const int at = round * kRound + threadIdx.x * kPer;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p = at + j;
            key[j] = p < np && !forced(p) ? float_to_key(__ldcg(scores + p)) : 0u;
        }
    };
    int turn = 0;
    load_keys(0);
    __syncthreads();
    const float margin = 2.f * 6.2e-5f * q_sum * __uint_as_float(__ldcg(a.row_max + row));  // 2E (2^-14 and its rounding)
    // ---- the want-th largest key, two bits at a time, until the interval is within E
    uint32_t t = 0;
    int sh = 30;
    for (;; sh -= 2) {
        const uint32_t c1 = t | (1u << sh), c2 = t | (2u << sh), c3 = t | (3u << sh);
        int3 n = make_int3(0, 0, 0);
        for (int r = 0; r < rounds; ++r) {
            if (rounds > 1) load_keys(r);
            uint32_t packed = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                packed += (key[j] >= c1 ? 1u : 0u) + (key[j] >= c2 ? 1u << 10 : 0u) + (key[j] >= c3 ? 1u << 20 : 0u);
            const int3 m = block_sum3(packed, sums, turn);
            n.x += m.x, n.y += m.y, n.z += m.z;
        }
        t = n.z >= want ? c3 : n.y >= want ? c2 : n.x >= want ? c1 : t;
        if (sh == 0) break;
        const float lo = key_to_float(t), hi = key_to_float(t | ((1u << sh) - 1u));
        if (hi - lo <= 0.5f * margin) break;
    }
    float cut_lo = key_to_float(t) - margin, cut_hi = key_to_float(t | ((1u << sh) - 1u)) + margin;
    // (no page but the forced ones is wanted: none above the cut)
    if (want == 0) cut_lo = cut_hi = kInf;
    // ---- the pages above the cut, and those the fp32 scores leave open
    int above = 0;
    for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load_keys(r);
        int n = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (key[j] == 0u) continue;
            const float s = key_to_float(key[j]);
            if (s > cut_hi) {
                ++n;
            } else if (s >= cut_lo) {
                const int at = atomicAdd(&n_band, 1);
                if (at < kBand) band_page[at] = r * kRound + threadIdx.x * kPer + j;
            }
        }
        above += block_sum(n, sums, turn);
    }
    __syncthreads();
    const int open = n_band, take = want - above;
    // ---- open pages in 64 bits; the taken ones' scores become +inf, the others' -inf
    auto exact_key = [&](int p) {  // by a warp
        const int phys = table[p];
        double best = -static_cast<double>(kInf);
        if (phys >= 0 && phys < g.n_pages) {
            const __nv_bfloat16* box = boxes + (static_cast<size_t>(phys) * g.hk + kh) * 2 * DK;
            for (int h = 0; h < g.Gk; ++h) {
                double s = 0.0;
#pragma unroll
                for (int i = lane; i < DK; i += 32) {
                    const float x = __bfloat162float(q[h * DK + i]);
                    s += static_cast<double>(fmaxf(x * __bfloat162float(box[i]), x * __bfloat162float(box[DK + i])));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                best = fmax(best, s);
            }
        }
        return double_to_key(best);
    };
    const bool all_open = open == take;
    if (!all_open && open <= kBand) {
        for (int i = warp; i < open; i += kWarps) {
            const unsigned long long k = exact_key(band_page[i]);
            if (lane == 0) band_key[i] = k;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < open; i += kThreads) {
            const unsigned long long k = band_key[i];
            const int p = band_page[i];
            int better = 0;
            for (int j = 0; j < open; ++j) better += band_key[j] > k || (band_key[j] == k && band_page[j] < p);
            scores[p] = better < take ? kInf : -kInf;
        }
        __syncthreads();
    } else if (!all_open) {  // many equal or nearly equal scores: their keys in the workspace, a search over 64 bits
        unsigned long long* keys = a.keys + static_cast<size_t>(row) * g.max_pages;
        auto is_open = [&](int p) {
            const float s = __ldcg(scores + p);
            return !forced(p) && s >= cut_lo && s <= cut_hi;
        };
        for (int p = warp; p < np; p += kWarps) {
            const unsigned long long k = is_open(p) ? exact_key(p) : 0ull;
            if (lane == 0) keys[p] = k;
        }
        __syncthreads();
        unsigned long long cut = 0;
        for (int bit = 63; bit >= 0; --bit) {
            int n = 0;
            for (int p = threadIdx.x; p < np; p += kThreads) n += keys[p] >= (cut | 1ull << bit);
            if (block_sum(n, sums, turn) >= take) cut |= 1ull << bit;
        }
        int n = 0;
        for (int p = threadIdx.x; p < np; p += kThreads) n += keys[p] > cut;
        int ties = take - block_sum(n, sums, turn);
        for (int at = 0; at < np; at += kThreads) {  // in order: the first ones of equal keys
            const int p = at + threadIdx.x;
            const unsigned long long k = p < np ? keys[p] : 0ull;
            int total;
            const int before = block_prefix(k == cut && k != 0ull, total, sums, turn);
            if (k != 0ull) scores[p] = k > cut || (k == cut && before < ties) ? kInf : -kInf;
            ties -= total;
        }
        __syncthreads();
    }
    // ---- the list, in order
    const float least = all_open ? cut_lo : cut_hi;
    int base = 0;
    for (int r = 0; r < rounds; ++r) {
        const int at = r * kRound + threadIdx.x * kPer;
        uint32_t in = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p = at + j;
            if (p >= np) continue;
            const float s = __ldcg(scores + p);
            if (forced(p) || (want > 0 && (all_open ? s >= least : s > least))) in |= 1u << j;
        }
        int total;
        int to = base + block_prefix(__popc(in), total, sums, turn);
        base += total;
        for (; in; in &= in - 1, ++to)
            if (to < a.n_sel) sel[to] = at + __ffs(in) - 1;
    }
    if (threadIdx.x == 0) {
        a.sel_cnt[row] = a.n_sel;
        a.tickets[row] = 0u;
        a.row_max[row] = 0u;
    }
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectArgs& a, cudaStream_t stream) {
    const PagedGeom& g = a.g;
    const dim3 grid((g.max_pages + kChunk - 1) / kChunk, g.b * g.hk);
    auto kern = g.Gk <= 8 ? (g.dk == 128  ? select_kernel<128, 1>
                             : g.dk == 64 ? select_kernel<64, 1>
                                          : select_kernel<32, 1>)
                          : (g.dk == 128  ? select_kernel<128, 2>
                             : g.dk == 64 ? select_kernel<64, 2>
                                          : select_kernel<32, 2>);
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace saga
