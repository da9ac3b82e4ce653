// Page selection of the sparse decode: the pages of each (sequence, key head)
// whose keys can reach the largest logits.
//
// A page's key bounds lo, hi (per dim the smallest and largest key, as they were
// before rounding to 4 bits) bound the logit of each of those keys: q.k <=
// sum_d max(q_d lo_d, q_d hi_d) = q+ . hi + q- . lo, with q+ = max(q, 0) and
// q- = min(q, 0) (a published way to rank pages).  The rounded keys, which the
// decode reads, may pass it by half a step.  The score of a page is the
// largest such bound over the key head's query heads, compared in 64 bits (the
// lower index first where equal).
//
// Scores come from the tensor cores in bf16 with fp32 sums, 16 pages by 8
// query heads a tile, straight from global memory (each bound is used once,
// its fragment is 16 contiguous bytes per lane).  A score is off by less than
// E = 2^-14 max_h sum_d |q_d| max(|lo_d|, |hi_d|), which a third product gives
// (at most 16 tile products of 17 addends, each cut at 2^-23 of the largest).
// The row's last CTA finds the bin of the n-th largest fp32 score in a
// histogram over equal steps between the row's extremes (again between the bin's own while it is full), which leaves an
// interval [lo, hi] that the score lies in; pages 2E above it are in, pages 2E
// below out, and only those between (a few, unless scores tie) are scored
// again in 64 bits, as are all where fp32 does not hold the scores.  One launch.
// Measured: batch 16 x 128K (64 rows of 2048 pages of 64 positions, 34 MB of
// bounds) 17.7 us, of which the scores take 5.4 (6.3 TB/s) and the last CTAs' chain
// (ticket, extremes, histogram, cut, open pages, list) the rest; one row of 2048
// pages 12.6 us, the same chain.
#include <cuda_bf16.h>

#include "paged.h"
#include "paged_device.cuh"

namespace saga {

namespace {

constexpr int kPer = 16;     // pages a thread holds in registers
constexpr int kBand = 1024;  // pages scored again in shared memory
constexpr int kBins = 2048;
constexpr int kFewInBin = 24;  // pages in the threshold's bin that need no finer histogram
constexpr float kLeast = 1e-34f;  // above what products and sums below fp32's normal range are off by in a score
constexpr float kMost = 1e33f;    // margins below: scores (2^14 of it) and their sums are finite
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ unsigned long long double_to_key(double x) {
    unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    if (u == 0x8000000000000000ull) u = 0ull;
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Sum over the block (two buffers in turn: one barrier a call).
template <int kWarps>
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
template <int kWarps>
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

template <int DK, int NT, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) select_kernel(const PagedSelectArgs a, const int groups) {
    constexpr int CH = DK / 32;  // 16-byte chunks of a bound row per lane
    constexpr int kWarps = kThreads / 32, kChunk = kWarps * 16, kRound = kThreads * kPer;  // kChunk: pages a CTA scores at once
    extern __shared__ uint32_t words[];  // the picked pages' bits, then each word's rank
    __shared__ uint32_t sums[2][kWarps];
    __shared__ uint32_t bins[kBins];
    __shared__ int band_page[kBand];
    __shared__ unsigned long long band_key[kBand];
    __shared__ int n_band, is_last, the_bin, the_rank;
    __shared__ uint32_t bin_lo, bin_hi;
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
    const int chunks = (np + groups * kChunk - 1) / (groups * kChunk);
    if (static_cast<int>(blockIdx.x) >= chunks) return;
    const int32_t* table = a.page_table + static_cast<size_t>(b) * g.max_pages;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * g.hq + kh * g.Gk) * DK;
    const __nv_bfloat16* boxes = reinterpret_cast<const __nv_bfloat16*>(a.bounds);
    float* scores = a.scores + static_cast<size_t>(row) * g.max_pages;
    // what the pick starts from, cleared while the first loads are on their way
    const int n_words = (np + 31) / 32;
    uint32_t* ranks = words + n_words;
    for (int i = threadIdx.x; i < kBins; i += kThreads) bins[i] = 0u;
    for (int i = threadIdx.x; i < n_words; i += kThreads) words[i] = 0u;
    if (threadIdx.x == 0) n_band = 0, bin_lo = 0xffffffffu, bin_hi = 0u, the_bin = 0, the_rank = 1;
    // the queries' fragments, for hi, lo and the sum of magnitudes (k-steps of 16 dims: two to a lane's chunk)
    uint4 qraw[NT][CH];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            qraw[nt][c] = make_uint4(0u, 0u, 0u, 0u);
            if (8 * nt + gq < g.Gk) qraw[nt][c] = *(reinterpret_cast<const uint4*>(q + (8 * nt + gq) * DK) + tq + 4 * c);
        }
    float size = 0.f;  // the largest sum of |q| max(|lo|, |hi|) over this lane's pages and heads
    for (int group = 0; group < groups; ++group) {
        const int p0 = ((blockIdx.x * groups + group) * kWarps + warp) * 16;
        if (p0 >= np) break;
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
        float d[NT][4] = {}, z[NT][4] = {};
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        auto larger = [](uint32_t x, uint32_t y) { return as_u32(__hmax2(__habs2(as_bf162(x)), __habs2(as_bf162(y)))); };
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t l0[4] = {lo[0][c].x, lo[0][c].y, lo[0][c].z, lo[0][c].w}, l1[4] = {lo[1][c].x, lo[1][c].y, lo[1][c].z, lo[1][c].w};
            const uint32_t h0[4] = {hi[0][c].x, hi[0][c].y, hi[0][c].z, hi[0][c].w}, h1[4] = {hi[1][c].x, hi[1][c].y, hi[1][c].z, hi[1][c].w};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int i = 2 * s;
                const uint32_t m0 = larger(l0[i], h0[i]), m1 = larger(l1[i], h1[i]);
                const uint32_t m2 = larger(l0[i + 1], h0[i + 1]), m3 = larger(l1[i + 1], h1[i + 1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t q0 = s ? qraw[nt][c].z : qraw[nt][c].x, q1 = s ? qraw[nt][c].w : qraw[nt][c].y;
                    mma_16816(d[nt], l0[i], l1[i], l0[i + 1], l1[i + 1], as_u32(__hmin2(as_bf162(q0), zero)), as_u32(__hmin2(as_bf162(q1), zero)));
                    mma_16816(d[nt], h0[i], h1[i], h0[i + 1], h1[i + 1], as_u32(__hmax2(as_bf162(q0), zero)), as_u32(__hmax2(as_bf162(q1), zero)));
                    mma_16816(z[nt], m0, m1, m2, m3, q0 & 0x7fff7fffu, q1 & 0x7fff7fffu);
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) size = fmaxf(size, z[nt][i]);
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
    }
    size = warp_max(size);
    if (lane == 0 && size > 0.f) atomicMax(a.row_max + row, __float_as_uint(size));  // positive: ordered as bits
    // ---- the row's last CTA picks
    __syncthreads();
    if (threadIdx.x == 0) is_last = take_ticket(a.tickets + row) == static_cast<unsigned>(chunks - 1);
    __syncthreads();
    if (!is_last) return;
    auto forced = [&](int p) { return p < a.n_first || p >= np - a.n_last; };
    const int want = a.n_sel - a.n_first - a.n_last;  // pages to pick beside the forced ones
    // this thread's scores: every kThreads-th page, 16 in registers (all there are, as a rule); no page: -inf
    const int rounds = (np + kRound - 1) / kRound;
    float x[kPer];
    auto load = [&](int round) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p = round * kRound + j * kThreads + threadIdx.x;
            x[j] = p < np && !forced(p) ? __ldcg(scores + p) : -kInf;
        }
    };
    auto each = [&](auto&& f) {  // f(score, page) for the pages that are not forced
        for (int r = 0; r < rounds; ++r) {
            if (rounds > 1) load(r);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int p0j = r * kRound + j * kThreads;
                if (p0j >= np) break;
                const int p = p0j + threadIdx.x;
                if (p < np && !forced(p)) f(x[j], p);
            }
        }
    };
    int turn = 0;
    load(0);
    // 2E: 2^-14 of the row's largest size, itself within 2^-14, and what fp32's subnormals may lose
    const float margin = 2.f * 6.2e-5f * __uint_as_float(__ldcg(a.row_max + row)) + kLeast;
    float top = -kInf, low = -kInf;
    each([&](float s, int) {
        if (s > -kInf) top = fmaxf(top, s), low = fmaxf(low, -s);
    });
    top = warp_max(top), low = warp_max(low);
    if (lane == 0) sums[0][warp] = __float_as_uint(top), sums[1][warp] = __float_as_uint(low);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        top = fmaxf(top, __uint_as_float(sums[0][w])), low = fmaxf(low, __uint_as_float(sums[1][w]));
    low = -low;
    // ---- the interval [lo, hi] of the want-th largest
    float lo = -kInf, hi = kInf;
    int rank = want;  // of it among the scores in (.., top]
    for (int level = 0; level < 4 && want > 0; ++level) {
        if (level > 0) {
            for (int i = threadIdx.x; i < kBins; i += kThreads) bins[i] = 0u;
            if (threadIdx.x == 0) bin_lo = 0xffffffffu, bin_hi = 0u, the_bin = 0, the_rank = 1;
            __syncthreads();
        }
        const float step = top > low ? (kBins - 1) / (top - low) : 0.f;
        auto bin_of = [&](float s) { return static_cast<int>(fminf(fmaxf((s - low) * step, 0.f), kBins - 1.f)); };
        auto in = [&](float s) { return s >= lo && s <= hi; };  // of the level above's bin
        each([&](float s, int) {
            if (in(s)) atomicAdd(&bins[bin_of(s)], 1u);
        });
        __syncthreads();
        // bins from the top: thread i has the i-th four
        uint32_t n[kBins / kThreads], sum = 0;
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) sum += n[i] = bins[kBins - 1 - (threadIdx.x * (kBins / kThreads) + i)];
        int total;
        int before = block_prefix(sum, total, sums, turn);
#pragma unroll
        for (int i = 0; i < kBins / kThreads; ++i) {
            if (before < rank && before + static_cast<int>(n[i]) >= rank) {
                the_bin = kBins - 1 - (threadIdx.x * (kBins / kThreads) + i);
                the_rank = rank - before;
            }
            before += n[i];
        }
        __syncthreads();
        const int bin = the_bin;
        each([&](float s, int) {
            if (in(s) && bin_of(s) == bin) {
                atomicMin(&bin_lo, float_to_key(s));
                atomicMax(&bin_hi, float_to_key(s));
            }
        });
        __syncthreads();
        const bool few = bins[bin] <= kFewInBin;
        rank = the_rank;
        lo = key_to_float(bin_lo);
        hi = key_to_float(bin_hi);
        top = hi, low = lo;
        if (few || hi - lo <= 0.25f * margin) break;
        __syncthreads();  // the bins are cleared next
    }
    float cut_lo = lo - margin, cut_hi = hi + margin;
    if (!(margin < kMost)) cut_lo = -kInf, cut_hi = kInf;  // scores past fp32's end: every page is open
    if (want == 0) cut_lo = cut_hi = kInf;                 // the forced pages only
    auto is_open = [&](float s) { return !(s < cut_lo) && !(s > cut_hi); };  // (a score that is no number too)
    // ---- the pages above the cut and the forced ones, and those that the fp32 scores leave open
    __syncthreads();
    int above = 0;
    for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int p0j = r * kRound + j * kThreads;
            if (p0j >= np) break;
            const int p = p0j + threadIdx.x;
            const bool must = p < np && forced(p), over = p < np && !must && x[j] > cut_hi;
            const uint32_t bits = __ballot_sync(kFull, must || over);
            if (lane == 0 && p < np) words[p / 32] = bits;
            above += over;
            if (p < np && !must && is_open(x[j])) {
                const int at = atomicAdd(&n_band, 1);
                if (at < kBand) band_page[at] = p, band_key[at] = 0ull;
            }
        }
    }
    above = block_sum(above, sums, turn);
    auto set = [&](int p) { atomicOr(&words[p / 32], 1u << (p % 32)); };
    const int open = n_band, take = want - above;
    // ---- open pages in 64 bits
    auto partial = [&](int p, int h) {  // this lane's share of a head's score
        const int phys = table[p];
        if (phys < 0 || phys >= g.n_pages) return -static_cast<double>(kInf);
        const __nv_bfloat16* box = boxes + (static_cast<size_t>(phys) * g.hk + kh) * 2 * DK;
        double s = 0.0;
#pragma unroll
        for (int i = lane; i < DK; i += 32) {
            const float v = __bfloat162float(q[h * DK + i]);
            s += static_cast<double>(v) * __bfloat162float(box[v > 0.f ? DK + i : i]);  // exact: 16 bits
        }
        return s;
    };
    if (open == take) {
        each([&](float s, int p) {
            if (is_open(s)) set(p);
        });
    } else if (open <= kBand) {
        // a page and head per warp, four at a time (their loads and sums overlap)
        const int pairs = open * g.Gk;
        for (int i0 = warp; i0 < pairs; i0 += 4 * kWarps) {
            double s[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = min(i0 + u * kWarps, pairs - 1);
                s[u] = partial(band_page[i / g.Gk], i % g.Gk);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(kFull, s[u], o);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (lane == u && i0 + u * kWarps < pairs) atomicMax(&band_key[(i0 + u * kWarps) / g.Gk], double_to_key(s[u]));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < open; i += kThreads) {
            const unsigned long long k = band_key[i];
            const int p = band_page[i];
            int better = 0;
            for (int j = 0; j < open; ++j) better += band_key[j] > k || (band_key[j] == k && band_page[j] < p);
            if (better < take) set(p);
        }
    } else {  // many equal or nearly equal scores: their keys in the workspace, a search over 64 bits
        unsigned long long* keys = a.keys + static_cast<size_t>(row) * g.max_pages;
        for (int p = warp; p < np; p += kWarps) {
            const float s = __ldcg(scores + p);
            unsigned long long k = 0ull;
            if (!forced(p) && is_open(s))
                for (int h = 0; h < g.Gk; ++h) {
                    double v = partial(p, h);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
                    k = max(k, double_to_key(v));
                }
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
            if (k != 0ull && (k > cut || (k == cut && before < ties))) set(p);
            ties -= total;
        }
    }
    __syncthreads();
    // ---- the list, in order: each word's rank, then every picked page at its own
    int picked = 0;
    for (int w0 = 0; w0 < n_words; w0 += kThreads) {
        const int w = w0 + threadIdx.x;
        int total;
        const int before = block_prefix(w < n_words ? __popc(words[w]) : 0, total, sums, turn);
        if (w < n_words) ranks[w] = picked + before;
        picked += total;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < np; p += kThreads) {
        const uint32_t word = words[p / 32];
        const int to = ranks[p / 32] + __popc(word & lanemask_lt());
        if ((word >> (p % 32) & 1u) && to < a.n_sel) sel[to] = p;
    }
    if (threadIdx.x == 0) {
        a.sel_cnt[row] = min(picked, a.n_sel);  // (n_sel, unless scores are no numbers)
        a.tickets[row] = 0u;
        a.row_max[row] = 0u;
    }
}

template <int kThreads>
cudaError_t launch(const PagedSelectArgs& a, int ctas, cudaStream_t stream) {
    const PagedGeom& g = a.g;
    // 16-page groups per warp: one wave of CTAs where the batch needs no more
    constexpr int kChunk = kThreads / 2;
    const int rows = g.b * g.hk, chunks = (g.max_pages + kChunk - 1) / kChunk;
    int groups = static_cast<int>((static_cast<long long>(chunks) * rows + ctas - 1) / ctas);
    groups = groups < 1 ? 1 : groups > 4 ? 4 : groups;
    const dim3 grid((chunks + groups - 1) / groups, rows);
    auto kern = g.Gk <= 8 ? (g.dk == 128  ? select_kernel<128, 1, kThreads>
                             : g.dk == 64 ? select_kernel<64, 1, kThreads>
                                          : select_kernel<32, 1, kThreads>)
                          : (g.dk == 128  ? select_kernel<128, 2, kThreads>
                             : g.dk == 64 ? select_kernel<64, 2, kThreads>
                                          : select_kernel<32, 2, kThreads>);
    const int smem = (g.max_pages + 31) / 32 * 8;  // at most 64 KB (kPagedMaxSelectPages)
    const cudaError_t e = allow_dynamic_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, grid, dim3(kThreads), smem, stream, a, groups);
}

}  // namespace

cudaError_t launch_paged_select(const PagedSelectArgs& a, int sms, cudaStream_t stream) {
    // More rows than SMs: their last CTAs' chains queue up, so smaller CTAs, two or three to an SM (1600 rows of
    // 157 pages 88 -> 51 us, 240 rows of 625 24.2 -> 21.5, with 64 rows of 2048 17.6 -> 19.6).
    return a.g.b * a.g.hk > sms ? launch<256>(a, 2 * sms, stream) : launch<512>(a, sms, stream);
}

}  // namespace saga
