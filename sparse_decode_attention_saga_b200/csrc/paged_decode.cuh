// Attention of one query token per sequence over the paged 4-bit cache.
//
//   l_j = q . n^k_j s^k_j / sqrt(d),   out = sum_j softmax(l)_j n^v_j s^v_j
//
// over every cached position, or over the positions of the listed pages of
// each key head, in one pass with the running maximum and sum.
//
// Arithmetic.  Both products run on the tensor cores in fp16 with fp32 sums,
// positions as the tile's rows and query heads as its columns, and are exact
// up to the sums: a number's nibble is an fp16 integer (keys: the bare nibble
// u = n + 8 as a subnormal, u 2^-24, its -8 sum(q) put into the accumulator's
// start; values: 1024 + u less 1032), a query is shifted by a power of two
// per head into fp16's range (its 8 bits stay whole), and a probability times
// its row's scale goes in as two fp16 halves (22 bits), relative to the
// largest scale met so far.  The row scale of the keys multiplies the logit.
//
// Work.  A work row is a (sequence, key head, group of its value heads); its
// tile is 64 positions (64/page_size pages).  All rows' tiles, counted on the
// device from the lengths, are cut into equal contiguous ranges, one per
// warp, whatever the rows' lengths: a warp runs through its tiles with its
// own ring of bulk copies (one for the key block and one for the value blocks
// of a page), no barrier between warps.  A row that ends inside a warp's
// range is finished there; the pieces of a row that crosses ranges are merged
// per CTA in shared memory and across CTAs by the row's last one (a ticket,
// fixed order: results do not depend on timing).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.h"
#include "saga_device.cuh"

namespace saga {

namespace {

constexpr int kWarps = kPagedWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;  // positions per tile
constexpr int kMaxEntries = kTile / 16;
constexpr int kMaxStages = 4;
constexpr uint32_t kFull = 0xffffffffu;
// Shared memory for a CTA's rings when two CTAs share an SM, and when one has
// it (228 KB an SM; the static part is below 8 KB a CTA).
constexpr int kHalfRing = 104 * 1024, kWholeRing = 216 * 1024;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// D = A(16x16, row) * B(16x8, col) + C, fp16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// D += A(16x16, row) * B(16x8, col).
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// What a ring stage holds: its work row, whether the tile is the row's first
// (bit 0) or last (bit 1), and the valid positions of each of its pages.
struct StageMeta {
    int row, flags;
    int full;  // every position of every page is valid
    int pad;
    int valid[kMaxEntries];
};

template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

// A warp's unfinished piece of a row, for the merge.
struct Piece {
    int row;    // -1: none
    int flags;  // bit 0: holds the row's first tile, bit 1: its last
};

template <int DK, int DV, int CW, int NVU>
struct Shape {
    static constexpr int NT = CW == 4 ? (NVU + 1) / 2 : CW == 8 ? NVU : 2;  // tiles of 8 columns
    static constexpr int KS = DK / 16;                                       // k-steps of q.k
    static constexpr int WK = DK / 32;                                       // words of a key row per lane
    static constexpr int MT = DV / 16;                                       // tiles of 16 value dims
    static constexpr int ACC = CW == 16 ? 2 : NVU;                           // accumulators of MT tiles
    static constexpr int GRP = NT == 1 ? 4 : 2;  // groups of 16 positions between softmax updates
    static constexpr int stage_bytes = kTile * (DK / 2 + 2) + NVU * kTile * (DV / 2 + 2);
    // CTAs per SM: two where 128 registers a thread and half the shared memory (two stages) do
    static constexpr int MINB = (NT == 1 && 2 * kWarps * stage_bytes <= kHalfRing) ? 2 : 1;
};

struct Partition {
    int items, mult;  // items (sequences, or sequence x key head) and work rows of each
    long long T;      // tiles of all rows
    int C;            // CTAs that share them
};

// P: positions per page (a template parameter: every offset inside a tile is
// then an immediate).
template <int DK, int DV, int CW, int NVU, int P>
__global__ void __launch_bounds__(kThreads, (Shape<DK, DV, CW, NVU>::MINB))
    paged_decode_kernel(const PagedDecodeArgs a, const int stages, const int min_tiles) {
    using S = Shape<DK, DV, CW, NVU>;
    constexpr int NT = S::NT, KS = S::KS, WK = S::WK, MT = S::MT, ACC = S::ACC, GRP = S::GRP;
    extern __shared__ __align__(16) uint8_t ring[];  // [kWarps][stages][stage bytes]
    __shared__ uint64_t bars[kWarps][kMaxStages];
    __shared__ StageMeta metas[kWarps][kMaxStages];
    __shared__ long long prefix[kThreads + 1];
    __shared__ long long warp_sums[kWarps];
    __shared__ Piece pieces[2 * kWarps];
    __shared__ int group_begin[2 * kWarps + 1], n_groups, group_last[2 * kWarps];
    __shared__ int abort_flag;

    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    constexpr int EPT = kTile / P;                                        // pages per tile
    constexpr int KBLK = paged_block_bytes(P, DK), VBLK = paged_block_bytes(P, DV);
    const int nvg = g.nvk / NVU;
    const int heads = NVU * g.Gv;  // of a work row
    const int rec = g.dv + kPagedRecHeader;

    if (lane < stages) mbar_init(&bars[warp][lane], 1);
    if (threadIdx.x < 2 * kWarps) pieces[threadIdx.x].row = -1;
    if (threadIdx.x == 0) abort_flag = 0;
    fence_mbar_init();
    pdl_wait();
    pdl_trigger();

    // ---- the partition of all tiles, from the lengths
    auto seq_len = [&](int b) {
        const int len = a.seq_lens[b];
        if (len < 0 || len > g.max_pages * P) {
            if (lane == 0) raise_device_error(a.err, kErrBounds);
            return len < 0 ? 0 : g.max_pages * P;
        }
        return len;
    };
    auto item_entries = [&](int item) {  // pages of the item's rows
        if (!a.sel) return (seq_len(item) + P - 1) / P;
        const int n = a.sel_cnt[item];
        if (n < 0 || n > a.n_sel) {
            raise_device_error(a.err, kErrBounds);
            return 0;
        }
        return n;
    };
    auto tiles_of = [&](int entries) { return (entries + EPT - 1) / EPT; };
    Partition part;
    part.items = a.sel ? g.b * g.hk : g.b;
    part.mult = a.sel ? nvg : g.hk * nvg;
    const int chunk = (part.items + kThreads - 1) / kThreads;
    {
        long long n = 0;
        const int i0 = threadIdx.x * chunk, i1 = min(i0 + chunk, part.items);
        for (int i = i0; i < i1; ++i) n += static_cast<long long>(tiles_of(item_entries(i))) * part.mult;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        long long before = 0;
        part.T = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_sums[w];
            part.T += warp_sums[w];
        }
        prefix[threadIdx.x] = before + incl - n;
        if (threadIdx.x == 0) prefix[kThreads] = part.T;
        __syncthreads();
    }
    // rows without a position
    for (int i = blockIdx.x; i < part.items; i += gridDim.x)
        if (item_entries(i) == 0) {
            const int per = a.sel ? g.Gk : g.hq;
            for (int j = threadIdx.x; j < per * DV; j += kThreads) a.out[static_cast<size_t>(i) * per * DV + j] = 0.f;
        }
    const long long by_work = (part.T + min_tiles - 1) / min_tiles;
    part.C = static_cast<int>(by_work < gridDim.x ? by_work : gridDim.x);
    if (static_cast<int>(blockIdx.x) >= part.C) return;
    const long long cta0 = cta_tile_begin(part.T, part.C, blockIdx.x), cta1 = cta_tile_begin(part.T, part.C, blockIdx.x + 1);
    const long long w0 = cta0 + (cta1 - cta0) * warp / kWarps, w1 = cta0 + (cta1 - cta0) * (warp + 1) / kWarps;
    const int n_my = static_cast<int>(w1 - w0);

    uint8_t* my_ring = ring + static_cast<size_t>(warp) * stages * S::stage_bytes;
    constexpr int k_bytes = EPT * KBLK;

    // ---- producer state: where in which row the next tile to load is
    int p_item = 0, p_sub = 0, p_tile = 0, p_tiles = 0, p_entries = 0, p_len = 0, p_b = 0, p_kh = 0, p_vg = 0;
    int win_lo = 0, win_page = -1, win_phys = -1;  // this lane's entry of a window of 32
    auto enter_row = [&]() {
        const int r = p_item * part.mult + p_sub;  // = (b * hk + kh) * nvg + vg
        p_vg = r % nvg;
        p_kh = r / nvg % g.hk;
        p_b = r / nvg / g.hk;
        p_len = seq_len(p_b);
        win_lo = -32;
    };
    if (n_my > 0) {
        int c = 0;  // the chunk of items that holds tile w0: the last with prefix <= w0 (never an empty one)
        for (int step = kThreads / 2; step > 0; step >>= 1)
            if (prefix[c + step] <= w0) c += step;
        long long at = prefix[c];
        p_item = c * chunk;
        while (true) {
            p_entries = item_entries(p_item);
            p_tiles = tiles_of(p_entries);
            const long long n = static_cast<long long>(p_tiles) * part.mult;
            if (w0 < at + n) break;
            at += n;
            ++p_item;
        }
        p_sub = static_cast<int>((w0 - at) / p_tiles);
        p_tile = static_cast<int>((w0 - at) % p_tiles);
        enter_row();
    }
    auto load_window = [&]() {
        const int e = p_tile * EPT + lane;
        win_lo = p_tile * EPT;
        win_page = -1;
        win_phys = -1;
        if (e < p_entries) {
            const int np = (p_len + P - 1) / P;
            win_page = a.sel ? a.sel[(static_cast<size_t>(p_b) * g.hk + p_kh) * a.n_sel + e] : e;
            if (win_page >= 0 && win_page < np) win_phys = a.page_table[static_cast<size_t>(p_b) * g.max_pages + win_page];
            if (win_phys < 0 || win_phys >= g.n_pages) {
                raise_device_error(a.err, kErrBounds);
                win_phys = -1;
            }
        }
    };
    // loads the next tile into stage s
    auto produce = [&](int s) {
        const int e0 = p_tile * EPT;
        if (e0 < win_lo || e0 - win_lo >= 32) load_window();
        const int src = e0 - win_lo + lane;
        const int phys = __shfl_sync(kFull, win_phys, src & 31), page = __shfl_sync(kFull, win_page, src & 31);
        const bool mine = lane < EPT && phys >= 0;
        constexpr uint32_t v_bytes = NVU * VBLK;
        const int live = __popc(__ballot_sync(kFull, mine));
        const int valid = mine ? min(P, p_len - page * P) : 0;
        const bool full = __all_sync(kFull, lane >= EPT || valid == P);
        StageMeta& meta = metas[warp][s];
        if (lane == 0) {
            meta.row = p_item * part.mult + p_sub;
            meta.flags = (p_tile == 0 ? 1 : 0) | (p_tile == p_tiles - 1 ? 2 : 0);
            meta.full = full;
            mbar_arrive_expect_tx(&bars[warp][s], live * (KBLK + v_bytes));
        }
        if (lane < EPT) meta.valid[lane] = valid;
        __syncwarp();
        if (mine) {
            const uint32_t dst = smem_addr(my_ring + static_cast<size_t>(s) * S::stage_bytes);
            bulk_load(dst + lane * KBLK, a.k_pages + (static_cast<size_t>(phys) * g.hk + p_kh) * KBLK, KBLK,
                      &bars[warp][s]);
            bulk_load(dst + k_bytes + lane * v_bytes,
                      a.v_pages + (static_cast<size_t>(phys) * g.hv + p_kh * g.nvk + p_vg * NVU) * VBLK, v_bytes,
                      &bars[warp][s]);
        }
        if (++p_tile == p_tiles) {  // on to the next row that has a tile
            p_tile = 0;
            if (++p_sub == part.mult) {
                p_sub = 0;
                do {
                    ++p_item;
                    p_entries = p_item < part.items ? item_entries(p_item) : 1;
                } while (p_entries == 0);
                p_tiles = tiles_of(p_entries);
            }
            if (p_item < part.items) enter_row();
        }
    };

    // ---- consumer state
    int row = -1, seen = 0, expo = 0;  // seen: flags of the row's tiles so far; expo: biased exponent of the largest scale
    uint32_t qf[NT][KS][2];
    float c0[NT][2], colf[NT][2], m[NT][2], l[NT][2];
    float acc[ACC][MT][4];
    const int pos_a = (gq >> 1) + 4 * (gq & 1);  // position (of 16) of tile row gq; row gq + 8: 8 more

    // query head (of the work row) in column c of tile nt, or -1
    auto head_of = [&](int nt, int c) {
        const int j = CW == 4 ? 2 * nt + (c >> 2) : CW == 8 ? nt : 0;
        const int i = CW == 4 ? (c & 3) : CW == 8 ? c : 8 * nt + c;
        return j < NVU && i < g.Gv ? j * g.Gv + i : -1;
    };
    auto begin_row = [&](int r) {
        row = r;
        seen = 0;
        expo = 20;
        const int vg = r % nvg, bk = r / nvg;  // bk = b * hk + kh
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                 (static_cast<size_t>(bk) * g.nvk + vg * NVU) * g.Gv * DK;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = head_of(nt, gq);
            uint32_t raw[WK][4];
            float big = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (h >= 0) v = *reinterpret_cast<const uint4*>(q + h * DK + 8 * (tq * WK + w));
                raw[w][0] = v.x, raw[w][1] = v.y, raw[w][2] = v.z, raw[w][3] = v.w;
#pragma unroll
                for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf16_lo(raw[w][i])), fabsf(bf16_hi(raw[w][i]))));
            }
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
            // the head's largest query in [2^14, 2^15): 8 bits of any one down to 2^-27 of it stay whole
            const int e = big > 0.f ? ilogbf(big) : 0;
            const int sh = 14 - e;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = ldexpf(bf16_lo(raw[w][i]), sh);
                    x[2 * i + 1] = ldexpf(bf16_hi(raw[w][i]), sh);
                }
                // pair j holds dims j and j + 4 of the word; odd pairs meet nibbles 16 times their number
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float f = (j & 1) ? 0.0625f : 1.f;
                    const __half2 p = __floats2half2_rn(x[j] * f, x[j + 4] * f);
                    qf[nt][2 * w + (j >> 1)][j & 1] = half2_bits(p);
                    const float2 back = __half22float2(p);
                    sum += (back.x + back.y) * ((j & 1) ? 16.f : 1.f);
                }
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            const float start = -8.f * sum * 5.9604644775390625e-08f;  // 2^-24: a nibble as an fp16 subnormal
            const float f = ldexpf(kLog2e * rsqrtf(static_cast<float>(DK)), min(24 - sh, 126));
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // this lane's columns 2 tq + i
                c0[nt][i] = __shfl_sync(kFull, start, (2 * tq + i) * 4);
                colf[nt][i] = __shfl_sync(kFull, f, (2 * tq + i) * 4);
                m[nt][i] = -kInf;
                l[nt][i] = 0.f;
            }
        }
#pragma unroll
        for (int x = 0; x < ACC; ++x)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[x][mt][i] = 0.f;
    };
    // a value per column (lane's columns 2 tq + i of tile nt) as it is laid out beside accumulator x
    auto beside = [&](const float (&v)[NT][2], int x, float (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (CW == 4) f[i] = __shfl_sync(kFull, v[x >> 1][i], (lane & ~3) | (tq & 1) | ((x & 1) << 1));
            else f[i] = v[x][i];
        }
    };
    // o (times factor per column) of the current row to dst[head * stride + dim]
    auto write_o = [&](const float (&factor)[NT][2], float* dst, int stride) {
#pragma unroll
        for (int x = 0; x < ACC; ++x) {
            float f[2];
            beside(factor, x, f);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = acc[x][mt][i];
                    if (CW == 4) v += __shfl_xor_sync(kFull, v, 2);  // the two halves of the probabilities
                    const int col = CW == 4 ? 2 * (tq & 1) + (i & 1) : 2 * tq + (i & 1);
                    const int hl = CW == 16 ? 8 * x + col : col;  // head of the value head
                    const int dim = 8 * (gq + 8 * (mt >> 2)) + 2 * (mt & 3) + (i >> 1);
                    if (hl < g.Gv && (CW != 4 || tq < 2)) dst[((CW == 16 ? 0 : x) * g.Gv + hl) * stride + dim] = v * f[i & 1];
                }
        }
    };
    auto finish_row = [&](bool end_of_range) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], o);
        const float unit = pow2i(expo - 127 - 13);
        float f[NT][2];
        if (seen == 3) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) f[nt][i] = l[nt][i] > 0.f ? unit / l[nt][i] : 0.f;
            write_o(f, a.out + (static_cast<size_t>(row / nvg) * g.nvk + row % nvg * NVU) * g.Gv * DV, DV);
            return;
        }
        // an end of the range stays in this warp's ring (its copies are all in), an earlier piece goes to the workspace
        float* dst = end_of_range ? reinterpret_cast<float*>(my_ring)
                                  : a.firsts + (static_cast<size_t>(blockIdx.x) * kWarps + warp) * heads * rec;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[nt][i] = unit;
                const int h = head_of(nt, 2 * tq + i);
                if (gq == 0 && h >= 0) dst[h * rec] = m[nt][i], dst[h * rec + 1] = l[nt][i];
            }
        write_o(f, dst + kPagedRecHeader, rec);
        if (lane == 0) {
            Piece& p = pieces[2 * warp + (end_of_range ? 1 : 0)];
            p.row = row;
            p.flags = seen;
        }
    };

    // ---- GRP groups of 16 positions from group g0 of the stage's tile; full: every position of it is valid
    auto consume = [&](const uint8_t* buf, const StageMeta& meta, auto g0_, auto full_) {
        constexpr int g0 = decltype(g0_)::value;
        constexpr bool full = decltype(full_)::value;
        float x[GRP][NT][4];
        float sv[GRP][NT][2];
        uint32_t sv_max = 0;
#pragma unroll
        for (int gi = 0; gi < GRP; ++gi) {
            const int p0 = (g0 + gi) * 16, e = p0 / P, in = p0 % P;  // the group's page and its place in it
            const int valid = full ? 16 : meta.valid[e] - in;
            const uint8_t* kb = buf + e * KBLK;
            const uint8_t* krow = kb + (in + pos_a) * (DK / 2) + tq * (WK * 4);
            uint32_t w[2][WK];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t* src = krow + r * 8 * (DK / 2);
                if constexpr (WK == 1) {
                    w[r][0] = *reinterpret_cast<const uint32_t*>(src);
                } else if constexpr (WK == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    w[r][0] = v.x, w[r][1] = v.y;
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
                }
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint32_t lo = (k & 1) ? w[0][k / 2] >> 8 : w[0][k / 2], hi = (k & 1) ? w[1][k / 2] >> 8 : w[1][k / 2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float (&c)[4] = x[gi][nt];
                    mma_f16(x[gi][nt], lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u,
                            qf[nt][k][0], qf[nt][k][1], k ? c[0] : c0[nt][0], k ? c[1] : c0[nt][1],
                            k ? c[2] : c0[nt][0], k ? c[3] : c0[nt][1]);
                }
            }
            const __nv_bfloat16* ks = reinterpret_cast<const __nv_bfloat16*>(kb + P * (DK / 2)) + in + pos_a;
            const uint8_t* vb = buf + k_bytes + e * NVU * VBLK;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool ok = full || pos_a + 8 * r < valid;
                const float s = __bfloat162float(ks[8 * r]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float y = x[gi][nt][2 * r + i] * colf[nt][i] * s;
                        x[gi][nt][2 * r + i] = ok ? y : -kInf;
                    }
                    // the value head of this lane's columns
                    const int j = CW == 4 ? min(2 * nt + (tq >> 1), NVU - 1) : CW == 8 ? nt : 0;
                    const uint16_t raw = reinterpret_cast<const uint16_t*>(vb + j * VBLK + P * (DV / 2))[in + pos_a + 8 * r];
                    const uint32_t bits = ok ? raw : 0u;
                    sv_max = max(sv_max, bits & 0x7fffu);
                    sv[gi][nt][r] = __uint_as_float(bits << 16);
                }
            }
        }
        // running maxima; accumulators follow when one grows
        const int top = static_cast<int>(__reduce_max_sync(kFull, sv_max) >> 7);
        float mn[NT][2];
        bool grew = top > expo;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = -kInf;
#pragma unroll
                for (int gi = 0; gi < GRP; ++gi) v = fmaxf(v, fmaxf(x[gi][nt][i], x[gi][nt][2 + i]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
                mn[nt][i] = fmaxf(v, m[nt][i]);
                grew |= mn[nt][i] > m[nt][i];
            }
        if (__any_sync(kFull, grew)) {
            const int en = max(expo, top);
            const float shift = en - expo < 126 ? pow2i(expo - en) : 0.f;
            expo = en;
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f[nt][i] = mn[nt][i] == -kInf ? 1.f : exp2_approx(m[nt][i] - mn[nt][i]);
                    l[nt][i] *= f[nt][i];
                    m[nt][i] = mn[nt][i];
                    f[nt][i] *= shift;
                }
#pragma unroll
            for (int xx = 0; xx < ACC; ++xx) {
                float fx[2];
                beside(f, xx, fx);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[xx][mt][i] *= fx[i & 1];
            }
        }
        const float unit = pow2i(13 - (expo - 127) < 127 ? 13 - (expo - 127) : 127);
        float base[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) base[nt][i] = m[nt][i] == -kInf ? 0.f : m[nt][i];
#pragma unroll
        for (int gi = 0; gi < GRP; ++gi) {
            const int p0 = (g0 + gi) * 16, e = p0 / P, in = p0 % P;
            const uint8_t* vb = buf + k_bytes + e * NVU * VBLK;
            uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0f = exp2_approx(x[gi][nt][2 * r] - base[nt][0]);
                    const float p1f = exp2_approx(x[gi][nt][2 * r + 1] - base[nt][1]);
                    l[nt][0] += p0f;
                    l[nt][1] += p1f;
                    const float s = sv[gi][nt][r] * unit;
                    const float y0 = p0f * s, y1 = p1f * s;
                    const __half2 h = __floats2half2_rn(y0, y1);
                    const float2 back = __half22float2(h);
                    hi[nt][r] = half2_bits(h);
                    lo[nt][r] = half2_bits(__floats2half2_rn(y0 - back.x, y1 - back.y));
                }
            // probabilities with positions along the contraction: per value head (CW 4: both halves in one tile)
            [[maybe_unused]] uint32_t ph[ACC][2], pl[ACC][2];
            if constexpr (CW == 4) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool left = tq < 2;
                        const uint32_t got = __shfl_xor_sync(kFull, left ? lo[nt][r] : hi[nt][r], 2);
                        ph[2 * nt][r] = transpose8x8(left ? hi[nt][r] : got);
                        if (2 * nt + 1 < NVU) ph[2 * nt + 1 < NVU ? 2 * nt + 1 : 0][r] = transpose8x8(left ? got : lo[nt][r]);
                    }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) ph[nt][r] = transpose8x8(hi[nt][r]), pl[nt][r] = transpose8x8(lo[nt][r]);
            }
#pragma unroll
            for (int j = 0; j < NVU; ++j) {
#pragma unroll
                for (int half = 0; half < DV / 64; ++half) {
                    // word gq (+ 8) of rows tq, tq + 4, tq + 8, tq + 12
                    const uint32_t* row0 = reinterpret_cast<const uint32_t*>(vb + j * VBLK + (in + tq) * (DV / 2)) + gq + 8 * half;
                    const uint32_t u0 = row0[0], u1 = row0[4 * DV / 8], u2 = row0[8 * DV / 8], u3 = row0[12 * DV / 8];
#pragma unroll
                    for (int part_ = 0; part_ < 2; ++part_) {  // nibbles 0-3, 4-7 of the words
                        const uint32_t sel = part_ ? 0x7632u : 0x5410u;
                        const uint32_t a_ = __byte_perm(u0, u1, sel), b_ = __byte_perm(u2, u3, sel);
#pragma unroll
                        for (int by = 0; by < 2; ++by) {
                            const uint32_t av = by ? a_ >> 8 : a_, bv = by ? b_ >> 8 : b_;
                            const __half2 k1032 = __float2half2_rn(1032.f), k16 = __float2half2_rn(0.0625f), k72 = __float2half2_rn(-72.f);
                            const uint32_t f0 = half2_bits(__hsub2(bits_half2((av & 0x000f000fu) | 0x64006400u), k1032));
                            const uint32_t f1 = half2_bits(__hfma2(bits_half2((av & 0x00f000f0u) | 0x64006400u), k16, k72));
                            const uint32_t f2 = half2_bits(__hsub2(bits_half2((bv & 0x000f000fu) | 0x64006400u), k1032));
                            const uint32_t f3 = half2_bits(__hfma2(bits_half2((bv & 0x00f000f0u) | 0x64006400u), k16, k72));
                            const int mt = 4 * half + 2 * part_ + by;
                            if constexpr (CW == 4) {
                                mma_f16(acc[j][mt], f0, f1, f2, f3, ph[j][0], ph[j][1]);
                            } else if constexpr (CW == 8) {
                                mma_f16(acc[j][mt], f0, f1, f2, f3, ph[j][0], ph[j][1]);
                                mma_f16(acc[j][mt], f0, f1, f2, f3, pl[j][0], pl[j][1]);
                            } else {
#pragma unroll
                                for (int nt = 0; nt < 2; ++nt) {
                                    mma_f16(acc[nt][mt], f0, f1, f2, f3, ph[nt][0], ph[nt][1]);
                                    mma_f16(acc[nt][mt], f0, f1, f2, f3, pl[nt][0], pl[nt][1]);
                                }
                            }
                        }
                    }
                }
            }
        }
    };

    // ---- the warp's tiles
    int produced = 0, done = 0;
    uint32_t phase = 0;  // bit s: parity to wait for in stage s
    bool ok = true;
    for (; produced < stages && produced < n_my; ++produced) produce(produced);
    for (int s = 0; done < n_my; ++done) {
        if (!mbar_wait(&bars[warp][s], (phase >> s) & 1u, &abort_flag)) {
            ok = false;
            break;
        }
        phase ^= 1u << s;
        const StageMeta& meta = metas[warp][s];
        const int r = meta.row;
        if (r != row) {
            if (row >= 0) finish_row(false);
            begin_row(r);
        }
        seen |= meta.flags;
        const uint8_t* buf = my_ring + static_cast<size_t>(s) * S::stage_bytes;
        if (meta.full) {
            consume(buf, meta, Int<0>{}, Bool<true>{});
            if constexpr (GRP == 2) consume(buf, meta, Int<2>{}, Bool<true>{});
        } else {
            consume(buf, meta, Int<0>{}, Bool<false>{});
            if constexpr (GRP == 2) consume(buf, meta, Int<2>{}, Bool<false>{});
        }
        __syncwarp();
        if (produced < n_my) {
            produce(s);
            ++produced;
        }
        s = s + 1 == stages ? 0 : s + 1;
    }
    if (!ok) {  // a wait ran out: let the copies in flight land (each wait limited again), then leave
        if (lane == 0) raise_device_error(a.err, kErrTimeout);
        int given_up = 0;
        for (int i = done; i < produced; ++i) {
            const int s = i % stages;
            mbar_wait(&bars[warp][s], (phase >> s) & 1u, &given_up);
            phase ^= 1u << s;
        }
    } else if (row >= 0) {
        finish_row(true);
    }

    // ---- pieces of the CTA, row by row
    __syncthreads();
    if (abort_flag) return;
    if (threadIdx.x == 0) {
        int n = 0, prev = -2;
        for (int i = 0; i < 2 * kWarps; ++i) {
            if (pieces[i].row < 0) continue;
            if (pieces[i].row != prev) group_begin[n++] = i, prev = pieces[i].row;
        }
        group_begin[n] = 2 * kWarps;
        n_groups = n;
    }
    __syncthreads();
    auto piece_rec = [&](int i, int h) -> const float* {
        return (i & 1) ? reinterpret_cast<const float*>(ring + static_cast<size_t>(i >> 1) * stages * S::stage_bytes) + h * rec
                       : a.firsts + ((static_cast<size_t>(blockIdx.x) * kWarps + (i >> 1)) * heads + h) * rec;
    };
    // the row's first tile among all and its number of tiles
    auto locate = [&](int r, long long& tile0, int& tiles) {
        const int item = r / part.mult;
        const int c = item / chunk;
        tile0 = prefix[c];
        for (int i = c * chunk; i < item; ++i) tile0 += static_cast<long long>(tiles_of(item_entries(i))) * part.mult;
        tiles = tiles_of(item_entries(item));
        tile0 += static_cast<long long>(r % part.mult) * tiles;
    };
    auto row_out = [&](int r) { return a.out + (static_cast<size_t>(r / nvg) * g.nvk + r % nvg * NVU) * g.Gv * DV; };
    for (int w = warp; w < n_groups * heads; w += kWarps) {
        const int gi = w / heads, h = w % heads;
        const int i0 = group_begin[gi], i1 = group_begin[gi + 1], r = pieces[i0].row;
        float M = -kInf, L = 0.f, o[DV / 32] = {};
        int flags = 0;
        for (int i = i0; i < i1; ++i)
            if (pieces[i].row == r) {
                M = fmaxf(M, piece_rec(i, h)[0]);
                flags |= pieces[i].flags;
            }
        for (int i = i0; i < i1; ++i)
            if (pieces[i].row == r) {
                const float* src = piece_rec(i, h);
                const float f = src[0] == -kInf ? 0.f : exp2_approx(src[0] - M);
                L += f * src[1];
#pragma unroll
                for (int d = 0; d < DV / 32; ++d) o[d] += f * src[kPagedRecHeader + lane + 32 * d];
            }
        if (flags == 3) {
            float* dst = row_out(r) + h * DV;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d) dst[lane + 32 * d] = L > 0.f ? o[d] / L : 0.f;
        } else {
            long long tile0;
            int tiles;
            locate(r, tile0, tiles);
            float* dst = a.records + ((static_cast<size_t>(blockIdx.x) * 2 + (tile0 < cta0 ? 0 : 1)) * heads + h) * rec;
            if (lane == 0) dst[0] = M, dst[1] = L;
#pragma unroll
            for (int d = 0; d < DV / 32; ++d) dst[kPagedRecHeader + lane + 32 * d] = o[d];
        }
    }
    __threadfence();
    __syncthreads();
    // the last CTA of a row that crosses CTAs merges its records
    if (threadIdx.x < n_groups) {
        const int i0 = group_begin[threadIdx.x], i1 = group_begin[threadIdx.x + 1], r = pieces[i0].row;
        int flags = 0;
        for (int i = i0; i < i1; ++i) flags |= pieces[i].row == r ? pieces[i].flags : 0;
        int last = 0;
        if (flags != 3) {
            long long tile0;
            int tiles;
            locate(r, tile0, tiles);
            const int n = cta_of_tile(tile0 + tiles - 1, part.T, part.C) - cta_of_tile(tile0, part.T, part.C) + 1;
            last = atomicAdd(a.tickets + r, 1u) == static_cast<unsigned>(n - 1);
            if (last) a.tickets[r] = 0u;
        }
        group_last[threadIdx.x] = last;
    }
    __syncthreads();
    for (int gi = 0; gi < n_groups; ++gi) {
        if (!group_last[gi]) continue;
        __threadfence();
        const int r = pieces[group_begin[gi]].row;
        long long tile0;
        int tiles;
        locate(r, tile0, tiles);
        const int first = cta_of_tile(tile0, part.T, part.C), n = cta_of_tile(tile0 + tiles - 1, part.T, part.C) - first + 1;
        // 4 dims a lane, 32 / (DV / 4) records at a time
        constexpr int LD = DV / 4, RP = 32 / LD;
        const int sub = lane / LD, d4 = lane % LD;
        for (int h = warp; h < heads; h += kWarps) {
            auto record = [&](int i) {
                return a.records + ((static_cast<size_t>(first + i) * 2 + (i == 0 ? 1 : 0)) * heads + h) * rec;
            };
            float M = -kInf;
            for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(record(i)));
            M = warp_max(M);
            float L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = sub; i < n; i += RP) {
                const float* src = record(i);
                const float mm = __ldcg(src), ll = __ldcg(src + 1);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src + kPagedRecHeader) + d4);
                const float f = mm == -kInf ? 0.f : exp2_approx(mm - M);
                L += f * ll;
                o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
            }
#pragma unroll
            for (int s = LD; s < 32; s <<= 1) {
                L += __shfl_xor_sync(kFull, L, s);
                o.x += __shfl_xor_sync(kFull, o.x, s), o.y += __shfl_xor_sync(kFull, o.y, s);
                o.z += __shfl_xor_sync(kFull, o.z, s), o.w += __shfl_xor_sync(kFull, o.w, s);
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            if (sub == 0)
                reinterpret_cast<float4*>(row_out(r) + h * DV)[d4] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
    }
}

template <int DK, int DV, int CW, int NVU, int P>
cudaError_t run(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    using S = Shape<DK, DV, CW, NVU>;
    int stages = (S::MINB == 2 ? kHalfRing : kWholeRing) / (kWarps * S::stage_bytes);
    stages = stages > kMaxStages ? kMaxStages : stages;
    const int smem = kWarps * stages * S::stage_bytes;
    auto kern = paged_decode_kernel<DK, DV, CW, NVU, P>;
    const cudaError_t e = allow_dynamic_smem(kern, smem);
    if (e != cudaSuccess) return e;
    int ctas = sms * S::MINB;
    if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
    return launch_dependent(kern, dim3(ctas), dim3(kThreads), smem, stream, a, stages, kWarps);
}

template <int DK, int DV, int CW, int NVU>
cudaError_t run_page(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    if (a.g.P == 16) return run<DK, DV, CW, NVU, 16>(a, sms, stream);
    if (a.g.P == 32) return run<DK, DV, CW, NVU, 32>(a, sms, stream);
    return run<DK, DV, CW, NVU, 64>(a, sms, stream);
}

template <int DK, int DV>
cudaError_t run_shape(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    const PagedRowShape r = paged_row_shape(a.g);
    if (r.CW == 4) {
        if (r.NVU == 1) return run_page<DK, DV, 4, 1>(a, sms, stream);
        if constexpr (DV == 64)
            if (r.NVU == 4) return run_page<DK, DV, 4, 4>(a, sms, stream);
        return run_page<DK, DV, 4, 2>(a, sms, stream);
    }
    if (r.CW == 8) return r.NVU == 1 ? run_page<DK, DV, 8, 1>(a, sms, stream) : run_page<DK, DV, 8, 2>(a, sms, stream);
    return run_page<DK, DV, 16, 1>(a, sms, stream);
}

}  // namespace

}  // namespace saga
