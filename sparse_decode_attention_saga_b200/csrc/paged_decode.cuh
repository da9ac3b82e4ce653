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
// its row's scale goes in as two fp16 halves (22 bits, none below 2^-31 of the
// largest such product of its query head so far: neither a row of little weight
// nor another head takes bits away).  The row scale of the keys multiplies the logit.
// A new reference for the exponentials (a whole number: rescaling and merging
// are exact) is taken only when a product nears fp16's end or the sum of the
// exponentials fp32's.  The contraction's order is free, so the nibbles of a word pair
// up as they lie (dims of the keys, queries laid out alike), and the values,
// which need pairs of positions, are transposed byte-wise on the way out of
// shared memory.
//
// Work.  A work row is a (sequence, key head, group of its value heads); its
// tile is 64 positions (64/page_size pages).  All rows' tiles, counted on the
// device from the lengths, are cut into equal contiguous ranges, one per
// warp, whatever the rows' lengths: a warp runs through its tiles with its
// own ring of bulk copies (one for the key block and one for the value blocks
// of a page).  A row that ends inside a warp's range is finished there; the
// pieces of a row that crosses ranges are merged per CTA in shared memory and
// across CTAs by the row's last one (a ticket, fixed order: results do not
// depend on timing).  One CTA has an SM to itself, and its warps keep within
// a round of four tiles of one another (a barrier that a warp arrives at after
// a round and waits for a round later): with two CTAs and no such pace the
// SM's older warps ran first and left the younger ones to finish alone, at
// half the issue rate (batch 16 x 128K: CTAs ended at 150 and at 215 us).
//
// Measured (32/4/8 heads of 64, batch 16 x 128K, 856 MB): 174 us, 4.9 TB/s, 0.75
// of the copy rate, at 1965 MHz; 195 us when repeated until the power cap holds
// the clock at 1750 MHz (time goes by the clock).  864 warp instructions a tile
// (384 on the half-rate integer pipe, unpacking nibbles): 56 % of the issue
// slots, 50 % of that pipe, tensor pipe 21 %, DRAM reads 1.00 times the cache.
// None is full: what is left is latency with the four warps a scheduler that the
// registers allow (of the 7.4 cycles from one issue of a warp to the next, 1.6
// wait for a result of fixed latency, 1.1 for another warp's turn, 1.0 for a
// pipe, 0.7 at barriers, 0.6 for memory).
// Batch 1 at 8K: 14.1 us, the chain of lengths, table, copies, one tile, two
// merges; most of it waits at barriers (8.6 of 20) for warps that fetch the body's
// instructions for the first time (4.4).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.h"
#include "paged_device.cuh"

namespace saga {

namespace {

constexpr int kTile = 64;  // positions per tile
constexpr int kMaxStages = 4;
constexpr uint32_t kFull = 0xffffffffu;
// Shared memory for a CTA's rings (227 KB at most; the static part is below 10 KB).
constexpr int kRingBytes = 216 * 1024;
// Tiles of a CTA at least: fewer CTAs than SMs where there is less work, as each adds a record to merge
// (batch 1 at 8K: 14.9 us at 16, 14.2 at 8, 14.8 at 4).
constexpr int kMinTiles = 8;
constexpr int kRound = 4;  // tiles between two arrivals at the pace barrier
// A probability times its row's scale is 2^6 to 2^kUnit where it sets its
// column's reference: room for others to pass it before a new one is taken,
// when a product reaches 2^15.
constexpr int kUnit = 8;
// Biased exponent that a scale is taken for at least (2^-45) where a reference is
// set: exponentials (2^53 then) and their sums stay far from fp32's end, rows of zeros among them.
constexpr int kLeastExpo = 82;
// A new reference where a lane's sums of exponentials reach this (by rows whose
// scale is too small for their products to ask for one).
constexpr float kMostSum = 1.2676506e30f;  // 2^100
// A reference from this on is no number: fp32 would leave the unit out of it.
constexpr float kMostLogit = 67108864.f;  // 2^26, logits in powers of two
// The reference before a row's first position: its exponential overflows and brings one.
constexpr float kNone = -3e38f;
// log2(e) / sqrt(d): logits count in powers of two
template <int D>
constexpr float kLogitScaleOf = D == 32 ? 0.25503486f : D == 64 ? 0.18033688f : 0.12751743f;

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

// Two 16x16 byte matrices (lanes 0-15 and 16-31 give the rows' addresses):
// register 2i + j gets bytes (rows 4 (lane % 4) .. + 3, column lane / 4 + 8 j) of matrix i.
__device__ __forceinline__ void load_columns(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
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

// (x & MASK) | magic in one instruction.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "n"(MASK), "r"(magic));
    return r;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// What a ring stage holds: its work row, which of the row's tiles it is, and
// the valid positions of each of its pages (a byte each).
struct StageMeta {
    int row, tile, tiles;
    uint32_t valid;
};

// A warp's unfinished piece of a row, for the merge.
struct Piece {
    int row;          // -1: none
    int flags;        // bit 0: holds the row's first tile, bit 1: its last
    int tiles;        // of the whole row
    long long tile0;  // the row's first tile among all
};

template <int DK, int DV, int CW, int NVU>
struct Shape {
    static constexpr int NT = CW == 4 ? (NVU + 1) / 2 : CW == 8 ? NVU : 2;  // tiles of 8 columns
    static constexpr int KS = DK / 16;                                       // k-steps of q.k
    static constexpr int WK = DK / 32;                                       // words of a key row per lane
    static constexpr int MT = DV / 16;                                       // tiles of 16 value dims
    static constexpr int ACC = CW == 16 ? 2 : NVU;                           // accumulators of MT tiles
    static constexpr int stage_bytes = kTile * (DK / 2 + 2) + NVU * kTile * (DV / 2 + 2);
    // warps: as many as two stages each leave room for and their registers
    // (accumulators and queries beside about 90 to 105 others)
    static constexpr int by_smem = kRingBytes / (2 * stage_bytes), regs = ACC * MT * 4 + NT * KS * 2 + 72 + 16 * NT;
    static constexpr int W = by_smem >= 16 && regs <= 128 ? 16 : by_smem >= 12 && regs <= 168 ? 12 : 8;
    static constexpr int stages = kRingBytes / (W * stage_bytes) < kMaxStages ? kRingBytes / (W * stage_bytes) : kMaxStages;
};

struct Partition {
    int items, mult;  // items (sequences, or sequence x key head) and work rows of each
    long long T;      // tiles of all rows
    int C;            // CTAs that share them
};

// P: positions per page (a template parameter: every offset inside a tile is
// then an immediate).
template <int DK, int DV, int CW, int NVU, int P>
__global__ void __launch_bounds__((Shape<DK, DV, CW, NVU>::W * 32), 1)
    paged_decode_kernel(const PagedDecodeArgs a, const int min_tiles) {
    using S = Shape<DK, DV, CW, NVU>;
    constexpr int NT = S::NT, KS = S::KS, WK = S::WK, MT = S::MT, ACC = S::ACC;
    constexpr float kLogitScale = kLogitScaleOf<DK>;
    constexpr int kWarps = S::W, kThreads = kWarps * 32, stages = S::stages;
    extern __shared__ __align__(16) uint8_t ring[];  // [kWarps][stages][stage bytes]
    __shared__ uint64_t bars[kWarps][stages], pace;
    __shared__ __align__(16) StageMeta metas[kWarps][stages];
    __shared__ long long prefix[kThreads + 1];
    __shared__ long long warp_sums[kWarps];
    __shared__ Piece pieces[2 * kWarps];
    __shared__ int piece_list[2 * kWarps], group_begin[2 * kWarps + 1], group_flags[2 * kWarps], n_groups;
    __shared__ int group_last[2 * kWarps];
    __shared__ int abort_flag;

    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    constexpr int EPT = kTile / P;                                        // pages per tile
    constexpr int KBLK = paged_block_bytes(P, DK), VBLK = paged_block_bytes(P, DV);
    const int nvg = g.nvk / NVU;
    // A record of a work row: (reference, sum of exponentials) of its columns, then
    // o as the lanes hold it, four values of each of the 32 lanes after another.
    constexpr int kColumns = NVU * CW, NV = CW == 4 ? ACC * MT * 2 : ACC * MT * 4, kRecord = kColumns * (2 + DV);
    static_assert(32 * NV == kColumns * DV, "every value once");

    if (lane < stages) mbar_init(&bars[warp][lane], 1);
    if (threadIdx.x == 0) mbar_init(&pace, kWarps);
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
    constexpr uint32_t kAllValid = EPT == 1 ? P : EPT == 2 ? P * 0x0101u : P * 0x01010101u;  // a byte per page
    constexpr int k_bytes = EPT * KBLK;
    constexpr uint32_t v_bytes = NVU * VBLK;

    // ---- producer state: where in which row the next tile to load is
    int p_item = 0, p_sub = 0, p_tile = 0, p_tiles = 0, p_entries = 0;
    // a window of 32 pages of the row: this lane's page, loaded once for all
    // the window's tiles and copied by this lane when its tile is due
    int win_left = 0;  // tiles left in the window
    const uint8_t *win_k = nullptr, *win_v = nullptr;
    bool win_live = false;
    uint32_t win_valid = 0;  // valid positions of the pages of this lane's tile, a byte each
    const uint32_t lane_dst = smem_addr(my_ring) + (lane % EPT) * KBLK, lane_vdst = smem_addr(my_ring) + k_bytes + (lane % EPT) * v_bytes;
    if (n_my > 0) {
        int c = 0;  // the chunk of items that holds tile w0: the last with prefix <= w0 (never an empty one)
#pragma unroll
        for (int step = 256; step > 0; step >>= 1)
            if (c + step < kThreads && prefix[c + step] <= w0) c += step;
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
        const unsigned rest = static_cast<unsigned>(w0 - at);  // below tiles x rows of one sequence
        p_sub = static_cast<int>(rest / p_tiles);
        p_tile = static_cast<int>(rest % p_tiles);
    }
    auto load_window = [&]() {
        const int r = p_item * part.mult + p_sub;  // = (b * hk + kh) * nvg + vg
        const int vg = r % nvg, bk = r / nvg, kh = bk % g.hk, b = bk / g.hk;
        const int len = seq_len(b);
        const int e = p_tile * EPT + lane;
        win_left = 32 / EPT;
        win_live = false;
        uint32_t valid = 0;
        if (e < p_entries) {
            const int np = (len + P - 1) / P;
            const int page = a.sel ? a.sel[static_cast<size_t>(bk) * a.n_sel + e] : e;
            const int phys = page >= 0 && page < np ? a.page_table[static_cast<size_t>(b) * g.max_pages + page] : -1;
            win_live = phys >= 0 && phys < g.n_pages;
            if (win_live) {
                win_k = a.k_pages + (static_cast<size_t>(phys) * g.hk + kh) * KBLK;
                win_v = a.v_pages + (static_cast<size_t>(phys) * g.hv + kh * g.nvk + vg * NVU) * VBLK;
                valid = min(P, len - page * P);
            } else {
                raise_device_error(a.err, kErrBounds);
            }
        }
        win_valid = valid << (8 * (lane % EPT));
#pragma unroll
        for (int o = 1; o < EPT; o <<= 1) win_valid |= __shfl_xor_sync(kFull, win_valid, o);
    };
    // loads the next tile into stage s
    auto produce = [&](int s) {
        if (win_left == 0) load_window();
        const int first = 32 - win_left * EPT;  // the lane of the tile's first page
        if (lane >= first && lane < first + EPT) {
            uint64_t* bar = &bars[warp][s];
            if (EPT > 1) {
                if (win_live) mbar_expect_tx(bar, KBLK + v_bytes);
                __syncwarp(((1u << EPT) - 1u) << first);
            }
            if (lane == first) {
                *reinterpret_cast<int4*>(&metas[warp][s]) =
                    make_int4(p_item * part.mult + p_sub, p_tile, p_tiles, static_cast<int>(win_valid));
                if (EPT == 1) mbar_arrive_expect_tx(bar, win_live ? KBLK + v_bytes : 0u);
                else mbar_arrive(bar);
            }
            if (win_live) {
                bulk_load(lane_dst + s * S::stage_bytes, win_k, KBLK, bar);
                bulk_load(lane_vdst + s * S::stage_bytes, win_v, v_bytes, bar);
            }
        }
        __syncwarp();
        --win_left;
        if (++p_tile == p_tiles) {  // on to the next row that has a tile
            p_tile = 0;
            win_left = 0;
            if (++p_sub == part.mult) {
                p_sub = 0;
                do {
                    ++p_item;
                    p_entries = p_item < part.items ? item_entries(p_item) : 1;
                } while (p_entries == 0);
                p_tiles = tiles_of(p_entries);
            }
        }
    };

    // ---- consumer state
    int row = -1, seen = 0;  // seen: flags of the row's tiles so far
    uint32_t qf[NT][KS][2];
    float c0[NT][2], colf[NT][2], m[NT][2], l[NT][2];  // m: the reference of the exponentials
    float acc[ACC][MT][4];
    // Rows gq and gq + 8 of a key tile are positions 2 gq and 2 gq + 1 (of 16): after the transposition a lane
    // then has the probabilities of positions 4 tq, 4 tq + 2 and 4 tq + 1, 4 tq + 3, as it has the values.
    const int pos_a = 2 * gq;
    const uint32_t v_lane_row = (lane & 15) * (DV / 2) + (lane >> 4) * 16;  // its address for load_columns

    // query head (of the work row) in column c of tile nt, or -1
    auto head_of = [&](int nt, int c) {
        const int j = CW == 4 ? 2 * nt + (c >> 2) : CW == 8 ? nt : 0;
        const int i = CW == 4 ? (c & 3) : CW == 8 ? c : 8 * nt + c;
        return j < NVU && i < g.Gv ? j * g.Gv + i : -1;
    };
    auto begin_row = [&](int r) {
        row = r;
        seen = 0;
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
            const int sh = min(14 + 127 - static_cast<int>(__float_as_uint(big) >> 23), 126);
            const float up = pow2i(sh);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = bf16_lo(raw[w][i]) * up;
                    x[2 * i + 1] = bf16_hi(raw[w][i]) * up;
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
            const float f = kLogitScale * pow2i(min(24 - sh, 126));
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // this lane's columns 2 tq + i
                c0[nt][i] = __shfl_sync(kFull, start, (2 * tq + i) * 4);
                colf[nt][i] = __shfl_sync(kFull, f, (2 * tq + i) * 4);
                m[nt][i] = kNone;
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
    // The values of o that this lane has, NV of them: for CW 4 the sums of the
    // two halves (columns c and c + 4 of a tile are one head; the left lanes
    // add them up for the even dims, the right ones for the odd).
    // Value k belongs to head (of the work row's columns) lane_head + head_at(k)
    // and dim lane_dim + dim_at(k).
    auto fragment = [&](int k) {
        if constexpr (CW == 4) {
            const int x = k / (2 * MT), mt = k / 2 % MT, i = k % 2;
            const bool left = tq < 2;
            const float mine = left ? acc[x][mt][i] : acc[x][mt][2 + i];
            const float other = left ? acc[x][mt][2 + i] : acc[x][mt][i];
            return mine + __shfl_xor_sync(kFull, other, 2);
        } else {
            return acc[k / (4 * MT)][k / 4 % MT][k % 4];
        }
    };
    auto frag_head = [](int k) { return CW == 4 ? 4 * (k / (2 * MT)) + k % 2 : 8 * (k / (4 * MT)) + k % 2; };
    auto frag_dim = [](int k) {
        const int mt = CW == 4 ? k / 2 % MT : k / 4 % MT;
        return 16 * mt + (CW == 4 ? 0 : k / 2 % 2);
    };
    auto lane_head = [](int ln) { return CW == 4 ? 2 * (ln & 1) : 2 * (ln & 3); };
    auto lane_dim = [](int ln) { return 2 * (ln >> 2) + (CW == 4 ? (ln >> 1) & 1 : 0); };
    // a column's place among the row's heads in the output, or -1
    auto out_head = [&](int c) { return c % CW < g.Gv ? c / CW * g.Gv + c % CW : -1; };
    auto row_out = [&](int r) { return a.out + (static_cast<size_t>(r / nvg) * g.nvk + r % nvg * NVU) * g.Gv * DV; };

    // (the row's number of tiles, and its first among all)
    auto finish_row = [&](bool end_of_range, int tiles, long long tile0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], o);
        float f[NT][2];
        const bool whole = seen == 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) f[nt][i] = !whole ? 1.f : l[nt][i] > 0.f ? __fdividef(1.f, l[nt][i]) : 0.f;
        // an end of the range stays in this warp's ring (its copies are all in), an earlier piece goes to the workspace
        float* dst = end_of_range ? reinterpret_cast<float*>(my_ring)
                                  : a.firsts + (static_cast<size_t>(blockIdx.x) * kWarps + warp) * kRecord;
        if (!whole && gq == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * nt + 2 * tq + i < kColumns)
                        reinterpret_cast<float2*>(dst)[8 * nt + 2 * tq + i] = make_float2(m[nt][i], l[nt][i]);
        }
        float* to = row_out(row) + lane_dim(lane);
        float fx[ACC][2];
#pragma unroll
        for (int x = 0; x < ACC; ++x) beside(f, x, fx[x]);
#pragma unroll
        for (int j = 0; j < NV / 4; ++j) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 4 * j + i;
                v[i] = fragment(k) * fx[CW == 4 ? k / (2 * MT) : k / (4 * MT)][k % 2];
            }
            if (whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = out_head(lane_head(lane) + frag_head(4 * j + i));
                    if (h >= 0) to[h * DV + frag_dim(4 * j + i)] = v[i];
                }
            } else {
                reinterpret_cast<float4*>(dst + 2 * kColumns)[j * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (whole) return;
        if (lane == 0) {
            Piece& p = pieces[2 * warp + (end_of_range ? 1 : 0)];
            p.row = row;
            p.flags = seen;
            p.tiles = tiles;
            p.tile0 = tile0;
        }
    };

    // fp16 pairs of 1024, 1032, 1/16 and -72
    constexpr uint32_t k1024 = 0x64006400u;
    const __half2 k1032 = bits_half2(0x64086408u), k16th = bits_half2(0x2c002c00u), k72 = bits_half2(0xd480d480u);
    // the value head of this lane's columns of a tile (CW 4: two value heads to a tile)
    const int v_lane = CW == 4 ? min(tq >> 1, NVU - 1) * VBLK : 0;

    // ---- 16 positions: group gi of the stage's tile
    auto consume = [&](const uint8_t* buf, uint32_t tile_valid, uint32_t gi, auto all_valid) {
        const uint32_t e = gi * 16 / P, in = gi * 16 % P;  // the group's page and its place in it
        const int valid = static_cast<int>((tile_valid >> (8 * e)) & 0xffu) - static_cast<int>(in);
        const uint8_t* kb = buf + e * KBLK;
        const uint8_t* krow = kb + (in + pos_a) * (DK / 2) + tq * (WK * 4);
        const uint8_t* vb = buf + k_bytes + e * NVU * VBLK;
        uint32_t w[2][WK];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint8_t* src = krow + r * (DK / 2);
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
        // the scales of the two positions, the first in the low half
        uint32_t kscale = *reinterpret_cast<const uint32_t*>(kb + P * (DK / 2) + 2 * (in + pos_a)), vscale[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int j = CW == 4 ? 2 * nt : CW == 8 ? nt : 0;
            vscale[nt] = *reinterpret_cast<const uint32_t*>(vb + j * VBLK + v_lane + P * (DV / 2) + 2 * (in + pos_a));
        }
        float x[NT][4];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const uint32_t lo = (k & 1) ? w[0][k / 2] >> 8 : w[0][k / 2], hi = (k & 1) ? w[1][k / 2] >> 8 : w[1][k / 2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float (&c)[4] = x[nt];
                mma_f16(x[nt], lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u, qf[nt][k][0],
                        qf[nt][k][1], k ? c[0] : c0[nt][0], k ? c[1] : c0[nt][1], k ? c[2] : c0[nt][0],
                        k ? c[3] : c0[nt][1]);
            }
        }
        float off[2] = {0.f, 0.f};  // -inf at the positions past the end, whose scales count as 0
        if (!decltype(all_valid)::value && valid < 16) {
            const uint32_t keep = pos_a + 1 < valid ? 0xffffffffu : pos_a < valid ? 0x0000ffffu : 0u;
            off[0] = pos_a < valid ? 0.f : -kInf;
            off[1] = pos_a + 1 < valid ? 0.f : -kInf;
            kscale &= keep;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) vscale[nt] &= keep;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float s = r ? bf16_hi(kscale) : bf16_lo(kscale);
#pragma unroll
                for (int i = 0; i < 2; ++i) x[nt][2 * r + i] = __fmaf_rn(x[nt][2 * r + i], s, off[r]);
            }
        // p = 2^(logit - reference), y = p times its row's scale, in two fp16 halves, sum = l and the p of its column
        float p[NT][4], y[NT][4], sum[NT][2];
        uint32_t hi[NT][2], lo[NT][2];
        auto products = [&]() {
            __half2 top = bits_half2(0u);
            float all = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float s = r ? bf16_hi(vscale[nt]) : bf16_lo(vscale[nt]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        p[nt][2 * r + i] = exp2_approx(__fmaf_rn(x[nt][2 * r + i], colf[nt][i], -m[nt][i]));
                        y[nt][2 * r + i] = p[nt][2 * r + i] * s;
                    }
                    const __half2 h = __floats2half2_rn(y[nt][2 * r], y[nt][2 * r + 1]);
                    hi[nt][r] = half2_bits(h);
                    top = __hmax2_nan(top, h);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sum[nt][i] = l[nt][i] + p[nt][i] + p[nt][2 + i];
                    all += sum[nt][i];
                }
            }
            // a half at 2^15 or above, sums far up, or no number
            return ((half2_bits(top) + 0x08000800u) & 0x80008000u) != 0u || !(all < kMostSum);
        };
        if (__any_sync(kFull, products())) {  // a new reference: the largest product so far is below 2^kUnit of it
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float e0 = static_cast<float>(max((vscale[nt] >> 7) & 0xffu, static_cast<uint32_t>(kLeastExpo)));
                const float e1 = static_cast<float>(max((vscale[nt] >> 23) & 0xffu, static_cast<uint32_t>(kLeastExpo)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(__fmaf_rn(x[nt][i], colf[nt][i], e0), __fmaf_rn(x[nt][2 + i], colf[nt][i], e1));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
                    v = fmaxf(ceilf(v) - static_cast<float>(kUnit + 126), m[nt][i]);
                    if (fabsf(v) >= kMostLogit && v != kNone) v = __uint_as_float(0x7fffffffu);
                    f[nt][i] = exp2_approx(m[nt][i] - v);
                    m[nt][i] = v;
                    l[nt][i] = f[nt][i] > 0.f ? l[nt][i] * f[nt][i] : 0.f;
                }
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
            products();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[nt][r] = sum[nt][r];
                const float2 back = __half22float2(bits_half2(hi[nt][r]));
                lo[nt][r] = half2_bits(__floats2half2_rn(y[nt][2 * r] - back.x, y[nt][2 * r + 1] - back.y));
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
                uint32_t u[4];
                load_columns(smem_addr(vb + j * VBLK + in * (DV / 2)) + v_lane_row + 32 * half, u);
                {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 16 dims: the bytes' low numbers are row gq, the high ones row gq + 8
                        const uint32_t odd = u[i] >> 8;
                        const uint32_t f0 = half2_bits(__hsub2(bits_half2(and_or<0x000f000fu>(u[i], k1024)), k1032));
                        const uint32_t f1 = half2_bits(__hfma2(bits_half2(and_or<0x00f000f0u>(u[i], k1024)), k16th, k72));
                        const uint32_t f2 = half2_bits(__hsub2(bits_half2(and_or<0x000f000fu>(odd, k1024)), k1032));
                        const uint32_t f3 = half2_bits(__hfma2(bits_half2(and_or<0x00f000f0u>(odd, k1024)), k16th, k72));
                        const int mt = 4 * half + i;
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
    };

    // ---- the warp's tiles
    // (lanes leave a wait one by one: the vote brings the warp together again)
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait(bar, parity, &abort_flag)) != 0; };
    int produced = 0, done = 0, tiles = 0;
    long long tile0 = 0;
    uint32_t phase = 0;  // bit s: parity to wait for in stage s
    bool ok = true;
    for (; produced < stages && produced < n_my; ++produced) produce(produced);
    for (int s = 0;; ++done) {
        int4 meta = make_int4(-1, 0, 0, 0);
        if (done < n_my) {
            if (!(ok = warp_wait(&bars[warp][s], (phase >> s) & 1u))) break;
            phase ^= 1u << s;
            meta = *reinterpret_cast<const int4*>(&metas[warp][s]);
        } else {  // the warp's last round is over: the others no longer count on it
            const int round = n_my > 0 ? (n_my - 1) / kRound : 0;
            if (round > 0 && !(ok = warp_wait(&pace, (round - 1) & 1))) break;
            if (lane == 0) mbar_arrive_drop(&pace);
        }
        if (meta.x != row) {
            if (row >= 0) finish_row(done == n_my, tiles, tile0);
            if (done == n_my) break;
            begin_row(meta.x);
            tiles = meta.z;
            tile0 = w0 + done - meta.y;
        }
        if (done == n_my) break;  // (a warp without a tile)
        seen |= (meta.y == 0 ? 1 : 0) | (meta.y == tiles - 1 ? 2 : 0);
        const uint8_t* buf = my_ring + s * S::stage_bytes;
        if (static_cast<uint32_t>(meta.w) == kAllValid) {
#pragma unroll
            for (uint32_t gi = 0; gi < kTile / 16; ++gi) consume(buf, meta.w, gi, std::true_type{});
        } else {
#pragma unroll 1
            for (uint32_t gi = 0; gi < kTile / 16; ++gi) consume(buf, meta.w, gi, std::false_type{});
        }
        __syncwarp();
        if (produced < n_my) {
            produce(s);
            ++produced;
        }
        s = s + 1 == stages ? 0 : s + 1;
        if (done % kRound == kRound - 1 && done + 1 < n_my) {  // end of round done / kRound
            const int round = done / kRound;
            if (round > 0 && !(ok = warp_wait(&pace, (round - 1) & 1))) {
                ++done;
                break;
            }
            if (lane == 0) mbar_arrive(&pace);
        }
    }
    if (!ok) {  // a wait ran out: let the copies in flight land (each wait limited again), then leave
        if (lane == 0) raise_device_error(a.err, kErrTimeout);
        int given_up = 0;
        for (int i = done; i < produced; ++i) {
            const int s = i % stages;
            mbar_wait(&bars[warp][s], (phase >> s) & 1u, &given_up);
            __syncwarp();
            phase ^= 1u << s;
        }
    }

    // ---- pieces of the CTA, row by row
    __syncthreads();
    if (abort_flag) return;
    if (warp == 0) {  // the pieces there are, in order; those of one row follow one another
        const int r = lane < 2 * kWarps ? pieces[lane].row : -1;
        const uint32_t have = __ballot_sync(kFull, r >= 0);
        const int at = __popc(have & lanemask_lt());
        const uint32_t before = have & lanemask_lt();
        const int prev = __shfl_sync(kFull, r, before ? 31 - __clz(before) : 0);
        const uint32_t starts = __ballot_sync(kFull, r >= 0 && (before == 0 || prev != r));
        const int gi = __popc(starts & (lanemask_lt() | (1u << lane))) - 1;
        if (r >= 0) piece_list[at] = lane;
        if (starts >> lane & 1u) group_begin[gi] = at;
        if (lane < 2 * kWarps) group_flags[lane] = 0;
        __syncwarp();
        if (r >= 0) atomicOr(&group_flags[gi], pieces[lane].flags);
        if (lane == 0) n_groups = __popc(starts), group_begin[__popc(starts)] = __popc(have);
    }
    __syncthreads();
    auto piece_rec = [&](int i) -> const float* {
        return (i & 1) ? reinterpret_cast<const float*>(ring + static_cast<size_t>(i >> 1) * stages * S::stage_bytes)
                       : a.firsts + (static_cast<size_t>(blockIdx.x) * kWarps + (i >> 1)) * kRecord;
    };
    // a thread's four values: place `at` of kPlaces in the records, of two columns
    constexpr int kPlaces = kColumns * DV / 4;
    auto columns_of = [&](int at, int (&c)[2]) {
        c[0] = lane_head(at % 32) + frag_head(at / 32 * 4);
        c[1] = c[0] + 1;
    };
    auto write_place = [&](int r, int at, const float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = at / 32 * 4 + i, h = out_head(lane_head(at % 32) + frag_head(k));
            if (h >= 0) row_out(r)[h * DV + lane_dim(at % 32) + frag_dim(k)] = v[i];
        }
    };
    bool crosses = false;  // a row of this CTA's goes on in another
    for (int gi = 0; gi < n_groups; ++gi) crosses |= group_flags[gi] != 3;
    {
        for (int item = threadIdx.x; item < n_groups * kPlaces; item += kThreads) {
            const int gi = item / kPlaces, at = item % kPlaces;
            const int i0 = group_begin[gi], i1 = group_begin[gi + 1];
            const bool whole = group_flags[gi] == 3;
            const Piece first = pieces[piece_list[i0]];
            int c[2];
            columns_of(at, c);
            float M[2] = {kNone, kNone}, L[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const float* src = piece_rec(piece_list[i]);
                M[0] = fmaxf(M[0], src[2 * c[0]]);
                M[1] = fmaxf(M[1], src[2 * c[1]]);
            }
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const float* src = piece_rec(piece_list[i]);
                const float2 h0 = reinterpret_cast<const float2*>(src)[c[0]], h1 = reinterpret_cast<const float2*>(src)[c[1]];
                const float4 v = reinterpret_cast<const float4*>(src + 2 * kColumns)[at];
                const float f0 = exp2_approx(h0.x - M[0]), f1 = exp2_approx(h1.x - M[1]);
                L[0] += f0 * h0.y, L[1] += f1 * h1.y;
                o[0] += f0 * v.x, o[1] += f1 * v.y, o[2] += f0 * v.z, o[3] += f1 * v.w;
            }
            if (whole) {
                const float i0f = L[0] > 0.f ? __fdividef(1.f, L[0]) : 0.f, i1f = L[1] > 0.f ? __fdividef(1.f, L[1]) : 0.f;
                const float v[4] = {o[0] * i0f, o[1] * i1f, o[2] * i0f, o[3] * i1f};
                write_place(first.row, at, v);
            } else {
                float* dst = a.records + (static_cast<size_t>(blockIdx.x) * 2 + (first.tile0 < cta0 ? 0 : 1)) * kRecord;
                reinterpret_cast<float4*>(dst + 2 * kColumns)[at] = make_float4(o[0], o[1], o[2], o[3]);
                if (lane_dim(at % 32) < 2 && at / 32 * 4 % (NV / ACC) == 0) {  // one thread of a column pair (CW 4: either dim's)
                    reinterpret_cast<float2*>(dst)[c[0]] = make_float2(M[0], L[0]);
                    reinterpret_cast<float2*>(dst)[c[1]] = make_float2(M[1], L[1]);
                }
            }
        }
    }
    if (!crosses) return;
    // ---- the last CTA of a row that crosses CTAs merges its records
    __syncthreads();
    if (threadIdx.x < n_groups) {
        const Piece p = pieces[piece_list[group_begin[threadIdx.x]]];
        int n = 0;
        if (group_flags[threadIdx.x] != 3) {
            n = cta_of_tile(p.tile0 + p.tiles - 1, part.T, part.C) - cta_of_tile(p.tile0, part.T, part.C) + 1;
            if (take_ticket(a.tickets + p.row) == static_cast<unsigned>(n - 1)) a.tickets[p.row] = 0u;
            else n = 0;
        }
        group_last[threadIdx.x] = n;  // records to merge, if this is the last CTA
    }
    __syncthreads();
    for (int gi = 0; gi < n_groups; ++gi) {
        const int n = group_last[gi];
        if (n == 0) continue;
        const Piece p = pieces[piece_list[group_begin[gi]]];
        const int first = cta_of_tile(p.tile0, part.T, part.C);
        auto record = [&](int i) { return a.records + (static_cast<size_t>(first + i) * 2 + (i == 0 ? 1 : 0)) * kRecord; };
        // a place per thread; groups of threads take every kSubs-th record and are joined in the (free) rings
        constexpr int kSubs = kThreads / kPlaces > 0 ? kThreads / kPlaces : 1;
        float4* parts = reinterpret_cast<float4*>(ring);
        const int sub = threadIdx.x / kPlaces;
        for (int at = threadIdx.x % kPlaces; at < kPlaces && sub < kSubs; at += kThreads) {
            int c[2];
            columns_of(at, c);
            float M[2] = {kNone, kNone}, L[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
            auto join = [&](float2 h0, float2 h1, float4 v) {
                const float m0 = fmaxf(M[0], h0.x), m1 = fmaxf(M[1], h1.x);
                const float f0 = exp2_approx(h0.x - m0), f1 = exp2_approx(h1.x - m1);
                const float g0 = exp2_approx(M[0] - m0), g1 = exp2_approx(M[1] - m1);
                M[0] = m0, M[1] = m1;
                L[0] = L[0] * g0 + f0 * h0.y, L[1] = L[1] * g1 + f1 * h1.y;
                o[0] = o[0] * g0 + f0 * v.x, o[1] = o[1] * g1 + f1 * v.y;
                o[2] = o[2] * g0 + f0 * v.z, o[3] = o[3] * g1 + f1 * v.w;
            };
            for (int i0 = sub; i0 < n; i0 += 8 * kSubs) {
                float2 h0[8], h1[8];
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int i = i0 + u * kSubs;
                    h0[u] = h1[u] = make_float2(kNone, 0.f);
                    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < n) {
                        const float* src = record(i);
                        h0[u] = __ldcg(reinterpret_cast<const float2*>(src) + c[0]);
                        h1[u] = __ldcg(reinterpret_cast<const float2*>(src) + c[1]);
                        v[u] = __ldcg(reinterpret_cast<const float4*>(src + 2 * kColumns) + at);
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) join(h0[u], h1[u], v[u]);
            }
            if constexpr (kSubs > 1) {
                if (sub > 0) {
                    parts[(sub * kPlaces + at) * 2] = make_float4(o[0], o[1], o[2], o[3]);
                    parts[(sub * kPlaces + at) * 2 + 1] = make_float4(M[0], L[0], M[1], L[1]);
                }
                named_barrier(1, kSubs * kPlaces);
                if (sub == 0) {
#pragma unroll
                    for (int s = 1; s < kSubs; ++s) {
                        const float4 h = parts[(s * kPlaces + at) * 2 + 1];
                        join(make_float2(h.x, h.y), make_float2(h.z, h.w), parts[(s * kPlaces + at) * 2]);
                    }
                }
            }
            if (sub == 0) {
                const float i0f = L[0] > 0.f ? __fdividef(1.f, L[0]) : 0.f, i1f = L[1] > 0.f ? __fdividef(1.f, L[1]) : 0.f;
                const float v[4] = {o[0] * i0f, o[1] * i1f, o[2] * i0f, o[3] * i1f};
                write_place(p.row, at, v);
            }
        }
        __syncthreads();  // the rings are used again
    }
}

template <int DK, int DV, int CW, int NVU, int P>
cudaError_t run(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    using S = Shape<DK, DV, CW, NVU>;
    constexpr int smem = S::W * S::stages * S::stage_bytes;
    auto kern = paged_decode_kernel<DK, DV, CW, NVU, P>;
    const cudaError_t e = allow_dynamic_smem(kern, smem);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kPagedMaxCtas ? sms : kPagedMaxCtas;
    return launch_dependent(kern, dim3(ctas), dim3(S::W * 32), smem, stream, a, kMinTiles);
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
