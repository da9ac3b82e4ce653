// The paged cache's way in and out: new key, value and query rows take the
// position rotation, keys and values are rounded to 4 bits and written into
// their pages; the same walk reads rows back as bf16.
//
// Rotation of a pair (x1, x2) by the table's angle row of its position:
// y1 = x1 c - x2 s, y2 = x2 c + x1 s, rounded to fp32 and then to bf16.
// 4 bits: scale = bf16(max|y| / 7) per row and head, n = clamp(rint(y /
// scale), -7, 7).  y has 8 significant bits and the scale 8, so no quotient
// comes within an fp32 rounding of a half without being one: n is the exact
// one, whatever computes it.
//
// Work unit: the new tokens of one page (the pages a sequence's run touches
// are found from its length and the run's start alone), so that one CTA owns
// a page's key bounds (each warp has its own, joined at the end): no atomics,
// results do not depend on the order of CTAs.  A row is handled by d/16 lanes, each with two 16-byte
// chunks that hold both halves of its pairs; a group of lanes keeps its
// position's angles for all heads.
//
// Bound by the rows' traffic, so the arithmetic is kept short: a rotated value
// is two operations and an error bound, recomputed exactly only where the
// bound leaves its bf16 rounding open (one value in some 2000); a quotient is
// a product with the scale's reciprocal, put on a grid of 2^-12 (halves stay
// halves, and no other quotient is within 2^-11 of one).  Measured on the device
// (graph replays): 20.7K tokens of 32/4/8 heads of 64 in 12 runs 50.6 us and their
// rows read back 12.7 (together 248 MB, 0.60 of the copy rate; the append is bound
// by issue); 256 single tokens 4.6 us, with the lengths grown in place 5.6 us (a
// ticket and the last CTA's pass over the lengths), from Python without a graph
// 11.2 us: the host's share.
#include <cuda_bf16.h>

#include "paged.h"
#include "paged_device.cuh"

namespace saga {

namespace {

// Small CTAs, many to an SM: a unit's start is a chain of dependent loads (run,
// length, page) that only other CTAs hide.
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kResident = 5;
constexpr int kDepth = 4;        // rows of a lane in flight
constexpr int kPartsPerSm = 12;  // CTAs per SM that a launch aims for by splitting the heads of its units
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kHole = 1u << 31;  // in the ticket: a page of the call's was missing
// Where a work unit's tokens are: sequence, logical page, rows [first, first +
// rows) of positions, and the index of the first one among the new tokens.
struct Unit {
    int seq, page, off, rows, token, phys;
    bool old_rows;  // the page held rows of the sequence before
};

// Units of sequence i start at cu[i]/P + 2i: a run of n tokens touches at
// most n/P + 2 pages, so that the ranges do not overlap.
__device__ __forceinline__ int unit_start(int cu, int i, int shift) { return (max(cu, 0) >> shift) + 2 * i; }

// (w.phys is the table's entry as it is, still on its way: has_page checks it.)
__device__ __forceinline__ bool find_unit(const PagedAppendArgs& a, int u, Unit& w) {
    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31, shift = 31 - __clz(g.P);
    int seq, j, n, t0, len0;
    if (!a.cu) {
        if (u >= g.b) return false;
        seq = u, j = 0, n = 1, t0 = u;
        len0 = a.seq_lens[seq];
    } else {
        int lo = 0, len = g.b;
        // 32-ary search for the last sequence that starts at or before u; the last level's lanes bring all that
        // is needed of theirs
        while (len > 32) {
            const int step = (len + 31) / 32;
            const bool in = lane * step < len && unit_start(a.cu[lo + lane * step], lo + lane * step, shift) <= u;
            const int c = __popc(__ballot_sync(kFull, in));
            if (c == 0) return false;
            lo += (c - 1) * step;
            len = min(step, len - (c - 1) * step);
        }
        const int i = lo + min(lane, len - 1);
        const int c0 = a.cu[i], c1 = a.cu[i + 1], start = unit_start(c0, i, shift), l0 = a.seq_lens[i];
        const int c = __popc(__ballot_sync(kFull, lane < len && start <= u));
        if (c == 0) return false;
        seq = lo + c - 1;
        t0 = __shfl_sync(kFull, c0, c - 1);
        n = __shfl_sync(kFull, c1, c - 1) - t0;
        j = u - __shfl_sync(kFull, start, c - 1);
        len0 = __shfl_sync(kFull, l0, c - 1);
        if (t0 < 0 || n < 0 || t0 > a.n_tokens - n) {
            if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
            return false;
        }
    }
    if (n == 0) return false;
    if (len0 < 0 || len0 > g.max_pages * g.P) {
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        return false;
    }
    const int page = (len0 >> shift) + j;
    const int first = max(len0, page * g.P), last = min(len0 + n, (page + 1) * g.P);
    if (first >= last) return false;
    w.phys = page < g.max_pages ? a.page_table[static_cast<size_t>(seq) * g.max_pages + page] : -1;
    w.seq = seq;
    w.page = page;
    w.off = first - page * g.P;
    w.rows = last - first;
    w.token = t0 + (first - len0);
    w.old_rows = len0 > page * g.P;
    return true;
}

// Whether the unit's page is in the pool; its rows are left alone otherwise.
__device__ __forceinline__ bool has_page(const PagedAppendArgs& a, const Unit& w) { return w.phys >= 0 && w.phys < a.g.n_pages; }

// x1 a + x2 b rounded once to fp32 (products and sum split into value and error).
__device__ __forceinline__ float dot2_rn(float x1, float a, float x2, float b) {
    const float p = __fmul_rn(x1, a), pe = __fmaf_rn(x1, a, -p);
    const float q = __fmul_rn(x2, b), qe = __fmaf_rn(x2, b, -q);
    const float s = __fadd_rn(p, q);
    const float z = __fsub_rn(s, p);
    const float se = __fadd_rn(__fsub_rn(p, __fsub_rn(s, z)), __fsub_rn(q, z));
    return __fadd_rn(s, __fadd_rn(se, __fadd_rn(pe, qe)));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
}

enum Rotation : int { kNoRotation = 0, kHalves = 1, kInterleaved = 2 };  // pairs (i, i + rot/2), (2i, 2i + 1)

// A lane's two chunks of 8 dims, and the angles of its 8 pairs.
template <int D, int MODE>
struct Pairs {
    int ca, cb;
    bool turned;
    float c[8], s[8];

    __device__ __forceinline__ Pairs(int rot) {
        const int i = threadIdx.x % (D / 16);
        const bool split = MODE == kHalves && i < rot / 16;
        ca = split ? i : 2 * i;
        cb = split ? i + rot / 16 : 2 * i + 1;
        turned = MODE == kHalves ? split : MODE == kInterleaved && 16 * i < rot;
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
    }
    __device__ __forceinline__ void load(const float* table, int rot, int pos) {
        if (MODE == kNoRotation || !turned) return;
        const float* at = table + static_cast<size_t>(pos) * rot + 8 * (threadIdx.x % (D / 16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(at) + h), y = __ldg(reinterpret_cast<const float4*>(at + rot / 2) + h);
            c[4 * h] = x.x, c[4 * h + 1] = x.y, c[4 * h + 2] = x.z, c[4 * h + 3] = x.w;
            s[4 * h] = y.x, s[4 * h + 1] = y.y, s[4 * h + 2] = y.z, s[4 * h + 3] = y.w;
        }
    }
    // The rotated chunks.
    __device__ __forceinline__ void turn(uint4& ra, uint4& rb) const {
        if (MODE == kNoRotation) return;
        float xa[8], xb[8];
        unpack8(ra, xa);
        unpack8(rb, xb);
        float u[8], v[8];  // the pairs
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = MODE == kHalves ? xa[j] : j < 4 ? xa[2 * j] : xb[2 * j - 8];
            v[j] = MODE == kHalves ? xb[j] : j < 4 ? xa[2 * j + 1] : xb[2 * j - 7];
        }
        uint32_t out[8], up[8], open = 0u;
        constexpr float k = 1.2e-7f;  // above 2^-23: a product's and a sum's rounding, with room
        float y[8], z[8], ye[8], ze[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = v[j] * s[j], q = u[j] * s[j];
            const float r = __fmaf_rn(u[j], c[j], -p), t = __fmaf_rn(v[j], c[j], q);
            const float re = fabsf(p) + fabsf(r), te = fabsf(q) + fabsf(t);
            y[j] = __fmaf_rn(-k, re, r), ye[j] = __fmaf_rn(k, re, r);
            z[j] = __fmaf_rn(-k, te, t), ze[j] = __fmaf_rn(k, te, t);
        }
        auto pack = [&](const float (&a)[8], const float (&b)[8], uint32_t (&o)[8]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j] = MODE == kHalves ? pack2(a[2 * j], a[2 * j + 1]) : pack2(a[j], b[j]);
                o[4 + j] = MODE == kHalves ? pack2(b[2 * j], b[2 * j + 1]) : pack2(a[4 + j], b[4 + j]);
            }
        };
        pack(y, z, out);
        pack(ye, ze, up);
#pragma unroll
        for (int j = 0; j < 8; ++j) open |= out[j] ^ up[j];
        if (open) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = dot2_rn(u[j], c[j], v[j], -s[j]);
                z[j] = dot2_rn(v[j], c[j], u[j], s[j]);
            }
            pack(y, z, out);
        }
        if (turned) {
            ra = make_uint4(out[0], out[1], out[2], out[3]);
            rb = make_uint4(out[4], out[5], out[6], out[7]);
        }
    }
};

// How a unit's rows and heads are spread over the CTA's groups of d/16 lanes:
// rp groups side by side on rows, the rest on heads.
struct Spread {
    int r, gh, rp, hp;
};
template <int D>
__device__ __forceinline__ Spread spread(int rows) {
    constexpr int GROUPS = kThreads / (D / 16);
    int rp = 1;
    while (rp < rows && rp < GROUPS) rp *= 2;
    const int grp = threadIdx.x / (D / 16);
    return Spread{grp % rp, grp / rp, rp, GROUPS / rp};
}

// Eight values to the word of n + 8 (value i in bits 4i .. 4i+3) for the
// scale s with reciprocal inv; 0x88888888 where s is 0.
__device__ __forceinline__ uint32_t nibbles(const float (&y)[8], float s, float inv) {
    uint32_t word = 0;
    if (s >= 1e-30f) {
        // n + 8 in the low bits of 1.5 2^23 + 8 + n; the other bits of the eight words add up to a constant
        constexpr float grid = 1.5f * 2048.f, whole = 12582912.f + 8.f;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float t = __fadd_rn(__fadd_rn(__fmul_rn(y[i], inv), grid), -grid);
            word = word * 16u + __float_as_uint(__fadd_rn(t, whole));
        }
        return word - 0x4b400000u * 0x11111111u;
    }
#pragma unroll
    for (int i = 7; i >= 0; --i) {  // scales that are 0 or have few bits
        const float n = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(y[i], s)), -7.f), 7.f) : 0.f;
        word = word * 16u + static_cast<uint32_t>(static_cast<int>(n) + 8);
    }
    return word;
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The larger magnitudes of two pairs of bf16 values, as bits.
__device__ __forceinline__ uint32_t magnitudes(uint32_t x, uint32_t y) { return __vmaxu2(x & 0x7fff7fffu, y & 0x7fff7fffu); }

// Eight bf16 values, each the smaller or larger of two.
__device__ __forceinline__ uint4 least(uint4 x, uint4 y) {
    auto f = [](uint32_t a, uint32_t b) { return as_u32(__hmin2(as_bf162(a), as_bf162(b))); };
    return make_uint4(f(x.x, y.x), f(x.y, y.y), f(x.z, y.z), f(x.w, y.w));
}
__device__ __forceinline__ uint4 most(uint4 x, uint4 y) {
    auto f = [](uint32_t a, uint32_t b) { return as_u32(__hmax2(as_bf162(a), as_bf162(b))); };
    return make_uint4(f(x.x, y.x), f(x.y, y.y), f(x.z, y.z), f(x.w, y.w));
}
__device__ __forceinline__ uint4 shfl_xor4(uint4 v, int o) {
    return make_uint4(__shfl_xor_sync(kFull, v.x, o), __shfl_xor_sync(kFull, v.y, o), __shfl_xor_sync(kFull, v.z, o),
                      __shfl_xor_sync(kFull, v.w, o));
}

// The unit's rows of nk key heads from k0, nv value heads from v0 (rows of the
// keys' width) and nq query heads from q0, one after another: keys and queries
// rotated, keys and values rounded into the pages, queries to q_out.  A lane's
// chunks come through kDepth slots of its own in shared memory, filled
// asynchronously (loads in flight cost no registers).  One body for the three
// kinds of rows: a short call is bound by fetching its instructions.
struct Heads {
    int k0, nk, v0, nv, q0, nq;
};
template <int D, int MODE>
__device__ __forceinline__ void write_rows(const PagedAppendArgs& a, const Unit& w, const Heads& n, bool value_rows,
                                           uint4 (*lo_hi)[2][D / 8], uint4 (*slots)[2][kThreads]) {
    constexpr int LPR = D / 16;
    const PagedGeom& g = a.g;
    const Spread sp = spread<D>(w.rows);
    const int total = n.nk + n.nv + n.nq;
    const size_t page_row = static_cast<size_t>(w.phys);
    Pairs<D, MODE> pairs(a.rot);
    for (int rb = 0; rb < w.rows; rb += sp.rp) {
        const int r = rb + sp.r;
        const bool row_live = r < w.rows;
        if (row_live && !value_rows) pairs.load(a.rope, a.rot, w.page * g.P + w.off + r);
        const long long token = w.token + r;
        const int row_at = (w.off + r) * (D / 2), scale_at = g.P * (D / 2) + 2 * (w.off + r);
        auto issue = [&](int slot, int at) {
            const int i = at + sp.gh;
            if (row_live && i < total) {
                const void* base = i < n.nk ? a.k_new : i < n.nk + n.nv ? a.v_new : a.q_new;
                const long long stride = i < n.nk ? a.k_stride : i < n.nk + n.nv ? a.v_stride : a.q_stride;
                const int h = i < n.nk ? n.k0 + i : i < n.nk + n.nv ? n.v0 + i - n.nk : n.q0 + i - n.nk - n.nv;
                const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + token * stride + h * D);
                cp_async_16(smem_addr(&slots[slot][0][threadIdx.x]), row + pairs.ca, 16);
                cp_async_16(smem_addr(&slots[slot][1][threadIdx.x]), row + pairs.cb, 16);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kDepth; ++i) issue(i, i * sp.hp);
        if (!has_page(a, w)) break;  // (looked at once the rows are on their way)
        int slot = 0;
        for (int at = 0; at < total; at += sp.hp) {  // every warp of the CTA the same number of times
            cp_async_wait<kDepth - 1>();
            const int i = at + sp.gh;
            const bool live = row_live && i < total, key = i < n.nk, value = !key && i < n.nk + n.nv;
            uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
            if (live) va = slots[slot][0][threadIdx.x], vb = slots[slot][1][threadIdx.x];
            if (MODE != kNoRotation && !value && !value_rows) pairs.turn(va, vb);
            if (live && !key && !value) {
                uint4* to = reinterpret_cast<uint4*>(a.q_out) + (static_cast<size_t>(token) * g.hq + n.q0 + i - n.nk - n.nv) * (D / 8);
                to[pairs.ca] = va;
                to[pairs.cb] = vb;
            }
            if (at < n.nk + n.nv) {  // rounding: keys or values among the CTA's heads of this time
                float ya[8], yb[8];
                unpack8(va, ya);
                unpack8(vb, yb);
                // the largest magnitude, by its bits: what is not finite is above all that is
                uint32_t most2 = __vmaxu2(__vmaxu2(magnitudes(va.x, va.y), magnitudes(va.z, va.w)),
                                          __vmaxu2(magnitudes(vb.x, vb.y), magnitudes(vb.z, vb.w)));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) most2 = __vmaxu2(most2, __shfl_xor_sync(kFull, most2, o));
                const uint32_t top = max(most2 & 0xffffu, most2 >> 16);
                const float m = __uint_as_float(top << 16);
                // (a seventh of 8 bits is at least a fourteenth of a step from every middle: the product rounds like the quotient)
                const __nv_bfloat16 scale = __float2bfloat16_rn(top < 0x7f80u ? m * 0.142857149f : __uint_as_float(0x7fffffffu));
                const float s = __bfloat162float(scale), inv = __fdividef(1.f, s);
                const uint32_t wa = nibbles(ya, s, inv), wb = nibbles(yb, s, inv);
                if (live && (key || value)) {
                    const int heads = key ? g.hk : g.hv, h = key ? n.k0 + i : n.v0 + i - n.nk, blk = key ? g.kblk : g.vblk;
                    uint8_t* to = (key ? a.k_pages : a.v_pages) + (page_row * heads + h) * blk;
                    reinterpret_cast<uint32_t*>(to + row_at)[pairs.ca] = wa;
                    reinterpret_cast<uint32_t*>(to + row_at)[pairs.cb] = wb;
                    if (threadIdx.x % LPR == 0) *reinterpret_cast<__nv_bfloat16*>(to + scale_at) = scale;
                }
            }
            if (a.bounds && at < n.nk && w.rows == 1) {  // a single row: straight to the page's bounds
                if (live && key) {
                    uint4* box = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.bounds) + (page_row * g.hk + n.k0 + i) * 2 * D);
                    auto widen = [&](uint4* to, uint4 v, bool up) { *to = w.old_rows ? up ? most(v, *to) : least(v, *to) : v; };
                    widen(box + pairs.ca, va, false);
                    widen(box + pairs.cb, vb, false);
                    widen(box + D / 8 + pairs.ca, va, true);
                    widen(box + D / 8 + pairs.cb, vb, true);
                }
            } else if (a.bounds && at < n.nk) {  // the warp's rows of each key head, into the warp's own boxes
                const uint4 none_lo = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);
                const uint4 none_hi = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                uint4 la = row_live ? va : none_lo, lb = row_live ? vb : none_lo, ha = row_live ? va : none_hi, hb = row_live ? vb : none_hi;
                const int span = min(32, sp.rp * LPR);
                for (int o = LPR; o < span; o <<= 1) {
                    la = least(la, shfl_xor4(la, o)), lb = least(lb, shfl_xor4(lb, o));
                    ha = most(ha, shfl_xor4(ha, o)), hb = most(hb, shfl_xor4(hb, o));
                }
                if (key && (threadIdx.x & 31) % span < LPR) {
                    uint4 (*box)[D / 8] = lo_hi[threadIdx.x / 32 * n.nk + i];
                    box[0][pairs.ca] = least(la, box[0][pairs.ca]);
                    box[0][pairs.cb] = least(lb, box[0][pairs.cb]);
                    box[1][pairs.ca] = most(ha, box[1][pairs.ca]);
                    box[1][pairs.cb] = most(hb, box[1][pairs.cb]);
                }
            }
            issue(slot, at + kDepth * sp.hp);
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }
        cp_async_wait<0>();
    }
    cp_async_wait<0>();
}

// The grown lengths: each sequence's up to the first position that the call
// does not write (none of a run or length out of range, none from a page on
// that reaches past the rotation table or is not in the pool).  pages: whether
// the runs' table entries have to be looked up for that.
__device__ __forceinline__ void write_lens(const PagedAppendArgs& a, bool pages) {
    constexpr int kAhead = 4, kOwn = 16;  // entries on their way at once; pages that a lane looks up by itself
    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31, shift = 31 - __clz(g.P), cap = g.max_pages * g.P;
    // the first of pages p, p + step, .. up to p1 that is not in the pool, or p1 + 1
    auto first_hole = [&](const int32_t* table, int p, int p1, int step) {
        for (; p <= p1; p += kAhead * step) {
            int e[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) e[k] = p + k * step <= p1 ? table[p + k * step] : 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (e[k] < 0 || e[k] >= g.n_pages) return p + k * step;
        }
        return p1 + 1;
    };
    for (int i0 = threadIdx.x - lane; i0 < g.b; i0 += kThreads) {
        const int i = i0 + lane;
        int len = 0, end = 0;
        if (i < g.b) {
            end = len = a.seq_lens[i];
            const int t0 = a.cu ? a.cu[i] : 0, n = a.cu ? a.cu[i + 1] - t0 : 1;
            if (t0 < 0 || n < 0 || t0 > a.n_tokens - n) {
                raise_device_error(a.err, kErrBounds);
            } else if (len >= 0 && len <= cap) {
                end = min(len + n, cap);
                if (a.rope && len + n > a.max_pos) end = max(len, min(end, a.max_pos >> shift << shift));
            }
        }
        if (!pages) {
            if (i < g.b) a.lens_out[i] = end;
            continue;
        }
        const int p0 = len >> shift, p1 = (end - 1) >> shift;
        int hole = p1 + 1;
        const bool any = end > len, many = any && p1 - p0 >= kOwn;
        if (any && !many) hole = first_hole(a.page_table + static_cast<size_t>(i) * g.max_pages, p0, p1, 1);
        for (uint32_t left = __ballot_sync(kFull, many); left; left &= left - 1u) {  // long runs: by the whole warp
            const int src = __ffs(left) - 1, q0 = __shfl_sync(kFull, p0, src), q1 = __shfl_sync(kFull, p1, src);
            const int32_t* table = a.page_table + static_cast<size_t>(i0 + src) * g.max_pages;
            const int h = __reduce_min_sync(kFull, first_hole(table, q0 + lane, q1, 32));
            if (lane == src) hole = h;
        }
        if (i < g.b) a.lens_out[i] = hole > p1 ? end : max(len, hole << shift);
    }
}

// Heads are numbered keys, values, queries; CTA y takes [y*per, (y+1)*per).
template <int DK, int DV, int MODE>
__global__ void __launch_bounds__(kThreads, kResident) append_kernel(const PagedAppendArgs a, int per) {
    __shared__ uint4 lo_hi[kWarps * 8][2][DK / 8];  // a warp's bounds of each key head of the CTA's
    __shared__ uint4 slots[kDepth][2][kThreads];
    pdl_wait();  // lengths, tables and pages may be the previous kernels' results
    pdl_trigger();
    const PagedGeom& g = a.g;
    if (blockIdx.x == a.lens_cta) {
        if (blockIdx.y == 0) write_lens(a, true);
        return;
    }
    Unit w;
    bool live = find_unit(a, blockIdx.x, w);
    if (live && a.rope && w.page * g.P + w.off + w.rows > a.max_pos) {  // positions past the table: not written
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        live = false;
    }
    if (live) {
        const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.hk + g.hv + (a.q_new ? g.hq : 0));
        const int k1 = min(h1, g.hk);
        const bool bounds = a.bounds && h0 < k1 && w.rows > 1;
        if (bounds) {
            for (int i = threadIdx.x; i < kWarps * (k1 - h0) * 2 * (DK / 8); i += kThreads) {
                const uint32_t none = i / (DK / 8) & 1 ? 0xff80ff80u : 0x7f807f80u;
                (&lo_hi[0][0][0])[i] = make_uint4(none, none, none, none);
            }
            __syncthreads();
        }
        const int v0 = max(h0 - g.hk, 0), v1 = min(h1 - g.hk, g.hv);
        const int q0 = max(h0 - g.hk - g.hv, 0), q1 = h1 - g.hk - g.hv;
        Heads n{h0, max(k1 - h0, 0), v0, max(v1 - v0, 0), q0, max(q1 - q0, 0)};
        if constexpr (DK != DV) {  // narrower keys: the value rows on their own
            const Heads values{0, 0, n.v0, n.nv, 0, 0};
            n.nv = 0;
            if (values.nv) write_rows<DV, kNoRotation>(a, w, values, true, nullptr, slots);
        }
        if (n.nk + n.nv + n.nq) write_rows<DK, MODE>(a, w, n, false, lo_hi, slots);
        if (!has_page(a, w) && threadIdx.x == 0) {
            raise_device_error(a.err, kErrBounds);
            if (a.lens_out == a.seq_lens) atomicOr(a.ticket, kHole);
        }
        if (bounds && has_page(a, w)) {
            __syncthreads();
            uint4* box = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.bounds) +
                                                  (static_cast<size_t>(w.phys) * g.hk + h0) * 2 * DK);
            const int all = (k1 - h0) * 2 * (DK / 8);
            for (int i = threadIdx.x; i < all; i += kThreads) {
                const bool up = i / (DK / 8) & 1;
                const uint4* own = &lo_hi[0][0][0] + i;
                uint4 x = own[0];
#pragma unroll
                for (int k = 1; k < kWarps; ++k) x = up ? most(x, own[k * all]) : least(x, own[k * all]);
                if (w.old_rows) x = up ? most(x, box[i]) : least(x, box[i]);
                box[i] = x;
            }
        }
    }
    if (a.lens_out == a.seq_lens) {  // grown in place: once every CTA has read the old lengths
        __shared__ uint32_t before;
        __syncthreads();
        if (threadIdx.x == 0) before = atomicAdd(a.ticket, 1u);
        __syncthreads();
        if ((before & ~kHole) != gridDim.x * gridDim.y - 1) return;
        if (threadIdx.x == 0) *a.ticket = 0u;
        write_lens(a, before & kHole);
    }
}

// Rows of heads [h0, h1) of the unit's positions out of the pages.
template <int D>
__device__ __forceinline__ void read_rows(const PagedAppendArgs& a, const Unit& w, const uint8_t* pages, int heads,
                                          int blk, void* out, int h0, int h1) {
    const Spread sp = spread<D>(w.rows);
    const int i = threadIdx.x % (D / 16);
    const uint8_t* block = pages + static_cast<size_t>(w.phys) * heads * blk;
    for (int r = sp.r; r < w.rows; r += sp.rp) {
        const int row_at = (w.off + r) * (D / 2) + 8 * i, scale_at = a.g.P * (D / 2) + 2 * (w.off + r);
        uint4* dst = reinterpret_cast<uint4*>(out) + static_cast<size_t>(w.token + r) * heads * (D / 8) + 2 * i;
#pragma unroll 2
        for (int h = h0 + sp.gh; h < h1; h += sp.hp) {
            const uint2 words = *reinterpret_cast<const uint2*>(block + h * blk + row_at);
            const float s = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(block + h * blk + scale_at));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t word = c ? words.y : words.x;
                float y[8];  // (n + 8 in the low bits of 2^23 + 8 + n)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = (__uint_as_float(0x4b000000u | (word >> (4 * j) & 15u)) - 8388616.f) * s;
                dst[h * (D / 8) + c] = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
            }
        }
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) read_kernel(const PagedAppendArgs a, int per) {
    pdl_wait();
    pdl_trigger();
    const PagedGeom& g = a.g;
    Unit w;
    if (!find_unit(a, blockIdx.x, w)) return;
    if (!has_page(a, w)) {
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        return;
    }
    const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.hk + g.hv);
    if (h0 < g.hk) read_rows<DK>(a, w, a.k_pages, g.hk, g.kblk, a.k_out, h0, min(h1, g.hk));
    const int v0 = max(h0 - g.hk, 0), v1 = h1 - g.hk;
    if (v0 < v1) read_rows<DV>(a, w, a.v_pages, g.hv, g.vblk, a.v_out, v0, v1);
}

using AppendKernel = void (*)(const PagedAppendArgs, int);

cudaError_t launch(AppendKernel kern, PagedAppendArgs a, int heads, int sms, cudaStream_t stream) {
    const PagedGeom& g = a.g;
    const int units = a.cu ? a.n_tokens / g.P + 2 * g.b : g.b;
    // two waves of CTAs even the ends out: 20.7K tokens in 12 runs 68.8 us at 5 CTAs an SM, 65.6 at 8, 63.5 at 12,
    // 64.2 at 16 (single rows: one CTA per SM)
    int parts = ((a.cu ? kPartsPerSm : 1) * sms + units - 1) / units;
    parts = parts < 1 ? 1 : parts > heads ? heads : parts;
    const int per = (heads + parts - 1) / parts;
    const bool apart = a.lens_out && a.lens_out != a.seq_lens;
    a.lens_cta = apart ? units : ~0u;
    const dim3 grid(units + apart, (heads + per - 1) / per);
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, a, per);
}

template <int MODE>
AppendKernel append_of(int dk) {
    return dk == 128 ? append_kernel<128, 128, MODE> : dk == 64 ? append_kernel<64, 64, MODE> : append_kernel<32, 64, MODE>;
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int sms, cudaStream_t stream) {
    const AppendKernel kern = !a.rope          ? append_of<kNoRotation>(a.g.dk)
                              : a.interleaved ? append_of<kInterleaved>(a.g.dk)
                                              : append_of<kHalves>(a.g.dk);
    return launch(kern, a, a.g.hk + a.g.hv + (a.q_new ? a.g.hq : 0), sms, stream);
}

cudaError_t launch_paged_read(const PagedAppendArgs& a, int sms, cudaStream_t stream) {
    const AppendKernel kern = a.g.dk == 128 ? read_kernel<128, 128> : a.g.dk == 64 ? read_kernel<64, 64> : read_kernel<32, 64>;
    return launch(kern, a, a.g.hk + a.g.hv, sms, stream);
}

}  // namespace saga
