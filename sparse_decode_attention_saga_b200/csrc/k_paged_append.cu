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
// a page's key bounds: no atomics on global memory, results do not depend on
// the order of CTAs.  Rows are handled by d/8 lanes with 16-byte loads.
#include <cuda_bf16.h>

#include "paged.h"
#include "saga_device.cuh"

namespace saga {

namespace {

constexpr int kThreads = 256;

// Where a work unit's tokens are: sequence, logical page, rows [first, first +
// rows) of positions, and the index of the first one among the new tokens.
struct Unit {
    int seq, page, off, rows, token, phys;
    bool old_rows;  // the page held rows of the sequence before
};

// Units of sequence i start at cu[i]/P + 2i: a run of n tokens touches at
// most n/P + 2 pages, so that the ranges do not overlap.
__device__ __forceinline__ int unit_start(const int32_t* cu, int i, int P) { return max(cu[i], 0) / P + 2 * i; }

__device__ __forceinline__ bool find_unit(const PagedAppendArgs& a, int u, Unit& w) {
    const PagedGeom& g = a.g;
    const int lane = threadIdx.x & 31;
    int seq, j, n, t0;
    if (!a.cu) {
        if (u >= g.b) return false;
        seq = u, j = 0, n = 1, t0 = u;
    } else {
        int lo = 0, len = g.b;
        while (true) {  // 32-ary search for the last sequence that starts at or before u
            const int step = (len + 31) / 32;
            const bool in = lane * step < len && unit_start(a.cu, lo + lane * step, g.P) <= u;
            const int c = __popc(__ballot_sync(0xffffffffu, in));
            if (c == 0) return false;
            lo += (c - 1) * step;
            len = min(step, len - (c - 1) * step);
            if (step == 1) break;
        }
        seq = lo;
        t0 = a.cu[seq];
        n = a.cu[seq + 1] - t0;
        j = u - unit_start(a.cu, seq, g.P);
        if (t0 < 0 || n < 0 || t0 > a.n_tokens - n) {
            if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
            return false;
        }
    }
    if (n == 0) return false;
    const int len0 = a.seq_lens[seq];
    if (len0 < 0 || len0 > g.max_pages * g.P) {
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        return false;
    }
    const int page = len0 / g.P + j;
    const int first = max(len0, page * g.P), last = min(len0 + n, (page + 1) * g.P);
    if (first >= last) return false;
    const int phys = page < g.max_pages ? a.page_table[static_cast<size_t>(seq) * g.max_pages + page] : -1;
    if (phys < 0 || phys >= g.n_pages) {  // no such page: its rows are not written
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        return false;
    }
    w.seq = seq;
    w.page = page;
    w.off = first - page * g.P;
    w.rows = last - first;
    w.token = t0 + (first - len0);
    w.phys = phys;
    w.old_rows = len0 > page * g.P;
    return true;
}

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

// Dims 8c .. 8c+7 of a row, rotated, as bf16.
__device__ __forceinline__ uint4 rotated8(const __nv_bfloat16* row, int c, const float* cs, int rot, bool interleaved) {
    const uint4 raw = *reinterpret_cast<const uint4*>(row + 8 * c);
    if (8 * c >= rot) return raw;
    const int half = rot / 2;
    float x[8], y[8];
    unpack8(raw, x);
    if (interleaved) {
        const float4 co = *reinterpret_cast<const float4*>(cs + 4 * c);
        const float4 si = *reinterpret_cast<const float4*>(cs + half + 4 * c);
        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = dot2_rn(x[2 * i], cc[i], x[2 * i + 1], -ss[i]);
            y[2 * i + 1] = dot2_rn(x[2 * i + 1], cc[i], x[2 * i], ss[i]);
        }
    } else {
        const bool upper = 8 * c >= half;
        const int i0 = upper ? 8 * c - half : 8 * c;
        float o[8];
        unpack8(*reinterpret_cast<const uint4*>(row + (upper ? i0 : i0 + half)), o);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 co = *reinterpret_cast<const float4*>(cs + i0 + 4 * h);
            const float4 si = *reinterpret_cast<const float4*>(cs + half + i0 + 4 * h);
            const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[4 * h + i] = dot2_rn(x[4 * h + i], cc[i], o[4 * h + i], upper ? ss[i] : -ss[i]);
        }
    }
    return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// How a unit's rows and heads are spread over the CTA's groups of d/8 lanes:
// rp groups side by side on rows, the rest on heads.
struct Spread {
    int gr, gh, rp, hp;
};
template <int D>
__device__ __forceinline__ Spread spread(int rows) {
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    int rp = 1;
    while (rp < rows && rp < GROUPS) rp *= 2;
    const int grp = threadIdx.x / LPR;
    return Spread{grp % rp, grp / rp, rp, GROUPS / rp};
}

// One head group of 8 values to 4 bits: the row's scale (all its lanes) and
// the word of n + 8, dim 8c + i in bits 4i .. 4i+3.
template <int LPR>
__device__ __forceinline__ uint32_t quantise8(const float (&y)[8], __nv_bfloat16& scale) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    scale = __float2bfloat16_rn(m / 7.0f);
    const float s = __bfloat162float(scale);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float n = s > 0.f ? fminf(fmaxf(rintf(y[i] / s), -7.f), 7.f) : 0.f;
        word |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * i);
    }
    return word;
}

// Key or value rows of heads [h0, h1) of the unit into the pages.
template <int D, bool KEYS>
__device__ __forceinline__ void write_rows(const PagedAppendArgs& a, const Unit& w, int h0, int h1,
                                           uint32_t (*lo_hi)[2][D]) {
    constexpr int LPR = D / 8;
    const PagedGeom& g = a.g;
    const Spread sp = spread<D>(w.rows);
    const int c = threadIdx.x % LPR;
    const int heads = KEYS ? g.hk : g.hv, blk = KEYS ? g.kblk : g.vblk;
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(KEYS ? a.k_new : a.v_new);
    const long long stride = KEYS ? a.k_stride : a.v_stride;
    uint8_t* pages = KEYS ? a.k_pages : a.v_pages;
    for (int hb = h0; hb < h1; hb += sp.hp) {
        const int h = hb + sp.gh;
        float mn[8], mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mn[i] = kInf, mx[i] = -kInf;
        for (int rb = 0; rb < w.rows; rb += sp.rp) {
            const int r = rb + sp.gr;
            const bool live = h < h1 && r < w.rows;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live) {
                const __nv_bfloat16* row = src + (w.token + r) * stride + h * D;
                const int pos = w.page * g.P + w.off + r;
                if (KEYS && a.rope) v = rotated8(row, c, a.rope + static_cast<size_t>(pos) * a.rot, a.rot, a.interleaved);
                else v = *reinterpret_cast<const uint4*>(row + 8 * c);
            }
            float y[8];
            unpack8(v, y);
            __nv_bfloat16 scale;
            const uint32_t word = quantise8<LPR>(y, scale);
            if (live) {
                uint8_t* block = pages + (static_cast<size_t>(w.phys) * heads + h) * blk;
                reinterpret_cast<uint32_t*>(block + (w.off + r) * (D / 2))[c] = word;
                if (c == 0) reinterpret_cast<__nv_bfloat16*>(block + g.P * (D / 2))[w.off + r] = scale;
                if (KEYS) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) mn[i] = fminf(mn[i], y[i]), mx[i] = fmaxf(mx[i], y[i]);
                }
            }
        }
        if (KEYS && a.bounds && h < h1 && sp.gr < w.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                atomicMin(&lo_hi[h - h0][0][8 * c + i], float_to_key(mn[i]));
                atomicMax(&lo_hi[h - h0][1][8 * c + i], float_to_key(mx[i]));
            }
        }
    }
}

// Heads are numbered keys, values, queries; CTA y takes [y*per, (y+1)*per).
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) append_kernel(const PagedAppendArgs a, int per) {
    __shared__ uint32_t lo_hi[8][2][DK];
    pdl_wait();  // lengths, tables and pages may be the previous kernels' results
    pdl_trigger();
    const PagedGeom& g = a.g;
    Unit w;
    bool live = find_unit(a, blockIdx.x, w);
    if (live && a.rope && w.page * g.P + w.off + w.rows > a.max_pos) {  // positions past the table: not written
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        live = false;
    }
    if (live) {
        const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.hk + g.hv + (a.q_new ? g.hq : 0));
        const int k1 = min(h1, g.hk);
        const bool bounds = a.bounds && h0 < k1;
        if (bounds) {
            for (int i = threadIdx.x; i < (k1 - h0) * 2 * DK; i += kThreads)
                (&lo_hi[0][0][0])[i] = (i / DK) & 1 ? 0u : 0xffffffffu;
            __syncthreads();
        }
        if (h0 < k1) write_rows<DK, true>(a, w, h0, k1, lo_hi);
        const int v0 = max(h0 - g.hk, 0), v1 = min(h1 - g.hk, g.hv);
        if (v0 < v1) write_rows<DV, false>(a, w, v0, v1, nullptr);
        const int q0 = max(h0 - g.hk - g.hv, 0), q1 = h1 - g.hk - g.hv;
        if (q0 < q1) {
            constexpr int LPR = DK / 8;
            const Spread sp = spread<DK>(w.rows);
            const int c = threadIdx.x % LPR;
            for (int h = q0 + sp.gh; h < q1; h += sp.hp)
                for (int r = sp.gr; r < w.rows; r += sp.rp) {
                    const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(a.q_new) +
                                               (w.token + r) * a.q_stride + h * DK;
                    const int pos = w.page * g.P + w.off + r;
                    const uint4 v = a.rope ? rotated8(row, c, a.rope + static_cast<size_t>(pos) * a.rot, a.rot, a.interleaved)
                                           : *reinterpret_cast<const uint4*>(row + 8 * c);
                    reinterpret_cast<uint4*>(a.q_out)[(static_cast<size_t>(w.token + r) * g.hq + h) * LPR + c] = v;
                }
        }
        if (bounds) {
            __syncthreads();
            __nv_bfloat16* box = reinterpret_cast<__nv_bfloat16*>(a.bounds) +
                                 (static_cast<size_t>(w.phys) * g.hk + h0) * 2 * DK;
            for (int i = threadIdx.x; i < (k1 - h0) * 2 * DK; i += kThreads) {
                float x = key_to_float((&lo_hi[0][0][0])[i]);
                if (w.old_rows) {
                    const float old = __bfloat162float(box[i]);
                    x = (i / DK) & 1 ? fmaxf(x, old) : fminf(x, old);
                }
                box[i] = __float2bfloat16_rn(x);
            }
        }
    }
    // The grown lengths, once every CTA has read the old ones.
    if (a.lens_out) {
        __shared__ bool last;
        __syncthreads();
        if (threadIdx.x == 0) {
            const unsigned n = gridDim.x * gridDim.y;
            last = atomicAdd(a.ticket, 1u) == n - 1;
            if (last) *a.ticket = 0u;
        }
        __syncthreads();
        if (last)
            for (int i = threadIdx.x; i < g.b; i += kThreads) {
                const int n = a.cu ? max(a.cu[i + 1] - a.cu[i], 0) : 1;
                a.lens_out[i] = min(a.seq_lens[i] + n, g.max_pages * g.P);
            }
    }
}

// Rows [h0, h1) of heads of the unit's positions out of the pages.
template <int D>
__device__ __forceinline__ void read_rows(const PagedAppendArgs& a, const Unit& w, const uint8_t* pages, int heads,
                                          int blk, void* out, int h0, int h1) {
    constexpr int LPR = D / 8;
    const Spread sp = spread<D>(w.rows);
    const int c = threadIdx.x % LPR;
    for (int h = h0 + sp.gh; h < h1; h += sp.hp)
        for (int r = sp.gr; r < w.rows; r += sp.rp) {
            const uint8_t* block = pages + (static_cast<size_t>(w.phys) * heads + h) * blk;
            const uint32_t word = reinterpret_cast<const uint32_t*>(block + (w.off + r) * (D / 2))[c];
            const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(block + a.g.P * (D / 2))[w.off + r]);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = static_cast<float>(static_cast<int>((word >> (4 * i)) & 15u) - 8) * s;
            reinterpret_cast<uint4*>(out)[(static_cast<size_t>(w.token + r) * heads + h) * LPR + c] =
                make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
        }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) read_kernel(const PagedAppendArgs a, int per) {
    pdl_wait();
    pdl_trigger();
    const PagedGeom& g = a.g;
    Unit w;
    if (!find_unit(a, blockIdx.x, w)) return;
    const int h0 = blockIdx.y * per, h1 = min(h0 + per, g.hk + g.hv);
    if (h0 < g.hk) read_rows<DK>(a, w, a.k_pages, g.hk, g.kblk, a.k_out, h0, min(h1, g.hk));
    const int v0 = max(h0 - g.hk, 0), v1 = h1 - g.hk;
    if (v0 < v1) read_rows<DV>(a, w, a.v_pages, g.hv, g.vblk, a.v_out, v0, v1);
}

using AppendKernel = void (*)(const PagedAppendArgs, int);

cudaError_t launch(AppendKernel k64, AppendKernel k128, AppendKernel k32, const PagedAppendArgs& a, int heads, int sms,
                   cudaStream_t stream) {
    const PagedGeom& g = a.g;
    const int units = a.cu ? a.n_tokens / g.P + 2 * g.b : g.b;
    // few units: the heads are split over several CTAs each, down to one head
    int parts = (4 * sms + units - 1) / units;
    parts = parts < 1 ? 1 : parts > heads ? heads : parts;
    const int per = (heads + parts - 1) / parts;
    const dim3 grid(units, (heads + per - 1) / per);
    return launch_dependent(g.dk == 128 ? k128 : g.dk == 64 ? k64 : k32, grid, dim3(kThreads), 0, stream, a, per);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int sms, cudaStream_t stream) {
    return launch(append_kernel<64, 64>, append_kernel<128, 128>, append_kernel<32, 64>, a,
                  a.g.hk + a.g.hv + (a.q_new ? a.g.hq : 0), sms, stream);
}

cudaError_t launch_paged_read(const PagedAppendArgs& a, int sms, cudaStream_t stream) {
    return launch(read_kernel<64, 64>, read_kernel<128, 128>, read_kernel<32, 64>, a, a.g.hk + a.g.hv, sms, stream);
}

}  // namespace saga
