// Attention of one query token per sequence over the paged 4-bit cache.
//
//   l_j = q . n^k_j s^k_j / sqrt(d),   out = sum_j softmax(l)_j n^v_j s^v_j
//
// over every cached position, or over the positions of the listed pages of
// each key head.  One pass with the running maximum and sum.
#include <cuda_bf16.h>

#include "paged.h"
#include "saga_device.cuh"

namespace saga {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One CTA per (query head, sequence), a warp per position.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) decode_kernel(const PagedDecodeArgs a) {
    __shared__ float part[kWarps][DV + 2];
    pdl_wait();
    pdl_trigger();
    const PagedGeom& g = a.g;
    const int i = blockIdx.x, b = blockIdx.y, kh = i / g.Gk, vh = i / g.Gv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int KB = DK / 64, VB = DV / 64;  // bytes of a row per lane (32-dim keys: half the lanes)
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(b) * g.hq + i) * DK;
    float qr[KB > 0 ? 2 * KB : 2] = {};
    const bool klane = lane < DK / 2;
    constexpr int KN = KB > 0 ? KB : 1;
    if (klane)
#pragma unroll
        for (int c = 0; c < 2 * KN; ++c) qr[c] = __bfloat162float(q[2 * KN * lane + c]);
    int len = a.seq_lens[b];
    if (len < 0 || len > g.max_pages * g.P) {
        if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
        len = len < 0 ? 0 : g.max_pages * g.P;
    }
    const int np = (len + g.P - 1) / g.P;
    int entries = np;
    const int32_t* sel = nullptr;
    if (a.sel) {
        const int row = b * g.hk + kh;
        sel = a.sel + static_cast<size_t>(row) * a.n_sel;
        entries = a.sel_cnt[row];
        if (entries < 0 || entries > a.n_sel) {
            if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
            entries = 0;
        }
    }
    const float scale = rsqrtf(static_cast<float>(DK));
    float m = -kInf, l = 0.f, o[2 * VB] = {};
    for (int e = 0; e < entries; ++e) {
        const int page = sel ? sel[e] : e;
        const int phys = page >= 0 && page < np ? a.page_table[static_cast<size_t>(b) * g.max_pages + page] : -1;
        if (phys < 0 || phys >= g.n_pages) {
            if (threadIdx.x == 0) raise_device_error(a.err, kErrBounds);
            continue;
        }
        const int rows = min(g.P, len - page * g.P);
        const uint8_t* kb = a.k_pages + (static_cast<size_t>(phys) * g.hk + kh) * g.kblk;
        const uint8_t* vb = a.v_pages + (static_cast<size_t>(phys) * g.hv + vh) * g.vblk;
        for (int r = warp; r < rows; r += kWarps) {
            float s = 0.f;
            if (klane)
#pragma unroll
                for (int c = 0; c < KN; ++c) {
                    const uint32_t u = kb[r * (DK / 2) + KN * lane + c];
                    s += qr[2 * c] * static_cast<float>(static_cast<int>(u & 15u) - 8) +
                         qr[2 * c + 1] * static_cast<float>(static_cast<int>(u >> 4) - 8);
                }
            s = warp_sum(s) * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(kb + g.P * (DK / 2))[r]) * scale;
            const float mn = fmaxf(m, s);
            const float f = expf(m - mn), p = expf(s - mn);
            m = mn;
            l = l * f + p;
            const float pv = p * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(vb + g.P * (DV / 2))[r]);
#pragma unroll
            for (int c = 0; c < VB; ++c) {
                const uint32_t u = vb[r * (DV / 2) + VB * lane + c];
                o[2 * c] = o[2 * c] * f + pv * static_cast<float>(static_cast<int>(u & 15u) - 8);
                o[2 * c + 1] = o[2 * c + 1] * f + pv * static_cast<float>(static_cast<int>(u >> 4) - 8);
            }
        }
    }
    if (lane == 0) part[warp][0] = m, part[warp][1] = l;
#pragma unroll
    for (int c = 0; c < 2 * VB; ++c) part[warp][2 + 2 * VB * lane + c] = o[c];
    __syncthreads();
    for (int d = threadIdx.x; d < DV; d += kThreads) {
        float M = -kInf, L = 0.f, x = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part[w][0]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = part[w][0] == -kInf ? 0.f : expf(part[w][0] - M);
            L += f * part[w][1];
            x += f * part[w][2 + d];
        }
        a.out[(static_cast<size_t>(b) * g.hq + i) * DV + d] = L > 0.f ? x / L : 0.f;
    }
}

}  // namespace

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int sms, cudaStream_t stream) {
    (void)sms;
    const dim3 grid(a.g.hq, a.g.b);
    auto kern = a.g.dk == 128 ? decode_kernel<128, 128> : a.g.dk == 64 ? decode_kernel<64, 64> : decode_kernel<32, 64>;
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace saga
