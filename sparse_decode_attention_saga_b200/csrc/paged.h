// The paged 4-bit cache: shapes, formats, workspace layout and the launch
// interface of its kernels (internal to libsaga.so).
#pragma once

#include <cuda_runtime.h>

#include "saga_kernels.h"
#include "saga_params.h"

namespace saga {

// Grid of the paged decode kernel and its warps per CTA at most (they size
// the partial records).
constexpr int kPagedMaxCtas = 160;
constexpr int kPagedWarps = 16;
// Pages of a sequence that the selection takes at most (their bits in shared memory).
constexpr int kPagedMaxSelectPages = 1 << 18;
struct PagedGeom {
    int b, hq, hk, hv, dk, dv;
    int P;          // positions per page: 16, 32 or 64
    int max_pages;  // columns of the page table
    int n_pages;    // pages in the pool
    int Gk, Gv;     // query heads per key head / per value head
    int nvk;        // value heads per key head
    int kblk, vblk; // bytes of one head's block: P rows of d/2 bytes, then P bf16 scales
};

SAGA_HD constexpr int paged_block_bytes(int P, int d) { return P * (d / 2 + 2); }

// Offsets up to `scores` depend on the batch, the heads and their dims only;
// the tickets are zero on entry and left at zero.
struct PagedWsLayout {
    size_t err;      // uint32 sticky flag; word 2: the append's ticket (256-byte header)
    size_t tickets;  // uint32 [b*hv]
    size_t records;  // float  [kPagedMaxCtas][2][columns of a work row * (2 + dv)]
    size_t firsts;   // float  [kPagedMaxCtas][kPagedWarps][columns of a work row * (2 + dv)]
    size_t sel_tickets;  // uint32 [b*hk]
    size_t row_max;      // uint32 [b*hk]  largest size of a row's scores (bits of a float; zero on entry and exit)
    size_t scores;   // float  [b*hk][max_pages]
    size_t keys;     // uint64 [b*hk][max_pages]
    size_t total;
};

// How the decode kernel cuts a key head's value heads into work rows: NVU of
// them, whose query heads stand in columns of the tensor-core tiles, CW
// columns to a value head.
struct PagedRowShape {
    int CW, NVU;
};
SAGA_HD PagedRowShape paged_row_shape(const PagedGeom& g) {
    const int CW = g.Gv <= 4 ? 4 : g.Gv <= 8 ? 8 : 16;
    // four value heads only where their accumulators fit in registers
    const int most = CW == 16 ? 1 : CW == 8 ? 2 : g.dv == 64 ? 4 : 2;
    int NVU = 1;
    while (NVU * 2 <= most && g.nvk % (NVU * 2) == 0) NVU *= 2;
    return PagedRowShape{CW, NVU};
}

inline PagedWsLayout paged_workspace_layout(const PagedGeom& g) {
    PagedWsLayout w{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    w.err = take(256);
    w.tickets = take(static_cast<size_t>(g.b) * g.hv * sizeof(uint32_t));
    w.sel_tickets = take(static_cast<size_t>(g.b) * g.hk * sizeof(uint32_t));
    w.row_max = take(static_cast<size_t>(g.b) * g.hk * sizeof(uint32_t));
    const PagedRowShape shape = paged_row_shape(g);
    const size_t rec = static_cast<size_t>(shape.NVU) * shape.CW * (2 + g.dv) * sizeof(float);
    w.records = take(kPagedMaxCtas * 2 * rec);
    w.firsts = take(static_cast<size_t>(kPagedMaxCtas) * kPagedWarps * rec);
    w.scores = take(static_cast<size_t>(g.b) * g.hk * g.max_pages * sizeof(float));
    w.keys = take(static_cast<size_t>(g.b) * g.hk * g.max_pages * sizeof(unsigned long long));
    w.total = off;
    return w;
}

// Rotation, rounding to 4 bits and the write into the pages; with `read` the
// way back (rows out of the pages as bf16).
struct PagedAppendArgs {
    PagedGeom g;
    int n_tokens;
    const int32_t* cu;        // [b+1], null: one token per sequence
    const int32_t* seq_lens;  // [b]
    const int32_t* page_table;
    const void *k_new, *v_new, *q_new;  // bf16 rows, strides in elements
    long long k_stride, v_stride, q_stride;
    const float* rope;  // [max_pos][rot] (cosines, then sines), null: no rotation
    int max_pos, rot, interleaved;
    uint8_t *k_pages, *v_pages;
    void* bounds;      // nullable
    void* q_out;       // [n_tokens][hq][dk]
    void *k_out, *v_out;  // read: [n_tokens][hk][dk], [n_tokens][hv][dv]
    int32_t* lens_out;  // nullable; may be seq_lens
    uint32_t* ticket;  // zero on entry and exit
    uint32_t lens_cta;  // column of CTAs that writes lengths apart from seq_lens (~0: none; set by the launch)
    uint32_t* err;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedAppendArgs& a, int sms, cudaStream_t stream);

struct PagedSelectArgs {
    PagedGeom g;
    int n_sel, n_first, n_last;
    const void* q;
    const void* bounds;
    const int32_t* seq_lens;
    const int32_t* page_table;
    int32_t* sel;      // [b][hk][n_sel]
    int32_t* sel_cnt;  // [b][hk]
    float* scores;
    unsigned long long* keys;
    uint32_t* tickets;
    uint32_t* row_max;
    uint32_t* err;
};
cudaError_t launch_paged_select(const PagedSelectArgs& a, int sms, cudaStream_t stream);

struct PagedDecodeArgs {
    PagedGeom g;
    const void* q;
    const uint8_t *k_pages, *v_pages;
    const int32_t* seq_lens;
    const int32_t* page_table;
    const int32_t* sel;      // nullable [b][hk][n_sel]
    const int32_t* sel_cnt;  // [b][hk] with sel
    int n_sel;
    float* out;
    float* records;
    float* firsts;
    uint32_t* tickets;
    uint32_t* err;
};
// by key head dim (one source file each)
cudaError_t launch_paged_decode_d32(const PagedDecodeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_paged_decode_d64(const PagedDecodeArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_paged_decode_d128(const PagedDecodeArgs& a, int sms, cudaStream_t stream);

}  // namespace saga
