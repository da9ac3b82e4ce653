// C entries of the paged 4-bit cache (declared in include/saga.h): argument
// validation and dispatch.  Every check happens before anything is enqueued.
#include <cstdint>

#include "paged.h"
#include "saga.h"

using namespace saga;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int make_paged(const saga_paged_dims* d, PagedGeom* out) {
    if (!d) return SAGA_ERR_INVALID_ARG;
    if (d->batch <= 0 || d->h_q <= 0 || d->h_k <= 0 || d->h_v <= 0 || d->head_dim <= 0 || d->v_head_dim < 0 ||
        d->page_size <= 0 || d->max_pages <= 0 || d->n_pages <= 0)
        return SAGA_ERR_INVALID_ARG;
    const int dv = d->v_head_dim ? d->v_head_dim : d->head_dim;
    const bool same = (d->head_dim == 64 || d->head_dim == 128) && dv == d->head_dim;
    if (!same && !(d->head_dim == 32 && dv == 64)) return SAGA_ERR_UNSUPPORTED;
    if (d->h_k != 1 && d->h_k != 2 && d->h_k != 4 && d->h_k != 8) return SAGA_ERR_UNSUPPORTED;
    if (d->h_v % d->h_k || d->h_q % d->h_v || d->h_q / d->h_k > 16 || d->h_q > 128) return SAGA_ERR_UNSUPPORTED;
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64) return SAGA_ERR_UNSUPPORTED;
    if (d->max_pages > (1 << 30) / d->page_size) return SAGA_ERR_UNSUPPORTED;
    if (static_cast<long long>(d->batch) * d->h_q > 65535) return SAGA_ERR_UNSUPPORTED;
    PagedGeom& g = *out;
    g = PagedGeom{};
    g.b = d->batch;
    g.hq = d->h_q;
    g.hk = d->h_k;
    g.hv = d->h_v;
    g.dk = d->head_dim;
    g.dv = dv;
    g.P = d->page_size;
    g.max_pages = d->max_pages;
    g.n_pages = d->n_pages;
    g.Gk = g.hq / g.hk;
    g.Gv = g.hq / g.hv;
    g.nvk = g.hv / g.hk;
    g.kblk = paged_block_bytes(g.P, g.dk);
    g.vblk = paged_block_bytes(g.P, g.dv);
    return SAGA_OK;
}

int check_ws(const PagedGeom& g, const void* ws, size_t ws_bytes) {
    if (!ws || !aligned(ws, 256)) return SAGA_ERR_INVALID_ARG;
    return ws_bytes < paged_workspace_layout(g).total ? SAGA_ERR_WORKSPACE : SAGA_OK;
}

template <typename T>
T* ws_at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

bool ok16(const void* p) { return p && aligned(p, 16); }
bool ok4(const void* p) { return p && aligned(p, 4); }
// rows of `heads` x `dim` elements, `stride` elements apart, read 16 bytes at a time
bool rows_ok(const void* p, int64_t stride, int heads, int dim) {
    return ok16(p) && stride >= static_cast<int64_t>(heads) * dim && stride % 8 == 0;
}

int finish(cudaError_t e) { return e == cudaSuccess ? SAGA_OK : SAGA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t saga_paged_workspace_bytes(const saga_paged_dims* dims) {
    PagedGeom g;
    return make_paged(dims, &g) == SAGA_OK ? paged_workspace_layout(g).total : 0;
}

int saga_paged_append(const saga_paged_dims* dims, int32_t n_tokens, const int32_t* cu_new, const int32_t* seq_lens,
                      const int32_t* page_table, const void* k_new, int64_t k_stride, const void* v_new,
                      int64_t v_stride, const void* q_new, int64_t q_stride, const saga_rope* rope, void* k_pages,
                      void* v_pages, void* bounds, void* q_out, int32_t* lens_out, void* ws, size_t ws_bytes,
                      saga_stream_t stream) {
    PagedGeom g;
    int st = make_paged(dims, &g);
    if (st) return st;
    if (n_tokens < 0 || n_tokens > (1 << 29) || (!cu_new && n_tokens != g.b)) return SAGA_ERR_INVALID_ARG;
    if ((cu_new && !aligned(cu_new, 4)) || !ok4(seq_lens) || !ok4(page_table) || (lens_out && !aligned(lens_out, 4)))
        return SAGA_ERR_INVALID_ARG;
    if (n_tokens) {
        if (!rows_ok(k_new, k_stride, g.hk, g.dk) || !rows_ok(v_new, v_stride, g.hv, g.dv)) return SAGA_ERR_INVALID_ARG;
        if (!q_new != !q_out) return SAGA_ERR_INVALID_ARG;
        if (q_new && (!rows_ok(q_new, q_stride, g.hq, g.dk) || !ok16(q_out))) return SAGA_ERR_INVALID_ARG;
    }
    if (!ok16(k_pages) || !ok16(v_pages) || (bounds && !aligned(bounds, 16))) return SAGA_ERR_INVALID_ARG;
    if (rope) {
        if (!ok16(rope->table) || rope->max_pos <= 0 || rope->rot_dim <= 0) return SAGA_ERR_INVALID_ARG;
        if (rope->rot_dim % 16 || rope->rot_dim > g.dk) return SAGA_ERR_UNSUPPORTED;
    }
    if ((st = check_ws(g, ws, ws_bytes))) return st;
    int sms = 0;
    if ((st = require_device(&sms))) return st;
    const PagedWsLayout L = paged_workspace_layout(g);
    PagedAppendArgs a{};
    a.g = g;
    a.n_tokens = n_tokens;
    a.cu = cu_new;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.k_new = k_new;
    a.v_new = v_new;
    a.q_new = q_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    if (rope) {
        a.rope = rope->table;
        a.max_pos = rope->max_pos;
        a.rot = rope->rot_dim;
        a.interleaved = rope->interleaved != 0;
    }
    a.k_pages = static_cast<uint8_t*>(k_pages);
    a.v_pages = static_cast<uint8_t*>(v_pages);
    a.bounds = bounds;
    a.q_out = q_out;
    a.lens_out = lens_out;
    a.ticket = ws_at<uint32_t>(ws, L.err) + 2;
    a.err = ws_at<uint32_t>(ws, L.err);
    note_launches(1);
    return finish(launch_paged_append(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int saga_paged_read(const saga_paged_dims* dims, int32_t n_tokens, const int32_t* cu, const int32_t* start,
                    const int32_t* page_table, const void* k_pages, const void* v_pages, void* k_out, void* v_out,
                    void* ws, size_t ws_bytes, saga_stream_t stream) {
    PagedGeom g;
    int st = make_paged(dims, &g);
    if (st) return st;
    if (n_tokens < 0 || n_tokens > (1 << 29) || (!cu && n_tokens != g.b)) return SAGA_ERR_INVALID_ARG;
    if ((cu && !aligned(cu, 4)) || !ok4(start) || !ok4(page_table)) return SAGA_ERR_INVALID_ARG;
    if (!ok16(k_pages) || !ok16(v_pages)) return SAGA_ERR_INVALID_ARG;
    if (n_tokens && (!ok16(k_out) || !ok16(v_out))) return SAGA_ERR_INVALID_ARG;
    if ((st = check_ws(g, ws, ws_bytes))) return st;
    int sms = 0;
    if ((st = require_device(&sms))) return st;
    if (n_tokens == 0) return SAGA_OK;
    PagedAppendArgs a{};
    a.g = g;
    a.n_tokens = n_tokens;
    a.cu = cu;
    a.seq_lens = start;
    a.page_table = page_table;
    a.k_pages = static_cast<uint8_t*>(const_cast<void*>(k_pages));
    a.v_pages = static_cast<uint8_t*>(const_cast<void*>(v_pages));
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = ws_at<uint32_t>(ws, paged_workspace_layout(g).err);
    note_launches(1);
    return finish(launch_paged_read(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int saga_paged_select(const saga_paged_dims* dims, int32_t n_sel, int32_t n_first, int32_t n_last, const void* q,
                      const void* bounds, const int32_t* seq_lens, const int32_t* page_table, int32_t* sel_pages,
                      int32_t* sel_cnt, void* ws, size_t ws_bytes, saga_stream_t stream) {
    PagedGeom g;
    int st = make_paged(dims, &g);
    if (st) return st;
    if (n_sel <= 0 || n_first < 0 || n_last < 0 || n_first > n_sel || n_last > n_sel - n_first)
        return SAGA_ERR_INVALID_ARG;
    if (!ok16(q) || !ok16(bounds) || !ok4(seq_lens) || !ok4(page_table) || !ok4(sel_pages) || !ok4(sel_cnt))
        return SAGA_ERR_INVALID_ARG;
    if (g.max_pages > kPagedMaxSelectPages) return SAGA_ERR_UNSUPPORTED;
    if ((st = check_ws(g, ws, ws_bytes))) return st;
    int sms = 0;
    if ((st = require_device(&sms))) return st;
    const PagedWsLayout L = paged_workspace_layout(g);
    PagedSelectArgs a{};
    a.g = g;
    a.n_sel = n_sel;
    a.n_first = n_first;
    a.n_last = n_last;
    a.q = q;
    a.bounds = bounds;
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.sel = sel_pages;
    a.sel_cnt = sel_cnt;
    a.scores = ws_at<float>(ws, L.scores);
    a.keys = ws_at<unsigned long long>(ws, L.keys);
    a.tickets = ws_at<uint32_t>(ws, L.sel_tickets);
    a.row_max = ws_at<uint32_t>(ws, L.row_max);
    a.err = ws_at<uint32_t>(ws, L.err);
    note_launches(1);
    return finish(launch_paged_select(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int saga_paged_decode(const saga_paged_dims* dims, const void* q, const void* k_pages, const void* v_pages,
                      const int32_t* seq_lens, const int32_t* page_table, const int32_t* sel_pages,
                      const int32_t* sel_cnt, int32_t n_sel, float* out, void* ws, size_t ws_bytes,
                      saga_stream_t stream) {
    PagedGeom g;
    int st = make_paged(dims, &g);
    if (st) return st;
    if (!ok16(q) || !ok16(k_pages) || !ok16(v_pages) || !ok4(seq_lens) || !ok4(page_table) || !ok16(out))
        return SAGA_ERR_INVALID_ARG;
    if (!sel_pages != !sel_cnt) return SAGA_ERR_INVALID_ARG;
    if (sel_pages && (!aligned(sel_pages, 4) || !aligned(sel_cnt, 4) || n_sel <= 0)) return SAGA_ERR_INVALID_ARG;
    if ((st = check_ws(g, ws, ws_bytes))) return st;
    int sms = 0;
    if ((st = require_device(&sms))) return st;
    const PagedWsLayout L = paged_workspace_layout(g);
    PagedDecodeArgs a{};
    a.g = g;
    a.q = q;
    a.k_pages = static_cast<const uint8_t*>(k_pages);
    a.v_pages = static_cast<const uint8_t*>(v_pages);
    a.seq_lens = seq_lens;
    a.page_table = page_table;
    a.sel = sel_pages;
    a.sel_cnt = sel_cnt;
    a.n_sel = sel_pages ? n_sel : 0;
    a.out = out;
    a.records = ws_at<float>(ws, L.records);
    a.firsts = ws_at<float>(ws, L.firsts);
    a.tickets = ws_at<uint32_t>(ws, L.tickets);
    a.err = ws_at<uint32_t>(ws, L.err);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kernel_event(false, s);
    const cudaError_t e = g.dk == 128  ? launch_paged_decode_d128(a, sms, s)
                          : g.dk == 64 ? launch_paged_decode_d64(a, sms, s)
                                       : launch_paged_decode_d32(a, sms, s);
    kernel_event(true, s);
    note_launches(1);
    return finish(e);
}

}  // extern "C"
