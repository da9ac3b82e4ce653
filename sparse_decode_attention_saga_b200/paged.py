"""Host-side driver of the paged 4-bit cache over the C ABI.

``PagedCache`` owns the caller-side state of one layer: the pages, the page
table, the sequences' lengths (all on the device), the pages' key bounds and
the workspace.  ``append`` takes a step's or a prompt's new rows in, ``decode``
attends over every cached position, ``select`` picks the pages a sparse
``decode`` attends to, ``read`` gives rows back as bf16, and ``step`` is one
token of every sequence through append, select and decode.  Handing pages to
sequences (filling ``page_table``) is the caller's, ``grow_table`` a helper for
the plain case.  All compute runs in libsaga.so; calls only enqueue work on the
current (or given) stream and follow lengths, table and lists on the device, so
they can be captured in a CUDA graph (after one uncaptured call of each).  What
a call returns without an output buffer belongs to that stream.  Calls of one
cache share its workspace and are ordered on one stream.
"""
from __future__ import annotations

import torch

from . import _lib


def block_bytes(page_size: int, dim: int) -> int:
    """Bytes of one head's block of a page: rows of dim/2 bytes, then bf16 scales."""
    return page_size * (dim // 2 + 2)


def _need(name, t, dtype, shape, device, rows=False):
    """rows: only the dims after the first have to be contiguous (rows a stride apart)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:  # not a tensor
        pass
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}, got "
                         f"{f'{t.dtype} {tuple(t.shape)}' if isinstance(t, torch.Tensor) else type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    step, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
    if shape[1:2] == (1,):  # a single head's stride means nothing
        head = shape[2]
    if not rows or one != 1 or head != shape[2] or step < shape[1] * shape[2] or step % 8:
        raise ValueError(f"{name} must be contiguous" + (" in each row, rows a multiple of 8 elements apart"
                                                         if rows else ""))


class PagedCache:
    """See the module's text.  ``rope`` is the rotation table [max_pos, rot_dim]
    fp32 (cosines, then sines); None: keys and queries come rotated.  Buffers
    that are not given are allocated: pages uninitialised, the table filled
    with -1, lengths with 0."""

    def __init__(self, batch, h_q, h_k, h_v, head_dim, n_pages, max_pages, page_size=64, v_head_dim=None, rope=None,
                 rot_dim=None, interleaved=False, k_pages=None, v_pages=None, bounds=None, page_table=None,
                 seq_lens=None, device="cuda"):
        self.dv = int(head_dim if v_head_dim is None else v_head_dim)
        self.dims = _lib.paged_dims(batch, h_q, h_k, h_v, head_dim, page_size, max_pages, n_pages, self.dv)
        nbytes = _lib.paged_workspace_bytes(self.dims)
        if nbytes == 0:
            raise _lib.SagaError("saga_paged_workspace_bytes", _lib.SAGA_ERR_UNSUPPORTED)
        given = [t for t in (k_pages, v_pages, bounds, page_table, seq_lens, rope) if t is not None]
        device = given[0].device if given else torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self._elsewhere = device.type == "cuda" and torch.cuda.device_count() > 1  # may not be the current device

        def buffer(name, t, dtype, shape, fill=None):
            if t is None:
                return torch.empty(shape, dtype=dtype, device=device) if fill is None else \
                    torch.full(shape, fill, dtype=dtype, device=device)
            _need(name, t, dtype, shape, device)
            return t

        u8, i32 = torch.uint8, torch.int32
        self.k_pages = buffer("k_pages", k_pages, u8, (n_pages, h_k, block_bytes(page_size, head_dim)))
        self.v_pages = buffer("v_pages", v_pages, u8, (n_pages, h_v, block_bytes(page_size, self.dv)))
        self.bounds = buffer("bounds", bounds, torch.bfloat16, (n_pages, h_k, 2, head_dim), 0)
        self.page_table = buffer("page_table", page_table, i32, (batch, max_pages), -1)
        self.seq_lens = buffer("seq_lens", seq_lens, i32, (batch,), 0)
        self.rope, self._rope = rope, None
        if rope is not None:
            rot = int(rope.shape[-1] if rot_dim is None else rot_dim)
            _need("rope", rope, torch.float32, (rope.shape[0], rot), device)
            self._rope = _lib.SagaRope(rope.data_ptr(), rope.shape[0], rot, int(bool(interleaved)))
        elif rot_dim:
            raise ValueError("rot_dim without a rotation table")
        self.ws = torch.zeros(nbytes, dtype=u8, device=device)
        # (a ctypes field costs as much to read as a check: the shapes once)
        self._batch = batch
        self._k_row, self._v_row, self._q_row = (h_k, head_dim), (h_v, self.dv), (h_q, head_dim)
        self._q, self._out, self._count = (batch, h_q, head_dim), (batch, h_q, self.dv), (batch, h_k)

    def _on(self, stream):
        """The stream to enqueue on: the given one, or the cache's device's current one (its handle)."""
        return torch._C._cuda_getCurrentRawStream(self.device.index) if stream is None else stream

    def _new(self, shape, dtype, stream, zero=False):
        """A tensor made on the stream that the call runs on."""
        make = torch.zeros if zero else torch.empty
        if stream is None:
            return make(shape, dtype=dtype, device=self.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        with torch.cuda.stream(stream):
            return make(shape, dtype=dtype, device=self.device)

    def _call(self, fn, *args, stream):
        if self._elsewhere and self.device.index != torch.cuda.current_device():
            with torch.cuda.device(self.device):
                fn(*args, self._on(stream))
        else:
            fn(*args, self._on(stream))

    def grow_table(self, lens) -> None:
        """Hands pool pages to sequences, enough for lens[b] positions of
        sequence b each (host numbers).  Pages that hold cached positions (the
        first seq_lens[b] of each sequence) stay with it; all others are dealt
        out in order, and the whole table is written.  Waits for the device."""
        d = self.dims
        need = [-(-int(n) // d.page_size) for n in lens]
        if len(need) != d.batch or any(n < 0 for n in lens):
            raise ValueError("the pool or the table does not hold these lengths (one of each sequence, 0 or more)")
        cached, table = self.seq_lens.tolist(), self.page_table.cpu()
        rows = torch.full((d.batch, d.max_pages), -1, dtype=torch.int32)
        held = set()
        for b, n in enumerate(cached):
            if not 0 <= n <= d.max_pages * d.page_size:
                raise ValueError(f"sequence {b}'s cached length is {n}")
            n = -(-n // d.page_size)
            own = table[b, :n].tolist()
            if any(not 0 <= p < d.n_pages for p in own):
                raise ValueError(f"the table does not hold the cached pages of sequence {b}")
            rows[b, :n] = table[b, :n]
            need[b] = max(need[b], n)
            held.update(own)
            cached[b] = n
        free = [p for p in range(d.n_pages) if p not in held]
        if max(need) > d.max_pages or sum(need) - sum(cached) > len(free):
            raise ValueError("the pool or the table does not hold these lengths")
        at = 0
        for b, n in enumerate(need):
            more = n - cached[b]
            rows[b, cached[b]:n] = torch.tensor(free[at:at + more], dtype=torch.int32)
            at += more
        self.page_table.copy_(rows)

    def append(self, k_new, v_new, q_new=None, cu_new=None, q_out=None, lens_out=None, stream=None):
        """New rows ([T, h_k, d], [T, h_v, d_v], queries [T, h_q, d], bf16) at the
        ends of the sequences: rows cu_new[b] .. cu_new[b+1]-1 are sequence b's
        (None: one row each).  Returns the rotated queries (None without
        q_new).  The grown lengths go to seq_lens, or to lens_out if given
        (seq_lens then stays); a sequence grows up to the first row that could
        not be written (its page not in the pool, its position past the rotation
        table: error() tells), and skipped rows' queries are left as they were
        (without q_out: uninitialised)."""
        dev, bf, batch = self.device, torch.bfloat16, self._batch
        T = k_new.shape[0]
        _need("k_new", k_new, bf, (T, *self._k_row), dev, rows=True)
        _need("v_new", v_new, bf, (T, *self._v_row), dev, rows=True)
        if cu_new is not None:
            _need("cu_new", cu_new, torch.int32, (batch + 1,), dev)
        elif T != batch:
            raise ValueError("without cu_new there is one new row per sequence")
        if q_new is not None:
            _need("q_new", q_new, bf, (T, *self._q_row), dev, rows=True)
            if q_out is None:
                q_out = self._new((T, *self._q_row), bf, stream)
            else:
                _need("q_out", q_out, bf, (T, *self._q_row), dev)
        elif q_out is not None:
            raise ValueError("q_out without q_new")
        if lens_out is None:
            lens_out = self.seq_lens
        else:
            _need("lens_out", lens_out, torch.int32, (batch,), dev)
        self._call(_lib.paged_append, self.dims, T, cu_new, self.seq_lens, self.page_table, k_new, v_new, q_new, self._rope,
                   self.k_pages, self.v_pages, self.bounds, q_out, lens_out, self.ws, stream=stream)
        return q_out

    def read(self, n_tokens, cu=None, start=None, k_out=None, v_out=None, stream=None):
        """Rows start[b] .. of each sequence (None: from seq_lens, the rows an
        append with lens_out wrote) as bf16 ([T, h_k, d], [T, h_v, d_v])."""
        dev, bf, batch = self.device, torch.bfloat16, self._batch
        if cu is not None:
            _need("cu", cu, torch.int32, (batch + 1,), dev)
        elif n_tokens != batch:
            raise ValueError("without cu one row of each sequence is read")
        if start is None:
            start = self.seq_lens
        else:
            _need("start", start, torch.int32, (batch,), dev)
        k_shape, v_shape = (n_tokens, *self._k_row), (n_tokens, *self._v_row)
        if k_out is None:
            k_out = self._new(k_shape, bf, stream)
        else:
            _need("k_out", k_out, bf, k_shape, dev)
        if v_out is None:
            v_out = self._new(v_shape, bf, stream)
        else:
            _need("v_out", v_out, bf, v_shape, dev)
        self._call(_lib.paged_read, self.dims, n_tokens, cu, start, self.page_table, self.k_pages, self.v_pages, k_out, v_out,
                   self.ws, stream=stream)
        return k_out, v_out

    def select(self, q, n_sel, first=1, last=1, pages_out=None, count_out=None, stream=None):
        """The pages (at most n_sel, [batch, h_k, n_sel] int32, ascending, and
        their number [batch, h_k]) that each key head's queries attend to: the
        first and last ones and those with the largest bounds on their logits."""
        dev, i32 = self.device, torch.int32
        _need("q", q, torch.bfloat16, self._q, dev)
        if pages_out is None:
            pages_out = self._new((*self._count, n_sel), i32, stream, zero=True)
        else:
            _need("pages_out", pages_out, i32, (*self._count, n_sel), dev)
        if count_out is None:
            count_out = self._new(self._count, i32, stream)
        else:
            _need("count_out", count_out, i32, self._count, dev)
        self._call(_lib.paged_select, self.dims, n_sel, first, last, q, self.bounds, self.seq_lens, self.page_table,
                   pages_out, count_out, self.ws, stream=stream)
        return pages_out, count_out

    def decode(self, q, pages=None, count=None, out=None, stream=None):
        """Attention of one query token per sequence ([batch, h_q, d] bf16,
        rotated) over every cached position, or over select's pages; fp32."""
        dev = self.device
        _need("q", q, torch.bfloat16, self._q, dev)
        if (pages is None) != (count is None):
            raise ValueError("pages and count go together")
        n_sel = 0
        if pages is not None:
            n_sel = pages.shape[-1]
            _need("pages", pages, torch.int32, (*self._count, n_sel), dev)
            _need("count", count, torch.int32, self._count, dev)
        if out is None:
            out = self._new(self._out, torch.float32, stream)
        else:
            _need("out", out, torch.float32, self._out, dev)
        self._call(_lib.paged_decode, self.dims, q, self.k_pages, self.v_pages, self.seq_lens, self.page_table, pages, count,
                   n_sel, out, self.ws, stream=stream)
        return out

    def step(self, k_new, v_new, q_new, n_sel=None, first=1, last=1, out=None, stream=None):
        """One token of every sequence: its rows appended, its query attended
        over the grown cache (over at most n_sel pages per key head if given).
        A sequence whose row could not be written (error() tells) keeps its
        length, and its output row means nothing."""
        q = self.append(k_new, v_new, q_new, stream=stream)
        pages = count = None
        if n_sel is not None:
            pages, count = self.select(q, n_sel, first, last, stream=stream)
        return self.decode(q, pages, count, out, stream=stream)

    def error(self, stream=None) -> int:
        """The sticky device flag (read and cleared; synchronises the stream)."""
        if self._elsewhere and self.device.index != torch.cuda.current_device():
            with torch.cuda.device(self.device):
                return _lib.workspace_error(self.ws, self._on(stream))
        return _lib.workspace_error(self.ws, self._on(stream))
