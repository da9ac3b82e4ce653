"""The paged cache's refusals and host logic (CPU): every bad argument is
turned down before anything is enqueued, by the C entries with a status and
by PagedCache with a ValueError."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_decode_attention_saga_b200 import _lib
from sparse_decode_attention_saga_b200 import paged
from sparse_decode_attention_saga_b200.paged import PagedCache, block_bytes

from tests import paged_reference as ref

INVALID, UNSUPPORTED, WORKSPACE = _lib.SAGA_ERR_INVALID_ARG, _lib.SAGA_ERR_UNSUPPORTED, _lib.SAGA_ERR_WORKSPACE
NO_DEVICE = (_lib.SAGA_ERR_DEVICE, _lib.SAGA_ERR_CUDA)
BASE = dict(batch=2, h_q=32, h_k=4, h_v=8, head_dim=64, page_size=64, max_pages=10, n_pages=30, v_head_dim=0)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def dims(**kw):
    b = dict(BASE, **kw)
    return _lib.paged_dims(b["batch"], b["h_q"], b["h_k"], b["h_v"], b["head_dim"], b["page_size"], b["max_pages"],
                           b["n_pages"], b["v_head_dim"])


class Ws:
    def __init__(self, d):
        self.n = _lib.paged_workspace_bytes(d)
        self.buf = torch.zeros(self.n + 512, dtype=torch.uint8)
        self.p = (self.buf.data_ptr() + 255) // 256 * 256


@pytest.mark.parametrize("bad", [dict(batch=0), dict(h_q=0), dict(h_k=-1), dict(h_v=0), dict(head_dim=0),
                                 dict(page_size=0), dict(max_pages=0), dict(n_pages=0), dict(v_head_dim=-64)])
def test_invalid_dims(lib, bad):
    d = dims(**bad)
    assert _lib.paged_workspace_bytes(d) == 0
    assert lib.saga_paged_decode(ctypes.byref(d), 16, 16, 16, 16, 16, None, None, 0, 16, 256, 1 << 30, None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=32), dict(v_head_dim=128), dict(h_k=3, h_v=6, h_q=6), dict(h_k=16, h_v=16),
    dict(h_v=2), dict(h_v=6), dict(h_q=20), dict(h_q=128, h_k=4), dict(h_q=256, h_k=8, h_v=32), dict(page_size=8),
    dict(page_size=128), dict(page_size=48), dict(max_pages=(1 << 24) + 1), dict(batch=2048)])
def test_unsupported_dims(lib, bad):
    d = dims(**bad)
    assert _lib.paged_workspace_bytes(d) == 0
    assert lib.saga_paged_select(ctypes.byref(d), 4, 0, 0, 16, 16, 16, 16, 16, 16, 256, 1 << 30, None) == UNSUPPORTED


@pytest.mark.parametrize("ok", [dict(), dict(head_dim=128), dict(head_dim=32, v_head_dim=64), dict(page_size=16),
                                dict(page_size=32), dict(h_q=16, h_k=1, h_v=8), dict(h_q=12, h_k=2, h_v=6),
                                dict(h_q=16, h_k=1, h_v=1, head_dim=32, v_head_dim=64)])
def test_supported_dims_have_a_workspace(ok):
    assert _lib.paged_workspace_bytes(dims(**ok)) > 0


def rope(table=16, max_pos=100, rot=64, inter=0):
    return _lib.SagaRope(table, max_pos, rot, inter)


def append_args(w, **kw):
    a = dict(n=2, cu=None, lens=16, table=16, k=16, ks=256, v=16, vs=512, q=16, qs=2048, rope=rope(), kp=16, vp=16,
             bounds=16, qo=16, lo=16, ws=w.p, bytes=w.n)
    a.update(kw)
    a["rope"] = None if a["rope"] is None else ctypes.byref(a["rope"])
    return list(a.values()) + [None]


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), INVALID), (dict(n=3), INVALID), (dict(n=(1 << 30) + 1, cu=16), INVALID), (dict(cu=18), INVALID),
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(table=2), INVALID), (dict(k=None), INVALID),
    (dict(k=8), INVALID), (dict(v=None), INVALID), (dict(ks=255), INVALID), (dict(ks=260), INVALID),
    (dict(vs=504), INVALID), (dict(qs=2040), INVALID), (dict(qs=2052), INVALID), (dict(q=None), INVALID),
    (dict(qo=None), INVALID), (dict(qo=24), INVALID), (dict(kp=None), INVALID), (dict(vp=40), INVALID),
    (dict(bounds=8), INVALID), (dict(lo=2), INVALID), (dict(ws=None), INVALID), (dict(rope=rope(None)), INVALID),
    (dict(rope=rope(20)), INVALID), (dict(rope=rope(max_pos=0)), INVALID), (dict(rope=rope(rot=0)), INVALID),
    (dict(rope=rope(rot=24)), UNSUPPORTED), (dict(rope=rope(rot=80)), UNSUPPORTED),
])
def test_append_refuses(lib, bad, code):
    d = dims()
    w = Ws(d)
    assert lib.saga_paged_append(ctypes.byref(d), *append_args(w, **bad)) == code


def test_workspaces_are_checked(lib):
    d = dims()
    w = Ws(d)
    assert lib.saga_paged_append(ctypes.byref(d), *append_args(w, bytes=w.n - 1)) == WORKSPACE
    assert lib.saga_paged_append(ctypes.byref(d), *append_args(w, ws=w.p + 16)) == INVALID
    assert lib.saga_paged_read(ctypes.byref(d), 2, None, 16, 16, 16, 16, 16, 16, w.p, w.n - 1, None) == WORKSPACE
    assert lib.saga_paged_select(ctypes.byref(d), 4, 0, 1, 16, 16, 16, 16, 16, 16, w.p, w.n - 1, None) == WORKSPACE
    assert lib.saga_paged_decode(ctypes.byref(d), 16, 16, 16, 16, 16, None, None, 0, 16, w.p, w.n - 1, None) == WORKSPACE


def test_read_select_and_decode_refuse(lib):
    d = dims()
    w = Ws(d)
    D = ctypes.byref(d)
    good = [2, None, 16, 16, 16, 16, 16, 16]
    for i, bad in ((0, -1), (0, 5), (1, 6), (2, None), (3, None), (4, 8), (5, None), (6, None), (7, 24)):
        a = list(good)
        a[i] = bad
        assert lib.saga_paged_read(D, *a, w.p, w.n, None) == INVALID, (i, bad)
    good = [4, 1, 1, 16, 16, 16, 16, 16, 16]
    for i, bad in ((0, 0), (0, 1), (1, -1), (2, -1), (1, 5), (2, 4), (3, None), (3, 8), (4, None), (5, 2), (6, None),
                   (7, None), (8, 18)):
        a = list(good)
        a[i] = bad
        assert lib.saga_paged_select(D, *a, w.p, w.n, None) == INVALID, (i, bad)
    good = [16, 16, 16, 16, 16, 16, 16, 4, 16]
    for i, bad in ((0, None), (1, 8), (2, None), (3, None), (4, 2), (5, None), (6, None), (7, 0), (8, 8), (8, None)):
        a = list(good)
        a[i] = bad
        assert lib.saga_paged_decode(D, *a, w.p, w.n, None) == INVALID, (i, bad)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_get_as_far_as_the_device(lib):
    d = dims()
    w = Ws(d)
    D = ctypes.byref(d)
    assert lib.saga_paged_append(D, *append_args(w)) in NO_DEVICE
    assert lib.saga_paged_append(D, *append_args(w, q=None, qo=None, rope=None, bounds=None, lo=None)) in NO_DEVICE
    assert lib.saga_paged_append(D, *append_args(w, n=0, cu=16, k=None, v=None, q=None, qo=None)) in NO_DEVICE
    assert lib.saga_paged_read(D, 7, 16, 16, 16, 16, 16, 16, 16, w.p, w.n, None) in NO_DEVICE
    assert lib.saga_paged_select(D, 4, 1, 3, 16, 16, 16, 16, 16, 16, w.p, w.n, None) in NO_DEVICE
    assert lib.saga_paged_decode(D, 16, 16, 16, 16, 16, None, None, 0, 16, w.p, w.n, None) in NO_DEVICE


def cache(**kw):
    return PagedCache(2, 32, 4, 8, 64, 30, 10, page_size=64, device="cpu", **kw)


def test_paged_cache_buffers_and_table():
    c = cache()
    assert c.k_pages.shape == (30, 4, 64 * 34) and c.v_pages.shape == (30, 8, 64 * 34)
    assert c.bounds.shape == (30, 4, 2, 64) and c.seq_lens.tolist() == [0, 0]
    c.grow_table([65, 640])
    assert c.page_table[0].tolist() == [0, 1] + [-1] * 8 and c.page_table[1].tolist() == list(range(2, 12))
    for bad in ([1], [641, 1], [-1, 5], [64 * 40, 1]):
        with pytest.raises(ValueError, match="hold"):
            c.grow_table(bad)
    with pytest.raises(ValueError, match="k_pages"):
        cache(k_pages=torch.zeros(30, 4, 64 * 32, dtype=torch.uint8))
    with pytest.raises(ValueError, match="page_table"):
        cache(page_table=torch.zeros(2, 10, dtype=torch.int64))
    with pytest.raises(ValueError, match="rope"):
        cache(rope=torch.zeros(100, 64), rot_dim=32)
    with pytest.raises(ValueError, match="rotation table"):
        cache(rot_dim=32)
    with pytest.raises(_lib.SagaError):
        PagedCache(2, 32, 4, 8, 96, 30, 10, device="cpu")


def test_paged_cache_refuses_wrong_tensors():
    c = cache()
    bf = torch.bfloat16
    k, v, q = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 32, 64, dtype=bf)
    for args, kw, what in [
        ((k.float(), v), {}, "k_new"), ((k, v[:, :4]), {}, "v_new"), ((k, v, q[:1]), {}, "q_new"),
        ((k[:1], v[:1]), {}, "one new row"), ((k, v), dict(q_out=q), "q_out"), ((k, v, q), dict(q_out=q[:, :3]), "q_out"),
        ((k, v), dict(cu_new=torch.zeros(2, dtype=torch.int32)), "cu_new"),
        ((k, v), dict(lens_out=torch.zeros(2)), "lens_out"),
        ((k.transpose(1, 2).contiguous().transpose(1, 2), v), {}, "contiguous"),
        ((torch.zeros(2, 4 * 64 + 4, dtype=bf)[:, :256].unflatten(-1, (4, 64)), v), {}, "multiple of 8"),
        ((k[:1].expand(2, 4, 64), v), {}, "contiguous"),
    ]:
        with pytest.raises(ValueError, match=what):
            c.append(*args, **kw)
    for kw, what in [(dict(n_tokens=3), "one row"), (dict(n_tokens=2, k_out=v), "k_out"), (dict(n_tokens=2, start=q), "start")]:
        with pytest.raises(ValueError, match=what):
            c.read(**kw)
    i32 = torch.zeros(2, 4, 6, dtype=torch.int32)
    for args, kw, what in [((q[:1], 6), {}, "q must"), ((q, 5), dict(pages_out=i32), "pages_out"),
                           ((q, 6), dict(count_out=i32), "count_out")]:
        with pytest.raises(ValueError, match=what):
            c.select(*args, **kw)
    for args, kw, what in [((q.float(),), {}, "q must"), ((q, i32), {}, "together"), ((q, i32, i32), {}, "count"),
                           ((q,), dict(out=torch.zeros(2, 32, 64, dtype=bf)), "out must")]:
        with pytest.raises(ValueError, match=what):
            c.decode(*args, **kw)
    with pytest.raises(ValueError, match="on meta"):
        c.decode(torch.zeros(2, 32, 64, dtype=bf, device="meta"))


def test_reference_holds_rows_within_half_a_step():
    """The numpy form itself: what a row stands for is within half a step of it (7 steps either side of 0),
    plus the scale's own rounding (2^-9 of it, 7 steps far); a page is its rows."""
    rng = np.random.default_rng(0)
    x = ref.bf16(rng.normal(size=(5, 64)))
    block = np.zeros(block_bytes(16, 64), np.uint8)
    for i in range(5):
        ref.write_row(block, 16, 64, 3 + i, x[i])
        _, scale = ref.quantise(x[i])
        got = ref.row(block, 16, 64, 3 + i)
        assert np.abs(got - x[i]).max() <= scale * (0.5 + 7 * 2.0 ** -8)
    assert paged.block_bytes(64, 128) == 64 * 66


def test_grow_table_keeps_the_pages_of_cached_rows():
    c = cache()
    c.grow_table([64, 64])
    c.seq_lens.copy_(torch.tensor([64, 1], dtype=torch.int32))
    c.grow_table([129, 128])
    assert c.page_table[0, :4].tolist() == [0, 2, 3, -1] and c.page_table[1, :3].tolist() == [1, 4, -1]
    c.seq_lens.copy_(torch.tensor([65, 1], dtype=torch.int32))
    c.grow_table([640, 0])  # a sequence keeps what its rows are in; pages without rows are dealt out anew
    assert c.page_table[0].tolist() == [0, 2] + list(range(3, 11)) and c.page_table[1].tolist() == [1] + [-1] * 9
    before = c.page_table.clone()
    for bad in ([641, 1], [640], [-1, 1]):
        with pytest.raises(ValueError):
            c.grow_table(bad)
    c.seq_lens[1] = 65  # more rows than the table has pages of
    with pytest.raises(ValueError, match="cached pages of sequence 1"):
        c.grow_table([640, 65])
    c.seq_lens[1] = 641
    with pytest.raises(ValueError, match="cached length"):
        c.grow_table([640, 65])
    assert torch.equal(c.page_table, before)
    c.seq_lens.zero_()  # all over: dealt out anew
    c.grow_table([65, 64])
    assert c.page_table[:, :3].tolist() == [[0, 1, -1], [2, -1, -1]]


def test_grow_table_with_shared_and_few_pages():
    """Sequences that share their first page (a common prefix); a pool that is just large enough."""
    c = PagedCache(3, 4, 1, 2, 64, 5, 4, page_size=16, device="cpu")
    c.page_table[0, :2] = torch.tensor([4, 1])
    c.page_table[1, 0] = c.page_table[2, 0] = 4
    c.seq_lens.copy_(torch.tensor([20, 16, 9], dtype=torch.int32))
    c.grow_table([32, 48, 20])
    assert c.page_table.tolist() == [[4, 1, -1, -1], [4, 0, 2, -1], [4, 3, -1, -1]]
    with pytest.raises(ValueError, match="hold these"):
        c.grow_table([33, 48, 20])


def test_rows_of_one_head_may_have_any_head_stride():
    """x[:, None, :d] of a wider matrix: the head dim of size 1 has an arbitrary stride."""
    bf = torch.bfloat16
    wide = torch.zeros(5, 200, dtype=bf)
    paged._need("k_new", wide[:, None, :64], bf, (5, 1, 64), wide.device, rows=True)
    odd = wide.as_strided((5, 1, 64), (200, 3, 1))
    paged._need("k_new", odd, bf, (5, 1, 64), wide.device, rows=True)
    for bad in (wide.as_strided((5, 1, 64), (200, 3, 2)), wide.as_strided((5, 1, 64), (36, 3, 1)),
                wide.as_strided((5, 1, 64), (100, 3, 1)), wide.as_strided((5, 2, 64), (200, 65, 1))):
        with pytest.raises(ValueError, match="k_new"):
            paged._need("k_new", bad, bf, tuple(bad.shape), wide.device, rows=True)
