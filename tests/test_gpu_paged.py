"""The paged 4-bit cache on the GPU against its 64-bit numpy form: append
(bytes, bounds, rotated queries and lengths bit for bit), read, page
selection (lists exactly) and decode (within what fp32 arithmetic may be off
by, derived from the inputs in paged_reference.decode)."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_saga_b200 import _lib
from sparse_decode_attention_saga_b200.paged import PagedCache, block_bytes

from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

# (h_q, h_k, h_v, d_k, d_v): every pairing of value-head group size and value
# heads per key head that a layout can have
LAYOUTS = [
    (4, 1, 2, 64, 64), (32, 4, 8, 64, 64), (32, 8, 8, 64, 64), (8, 8, 8, 64, 64), (12, 1, 2, 128, 128),
    (12, 2, 2, 128, 128), (16, 2, 8, 32, 64), (16, 1, 8, 64, 64), (16, 1, 1, 128, 128), (12, 2, 6, 64, 64),
    (16, 1, 1, 64, 64), (16, 2, 2, 32, 64), (14, 1, 2, 64, 64), (16, 1, 4, 128, 128), (8, 1, 8, 128, 128),
    (32, 2, 4, 64, 64), (20, 2, 4, 64, 64),
]


def rope_table(max_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), -1).float()


def randn_bf16(gen, *shape):
    return torch.randn(*shape, generator=gen).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


class Pair:
    """A PagedCache and its numpy twin over the same pool."""

    def __init__(self, layout, P, caps, lens, seed=0, rot=None, interleaved=False, max_pos=None, spare=2):
        hq, hk, hv, dk, dv = layout
        self.layout, self.P = layout, P
        gen = self.gen = torch.Generator().manual_seed(seed)
        need = [-(-max(c, 1) // P) for c in caps]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=gen).int()
        table = torch.full((len(caps), max(need)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        kp = torch.randint(0, 256, (n_pages, hk, block_bytes(P, dk)), generator=gen, dtype=torch.uint8)
        vp = torch.randint(0, 256, (n_pages, hv, block_bytes(P, dv)), generator=gen, dtype=torch.uint8)
        bounds = torch.zeros(n_pages, hk, 2, dk, dtype=torch.bfloat16)
        self.rot, self.inter = dk if rot is None else rot, interleaved
        self.table = rope_table(max_pos or max(need) * P, self.rot) if self.rot else None
        self.state = dict(P=P, k_pages=kp.numpy().copy(), v_pages=vp.numpy().copy(), bounds=f64(bounds).copy(),
                          page_table=table.numpy().copy(), seq_lens=np.asarray(lens, np.int32))
        self.cache = PagedCache(len(caps), hq, hk, hv, dk, n_pages, max(need), page_size=P, v_head_dim=dv,
                                rope=None if self.table is None else self.table.cuda(), interleaved=interleaved,
                                k_pages=kp.cuda(), v_pages=vp.cuda(), bounds=bounds.cuda(), page_table=table.cuda(),
                                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def rows(self, T):
        hq, hk, hv, dk, dv = self.layout
        return randn_bf16(self.gen, T, hk, dk), randn_bf16(self.gen, T, hv, dv), randn_bf16(self.gen, T, hq, dk)

    def append(self, news, k=None, v=None, q=None, **kw):
        """Ragged runs (news: rows per sequence, or None for one each) through both; rows checked."""
        B = len(self.state["seq_lens"])
        cu = np.concatenate(([0], np.cumsum([1] * B if news is None else news))).astype(np.int32)
        if k is None:
            k, v, q = self.rows(int(cu[-1]))
        want = ref.append(self.state, f64(k), f64(v), None if q is None else f64(q), cu,
                          None if self.table is None else self.table.numpy(), self.rot, self.inter)
        got = self.cache.append(k.cuda(), v.cuda(), None if q is None else q.cuda(),
                                cu_new=None if news is None else torch.from_numpy(cu).cuda(), **kw)
        if q is not None:
            assert np.array_equal(f64(got), want)
        return got

    def check_pool(self):
        assert self.cache.error() == _lib.SAGA_OK
        assert np.array_equal(self.cache.k_pages.cpu().numpy(), self.state["k_pages"])
        assert np.array_equal(self.cache.v_pages.cpu().numpy(), self.state["v_pages"])
        assert np.array_equal(f64(self.cache.bounds), self.state["bounds"])
        assert np.array_equal(self.cache.seq_lens.cpu().numpy(), self.state["seq_lens"])

    def kill_dead_rows(self):
        """NaN scales in the rows past each sequence's end (all of a page's after it)."""
        P, (hq, hk, hv, dk, dv) = self.P, self.layout
        nan = ref.scale_bytes(float("nan"))
        for b, n in enumerate(self.state["seq_lens"]):
            if n % P:
                phys = self.state["page_table"][b, n // P]
                for name, d in (("k_pages", dk), ("v_pages", dv)):
                    self.state[name][phys, :, P * d // 2 + 2 * (n % P):] = np.tile(nan, P - n % P)
        self.cache.k_pages.copy_(torch.from_numpy(self.state["k_pages"]))
        self.cache.v_pages.copy_(torch.from_numpy(self.state["v_pages"]))

    def expect(self, q, lists=None):
        hq, hk, hv, dk, dv = self.layout
        s = self.state
        return ref.decode(f64(q), s["k_pages"], s["v_pages"], s["seq_lens"], s["page_table"], self.P, dk, dv, lists)

    def check_decode(self, q, lists=None, out=None, **kw):
        want, bound = self.expect(q, lists)
        pages = count = None
        if lists is not None:
            hk, n = self.layout[1], max(1, max(len(r) for rows in lists for r in rows))
            pages = torch.full((len(lists), hk, n), -7, dtype=torch.int32)  # past the count: anything
            count = torch.tensor([[len(r) for r in rows] for rows in lists], dtype=torch.int32).cuda()
            for b, rows in enumerate(lists):
                for h, r in enumerate(rows):
                    pages[b, h, :len(r)] = torch.tensor(r, dtype=torch.int32)
            pages = pages.cuda()
        got = f64(self.cache.decode(q.cuda(), pages, count, out, **kw))
        assert self.cache.error() == _lib.SAGA_OK
        assert np.all(np.abs(got - want) <= bound[..., None]), float((np.abs(got - want) - bound[..., None]).max())
        return got

    def query(self):
        hq, hk, hv, dk, dv = self.layout
        return (2 * torch.randn(len(self.state["seq_lens"]), hq, dk, generator=self.gen)).bfloat16()


def filled(layout, P, lens, seed=0, **kw):
    """A pair whose sequences hold lens rows, quantised from normal rows without a call (rotation off)."""
    p = Pair(layout, P, lens, lens, seed, rot=0, **kw)
    hq, hk, hv, dk, dv = layout
    s = p.state
    for name, heads, d in (("k_pages", hk, dk), ("v_pages", hv, dv)):
        n_pages = s[name].shape[0]
        x = torch.randn(n_pages, heads, P, d, generator=p.gen).bfloat16().float()
        scale = (x.abs().amax(-1) / 7).bfloat16()
        u = (torch.round(x / scale.float()[..., None]).clamp(-7, 7) + 8).to(torch.uint8)
        s[name][:, :, :P * d // 2] = (u[..., 0::2] | (u[..., 1::2] << 4)).flatten(2).numpy()
        s[name][:, :, P * d // 2:] = scale.view(torch.uint8).view(n_pages, heads, 2 * P).numpy()
        if name == "k_pages":
            s["bounds"][:, :, 0], s["bounds"][:, :, 1] = x.amin(2).numpy(), x.amax(2).numpy()
    p.cache.bounds.copy_(torch.from_numpy(s["bounds"]))
    p.kill_dead_rows()
    return p


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("layout,rot,inter", [
    ((4, 1, 2, 64, 64), None, False), ((32, 4, 8, 64, 64), 32, True), ((12, 1, 2, 128, 128), 96, False),
    ((12, 2, 2, 128, 128), None, True), ((16, 2, 8, 32, 64), 16, False), ((16, 2, 8, 32, 64), None, True),
    ((32, 8, 8, 64, 64), 0, False),
])
def test_append_ragged_runs(layout, rot, inter, P):
    """Runs that start anywhere in a page, cross pages, are empty, or one row long; then one row each."""
    lens = [0, 5, P - 1, P, 2 * P + 3, 40, 0]
    news = [P + 1, 0, 1, 2 * P, 3 * P - 3, 1, 7]
    p = Pair(layout, P, [a + b + 2 for a, b in zip(lens, news)], lens, 1, rot, inter)
    p.append(news)
    p.check_pool()
    p.append(None)
    p.append(None)
    p.check_pool()


def test_append_values_at_the_edges():
    """Zero rows (scale 0), rows of equal values, halves between numbers, very large and very small values."""
    p = Pair((4, 1, 2, 64, 64), 16, [40], [3], 2, rot=0)
    k = torch.zeros(9, 1, 64, dtype=torch.bfloat16)
    v = torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    k[1] = 3.5
    k[2] = torch.arange(64) / 8 - 4.0
    k[3] = (torch.arange(64) % 15 - 7) / 2
    k[4, 0, 5] = 3e38
    k[5, 0, 63] = -1e-38
    k[6] = torch.where(torch.arange(64) % 2 == 0, 7.0, 0.5)  # scale 1: halves, to even
    k[7] = torch.where(torch.arange(64) % 3 == 0, -7.0, -2.5)
    k[8, 0, 0] = 1e-40
    v[:, 0] = k[:, 0]
    v[:, 1] = -k[:, 0]
    p.append([9], k, v, randn_bf16(p.gen, 9, 4, 64))
    p.check_pool()


def test_append_rows_of_a_fused_projection():
    """Rows that are slices of one wide output, queries among them."""
    layout = hq, hk, hv, dk, dv = (32, 4, 8, 64, 64)
    p = Pair(layout, 32, [90, 90, 90], [10, 0, 31], 3)
    wide = randn_bf16(p.gen, 50, hq * dk + hk * dk + hv * dv).cuda()
    q, k, v = (t.unflatten(-1, (h, d)) for t, h, d in zip(wide.split((hq * dk, hk * dk, hv * dv), -1), (hq, hk, hv), (dk, dk, dv)))
    cu = np.array([0, 20, 45, 50], np.int32)
    want = ref.append(p.state, f64(k), f64(v), f64(q), cu, p.table.numpy(), p.rot, False)
    got = p.cache.append(k, v, q, cu_new=torch.from_numpy(cu).cuda())
    assert np.array_equal(f64(got), want)
    p.check_pool()


def test_append_without_queries_without_bounds_and_nothing():
    p = Pair((4, 1, 2, 64, 64), 16, [100, 60], [10, 0], 4)
    k, v, _ = p.rows(30)
    p.append([13, 17], k, v, None)
    p.check_pool()
    d, c = p.cache.dims, p.cache
    empty = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    assert c.append(empty, torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"),
                    cu_new=torch.zeros(3, dtype=torch.int32, device="cuda")) is None
    p.check_pool()
    before = c.bounds.clone()
    k, v, _ = p.rows(2)
    ref.append(p.state, f64(k), f64(v), None, np.array([0, 1, 2]), p.table.numpy(), p.rot, False)
    p.state["bounds"] = f64(before)
    _lib.paged_append(d, 2, None, c.seq_lens, c.page_table, k.cuda(), v.cuda(), None, c._rope, c.k_pages, c.v_pages,
                      None, None, c.seq_lens, c.ws)
    p.check_pool()


def test_append_keeps_seq_lens_with_lens_out_and_is_repeatable():
    p = Pair((12, 1, 2, 128, 128), 32, [200, 200], [33, 64], 5)
    k, v, q = (t.cuda() for t in p.rows(70))
    cu = torch.tensor([0, 31, 70], dtype=torch.int32, device="cuda")
    grown = torch.zeros(2, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(2):
        qo = p.cache.append(k, v, q, cu_new=cu, lens_out=grown)
        outs.append([t.clone() for t in (qo, p.cache.k_pages, p.cache.v_pages, p.cache.bounds)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert grown.tolist() == [64, 103] and p.cache.seq_lens.tolist() == [33, 64]


@pytest.mark.parametrize("layout", [(4, 1, 2, 64, 64), (12, 1, 2, 128, 128), (16, 2, 8, 32, 64)])
def test_read_gives_the_rows_back(layout):
    hq, hk, hv, dk, dv = layout
    lens = [0, 37, 150, 64]
    p = filled(layout, 32, lens, 6)
    cu = torch.tensor([0, 0, 37, 187, 251], dtype=torch.int32, device="cuda")
    k, v = p.cache.read(251, cu, torch.zeros(4, dtype=torch.int32, device="cuda"))
    s = p.state
    for out, name, heads, d in ((k, "k_pages", hk, dk), (v, "v_pages", hv, dv)):
        want = np.concatenate([np.stack([ref.rows(s[name], 32, d, s["page_table"][b], h, n) for h in range(heads)], 1)
                               for b, n in enumerate(lens)])
        assert np.array_equal(f64(out), ref.bf16(want))
    # one row of each sequence, from a start of its own
    start = torch.tensor([0, 36, 149, 3], dtype=torch.int32, device="cuda")
    k1, v1 = p.cache.read(4, None, start)
    assert torch.equal(k1[1:], k[[36, 37 + 149, 187 + 3]]) and torch.equal(v1[1:], v[[36, 37 + 149, 187 + 3]])


def test_append_out_of_range_is_skipped_and_flagged():
    """A length past the table, a negative one, a page outside the pool, a position past the rotation
    table and run bounds outside the rows: nothing of them is written, the others are."""
    p = Pair((4, 1, 2, 64, 64), 16, [64] * 5, [3, 3, 3, 3, 3], 7, max_pos=40)
    good = {n: p.state[n].copy() for n in ("k_pages", "v_pages", "bounds")}
    c = p.cache
    k, v, q = p.rows(5)
    c.seq_lens.copy_(torch.tensor([3, 64, -1, 3, 41], dtype=torch.int32))
    c.page_table[3, 0] = c.dims.n_pages
    out = torch.full((5, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    c.append(k.cuda(), v.cuda(), q.cuda(), q_out=out, lens_out=torch.empty_like(c.seq_lens))
    torch.cuda.synchronize()
    assert c.error() == _lib.SAGA_ERR_BOUNDS and c.error() == _lib.SAGA_OK
    assert torch.all(out[1:] == 9.0)
    sub = dict(p.state, seq_lens=np.array([3], np.int32))
    want = ref.append(sub, f64(k[:1]), f64(v[:1]), f64(q[:1]), np.array([0, 1]), p.table.numpy(), 64, False)
    assert np.array_equal(f64(out[:1]), want)
    assert np.array_equal(c.k_pages.cpu().numpy(), p.state["k_pages"])
    assert np.array_equal(c.v_pages.cpu().numpy(), p.state["v_pages"])
    assert not np.array_equal(good["k_pages"], p.state["k_pages"])
    # runs that leave the rows
    c.seq_lens.fill_(3)
    before = c.k_pages.clone()
    c.append(k.cuda(), v.cuda(), cu_new=torch.tensor([-4, 9, 3, 3, 5, 5], dtype=torch.int32, device="cuda"),
             lens_out=torch.empty_like(c.seq_lens))
    assert c.error() == _lib.SAGA_ERR_BOUNDS
    p.state["k_pages"] = before.cpu().numpy()
    bad = {int(c.page_table[b, 0]) for b in (0, 1)}
    after = c.k_pages.cpu().numpy()
    assert all(np.array_equal(after[i], p.state["k_pages"][i]) for i in bad)


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("layout,P", [((4, 1, 2, 64, 64), 16), ((32, 4, 8, 64, 64), 64), ((12, 1, 2, 128, 128), 16),
                                      ((16, 2, 8, 32, 64), 32), ((16, 1, 1, 128, 128), 64), ((32, 2, 4, 64, 64), 16)])
@pytest.mark.parametrize("n_sel,first,last", [(1, 0, 0), (1, 0, 1), (7, 1, 2), (40, 2, 38), (64, 0, 1)])
def test_select_lists(layout, P, n_sel, first, last):
    lens = [0, 1, P, 7 * P, 7 * P + 1, 41 * P - 5, 65 * P, 301 * P + 2]
    p = filled(layout, P, lens, 8)
    q = p.query()
    s = p.state
    want = ref.select(f64(q), s["bounds"], lens, s["page_table"], P, n_sel, first, last)
    out = torch.full((len(lens), layout[1], n_sel), -5, dtype=torch.int32, device="cuda")
    pages, count = p.cache.select(q.cuda(), n_sel, first, last, pages_out=out)
    assert p.cache.error() == _lib.SAGA_OK
    pages, count = pages.cpu().numpy(), count.cpu().numpy()
    for b in range(len(lens)):
        for h in range(layout[1]):
            n = len(want[b][h])
            assert count[b, h] == n
            assert pages[b, h, :n].tolist() == want[b][h]
            assert (pages[b, h, n:] == -5).all()


def test_select_ties_go_to_the_lowest_index():
    """Equal pages, and pages whose scores differ only far behind fp32's last bit."""
    layout = (8, 2, 2, 64, 64)
    p = filled(layout, 16, [16 * 200, 16 * 90], 9)
    box = p.state["bounds"]
    box[:] = box[0]
    q = p.query()
    # one dim of a few pages wider by the smallest step: products apart by 2^-30 of the score
    tiny = [17, 60, 61, 150]
    for i in tiny:
        phys = p.state["page_table"][0, i]
        box[phys, :, 1, 3] = box[phys, :, 0, 3] = 1e-6 * (1 + i % 2)
    for i in range(200):
        if i not in tiny:
            phys = p.state["page_table"][0, i]
            box[phys, :, 1, 3] = box[phys, :, 0, 3] = 0.0
    q[:, :, 3] = 1.0
    box[:] = ref.bf16(box)
    p.cache.bounds.copy_(torch.from_numpy(box))
    for n_sel, first, last in ((5, 0, 0), (5, 1, 1), (3, 0, 0), (80, 3, 4)):
        want = ref.select(f64(q), box, [3200, 1440], p.state["page_table"], 16, n_sel, first, last)
        pages, count = p.cache.select(q.cuda(), n_sel, first, last)
        assert pages.cpu().numpy().tolist() == want
        assert (count == n_sel).all()


def test_select_zero_queries_and_long_rows():
    """q = 0: every score ties.  Thousands of pages of one row."""
    p = filled((4, 1, 2, 64, 64), 16, [16 * 5000 + 3], 10)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    pages, _ = p.cache.select(q.cuda(), 100, 2, 3)
    assert pages[0, 0].tolist() == list(range(97)) + [4998, 4999, 5000]
    q = p.query()
    want = ref.select(f64(q), p.state["bounds"], [16 * 5000 + 3], p.state["page_table"], 16, 1000, 1, 1)
    pages, _ = p.cache.select(q.cuda(), 1000, 1, 1)
    assert pages.cpu().numpy().tolist() == want


def test_select_flags_what_is_out_of_range():
    p = filled((4, 1, 2, 64, 64), 16, [320, 320, 320], 11)
    c, q = p.cache, p.query()
    want = ref.select(f64(q), p.state["bounds"], [320, 320, 320], p.state["page_table"], 16, 6, 0, 1)
    c.seq_lens.copy_(torch.tensor([320, -9, 10 ** 6], dtype=torch.int32))
    pages, count = c.select(q.cuda(), 6, 0, 1)
    assert c.error() == _lib.SAGA_ERR_BOUNDS
    assert pages[0].tolist() == want[0] and count[1].tolist() == [0] and count[2].tolist() == [6]
    c.seq_lens.fill_(320)
    c.page_table[1, 4] = -3
    c.page_table[2, 19] = 10 ** 6
    pages, count = c.select(q.cuda(), 6, 0, 1)
    assert c.error() == _lib.SAGA_ERR_BOUNDS
    assert pages[0].tolist() == want[0] and (count == 6).all()
    assert 4 not in pages[1, 0].tolist()


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_decode_every_layout_ragged(layout, P):
    """Lengths of zero and one, ends at, before and behind page and tile edges, NaN scales behind them."""
    lens = [0, 1, P - 1, P, P + 1, 63, 64, 65, 129, 700, 0, 1500]
    p = filled(layout, P, lens, 12)
    q = p.query()
    got = p.check_decode(q)
    assert np.all(got[0] == 0) and np.all(got[10] == 0)
    again = f64(p.cache.decode(q.cuda()))
    assert np.array_equal(got, again)


@pytest.mark.parametrize("layout", [(4, 1, 2, 64, 64), (32, 4, 8, 64, 64), (12, 1, 2, 128, 128), (16, 2, 8, 32, 64),
                                    (16, 1, 8, 64, 64), (14, 1, 2, 64, 64)])
@pytest.mark.parametrize("lens", [[20000], [9001, 3, 0, 12000], [1] * 200, [130] * 60])
def test_decode_split_and_packed(layout, lens):
    """Few long rows (split over the GPU), many short ones (several per CTA)."""
    p = filled(layout, 32, lens, 13)
    p.check_decode(p.query())


@pytest.mark.parametrize("layout", [(4, 1, 2, 64, 64), (32, 4, 8, 64, 64), (12, 2, 2, 128, 128), (16, 2, 8, 32, 64)])
@pytest.mark.parametrize("P", [16, 32, 64])
def test_decode_over_lists(layout, P):
    """Lists of their own per key head: any order, the ragged last page in the middle, empty ones."""
    lens = [0, 1, 5 * P + 3, 40 * P - 1, 90 * P, 17]
    p = filled(layout, P, lens, 14)
    rng = np.random.default_rng(1)
    lists = []
    for n in lens:
        np_ = -(-n // P)
        lists.append([rng.permutation(np_)[:rng.integers(0, min(np_, 23) + 1)].tolist() for _ in range(layout[1])])
    lists[3][0] = [39, 0, 7, 38, 2]
    lists[2][-1] = [5]
    p.check_decode(p.query(), lists)
    whole = [[list(range(-(-n // P))) for _ in range(layout[1])] for n in lens]
    p.check_decode(p.query(), whole)


def test_decode_extreme_logits_and_large_offsets():
    """Queries so large that one position takes all; a pool past 4 GB with the pages at its end."""
    p = filled((32, 4, 8, 64, 64), 64, [1000, 77], 15)
    q = (200 * torch.randn(2, 32, 64, generator=p.gen)).bfloat16()
    p.check_decode(q)
    q = torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    p.check_decode(q)
    n_big, c = 260_000, p.cache
    n = c.dims.n_pages
    kp = torch.empty(n_big, 4, block_bytes(64, 64), dtype=torch.uint8, device="cuda")
    vp = torch.empty(n_big, 8, block_bytes(64, 64), dtype=torch.uint8, device="cuda")
    kp[-n:], vp[-n:] = c.k_pages, c.v_pages
    big = PagedCache(2, 32, 4, 8, 64, n_big, c.dims.max_pages, k_pages=kp, v_pages=vp,
                     page_table=torch.where(c.page_table >= 0, c.page_table + (n_big - n), -1), seq_lens=c.seq_lens)
    q = p.query().cuda()
    assert torch.equal(big.decode(q), c.decode(q))
    k, v, qn = (t.cuda() for t in p.rows(2))
    c.page_table[:, -1] = c.page_table.max()
    grown = torch.empty(2, dtype=torch.int32, device="cuda")
    big.page_table.copy_(torch.where(c.page_table >= 0, c.page_table + (n_big - n), -1))
    big.append(k[:, :, :], v, qn, lens_out=grown)
    c.append(k, v, qn, lens_out=grown)
    assert torch.equal(big.k_pages[-n:], c.k_pages) and torch.equal(big.v_pages[-n:], c.v_pages)


def test_decode_query_scales():
    """Each head's queries at magnitudes of their own, subnormal and near the largest bf16 values among them."""
    p = filled((32, 4, 8, 64, 64), 32, [300, 129], 16)
    q = p.query()
    mag = torch.tensor([1e-39, 1e-30, 1e-4, 1.0, 3.0, 1e-3, 50.0, 0.25] * 4)[None, :, None]
    p.check_decode((q.float() * mag).bfloat16())
    q[:, :, 5] = 1e-20  # next to normal ones
    q[:, 3] = 0
    p.check_decode(q)


def test_decode_flags_what_is_out_of_range():
    p = filled((4, 1, 2, 64, 64), 16, [100, 100, 100, 100], 17)
    c, q = p.cache, p.query()
    want = f64(c.decode(q.cuda()))
    c.page_table[1, 2] = c.dims.n_pages  # the page's positions are left out
    got = f64(c.decode(q.cuda()))
    assert c.error() == _lib.SAGA_ERR_BOUNDS and c.error() == _lib.SAGA_OK
    assert np.array_equal(got[[0, 2, 3]], want[[0, 2, 3]])
    lists = [[[0, 1, 3, 4, 5, 6]] if b == 1 else [list(range(7))] for b in range(4)]
    w, bound = p.expect(q, lists)
    assert np.all(np.abs(got[1] - w[1]) <= bound[1][:, None])
    c.page_table.copy_(torch.from_numpy(p.state["page_table"]))
    c.seq_lens.copy_(torch.tensor([100, -5, 10 ** 9, 100], dtype=torch.int32))
    got = f64(c.decode(q.cuda()))
    assert c.error() == _lib.SAGA_ERR_BOUNDS
    assert np.array_equal(got[[0, 3]], want[[0, 3]]) and np.all(got[1] == 0)
    c.seq_lens.fill_(100)
    pages = torch.tensor([[[0, 7, 2]], [[0, -1, 2]], [[0, 2, 5]], [[0, 2, 5]]], dtype=torch.int32, device="cuda")
    count = torch.tensor([[3], [3], [9], [-2]], dtype=torch.int32, device="cuda")
    got = f64(c.decode(q.cuda(), pages, count))
    assert c.error() == _lib.SAGA_ERR_BOUNDS
    w, bound = p.expect(q, [[[0, 2]], [[0, 2]], [[]], [[]]])
    assert np.all(np.abs(got[:2] - w[:2]) <= bound[:2][..., None]) and np.all(got[2:] == 0)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("layout,P,n_sel", [((32, 4, 8, 64, 64), 64, None), ((12, 1, 2, 128, 128), 16, 12),
                                            ((16, 2, 8, 32, 64), 32, 5)])
def test_prompt_then_steps(layout, P, n_sel):
    """A ragged prompt, then steps of one token each: append, select and decode against the 64-bit forms."""
    news = [150, 1, 333, 64]
    p = Pair(layout, P, [n + 70 for n in news], [0] * 4, 18)
    p.append(news)
    for _ in range(66):
        k, v, q = p.rows(4)
        qr = ref.append(p.state, f64(k), f64(v), f64(q), np.arange(5), p.table.numpy(), p.rot, p.inter)
        out = p.cache.step(k.cuda(), v.cuda(), q.cuda(), n_sel, 1, 2)
    s = p.state
    lists = None if n_sel is None else ref.select(qr, s["bounds"], s["seq_lens"], s["page_table"], P, n_sel, 1, 2)
    want, bound = ref.decode(qr, s["k_pages"], s["v_pages"], s["seq_lens"], s["page_table"], P, layout[3], layout[4], lists)
    assert np.all(np.abs(f64(out) - want) <= bound[..., None])
    p.check_pool()


def test_captured_steps_grow_the_cache():
    """One step captured on a side stream and replayed: lengths grow in place, the outputs are those of
    eager steps; a second graph sharing the workspace, replayed in turn on the same stream."""
    layout, P = (32, 4, 8, 64, 64), 16
    caps, lens = [400, 90, 60], [300, 0, 31]
    a, b = Pair(layout, P, caps, lens, 19), Pair(layout, P, caps, lens, 19)
    k, v, q = (t.cuda() for t in a.rows(3))
    outs = [b.cache.step(k, v, q, 4).clone() for _ in range(6)]
    warm = Pair(layout, P, caps, lens, 19)
    warm.cache.step(k, v, q, 4)
    out1, out2 = (torch.empty(3, 32, 64, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g1, stream=side):
        a.cache.step(k, v, q, 4, out=out1)
    with torch.cuda.graph(g2, stream=side):
        a.cache.step(k, v, q, 4, out=out2)
    got = []
    with torch.cuda.stream(side):
        for i in range(3):
            g1.replay()
            got.append(out1.clone())
            g2.replay()
            got.append(out2.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.int32), y.view(torch.int32)) for x, y in zip(got, outs))  # NaN rows too
    assert a.cache.seq_lens.tolist() == [306, 6, 37]
    assert torch.equal(a.cache.k_pages, b.cache.k_pages)
    assert a.cache.error() == _lib.SAGA_OK


def test_other_stream_and_read_into_the_contiguous_path():
    """Calls on a stream of the caller's; a sequence read back feeds the bf16 decode of the framework."""
    layout = (32, 4, 8, 64, 64)
    p = filled(layout, 64, [1000], 20)
    s = torch.cuda.Stream()
    q = p.query().cuda()
    torch.cuda.synchronize()
    out = torch.empty(1, 32, 64, device="cuda")
    p.cache.decode(q, out=out, stream=s)
    k, v = p.cache.read(1000, torch.tensor([0, 1000], dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"))
    s.synchronize()
    want, bound = p.expect(q.cpu())
    assert np.all(np.abs(f64(out) - want) <= bound[..., None])
    d = _lib.dims(1, 32, 4, 8, 64, 1000)
    ws = torch.zeros(_lib.workspace_bytes(d, 1), dtype=torch.uint8, device="cuda")
    dense = torch.empty(1, 32, 64, device="cuda")
    _lib.decode_dense(d, q, k, v, dense, ws)
    # bf16 rounding of the rows: 2^-8 of a value, and of a logit's terms
    rows = np.abs(f64(k)).max() * np.abs(f64(q)).sum(-1).max() / 8
    assert np.abs(f64(dense) - want).max() <= (2 ** -8 + 2 * 2 ** -8 * rows) * np.abs(f64(v)).max()


def test_launches_are_counted():
    p = filled((4, 1, 2, 64, 64), 16, [100], 21)
    n = _lib.launch_count()
    p.cache.decode(p.query().cuda())
    assert _lib.launch_count() == n + 1


# ---------------------------------------------------------------- further shapes, streams and orders

@pytest.mark.parametrize("layout", [(8, 2, 2, 64, 64), (16, 2, 8, 32, 64)])
def test_many_short_sequences(layout):
    """More sequences than a CTA has threads, most of them a few positions or none."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 40, 1100)]
    lens[7], lens[600] = 900, 333
    lens[1099] = 0
    p = filled(layout, 16, lens, 22)
    q = p.query()
    p.check_decode(q)
    lists = [[rng.permutation(-(-n // 16))[:rng.integers(0, 3)].tolist() for _ in range(layout[1])] for n in lens]
    lists[0][0] = []
    p.check_decode(q, lists)


def test_select_over_many_pages():
    """A row longer than what the search holds in registers, next to short ones."""
    lens = [16 * 20000 + 5, 100, 16 * 9000]
    p = filled((4, 1, 2, 64, 64), 16, lens, 23)
    q = p.query()
    for n_sel in (3, 700):
        want = ref.select(f64(q), p.state["bounds"], lens, p.state["page_table"], 16, n_sel, 1, 1)
        pages, count = p.cache.select(q.cuda(), n_sel, 1, 1)
        for b in range(3):
            assert pages[b, 0, :count[b, 0]].tolist() == want[b][0]
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)  # every score equal
    pages, _ = p.cache.select(q.cuda(), 9, 1, 1)
    assert pages[0, 0].tolist() == list(range(8)) + [20000]
    assert pages[2, 0].tolist() == list(range(8)) + [8999]


def test_select_outlying_scores():
    """A few pages far above the rest, equal runs among them, and bounds that cancel (score 0)."""
    p = filled((4, 1, 2, 64, 64), 32, [32 * 600], 24)
    box = p.state["bounds"]
    table = p.state["page_table"][0]
    for i in range(0, 600, 50):
        box[table[i]] *= 1024.0
    for i in range(100, 140):
        box[table[i]] = box[table[100]]
    box[table[300]] = 0.0
    box[:] = ref.bf16(box)
    p.cache.bounds.copy_(torch.from_numpy(box))
    q = p.query()
    for n_sel, first, last in ((5, 0, 0), (13, 1, 1), (40, 0, 2), (599, 0, 0)):
        want = ref.select(f64(q), box, [19200], p.state["page_table"], 32, n_sel, first, last)
        pages, count = p.cache.select(q.cuda(), n_sel, first, last)
        assert pages[0, 0].tolist() == want[0][0] and count.tolist() == [[n_sel]]


def test_every_call_on_another_stream_allocates_there():
    """Outputs that the calls make themselves, on a side stream whose work lags behind the current one's."""
    layout = (32, 4, 8, 64, 64)
    a, b = filled(layout, 16, [700, 90], 25), filled(layout, 16, [700, 90], 25)
    k, v, q = (t.cuda() for t in a.rows(2))
    want = b.cache.step(k, v, q, 5)
    start = b.cache.seq_lens - 1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    got = a.cache.step(k, v, q, 5, stream=side)
    pages, count = a.cache.select(q, 5, stream=side.cuda_stream)
    rows = a.cache.read(2, start=start, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    assert all(torch.equal(x, y) for x, y in zip(rows, b.cache.read(2, start=start)))
    want_pages, want_count = b.cache.select(q, 5)
    assert torch.equal(pages, want_pages) and torch.equal(count, want_count)


def test_append_rotates_in_place_and_takes_single_rows_of_any_stride():
    p = Pair((12, 1, 2, 128, 128), 16, [40], [7], 26)
    k, v, q = p.rows(1)
    cu = np.array([0, 1], np.int32)
    want = ref.append(p.state, f64(k), f64(v), f64(q), cu, p.table.numpy(), p.rot, False)
    odd = torch.empty(1, 12, 128, dtype=torch.bfloat16, device="cuda").as_strided((1, 12, 128), (3, 128, 1))
    odd.copy_(q)
    assert p.cache.append(k.cuda(), v.cuda(), odd, q_out=odd) is odd
    assert np.array_equal(f64(odd), want)
    p.check_pool()


def test_runs_out_of_range_do_not_grow_their_sequences():
    p = Pair((4, 1, 2, 64, 64), 16, [64] * 4, [3, 60, 5, 64], 27)
    k, v, _ = p.rows(10)
    cu = torch.tensor([0, 2, 40, 42, 10], dtype=torch.int32, device="cuda")
    grown = torch.zeros(4, dtype=torch.int32, device="cuda")
    p.cache.append(k.cuda(), v.cuda(), cu_new=cu, lens_out=grown)
    assert p.cache.error() == _lib.SAGA_ERR_BOUNDS
    assert grown.tolist() == [5, 60, 5, 64]


@pytest.mark.parametrize("layout,P", [((32, 4, 8, 64, 64), 64), ((12, 2, 2, 128, 128), 16), ((16, 1, 1, 64, 64), 32)])
def test_decode_scales_that_grow_and_vanish(layout, P):
    """Logits that rise from position to position (a new reference again and again), value scales from
    2^-40 to 2^40 in both orders, rows of scale zero (keys, values, the first ones of a sequence)."""
    hq, hk, hv, dk, dv = layout
    lens = [40 * 64, 700, 65, 3]
    p = filled(layout, P, lens, 28)
    s = p.state
    for b, n in enumerate(lens):
        pos = np.arange(n)
        up = 2.0 ** ((pos * 80) // max(1, n) - 40)
        for name, d, heads in (("k_pages", dk, hk), ("v_pages", dv, hv)):
            for h in range(heads):
                if name == "k_pages":
                    scale = ref.bf16(0.05 + 0.5 * pos / n) if b != 1 else ref.bf16(0.4 + 0 * pos)
                else:
                    scale = (up if b % 2 == 0 else up[::-1]).copy()
                scale[pos % 7 == 3] = 0.0
                scale[:min(2, n - 1)] = 0.0
                raw = torch.from_numpy(np.ascontiguousarray(scale)).bfloat16().view(torch.uint8).numpy().reshape(n, 2)
                for i in range(n):
                    block = s[name][s["page_table"][b, i // P], h]
                    at = P * d // 2 + 2 * (i % P)
                    block[at:at + 2] = raw[i]
    p.cache.k_pages.copy_(torch.from_numpy(s["k_pages"]))
    p.cache.v_pages.copy_(torch.from_numpy(s["v_pages"]))
    p.check_decode(p.query())
    q = p.query()
    q[:] = q[:1, :1].abs()  # the same sign everywhere: large logits
    p.check_decode((8 * q.float()).bfloat16())
