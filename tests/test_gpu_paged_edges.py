"""The paged 4-bit cache at the edges of its ranges, on the GPU against the
64-bit numpy form: what a call skips, magnitudes far apart, many sequences."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_saga_b200 import _lib

from tests import paged_reference as ref
from tests.test_gpu_paged import Pair, f64, filled, randn_bf16

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- lengths over rows that are not written

def grown_by(p, news, in_place, k, v, q=None, single=False):
    """One append through the cache; the grown lengths, in place or apart."""
    c = p.cache
    cu = None if single else torch.tensor(np.concatenate(([0], np.cumsum(news))), dtype=torch.int32, device="cuda")
    out = None if in_place else torch.full_like(c.seq_lens, -77)
    before = c.seq_lens.tolist()
    c.append(k.cuda(), v.cuda(), None if q is None else q.cuda(), cu_new=cu, lens_out=out)
    if not in_place:
        assert c.seq_lens.tolist() == before
        c.seq_lens.copy_(out)
    return c.seq_lens.tolist()


@pytest.mark.parametrize("in_place", [True, False])
def test_lengths_stop_at_a_missing_page(in_place):
    """A sequence grows up to the first position whose page is not in the pool, the others by their whole
    runs; with the page there, the rest of the run goes on from that length."""
    P, lens = 16, [3, 40, 0, 17, 16, 5]
    news = [30, 900, 16 * 300, 1, 20, 0]
    p = Pair((4, 1, 2, 64, 64), P, [a + b + 40 for a, b in zip(lens, news)], lens, 31, rot=0)
    table = p.cache.page_table
    whole = table.clone()
    # holes: none, page 30 of the run's 3 .. 58, page 270 (and 290), the run's only one, its second one
    table[1, 30], table[2, 270], table[2, 290], table[3, 1], table[4, 2] = -1, p.cache.dims.n_pages, -5, -1, 2 ** 30
    k, v, _ = p.rows(sum(news))
    got = grown_by(p, news, in_place, k, v)
    assert p.cache.error() == _lib.SAGA_ERR_BOUNDS
    want = [33, 480, 16 * 270, 17, 32, 5]
    assert got == want
    # the pages arrive: each sequence's rest
    table.copy_(whole)
    rest = [a + b - c for a, b, c in zip(lens, news, want)]
    at = np.concatenate(([0], np.cumsum(news)))
    rows = np.concatenate([np.arange(at[b + 1] - r, at[b + 1]) for b, r in enumerate(rest)])
    got = grown_by(p, rest, in_place, k[rows], v[rows])
    assert got == [a + b for a, b in zip(lens, news)]
    ref.append(p.state, f64(k), f64(v), None, at, None, 0, False)
    p.check_pool()


@pytest.mark.parametrize("in_place", [True, False])
def test_lengths_of_single_rows_without_a_page(in_place):
    lens = [0, 15, 16, 47, 64, 2 ** 31 - 1, -3] + [20] * 300
    p = Pair((4, 1, 2, 64, 64), 16, [64] * len(lens), [0] * len(lens), 32, rot=0)
    p.cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    p.cache.page_table[2, 1] = -1   # sequence 2's next page
    p.cache.page_table[1, 0] = -1   # the page that sequence 1's row is due in
    p.cache.page_table[200, 1] = -1
    p.cache.page_table[3, 0] = -1   # a page before the row: nothing of this call
    k, v, _ = p.rows(len(lens))
    got = grown_by(p, None, in_place, k, v, single=True)
    assert p.cache.error() == _lib.SAGA_ERR_BOUNDS
    want = [1, 15, 16, 48, 64, 2 ** 31 - 1, -3] + [21] * 300
    want[200] = 20
    assert got == want
    # nothing is left behind for the next call: the same with every page there
    p.cache.seq_lens.fill_(20)
    p.cache.page_table.copy_(torch.from_numpy(p.state["page_table"]))
    assert grown_by(p, None, in_place, k, v, single=True) == [21] * len(lens)
    assert p.cache.error() == _lib.SAGA_OK


@pytest.mark.parametrize("in_place", [True, False])
def test_lengths_stop_at_the_end_of_the_rotation_table(in_place):
    """Positions past the table are not written, nor the rest of their page's part of the run; the length
    stays in front of them.  40 rows in the table, pages of 16."""
    lens = [3, 3, 33, 41, 40, 0, 39]
    news = [50, 37, 3, 2, 1, 40, 1]
    p = Pair((12, 1, 2, 128, 128), 16, [80] * len(lens), lens, 33, max_pos=40)
    k, v, q = p.rows(sum(news))
    got = grown_by(p, news, in_place, k, v, q)
    assert p.cache.error() == _lib.SAGA_ERR_BOUNDS
    assert got == [32, 40, 36, 41, 40, 40, 40]


# ---------------------------------------------------------------- magnitudes far apart

def weighted(p, q, lists=None):
    """(out, bound) in 64 bits; the bound goes by the rows' weights, not by the largest value.

    With w = softmax and e the relative error of a weight (a logit's dk + 2 roundings of 2^-24 of its terms'
    magnitudes, 2^-20 for the exponential and the two halves of a product, 2^-16 for sums of a few hundred
    steps), numerator and denominator are off by e sum w |v| each.  A product w s of weight and row scale is
    held to 2^-25 of the column's own unit, in which the largest product is at least 2^6, and multiplies
    numbers up to 7: N 7 2^-31 max(w s)."""
    hq, hk, hv, dk, dv = p.layout
    s, P = p.state, p.P
    qn = f64(q)
    out, bound = np.zeros((len(s["seq_lens"]), hq, dv)), np.zeros((len(s["seq_lens"]), hq, dv))
    for b, n in enumerate(s["seq_lens"]):
        if not n:
            continue
        for i in range(hq):
            k = ref.rows(s["k_pages"], P, dk, s["page_table"][b], i * hk // hq, int(n))
            v = ref.rows(s["v_pages"], P, dv, s["page_table"][b], i * hv // hq, int(n))
            x = k @ qn[b, i] / np.sqrt(dk)
            w = np.exp(x - x.max())
            w /= w.sum()
            out[b, i] = w @ v
            e = (dk + 2) * 2.0 ** -24 * (np.abs(k) @ np.abs(qn[b, i])).max() / np.sqrt(dk) + 2.0 ** -20 + 2.0 ** -16
            bound[b, i] = 2 * e * (w @ np.abs(v)) + n * 7 * 2.0 ** -31 * (w * np.abs(v).max(1) / 7).max()
    return out, bound


def set_scales(p, name, b, head, scales):
    """The first len(scales) row scales of a head of sequence b (bf16 values)."""
    d, P, s = p.layout[3 if name == "k_pages" else 4], p.P, p.state
    raw = torch.from_numpy(np.ascontiguousarray(scales)).bfloat16().view(torch.uint8).numpy().reshape(-1, 2)
    for i, r in enumerate(raw):
        at = P * d // 2 + 2 * (i % P)
        s[name][s["page_table"][b, i // P], head, at:at + 2] = r


def set_rows(p, name, b, head, numbers):
    """The first rows of a head of sequence b: every number of row i is numbers[i]."""
    d, P, s = p.layout[3 if name == "k_pages" else 4], p.P, p.state
    for i, n in enumerate(numbers):
        u = int(n) + 8
        s[name][s["page_table"][b, i // P], head, i % P * d // 2:(i % P + 1) * d // 2] = u | u << 4


def push(p):
    p.cache.k_pages.copy_(torch.from_numpy(p.state["k_pages"]))
    p.cache.v_pages.copy_(torch.from_numpy(p.state["v_pages"]))


def check_weighted(p, q):
    want, bound = weighted(p, q)
    got = f64(p.cache.decode(q.cuda()))
    assert p.cache.error() == _lib.SAGA_OK
    worst = np.abs(got - want) / np.maximum(bound, 1e-300)
    assert worst.max() <= 1, "%.3g times the bound at %s" % (worst.max(), np.unravel_index(worst.argmax(), worst.shape))


# value heads per key head in one work row: 2, 4 and 2 of at most four, eight and four query heads
SHARED = [((32, 4, 8, 64, 64), 64), ((16, 1, 8, 64, 64), 16), ((32, 2, 4, 64, 64), 32), ((12, 1, 2, 128, 128), 16),
          ((16, 2, 8, 32, 64), 64)]


@pytest.mark.parametrize("layout,P", SHARED)
def test_value_heads_of_scales_far_apart(layout, P):
    """Value heads of one key head at scales 1, 2^-24, 2^-36 and 2^20 of each other: each is as exact as alone."""
    lens = [3000, 65, 700]
    p = filled(layout, P, lens, 41)
    hv = layout[2]
    for b, n in enumerate(lens):
        for h in range(hv):
            set_scales(p, "v_pages", b, h, ref.bf16(np.full(n, 0.3) * (1 + np.arange(n) % 5 / 8) *
                                                    2.0 ** (0, -24, -36, 20)[(h + b) % 4]))
    push(p)
    check_weighted(p, p.query())


@pytest.mark.parametrize("layout,P", SHARED + [((16, 1, 1, 128, 128), 64), ((4, 1, 2, 64, 64), 16)])
@pytest.mark.parametrize("up", [10, 20, 30])
def test_a_large_row_without_weight(layout, P, up):
    """Rows at the starts whose value scale is 2^up above the others' and whose weight is next to nothing
    do not take bits from the rows that carry it."""
    lens = [1500, 40, 9000]
    p = filled(layout, P, lens, 42)
    hq, hk, hv, dk, dv = layout
    for b, n in enumerate(lens):
        for h in range(hk):  # the first rows: logits far below all others
            set_rows(p, "k_pages", b, h, [-7] * 3)
            set_scales(p, "k_pages", b, h, np.full(3, 8.0))
        for h in range(hv):
            set_scales(p, "v_pages", b, h, np.full(3, 2.0 ** up))
    push(p)
    check_weighted(p, (0.1 + 0.4 * torch.rand(len(lens), hq, dk, generator=p.gen)).bfloat16())


@pytest.mark.parametrize("layout", [(32, 4, 8, 64, 64), (16, 1, 1, 128, 128), (32, 2, 4, 64, 64), (16, 2, 8, 32, 64)])
@pytest.mark.parametrize("up,sign", [(53, -7), (53, 7), (-34, -7), (-34, 7), (-40, -7)])
def test_logits_of_every_magnitude(layout, up, sign):
    """One row's logit far from the others, all of them large: it takes all, whatever their sign.  Where
    fp32's steps are larger than the unit (2^53: logits of 1e31, apart by 2^80 steps) the result is NaN."""
    hq, hk, hv, dk, dv = layout
    lens = [200, 17, 64]
    p = filled(layout, 32, lens, 43)
    best = [133, 4, 63]
    for b, n in enumerate(lens):
        pos = np.arange(n)
        near, far = (2.0 ** 50, 2.0 ** 51 * (1 + pos % 7 / 8)) if sign < 0 else (2.0 ** 52, 2.0 ** 50 * (1 + pos % 7 / 8))
        for h in range(hk):
            set_rows(p, "k_pages", b, h, [sign] * n)
            set_scales(p, "k_pages", b, h, np.where(pos == best[b], near, far))
    push(p)
    q = torch.full((3, hq, dk), 2.0 ** up).bfloat16()
    got = f64(p.cache.decode(q.cuda()))
    assert p.cache.error() == _lib.SAGA_OK
    for b, n in enumerate(lens):
        for i in range(hq):
            v = ref.rows(p.state["v_pages"], 32, dv, p.state["page_table"][b], i * hv // hq, n)[best[b]]
            if up > 0:
                assert np.isnan(got[b, i]).all()
            else:
                assert np.all(np.abs(got[b, i] - v) <= 2.0 ** -20 * np.abs(v) + 2.0 ** -31 * np.abs(v).max())


@pytest.mark.parametrize("layout", [(32, 4, 8, 64, 64), (16, 1, 1, 128, 128), (32, 2, 4, 64, 64), (16, 2, 8, 32, 64)])
@pytest.mark.parametrize("gap", [110.0, 119.3, 119.6, 130.0])
def test_zero_value_rows_far_above_the_first(layout, gap):
    """Rows of zeros whose weight is 2^gap times the ones' before them, then rows like those and as heavy:
    the zeros' weight counts, and nothing overflows."""
    hq, hk, hv, dk, dv = layout
    n = 96
    p = filled(layout, 32, [n], 44)
    pos = np.arange(n)
    scale = ref.bf16(gap * np.log(2) * np.sqrt(dk) / (7 * dk))  # logits of 7 dk scale / sqrt(dk) with queries of 1
    for h in range(hk):
        set_rows(p, "k_pages", 0, h, [7] * n)
        set_scales(p, "k_pages", 0, h, np.where(pos < 16, 0.0, scale))
    for h in range(hv):
        set_scales(p, "v_pages", 0, h, np.where((pos >= 16) & (pos < 64), 0.0, 1.0))
    push(p)
    check_weighted(p, torch.ones(1, hq, dk).bfloat16())


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("layout", [(4, 1, 2, 64, 64), (12, 1, 2, 128, 128), (16, 2, 8, 32, 64), (16, 1, 1, 64, 64)])
@pytest.mark.parametrize("qs,ks", [(1e-30, 1e-12), (1e-30, 1e-14), (1e-38, 1e-10), (1e-39, 1.0), (1e-39, 2.0 ** 60),
                                   (1e-20, 1e-20), (1.0, 1e-39), (2.0 ** 55, 2.0 ** 55), (2.0 ** 70, 2.0 ** 60), (1e35, 1e36)])
def test_select_scores_of_every_magnitude(layout, qs, ks):
    """Scores at and below fp32's smallest numbers and past its largest, subnormal queries and keys."""
    lens = [16 * 300 + 5, 16 * 90, 16 * 4]
    p = filled(layout, 16, lens, 45)
    box = ref.bf16(p.state["bounds"] * ks)
    p.cache.bounds.copy_(torch.from_numpy(box))
    q = (p.query().float() * qs).bfloat16()
    for n_sel, first, last in ((7, 0, 0), (40, 1, 2)):
        want = ref.select(f64(q), box, lens, p.state["page_table"], 16, n_sel, first, last)
        pages, count = p.cache.select(q.cuda(), n_sel, first, last)
        got = [[pages[b, h, :count[b, h]].tolist() for h in range(layout[1])] for b in range(len(lens))]
        assert got == want


# ---------------------------------------------------------------- rows as they come

def test_append_rows_of_one_head_out_of_a_wider_matrix():
    p = Pair((4, 1, 2, 64, 64), 16, [60, 60], [9, 0], 50)
    k, v, q = p.rows(30)
    wide = torch.zeros(30, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, :64] = k[:, 0].cuda()
    cu = np.array([0, 17, 30], np.int32)
    want = ref.append(p.state, f64(k), f64(v), f64(q), cu, p.table.numpy(), p.rot, False)
    got = p.cache.append(wide[:, None, :64], v.cuda(), q.cuda(), cu_new=torch.from_numpy(cu).cuda())
    assert np.array_equal(f64(got), want)
    p.check_pool()


# ---------------------------------------------------------------- rows that are not finite

@pytest.mark.parametrize("layout", [(4, 1, 2, 64, 64), (12, 1, 2, 128, 128), (16, 2, 8, 32, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite_stay_so(layout, bad):
    """A row with one number that is not finite reads back as NaN and makes a decode over it NaN; the rows
    beside it are whole."""
    hq, hk, hv, dk, dv = layout
    p = Pair(layout, 16, [80], [5], 48, rot=0)
    k, v, q = p.rows(40)
    k[7, 0, dk - 1] = bad
    v[21, hv - 1, 3] = bad
    p.cache.append(k.cuda(), v.cuda(), cu_new=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    got_k, got_v = p.cache.read(40, torch.tensor([0, 40], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"))
    k[7, 0], v[21, hv - 1] = 0, 0
    ref.append(p.state, f64(k), f64(v), None, np.array([0, 40]), None, 0, False)
    s = p.state
    for out, name, heads, d, at in ((got_k, "k_pages", hk, dk, (7, 0)), (got_v, "v_pages", hv, dv, (21, hv - 1))):
        want = np.stack([ref.rows(s[name], 16, d, s["page_table"][0], h, 45)[5:] for h in range(heads)], 1)
        got = f64(out)
        assert np.isnan(got[at]).all()
        got[at] = 0
        assert np.array_equal(got, ref.bf16(want))
    out = f64(p.cache.decode(q[:1].cuda()))[0]
    G = hq // hv
    assert np.isnan(out[:hq // hk]).all()             # key head 0's query heads
    assert np.isnan(out[(hv - 1) * G:]).all()         # the last value head's


# ---------------------------------------------------------------- many sequences

@pytest.mark.parametrize("layout,P,batch", [((32, 4, 8, 64, 64), 64, 60), ((8, 2, 2, 64, 64), 16, 1100), ((16, 2, 8, 32, 64), 32, 100),
                                            ((12, 1, 2, 128, 128), 16, 170), ((16, 1, 1, 64, 64), 16, 200),
                                            ((16, 1, 1, 128, 128), 32, 160), ((32, 2, 2, 32, 64), 16, 90)])
def test_select_more_rows_than_sms(layout, P, batch):
    """More rows than SMs (the smaller CTAs), most of a few pages, one beyond 4096 of them."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 60 * P, batch)]
    lens[3], lens[batch // 2], lens[-1] = 4200 * P + 1, 700 * P, 0
    p = filled(layout, P, lens, 46)
    q = p.query()
    for n_sel, first, last in ((1, 0, 0), (25, 1, 2)):
        want = ref.select(f64(q), p.state["bounds"], lens, p.state["page_table"], P, n_sel, first, last)
        pages, count = p.cache.select(q.cuda(), n_sel, first, last)
        assert p.cache.error() == _lib.SAGA_OK
        pages, count = pages.tolist(), count.tolist()
        assert [[r[:n] for r, n in zip(*rn)] for rn in zip(pages, count)] == want


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("batch", [32, 33, 64, 65, 1024, 1025, 1100])
def test_runs_of_many_sequences(batch, P):
    """Ragged runs over more sequences than a warp's search takes in one step, empty ones at its steps' borders;
    the rows read back by the same runs."""
    layout = (2, 1, 1, 64, 64)
    rng = np.random.default_rng(batch)
    news = rng.integers(0, 3, batch)
    for step in (31, 32, 33, 34, 63, 64, 65, 66, 1023, 1024, 1056):
        if step < batch:
            news[step] = step % 2 * 40
    news[0], news[-1] = 70, 5
    lens = rng.integers(0, 40, batch)
    p = Pair(layout, P, (lens + news).tolist(), lens.tolist(), 47)
    got = p.append(news.tolist())
    assert got.shape[0] == news.sum()
    p.check_pool()
    cu = torch.tensor(np.concatenate(([0], np.cumsum(news))), dtype=torch.int32, device="cuda")
    k, v = p.cache.read(int(news.sum()), cu, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    s = p.state
    for out, name in ((k, "k_pages"), (v, "v_pages")):
        want = np.concatenate([ref.rows(s[name], P, 64, s["page_table"][b], 0, int(lens[b] + news[b]))[lens[b]:]
                               for b in range(batch)])
        assert np.array_equal(f64(out)[:, 0], ref.bf16(want))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("mag,steps", [(1e30, 0), (1.0, 0), (1e-31, 0), (1e-36, 1), (1e-39, 1)])
def test_rotation_of_every_magnitude(inter, mag, steps):
    """Rotated rows bit for bit while a pair's products are above 2^-110, else to one step of bf16."""
    T, d = 3000, 128
    p = Pair((12, 1, 2, d, d), 64, [T], [0], 49, interleaved=inter)
    k, v, q = p.rows(T)
    # magnitudes within 2^-4 of each other: no pair's products are far below mag
    q = (torch.where(q < 0, -1.0, 1.0) * (1 + q.float().abs().clamp(max=3)) * mag).bfloat16()
    got = p.cache.append(k.cuda(), v.cuda(), q.cuda(), cu_new=torch.tensor([0, T], dtype=torch.int32, device="cuda")).cpu()
    c, s = p.table[:T, None, :d // 2].double(), p.table[:T, None, d // 2:].double()
    x = q.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :d // 2], x[..., d // 2:])
    y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2) if inter else torch.cat((a * c - b * s, b * c + a * s), -1)
    want = y.float().bfloat16()
    if steps == 0:
        small = torch.stack((torch.minimum((a * c).abs(), (b * s).abs()), torch.minimum((b * c).abs(), (a * s).abs())), -1) < 2.0 ** -110
        small = small.flatten(-2) if inter else torch.cat((small[..., 0], small[..., 1]), -1)
        assert small.float().mean() < 0.2
        assert torch.equal(got[~small], want[~small])
    one = torch.maximum(want.abs().double() * 2.0 ** -7, torch.tensor(2.0 ** -133, dtype=torch.float64))
    assert ((got.double() - want.double()).abs() <= one).all()
