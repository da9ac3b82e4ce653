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
