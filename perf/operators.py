"""Cases and plain forms of the paged 4-bit cache's operators.

A paged cache keeps the keys and values of many sequences in pages of
``page`` positions; every row of a head is held as signed 4-bit numbers with
one bfloat16 scale.  The operators measured here are

  append   new key and value rows (one per sequence, or ragged runs of them)
           and their queries take the position rotation; the rows are rounded
           to 4 bits and written into their pages, the pages' key bounds are
           kept up, and the written rows are read back;
  select   the pages that each key head's queries attend to, by the upper
           bound that a page's key bounds put on its logits;
  decode   one query token per sequence over the whole 4-bit cache;
  sparse   the same over the selected pages of each key head only.

Formats.  A block is one head's rows of one page: ``page * d / 2`` bytes of
numbers (byte k of a row holds dims 2k in the low and 2k + 1 in the high four
bits, as n + 8) and then ``page`` bfloat16 scales; it stands for n * scale.
Pages are ``[pages, heads, block bytes]``, bounds ``[pages, key heads, 2, d]``
bfloat16 (smallest, then largest key).  Rows past a sequence's end hold
anything, NaN scales among it.

``own`` false computes with elementary torch operations, ``own`` true with the
package's calls; ``exact`` computes in 64 bits, written on its own.
"""
import math
import random

import torch

own = False

# (query heads, key heads, value heads, key dim, value dim): the layouts of the
# repository's workloads
LAYOUTS = {
    "small": (4, 1, 2, 64, 64),       # its smallest shape
    "saga64": (32, 4, 8, 64, 64),     # 8 query heads and 2 value heads per key head
    "gqa64": (32, 8, 8, 64, 64),      # the grouped-query layer that one is converted from
    "saga128": (12, 1, 2, 128, 128),  # 128-dim heads, one key head
    "gqa128": (12, 2, 2, 128, 128),
    "narrow": (16, 2, 8, 32, 64),     # keys narrower than values
}
MAX_POS = 140_000  # rows of the rotation table


def _case(op, layout, page, batch, len_lo, len_hi, **kw):
    hq, hk, hv, dk, dv = LAYOUTS[layout]
    c = dict(op=op, hq=hq, hk=hk, hv=hv, dk=dk, dv=dv, page=page, batch=batch, len_lo=len_lo, len_hi=len_hi,
             new_lo=0, new_hi=0, rot=0, interleaved=False, fused=False, sel=0, first=0, last=0)
    c.update(kw)
    return c


def listed():
    return [
        # a few users' next tokens, short contexts: latency of the whole write path
        dict(_case("append", "small", 16, 4, 100, 900, new_lo=1, new_hi=1, rot=64), name="append 4 tokens"),
        # a serving step of a full batch: one token of each of 256 ragged sequences, rows out of the
        # fused projection's output
        dict(_case("append", "saga64", 64, 256, 1, 8000, new_lo=1, new_hi=1, rot=64, fused=True), name="append 256 tokens"),
        # prompts entering the cache: ragged runs, some behind a prefix that ends inside a page
        dict(_case("append", "saga64", 64, 12, 0, 700, new_lo=300, new_hi=4100, rot=64), name="prefill 12 prompts"),
        # interleaved pairs, part of the dims rotated, 128-dim heads, small pages
        dict(_case("append", "saga128", 16, 5, 0, 90_000, new_lo=1, new_hi=2500, rot=96, interleaved=True), name="prefill 5 chunks d128"),
        # one long context, small pages: few rows, thousands of pages each
        dict(_case("select", "saga128", 16, 1, 32768, 32768, sel=128, first=1, last=4), name="select b1 32k"),
        # ragged mid-size contexts, narrow keys; some shorter than the budget, one empty
        dict(_case("select", "narrow", 32, 40, 0, 40_000, sel=96, first=1, last=2), name="select b40 ragged"),
        # the largest: a full batch of long contexts
        dict(_case("select", "saga64", 64, 16, 131072, 131072, sel=64, first=1, last=2), name="select b16 128k"),
        # one user's step at a short context: latency
        dict(_case("decode", "saga64", 64, 1, 8191, 8191), name="decode b1 8k"),
        # a mixed batch: short, long and empty sequences, small pages, grouped-query heads
        dict(_case("decode", "gqa128", 16, 48, 0, 20_000), name="decode b48 ragged d128"),
        # the largest: every position of a full batch of long contexts
        dict(_case("decode", "saga64", 64, 16, 131072, 131072), name="decode b16 128k"),
        # the selected 4096 positions of each of a full batch of long contexts
        dict(_case("sparse", "saga64", 64, 16, 131072, 131072, sel=64, first=1, last=2), name="sparse b16 128k"),
        # a ragged batch with small pages, some shorter than the budget
        dict(_case("sparse", "narrow", 16, 70, 0, 30_000, sel=80, first=1, last=3), name="sparse b70 ragged"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "select", "decode", "sparse"))
    layout = rng.choice(sorted(LAYOUTS))
    hq, hk, hv, dk, dv = LAYOUTS[layout]
    page = rng.choice((16, 32, 64))
    batch = _log_int(rng, 1, 200)
    row = hk * (dk / 2 + 2) + hv * (dv / 2 + 2)
    most = int(min(131072, 5e8 / (row * batch)))  # at most the largest listed case's bytes
    hi = _log_int(rng, min(200, most), most)
    lo = rng.choice((0, 1, hi // 2, hi))
    kw = {}
    if op == "append":
        if rng.random() < 0.5:
            kw = dict(new_lo=1, new_hi=1)
        else:
            kw = dict(new_lo=rng.choice((0, 1, 17)), new_hi=_log_int(rng, 20, max(20, 30_000 // batch)))
        kw.update(rot=rng.choice((dk, dk, dk // 2, 0)), interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
        hi = min(hi, 100_000)
        lo = min(lo, hi)
    elif op != "decode":  # a budget below the longest sequence's pages
        hi = max(hi, 20 * page)
        kw = dict(sel=_log_int(rng, 8, min(300, hi // page // 2)), first=rng.choice((0, 1, 2)), last=rng.choice((1, 2, 4)))
    return _case(op, layout, page, batch, lo, hi, **kw)


# ---------------------------------------------------------------- shapes of a case (no seed: work() needs them)

def _lens(c):
    """Each sequence's cached length: spread over the logarithm between the case's bounds, the longest first."""
    rng = random.Random("lens %d %d %d" % (c["batch"], c["len_lo"], c["len_hi"]))
    lo, hi = c["len_lo"], c["len_hi"]
    out = [hi] + [lo if lo == hi else _log_int(rng, max(lo, 1), hi) for _ in range(c["batch"] - 1)]
    if lo == 0 and len(out) > 2:
        out[len(out) // 2] = 0
    return out


def _news(c):
    """New rows of each sequence."""
    rng = random.Random("news %d %d %d" % (c["batch"], c["new_lo"], c["new_hi"]))
    return [c["new_hi"]] + [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"] - 1)]


def _pages(n, page):
    return (n + page - 1) // page


def work(case):
    c, P = case, case["page"]
    lens = _lens(c)
    krow, vrow = c["hk"] * (c["dk"] // 2 + 2), c["hv"] * (c["dv"] // 2 + 2)
    if c["op"] == "append":
        news = _news(c)
        T = sum(news)
        touched = sum(_pages(n + m, P) - n // P for n, m in zip(lens, news) if m)
        rows_in = T * (2 * c["hq"] * c["dk"] + 2 * c["hk"] * c["dk"] + 2 * c["hv"] * c["dv"])
        rows_out = rows_in + T * (krow + vrow)  # rotated queries, the rows read back, the rows in 4 bits
        return {"bytes": rows_in + rows_out + T * c["rot"] * 4 + touched * c["hk"] * 4 * c["dk"],
                "flops": T * (6 * (c["hq"] + c["hk"]) * c["dk"] + 4 * c["hv"] * c["dv"])}
    if c["op"] == "select":
        scored = sum(_pages(n, P) for n in lens if _pages(n, P) > c["sel"])
        return {"bytes": scored * c["hk"] * 4 * c["dk"] + c["batch"] * (2 * c["hq"] * c["dk"] + 4 * c["hk"] * (c["sel"] + 1)),
                "flops": 4.0 * scored * c["hq"] * c["dk"]}
    rows = sum(lens)
    if c["op"] == "sparse":
        rows = sum(min(n, (c["sel"] - 1) * P + (n - 1) % P + 1) for n in lens)
    return {"bytes": rows * (krow + vrow) + c["batch"] * c["hq"] * (2 * c["dk"] + 4 * c["dv"]),
            "flops": 2.0 * rows * c["hq"] * (c["dk"] + c["dv"])}


# ---------------------------------------------------------------- inputs

def _quantise(x):
    """bfloat16 rows [..., d] -> (numbers + 8 as uint8 [..., d], bfloat16 scales [...])."""
    x = x.float()
    scale = (x.abs().amax(-1) / 7.0).bfloat16()
    s = scale.float()[..., None]
    n = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)), torch.zeros_like(x)).clamp(-7, 7)
    return (n + 8).to(torch.uint8), scale


def _pool(n_pages, heads, page, d, gen, shift):
    """Pages of normal rows (a fortieth of the key rows leaning on their head's topic), in chunks, and their bounds."""
    pages = torch.empty(n_pages, heads, page * d // 2 + 2 * page, dtype=torch.uint8, device="cuda")
    bounds = torch.empty(n_pages, heads, 2, d, dtype=torch.bfloat16, device="cuda") if shift is not None else None
    step = max(1, (1 << 26) // (heads * page * d))
    for a in range(0, n_pages, step):
        n = min(step, n_pages - a)
        x = torch.randn(n, heads, page, d, device="cuda", generator=gen)
        if shift is not None:
            lean = torch.rand(n, heads, page, 1, device="cuda", generator=gen) < 0.025
            x += lean * (2.0 * shift[None, :, None, :])
        x = x.bfloat16()
        u, s = _quantise(x)
        pages[a:a + n, :, :page * d // 2] = (u[..., 0::2] | (u[..., 1::2] << 4)).flatten(2)
        pages[a:a + n, :, page * d // 2:] = s.view(torch.uint8).view(n, heads, 2 * page)
        if bounds is not None:
            bounds[a:a + n, :, 0] = x.amin(2)
            bounds[a:a + n, :, 1] = x.amax(2)
    return pages, bounds


def prepare(case, seed):
    c, P = dict(case), case["page"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    lens, news = _lens(c), _news(c) if c["op"] == "append" else [0] * c["batch"]
    need = [_pages(n + m, P) for n, m in zip(lens, news)]
    max_pages = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["batch"], max_pages), -1, dtype=torch.int32, device="cuda")
    np_ = torch.tensor(need, device="cuda")
    slot = torch.arange(max_pages, device="cuda")[None]
    table[slot < np_[:, None]] = order[:sum(need)]
    s = {"case": c, "page_table": table, "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    topic = torch.randn(c["hk"], c["dk"], device="cuda", generator=gen)
    topic /= topic.norm(dim=-1, keepdim=True)
    s["k_pages"], s["bounds"] = _pool(n_pages, c["hk"], P, c["dk"], gen, topic)
    s["v_pages"], _ = _pool(n_pages, c["hv"], P, c["dv"], gen, None)
    # the last page's rows past the sequence's end: scales of NaN
    last = torch.tensor([[b, n // P, n % P] for b, n in enumerate(lens) if n % P], device="cuda").view(-1, 3)
    if len(last):
        phys = table[last[:, 0], last[:, 1]].long()
        for pages, d in ((s["k_pages"], c["dk"]), (s["v_pages"], c["dv"])):
            sc = pages.view(torch.bfloat16)[:, :, P * d // 4:]
            past = torch.arange(P, device="cuda")[None] >= last[:, 2:3]
            sc[phys] = torch.where(past[:, None], torch.nan, sc[phys])
    b, hq, hk, hv, dk, dv = (c[k] for k in ("batch", "hq", "hk", "hv", "dk", "dv"))
    topics = topic.repeat_interleave(hq // hk, 0)
    if c["op"] == "append":
        T = sum(news)
        x = torch.randn(T, hq * dk + hk * dk + hv * dv, device="cuda", generator=gen).bfloat16()
        q, k, v = x.split((hq * dk, hk * dk, hv * dv), -1)
        if not c["fused"]:  # rows of their own instead of the fused projection's
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        s["q_new"], s["k_new"], s["v_new"] = q.unflatten(-1, (hq, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (hv, dv))
        cu = torch.tensor([sum(news[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
        s["cu_new"] = None if c["new_lo"] == c["new_hi"] == 1 else cu
        s["cu"] = cu
        s["rope"] = None
        if c["rot"]:
            freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
            angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * freq
            s["rope"] = torch.cat((angle.cos(), angle.sin()), -1).float()
        s["q_out"] = torch.zeros(T, hq, dk, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(T, hk, dk, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(T, hv, dv, dtype=torch.bfloat16, device="cuda")
        s["lens_out"] = torch.zeros_like(s["seq_lens"])
    else:
        s["q"] = (torch.randn(b, hq, dk, device="cuda", generator=gen) + 2.0 * topics).bfloat16()
        s["out"] = torch.zeros(b, hq, dv, device="cuda")
        s["sel"] = torch.zeros(b, hk, max(1, c["sel"]), dtype=torch.int32, device="cuda")
        s["cnt"] = torch.zeros(b, hk, dtype=torch.int32, device="cuda")
    if c["op"] == "sparse":  # the first pages, the last, and random ones between, ascending
        n_pg = np_[:, None, None]
        r = torch.rand(b, hk, max_pages, device="cuda", generator=gen)
        forced = (slot < c["first"]) | (slot >= np_[:, None] - c["last"])
        r = torch.where(forced[:, None], 2.0, r).masked_fill(slot[None] >= n_pg, -1.0)
        pick = r.argsort(-1, descending=True)[..., :c["sel"]]
        count = np_.clamp(max=c["sel"])
        live = torch.arange(pick.shape[-1], device="cuda")[None] < count[:, None]
        pick = torch.where(live[:, None], pick, max_pages).sort(-1).values
        s["sel"][..., :pick.shape[-1]] = torch.where(live[:, None], pick, 0).int()
        s["cnt"][:] = count[:, None].int()
    if own:  # the handle that a program keeps: shapes, workspace, and the buffers above
        from sparse_decode_attention_saga_b200.paged import PagedCache
        s["cache"] = PagedCache(b, hq, hk, hv, dk, n_pages, max_pages, page_size=P, v_head_dim=dv,
                                rope=s.get("rope"), rot_dim=c["rot"], interleaved=c["interleaved"],
                                k_pages=s["k_pages"], v_pages=s["v_pages"], bounds=s["bounds"],
                                page_table=table, seq_lens=s["seq_lens"])
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, table, pos, rot, interleaved):
    if not rot:
        return x
    y = x.double()
    cos, sin = table[pos].double()[:, None, :].split(rot // 2, -1)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((turned, y[..., rot:]), -1).float().bfloat16()


def _views(pages, page, d):
    """The numbers [pages, heads, page, d/2] and scales [pages, heads, page] of pages, as views."""
    return pages[:, :, :page * d // 2].unflatten(-1, (page, d // 2)), pages.view(torch.bfloat16)[:, :, page * d // 4:]


def _write(pages, page, d, phys, off, rows):
    numbers, scales = _views(pages, page, d)
    u, s = _quantise(rows)
    numbers[phys, :, off] = u[..., 0::2] | (u[..., 1::2] << 4)
    scales[phys, :, off] = s


def _read(pages, page, d, phys, off):
    numbers, scales = _views(pages, page, d)
    u = numbers[phys, :, off]
    n = torch.stack((u & 15, u >> 4), -1).flatten(-2).float() - 8.0
    return (n * scales[phys, :, off].float()[..., None]).bfloat16()


def _plain_append(s):
    c, P = s["case"], s["case"]["page"]
    token = torch.arange(s["k_new"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"], token, right=True) - 1
    pos = s["seq_lens"][seq].long() + token - s["cu"][seq]
    phys, off = s["page_table"][seq, pos // P].long(), pos % P
    q = _rotate(s["q_new"], s["rope"], pos, c["rot"], c["interleaved"])
    k = _rotate(s["k_new"], s["rope"], pos, c["rot"], c["interleaved"])
    _write(s["k_pages"], P, c["dk"], phys, off, k)
    _write(s["v_pages"], P, c["dv"], phys, off, s["v_new"])
    fresh = torch.zeros(s["bounds"].shape[0], dtype=torch.int32, device="cuda").index_reduce_(
        0, phys, (off == 0).int(), "amax")[:, None, None] > 0
    low = torch.where(fresh, torch.inf, s["bounds"][:, :, 0].float()).index_reduce_(0, phys, k.float(), "amin")
    high = torch.where(fresh, -torch.inf, s["bounds"][:, :, 1].float()).index_reduce_(0, phys, k.float(), "amax")
    s["bounds"][:, :, 0] = low.bfloat16()
    s["bounds"][:, :, 1] = high.bfloat16()
    return {"q": q, "k": _read(s["k_pages"], P, c["dk"], phys, off), "v": _read(s["v_pages"], P, c["dv"], phys, off),
            "bounds": s["bounds"], "lens": s["seq_lens"] + (s["cu"][1:] - s["cu"][:-1])}


def _plain_select(s):
    c, P = s["case"], s["case"]["page"]
    b, hk, n = c["batch"], c["hk"], c["sel"]
    pages = s["page_table"].shape[1]
    bounds = s["bounds"][s["page_table"].clamp(min=0).long()].double()  # [b, pages, hk, 2, d]
    q = s["q"].double().view(b, 1, hk, c["hq"] // hk, c["dk"])
    score = torch.maximum(q * bounds[:, :, :, None, 0], q * bounds[:, :, :, None, 1]).sum(-1).amax(-1)
    score = score.transpose(1, 2)  # [b, hk, pages]
    count = ((s["seq_lens"] + P - 1) // P)[:, None, None]
    slot = torch.arange(pages, device="cuda")
    score = torch.where((slot < c["first"]) | (slot >= count - c["last"]), torch.inf, score)
    score = torch.where(slot < count, score, -torch.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    kept = count.clamp(max=n)
    live = torch.arange(order.shape[-1], device="cuda") < kept
    order = torch.where(live, order, pages).sort(-1).values
    sel = s["sel"]
    sel[..., :order.shape[-1]] = torch.where(live, order.int(), sel[..., :order.shape[-1]])
    s["cnt"][:] = kept[..., 0]
    return {"pages": sel, "count": s["cnt"]}


def _blocks(pages, page, d, phys):
    """Rows [b, heads, n * page, d] of the pages phys [b, heads, n], and their scales, in 32 bits."""
    blocks = pages[phys, torch.arange(pages.shape[1], device="cuda")[None, :, None]]
    u = blocks[..., :page * d // 2]
    n = torch.stack((u & 15, u >> 4), -1).flatten(-2).unflatten(-1, (page, d)).flatten(2, 3).float() - 8.0
    return n, blocks[..., page * d // 2:].contiguous().view(torch.bfloat16).flatten(2).float()


def _plain_decode(s):
    c, P = s["case"], s["case"]["page"]
    b, hq, hk, hv = c["batch"], c["hq"], c["hk"], c["hv"]
    if c["op"] == "sparse":
        logical = s["sel"].long()
        live = torch.arange(logical.shape[-1], device="cuda") < s["cnt"][..., None]
    else:
        logical = torch.arange(s["page_table"].shape[1], device="cuda").expand(b, hk, -1)
        live = torch.ones_like(logical, dtype=torch.bool)
    phys = s["page_table"].long()[:, None].expand(b, hk, -1).gather(-1, logical).clamp(min=0)
    pos = logical[..., None] * P + torch.arange(P, device="cuda")
    valid = ((pos < s["seq_lens"][:, None, None, None]) & live[..., None]).flatten(2)  # [b, hk, rows]
    k, ks = _blocks(s["k_pages"], P, c["dk"], phys)
    v, vs = _blocks(s["v_pages"], P, c["dv"], phys.repeat_interleave(hv // hk, 1))
    wide = valid.repeat_interleave(hv // hk, 1)
    k *= torch.where(valid, ks, 0.0)[..., None]
    v *= torch.where(wide, vs, 0.0)[..., None]
    logits = s["q"].float().view(b, hk, hq // hk, c["dk"]) @ k.transpose(-1, -2) / math.sqrt(c["dk"])
    logits = logits.masked_fill(~valid[:, :, None], -torch.inf).view(b, hv, hq // hv, -1)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return {"out": ((p @ v) / torch.where(total > 0, total, 1.0)).reshape(b, hq, c["dv"])}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_select(s) if op == "select" else _plain_decode(s)
    cache = s["cache"]
    if op == "append":
        cache.append(s["k_new"], s["v_new"], s["q_new"], cu_new=s["cu_new"], q_out=s["q_out"], lens_out=s["lens_out"])
        cache.read(s["k_new"].shape[0], cu=s["cu_new"], k_out=s["k_out"], v_out=s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "bounds": s["bounds"], "lens": s["lens_out"]}
    if op == "select":
        c = s["case"]
        cache.select(s["q"], c["sel"], first=c["first"], last=c["last"], pages_out=s["sel"], count_out=s["cnt"])
        return {"pages": s["sel"], "count": s["cnt"]}
    if op == "sparse":
        return {"out": cache.decode(s["q"], pages=s["sel"], count=s["cnt"], out=s["out"])}
    return {"out": cache.decode(s["q"], out=s["out"])}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_rows(x, s, starts, turn):
    """Rows of one sequence's run, rotated as complex numbers, and what 4 bits make of them."""
    c = s["case"]
    if turn and c["rot"]:
        half = c["rot"] // 2
        rows = s["rope"][starts:starts + x.shape[0]].to(torch.complex128)
        unit = (rows[:, :half] + 1j * rows[:, half:])[:, None]
        y = x.double()
        if c["interleaved"]:
            z = torch.complex(y[..., 0:c["rot"]:2].contiguous(), y[..., 1:c["rot"]:2].contiguous()) * unit
            y = y.index_copy(-1, torch.arange(0, c["rot"], 2, device="cuda"), z.real)
            y = y.index_copy(-1, torch.arange(1, c["rot"], 2, device="cuda"), z.imag)
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * unit
            y = torch.cat((z.real, z.imag, y[..., 2 * half:]), -1)
        x = y.float().bfloat16()
    y = x.double()
    scale = (y.abs().max(-1, keepdim=True).values / 7).float().bfloat16().double()
    held = torch.nan_to_num(y / scale, nan=0.0).round().clamp(-7, 7) * scale
    return x, held


def exact(case, seed):
    s = prepare(case, seed)
    c, P = s["case"], case["page"]
    lens = s["seq_lens"].tolist()
    hq, hk, hv, dk, dv = (c[k] for k in ("hq", "hk", "hv", "dk", "dv"))
    if c["op"] == "append":
        cu, table = s["cu"].tolist(), s["page_table"].tolist()
        parts, bounds = {"q": [], "k": [], "v": []}, s["bounds"].double()
        for b, start in enumerate(lens):
            at = slice(cu[b], cu[b + 1])
            if at.start == at.stop:
                continue
            parts["q"].append(_exact_rows(s["q_new"][at], s, start, True)[0].double())
            k, held = _exact_rows(s["k_new"][at], s, start, True)
            parts["k"].append(held)
            parts["v"].append(_exact_rows(s["v_new"][at], s, start, False)[1])
            for p in range(start // P, (start + len(k) - 1) // P + 1):
                rows = k[max(0, p * P - start):max(0, (p + 1) * P - start)].double()
                old = bounds[table[b][p]]
                new = torch.stack((rows.amin(0), rows.amax(0)), 1)
                if p * P < start:
                    new = torch.stack((torch.minimum(new[:, 0], old[:, 0]), torch.maximum(new[:, 1], old[:, 1])), 1)
                bounds[table[b][p]] = new
        return {"q": torch.cat(parts["q"]), "k": torch.cat(parts["k"]), "v": torch.cat(parts["v"]), "bounds": bounds,
                "lens": s["seq_lens"] + (s["cu"][1:] - s["cu"][:-1])}
    if c["op"] == "select":
        pages, count = s["sel"].clone(), s["cnt"].clone()
        for b, n in enumerate(lens):
            n = -(-n // P)
            box = s["bounds"][s["page_table"][b, :n].long()].double()
            for h in range(hk):
                q = s["q"][b, h * hq // hk:(h + 1) * hq // hk].double()
                up, down = q.clamp(min=0), q.clamp(max=0)
                score = (up @ box[:, h, 1].T + down @ box[:, h, 0].T)
                score = score.amax(0).tolist() if n else []
                rank = sorted(range(n), key=lambda p: (not (p < c["first"] or p >= n - c["last"]), -score[p], p))
                keep = sorted(rank[:c["sel"]])
                count[b, h] = len(keep)
                pages[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32, device="cuda")
        return {"pages": pages, "count": count}
    out = torch.zeros(c["batch"], hq, dv, dtype=torch.float64, device="cuda")
    values = torch.arange(256, device="cuda")
    values = torch.stack((values % 16 - 8, values // 16 - 8), -1).double()  # what a byte stands for

    def rows(pages, d, phys, h, n):
        blocks = pages[phys, h]
        x = values[blocks[:, :P * d // 2].long()].reshape(-1, d)[:n]
        return x * blocks[:, P * d // 2:].reshape(-1).view(torch.bfloat16).double()[:n, None]

    for b, n in enumerate(lens):
        for h in range(hk):
            logical = s["sel"][b, h, :int(s["cnt"][b, h])].long() if c["op"] == "sparse" else torch.arange(-(-n // P), device="cuda")
            if not len(logical):
                continue
            live = len(logical) * P - max(0, (int(logical[-1]) + 1) * P - n)  # only the last page can end early
            phys = s["page_table"][b, logical].long()
            k = rows(s["k_pages"], dk, phys, h, live)
            for i in range(h * hv // hk, (h + 1) * hv // hk):
                at = slice(i * hq // hv, (i + 1) * hq // hv)
                w = torch.softmax(s["q"][b, at].double() @ k.T / math.sqrt(dk), -1)
                out[b, at] = w @ rows(s["v_pages"], dv, phys, i, live)
    return {"out": out}
