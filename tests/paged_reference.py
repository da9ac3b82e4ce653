"""The paged 4-bit cache in 64-bit numpy, from its definitions: the pool as
bytes, row by row.  bf16 arrays are held as float64 of their values."""
import numpy as np
import torch


def bf16(x):
    """float64 -> nearest bf16 (by way of fp32, as the operators define it), as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().bfloat16().double().numpy()


def rotate(x, table, pos, rot, interleaved):
    """Row x [heads, d] at position pos."""
    if table is None:
        return x
    y = np.array(x, np.float64)
    c, s = table[pos, :rot // 2].astype(np.float64), table[pos, rot // 2:rot].astype(np.float64)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return bf16(y)


def quantise(x):
    """Row [d] (float64 of bf16 values) -> numbers int, scale (float64 of a bf16)."""
    scale = float(bf16(np.float64(np.float32(np.abs(x).max() / 7.0))))
    if scale == 0.0:
        return np.zeros(len(x), np.int64), 0.0
    return np.clip(np.rint(x / scale), -7, 7).astype(np.int64), scale


def scale_bytes(scale):
    return torch.tensor([scale], dtype=torch.float64).bfloat16().view(torch.uint8).numpy()


def write_row(block, P, d, off, x):
    n, scale = quantise(x)
    u = (n + 8).astype(np.uint8)
    block[off * d // 2:(off + 1) * d // 2] = u[0::2] | (u[1::2] << 4)
    block[P * d // 2 + 2 * off:P * d // 2 + 2 * off + 2] = scale_bytes(scale)


def row(block, P, d, off):
    u = block[off * d // 2:(off + 1) * d // 2]
    n = np.stack((u & 15, u >> 4), -1).reshape(-1).astype(np.int64) - 8
    raw = np.ascontiguousarray(block[P * d // 2 + 2 * off:P * d // 2 + 2 * off + 2])
    return n * float(torch.from_numpy(raw).view(torch.bfloat16).double())


def rows(pages, P, d, phys_list, head, count):
    """The first `count` rows of a sequence's pages, dequantised [count, d]."""
    if count == 0:
        return np.zeros((0, d))
    blk = pages[np.asarray(phys_list)[:-(-count // P)], head]
    u = blk[:, :P * d // 2].reshape(-1, d // 2)[:count]
    n = np.stack((u & 15, u >> 4), -1).reshape(count, d).astype(np.float64) - 8
    sc = torch.from_numpy(np.ascontiguousarray(blk[:, P * d // 2:])).view(torch.bfloat16).double().numpy()
    return n * sc.reshape(-1)[:count, None]


def append(state, k_new, v_new, q_new, cu, table, rot, interleaved):
    """state: dict of k_pages, v_pages (uint8 arrays), bounds (float64), page_table,
    seq_lens, P; changed in place.  Returns the rotated queries."""
    P = state["P"]
    dk, dv = k_new.shape[-1], v_new.shape[-1]
    q_out = None if q_new is None else np.zeros_like(q_new)
    for b, start in enumerate(state["seq_lens"]):
        for t in range(cu[b], cu[b + 1]):
            pos = int(start) + t - cu[b]
            phys = state["page_table"][b, pos // P]
            k = rotate(k_new[t], table, pos, rot, interleaved)
            if q_new is not None:
                q_out[t] = rotate(q_new[t], table, pos, rot, interleaved)
            for h in range(k.shape[0]):
                write_row(state["k_pages"][phys, h], P, dk, pos % P, k[h])
            for h in range(v_new.shape[1]):
                write_row(state["v_pages"][phys, h], P, dv, pos % P, v_new[t, h])
            if state["bounds"] is not None:
                box = state["bounds"][phys]
                if pos % P == 0:
                    box[:, 0], box[:, 1] = k, k
                else:
                    box[:, 0], box[:, 1] = np.minimum(box[:, 0], k), np.maximum(box[:, 1], k)
    state["seq_lens"] = state["seq_lens"] + np.diff(cu).astype(state["seq_lens"].dtype)
    return q_out


def select(q, bounds, seq_lens, page_table, P, n_sel, first, last):
    """Lists of page indices, [b][h_k]."""
    hk, out = bounds.shape[1], []
    G = q.shape[1] // hk
    for b, n in enumerate(seq_lens):
        n, rows_ = -(-int(n) // P), []
        box = bounds[page_table[b, :n]]  # [n, hk, 2, d]
        for h in range(hk):
            qq = q[b, h * G:(h + 1) * G]
            s = np.maximum(qq[:, None] * box[None, :, h, 0], qq[:, None] * box[None, :, h, 1]).sum(-1).max(0)
            forced = [p for p in range(n) if p < first or p >= n - last]
            rest = sorted((p for p in range(n) if p not in set(forced)), key=lambda p: (-s[p], p))
            rows_.append(sorted((forced + rest)[:n_sel]) if n > n_sel else list(range(n)))
        out.append(rows_)
    return out


def decode(q, k_pages, v_pages, seq_lens, page_table, P, dk, dv, lists=None):
    """(out [b, h_q, dv], bound): bound[b, i] is what fp32 arithmetic may be off by.

    A logit is a sum of dk products (exact in fp32) and two scale products: off
    by at most (dk + 2) 2^-24 sum|q k| / sqrt(dk), which is a relative error of
    its probability; the exponential and the probability's two 11-bit halves
    add 2^-20, the sums over positions (in any tree of at most a few hundred
    sequential steps) 2^-16 at the very most; numerator and denominator both."""
    b_, hq = q.shape[:2]
    hk, hv = k_pages.shape[1], v_pages.shape[1]
    out, bound = np.zeros((b_, hq, dv)), np.zeros((b_, hq))
    for b, n in enumerate(seq_lens):
        n = int(n)
        for h in range(hk):
            k = rows(k_pages, P, dk, page_table[b], h, n)
            keep = np.arange(n)
            if lists is not None:
                keep = np.concatenate([np.arange(p * P, min(n, (p + 1) * P)) for p in lists[b][h]] or
                                      [np.zeros(0)]).astype(np.int64)
            if not len(keep):
                continue
            k = k[keep]
            for j in range(h * hv // hk, (h + 1) * hv // hk):
                v = rows(v_pages, P, dv, page_table[b], j, n)[keep]
                for i in range(j * hq // hv, (j + 1) * hq // hv):
                    s = k @ q[b, i] / np.sqrt(dk)
                    p = np.exp(s - s.max())
                    out[b, i] = p @ v / p.sum()
                    off = (dk + 2) * 2.0 ** -24 * (np.abs(k) @ np.abs(q[b, i])).max() / np.sqrt(dk)
                    bound[b, i] = 2 * (off + 2.0 ** -20 + 2.0 ** -16) * np.abs(v).max()
    return out, bound
