"""Plain 64-bit implementations of the serving operators, written from their
definitions, and the bounds that rounding sets on a kernel's results."""
import math

import numpy as np
import torch


def bound_of(dtype):
    """Half a step of the type, relative to the value."""
    return torch.finfo(dtype).eps / 2


class Pools:
    """Owner slabs [cp][pages, ps, width] on the host, in the element type."""

    def __init__(self, rng, n_pages, ps, cp, width, dtype, device="cpu"):
        self.ps, self.cp = ps, cp
        cap = -(-(n_pages + 1) // cp)
        self.slabs = [torch.from_numpy(rng.standard_normal((cap, ps, width)).astype(np.float32)).to(dtype) for _ in range(cp)]

    def row(self, page, off):
        return self.slabs[page % self.cp][page // self.cp, off]

    def rows(self, pages, n):
        """Token rows 0 .. n - 1 of a page list, in 64 bits."""
        if n == 0:
            return torch.zeros((0, self.slabs[0].shape[2]), dtype=torch.float64)
        return torch.stack([self.row(int(pages[t // self.ps]), t % self.ps) for t in range(n)]).double()

    def cuda(self):
        return [s.cuda() for s in self.slabs]


def softmax_rows(q, k, v, sees, scale):
    """One query [d] over keys [n, d] and values [n, d] that it sees (bool [n]):
    output, log-sum-exp and sum of weight * |value|, in 64 bits."""
    k, v = k[sees], v[sees]
    if k.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=torch.float64), -math.inf, torch.zeros(q.shape[0], dtype=torch.float64)
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    w = torch.exp(s - lse)
    return w @ v, float(lse), w @ v.abs()


def window(q, q_lens, pages, kv_lens, pools, *, kv_heads, dim, window, sinks, scale, k_at=0, v_at=None):
    """(out, lse, weighted absolute values) of cpkv_attend_window, query by query."""
    v_at = kv_heads * dim if v_at is None else v_at
    heads = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    t = 0
    for b, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        visible = [[j for j in range(kv) if j <= kv - nq + i and (window == 0 or kv - nq + i - j < window or j < sinks)]
                   for i in range(nq)]
        used = sorted(set(j for v in visible for j in v))  # nothing else of the cache is looked at
        rows = {j: pools.row(int(pages[b][j // pools.ps]), j % pools.ps).double() for j in used}
        for i in range(nq):
            for h in range(heads):
                c = h // (heads // kv_heads) * dim
                if visible[i]:
                    kvs = torch.stack([rows[j] for j in visible[i]])
                    out[t, h], lse[t, h], size[t, h] = softmax_rows(
                        q[t, h].double(), kvs[:, k_at + c:k_at + c + dim], kvs[:, v_at + c:v_at + c + dim],
                        torch.ones(len(kvs), dtype=torch.bool), scale)
            t += 1
    return out, lse, size


def shared(q, sizes, prefix_lens, prefix_pages, pages, suffix_lens, pools, *, kv_heads, dim, scale):
    heads = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    first = p0 = 0
    for n, length in zip(sizes, prefix_lens):
        np_ = length // pools.ps
        prefix = pools.rows(prefix_pages[p0:p0 + np_], length)
        p0 += np_
        for b in range(first, first + n):
            kvs = torch.cat([prefix, pools.rows(pages[b], suffix_lens[b])])
            for h in range(heads):
                c = h // (heads // kv_heads) * dim
                out[b, h], lse[b, h], size[b, h] = softmax_rows(
                    q[b, h].double(), kvs[:, c:c + dim], kvs[:, (kv_heads * dim) + c:(kv_heads * dim) + c + dim],
                    torch.ones(len(kvs), dtype=torch.bool), scale)
        first += n
    return out, lse, size


def check(got, lse, want, dtype, what=""):
    """A kernel's output against (out, lse, size).  An element's error: the
    rounding of the result, half a step of its value; the rounding of each
    weight before the product, half a step of the weighted |value|s; and 32-bit
    scores, weights and sums, 2^-13 of them at these sizes (a score of a few
    dozen 32-bit products is off by less than 2^-16, a weight's exponential
    and the sums by less than that)."""
    out, want_lse, size = want
    got, lse = got.double().cpu(), None if lse is None else lse.double().cpu()
    u = bound_of(dtype)
    limit = u * out.abs() + (u + 2.0**-13) * size + 2.0**-24
    bad = ~((got - out).abs() <= limit)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements off, worst {float(((got - out).abs() / limit).max()):.3g} of the bound, first {tuple(bad.nonzero()[0].tolist())}"
    if lse is not None:
        empty = torch.isneginf(want_lse)
        assert torch.equal(torch.isneginf(lse), empty), what
        off = (lse - want_lse)[~empty].abs()
        assert off.numel() == 0 or float(off.max()) <= 2.0**-13, f"{what}: lse off by {float(off.max()):.3g}"


def append(pools, k, v, q, slots, positions, table, axis, interleaved, k_at, v_at):
    """Writes the rows into ``pools`` (64-bit copies) and returns (q_out, pools64); rows as lists of slabs."""
    slabs = [s.double().clone() for s in pools.slabs]
    rot = table.shape[1]
    half = rot // 2
    n = k.shape[0]

    def turned(x, t):
        x = x.double().clone()
        y = x.clone()
        for i in range(half):
            c, s = float(table[positions[axis[i]][t], i]), float(table[positions[axis[i]][t], half + i])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        return y

    q_out = None if q is None else torch.stack([turned(q[t], t) for t in range(n)]) if n else q.double()
    for t in range(n):
        slot = int(slots[t])
        if slot < 0:
            continue
        page, off = slot // pools.ps, slot % pools.ps
        row = slabs[page % pools.cp][page // pools.cp, off]
        kk, vv = turned(k[t], t).flatten(), v[t].double().flatten()
        row[k_at:k_at + kk.numel()] = kk
        row[v_at:v_at + vv.numel()] = vv
    return q_out, slabs
