"""The operators of a quantised paged KV cache, as measured: the cases, their inputs, their plain forms and their values in 64 bits.

Four operators on rows that hold e4m3 values with float32 scales: ``append`` (new keys, rotated by position, and values quantised as they
are written into the paged pools, queries rotated beside them), ``read`` (rows of the pools read back into 16 bits), ``window`` (causal
attention over the quantised rows with a sliding window and a few first tokens that stay visible, for prefill and for decode) and
``shared`` (one query token per request, groups of requests that share a long prefix).

A row keeps its key heads (one scale a head), its value heads (a scale for each 128 values, or for a head of 64), the key scales and the
value scales, in this order.  A latent row keeps 512 values, their 4 scales and 64 rotated elements in 16 bits (656 bytes).  A scale is the
smallest power of two (2^-126 at least) whose 448-fold reaches the largest magnitude of its group; a value is the group's element over the
scale, rounded once to e4m3 from the exact product of the rotation.  Pools are ``cp`` owner slabs of pages of ``ps`` token rows; logical
page ``lp`` lives on owner ``lp % cp`` at local page ``lp // cp``; page 0 is the dummy page.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step's rows of 32 requests: the call counts, not its 0.5 MB
        dict(name="append_decode", op="append", n=32, hq=32, hkv=8, d=128, rot=128, style="half", axes=1, ps=64, cp=8, dtype="bf16",
             latent=False, spare=96, pos=131072),
        # the fp8 batch's 131 072 tokens into latent rows of 656 bytes
        dict(name="append_latent", op="append", n=131072, hq=16, hkv=1, d=64, rot=64, style="pairs", axes=1, ps=64, cp=8, dtype="bf16",
             latent=True, spare=64, pos=196608),
        # the traced batch's 44 600 tokens, only half of each head rotated
        dict(name="append_traced", op="append", n=44600, hq=32, hkv=8, d=128, rot=64, style="half", axes=1, ps=64, cp=8, dtype="fp16",
             latent=False, spare=64, pos=65536),
        # four queries' lists of 2048 chosen tokens (one place of the last missing), padding among them, from latent rows
        dict(name="read_chosen", op="read", n=8191, cached=131072, hq=16, hkv=1, d=64, ps=64, cp=8, dtype="bf16", latent=True, pads=0.05, runs=False),
        # the traced batch's 88 832 prefix tokens, page by page, before a dense prefill
        dict(name="read_prefix", op="read", n=88832, cached=133432, hq=32, hkv=8, d=128, ps=64, cp=8, dtype="bf16", latent=False, pads=0.0,
             runs=True),
        # one request's decode step: latency
        dict(name="window_decode_one", op="window", b=1, q=1, total=0, kv=777, spread=False, window=256, sinks=4, hq=8, hkv=1, d=64, ps=16, cp=2,
             dtype="fp16", lens=11),
        # 64 requests of up to 65 536 tokens, each seeing its last 4096 and the first four
        dict(name="window_decode_batch", op="window", b=64, q=1, total=0, kv=65536, spread=True, window=4096, sinks=4, hq=64, hkv=8, d=64, ps=64,
             cp=8, dtype="bf16", lens=12),
        # three proposed tokens each checked at once, no window, one-token pages
        dict(name="window_verify_token_pages", op="window", b=12, q=3, total=0, kv=16384, spread=True, window=0, sinks=0, hq=32, hkv=8, d=128, ps=1,
             cp=8, dtype="bf16", lens=13),
        # the next chunks of five long prompts, 1501 tokens in all behind up to 32 768
        dict(name="window_chunks", op="window", b=5, q=0, total=1501, kv=32768, spread=True, window=0, sinks=0, hq=32, hkv=8, d=128, ps=64, cp=8,
             dtype="bf16", lens=14),
        # the traced batch: 44 600 current tokens of 12 requests behind prefixes of up to 16 384
        dict(name="window_prefill_traced", op="window", b=12, q=0, total=44600, kv=16384, spread=True, window=4096, sinks=64, hq=32, hkv=8, d=128,
             ps=64, cp=8, dtype="bf16", lens=15),
        # a batch of 32 on one long document
        dict(name="shared_document", op="shared", b=32, groups=1, prefix=16384, suffix=1024, hq=32, hkv=8, d=128, ps=64, cp=8, dtype="bf16", lens=22),
        # three prompts shared by 48 requests, one-token pages, odd lengths
        dict(name="shared_groups", op="shared", b=48, groups=3, prefix=9001, suffix=700, hq=64, hkv=8, d=64, ps=1, cp=8, dtype="fp16", lens=23),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 and n > lo else n  # odd rather than round


def draw(rng):
    op = rng.choice(["append", "read", "window", "shared"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hq=hkv * rng.choice([1, 2, 4, 5, 7, 8]), hkv=hkv, d=rng.choice([64, 128]), ps=rng.choice([1, 16, 64]),
             cp=rng.choice([1, 2, 8]), dtype=rng.choice(["bf16", "fp16"]))
    if op in ("append", "read"):
        latent = rng.random() < 0.3
        if latent:
            c.update(hkv=1, hq=rng.choice([8, 16, 32]), d=64)
        c["latent"] = latent
    if op == "append":
        c.update(n=_log(rng, 1, 44600), rot=rng.choice([16, 32, 48, 64] + ([] if c["d"] == 64 else [96, 128])),
                 style=rng.choice(["half", "pairs"]), axes=rng.choice([1, 1, 3]), spare=rng.randint(16, 128), pos=_log(rng, 2048, 131072))
    elif op == "read":
        n = _log(rng, 1, 88832)
        c.update(n=n, cached=n + rng.randint(1, 65536), pads=rng.choice([0.0, 0.05]), runs=rng.random() < 0.5)
    elif op == "window":
        c.update(lens=rng.randint(100, 10**6), window=rng.choice([0, _log(rng, 16, 4096), _log(rng, 16, 4096)]), sinks=rng.choice([0, 1, 4, 64, 130]))
        if rng.random() < 0.5:  # decode, one to four tokens each
            c.update(b=_log(rng, 1, 64), q=rng.choice([1, 1, 2, 4]), total=0, kv=_log(rng, 64, 16384), spread=True)
        else:  # prefill behind prefixes
            b = _log(rng, 1, 16)
            c.update(b=b, q=0, total=max(b, _log(rng, 16, 8192)), kv=_log(rng, 64, 16384), spread=True)
    else:
        b = _log(rng, 1, 128)
        c.update(b=b, groups=min(b, rng.choice([1, 1, 2, 5])), prefix=_log(rng, 64, 32768), suffix=_log(rng, 1, 1024), lens=rng.randint(100, 10**6))
    return c


# ---------------------------------------------------------------------------
# rows and lengths: they belong to the case (work() counts them), values to the seed
# ---------------------------------------------------------------------------

class _Row:
    """Where a row keeps what, in bytes."""

    def __init__(self, case):
        self.hkv, self.kd, self.latent = case["hkv"], case["d"], case.get("latent", False)
        self.vd = 512 if self.latent else case["d"]
        self.groups = max(1, self.vd // 128)  # scales of a value head
        if self.latent:
            self.v, self.vs, self.k, self.ks = 0, 512, 528, None
            self.bytes = self.used = 656
        else:
            self.k, self.v = 0, self.hkv * self.kd
            self.ks = self.v + self.hkv * self.vd
            self.vs = self.ks + 4 * self.hkv
            self.used = self.vs + 4 * self.hkv * self.groups
            self.bytes = -(-self.used // 16) * 16

    def values(self, rows):
        return rows[..., self.v:self.v + self.hkv * self.vd].view(E4M3)

    def value_scales(self, rows):
        return rows[..., self.vs:self.vs + 4 * self.hkv * self.groups].view(torch.float32)

    def keys(self, rows, t):
        return rows[..., self.k:self.k + 128].view(t) if self.latent else rows[..., self.k:self.k + self.hkv * self.kd].view(E4M3)

    def key_scales(self, rows):
        return rows[..., self.ks:self.ks + 4 * self.hkv].view(torch.float32)


def _window_lens(case):
    """(q_lens, kv_lens): kv_len counts the request's prefix and its queries."""
    rng = np.random.default_rng(case["lens"])
    b = case["b"]
    if case["total"]:
        w = np.exp(rng.normal(0.0, 1.0, b))
        q = 1 + np.floor(w / w.sum() * (case["total"] - b)).astype(np.int64)
        q[0] += case["total"] - q.sum()
        kv = q + rng.integers(0, case["kv"] + 1, b) // case["ps"] * case["ps"]
    else:
        q = np.full(b, case["q"])
        kv = np.maximum(q, rng.integers(1, case["kv"] + 1, b) if case["spread"] else np.full(b, case["kv"]))
    return q.astype(np.int32), kv.astype(np.int32)


def _shared_lens(case):
    """(requests, prefix_len) of each group and (suffix_len) of each request: a prefix is whole pages, a suffix holds the query's own token."""
    rng = np.random.default_rng(case["lens"])
    b, g = case["b"], case["groups"]
    cuts = np.sort(rng.choice(np.arange(1, b), g - 1, replace=False)) if g > 1 else np.zeros(0, np.int64)
    sizes = np.diff(np.concatenate([[0], cuts, [b]]))
    prefix = np.maximum(1, (case["prefix"] * (1.0 - 0.3 * np.arange(g) / g)).astype(np.int64) // case["ps"]) * case["ps"]
    return sizes.astype(np.int32), prefix.astype(np.int32), rng.integers(1, case["suffix"] + 1, b).astype(np.int32)


def _seen(q, kv, w, s):
    """Visible pairs of (query token, key), and keys seen by any query, of one request."""
    p = np.arange(int(kv) - int(q), int(kv), dtype=np.int64)
    p = p[p >= 0]
    if not p.size:
        return 0, 0
    w = w if w else int(kv) + 1
    pairs = np.minimum(p + 1, w) + np.minimum(s, np.maximum(0, p + 1 - w))
    first = max(0, int(p[0]) - w + 1)
    return int(pairs.sum()), int(kv) - first + min(s, first)


def work(case):
    hq, hkv, d, row = case["hq"], case["hkv"], case["d"], _Row(case)
    new = 2 * hkv * (d + row.vd)  # bytes of a token's keys and values in 16 bits
    if case["op"] == "append":
        n = case["n"]
        turns = min(n, case["pos"]) * case["rot"] * 4  # each position's table row once
        return dict(bytes=n * (4 * hq * d + new + row.used + 8 + 4 * case["axes"]) + turns, flops=n * (3 * (hq + hkv) * case["rot"] + 2 * hkv * (d + row.vd)))
    if case["op"] == "read":
        real = case["n"] - int(case["n"] * case["pads"])
        return dict(bytes=real * row.used + case["n"] * (new + 8), flops=real * hkv * (d + row.vd))
    if case["op"] == "window":
        q, kv = _window_lens(case)
        seen = [_seen(a, b, case["window"], case["sinks"]) for a, b in zip(q, kv)]
        n, pairs, keys = int(q.sum()), sum(x for x, _ in seen), sum(y for _, y in seen)
    else:
        sizes, prefix, suffix = _shared_lens(case)
        n, keys = case["b"], int(prefix.sum() + suffix.sum())
        pairs = int((sizes.astype(np.int64) * prefix).sum() + suffix.sum())
    return dict(bytes=n * hq * (4 * d + 4) + keys * row.used, flops=4 * d * hq * pairs)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, shape, dtype, factor=1.0):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(factor)


def _pool(case, gen, pages):
    """The owner slabs, one allocation: [cp, slab pages, ps, row bytes] of tokens as a model leaves them, whose magnitude differs from head to
    head; valid page ids are [1, pages]."""
    row, t = _Row(case), TYPES[case["dtype"]]
    pool = torch.zeros((case["cp"], -(-(pages + 1) // case["cp"]), case["ps"], row.bytes), dtype=torch.uint8, device="cuda")
    flat = pool.view(-1, row.bytes)
    step = max(1, (1 << 26) // row.bytes)
    for i in range(0, flat.shape[0], step):
        at = flat[i:i + step]
        parts = [(row.values(at), row.value_scales(at), row.vd // row.groups)]
        if row.latent:
            row.keys(at, t).copy_(_randn(gen, (at.shape[0], 64), t))
        else:
            parts.append((row.keys(at, t), row.key_scales(at), row.kd))
        for to, scales, size in parts:
            x = _randn(gen, (*scales.shape, size), torch.float32)
            x *= _randn(gen, scales.shape, torch.float32, 0.4).exp_()[..., None]
            scale = _scale_of(x.abs().amax(-1))
            scales.copy_(scale)
            to.copy_((x / scale[..., None]).to(E4M3).flatten(1))
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, ps, hq, hkv, d, row = TYPES[case["dtype"]], case["ps"], case["hq"], case["hkv"], case["d"], _Row(case)
    st = dict(case=case)
    if case["op"] == "append":
        n = case["n"]
        pages = -(-n // ps) + case["spare"]
        st["pool"] = _pool(case, gen, pages)
        slots = ps + rng.permutation(pages * ps)[:n] if n < 1024 else ps + np.concatenate(
            [np.arange(p * ps, p * ps + ps) for p in rng.permutation(pages)[:-(-n // ps)]])[:n]
        st["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        first = torch.randint(0, max(1, case["pos"] - n), (), generator=gen, device="cuda")
        run_ = first + torch.arange(n, device="cuda")
        axes = [run_] if case["axes"] == 1 else [run_ // 64, run_ // 8 % 64, run_ % 64]
        st["positions"] = torch.stack([(a % case["pos"]).to(torch.int32) for a in axes])
        half = case["rot"] // 2
        st["axis"] = [0] * half if case["axes"] == 1 else [(0 if i < half // 4 else 1 if i < half // 4 + (half - half // 4) // 2 else 2)
                                                            for i in range(half)]
        angle = torch.arange(case["pos"], dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(half, dtype=torch.float64, device="cuda") / half)
        st["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        if row.latent:  # the latent part is the row's value, the rotated part its key
            latent = _randn(gen, (n, 576), t)
            st["q"], st["k"], st["v"] = _randn(gen, (n, hq, d), t), latent[:, 512:].unflatten(1, (1, 64)), latent[:, :512].unflatten(1, (1, 512))
        else:  # slices of the projection's one output
            qkv = _randn(gen, (n, hq + 2 * hkv, d), t)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_out"] = torch.empty((n, hq, d), dtype=t, device="cuda")
    elif case["op"] == "read":
        n, pages = case["n"], -(-case["cached"] // ps)
        st["pool"] = _pool(case, gen, pages)
        if case["runs"]:
            slots = ps + np.concatenate([np.arange(p * ps, p * ps + ps) for p in rng.permutation(pages)[:-(-n // ps)]])[:n]
        else:
            slots = ps + rng.permutation(pages * ps)[:n]
        slots[rng.permutation(n)[:int(n * case["pads"])]] = -1
        st["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        dense = torch.empty((n, hkv * (d + row.vd)), dtype=t, device="cuda")  # a dense row as the unquantised cache keeps it
        if row.latent:
            st["v_out"], st["k_out"] = dense[:, :512].unflatten(1, (1, 512)), dense[:, 512:].unflatten(1, (1, 64))
        else:
            st["k_out"], st["v_out"] = (x.unflatten(1, (hkv, d)) for x in dense.split(hkv * d, 1))
    elif case["op"] == "window":
        q_lens, kv_lens = _window_lens(case)
        need = -(-kv_lens.astype(np.int64) // ps)
        pages = int(need.sum())
        st["pool"] = _pool(case, gen, pages)
        table = np.zeros((case["b"], int(need.max())), np.int32)
        table[np.arange(table.shape[1]) < need[:, None]] = 1 + rng.permutation(pages)
        st["table"], st["kv_lens"] = torch.from_numpy(table).cuda(), torch.from_numpy(kv_lens).cuda()
        st["q_lens"], st["max_kv"] = q_lens, int(kv_lens.max())
        st["q"] = _randn(gen, (int(q_lens.sum()), hq, d), t, 1.5)
    else:
        sizes, prefix, suffix = _shared_lens(case)
        need = -(-suffix.astype(np.int64) // ps)
        n_prefix = int((prefix // ps).sum())
        pages = n_prefix + int(need.sum())
        st["pool"] = _pool(case, gen, pages)
        perm = (1 + rng.permutation(pages)).astype(np.int32)
        table = np.zeros((case["b"], int(need.max())), np.int32)
        table[np.arange(table.shape[1]) < need[:, None]] = perm[n_prefix:]
        st["prefix_pages"], st["table"] = torch.from_numpy(perm[:n_prefix]).cuda(), torch.from_numpy(table).cuda()
        st["suffix_lens"], st["sizes"], st["prefix"], st["max_suffix"] = torch.from_numpy(suffix).cuda(), sizes, prefix, int(suffix.max())
        st["q"] = _randn(gen, (case["b"], hq, d), t, 1.5)
    if case["op"] in ("window", "shared"):
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
    if own:  # the handle a serving program keeps: the pools' addresses, the row layout, a workspace
        from paged_kv_cache_compose_gb300.runtime import QuantisedCache

        st["cache"] = QuantisedCache(list(st["pool"]), page_size=ps, kv_heads=hkv, key_dim=d, value_dim=row.vd, dtype=t, keep_keys=row.latent)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        cache = state["cache"]
        if case["op"] == "append":
            cache.append_rotary(state["k"], state["v"], state["slots"], state["positions"], state["table"], q=state["q"], q_out=state["q_out"],
                                axis_of_freq=state["axis"] if case["axes"] > 1 else None, interleaved=case["style"] == "pairs")
            return _written(state, state["q_out"])
        if case["op"] == "read":
            cache.read_rows(state["slots"], k_out=state["k_out"], v_out=state["v_out"])
            return dict(k=state["k_out"], v=state["v_out"])
        if case["op"] == "window":
            cache.attend_window(state["q"], state["q_lens"], state["table"], state["kv_lens"], max_kv_len=state["max_kv"],
                                window=case["window"], sinks=case["sinks"], out=state["out"], lse=state["lse"])
        else:
            cache.attend_shared(state["q"], state["sizes"], state["prefix"], state["prefix_pages"], state["table"], state["suffix_lens"],
                                max_suffix_len=state["max_suffix"], out=state["out"], lse=state["lse"])
        return dict(out=state["out"], lse=state["lse"])
    return {"append": _append, "read": _read, "window": _window, "shared": _shared}[case["op"]](state)


def _written(st, q):
    """An append's outputs: the queries, and the pools as the e4m3 values and scales that they hold."""
    row, pool = _Row(st["case"]), st["pool"]
    r = dict(q=q, keys=row.keys(pool, q.dtype), values=row.values(pool), value_scales=row.value_scales(pool))
    return r if row.latent else dict(r, key_scales=row.key_scales(pool))


def _scale_of(largest):
    """The smallest power of two, 2^-126 at least, whose 448-fold reaches ``largest``."""
    m, e = torch.frexp(largest)
    return _power(torch.where(largest > 0, (e - 9 + (m > 0.875)).clamp(min=-126), -126)).to(largest.dtype)


def _power(e):
    """2^e in 64 bits, put together from its bits: ldexp goes through pow, which is off by a bit here and there."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _quantised(x):
    """e4m3 values and scales of [..., group] in 64 bits: rounded once, ties to even."""
    scale = _scale_of(x.abs().amax(-1))
    y = x / scale[..., None]
    step = _power(torch.frexp(y)[1].sub_(1).clamp_(min=-6) - 3)
    return torch.round(y / step).mul_(step).float().to(E4M3), scale.float()


def _rotated(x, cos, sin, rot, style):
    """x [n, heads, d] with its first ``rot`` elements rotated."""
    half = rot // 2
    a, b = (x[..., :half], x[..., half:rot]) if style == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    c, s = cos[:, None], sin[:, None]
    y1, y2 = a * c - b * s, b * c + a * s
    turned = torch.cat([y1, y2], -1) if style == "half" else torch.stack([y1, y2], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rows(case, pool, pages, offsets):
    """Row of the flat pool of each (page, offset)."""
    cp, slab = pool.shape[:2]
    return ((pages % cp) * slab + pages // cp) * case["ps"] + offsets


def _append(st):
    case, pool, row = st["case"], st["pool"], _Row(st["case"])
    half, t = case["rot"] // 2, st["q"].dtype
    axis = torch.tensor(st["axis"], device="cuda")
    angle = st["positions"].long()[axis].T  # [n, half]: each frequency's own position
    freq = torch.arange(half, device="cuda")
    cos, sin = st["table"][angle, freq], st["table"][angle, half + freq]
    q = _rotated(st["q"].float(), cos, sin, case["rot"], case["style"]).to(t)
    k = _rotated(st["k"].double(), cos.double(), sin.double(), case["rot"], case["style"])  # next to a border between two e4m3 values 32 bits lose which side
    v, v_scale = _quantised(st["v"].double().unflatten(-1, (row.groups, -1)))
    flat = pool.view(-1, row.bytes)
    at = _rows(case, pool, st["slots"] // case["ps"], st["slots"] % case["ps"])
    new = flat[at]
    row.values(new).copy_(v.flatten(1))
    row.value_scales(new).copy_(v_scale.flatten(1))
    if row.latent:
        row.keys(new, t).copy_(k.to(t).flatten(1))
    else:
        k8, k_scale = _quantised(k)
        row.keys(new, t).copy_(k8.flatten(1))
        row.key_scales(new).copy_(k_scale)
    flat[at] = new
    return _written(st, q)


def _read_back(row, rows, t):
    """Keys [..., hkv, kd] and values [..., hkv, vd] of gathered rows in 32 bits."""
    v = row.values(rows).float().unflatten(-1, (row.hkv * row.groups, -1)) * row.value_scales(rows)[..., None]
    v = v.reshape(*rows.shape[:-1], row.hkv, row.vd)
    k = row.keys(rows, t).float().unflatten(-1, (row.hkv, -1))
    return (k if row.latent else k * row.key_scales(rows)[..., None]), v


def _read(st):
    case, row = st["case"], _Row(st["case"])
    t, slots = TYPES[case["dtype"]], st["slots"]
    rows = st["pool"].view(-1, row.bytes)[_rows(case, st["pool"], slots.clamp(min=0) // case["ps"], slots.clamp(min=0) % case["ps"])]
    there = (slots >= 0)[:, None, None]
    return dict(zip("kv", (torch.where(there, x, 0.0).to(t) for x in _read_back(row, rows, t))))


def _parts(q, keys, values, mask, scale):
    """Maximum, sum and weighted values of [n, hkv, rows, d] queries over [n, keys, hkv, d] rows; mask [n, rows, keys] or None."""
    s = q @ keys.permute(0, 2, 3, 1) * scale
    if mask is not None:
        s.masked_fill_(~mask[:, None], -math.inf)
    m = s.amax(-1)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)[..., None]).exp_()
    return m, p.sum(-1), p @ values.permute(0, 2, 1, 3)


def _finished(m, l, o, t):
    return (o / torch.where(l == 0, 1.0, l)[..., None]).to(t), m + l.log()


def _window(st):
    """Blocks of up to 64 query tokens of one request, each against the keys it can see; as many blocks at once as fit 4 GB."""
    case, pool, q, row = st["case"], st["pool"], st["q"], _Row(st["case"])
    hkv, d, g, ps = case["hkv"], case["d"], case["hq"] // case["hkv"], case["ps"]
    flat = pool.view(-1, row.bytes)
    ql, kv = torch.from_numpy(st["q_lens"]).cuda().long(), st["kv_lens"].long()
    step = min(64, int(st["q_lens"].max()))
    w = case["window"] or st["max_kv"] + 1
    per = (ql + step - 1) // step
    req = torch.repeat_interleave(torch.arange(case["b"], device="cuda"), per)
    at = (torch.arange(req.numel(), device="cuda") - (per.cumsum(0) - per)[req]) * step  # first query token of the block
    tok = at[:, None] + torch.arange(step, device="cuda")
    place = torch.where(tok < ql[req][:, None], (ql.cumsum(0) - ql)[req][:, None] + tok, -1)
    pos = (kv - ql)[req][:, None] + tok
    n_sink = min(case["sinks"], st["max_kv"])
    first = (pos[:, :1] - w + 1).clamp(min=n_sink)
    span = min(w + step - 1, st["max_kv"])
    key = torch.cat([torch.arange(n_sink, device="cuda").expand(req.numel(), -1), first + torch.arange(span, device="cuda")], 1)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    count = max(1, int(4e9 / (4 * key.shape[1] * (case["hq"] * step + 3 * hkv * d))))
    for i in range(0, req.numel(), count):
        b, j, p, r = req[i:i + count], key[i:i + count], pos[i:i + count], place[i:i + count]
        page = st["table"][b[:, None], (j // ps).clamp(max=st["table"].shape[1] - 1)].long()
        k, v = _read_back(row, flat[_rows(case, pool, page, j % ps)], q.dtype)
        seen = (j[:, None] <= p[..., None]) & (j[:, None] < kv[b][:, None, None]) & ((p[..., None] - j[:, None] < w) | (j[:, None] < case["sinks"]))
        qs = q[r.clamp(min=0)].float().view(-1, step, hkv, g, d).transpose(1, 2).reshape(-1, hkv, step * g, d)
        o, e = _finished(*_parts(qs, k, v, seen.repeat_interleave(g, 1), d ** -0.5), q.dtype)
        keep = r >= 0
        out[r[keep]] = o.view(-1, hkv, step, g, d).transpose(1, 2).reshape(-1, step, case["hq"], d)[keep]
        lse[r[keep]] = e.view(-1, hkv, step, g).transpose(1, 2).reshape(-1, step, case["hq"])[keep]
    return dict(out=out, lse=lse)


def _shared(st):
    """Each group's queries against its prefix in one product, every request against its own suffix, joined by maximum and sum."""
    case, pool, ps, row = st["case"], st["pool"], st["case"]["ps"], _Row(st["case"])
    b, hkv, d, g = case["b"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    flat, scale, t = pool.view(-1, row.bytes), case["d"] ** -0.5, st["q"].dtype
    q = st["q"].float().view(b, hkv, g, d)
    parts, r0, p0 = [], 0, 0
    for size, length in zip(st["sizes"].tolist(), st["prefix"].tolist()):
        pages = st["prefix_pages"][p0:p0 + length // ps].long()
        k, v = _read_back(row, flat[_rows(case, pool, pages[:, None], torch.arange(ps, device="cuda")).view(1, -1)], t)
        x = _parts(q[r0:r0 + size].transpose(0, 1).reshape(1, hkv, size * g, d), k, v, None, scale)
        parts.append([y.view(hkv, size, g, *y.shape[3:]).transpose(0, 1) for y in x])
        r0, p0 = r0 + size, p0 + length // ps
    m1, l1, o1 = (torch.cat(x) for x in zip(*parts))
    j = torch.arange(st["max_suffix"], device="cuda")
    k, v = _read_back(row, flat[_rows(case, pool, st["table"].long()[:, j // ps], j % ps)], t)
    m2, l2, o2 = _parts(q, k, v, (j < st["suffix_lens"][:, None])[:, None].expand(-1, g, -1), scale)
    m = torch.maximum(m1, m2)
    w1, w2 = (m1 - m).exp(), (m2 - m).exp()
    out, lse = _finished(m, w1 * l1 + w2 * l2, w1[..., None] * o1 + w2[..., None] * o2, t)
    return dict(out=out.view_as(st["q"]), lse=lse.view(b, -1))


# ---------------------------------------------------------------------------
# the values in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _e4m3_64():
    """The 256 values of e4m3 by their bits: sign, 4 bits of exponent (bias 7), 3 of fraction; all ones are no number."""
    byte = np.arange(256)
    e, f = byte >> 3 & 15, byte & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    return np.where((byte & 127) == 127, np.nan, np.where(byte < 128, v, -v))


def _nearest64(x):
    """[..., group] -> its e4m3 values and scales, by looking the nearest value up."""
    top = x.abs().amax(-1)
    scale = torch.full_like(top, 2.0 ** -126)
    for shift in range(-126, 127):  # the first power that is large enough
        scale = torch.where(448.0 * 2.0 ** shift < top, 2.0 ** (shift + 1), scale)
    have = torch.from_numpy(_e4m3_64()[:127]).cuda()
    y = (x / scale[..., None]).contiguous()
    up = torch.searchsorted(have, y.abs(), right=False).clamp(1, 126)  # have[up - 1] < |y| <= have[up]
    low, high = y.abs() - have[up - 1], have[up] - y.abs()
    take = torch.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)
    return torch.copysign(have[take], y), scale


def _softmax64(q, k, v, hidden):
    """One request's [tokens, hq, d] queries over [keys, hkv, d] rows in 64 bits; hidden [tokens, keys] or None."""
    g = q.shape[1] // k.shape[1]
    out, lse = [], []
    for h in range(k.shape[1]):
        s = torch.einsum("tgd,kd->tgk", q[:, h * g:(h + 1) * g], k[:, h]) / math.sqrt(q.shape[-1])
        if hidden is not None:
            s = s.masked_fill(hidden[:, None], -math.inf)
        e = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.nan_to_num(e, neginf=0.0)[..., None])
        out.append(torch.einsum("tgk,kd->tgd", w, v[:, h]))
        lse.append(e)
    return torch.cat(out, 1), torch.cat(lse, 1)


def _slots64(st, tokens, pages):
    """Keys and values of a request's token numbers in 64 bits, looked up page by page."""
    case, pool, row = st["case"], st["pool"], _Row(st["case"])
    page = pages[tokens // case["ps"]].long()
    rows = pool[page % case["cp"], page // case["cp"], tokens % case["ps"]]
    value = torch.from_numpy(_e4m3_64()).cuda()
    v = value[rows[:, row.v:row.v + row.hkv * row.vd].long()].view(len(rows), row.hkv, row.groups, -1)
    v = v * row.value_scales(rows).double().view(len(rows), row.hkv, row.groups, 1)
    if row.latent:
        k = row.keys(rows, TYPES[case["dtype"]]).double().view(len(rows), 1, 64)
    else:
        k = value[rows[:, row.k:row.k + row.hkv * row.kd].long()].view(len(rows), row.hkv, -1) * row.key_scales(rows).double()[..., None]
    return k, v.flatten(2)


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    row, t = _Row(case), TYPES[case["dtype"]]
    if case["op"] == "append":
        rot, half, pool = case["rot"], case["rot"] // 2, st["pool"]
        at = [st["table"].double()[st["positions"][a].long()] for a in range(case["axes"])]
        cos = torch.stack([at[a][:, i] for i, a in enumerate(st["axis"])], 1)
        sin = torch.stack([at[a][:, half + i] for i, a in enumerate(st["axis"])], 1)
        turn = torch.complex(cos, sin)[:, None]
        q, k = st["q"].double().clone(), st["k"].double().clone()
        for x in (q, k):
            one, two = (slice(0, half), slice(half, rot)) if case["style"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
            z = torch.complex(x[..., one].clone(), x[..., two].clone()) * turn
            x[..., one], x[..., two] = z.real, z.imag
        page, off = st["slots"] // case["ps"], st["slots"] % case["ps"]
        place = (page % case["cp"], page // case["cp"], off)
        r = {name: x.double() for name, x in _written(st, q.to(t)).items()}
        r["q"] = q
        v, scale = _nearest64(st["v"].double().view(case["n"], -1, row.vd // row.groups))
        r["values"][place], r["value_scales"][place] = v.flatten(1), scale
        if row.latent:
            r["keys"][place] = k.flatten(1)
        else:
            k, scale = _nearest64(k)
            r["keys"][place], r["key_scales"][place] = k.flatten(1), scale
        return r
    if case["op"] == "read":
        there = st["slots"] >= 0
        page = torch.where(there, st["slots"] // case["ps"], 0)
        k = torch.zeros((case["n"], row.hkv, row.kd), dtype=torch.float64, device="cuda")
        v = torch.zeros((case["n"], row.hkv, row.vd), dtype=torch.float64, device="cuda")
        for i in range(0, case["n"], 16384):
            some = slice(i, i + 16384)
            # a page of its own for each token, at the token's place in it
            a, b = _slots64(st, torch.arange(len(page[some]), device="cuda") * case["ps"] + torch.where(there, st["slots"] % case["ps"], 0)[some], page[some])
            k[some], v[some] = a * there[some, None, None], b * there[some, None, None]
        return dict(k=k, v=v)
    out, lse = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    q = st["q"].double()
    if case["op"] == "window":
        r = 0
        for b, (n, kv) in enumerate(zip(st["q_lens"].tolist(), st["kv_lens"].tolist())):
            for i in range(0, n, 512):
                p = torch.arange(kv - n + i, kv - n + min(n, i + 512), device="cuda")
                lo = max(0, kv - n + i - case["window"] + 1) if case["window"] else 0
                j = torch.arange(lo, int(p[-1]) + 1, device="cuda")
                j = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), j])
                hidden = j > p[:, None]
                if case["window"]:
                    hidden |= (j <= p[:, None] - case["window"]) & (j >= case["sinks"])
                k, v = _slots64(st, j, st["table"][b])
                out[r:r + len(p)], lse[r:r + len(p)] = _softmax64(q[r:r + len(p)], k, v, hidden)
                r += len(p)
    else:
        r, p0, ps = 0, 0, case["ps"]
        for size, length in zip(st["sizes"].tolist(), st["prefix"].tolist()):
            k0, v0 = _slots64(st, torch.arange(length, device="cuda"), st["prefix_pages"][p0:p0 + length // ps])
            p0 += length // ps
            o0, e0 = _softmax64(q[r:r + size], k0, v0, None)
            for b in range(r, r + size):
                k1, v1 = _slots64(st, torch.arange(int(st["suffix_lens"][b]), device="cuda"), st["table"][b])
                o1, e1 = _softmax64(q[b:b + 1], k1, v1, None)
                lse[b] = torch.logaddexp(e0[b - r], e1[0])
                out[b] = o0[b - r] * (e0[b - r] - lse[b]).exp()[:, None] + o1[0] * (e1[0] - lse[b]).exp()[:, None]
            r += size
    return dict(out=out, lse=lse)
