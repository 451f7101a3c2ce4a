"""The serving operators on paged KV rows, as measured: the cases, their inputs, their plain forms and their values in 64 bits.

Three operators: ``append`` (new keys and values rotated by position and written into the paged pools, queries rotated beside them),
``window`` (causal attention over the pages with a sliding window and a few first tokens that stay visible, for prefill and for decode) and
``shared`` (one query token per request, groups of requests that share a long prefix).  Pools are ``cp`` owner slabs of pages of ``ps``
token rows; logical page ``lp`` lives on owner ``lp % cp`` at local page ``lp // cp``; page 0 is the dummy page.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decode step's rows of 32 requests: the call counts, not its 0.5 MB
        dict(name="append_decode", op="append", n=32, hq=32, hkv=8, d=128, rot=128, style="half", axes=1, ps=64, cp=8, dtype="bf16",
             latent=False, spare=96, pos=131072),
        # an image-and-text chunk into latent rows (512 latent + 64 rotated), three position axes, odd count
        dict(name="append_latent_axes", op="append", n=8191, hq=16, hkv=1, d=64, rot=64, style="pairs", axes=3, ps=16, cp=2, dtype="bf16",
             latent=True, spare=64, pos=16384),
        # the traced batch's 44 600 tokens, only half of each head rotated
        dict(name="append_traced", op="append", n=44600, hq=32, hkv=8, d=128, rot=64, style="half", axes=1, ps=64, cp=8, dtype="fp16",
             latent=False, spare=64, pos=65536),
        # one request's decode step: latency
        dict(name="window_decode_one", op="window", b=1, q=1, total=0, kv=777, spread=False, window=256, sinks=4, hq=8, hkv=1, d=64, ps=16, cp=2,
             dtype="fp16", lens=11),
        # 64 requests of up to 65 536 tokens, each seeing its last 4096 and the first four
        dict(name="window_decode_batch", op="window", b=64, q=1, total=0, kv=65536, spread=True, window=4096, sinks=4, hq=64, hkv=8, d=64, ps=64,
             cp=8, dtype="bf16", lens=12),
        # three proposed tokens each checked at once, no window, one-token pages
        dict(name="window_verify_token_pages", op="window", b=12, q=3, total=0, kv=16384, spread=True, window=0, sinks=0, hq=32, hkv=8, d=128, ps=1,
             cp=8, dtype="bf16", lens=13),
        # a few short prompts behind short prefixes
        dict(name="window_prefill_tiny", op="window", b=4, q=48, total=0, kv=64, spread=True, window=40, sinks=2, hq=16, hkv=4, d=64, ps=16, cp=2,
             dtype="bf16", lens=14),
        # the traced batch: 44 600 current tokens of 12 requests behind prefixes of up to 16 384
        dict(name="window_prefill_traced", op="window", b=12, q=0, total=44600, kv=16384, spread=True, window=4096, sinks=64, hq=32, hkv=8, d=128,
             ps=64, cp=8, dtype="bf16", lens=15),
        # a handful of chats on a short system prompt
        dict(name="shared_few", op="shared", b=4, groups=1, prefix=512, suffix=64, hq=32, hkv=8, d=128, ps=16, cp=2, dtype="bf16", lens=21),
        # a batch of 32 on one long document
        dict(name="shared_document", op="shared", b=32, groups=1, prefix=16384, suffix=1024, hq=32, hkv=8, d=128, ps=64, cp=8, dtype="bf16", lens=22),
        # three prompts shared by 48 requests, one-token pages, odd lengths
        dict(name="shared_groups", op="shared", b=48, groups=3, prefix=9001, suffix=700, hq=64, hkv=8, d=64, ps=1, cp=8, dtype="fp16", lens=23),
        # 256 samples of one very long context
        dict(name="shared_samples", op="shared", b=256, groups=1, prefix=65536, suffix=2048, hq=64, hkv=8, d=128, ps=64, cp=8, dtype="bf16",
             lens=24),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 and n > lo else n  # odd rather than round


def draw(rng):
    op = rng.choice(["append", "window", "shared"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hq=hkv * rng.choice([1, 2, 4, 5, 7, 8]), hkv=hkv, d=rng.choice([64, 128]), ps=rng.choice([1, 16, 64]),
             cp=rng.choice([1, 2, 8]), dtype=rng.choice(["bf16", "fp16"]))
    if (c["hq"] + 2 * hkv) * c["d"] == 3072:  # another width of the projection's output
        c["d"] = 192 - c["d"]
    if op == "append":
        latent = rng.random() < 0.3
        if latent:
            c.update(hkv=1, hq=rng.choice([8, 16, 32]), d=64)
        c.update(n=_log(rng, 1, 44600), rot=rng.choice([16, 32, 48, 64] + ([] if c["d"] == 64 else [96, 128])),
                 style=rng.choice(["half", "pairs"]), axes=rng.choice([1, 1, 3]), latent=latent, spare=rng.randint(16, 128),
                 pos=_log(rng, 2048, 131072))
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
# lengths: they belong to the case (work() counts them), values to the seed
# ---------------------------------------------------------------------------

def _window_lens(case):
    """(q_lens, kv_lens): kv_len counts the request's prefix and its queries."""
    rng = np.random.default_rng(case["lens"])
    b = case["b"]
    if case["total"]:
        w = np.exp(rng.normal(0.0, 1.0, b))
        q = 1 + np.floor(w / w.sum() * (case["total"] - b)).astype(np.int64)
        q[0] += case["total"] - q.sum()
        kv = q + rng.integers(0, case["kv"] + 1, b) // case["ps"] * case["ps"]
    elif case["q"] > 4:
        q = rng.integers(1, case["q"] + 1, b)
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
    e, hq, hkv, d = 2, case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        n, row = case["n"], (576 if case["latent"] else 2 * hkv * d) * e
        rows = min(n, case["pos"]) * case["rot"] * 4  # each position's table row once
        return dict(bytes=n * (2 * hq * d * e + 2 * row + 8 + 4 * case["axes"]) + rows, flops=3 * n * (hq + hkv) * case["rot"])
    if case["op"] == "window":
        q, kv = _window_lens(case)
        seen = [_seen(a, b, case["window"], case["sinks"]) for a, b in zip(q, kv)]
        n, pairs, keys = int(q.sum()), sum(x for x, _ in seen), sum(y for _, y in seen)
    else:
        sizes, prefix, suffix = _shared_lens(case)
        n, keys = case["b"], int(prefix.sum() + suffix.sum())
        pairs = int((sizes.astype(np.int64) * prefix).sum() + suffix.sum())
    return dict(bytes=n * hq * (2 * d * e + 4) + keys * 2 * hkv * d * e, flops=4 * d * hq * pairs)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, shape, dtype, factor=1.0):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(factor)


def _pool(case, gen, pages, width):
    """The owner slabs, one allocation: [cp, slab pages, ps, width]; valid page ids are [1, pages]."""
    return _randn(gen, (case["cp"], -(-(pages + 1) // case["cp"]), case["ps"], width), TYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, ps, hq, hkv, d = TYPES[case["dtype"]], case["ps"], case["hq"], case["hkv"], case["d"]
    st = dict(case=case)
    if case["op"] == "append":
        n = case["n"]
        width = 576 if case["latent"] else 2 * hkv * d
        pages = -(-n // ps) + case["spare"]
        st["pool"] = _pool(case, gen, pages, width)
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
        if case["latent"]:  # the latent part is the row's value, the rotated part its key
            latent = _randn(gen, (n, 576), t)
            st["q"], st["k"], st["v"] = _randn(gen, (n, hq, d), t), latent[:, 512:].unflatten(1, (1, 64)), latent[:, :512].unflatten(1, (1, 512))
            st["offsets"] = (512, 0)
        else:  # slices of the projection's one output
            qkv = _randn(gen, (n, hq + 2 * hkv, d), t)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            st["offsets"] = (0, hkv * d)
        st["q_out"] = torch.empty((n, hq, d), dtype=t, device="cuda")
    elif case["op"] == "window":
        q_lens, kv_lens = _window_lens(case)
        need = -(-kv_lens.astype(np.int64) // ps)
        pages = int(need.sum())
        st["pool"] = _pool(case, gen, pages, 2 * hkv * d)
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
        st["pool"] = _pool(case, gen, pages, 2 * hkv * d)
        perm = (1 + rng.permutation(pages)).astype(np.int32)
        table = np.zeros((case["b"], int(need.max())), np.int32)
        table[np.arange(table.shape[1]) < need[:, None]] = perm[n_prefix:]
        st["prefix_pages"], st["table"] = torch.from_numpy(perm[:n_prefix]).cuda(), torch.from_numpy(table).cuda()
        st["suffix_lens"], st["sizes"], st["prefix"], st["max_suffix"] = torch.from_numpy(suffix).cuda(), sizes, prefix, int(suffix.max())
        st["q"] = _randn(gen, (case["b"], hq, d), t, 1.5)
    if case["op"] != "append":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
    if own:  # the handle a serving program keeps: the pools' addresses, the row layout, a workspace
        from paged_kv_cache_compose_gb300.runtime import PagedCache

        k_off, v_off = st.get("offsets", (0, hkv * d))
        st["cache"] = PagedCache(list(st["pool"]), page_size=ps, kv_heads=hkv, key_dim=d, value_dim=512 if case.get("latent") else d,
                                 key_offset=k_off, value_offset=v_off)
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
            return dict(q=state["q_out"], pool=state["pool"])
        if case["op"] == "window":
            cache.attend_window(state["q"], state["q_lens"], state["table"], state["kv_lens"], max_kv_len=state["max_kv"],
                                window=case["window"], sinks=case["sinks"], out=state["out"], lse=state["lse"])
        else:
            cache.attend_shared(state["q"], state["sizes"], state["prefix"], state["prefix_pages"], state["table"], state["suffix_lens"],
                                max_suffix_len=state["max_suffix"], out=state["out"], lse=state["lse"])
        return dict(out=state["out"], lse=state["lse"])
    return {"append": _append, "window": _window, "shared": _shared}[case["op"]](state)


def _rotated(x, cos, sin, rot, style):
    """x [n, heads, d] in 32 bits with its first ``rot`` elements rotated."""
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
    case, pool = st["case"], st["pool"]
    half = case["rot"] // 2
    axis = torch.tensor(st["axis"], device="cuda")
    angle = st["positions"].long()[axis].T  # [n, half]: each frequency's own position
    freq = torch.arange(half, device="cuda")
    cos, sin = st["table"][angle, freq], st["table"][angle, half + freq]
    q = _rotated(st["q"].float(), cos, sin, case["rot"], case["style"]).to(pool.dtype)
    k = _rotated(st["k"].float(), cos, sin, case["rot"], case["style"]).to(pool.dtype)
    flat = pool.view(-1, pool.shape[-1])
    at = _rows(case, pool, st["slots"] // case["ps"], st["slots"] % case["ps"])
    flat[at] = torch.cat([st["v"].flatten(1), k.flatten(1)] if case["latent"] else [k.flatten(1), st["v"].flatten(1)], 1)
    return dict(q=q, pool=pool)


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
    case, pool, q = st["case"], st["pool"], st["q"]
    hkv, d, g, ps = case["hkv"], case["d"], case["hq"] // case["hkv"], case["ps"]
    flat = pool.view(-1, 2, hkv, d)
    ql, kv = torch.from_numpy(st["q_lens"]).cuda().long(), st["kv_lens"].long()
    step = min(64, int(st["q_lens"].max()))
    w = case["window"] or st["max_kv"] + 1
    per = (ql + step - 1) // step
    req = torch.repeat_interleave(torch.arange(case["b"], device="cuda"), per)
    at = (torch.arange(req.numel(), device="cuda") - (per.cumsum(0) - per)[req]) * step  # first query token of the block
    tok = at[:, None] + torch.arange(step, device="cuda")
    row = torch.where(tok < ql[req][:, None], (ql.cumsum(0) - ql)[req][:, None] + tok, -1)
    pos = (kv - ql)[req][:, None] + tok
    n_sink = min(case["sinks"], st["max_kv"])
    first = (pos[:, :1] - w + 1).clamp(min=n_sink)
    span = min(w + step - 1, st["max_kv"])
    key = torch.cat([torch.arange(n_sink, device="cuda").expand(req.numel(), -1), first + torch.arange(span, device="cuda")], 1)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    count = max(1, int(4e9 / (4 * key.shape[1] * (case["hq"] * step + 2 * hkv * d))))
    for i in range(0, req.numel(), count):
        b, j, p, r = req[i:i + count], key[i:i + count], pos[i:i + count], row[i:i + count]
        page = st["table"][b[:, None], (j // ps).clamp(max=st["table"].shape[1] - 1)].long()
        kvs = flat[_rows(case, pool, page, j % ps)].float()
        seen = (j[:, None] <= p[..., None]) & (j[:, None] < kv[b][:, None, None]) & ((p[..., None] - j[:, None] < w) | (j[:, None] < case["sinks"]))
        qs = q[r.clamp(min=0)].float().view(-1, step, hkv, g, d).transpose(1, 2).reshape(-1, hkv, step * g, d)
        o, e = _finished(*_parts(qs, kvs[:, :, 0], kvs[:, :, 1], seen.repeat_interleave(g, 1), d ** -0.5), q.dtype)
        keep = r >= 0
        out[r[keep]] = o.view(-1, hkv, step, g, d).transpose(1, 2).reshape(-1, step, case["hq"], d)[keep]
        lse[r[keep]] = e.view(-1, hkv, step, g).transpose(1, 2).reshape(-1, step, case["hq"])[keep]
    return dict(out=out, lse=lse)


def _shared(st):
    """Each group's queries against its prefix in one product, every request against its own suffix, joined by maximum and sum."""
    case, pool, ps = st["case"], st["pool"], st["case"]["ps"]
    b, hkv, d, g = case["b"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    flat, scale = pool.view(-1, 2, hkv, d), case["d"] ** -0.5
    q = st["q"].float().view(b, hkv, g, d)
    parts, r0, p0 = [], 0, 0
    for size, length in zip(st["sizes"].tolist(), st["prefix"].tolist()):
        pages = st["prefix_pages"][p0:p0 + length // ps].long()
        rows = _rows(case, pool, pages[:, None], torch.arange(ps, device="cuda")).view(1, -1)
        kvs = flat[rows].float()
        x = _parts(q[r0:r0 + size].transpose(0, 1).reshape(1, hkv, size * g, d), kvs[:, :, 0], kvs[:, :, 1], None, scale)
        parts.append([y.view(hkv, size, g, *y.shape[3:]).transpose(0, 1) for y in x])
        r0, p0 = r0 + size, p0 + length // ps
    m1, l1, o1 = (torch.cat(x) for x in zip(*parts))
    j = torch.arange(st["max_suffix"], device="cuda")
    kvs = flat[_rows(case, pool, st["table"].long()[:, j // ps], j % ps)].float()
    m2, l2, o2 = _parts(q, kvs[:, :, 0], kvs[:, :, 1], (j < st["suffix_lens"][:, None])[:, None].expand(-1, g, -1), scale)
    m = torch.maximum(m1, m2)
    w1, w2 = (m1 - m).exp(), (m2 - m).exp()
    out, lse = _finished(m, w1 * l1 + w2 * l2, w1[..., None] * o1 + w2[..., None] * o2, st["q"].dtype)
    return dict(out=out.view_as(st["q"]), lse=lse.view(b, -1))


# ---------------------------------------------------------------------------
# the values in 64 bits, from the definitions
# ---------------------------------------------------------------------------

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
    case, pool = st["case"], st["pool"]
    page = pages[tokens // case["ps"]].long()
    rows = pool[page % case["cp"], page // case["cp"], tokens % case["ps"]].double()
    return rows.unflatten(1, (2, case["hkv"], case["d"])).unbind(1)


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
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
        full, page, off = pool.double(), st["slots"] // case["ps"], st["slots"] % case["ps"]
        parts = (st["v"].double(), k) if case["latent"] else (k, st["v"].double())
        full[page % case["cp"], page // case["cp"], off] = torch.cat([p.reshape(case["n"], -1) for p in parts], 1)
        return dict(q=q, pool=full)
    out, lse = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    q = st["q"].double()
    if case["op"] == "window":
        row = 0
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
                out[row:row + len(p)], lse[row:row + len(p)] = _softmax64(q[row:row + len(p)], k, v, hidden)
                row += len(p)
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
