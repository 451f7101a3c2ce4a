"""Plain 64-bit implementations of quantised rows, written from their definition."""
import numpy as np
import torch

from paged_kv_cache_compose_gb300.cpkv import QuantisedRow

NAN = 0x7F


def e4m3_values():
    """The numbers of the 256 bytes: sign, four bits of exponent (bias 7), three of fraction; all ones are no number."""
    byte = np.arange(256)
    e, f = byte >> 3 & 15, byte & 7
    v = np.where(e == 0, f / 8 * 2.0**-6, (1 + f / 8) * 2.0 ** (e - 7.0))
    return np.where((byte & 127) == NAN, np.nan, np.where(byte < 128, v, -v))


VALUES = e4m3_values()


def scale_of(x):
    """The smallest power of two, 2^-126 at least, whose 448-fold reaches the largest finite magnitude of [..., group]."""
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    scale = np.full(top.shape, 2.0**-126)
    while (small := 448.0 * scale < top).any():
        scale = np.where(small, 2 * scale, scale)
    return scale


def to_e4m3(y):
    """The nearest byte, of two equally near the even one; no number for what is infinite or none."""
    mag = np.where(np.isfinite(y), np.abs(y), 0.0)
    up = np.clip(np.searchsorted(VALUES[:127], mag), 1, 126)
    low, high = mag - VALUES[up - 1], VALUES[up] - mag
    byte = np.where((low < high) | ((low == high) & (up % 2 == 1)), up - 1, up)
    return np.where(np.isfinite(y), byte | np.where(np.signbit(y), 128, 0), NAN).astype(np.uint8)


def quantise(x):
    """[..., group] in 64 bits -> (bytes, scales)."""
    scale = scale_of(x)
    return to_e4m3(x / scale[..., None]), scale.astype(np.float32)


def groups(row: QuantisedRow) -> int:
    """Scales of a value head."""
    return max(1, row.value_dim // 128)


class Pools:
    """Owner slabs [cp][pages, ps, row bytes] on the host; kept keys in ``dtype``."""

    def __init__(self, n_pages, ps, cp, row: QuantisedRow, dtype, width=None):
        self.ps, self.cp, self.row, self.dtype = ps, cp, row, dtype
        cap = -(-(n_pages + 1) // cp)
        self.slabs = [np.zeros((cap, ps, width or row.row_bytes), np.uint8) for _ in range(cp)]

    def at(self, page, off):
        return self.slabs[page % self.cp][page // self.cp, off]

    def put(self, page, off, k, v):
        """Keys [kv_heads, key_dim] and values [kv_heads, value_dim] in 64 bits."""
        row, to = self.row, self.at(page, off)
        bytes_, scales = quantise(v.reshape(row.kv_heads * groups(row), -1))
        to[row.value_offset:row.value_offset + bytes_.size] = bytes_.reshape(-1)
        to[row.value_scale_offset:row.value_scale_offset + 4 * scales.size] = scales.view(np.uint8)
        if row.keep_keys:
            bits = torch.from_numpy(k.reshape(-1)).to(self.dtype).view(torch.uint8).numpy()
            to[row.key_offset:row.key_offset + bits.size] = bits
        else:
            bytes_, scales = quantise(k)
            to[row.key_offset:row.key_offset + bytes_.size] = bytes_.reshape(-1)
            to[row.key_scale_offset:row.key_scale_offset + 4 * scales.size] = scales.view(np.uint8)

    def fill(self, rng, spread=0.4):
        """Every row: normal keys and values, whose magnitude differs from head to head."""
        row = self.row
        for slab in self.slabs:
            n = slab.shape[0] * slab.shape[1]
            k = rng.standard_normal((n, row.kv_heads, row.key_dim)) * np.exp(spread * rng.standard_normal((n, row.kv_heads, 1)))
            v = rng.standard_normal((n, row.kv_heads, row.value_dim)) * np.exp(spread * rng.standard_normal((n, row.kv_heads, 1)))
            flat = slab.reshape(n, -1)
            bytes_, scales = quantise(v.reshape(n, row.kv_heads * groups(row), -1))
            flat[:, row.value_offset:row.value_offset + row.kv_heads * row.value_dim] = bytes_.reshape(n, -1)
            flat[:, row.value_scale_offset:row.value_scale_offset + 4 * scales.shape[1]] = scales.view(np.uint8).reshape(n, -1)
            if row.keep_keys:
                bits = torch.from_numpy(k.reshape(n, -1)).to(self.dtype).view(torch.uint8).numpy()
                flat[:, row.key_offset:row.key_offset + bits.shape[1]] = bits
            else:
                bytes_, scales = quantise(k)
                flat[:, row.key_offset:row.key_offset + row.kv_heads * row.key_dim] = bytes_.reshape(n, -1)
                flat[:, row.key_scale_offset:row.key_scale_offset + 4 * row.kv_heads] = scales.view(np.uint8).reshape(n, -1)
        return self

    def rows(self, raw):
        """(keys [n, kv_heads, key_dim], values [n, kv_heads, value_dim]) of raw rows [n, bytes], in 64 bits."""
        row = self.row
        n, raw = len(raw), np.ascontiguousarray(raw)

        def floats(at, count):
            return np.ascontiguousarray(raw[:, at:at + 4 * count]).view(np.float32).reshape(n, count).astype(np.float64)

        v = VALUES[raw[:, row.value_offset:row.value_offset + row.kv_heads * row.value_dim]].reshape(n, row.kv_heads * groups(row), -1)
        v = (v * floats(row.value_scale_offset, row.kv_heads * groups(row))[..., None]).reshape(n, row.kv_heads, row.value_dim)
        if row.keep_keys:
            bits = np.ascontiguousarray(raw[:, row.key_offset:row.key_offset + 2 * row.kv_heads * row.key_dim])
            k = torch.from_numpy(bits).view(self.dtype).double().numpy().reshape(n, row.kv_heads, row.key_dim)
        else:
            k = VALUES[raw[:, row.key_offset:row.key_offset + row.kv_heads * row.key_dim]].reshape(n, row.kv_heads, row.key_dim)
            k = k * floats(row.key_scale_offset, row.kv_heads)[..., None]
        return k, v

    def cuda(self):
        return [torch.from_numpy(s).cuda() for s in self.slabs]


class Dense:
    """The rows read back, as the models of attention over plain rows look them up: keys, then values."""

    def __init__(self, pools: Pools):
        self.pools, self.ps = pools, pools.ps

    def row(self, page, off):
        k, v = self.pools.rows(self.pools.at(page, off)[None])
        return torch.from_numpy(np.concatenate([k.reshape(-1), v.reshape(-1)]))

    def rows(self, pages, n):
        if n == 0:
            return torch.zeros((0, self.pools.row.kv_heads * (self.pools.row.key_dim + self.pools.row.value_dim)), dtype=torch.float64)
        k, v = self.pools.rows(np.stack([self.pools.at(int(pages[t // self.ps]), t % self.ps) for t in range(n)]))
        return torch.from_numpy(np.concatenate([k.reshape(n, -1), v.reshape(n, -1)], 1))


def rotated(x, table, positions, axis, interleaved):
    """[n, heads, dim] in 64 bits, rotated."""
    half = table.shape[1] // 2
    y = x.copy()
    for i in range(half):
        c = table[positions[axis[i]], i].astype(np.float64)[:, None]
        s = table[positions[axis[i]], half + i].astype(np.float64)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y
