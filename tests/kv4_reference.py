"""Plain implementations, in 64 bits, of the operators around the 4-bit KV cache (test infrastructure).

Written from the header's definitions: loops and index formulas, no code shared with the kernels.
"""
import math

import numpy as np
import torch

SLOTS, GROUP = 16, 32


def to_bf16(x):
    """Round float64 to bf16 (half to even) and back. Values here have at most 24 bits: float32 holds them."""
    return torch.as_tensor(np.asarray(x, dtype=np.float64)).to(torch.float32).to(torch.bfloat16).double().numpy()


def quantise(x):
    """Rows [..., d] -> (codes [..., d] int, scales [..., d / 32])."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    codes = np.zeros(g.shape, dtype=np.int64)
    a = np.abs(g).max(-1)                       # NaN propagates
    over = ~(to_bf16(np.where(np.isfinite(a), a, 0.0)) <= 2.0 ** 60) | ~np.isfinite(a)
    a = to_bf16(np.where(over, 0.0, a))
    scale = np.where(a < 2.0 ** -60, 0.0, to_bf16(a / 7.0))
    live = scale > 0
    q = g[live] / scale[live][:, None]          # 24 by 8 bits: no quotient is within 2^-53 of a border without being on it
    codes[live] = np.rint(q)
    return codes.reshape(x.shape), np.where(over, math.nan, scale)


def values(codes, scale):
    with np.errstate(invalid="ignore"):
        return codes * np.repeat(scale, GROUP, axis=-1)


def place(which, slot, col, d):
    """(byte, half of the byte) of a code in a K (0) or V (1) tile."""
    j, r = divmod(col, 32)
    if which == 0:
        t, p, h = r // 8, r % 8 // 2, r % 2
        return slot * (d // 2) + t * (d // 8) + 4 * j + 2 * h + p // 2, p % 2
    g, p = divmod(r, 4)
    e, t, h = slot // 8, slot % 8 // 2, slot % 2
    return e * 4 * d + t * d + g * (d // 8) + 4 * j + 2 * h + p // 2, p % 2


class Pool:
    """A pool as bytes on the host; rows written and read code by code."""

    def __init__(self, pages, nkv, d, fill=None):
        self.nkv, self.d, self.pages = nkv, d, pages
        self.raw = np.zeros((pages, nkv, 2, 9 * d), dtype=np.uint8) if fill is None else fill.reshape(
            pages, nkv, 2, 9 * d).copy()
        at = np.array([[[place(w, s, c, d) for c in range(d)] for s in range(SLOTS)] for w in (0, 1)])
        self.byte, self.half = at[..., 0], at[..., 1]

    def write(self, slots, k, v):
        for which, x in ((0, k), (1, v)):
            codes, scale = quantise(x)
            bits = (to_bits(scale)).view(np.uint8).reshape(*scale.shape, 2)
            for t, slot in enumerate(slots):
                if slot < 0 or slot // SLOTS >= self.pages:
                    continue
                page, s = divmod(int(slot), SLOTS)
                tile = self.raw[page, :, which]
                for half in (0, 1):
                    cols = np.nonzero(self.half[which, s] == half)[0]
                    b = self.byte[which, s, cols]
                    keep = 0xF0 if half == 0 else 0x0F
                    tile[:, b] = (tile[:, b] & keep) | ((codes[t][:, cols] + 8) << (4 * half)).astype(np.uint8)
                at = 8 * self.d + s * (self.d // GROUP) * 2
                tile[:, at:at + self.d // GROUP * 2] = bits[t].reshape(self.nkv, -1)

    def pages64(self, pages):
        """(K, V) [n, nkv, 16, d] float64 of whole pages."""
        out = []
        for which in (0, 1):
            tile = self.raw[pages][:, :, which]
            codes = (tile[:, :, self.byte[which]] >> (4 * self.half[which])) % 16
            scale = from_bits(np.ascontiguousarray(tile[:, :, 8 * self.d:]).view(np.uint16))
            scale = scale.reshape(*tile.shape[:2], SLOTS, -1)
            out.append(values(codes.astype(np.int64) - 8, scale))
        return out

    def rows(self, slots):
        slots = np.asarray(slots)
        k, v = self.pages64(slots // SLOTS)
        n = np.arange(len(slots))
        return k[n, :, slots % SLOTS], v[n, :, slots % SLOTS]


def to_bits(x):
    t = torch.as_tensor(np.asarray(x, dtype=np.float64)).to(torch.float32).to(torch.bfloat16)
    bits = t.view(torch.int16).numpy().view(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), bits)   # (torch's conversion gives NaN different bits by length)


def from_bits(b):
    return torch.from_numpy(b.view(np.int16).copy()).view(torch.bfloat16).double().numpy()


def attention(q, K, V, scale):
    """One KV head: q [G, d], K and V [n, d] -> (out [G, d], sum of weight times |V| [G, d])."""
    if len(K) == 0:
        z = np.zeros_like(q)
        return z, z
    x = q @ K.T * scale
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ V, w @ np.abs(V)


def page_map(ctx, new, table, free, free_count, num_pages, page_cap, token_cap):
    """The documented result: dict of lists, with the status words that may be latched."""
    R, stride = table.shape
    table = table.copy()
    status = set()
    if not 0 <= free_count <= len(free):
        status.add(6)
        free_count = min(max(free_count, 0), len(free))
    plan, asked, taken = [], 0, 0
    for r in range(R):
        c, n = int(ctx[r]), int(new[r])
        if c < 0 or n < 0:
            status.add(6)
            c = n = 0
        b, a = -(-c // 16), -(-(c + n) // 16)
        if b > stride:
            status.add(6)
            plan.append((c, n, 0, 0, None, True))
            continue
        if a > stride:
            status.add(6)
            plan.append((c, n, b, b, None, False))
            continue
        first = asked
        asked += a - b
        if a > b and asked > free_count:
            status.add(3)
            plan.append((c, n, b, b, None, False))
        else:
            taken += a - b
            plan.append((c, n, b, a, first, False))
    pages, tokens = sum(p[3] for p in plan), sum(p[1] for p in plan)
    if pages > page_cap or tokens > token_cap:
        return {"status": status | {6}, "table": table, "kv_len": [0] * R, "indptr": [0] * (R + 1), "indices": [],
                "slots": [-1] * min(tokens, token_cap), "positions": [], "left": free_count}
    out = {"status": status, "table": table, "kv_len": [], "indptr": [0], "indices": [], "slots": [], "positions": [],
           "left": free_count - taken}
    for r, (c, n, b, a, first, dead) in enumerate(plan):
        for i in range(b, a):
            table[r, i] = free[free_count - 1 - (first + i - b)]
        row = [int(x) for x in table[r, :a]]
        if any(not 0 <= x < num_pages for x in row):
            status.add(6)
        out["kv_len"].append(0 if dead else c + (n if first is not None else 0))
        out["indices"] += row
        out["indptr"].append(len(out["indices"]))
        for i in range(n):
            pos = c + i
            ok = first is not None and 0 <= row[pos // 16] < num_pages
            out["slots"].append(row[pos // 16] * 16 + pos % 16 if ok else -1)
            out["positions"].append(min(pos, 2 ** 31 - 1))
    return out


def rope(x, positions, freq, scale, rot, interleaved):
    """x [T, heads, d] float64."""
    y = np.array(x, dtype=np.float64)
    angle = positions.astype(np.float64)[:, None] * freq
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
