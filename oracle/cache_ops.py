"""CPU oracle of the operators around the cache -- TEST INFRASTRUCTURE ONLY.

Plain numpy float64 definitions of rotary positions with scaled frequencies, the
e4m3 cache with one scale per block and KV head, attention over it, and block
copies and compaction.  Shares no code with the CUDA library.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities, the codes
0x7f and 0xff are NaN, the largest value is 448, subnormals are multiples of 2^-9.
"""
from __future__ import annotations

import math

import numpy as np


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]                      # 0 .. 448 in code order


def e4m3_codes(x):
    """float64 values as e4m3 codes: nearest, ties to the even code, saturating; NaN kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POS, np.where(np.isnan(a), 0.0, a))          # first code with value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(np.isnan(x), 0x7F, pick)
    return (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def block_scale(amax):
    """The smallest power of two s >= 2^-117 with amax <= 448 s (0 for 0)."""
    if amax == 0:
        return 0.0
    e = -117
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


class PoolF8:
    """codes uint8 [num_blocks, n_kv_heads, block_size, head_dim], scales float64 [num_blocks, n_kv_heads]."""

    def __init__(self, k, v, k_scale, v_scale):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @property
    def block_size(self):
        return self.k.shape[2]

    def append(self, k, v, table, context_lens, cu):
        """k, v float64 [tokens, n_kv_heads, head_dim]; bad blocks are skipped."""
        bs = self.block_size
        for b in range(len(context_lens)):
            n = int(cu[b + 1] - cu[b])
            p = int(context_lens[b]) - n
            t = int(cu[b])
            while n > 0:
                off = p % bs
                m = min(bs - off, n)
                blk = int(table[b][p // bs])
                if 0 <= blk < len(self.k):
                    for x, codes, scale in ((k, self.k, self.k_scale), (v, self.v, self.v_scale)):
                        for h in range(codes.shape[1]):
                            rows = x[t:t + m, h]
                            fin = np.abs(rows[np.isfinite(rows)])
                            s = block_scale(fin.max() if fin.size else 0.0)
                            if off:
                                old = float(scale[blk, h])
                                s = max(s, old)
                                if s > old:
                                    codes[blk, h, :off] = e4m3_codes(E4M3[codes[blk, h, :off]] * (old / s))
                            with np.errstate(divide="ignore", invalid="ignore"):
                                y = rows / s if s > 0 else np.where(np.isnan(rows), rows, 0.0)
                            codes[blk, h, off:off + m] = e4m3_codes(y)
                            scale[blk, h] = s
                p, t, n = p + m, t + m, n - m

    def rows(self, table_row, n, h):
        """(k, v, valid): the first n cached rows of a sequence for KV head h; rows without a block are zeros."""
        bs, d = self.block_size, self.k.shape[3]
        k, v, ok = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n, bool)
        for j in range(-(-n // bs)):
            blk, m = int(table_row[j]), min(bs, n - j * bs)
            if 0 <= blk < len(self.k):
                k[j * bs:j * bs + m] = E4M3[self.k[blk, h, :m]] * self.k_scale[blk, h]
                v[j * bs:j * bs + m] = E4M3[self.v[blk, h, :m]] * self.v_scale[blk, h]
                ok[j * bs:j * bs + m] = True
        return k, v, ok


def attention_f8(q, pool, table, context_lens, cu, scale):
    """Causal attention of the new tokens (rows cu[b] .. cu[b+1]-1 of q float64 [tokens, heads, d]).  Returns
    (out, weight, spread): the output, sum p |v| per element, and per row (largest scale * sum |q k| over the
    keys seen, number of keys, largest |v| among them)."""
    T, H, d = q.shape
    Hkv = pool.k.shape[1]
    G = H // Hkv
    out, weight, info = np.zeros((T, H, d)), np.zeros((T, H, d)), np.zeros((T, H, 3))
    for b in range(len(context_lens)):
        n, ctx = int(cu[b + 1] - cu[b]), int(context_lens[b])
        if n == 0 or ctx == 0:
            continue
        for hk in range(Hkv):
            k, v, ok = pool.rows(table[b], ctx, hk)
            for h in range(hk * G, hk * G + G):
                x = q[cu[b]:cu[b + 1], h]
                s = (x @ k.T) * scale
                seen = (np.arange(ctx)[None, :] <= (ctx - n + np.arange(n))[:, None]) & ok[None, :]
                s = np.where(seen, s, -np.inf)
                m = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
                tot = p.sum(1, keepdims=True)
                p /= np.where(tot > 0, tot, 1.0)
                out[cu[b]:cu[b + 1], h] = p @ v
                weight[cu[b]:cu[b + 1], h] = p @ np.abs(v)
                mag = np.where(seen, (np.abs(x) @ np.abs(k).T) * scale, 0.0)
                vmax = np.where(seen, np.abs(v).max(1)[None, :], 0.0).max(1)
                info[cu[b]:cu[b + 1], h] = np.stack((mag.max(1), seen.sum(1), vmax), 1)
    return out, weight, info


def largest_term(q, pool, table, context_lens, cu, scale):
    """Per query row [tokens, heads, 1]: the largest probability times 448 times the V scale of its key, a bound on
    any one key's share of the output."""
    ones = PoolF8(pool.k, np.full_like(pool.v, e4m3_codes(448.0)), pool.k_scale, pool.v_scale)
    T, H, _ = q.shape
    Hkv, top = pool.k.shape[1], np.zeros((T, H, 1))
    for b in range(len(context_lens)):
        n, ctx = int(cu[b + 1] - cu[b]), int(context_lens[b])
        for h in range(H if n else 0):
            k, v, ok = ones.rows(table[b], ctx, h // (H // Hkv))
            seen = (np.arange(ctx)[None, :] <= (ctx - n + np.arange(n))[:, None]) & ok[None, :]
            s = np.where(seen, (q[cu[b]:cu[b + 1], h] @ k.T) * scale, -np.inf)
            p = np.exp(s - np.max(s, 1, keepdims=True, initial=-1e300))
            top[cu[b]:cu[b + 1], h, 0] = (p / np.maximum(p.sum(1, keepdims=True), 1e-300) * v[:, 0]).max(1, initial=0.0)
    return top


def inv_freq(rotary_dim, theta=10000.0, scaling="plain", factor=1.0, original=0, low=1.0, high=None, magnitude=0.0):
    """(inverse frequencies float64, factor on cos and sin)."""
    high = high if high is not None else (32.0 if scaling == "yarn" else 4.0)
    half = rotary_dim // 2
    if scaling == "ntk":
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2.0))
    w = np.array([theta ** (-2.0 * i / rotary_dim) for i in range(half)])
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "banded":
        out = np.empty(half)
        for i in range(half):
            turns = original * w[i] / (2 * math.pi)
            t = 0.0 if turns <= low else 1.0 if turns >= high else (turns - low) / (high - low)
            out[i] = t * w[i] + (1 - t) * w[i] / factor
        return out, 1.0
    if scaling == "yarn":
        pair = lambda turns: rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rotary_dim - 1)
        r = np.clip((np.arange(half) - lo) / max(hi - lo, 0.001), 0, 1)
        return (1 - r) * w + r * w / factor, magnitude if magnitude > 0 else 0.1 * math.log(factor) + 1.0
    return w, 1.0


def rope(x, positions, freq, magnitude, layout, backward=False):
    """x float64 [tokens, heads, d] turned pair by pair."""
    half = len(freq)
    out = np.array(x)
    for i in range(half):
        i0, i1 = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        ang = positions.astype(np.float64) * freq[i]
        c, s = magnitude * np.cos(ang)[:, None], magnitude * np.sin(ang)[:, None]
        if backward:
            s = -s
        out[:, :, i0] = x[:, :, i0] * c - x[:, :, i1] * s
        out[:, :, i1] = x[:, :, i1] * c + x[:, :, i0] * s
    return out


def compact(table, num_blocks):
    """(new table, moves [(from, to)], blocks in use, map) -- ids outside the pool stay."""
    used = sorted({int(v) for v in np.asarray(table).ravel() if 0 <= v < num_blocks})
    U = len(used)
    holes = sorted(set(range(U)) - set(used))
    moves = list(zip([v for v in used if v >= U], holes))
    to = {v: v for v in used}
    to.update(dict(moves))
    new = np.array([[to.get(int(v), int(v)) for v in row] for row in table], np.int32).reshape(np.shape(table))
    block_map = np.array([to.get(v, -1) for v in range(num_blocks)], np.int32)
    return new, moves, U, block_map
