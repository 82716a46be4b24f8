"""Attention weights of cached positions against their float64 definition on a GPU.

Tolerance of a weight.  A score's float32 error: d products and sums on the tensor core, which may cut instead of round,
2^-23 each of sum |q k| scale (d + 8 of them; INT8: the code is exact, the scale's product 2^-24 more, inside that), and
2^-22 of the score for the factors; exponentiated it is relative to the weight.  The exponentials 2^-21 each, the sum of
n probabilities in float32 (n / 16 + 160) 2^-23 relative, the logarithm of the sum 2^-22 of itself and of the largest
score (their difference from the score is rounded at that size).  The sum over the heads and rows adds
(heads * rows / 8 + 16) 2^-23 relative, and the sum so far one rounding.
"""
import math

import numpy as np
import pytest
import torch

from oracle import llama_layer as O
from oracle import weight_ops as W
from tests.helpers import f64
from transformer_decoder_layer_llama_gb300 import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api

LOG2E = 1.4426950408889634


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def check_status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


class Paged:
    """A paged cache of some sequences: blocks in random order, garbage (NaN in BF16 pools) behind every context."""

    def __init__(self, ctx, kv_heads, dim, block, seed, int8=False, spare=1):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // block) for n in ctx]
        wide, nb = max(need) + spare, sum(need) + 2
        perm = torch.randperm(nb, generator=g).tolist()
        self.table = np.full((len(ctx), wide), -1, np.int64)
        for b, n in enumerate(need):
            self.table[b, :n] = [perm.pop() for _ in range(n)]
        k, v = (torch.randn(nb, kv_heads, block, dim, generator=g).bfloat16() for _ in range(2))
        k[..., ::max(dim // 4, 1)] *= 4
        self.ctx, self.block, self.int8 = list(ctx), block, int8
        if int8:
            sets = []
            for x in (k, v):
                s = x.float().abs().amax(-1) / 127
                sets += [torch.round(x.float() / s[..., None]).to(torch.int8), s]
            self.kq, ks, vq, vs = sets
            self.pool = api.PoolQ8(self.kq.cuda(), vq.cuda(), ks.cuda(), vs.cuda())
            self.k_rows, self.v_rows = (c.numpy().astype(np.float64) * f64(s)[..., None] for c, s in ((self.kq, ks), (vq, vs)))
        else:
            self.k_rows, self.v_rows = f64(k), f64(v)
            for b, n in enumerate(ctx):                       # NaN behind the contexts, and in blocks of nobody
                if n % block:
                    k[self.table[b, n // block], :, n % block:] = math.nan
                    v[self.table[b, n // block], :, n % block:] = math.nan
            free = sorted(set(range(nb)) - set(self.table[self.table >= 0].tolist()))
            k[free], v[free] = math.nan, math.nan
            self.k, self.v = k.cuda(), v.cuda()
        self.d_table, self.d_ctx = i32(self.table), i32(ctx)

    def rows(self, which, b, h, hole=()):
        """float64 rows of sequence b and KV head h, and which positions have a block."""
        at = np.arange(self.ctx[b])
        blk = self.table[b, at // self.block]
        ok = np.array([j not in hole for j in at // self.block], dtype=bool) & (blk >= 0)
        x = (self.k_rows if which == "k" else self.v_rows)[np.where(ok, blk, 0), h, at % self.block]
        return x, ok


def reference(paged, q, cu, scale, base, holes={}):
    """(weights float64, their bounds) after the rows q [tokens, heads, d] of every sequence."""
    w, bound = f64(base), np.abs(f64(base)) * 2.0 ** -24
    B, Hkv, width = w.shape
    G = q.shape[1] // Hkv
    d = q.shape[2]
    for b, n in enumerate(paged.ctx):
        rows = q[cu[b]:cu[b + 1]]
        m = len(rows)
        if not m or not n:
            continue
        for h in range(Hkv):
            k, ok = paged.rows("k", b, h, holes.get(b, ()))
            qq = rows[:, h * G:(h + 1) * G]
            s = np.einsum("igd,md->igm", qq, k) * scale
            size = np.einsum("igd,md->igm", np.abs(qq), np.abs(k)) * scale
            seen = (np.arange(n)[None, None] <= (n - m + np.arange(m))[:, None, None]) & ok
            s = np.where(seen, s, -np.inf)
            top = s.max(-1, keepdims=True, initial=-np.inf)
            p = np.exp(s - np.where(np.isfinite(top), top, 0))
            tot = p.sum(-1, keepdims=True)
            p = np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)
            largest = np.where(np.isfinite(top), np.abs(top), 0) + np.log(np.maximum(tot, 1))
            score = (d + 8) * 2.0 ** -23 * size + 2.0 ** -22 * (np.where(seen, np.abs(s), 0) + 2 * largest)
            # a score's error moves its own weight, and the row's normaliser by at most the largest error among its weights
            own = score + (p * score).sum(-1, keepdims=True)
            rel = own + 2 * 2.0 ** -21 + (n / 16 + 160) * 2.0 ** -23 + (m * G / 8 + 16) * 2.0 ** -23
            end = min(n, width)
            w[b, h, :end] += p.sum((0, 1))[:end]
            bound[b, h, :end] += (p * rel).sum((0, 1))[:end] + p.sum((0, 1))[:end] * 2.0 ** -24
    return w, bound * 1.01 + 2.0 ** -120


def assert_weights(got, ref, bound):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all()
    assert (err <= bound + 2.0 ** -24 * np.abs(ref)).all(), float((err / bound).max())


DECODE = [  # contexts, heads, kv_heads, dim, block
    ([1], 1, 1, 64, 16), ([5, 64, 65], 4, 2, 64, 16), ([1, 0, 200], 8, 8, 128, 32), ([1024, 1025, 3, 2047], 6, 2, 128, 64),
    ([300, 77], 16, 1, 128, 128), ([129], 9, 1, 64, 256), ([4099, 31], 5, 1, 128, 256), ([2500] * 3, 14, 2, 64, 32),
    ([9000, 100, 8193], 8, 1, 128, 128)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, int8):
    ctx, H, Hkv, d, block = case
    if int8 and d != 128:
        d = 128
    c = Paged(ctx, Hkv, d, block, 7 * len(ctx) + H, int8)
    g = torch.Generator().manual_seed(H)
    q = torch.randn(len(ctx), H, d, generator=g).bfloat16().cuda()
    width = c.table.shape[1] * block + 3
    base = torch.rand(len(ctx), Hkv, width, generator=g).cuda()
    w, st, scale = base.clone(), api.new_status(), 1 / math.sqrt(d)
    if int8:
        out = api.paged_attention_decode_weights_q8(q, c.pool, c.d_table, c.d_ctx, scale, w, status=st)
        plain = api.paged_attention_decode_q8(q, c.pool, c.d_table, c.d_ctx, scale)
    else:
        out = api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, scale, w, status=st)
        plain = api.paged_attention_decode(q, c.k, c.v, c.d_table, c.d_ctx, scale)
    check_status(st)
    assert torch.equal(out, plain)                              # the output is that of the call without weights
    ref, bound = reference(c, f64(q), list(range(len(ctx) + 1)), scale, base)
    assert_weights(w, ref, bound)
    for b, n in enumerate(ctx):
        assert torch.equal(w[b, :, n:], base[b, :, n:])         # behind the context: left
        added = f64(w[b]).sum(-1) - f64(base[b]).sum(-1)
        assert np.allclose(added, H // Hkv if n else 0, atol=1e-3)
    again = base.clone()
    if not int8:
        ws = torch.full((api.attention_decode_weights_workspace_size(len(ctx), H, Hkv, d, c.table.shape[1], block),), 255,
                        dtype=torch.uint8, device="cuda")
        api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, scale, again, out=out, workspace=ws, status=st)
        check_status(st)
        assert torch.equal(again, w)                            # the same bits, whatever the workspace held


def test_decode_edges():
    """Bad blocks add nothing, narrow weights are flagged, bad contexts are cut, a scale of 0, an infinite query."""
    c = Paged([40, 90, 64], 2, 64, 16, 3)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    table = c.table.copy()
    table[1, 2] = 10 ** 6
    table[2, :] = -1
    base = torch.rand(3, 2, 112, generator=torch.Generator().manual_seed(2)).cuda()
    w, st = base.clone(), api.new_status()
    out = api.paged_attention_decode_weights(q, c.k, c.v, i32(table), c.d_ctx, 0.125, w, status=st)
    check_status(st, api.LL_DEV_BAD_BLOCK)
    ref, bound = reference(c, f64(q), [0, 1, 2, 3], 0.125, base, {1: (2,), 2: range(9)})
    assert_weights(w, ref, bound)
    assert torch.equal(w[1, :, 32:48], base[1, :, 32:48]) and torch.equal(w[2], base[2]) and (out[2] == 0).all()
    w, st = base[..., :48].contiguous(), api.new_status()
    api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, 0.125, w, status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    ref, bound = reference(c, f64(q), [0, 1, 2, 3], 0.125, base[..., :48])
    assert_weights(w, ref, bound)
    w, st = torch.zeros(3, 2, 112).cuda(), api.new_status()
    api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, 0.0, w, status=st)
    check_status(st)
    for b, n in enumerate(c.ctx):
        assert np.allclose(f64(w[b, :, :n]), 2 / n, rtol=1e-5) and (w[b, :, n:] == 0).all()
    w, st = base.clone(), api.new_status()
    api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, i32([40, -3, 5000]), 0.125, w, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & api.LL_DEV_BAD_POSITION and torch.equal(w[1], base[1])
    ref, bound = reference(c, f64(q), [0, 1, 1, 1], 0.125, base)
    assert (np.abs(f64(w[0]) - ref[0]) <= bound[0] + 2.0 ** -24 * np.abs(ref[0])).all()


def test_decode_streams_and_graphs():
    c = Paged([500, 1300], 2, 128, 64, 5)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    zero = lambda: torch.zeros(2, 2, c.table.shape[1] * 64, device="cuda")  # noqa: E731
    want = zero()
    out = api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, 0.1, want)
    torch.cuda.synchronize()
    side, w = torch.cuda.Stream(), zero()
    side.wait_stream(torch.cuda.current_stream())
    o2 = api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, 0.1, w, stream=side)
    side.synchronize()
    assert torch.equal(w, want) and torch.equal(o2, out)
    w, o3, st = zero(), torch.zeros_like(out), api.new_status()
    ws = torch.empty(api.attention_decode_weights_workspace_size(2, 8, 2, 128, c.table.shape[1], 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, c.d_ctx, 0.1, w, out=o3, workspace=ws, status=st)
    for step in (1, 2):
        graph.replay()
        check_status(st)
        assert torch.equal(o3, out)
        assert (f64(w) - step * f64(want) <= 2.0 ** -22 * step * f64(want)).all()


# ---------------------------------------------------------------- prompts, chunks, last rows

PROMPT = [  # contexts, new rows, heads, kv_heads, dim, block
    ([1], [1], 1, 1, 64, 16), ([5, 64, 65], [5, 3, 65], 4, 2, 64, 16), ([200, 17, 130], [1, 0, 130], 8, 8, 128, 32),
    ([700], [700], 2, 2, 128, 128), ([300, 77], [64, 77], 16, 1, 128, 128), ([129, 500], [40, 31], 9, 1, 64, 256),
    ([1100], [259], 5, 1, 128, 256), ([600] * 3, [32] * 3, 14, 2, 64, 32), ([2100, 100, 1025], [33, 100, 2], 8, 1, 128, 64),
    ([4000], [17], 6, 2, 128, 128), ([1300], [1300], 3, 1, 64, 64)]


def prompt(case, seed=0):
    ctx, new, H, Hkv, d, block = case
    c = Paged(ctx, Hkv, d, block, 11 * len(ctx) + H + seed)
    g = torch.Generator().manual_seed(H + seed)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    q = torch.randn(cu[-1], H, d, generator=g).bfloat16().cuda()
    base = torch.rand(len(ctx), Hkv, c.table.shape[1] * block + 3, generator=g).cuda()
    return c, q, cu, base


@pytest.mark.parametrize("case", PROMPT)
def test_prompt(case):
    ctx, new, H, Hkv, d, block = case
    c, q, cu, base = prompt(case)
    w, st, scale = base.clone(), api.new_status(), 1 / math.sqrt(d)
    got = api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, scale, w, max(new), status=st)
    check_status(st)
    assert got is w
    ref, bound = reference(c, f64(q), cu, scale, base)
    assert_weights(w, ref, bound)
    for b, n in enumerate(ctx):
        end = n if new[b] else 0
        assert torch.equal(w[b, :, end:], base[b, :, end:])
    # the same bits again, whatever the workspace held; an upper bound of the rows may split them otherwise
    for more in (max(new), max(new) + 50):
        again = base.clone()
        ws = torch.full((api.attention_weights_workspace_size(len(ctx), cu[-1], more, H, Hkv, d, c.table.shape[1], block),), 255,
                        dtype=torch.uint8, device="cuda")
        api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, scale, again, more, workspace=ws, status=st)
        check_status(st)
        assert_weights(again, ref, bound)
        assert more > max(new) or torch.equal(again, w)


@pytest.mark.parametrize("case", [
    ([(37 * i) % 900 for i in range(70)], [min((37 * i) % 900, i % 5) for i in range(70)], 4, 1, 64, 16), ([39000], [20], 8, 1, 128, 256),
    ([9000] + [300] * 90, [1] * 91, 16, 8, 64, 64), ([300] * 40 + [0, 7000], [2] * 40 + [0, 64], 4, 2, 128, 128), ([500], [84], 3, 1, 128, 32),
    ([500, 600], [85, 3], 3, 1, 128, 32), ([2600] * 5, [16] * 5, 32, 32, 64, 128)])
def test_windows(case):
    """Few rows: every CTA has a share of all sequences' and heads' keys, so that a head's may lie in many parts."""
    test_prompt(case)


def test_prompt_equals_its_single_tokens():
    """A chunk's weights are those of its rows as decode steps, but for rounding."""
    case = ([150, 90], [7, 3], 8, 2, 128, 32)
    c, q, cu, base = prompt(case)
    w = api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.09, base.clone(), 7)
    steps = base.clone()
    for i in range(7):
        ctx = [150 - 7 + i + 1, 90 - 3 + i + 1 if i < 3 else 0]
        rows = torch.stack([q[i], q[7 + min(i, 2)]])
        api.paged_attention_decode_weights(rows, c.k, c.v, c.d_table, i32(ctx), 0.09, steps)
    ref, bound = reference(c, f64(q), cu, 0.09, base)
    assert_weights(w, ref, bound)
    assert (np.abs(f64(w) - f64(steps)) <= 2 * bound + 2.0 ** -20 * np.abs(ref)).all()


def test_prompt_edges():
    """Counts that do not fit, bad blocks, rows of nobody (NaN), narrow weights, no rows."""
    case = ([60, 50, 90, 40], [20, 10, 30, 5], 4, 2, 64, 16)
    c, q, cu, base = prompt(case)
    pad = torch.full((9, 4, 64), math.nan).bfloat16().cuda()
    wide = torch.cat([pad, q, pad])
    cu9 = [x + 9 for x in cu]
    table = c.table.copy()
    table[2, 1] = 10 ** 6
    w, st = base.clone(), api.new_status()
    api.paged_attention_weights(wide, i32(cu9), c.k, i32(table), i32([60, 8, 90, 40]), 0.125, w, 30, status=st)     # 8 < 10 rows
    check_status(st, api.LL_DEV_BAD_POSITION | api.LL_DEV_BAD_BLOCK)
    ref, bound = reference(c, f64(q), cu, 0.125, base, {2: (1,)})
    for b in (0, 2, 3):
        assert (np.abs(f64(w[b]) - ref[b]) <= bound[b] + 2.0 ** -24 * np.abs(ref[b])).all()
    assert torch.equal(w[1], base[1]) and torch.equal(w[2, :, 16:32], base[2, :, 16:32])
    for bad in (dict(max_new=29), dict(cu=[9, 29, 25, 69, 74]), dict(cu=[9, 29, 39, 69, 200]), dict(cu=[-1, 29, 39, 69, 74])):
        w, st = base.clone(), api.new_status()
        api.paged_attention_weights(wide, i32(bad.get("cu", cu9)), c.k, c.d_table, c.d_ctx, 0.125, w, bad.get("max_new", 60), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == api.LL_DEV_BAD_POSITION
        assert torch.equal(w[0], base[0]) or bad.get("cu", [0])[0] != -1
    narrow, st = base[..., :70].contiguous(), api.new_status()
    api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.125, narrow, 30, status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    ref, bound = reference(c, f64(q), cu, 0.125, base[..., :70])
    assert_weights(narrow, ref, bound)
    w, st = torch.zeros_like(base), api.new_status()                    # a scale of 0: equal weights
    api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.0, w, 30, status=st)
    check_status(st)
    for b, n in enumerate(c.ctx):
        m = case[1][b]
        want = sum(np.where(np.arange(n) <= n - m + i, 2 / (n - m + i + 1), 0) for i in range(m))
        assert np.allclose(f64(w[b, :, :n]), want, rtol=1e-5) and (w[b, :, n:] == 0).all()
    w, st = base.clone(), api.new_status()
    api.paged_attention_weights(q[:0], i32([0] * 5), c.k, c.d_table, c.d_ctx, 0.125, w, 3, status=st)
    check_status(st)
    assert torch.equal(w, base)


def test_prompt_edges_of_many_rows():
    """As above where a sequence has more rows than stay beside its keys."""
    case = ([300, 350, 420, 40], [200, 150, 300, 5], 4, 2, 64, 16)
    c, q, cu, base = prompt(case)
    pad = torch.full((9, 4, 64), math.nan).bfloat16().cuda()
    wide, cu9 = torch.cat([pad, q, pad]), [x + 9 for x in cu]
    table = c.table.copy()
    table[2, [1, 20]] = 10 ** 6, -1
    w, st = base.clone(), api.new_status()
    api.paged_attention_weights(wide, i32(cu9), c.k, i32(table), i32([300, 149, 420, 40]), 0.125, w, 300, status=st)   # 149 < 150 rows
    check_status(st, api.LL_DEV_BAD_POSITION | api.LL_DEV_BAD_BLOCK)
    ref, bound = reference(c, f64(q), cu, 0.125, base, {2: (1, 20)})
    for b in (0, 2, 3):
        assert (np.abs(f64(w[b]) - ref[b]) <= bound[b] + 2.0 ** -24 * np.abs(ref[b])).all()
    assert torch.equal(w[1], base[1]) and torch.equal(w[2, :, 16:32], base[2, :, 16:32]) and torch.equal(w[2, :, 320:336], base[2, :, 320:336])
    w, st = torch.zeros_like(base), api.new_status()                    # a scale of 0: equal weights
    api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.0, w, 300, status=st)
    check_status(st)
    for b, n in enumerate(c.ctx):
        m = case[1][b]
        want = sum(np.where(np.arange(n) <= n - m + i, 2 / (n - m + i + 1), 0) for i in range(m))
        assert np.allclose(f64(w[b, :, :n]), want, rtol=1e-5) and (w[b, :, n:] == 0).all()


@pytest.mark.parametrize("which", ["a query row", "a key"])
def test_nan_in_a_window(which):
    """As below for few rows: their keys lie in several CTAs' shares."""
    n, m = 2900, 20
    for at in (0, 7, 19):
        c, q, cu, base = prompt(([n], [m], 4, 2, 64, 64))
        if which == "a query row":
            q[at, 1, 7] = math.nan
            head, end = 0, n - m + at + 1                     # its KV head; the positions that it sees
        else:
            key = n - m + at
            c.k[c.table[0, key // 64], 1, key % 64, 3] = math.nan
            head, end = 1, n                                  # rows from `at` on see it, the last of them all
        w, st = base.clone(), api.new_status()
        api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.125, w, m, status=st)
        check_status(st)
        nan = np.zeros(w.shape, dtype=bool)
        nan[0, head, :end] = True
        assert (np.isnan(f64(w)) == nan).all()


@pytest.mark.parametrize("which", ["a query row", "a key"])
def test_nan_reaches_what_it_is_a_score_of(which):
    """A NaN in a row's query: every position that the row sees.  In a key: every position, of every row that sees it."""
    ctx, new, H, Hkv, d, block = [700], [300], 4, 2, 64, 64
    for at in (0, 5, 123, 299):
        c, q, cu, base = prompt((ctx, new, H, Hkv, d, block))
        if which == "a query row":
            q[at, 1, 7] = math.nan
            hit = [0], range(400 + at + 1)                   # its KV head; the positions that it sees
        else:
            key = 400 + at
            c.k[c.table[0, key // block], 1, key % block, 3] = math.nan
            hit = [1], range(700)                            # rows from `at` on see it, the last of them all
        w, st = base.clone(), api.new_status()
        api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 0.125, w, 300, status=st)
        check_status(st)
        nan = np.zeros(w.shape, dtype=bool)
        for h in hit[0]:
            nan[0, h, list(hit[1])] = True
        assert (np.isnan(f64(w)) == nan).all()


def test_prompt_far_below_its_largest_score():
    """Scores far apart: what is far below the largest adds nothing to speak of, and no noise to the rest."""
    ctx, new, H, Hkv, d, block = [520], [40], 2, 1, 64, 64
    c, q, cu, _ = prompt((ctx, new, H, Hkv, d, block))
    w, st = torch.zeros(1, 1, c.table.shape[1] * block).cuda(), api.new_status()
    api.paged_attention_weights(q, i32(cu), c.k, c.d_table, c.d_ctx, 40.0, w, 40, status=st)
    check_status(st)
    ref, bound = reference(c, f64(q), cu, 40.0, torch.zeros(w.shape))
    assert_weights(w, ref, bound)


def test_prompt_streams_and_graphs():
    case = ([500, 300], [100, 90], 8, 2, 128, 64)
    c, q, cu, base = prompt(case)
    cu = i32(cu)
    want = api.paged_attention_weights(q, cu, c.k, c.d_table, c.d_ctx, 0.1, base.clone(), 100)
    torch.cuda.synchronize()
    side, w = torch.cuda.Stream(), base.clone()
    side.wait_stream(torch.cuda.current_stream())
    api.paged_attention_weights(q, cu, c.k, c.d_table, c.d_ctx, 0.1, w, 100, stream=side)
    side.synchronize()
    assert torch.equal(w, want)
    w, st = base.clone(), api.new_status()
    ws = torch.empty(api.attention_weights_workspace_size(2, 190, 100, 8, 2, 128, c.table.shape[1], 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention_weights(q, cu, c.k, c.d_table, c.d_ctx, 0.1, w, 100, workspace=ws, status=st)
    graph.replay()
    check_status(st)
    assert torch.equal(w, want)


# ---------------------------------------------------------------- calls that follow each other on one stream

@pytest.mark.parametrize("int8", [False, True])
def test_calls_of_a_stream_share_a_workspace(int8):
    """Prompts' weights and then a step's, and steps of other batches, over one workspace without a wait between: the same
    bits as with workspaces of their own.  (The step's first kernel starts before the one in front has ended.)"""
    H, Hkv, d, block = 8, 2, 128, 64
    long = Paged([1900], Hkv, d, block, 1)                               # the normalisers of its rows: 1900 x 8
    wide = Paged([700, 9000, 65, 3000, 1024, 8000], Hkv, d, block, 2, int8)
    few = Paged([8300, 20], Hkv, d, block, 3, int8)                      # (nine splits: BF16 calls have a dispatch order too)
    one = Paged([40], Hkv, d, block, 4, True)                            # one split: its dispatch order lies far in front
    g = torch.Generator().manual_seed(5)
    q = {n: torch.randn(n, H, d, generator=g).bfloat16().cuda() for n in (1, 2, 6, 1900)}
    cu, scale, st = i32([0, 1900]), 1 / math.sqrt(d), api.new_status()

    def step(c, w, ws):
        x = q[len(c.ctx)]
        if c.int8:
            return api.paged_attention_decode_weights_q8(x, c.pool, c.d_table, c.d_ctx, scale, w, workspace=ws, status=st)
        return api.paged_attention_decode_weights(x, c.k, c.v, c.d_table, c.d_ctx, scale, w, workspace=ws, status=st)

    def chain(ws):
        cases = (long, one, wide, few, wide, one, long)
        w = [torch.zeros(len(c.ctx), Hkv, c.table.shape[1] * block, device="cuda") for c in cases]
        torch.cuda.synchronize()
        out = []
        for c, x in zip(cases, w):
            if c is long:
                api.paged_attention_weights(q[1900], cu, c.k, c.d_table, c.d_ctx, scale, x, 1900, workspace=ws, status=st)
            else:
                out.append(step(c, x, ws))
        check_status(st)
        return w + out

    want = chain(None)
    size = max([api.attention_decode_weights_workspace_size(len(c.ctx), H, Hkv, d, c.table.shape[1], block) for c in (one, wide, few)] +
               [api.attention_weights_workspace_size(1, 1900, 1900, H, Hkv, d, long.table.shape[1], block)])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(chain(ws), want))


@pytest.mark.parametrize("int8", [False, True])
def test_context_lengths_from_the_kernel_in_front(int8):
    """The lengths are written by the kernel in front of the call, as a server's `ctx += 1` does: the call sees them."""
    H, Hkv, d, block = 8, 2, 128, 64
    c = Paged([8300, 8200], Hkv, d, block, 6, int8)
    q = torch.randn(2, H, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    scale, st, ctx = 1 / math.sqrt(d), api.new_status(), i32([0, 0])
    zero = lambda: torch.zeros(2, Hkv, c.table.shape[1] * block, device="cuda")  # noqa: E731

    def call(ctx, w):
        if int8:
            return api.paged_attention_decode_weights_q8(q, c.pool, c.d_table, ctx, scale, w, status=st)
        return api.paged_attention_decode_weights(q, c.k, c.v, c.d_table, ctx, scale, w, status=st)

    lens = [(8300, 8200), (1, 8193), (8300, 40), (0, 0), (8256, 8200)]
    for n in lens * 4:
        a, b, new = zero(), zero(), i32(n)
        torch.cuda.synchronize()
        ctx.copy_(new)
        out = call(ctx, a)
        check_status(st)
        assert torch.equal(out, call(new, b)) and torch.equal(a, b)
        ctx.zero_()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("group", [1, 2, 7])
def test_a_query_of_nan_reaches_what_it_sees_alone(group, int8):
    """A NaN query gives NaN to its sequence's and KV head's positions; those without a valid block, behind the context and of
    other heads and sequences keep their values, as in the prompts' call."""
    Hkv, d, block = 2, 128, 32
    c = Paged([1300, 90], Hkv, d, block, 8, int8)
    q = torch.randn(2, Hkv * group, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    q[0, group + group // 2, 5] = math.nan                    # sequence 0, KV head 1
    table = c.table.copy()
    table[0, [1, 35]] = 10 ** 6, -1
    table[1, 2] = -1
    q, base, st = q.cuda(), torch.rand(2, Hkv, c.table.shape[1] * block + 3, generator=torch.Generator().manual_seed(2)).cuda(), api.new_status()
    w = base.clone()
    if int8:
        api.paged_attention_decode_weights_q8(q, c.pool, i32(table), c.d_ctx, 0.1, w, status=st)
    else:
        api.paged_attention_decode_weights(q, c.k, c.v, i32(table), c.d_ctx, 0.1, w, status=st)
    check_status(st, api.LL_DEV_BAD_BLOCK)
    hole = torch.zeros(1300, dtype=torch.bool)
    hole[32:64] = hole[35 * 32:36 * 32] = True
    assert torch.equal(w[0, 1].cpu()[:1300].isnan(), ~hole) and torch.equal(w[0, 1].cpu()[:1300][hole], base[0, 1].cpu()[:1300][hole])
    assert torch.equal(w[0, :, 1300:], base[0, :, 1300:]) and torch.equal(w[1, :, 64:], base[1, :, 64:])
    assert torch.equal(w[0, 0, 32:64], base[0, 0, 32:64]) and not w[0, 0].isnan().any() and not w[1].isnan().any()
    if not int8:                                               # the prompts' call on the same query: the same places
        again = base.clone()
        api.paged_attention_weights(q, i32([0, 1, 2]), c.k, i32(table), c.d_ctx, 0.1, again, 1, status=st)
        check_status(st, api.LL_DEV_BAD_BLOCK)
        assert torch.equal(again.isnan(), w.isnan())


@pytest.mark.parametrize("heads,kv", [(16, 2), (4, 4), (8, 1)])
def test_one_workspace_for_smaller_calls(heads, kv):
    """A workspace of the largest call's size serves calls of fewer sequences, rows and tokens: the same bits as with their own."""
    ctx, d, block, most = [3000, 2000, 700, 3000, 90, 1500], 64, 32, 300
    c = Paged(ctx, kv, d, block, 9)
    wide = c.table.shape[1]
    q = torch.randn(6 * most, heads, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    st, n = api.new_status(), api.attention_weights_workspace_size(6, 6 * most, most, heads, kv, d, wide, block)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for batch in (6, 2, 1):
        for new in (90, 70, 64, 17, 1):
            cu = i32([new * b for b in range(batch + 1)])
            args = (q[:batch * new], cu, c.k, c.d_table[:batch].contiguous(), c.d_ctx[:batch].contiguous(), 0.125)
            a, b = (torch.zeros(batch, kv, wide * block, device="cuda") for _ in range(2))
            api.paged_attention_weights(*args, a, new, workspace=ws, status=st)
            api.paged_attention_weights(*args, b, new, status=st)
            assert torch.equal(a, b) and api.attention_weights_workspace_size(batch, batch * new, new, heads, kv, d, wide, block) <= n
    with pytest.raises(api.LayerError):
        api.paged_attention_weights(*args, a, 1, workspace=ws[:16], status=st)
    check_status(st)


@pytest.mark.parametrize("kind", ["bf16", "int8", "noalloc"])
def test_plain_decode_calls_of_a_stream_share_a_workspace(kind):
    """The calls without weights, of batches whose dispatch orders lie in each other's partials, without a wait between."""
    H, Hkv, d, block, scale = 8, 2, 128, 64, 0.09
    cases = [Paged(ctx, Hkv, d, block, 20 + i, kind == "int8") for i, ctx in enumerate(([8200, 9000, 8700], [8300], [8500, 8193], [700], [9000] * 4))]
    if kind != "int8":
        cases = [c for c in cases if c.table.shape[1] * block > 7 * 1024]       # (with a dispatch order)
    g = torch.Generator().manual_seed(6)
    q, st = [torch.randn(len(c.ctx), H, d, generator=g).bfloat16().cuda() for c in cases], api.new_status()
    size = max(api.attention_workspace_size(len(c.ctx), H, d, c.table.shape[1], block) for c in cases)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def call(c, x, **kw):
        if kind == "int8":
            return api.paged_attention_decode_q8(x, c.pool, c.d_table, c.d_ctx, scale, status=st, **kw)
        if kind == "noalloc" and kw:
            return api.paged_attention_decode_noalloc(x, c.k, c.v, c.d_table, c.d_ctx, scale, status=st)
        return api.paged_attention_decode(x, c.k, c.v, c.d_table, c.d_ctx, scale, status=st, **kw)

    want = []
    for c, x in zip(cases, q):
        want.append(call(c, x))
        check_status(st)
    for _ in range(30):
        got = [call(c, x, workspace=ws) for c, x in zip(cases, q)]
        check_status(st)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
