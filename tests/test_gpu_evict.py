"""Eviction of cached rows against its definition on a GPU: everything is exact (rows, weights, codes, lengths)."""
import numpy as np
import pytest
import torch

from oracle import weight_ops as W

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def check_status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


def bits(t):
    """The tensor's bytes as integers on the CPU (NaN compares by its bits)."""
    return t.cpu().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


class Cache:
    def __init__(self, ctx, kv_heads, dim, block, seed, kind="bf16", spare=1):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.block, self.H = list(ctx), block, kv_heads
        need = [-(-n // block) for n in ctx]
        wide, nb = max(max(need), 1) + spare, sum(need) + 2
        perm = torch.randperm(nb, generator=g).tolist()
        self.table = np.full((len(ctx), wide), -1, np.int64)
        for b, n in enumerate(need):
            self.table[b, :n] = [perm.pop() for _ in range(n)]
        shape = (nb, kv_heads, block, dim)
        if kind == "bf16":
            self.tensors = [torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16).view(torch.bfloat16).cuda()
                            for _ in range(2)]
            self.pool = tuple(self.tensors)
        else:
            codes = [torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda() for _ in range(2)]
            scales = [torch.rand(shape[:3], generator=g).cuda() for _ in range(2)]
            self.tensors = codes + scales
            self.pool = api.PoolQ8(*self.tensors)
        self.d_table, self.d_ctx = i32(self.table), i32(self.ctx)
        self.width = wide * block

    def rows(self, t, b, h):
        at = np.arange(self.ctx[b])
        return bits(t)[self.table[b, at // self.block], h, at % self.block]


def make_weights(kind, B, H, width, g):
    w = torch.exp(1.5 * torch.randn(B, H, width, generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0)
    elif kind == "odd":                                    # NaN, infinities, negative, subnormal, near the border
        pick = torch.randint(0, 8, w.shape, generator=g)
        vals = torch.tensor([float("nan"), float("inf"), -float("inf"), -1.0, 1e-42, -1e-42, 0.0, 2.0])
        w = vals[pick]
    return w


def run(c, weights, keep, sinks, recent, max_keep=None, separate=False, **kw):
    """Evicts, checks everything against the definition; returns (kept, new_lens)."""
    before = [bits(t).clone() for t in c.tensors]
    wd = weights.cuda()
    out = torch.full_like(wd, -7.0) if separate else None
    st = api.new_status()
    per = keep if isinstance(keep, int) else i32(keep)
    kept, lens = api.evict_rows(c.pool, c.d_table, c.d_ctx, wd, per, max_keep=max_keep, sinks=sinks, recent=recent, weights_out=out,
                                status=st, **kw)
    check_status(st)
    keeps = [keep] * len(c.ctx) if isinstance(keep, int) else keep
    assert lens.tolist() == [min(n, k) for n, k in zip(c.ctx, keeps)]
    want = [t.clone() for t in before]
    want_w = torch.full_like(weights, -7.0) if separate else weights.clone()
    for b, (n, k) in enumerate(zip(c.ctx, keeps)):
        for h in range(c.H):
            rows = W.keep_rows(weights[b, h, :n].numpy(), k, sinks, recent)
            got = kept[b, h].cpu().numpy()
            assert (got[:len(rows)] == rows).all() and (got[len(rows):] == -1).all()
            m = len(rows)
            want_w[b, h, :n] = 0
            want_w[b, h, :m] = weights[b, h, rows]
            at = np.arange(m)
            for t, old in zip(want, before):
                src = old[c.table[b, rows // c.block], h, rows % c.block]
                t[c.table[b, at // c.block], h, at % c.block] = src
    for t, w in zip(c.tensors, want):
        assert torch.equal(bits(t), w)
    assert torch.equal(bits(out if separate else wd), bits(want_w))
    if separate:
        assert torch.equal(bits(wd), bits(weights))
    return kept, lens


CASES = [  # contexts, kv_heads, dim, block, keep, sinks, recent
    ([1], 1, 64, 16, 1, 0, 0), ([2, 1, 5], 2, 64, 16, 1, 4, 0), ([40, 17, 0, 16], 2, 128, 16, 16, 2, 5), ([100, 33], 3, 64, 32, 20, 0, 20),
    ([300, 299, 257], 4, 128, 64, 128, 4, 31), ([1500], 2, 128, 128, 1499, 0, 0), ([1500], 2, 64, 256, 1, 0, 0), ([700] * 5, 8, 128, 128, 350, 700, 0),
    ([2049, 64], 1, 128, 256, 1025, 1, 1), ([3000], 1, 128, 64, 2999, 16, 1024)]


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("weights", ["spread", "ties", "zeros", "odd"])
@pytest.mark.parametrize("case", CASES)
def test_evict(case, weights, kind):
    ctx, H, dim, block, keep, sinks, recent = case
    c = Cache(ctx, H, dim, block, len(ctx) * 100 + keep, kind)
    w = make_weights(weights, len(ctx), H, c.width, torch.Generator().manual_seed(keep))
    run(c, w, keep, sinks, recent, separate=len(ctx) % 2 == 0)


@pytest.mark.parametrize("weights", ["spread", "ties", "odd"])
@pytest.mark.parametrize("ctx,keep", [([9000], 4500), ([20001], 1), ([20001], 20000), ([12345, 8192], 8191), ([33000], 3000)])
def test_long_rows_of_weights(ctx, keep, weights):
    """Few long rows of weights: the choice is spread over clusters of CTAs."""
    c = Cache(ctx, 2, 64, 256, keep, "bf16")
    run(c, make_weights(weights, len(ctx), 2, c.width, torch.Generator().manual_seed(keep)), keep, 4, min(keep, 100))


@pytest.mark.parametrize("weights", ["spread", "ties", "zeros", "some odd"])
@pytest.mark.parametrize("ctx,H,keep,spare,extra", [
    ([5000], 5, 1700, 1, 0), ([5000, 300], 10, 1234, 1, 1), ([4999] * 3, 20, 4000, 1, 2), ([5003] * 2, 50, 900, 1, 3), ([4100, 700], 100, 2000, 1, 0),
    ([300, 64], 2, 50, 900, 1), ([3000], 80, 1200, 3300, 0)])
def test_forms_of_the_choice(ctx, H, keep, spare, extra, weights):
    """Rows of weights in clusters of eight, four and two CTAs, in one with all or half of its threads, too long for shared
    memory by the table (and short in it), on 16 bytes or not; warps with and without odd values; part of the rows and outputs
    apart."""
    c = Cache(ctx, H, 16, 16, keep, spare=spare)
    g = torch.Generator().manual_seed(H)
    w = make_weights("spread" if weights == "some odd" else weights, len(ctx), H, c.width + extra, g)
    if weights == "some odd":                                 # few places, most warps have none
        odd = make_weights("odd", len(ctx), H, w.shape[2], g)
        w = torch.where(torch.rand(w.shape, generator=g) < 0.001, odd, w)
        w = torch.where(torch.rand(w.shape, generator=g) < 0.05, 0.0, w)
    run(c, w, keep, 4, min(keep, 100), separate=extra == 1)


def test_a_number_for_each_sequence():
    c = Cache([50, 60, 70, 16], 2, 64, 16, 1)
    w = make_weights("spread", 4, 2, c.width, torch.Generator().manual_seed(1))
    run(c, w, [10, 0, 100, 16], 2, 3, max_keep=70)


def test_twice_in_a_row():
    """Sums go on from the moved weights; a second eviction works on the result of the first."""
    c = Cache([200, 90], 2, 128, 32, 2)
    w = make_weights("spread", 2, 2, c.width, torch.Generator().manual_seed(2))
    wd, st = w.cuda(), api.new_status()
    k1, n1 = api.evict_rows(c.pool, c.d_table, c.d_ctx, wd, 64, sinks=2, recent=8, status=st)
    k2, n2 = api.evict_rows(c.pool, c.d_table, n1, wd, 32, sinks=2, recent=8, status=st)
    check_status(st)
    c2 = Cache([200, 90], 2, 128, 32, 2)
    for b, n in enumerate(c.ctx):
        for h in range(2):
            a = W.keep_rows(w[b, h, :n].numpy(), 64, 2, 8)
            r = W.keep_rows(w[b, h, a].numpy(), 32, 2, 8)
            assert (k2[b, h].cpu().numpy() == r).all()
            for t, old in zip(c.tensors, c2.tensors):
                at = np.arange(32)
                assert torch.equal(bits(t)[c.table[b, at // 32], h, at % 32], c2.rows(old, b, h)[a[r]])
    assert n2.tolist() == [32, 32]


def test_what_does_not_fit_is_flagged_and_left():
    ctx = [40, 50, 60, 30, 45]
    c = Cache(ctx, 2, 64, 16, 4)
    good = Cache(ctx, 2, 64, 16, 4)
    w = make_weights("spread", 5, 2, c.width, torch.Generator().manual_seed(4))
    table = c.table.copy()
    table[2, 3] = 10 ** 6                                  # a bad block of a sequence that loses rows
    table[3, 1] = -1                                       # of one that does not
    for d_ctx, keep, flagged, bad in ((ctx, [20, 20, 20, 30, 20], api.LL_DEV_BAD_BLOCK, [2]),
                                      ([40, -1, 10 ** 6, 30, 45], [20] * 3 + [30, 20], api.LL_DEV_BAD_POSITION, [1, 2]),
                                      (ctx, [20, -1, 20, 30, 41], api.LL_DEV_BAD_POSITION | api.LL_DEV_BAD_BLOCK, [1, 2, 4])):
        st, wd = api.new_status(), w.cuda()
        before = [bits(t).clone() for t in c.tensors]
        kept, lens = api.evict_rows(c.pool, i32(table), i32(d_ctx), wd, i32(keep), max_keep=40, sinks=1, recent=4, status=st)
        check_status(st, flagged)
        for b in range(5):
            if b in bad:
                assert (kept[b] == -1).all() and int(lens[b]) == d_ctx[b] and torch.equal(wd[b].cpu(), w[b])
                for t, old in zip(c.tensors, before):
                    blocks = c.table[b][c.table[b] >= 0]
                    assert torch.equal(bits(t)[blocks], old[blocks])
            else:
                assert int(lens[b]) == min(ctx[b], keep[b])
                for h in range(2):
                    r = W.keep_rows(w[b, h, :ctx[b]].numpy(), keep[b], 1, 4)
                    assert (kept[b, h, :len(r)].cpu().numpy() == r).all() and (kept[b, h, len(r):] == -1).all()
        for t, g in zip(c.tensors, good.tensors):          # the next turn starts from the same cache
            t.copy_(g)
    narrow, st = w[..., :48].contiguous().cuda(), api.new_status()
    _, lens = api.evict_rows(good.pool, good.d_table, good.d_ctx, narrow, 20, status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    assert lens.tolist() == [20, 50, 60, 20, 20]


def test_streams_and_graphs():
    w = make_weights("spread", 2, 2, 320, torch.Generator().manual_seed(4)).cuda()

    def fresh():
        c = Cache([300, 290], 2, 128, 64, 9, spare=0)
        assert c.width == 320
        return c
    a = fresh()
    wa = w.clone()
    kept, lens = api.evict_rows(a.pool, a.d_table, a.d_ctx, wa, 100, sinks=3, recent=10)
    torch.cuda.synchronize()
    b, wb, side = fresh(), w.clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kb, nb = api.evict_rows(b.pool, b.d_table, b.d_ctx, wb, 100, sinks=3, recent=10, stream=side)
    side.synchronize()
    assert torch.equal(kb, kept) and torch.equal(nb, lens) and torch.equal(wa, wb)
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a.tensors, b.tensors))
    c, wc, kc, nc, st = fresh(), w.clone(), torch.zeros_like(kept), torch.zeros_like(lens), api.new_status()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.evict_rows(c.pool, c.d_table, c.d_ctx, wc, 100, sinks=3, recent=10, kept=kc, new_lens=nc, status=st)
    graph.replay()
    check_status(st)
    assert torch.equal(kc, kept) and torch.equal(wa, wc) and all(torch.equal(bits(x), bits(y)) for x, y in zip(a.tensors, c.tensors))


def test_rows_of_weights_beyond_shared_memory():
    """A table so wide that the choice reads the weights from memory again; many heads and sequences, so no clusters."""
    c = Cache([60000, 70, 1000, 16], 48, 64, 256, 8, spare=150)
    w = make_weights("spread", 4, 48, c.width, torch.Generator().manual_seed(3))
    run(c, w, 64, 4, 10)


@pytest.mark.parametrize("separate", [False, True])
def test_one_very_long_row_of_weights(separate):
    c = Cache([420000], 1, 64, 256, 5, spare=0)
    w = make_weights("ties", 1, 1, c.width, torch.Generator().manual_seed(3))
    g = W.keep_rows
    before = [bits(t).clone() for t in c.tensors]
    wd, st = w.cuda(), api.new_status()
    out = torch.zeros_like(wd) if separate else None
    kept, lens = api.evict_rows(c.pool, c.d_table, c.d_ctx, wd, 5000, sinks=7, recent=11, weights_out=out, status=st)
    check_status(st)
    rows = g(w[0, 0, :420000].numpy(), 5000, 7, 11)
    assert (kept[0, 0].cpu().numpy() == rows).all() and lens.tolist() == [5000]
    at = np.arange(5000)
    for t, old in zip(c.tensors, before):
        assert torch.equal(bits(t)[c.table[0, at // 256], 0, at % 256], old[c.table[0, rows // 256], 0, rows % 256])
    got = (out if separate else wd)[0, 0].cpu()
    assert torch.equal(got[:5000], w[0, 0, rows]) and (got[5000:420000] == 0).all()


@pytest.mark.parametrize("weights", ["spread", "ties", "zeros", "odd"])
@pytest.mark.parametrize("ctx,block,keep", [([1024, 1023, 900, 31], 256, 33), ([2048, 2047, 1500, 1025], 256, 1024), ([1008, 640, 32, 64], 16, 640),
                                            ([2000, 1999, 2], 16, 1998)])
def test_rows_at_the_size_of_a_warp(ctx, block, keep, weights):
    """A table as wide as a warp's registers, and one block less."""
    c = Cache(ctx, 3, 64, block, keep, spare=0)
    run(c, make_weights(weights, len(ctx), 3, c.width, torch.Generator().manual_seed(keep)), keep, 3, 17)
