"""The operators around the cache where they can go wrong: what a serving program does between steps,
batches of very different sequences, values that a row does not see.  Tolerances are those of
test_gpu_cache_ops.py."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from tests.helpers import f64
from tests.test_gpu_cache_ops import assert_attention, assert_pool, bf16, check, dev, make_cache, status, to_gpu
from transformer_decoder_layer_llama_gb300 import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api


def test_compaction_renames_a_prefill_that_is_staged():
    """Requests whose rows lie in pf_table when the pools are packed: the prefill writes their new blocks."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, nb, mb, slots, n = synth.DIMS_TINY, 24, 4, 3, 20
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = [api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=7).items()})]
    pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim)]
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=n)
    eng = StackEngine(api, [cfg], packed, pools, slots, mb, slots * n)
    stream = torch.cuda.Stream()
    for s in range(slots):
        sch.start_resident(s, n)
    eng.pf_table.copy_(torch.from_numpy(sch.table))
    eng.pf_table[1, 2] = 10 ** 6                       # an id of no pool stays
    eng.pf_ctx.fill_(n)
    eng.pf_x.copy_(synth.make_x(slots * n, d.hidden, seed=1))
    sch.retire(2)
    torch.cuda.synchronize()
    assert eng.compact(sch, stream) > 0
    got = eng.pf_table.cpu().numpy()
    assert got[1, 2] == 10 ** 6 and (got[2] == -1).all()
    got[1, 2] = -1
    assert (got[:2] == sch.table[:2]).all() and set(got[got >= 0]) == set(range(4))
    eng.prefill(2, n, stream)
    torch.cuda.synchronize()
    assert int(eng.status.item()) == 0
    assert (pools[0].k_scale[:4] > 0).all() and (pools[0].k_scale[4:] == 0).all()


@pytest.mark.parametrize("f8", [False, True])
def test_a_stack_whose_pools_have_different_numbers_of_blocks(f8):
    """Each layer's call takes its own pool; only copies of blocks in all of them need as many everywhere."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, mb, slots, n = synth.DIMS_TINY, 4, 2, 20
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = [api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=7 + l).items()}) for l in range(2)]
    ys = []
    for blocks in ((12, 12), (12, 20)):
        pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim) if f8 else
                 tuple(t.cuda() for t in synth.make_pool(nb, d, seed=3)) for nb in blocks]
        sch = Scheduler(slots, d.block_size, mb, BlockAllocator(12, seed=5), seed=6, prompt_len=n)
        eng = StackEngine(api, [cfg] * 2, packed, pools, slots, mb, slots * n)
        for s in range(slots):
            sch.start_resident(s, n)
        eng.pf_table.copy_(torch.from_numpy(sch.table))
        eng.pf_ctx.fill_(n)
        eng.pf_pos.copy_(dev(np.tile(np.arange(n), slots)))
        eng.pf_x.copy_(synth.make_x(slots * n, d.hidden, seed=1))
        stream = torch.cuda.current_stream()
        ys.append(eng.prefill(slots, n, stream).clone())
        ctx = sch.grow_for_decode()
        eng.table.copy_(torch.from_numpy(sch.table))
        eng.ctx.copy_(torch.from_numpy(ctx))
        eng.x.copy_(synth.make_x(slots, d.hidden, seed=2))
        ys.append(eng.decode(stream).clone())
        check(eng.status)
    assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[3])
    before = sch.table.copy(), [list(r.blocks) for r in sch.slots]
    with pytest.raises(ValueError, match="number of blocks"):
        eng.compact(sch, stream)
    assert (sch.table == before[0]).all() and [r.blocks for r in sch.slots] == before[1]


def test_calls_refuse_status_words_that_are_no_int32():
    """The kernels set bits of a 4-byte word: a byte tensor's address may be any."""
    rng = np.random.default_rng(3)
    ref, table = make_cache(rng, [20, 9], 2, 64, 16)
    pool, t, ctx, cu = to_gpu(ref), dev(table), dev([20, 9]), dev([0, 1, 2])
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    tab = api.rope_table(api.make_rope_config(64), 16)
    d = synth.DIMS_TINY
    cfg = api.make_config(d, max_position=64)
    packed = api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=1).items()})
    layer = api.PoolF8.empty(4, d.n_kv_heads, d.block_size, d.head_dim)
    x = synth.make_x(2, d.hidden, seed=2).cuda()
    for bad, error in ((torch.zeros(8, dtype=torch.uint8, device="cuda")[1:], TypeError),
                       (torch.zeros(1, dtype=torch.int64, device="cuda"), TypeError),
                       (torch.zeros(0, dtype=torch.int32, device="cuda"), ValueError),
                       (torch.zeros(1, dtype=torch.int32), ValueError)):
        for call in (lambda st: api.rope(q, None, dev([0, 1]), tab, status=st),
                     lambda st: api.append_to_cache_f8(q[:, :2].contiguous(), q[:, 2:].contiguous(), pool, t, ctx, status=st),
                     lambda st: api.paged_attention_decode_f8(q, pool, t, ctx, 0.1, status=st),
                     lambda st: api.paged_attention_prefill_f8(q, cu, pool, t, ctx, 0.1, max_new=1, status=st),
                     lambda st: api.layer_decode_step_f8(cfg, packed, x, layer, dev([[0], [1]]), dev([1, 1]), status=st),
                     lambda st: api.layer_prefill_f8(cfg, packed, x, layer, dev([[0], [1]]), dev([1, 1]), 1, status=st),
                     lambda st: api.copy_blocks(api.BlockSet(pool.tensors()), dev([[0, 1]]), status=st),
                     lambda st: api.compact_blocks(t, len(ref.k), status=st)):
            with pytest.raises(error, match="status"):
                call(bad)
    torch.cuda.synchronize()
    assert_pool(pool, ref)


@pytest.mark.parametrize("B,H,Hkv,d", [(1025, 4, 2, 64), (2100, 6, 3, 128), (1300, 18, 2, 64)])
def test_decode_of_thousands_of_sequences_some_of_which_many_ctas_share(B, H, Hkv, d):
    """Beyond 1024 sequences a CTA of the join takes a run of them: long contexts first, last and side by side in a run,
    which are cut over several CTAs each, among short and empty ones."""
    rng = np.random.default_rng(B)
    bs = 16
    ctx = rng.integers(0, 40, B)
    ctx[[3, 4, B // 2 + 2, B - 2]] = 0
    long = [0, B // 2, B // 2 + 1, B - 1]              # (runs of B / 1024 rounded up: 2 or 3)
    ctx[long] = [5000, 3001, 2500, 4097]
    ref, table = make_cache(rng, list(ctx), Hkv, d, bs)
    q = torch.from_numpy(rng.normal(size=(B, H, d))).bfloat16()
    want = C.attention_f8(f64(q), ref, table, ctx, np.arange(B + 1), d ** -0.5)
    st = status()
    ws = torch.full((api.attention_decode_f8_workspace_size(B, H, Hkv, d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    api.paged_attention_decode_f8(q.cuda(), to_gpu(ref), dev(table), dev(ctx), d ** -0.5, out=out, workspace=ws, status=st)
    check(st)
    for some in (long, np.flatnonzero(ctx == 0)):      # (named first, so that a failure says which)
        assert_attention(out[torch.as_tensor(some).cuda()], *(w[some] for w in want), d)
    assert_attention(out, *want, d)
    assert (out[torch.from_numpy(ctx == 0).cuda()] == 0).all()


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 8, 2, 64), (128, 16, 2, 128), (64, 3, 3, 128)])
def test_prefill_of_a_prompt_beside_single_tokens_behind_long_prefixes(bs, H, Hkv, d):
    """Items of one query tile and of two side by side, each with its own number of key tiles; with an empty sequence,
    a short chunk, and more than a warp's lanes of sequences."""
    rng = np.random.default_rng(bs + H)
    for before, new in (([0, 5000, 3000, 17, 4100, 0, 700], [600, 1, 1, 0, 1, 33, 5]),
                        ([0] * 3 + [900] * 32, [300, 129, 0] + [1] * 32)):
        ctx = [b + n for b, n in zip(before, new)]
        ref, table = make_cache(rng, ctx, Hkv, d, bs)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = torch.from_numpy(rng.normal(size=(int(cu[-1]) + 2, H, d))).bfloat16()
        want = C.attention_f8(f64(q[:cu[-1]]), ref, table, ctx, cu, d ** -0.5)
        st = status()
        out = torch.full(tuple(q.shape), 5.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((api.attention_prefill_f8_workspace_size(len(new), len(q), max(new), H, Hkv, d),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        for _ in range(2):
            api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(ref), dev(table), dev(ctx), d ** -0.5, max_new=max(new),
                                           out=out, workspace=ws, status=st)
            check(st)
            assert_attention(out[:cu[-1]], *want, d)
            assert (out[cu[-1]:] == 5).all()


@pytest.mark.parametrize("rot", [64, 24])
def test_rope_leaves_the_rows_of_bad_positions_in_views_of_merged_rows(rot):
    """Whole 16-byte columns (64) and not (24 of 64, half-split): rows of a wider buffer, out of place and in place."""
    T, H, Hkv, d = 6, 3, 2, 64
    w = (H + 2 * Hkv) * d + 8
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(T, w, generator=g).bfloat16().cuda()
    q, k = x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
    tab, pos, bad = api.rope_table(api.make_rope_config(rot), 16), dev([0, -1, 15, 16, 3, 2 ** 31 - 1]), [1, 3, 5]
    good, st = [0, 2, 4], status()
    want = api.rope(q[good].contiguous(), k[good].contiguous(), pos[good].contiguous(), tab, status=st)
    check(st)
    y = torch.full_like(x, 7.0)
    q1, k1 = y[:, :H * d].view(T, H, d), y[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
    before = x.clone()
    for outs in ((q1, k1), (q, k)):
        st = status()
        api.rope(q, k, pos, tab, q_out=outs[0], k_out=outs[1], status=st)
        check(st, api.LL_DEV_BAD_POSITION)
        assert torch.equal(outs[0][good], want[0]) and torch.equal(outs[1][good], want[1])
    assert (y[bad] == 7).all() and (y[:, (H + Hkv) * d:] == 7).all()
    assert torch.equal(x[bad], before[bad]) and torch.equal(x[:, (H + Hkv) * d:], before[:, (H + Hkv) * d:])


# ---------------------------------------------------------------- values that a row does not see, or hardly weighs

def assert_by_terms(got, q, pool, table, ctx, cu, scale, extra=0.0):
    """As assert_attention, with what the FP16 probabilities lose counted against the largest term that the row
    itself sums, not the largest |v| around: a probability times its V scale enters P V relative to a base, times 2^6.
    The base is at most 2^4 above the largest such product of the row (keys whose scales differ by less share one),
    so where it is subnormal it is off by 2^-25 of 2^-2 of that product, and a code (448) may carry a factor below 2."""
    d = q.shape[2]
    ref, weight, info = C.attention_f8(f64(q), pool, table, ctx, cu, scale)
    mag, n = info[..., :1], info[..., 1:2]
    rel = 2.0 ** -11 + 2.0 ** -23 * (d + 4) * mag + 2.0 ** -20 + (n / 16 + n / 128 + 8) * 2.0 ** -23 + extra
    bound = 2.0 ** -8 * np.abs(ref) + 1.01 * rel * weight + (n + 1) * 2.0 ** -26 * C.largest_term(f64(q), pool, table, ctx, cu, scale)
    got = f64(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def one_large_value(rng, before, new, Hkv, d, bs, at, size, u=None):
    """A cache of contexts before + new in which position at[b] of sequence b has a V `size` times as large (and, with u,
    every position of its block the key u: a block's scale counts for each of its keys)."""
    ctx = [b + n for b, n in zip(before, new)]
    pool, table = make_cache(rng, ctx, Hkv, d, bs)
    k, v = (bf16(rng.normal(size=(sum(ctx), Hkv, d))) for _ in range(2))
    starts = np.concatenate([[0], np.cumsum(ctx)]).astype(int)
    for b, p in enumerate(at):
        v[starts[b] + p] *= size
        if u is not None:
            lo = p // bs * bs
            k[starts[b] + lo:starts[b] + min(lo + bs, ctx[b])] = u
    pool.append(bf16(k), bf16(v), table, ctx, starts)
    return pool, table, ctx


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 4, 2, 64), (128, 4, 4, 128), (32, 16, 1, 128)])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 60])
def test_a_large_value_does_not_reach_rows_that_do_not_see_it(bs, H, Hkv, d, size):
    """The last new tokens have V far above the others': the rows before them answer as without it (chunks, a prompt of
    two query tiles, and a few tokens behind a long prefix, whose keys several CTAs share)."""
    for before, new in (([40, 0, 200], [100, 300, 2]), ([3000], [20])):
        rng = np.random.default_rng(bs + d)
        ctx = [b + n for b, n in zip(before, new)]
        pool, table, ctx = one_large_value(rng, before, new, Hkv, d, bs, [c - 1 for c in ctx], size)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = torch.from_numpy(rng.normal(size=(int(cu[-1]), H, d))).bfloat16()
        st = status()
        out = api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), d ** -0.5, max_new=max(new), status=st)
        check(st)
        assert_by_terms(out, q, pool, table, ctx, cu, d ** -0.5)


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 4, 2, 64), (128, 4, 4, 128), (32, 16, 1, 128)])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 60])
def test_a_large_value_that_hardly_weighs_leaves_the_others_their_bits(bs, H, Hkv, d, size):
    """A block far from every query (its probabilities about e^-150) has a V far above the others': decode and prefill."""
    rng = np.random.default_rng(bs + d)
    u = rng.choice([-1.0, 1.0], size=d)
    before, new = [3000, 0, 300], [3, 300, 40]
    pool, table, ctx = one_large_value(rng, before, new, Hkv, d, bs, [1234, 0, 177], size, u=-4 * u)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    q = torch.from_numpy(4.0 * u + rng.normal(size=(T, H, d))).bfloat16()
    scale = 150.0 / (16 * d)
    st = status()
    out = api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), scale, max_new=max(new), status=st)
    one = api.paged_attention_decode_f8(q[:3].cuda(), to_gpu(pool), dev(table), dev(ctx), scale, status=st)
    check(st)
    assert_by_terms(one, q[:3], pool, table, ctx, np.arange(4), scale)
    assert_by_terms(out, q, pool, table, ctx, cu, scale)


@pytest.mark.parametrize("power", [-123, -110, 80, 117])
def test_value_scales_far_from_one(power):
    """V scales of 2^power and a few powers above, in blocks side by side."""
    rng = np.random.default_rng(power + 200)
    before, new, H, Hkv, d, bs = [600, 0], [5, 130], 4, 2, 64, 16
    ctx = [605, 130]
    pool, table = make_cache(rng, ctx, Hkv, d, bs)
    live = pool.v_scale == pool.v_scale
    pool.v_scale[live] = 2.0 ** (power + rng.integers(0, 3, size=int(live.sum())))
    cu = np.array([0, 5, 135], np.int32)
    q = torch.from_numpy(rng.normal(size=(135, H, d))).bfloat16()
    st = status()
    out = api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), 0.125, max_new=130, status=st)
    one = api.paged_attention_decode_f8(q[:2].cuda(), to_gpu(pool), dev(table), dev(ctx), 0.125, status=st)
    check(st)
    assert_by_terms(one, q[:2], pool, table, ctx, np.arange(3), 0.125)
    assert_by_terms(out, q, pool, table, ctx, cu, 0.125)


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 4, 2, 64), (128, 4, 2, 128), (32, 24, 2, 128)])
def test_a_large_value_that_hardly_weighs_in_long_runs_of_keys(bs, H, Hkv, d):
    """The same for decode where a CTA has several key tiles of a sequence, before and behind the large block."""
    rng = np.random.default_rng(bs)
    u = rng.choice([-1.0, 1.0], size=d)
    B = 20
    pool, table, ctx = one_large_value(rng, [2300] * B, list(range(B)), Hkv, d, bs, list(rng.integers(0, 2300, size=B)), 2.0 ** 40, u=-4 * u)
    q = torch.from_numpy(4.0 * u + rng.normal(size=(B, H, d))).bfloat16()
    st = status()
    out = api.paged_attention_decode_f8(q.cuda(), to_gpu(pool), dev(table), dev(ctx), 150.0 / (16 * d), status=st)
    check(st)
    assert_by_terms(out, q, pool, table, ctx, np.arange(B + 1), 150.0 / (16 * d))


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 8, 8, 64), (128, 32, 4, 128), (64, 4, 4, 128), (16, 32, 2, 64)])
def test_decode_gives_the_same_bits_every_time(bs, H, Hkv, d):
    """Long runs of key tiles, whose codes follow each other into the same shared memory, 300 times."""
    rng = np.random.default_rng(bs + H)
    B = 24
    nb = B * (8192 // bs)
    g = torch.Generator("cuda").manual_seed(bs)
    codes = [torch.randint(0, 256, (nb, Hkv, bs, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0                      # no NaN
    pool = api.PoolF8(*(c.view(torch.float8_e4m3fn) for c in codes),
                      *(torch.exp2(torch.randint(-9, -5, (nb, Hkv), generator=g, device="cuda").float()) for _ in range(2)))
    table = torch.randperm(nb, generator=g, device="cuda").int().view(B, -1)
    ctx = dev(rng.integers(1, 8193, size=B))
    q, st = torch.randn(B, H, d, generator=g, device="cuda").bfloat16(), status()
    ws = torch.empty(api.attention_decode_f8_workspace_size(B, H, Hkv, d), dtype=torch.uint8, device="cuda")
    first = api.paged_attention_decode_f8(q, pool, table, ctx, d ** -0.5, workspace=ws, status=st)
    out, differ = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        out.fill_(5.0)
        api.paged_attention_decode_f8(q, pool, table, ctx, d ** -0.5, out=out, workspace=ws, status=st)
        differ += (out != first).any()
    check(st)
    assert int(differ.item()) == 0 and torch.isfinite(first).all()


@pytest.mark.parametrize("bs,H,Hkv,d", [(16, 8, 2, 64), (128, 16, 2, 128)])
def test_values_far_apart_give_the_same_bits_every_time(bs, H, Hkv, d):
    """Prefill over tiles whose V scales lie far apart, among tiles whose scales are near or alike, 100 times."""
    rng = np.random.default_rng(bs)
    before, new = [900, 0, 3000], [150, 300, 2]
    pool, table, ctx = one_large_value(rng, before, new, Hkv, d, bs, [200, 77, 1500], 2.0 ** 9)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q, st = torch.from_numpy(rng.normal(size=(int(cu[-1]), H, d))).bfloat16(), status()
    args = (q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), d ** -0.5)
    first = api.paged_attention_prefill_f8(*args, max_new=max(new), status=st)
    assert_by_terms(first, q, pool, table, ctx, cu, d ** -0.5)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        differ += (api.paged_attention_prefill_f8(*args, max_new=max(new), status=st) != first).any()
    check(st)
    assert int(differ.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_subnormal_queries_of_large_keys(d):
    """Queries below BF16's normal range whose scores with very large keys are of ordinary size."""
    rng = np.random.default_rng(d)
    before, new, H, Hkv, bs = [200, 0], [4, 90], 4, 2, 16
    ctx = [204, 90]
    pool, table = make_cache(rng, ctx, Hkv, d, bs)
    live = pool.k_scale == pool.k_scale
    pool.k_scale[live] = 2.0 ** 119
    cu = np.array([0, 4, 94], np.int32)
    q = torch.from_numpy(rng.integers(-100, 101, size=(94, H, d)) * 2.0 ** -133).bfloat16()
    scale = float(np.float32(16.0 / d))
    st = status()
    out = api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), scale, max_new=90, status=st)
    one = api.paged_attention_decode_f8(q[:2].cuda(), to_gpu(pool), dev(table), dev(ctx), scale, status=st)
    check(st)
    # the factor of such a row, a power of two times scale * log2 e, is subnormal itself: 20 bits
    mag = C.attention_f8(f64(q), pool, table, ctx, cu, scale)[2][..., :1]
    assert 3 < mag.max() < 300
    assert_by_terms(out, q, pool, table, ctx, cu, scale, extra=2.0 ** -20 * mag)
    assert_by_terms(one, q[:2], pool, table, ctx, np.arange(3), scale, extra=2.0 ** -20 * mag[:2])


@pytest.mark.parametrize("B,H,Hkv,d,bs", [(40, 4, 1, 64, 16), (33, 16, 1, 128, 64), (64, 8, 1, 128, 32)])
def test_few_tokens_of_more_sequences_than_a_warp_has_lanes_behind_prefixes_that_ctas_share(B, H, Hkv, d, bs):
    rng = np.random.default_rng(B)
    before, new = rng.integers(0, 1500, B), rng.integers(0, 4, B)
    new[[2, B - 1]] = 0
    ctx = before + new
    pool, table = make_cache(rng, list(ctx), Hkv, d, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.normal(size=(int(cu[-1]), H, d))).bfloat16()
    st = status()
    out = api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(pool), dev(table), dev(ctx), d ** -0.5, max_new=3, status=st)
    check(st)
    assert_attention(out, *C.attention_f8(f64(q), pool, table, ctx, cu, d ** -0.5), d)


def test_rows_before_the_first_sequence_and_tables_with_more_rows_than_sequences():
    """cu_new may start behind row 0, and the table may hold rows of sequences that are not in the call."""
    rng = np.random.default_rng(12)
    H, Hkv, d, bs = 4, 2, 64, 16
    before, new, ctx = [20, 7], [5, 30], [25, 37]
    cu = np.array([3, 8, 38], np.int32)
    T = 45
    ref, table = make_cache(rng, ctx, Hkv, d, bs)
    gpu = to_gpu(ref)
    wide = dev(np.concatenate([table, np.full((2, table.shape[1]), 10 ** 6, np.int32)]))
    k, v = (bf16(rng.normal(size=(T, Hkv, d))) for _ in range(2))
    ref.append(k, v, table, ctx, cu)
    st = status()
    api.append_to_cache_f8(*(torch.from_numpy(x).bfloat16().cuda() for x in (k, v)), gpu, wide, dev(ctx), cu_new=dev(cu), max_new=30, status=st)
    check(st)
    assert_pool(gpu, ref)
    q = torch.from_numpy(rng.normal(size=(T, H, d))).bfloat16()
    out = torch.full((T, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    api.paged_attention_prefill_f8(q.cuda(), dev(cu), gpu, wide, dev(ctx), 0.125, max_new=30, out=out, status=st)
    check(st)
    want = C.attention_f8(f64(q), ref, table, ctx, cu, 0.125)
    assert_attention(out[3:38], *(w[3:38] for w in want), d)
    assert (out[:3] == 5).all() and (out[38:] == 5).all()
    one = api.paged_attention_decode_f8(q[:2].cuda(), gpu, wide, dev(ctx), 0.125, status=st)
    check(st)
    assert_attention(one, *C.attention_f8(f64(q[:2]), ref, table, ctx, np.arange(3), 0.125), d)
