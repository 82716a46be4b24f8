"""The operators around the cache against their float64 definitions on a GPU.

Tolerances.  Rounding errors relative to the value: BF16 2^-8, FP16 2^-11, float32 2^-24, counted once
for each rounding on the way:
* rope: c and s come from a float32 table (2^-24 each), each product and the sum round once in float32:
  4 * 2^-24 * magnitude * (|a| + |b|) covers them, then one rounding to the output's type.
* attention: a probability enters P V as FP16 (2^-11 relative; below 2^-14 of its base FP16 is
  subnormal, an absolute 2^-25, and the base is at most 2^8 above the row's largest and 2^6 shifted, so
  2^-30 of the largest |v| per key at most, in fact far less in sum), its exponent carries the score's
  float32 error (d products and sums on the tensor core, which may cut instead of round: 2^-23 each of
  sum |q k| scale, and 2^-22 of the score for the factor), exp2 itself 2^-21, and the sums of n weights
  and products in float32 cut n / 16 + n / 128 times 2^-23.  Weighted by sum p |v|.
  Then one rounding to BF16.
* codes, scales, tables of ids and copied bytes are exact.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import llama_layer as O
from tests.helpers import assert_close, bits, f64
from transformer_decoder_layer_llama_gb300 import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api

F8 = torch.float8_e4m3fn
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def status():
    return api.new_status()


def check(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


# ---------------------------------------------------------------- rope

def rope_bound(x, freq, magnitude, layout, dtype, ref):
    half = len(freq)
    pair = np.zeros_like(x)
    i0 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i1 = i0 + half if layout == "half" else i0 + 1
    s = np.abs(x[..., i0]) + np.abs(x[..., i1])
    pair[..., i0] = pair[..., i1] = s * magnitude
    return 4 * 2.0 ** -24 * pair + (UNIT[dtype] * np.abs(ref) if dtype != torch.float32 else 0) + 2.0 ** -140


ROPE_CASES = [  # tokens, heads, kv_heads, dim, rot, scaling
    (1, 1, 1, 64, 64, "plain"), (7, 4, 2, 128, 128, "plain"), (33, 5, 1, 128, 64, "linear"), (3, 8, 8, 64, 10, "ntk"),
    (64, 32, 32, 128, 128, "banded"), (5, 3, 2, 96, 34, "yarn"), (129, 64, 8, 128, 128, "yarn"), (2, 2, 0, 24, 8, "plain"),
    (1025, 64, 8, 128, 32, "banded"), (9, 1, 3, 256, 256, "plain"), (4, 2, 1, 80, 2, "plain")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("case", ROPE_CASES)
def test_rope_matches_the_definition(case, layout, backward, dtype):
    T, H, Hk, d, rot, scaling = case
    g = torch.Generator().manual_seed(T * 1000 + rot)
    qkv = torch.randn(T, (H + 2 * Hk) * d + 8, generator=g).to(dtype).cuda()
    q, k = qkv[:, :H * d].view(T, H, d), qkv[:, H * d:(H + Hk) * d].view(T, Hk, d)
    before = qkv.clone()
    maxpos = 140000
    pos = torch.randint(0, maxpos, (T,), generator=g, dtype=torch.int32)
    kw = dict(factor=8.0, original_max_position=4096) if scaling != "plain" else {}
    table = api.rope_table(api.make_rope_config(rot, scaling=scaling, **kw), maxpos)
    st = status()
    q2, k2 = api.rope(q, k if Hk else None, pos.cuda(), table, layout=layout, backward=backward, status=st)
    check(st)
    f, m = C.inv_freq(rot, scaling=scaling, factor=kw.get("factor", 1.0), original=4096)
    for x, got in ((q, q2), (k, k2)) if Hk else ((q, q2),):
        xn = f64(x)
        ref = C.rope(xn, pos.numpy(), f, m, layout, backward)
        assert got.is_contiguous() and got.dtype == dtype
        assert (np.abs(f64(got) - ref) <= rope_bound(xn, f, m, layout, dtype, ref)).all()
        assert (f64(got)[..., rot:] == xn[..., rot:]).all()
    assert torch.equal(qkv, before)                                      # the inputs are left alone
    # in place, through the views: the same bits, and nothing else of the merged rows changes
    api.rope(q, k if Hk else None, pos.cuda(), table, layout=layout, backward=backward, q_out=q,
             k_out=k if Hk else None, status=st)
    check(st)
    assert torch.equal(q, q2) and (not Hk or torch.equal(k, k2))
    assert torch.equal(qkv[:, (H + Hk) * d:], before[:, (H + Hk) * d:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_is_the_transpose_and_the_difference_quotient(layout):
    T, H, d, rot = 6, 3, 64, 48
    g = torch.Generator().manual_seed(4)
    x, y, h = (torch.randn(T, H, d, generator=g).cuda() for _ in range(3))
    pos = dev([0, 1, 5, 99, 1000, 4095])
    table = api.rope_table(api.make_rope_config(rot, scaling="yarn", factor=4.0, original_max_position=1024), 4096)
    fwd = lambda t: f64(api.rope(t, None, pos, table, layout=layout)[0])  # noqa: E731
    grad = f64(api.rope(y, None, pos, table, layout=layout, backward=True)[0])
    # <R(x), y> is linear in x, so its difference along h is <grad, h> but for rounding
    diff = ((fwd(x + h) - fwd(x)) * f64(y)).sum()
    bound = 2.0 ** -20 * (np.abs(f64(x)) + np.abs(f64(h))).sum() * np.abs(f64(y)).max()
    assert abs(diff - (grad * f64(h)).sum()) <= bound
    assert abs((fwd(x) * f64(y)).sum() - (f64(x) * grad).sum()) <= bound


def test_rope_bad_positions_are_flagged_and_left():
    q = torch.randn(5, 2, 64).bfloat16().cuda()
    table = api.rope_table(api.make_rope_config(64), 16)
    out = torch.full_like(q, 7.0)
    for stride_view in (False, True):
        st = status()
        api.rope(q, None, dev([0, -1, 15, 16, 3]), table, q_out=out, status=st)
        check(st, api.LL_DEV_BAD_POSITION)
        assert (out[[1, 3]] == 7).all() and torch.equal(out[0], q[0]) and not (out[[2, 4]] == 7).all()
    with pytest.raises(api.LayerError):                                  # shifted onto its own input
        flat = torch.zeros(5 * 128 + 64, dtype=torch.bfloat16, device="cuda")
        api.rope(flat[:640].view(5, 2, 64), None, dev([0] * 5), table, q_out=flat[64:].view(5, 2, 64))
    with pytest.raises(ValueError):
        api.rope(q, None, dev([0] * 5), table, q_out=out[:, :1])
    with pytest.raises(ValueError):
        api.rope(q.transpose(0, 1), None, dev([0] * 2), table)


def test_rope_special_values_and_empty():
    table = api.rope_table(api.make_rope_config(4), 4)
    q = torch.tensor([[[float("inf"), 1.0, 2.0, float("nan"), 3.0, -0.0, 5.0, 6.0]]]).cuda()
    out, _ = api.rope(q, None, dev([0]), table)                          # position 0: c = 1, s = 0
    assert torch.isinf(out[0, 0, 0]) and torch.isnan(out[0, 0, 3]) and torch.isnan(out[0, 0, 2])
    assert torch.equal(out[0, 0, 4:], q[0, 0, 4:])
    e, _ = api.rope(q[:0], None, dev([]), table)
    assert e.shape == (0, 1, 8)


def test_pack_rope_rescales_the_layer():
    """The plain configuration packs the table that ll_pack_weights made; under interpolation by 2 position 2 p
    turns as p did."""
    d = synth.DIMS_TINY
    W = {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=1).items()}
    cfg = api.make_config(d, max_position=64)
    base = api.pack_weights(cfg, W)
    same = base.clone()
    api.pack_rope(cfg, api.make_rope_config(d.head_dim, theta=d.rope_theta), same)
    assert torch.equal(base, same)
    api.pack_rope(cfg, api.make_rope_config(d.head_dim, theta=d.rope_theta, scaling="linear", factor=2.0), same)
    x = synth.make_x(8, d.hidden, seed=2).cuda()
    kp, vp = (t.cuda() for t in synth.make_pool(8, d, seed=3))
    table = dev([[0, 1, 2, 3]])
    q = []
    for packed, step in ((base, 1), (same, 2)):
        ws = api.new_workspace(cfg, 8, 4)
        api.layer_prefill(cfg, packed, x, dev(np.arange(8) * step), 1, 8, kp, vp, table, workspace=ws)
        torch.cuda.synchronize()
        q.append(api.checkpoints(cfg, ws, 8, 4, 8)["q"].clone())
    assert torch.equal(q[0], q[1])


# ---------------------------------------------------------------- the e4m3 cache

def make_cache(rng, ctx, Hkv, d, bs, extra=2, poison=True, spread=0.5):
    """(oracle pool, table) of cached contexts: values of differing size, blocks in random order, -1 behind a
    sequence's blocks, NaN codes in every row that holds no token."""
    need = [-(-c // bs) for c in ctx]
    nb = sum(need) + extra
    table = np.full((len(ctx), max(need + [1]) + 1), -1, np.int32)
    perm = rng.permutation(nb).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    fill = 0x7F if poison else 0
    pool = C.PoolF8(*(np.full((nb, Hkv, bs, d), fill, np.uint8) for _ in range(2)), *(np.full((nb, Hkv), np.nan) for _ in range(2)))
    size = np.exp(spread * rng.normal(size=(1, Hkv, 1)))
    T = int(sum(ctx))
    k, v = (bf16(rng.normal(size=(T, Hkv, d)) * size) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(ctx)]).astype(int)
    pool.append(k, v, table, ctx, cu)
    return pool, table


def bf16(x):
    return torch.as_tensor(x).bfloat16().double().numpy()


def to_gpu(pool):
    return api.PoolF8(*(torch.from_numpy(c.copy()).cuda().view(F8) for c in (pool.k, pool.v)),
                      *(torch.from_numpy(s.astype(np.float32)).cuda() for s in (pool.k_scale, pool.v_scale)))


def copy_pool(p):
    return C.PoolF8(p.k.copy(), p.v.copy(), p.k_scale.copy(), p.v_scale.copy())


def assert_pool(gpu, ref):
    for name in ("k", "v"):
        got = getattr(gpu, name).view(torch.uint8).cpu().numpy()
        want = getattr(ref, name)
        # -0 and +0 are the same value
        bad = (got != want) & ~(((got | want) & 0x7F) == 0)
        assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
        s = getattr(gpu, name + "_scale").cpu().numpy().astype(np.float64)
        assert np.array_equal(s, getattr(ref, name + "_scale"), equal_nan=True)


APPEND_CASES = [  # block, kv_heads, dim, contexts before, new tokens
    (16, 1, 64, [0], [1]), (16, 2, 128, [0, 5, 15, 16, 17], [1, 1, 1, 1, 1]), (256, 3, 128, [255, 256, 100, 0], [1, 1, 1, 1]),
    (64, 32, 128, [63, 1, 64], [1, 1, 1]), (16, 2, 64, [0, 3, 40], [100, 0, 7]), (32, 1, 128, [31, 32], [1, 33]),
    (64, 2, 128, [10, 0, 130], [300, 64, 63]), (128, 4, 64, [127, 5], [2, 250]), (128, 2, 128, [1, 128], [127, 128]),
    (256, 2, 128, [3, 255], [600, 2]), (256, 1, 64, [100], [400])]


@pytest.mark.parametrize("case", APPEND_CASES)
def test_append_matches_the_definition(case):
    bs, Hkv, d, before, new = case
    rng = np.random.default_rng(bs + Hkv + sum(new))
    ctx = [b + n for b, n in zip(before, new)]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    ref, table = make_cache(rng, ctx, Hkv, d, bs)      # every block of the contexts is in the table
    old, _ = make_cache(rng, before, Hkv, d, bs, extra=len(ref.k) - sum(-(-b // bs) for b in before))
    ref = copy_pool(old)
    # lay the earlier rows where the table has them, with their scales
    ref.k[:], ref.v[:], ref.k_scale[:], ref.v_scale[:] = 0x7F, 0x7F, np.nan, np.nan
    kb, vb = (bf16(0.1 * rng.normal(size=(sum(before), Hkv, d))) for _ in range(2))
    ref.append(kb, vb, table, before, np.concatenate([[0], np.cumsum(before)]).astype(int))
    gpu = to_gpu(ref)
    # magnitudes that make some blocks grow and others not; zeros, huge and tiny values, both infinities, NaN
    k, v = (rng.normal(size=(T, Hkv, d)) * np.exp(2 * rng.normal(size=(T, Hkv, 1))) for _ in range(2))
    if T > 4:
        k[0], v[1, 0], k[2, 0, 0], v[2, -1, 1], k[3, 0, 2] = 0.0, 1e-37, np.inf, -np.inf, np.nan
        v[3, 0, 3] = 3.3e38
    k, v = bf16(k), bf16(v)
    wide = torch.zeros(T, 2 * Hkv * d + 8, dtype=torch.bfloat16, device="cuda")
    kt, vt = wide[:, :Hkv * d].view(T, Hkv, d), wide[:, Hkv * d:2 * Hkv * d].view(T, Hkv, d)
    kt.copy_(torch.from_numpy(k))
    vt.copy_(torch.from_numpy(v))
    ref.append(k, v, table, ctx, cu)
    st = status()
    one = all(n == 1 for n in new)
    for cu_arg in ([None] if one else []) + [dev(cu)]:   # one token each: both ways to say it
        pool = api.PoolF8(gpu.k.clone(), gpu.v.clone(), gpu.k_scale.clone(), gpu.v_scale.clone())
        api.append_to_cache_f8(kt, vt, pool, dev(table), dev(ctx), cu_new=cu_arg, max_new=max(new), status=st)
        check(st)
        assert_pool(pool, ref)


def test_append_zeros_then_values_and_a_fresh_start():
    """A block of zeros has scale 0; a call that writes offset 0 forgets what the block held."""
    ref = C.PoolF8(*(np.full((2, 1, 16, 64), 0x55, np.uint8) for _ in range(2)), *(np.full((2, 1), 2.0 ** 60) for _ in range(2)))
    pool, table = to_gpu(ref), [[1, 0]]
    st = status()
    rng = np.random.default_rng(0)
    for ctx, x in ((1, 0.0), (2, 0.0), (3, 1.0), (4, 1000.0), (5, 1e-3)):
        k = bf16(rng.normal(size=(1, 1, 64)) * x)
        ref.append(k, -k, table, [ctx], [0, 1])
        t = torch.from_numpy(k).bfloat16().cuda()
        api.append_to_cache_f8(t, -t, pool, dev(table), dev([ctx]), status=st)
        check(st)
        assert_pool(pool, ref)


def test_append_flags_bad_counts_and_blocks():
    rng = np.random.default_rng(5)
    ref, table = make_cache(rng, [20, 20, 20], 2, 64, 16)
    T = 9
    k = bf16(rng.normal(size=(T, 2, 64)))
    t = torch.from_numpy(k).bfloat16().cuda()
    bad_table = table.copy()
    bad_table[1, 1], bad_table[2, 1] = len(ref.k), -1
    for cu, ctx, mx, tab, want in (([0, 3, 3, 3], [2, 20, 20], 3, table, api.LL_DEV_BAD_POSITION),       # n > context
                                   ([0, 0, 4, 4], [20, 20, 20], 3, table, api.LL_DEV_BAD_POSITION),      # n > max_new
                                   ([0, 0, 0, 12], [20, 20, 20], 20, table, api.LL_DEV_BAD_POSITION),    # beyond tokens
                                   ([5, 5, 5, 2], [20, 20, 20], 9, table, api.LL_DEV_BAD_POSITION),      # n < 0
                                   ([-1, 1, 1, 1], [20, 20, 20], 9, table, api.LL_DEV_BAD_POSITION),
                                   ([0, 3, 3, 3], [1000, 20, 20], 3, table, api.LL_DEV_BAD_POSITION),    # beyond the table
                                   ([0, 0, 3, 6], [20, 20, 20], 3, bad_table, api.LL_DEV_BAD_BLOCK)):
        gpu = to_gpu(ref)
        st = status()
        api.append_to_cache_f8(t, t, gpu, dev(tab), dev(ctx), cu_new=dev(cu), max_new=mx, status=st)
        check(st, want)
        assert_pool(gpu, ref)                                            # nothing was written
    gpu = to_gpu(ref)
    st = status()
    api.append_to_cache_f8(t[:3], t[:3], gpu, dev(bad_table), dev([0, 20, 20]), status=st)
    check(st, api.LL_DEV_BAD_BLOCK | api.LL_DEV_BAD_POSITION)
    assert_pool(gpu, ref)


# ---------------------------------------------------------------- attention over it

def attention_bound(ref, weight, info, d):
    mag, n, vmax = info[..., :1], info[..., 1:2], info[..., 2:]
    score = 2.0 ** -23 * (d + 4) * mag
    rel = 2.0 ** -11 + score + 2.0 ** -20 + (n / 16 + n / 128 + 8) * 2.0 ** -23
    return 2.0 ** -8 * np.abs(ref) + 1.01 * rel * weight + (n + 1) * 2.0 ** -31 * vmax


def assert_attention(got, ref, weight, info, d):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= attention_bound(ref, weight, info, d))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


DECODE_CASES = [  # block, heads, kv_heads, dim, contexts
    (16, 4, 2, 64, [1]), (16, 4, 2, 64, [0, 1, 15, 16, 17, 63, 64, 65, 200]), (128, 32, 32, 128, [700, 3, 129]),
    (128, 64, 8, 128, [1, 2000, 1024]), (64, 16, 1, 128, [777]), (256, 10, 2, 128, [256, 257, 600]),
    (32, 7, 1, 64, [0, 0, 33]), (16, 12, 4, 128, [5, 100]), (16, 9, 1, 128, [130, 64]), (32, 16, 1, 64, [500, 31]),
    (128, 2, 2, 128, [5000]), (16, 1, 1, 64, [3000, 0, 7])]


@pytest.mark.parametrize("case", DECODE_CASES)
def test_decode_matches_the_definition(case):
    bs, H, Hkv, d, ctx = case
    rng = np.random.default_rng(bs + H + sum(ctx))
    ref_pool, table = make_cache(rng, ctx, Hkv, d, bs)
    pool = to_gpu(ref_pool)
    q = torch.from_numpy(rng.normal(size=(len(ctx), H, d)) * np.exp(rng.normal(size=(len(ctx), H, 1)))).bfloat16()
    scale = d ** -0.5
    want = C.attention_f8(f64(q), ref_pool, table, ctx, np.arange(len(ctx) + 1), scale)
    st = status()
    ws = torch.full((api.attention_decode_f8_workspace_size(len(ctx), H, Hkv, d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((len(ctx), H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    first = None
    for _ in range(3):                                                   # the same workspace, whatever it holds
        api.paged_attention_decode_f8(q.cuda(), pool, dev(table), dev(ctx), scale, out=out, workspace=ws, status=st)
        check(st)
        assert_attention(out, *want, d)
        first = out.clone() if first is None else first
        assert torch.equal(out, first)                                   # the same bits every time


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scales_of_every_size(d):
    """Blocks whose scales lie far apart, scale 0, scales that are no powers of two, large and tiny queries."""
    rng = np.random.default_rng(d)
    ctx, bs, H, Hkv = [160, 96], 16, 6, 2
    ref_pool, table = make_cache(rng, ctx, Hkv, d, bs)
    live = ref_pool.k_scale == ref_pool.k_scale
    sizes = np.array([1.0, 0.37, 2.0 ** -12, 0.0, 1.9, 2.0 ** -20])
    for s in (ref_pool.k_scale, ref_pool.v_scale):
        s[live] = (rng.choice(sizes, size=s.shape) * 2.0 ** -6)[live]
    ref_pool.k_scale[live] = np.float32(ref_pool.k_scale[live]).astype(np.float64)
    ref_pool.v_scale[live] = np.float32(ref_pool.v_scale[live]).astype(np.float64)
    for size in (1.0, 1e-20, 30.0):
        q = torch.from_numpy(rng.normal(size=(2, H, d)) * size).bfloat16()
        ref, weight, info = C.attention_f8(f64(q), ref_pool, table, ctx, [0, 1, 2], 0.1)
        st = status()
        out = api.paged_attention_decode_f8(q.cuda(), to_gpu(ref_pool), dev(table), dev(ctx), 0.1, status=st)
        pre = api.paged_attention_prefill_f8(q.cuda(), dev([0, 1, 2]), to_gpu(ref_pool), dev(table), dev(ctx), 0.1,
                                             max_new=1, status=st)
        check(st)
        # a scale that is no power of two costs one more FP16 rounding, of the block's V (prefill) or of P (decode)
        extra = 2.0 ** -11 * weight
        for got in (out, pre):
            assert (np.abs(f64(got) - ref) <= attention_bound(ref, weight, info, d) + extra).all()


def test_decode_of_a_tiny_cache_keeps_its_size():
    """V of 1e-30 next to nothing larger comes back at its own size."""
    rng = np.random.default_rng(7)
    pool, table = make_cache(rng, [40], 1, 64, 16)
    live = pool.v_scale == pool.v_scale
    pool.v_scale[live] *= 2.0 ** -100
    q = torch.from_numpy(rng.normal(size=(1, 2, 64))).bfloat16()
    want = C.attention_f8(f64(q), pool, table, [40], [0, 1], 0.1)
    for got in (api.paged_attention_decode_f8(q.cuda(), to_gpu(pool), dev(table), dev([40]), 0.1),
                api.paged_attention_prefill_f8(q.cuda(), dev([0, 1]), to_gpu(pool), dev(table), dev([40]), 0.1, max_new=1)):
        assert_attention(got, *want, 64)


def test_attention_bad_blocks_and_contexts():
    rng = np.random.default_rng(11)
    pool, table = make_cache(rng, [100, 50, 16], 2, 64, 16)
    gpu = to_gpu(pool)
    table[0, 2], table[0, 4], table[2, 0] = -1, len(pool.k) + 5, -7      # holes, and a sequence without any block
    q = torch.from_numpy(rng.normal(size=(3, 4, 64))).bfloat16()
    want = C.attention_f8(f64(q), pool, table, [100, 50, 16], [0, 1, 2, 3], 0.1)
    for call in (lambda st, ctx: api.paged_attention_decode_f8(q.cuda(), gpu, dev(table), dev(ctx), 0.1, status=st),
                 lambda st, ctx: api.paged_attention_prefill_f8(q.cuda(), dev([0, 1, 2, 3]), gpu, dev(table), dev(ctx), 0.1,
                                                                max_new=1, out=torch.zeros_like(q, device="cuda"), status=st)):
        st = status()
        got = call(st, [100, 50, 16])
        check(st, api.LL_DEV_BAD_BLOCK)
        assert_attention(got, *want, 64)
        assert (got[2] == 0).all()
        st = status()
        got = call(st, [-5, 50, 10 ** 6])
        torch.cuda.synchronize()
        assert int(st.item()) & api.LL_DEV_BAD_POSITION
        assert_attention(got[1:2], *(w[1:2] for w in want), 64)
        assert (got[0] == 0).all()


PREFILL_CASES = [  # block, heads, kv_heads, dim, contexts before, new tokens
    (16, 4, 2, 64, [0], [1]), (16, 4, 2, 64, [0, 10, 0], [64, 5, 17]), (128, 4, 4, 128, [0], [300]),
    (128, 16, 2, 128, [100, 0, 1], [129, 1, 40]), (64, 16, 1, 128, [500], [33]), (256, 5, 1, 128, [0, 255], [128, 2]),
    (32, 3, 1, 64, [0, 0, 7], [0, 130, 0]), (16, 7, 7, 128, [2000], [3]), (16, 14, 2, 64, [129], [255]),
    (128, 9, 1, 128, [30], [60]), (32, 8, 8, 64, [0, 96], [127, 128]), (16, 1, 1, 128, [1000], [200]),
    (256, 16, 1, 64, [3000], [5]), (128, 8, 2, 128, [1500, 0], [1, 700]), (64, 2, 2, 64, [2500], [257])]


@pytest.mark.parametrize("case", PREFILL_CASES)
def test_prefill_matches_the_definition(case):
    bs, H, Hkv, d, before, new = case
    ctx = [b + n for b, n in zip(before, new)]
    rng = np.random.default_rng(bs + H + sum(ctx))
    ref_pool, table = make_cache(rng, ctx, Hkv, d, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    q = torch.from_numpy(rng.normal(size=(T + 3, H, d)) * np.exp(rng.normal(size=(T + 3, H, 1)))).bfloat16()
    scale = d ** -0.5
    want = C.attention_f8(f64(q[:T]), ref_pool, table, ctx, cu, scale)
    st = status()
    out = torch.full((T + 3, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    pool = to_gpu(ref_pool)
    first = None
    for mx in (max(new), max(new) + 200):                                # max_new is an upper bound
        api.paged_attention_prefill_f8(q.cuda(), dev(cu), pool, dev(table), dev(ctx), scale, max_new=mx, out=out, status=st)
        check(st)
        assert_attention(out[:T], *want, d)
        assert (out[T:] == 5).all()                                      # rows behind the last sequence
        first = out.clone() if first is None else first
    again = api.paged_attention_prefill_f8(q.cuda(), dev(cu), pool, dev(table), dev(ctx), scale, max_new=max(new), status=st)
    assert torch.equal(again[:T], first[:T])


def test_prefill_flags_bad_counts():
    rng = np.random.default_rng(5)
    pool, table = make_cache(rng, [20, 20], 2, 64, 16)
    gpu = to_gpu(pool)
    q = torch.from_numpy(rng.normal(size=(9, 4, 64))).bfloat16().cuda()
    for cu, ctx, mx in (([0, 3, 3], [2, 20], 3), ([0, 0, 4], [20, 20], 3), ([0, 0, 12], [20, 20], 20), ([5, 5, 2], [20, 20], 9),
                        ([-1, 1, 1], [20, 20], 9), ([0, 3, 3], [1000, 20], 3)):
        st = status()
        out = torch.full_like(q, 5.0)
        api.paged_attention_prefill_f8(q, dev(cu), gpu, dev(table), dev(ctx), 0.1, max_new=mx, out=out, status=st)
        check(st, api.LL_DEV_BAD_POSITION)
        assert (out == 5).all()


def test_attention_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes: blocks at both ends of it."""
    nb, Hkv, bs, d = 5000, 32, 256, 128                                  # 5.2 GB of codes per tensor
    pool = api.PoolF8.empty(nb, Hkv, bs, d)
    table = np.array([[nb - 1, 0, nb - 2]], np.int32)
    rng = np.random.default_rng(1)
    ctx, H = [600], 32
    k, v = (bf16(rng.normal(size=(600, Hkv, d))) for _ in range(2))
    st = status()
    kt, vt = (torch.from_numpy(x).bfloat16().cuda() for x in (k, v))
    api.append_to_cache_f8(kt, vt, pool, dev(table), dev(ctx), cu_new=dev([0, 600]), max_new=600, status=st)
    small = C.PoolF8(*(np.zeros((3, Hkv, bs, d), np.uint8) for _ in range(2)), *(np.zeros((3, Hkv)) for _ in range(2)))
    small.append(k, v, [[0, 1, 2]], ctx, [0, 600])
    q = torch.from_numpy(rng.normal(size=(1, H, d))).bfloat16()
    want = C.attention_f8(f64(q), small, [[0, 1, 2]], ctx, [0, 1], d ** -0.5)
    assert_attention(api.paged_attention_decode_f8(q.cuda(), pool, dev(table), dev(ctx), d ** -0.5, status=st), *want, d)
    assert_attention(api.paged_attention_prefill_f8(q.cuda(), dev([0, 1]), pool, dev(table), dev(ctx), d ** -0.5, max_new=1,
                                                    status=st), *want, d)
    blocks = api.BlockSet(pool.tensors())
    api.copy_blocks(blocks, dev([[nb - 1, 17], [0, nb - 3]]), status=st)
    check(st)
    assert torch.equal(pool.k.view(torch.uint8)[17], pool.k.view(torch.uint8)[nb - 1])
    assert torch.equal(pool.v.view(torch.uint8)[nb - 3], pool.v.view(torch.uint8)[0])
    assert torch.equal(pool.k_scale[17], pool.k_scale[nb - 1])


# ---------------------------------------------------------------- blocks

@pytest.mark.parametrize("n_tensors,inner,dtype", [(1, (4,), torch.uint8), (3, (2, 16, 64), torch.bfloat16), (2, (5,), torch.float32),
                                                   (130, (33,), torch.int32), (4, (8, 128, 128), torch.uint8)])
@pytest.mark.parametrize("n", [1, 7])
def test_copy_blocks(n_tensors, inner, dtype, n):
    nb = 24
    g = torch.Generator().manual_seed(n)
    ts = [torch.randint(0, 100, (nb, *inner), generator=g).to(dtype).cuda() for _ in range(n_tensors)]
    want = [t.clone() for t in ts]
    perm = torch.randperm(nb, generator=g)[:2 * n].view(n, 2)
    for t in want:
        t[perm[:, 1].cuda()] = t[perm[:, 0].cuda()]
    pad = torch.full((3, 2), -1)
    pairs = torch.cat((pad, perm, pad)).int().cuda()
    blocks = api.BlockSet(ts)
    st = status()
    api.copy_blocks(blocks, pairs, n_pairs=dev([0]), status=st)
    api.copy_blocks(blocks, pairs[:0], status=st)
    api.copy_blocks(blocks, pairs[3:], n_pairs=dev([n]), status=st)
    check(st)
    assert all(torch.equal(a, b) for a, b in zip(ts, want))
    api.copy_blocks(blocks, pairs, status=st)                            # the padding is skipped
    check(st)
    assert all(torch.equal(a, b) for a, b in zip(ts, want))
    api.copy_blocks(blocks, dev([[0, nb], [-1, 3], [-5, 0], [nb + 7, 2], [4, 4]]), status=st)
    check(st, api.LL_DEV_BAD_BLOCK)
    assert all(torch.equal(a, b) for a, b in zip(ts, want))


def test_copy_blocks_of_tensors_off_16_bytes():
    raw = torch.randint(0, 255, (4 + 12 * 20 + 16 * 20,), dtype=torch.uint8).cuda()
    a, b = raw[4:4 + 240].view(20, 12), raw[244:244 + 320].view(20, 16)  # 4-byte aligned only
    want_a, want_b = a.clone(), b.clone()
    want_a[7], want_b[7] = a[3], b[3]
    st = status()
    api.copy_blocks(api.BlockSet([a, b]), dev([[3, 7]]), status=st)
    check(st)
    assert torch.equal(a, want_a) and torch.equal(b, want_b)


@pytest.mark.parametrize("nb,rows,wide,used", [(1, 1, 1, 1), (2, 1, 1, 1), (33, 4, 8, 20), (33, 4, 9, 33), (100, 7, 20, 0),
                                               (1000, 16, 64, 700), (100003, 64, 200, 9000), (524288, 1, 5000, 5000)])
def test_compact_blocks(nb, rows, wide, used):
    rng = np.random.default_rng(nb)
    ids = rng.permutation(nb)[:used].astype(np.int32)
    table = np.full(rows * wide, -1, np.int32)
    table[rng.permutation(rows * wide)[:used]] = ids
    if used > 4:
        table[rng.integers(0, rows * wide, size=used // 4)] = rng.choice(ids, used // 4)    # shared blocks
    table = table.reshape(rows, wide)
    new, moves, U, block_map = C.compact(table, nb)
    st = status()
    t = dev(table)
    got, pairs, counts, bm = api.compact_blocks(t, nb, status=st)
    check(st)
    want = np.full((nb // 2, 2), -1, np.int32)
    want[:len(moves)] = np.array(moves, np.int32).reshape(-1, 2)
    assert counts.tolist() == [U, len(moves)] and (pairs.cpu().numpy() == want).all()
    assert (got.cpu().numpy() == new).all() and (bm.cpu().numpy() == block_map).all()
    assert (t.cpu().numpy() == table).all()
    api.compact_blocks(t, nb, new_table=t, status=st)                    # in place
    check(st)
    assert (t.cpu().numpy() == new).all()


def test_compact_blocks_bad_ids_and_no_rows():
    st = status()
    got, pairs, counts, _ = api.compact_blocks(dev([[9, -3, 5, 8]]), 8, status=st)
    check(st, api.LL_DEV_BAD_BLOCK)
    assert got.tolist() == [[9, -3, 0, 8]] and counts.tolist() == [1, 1] and pairs[0].tolist() == [5, 0]
    st = status()
    _, pairs, counts, bm = api.compact_blocks(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 6, status=st)
    check(st)
    assert counts.tolist() == [0, 0] and (pairs == -1).all() and (bm == -1).all()


# ---------------------------------------------------------------- together

def test_a_served_batch_from_prompt_to_compaction():
    """Prompts through rope, the cache write and the prefill attention; a fork; decode steps replayed as one CUDA
    graph on a stream of its own; compaction; the same answers from the packed pool."""
    H, Hkv, d, bs, nb = 8, 2, 64, 16, 40
    rng = np.random.default_rng(21)
    freq = dict(scaling="banded", factor=4.0, original_max_position=64)
    tab = api.rope_table(api.make_rope_config(d, **freq), 256)
    f, mag = C.inv_freq(d, scaling="banded", factor=4.0, original=64)
    pool = api.PoolF8.empty(nb, Hkv, bs, d)
    blocks = api.BlockSet(pool.tensors())
    ref = C.PoolF8(*(np.zeros((nb, Hkv, bs, d), np.uint8) for _ in range(2)), *(np.zeros((nb, Hkv)) for _ in range(2)))
    table = np.full((3, 8), -1, np.int32)
    table[0, :4], table[1, :3] = [30, 7, 39, 2], [11, 25, 38]
    new, ctx = [50, 33], [50, 33]
    cu = np.array([0, 50, 83], np.int32)
    st = status()

    def inputs(T):
        return torch.from_numpy(rng.normal(size=(T, (H + 2 * Hkv) * d))).bfloat16().cuda()

    def split(x):
        T = x.shape[0]
        return x[:, :H * d].view(T, H, d), x[:, H * d:(H + Hkv) * d].view(T, Hkv, d), x[:, (H + Hkv) * d:].view(T, Hkv, d)

    def oracle(x, pos, table, ctx, cu):
        q, k, v = (f64(t) for t in split(x))
        q, k = bf16(C.rope(q, pos, f, mag, "half")), bf16(C.rope(k, pos, f, mag, "half"))
        return q, k, v

    # the prompts; the oracle's cache takes the device's K, since a BF16 rounding may fall either way
    x = inputs(83)
    pos = np.concatenate([np.arange(50), np.arange(33)]).astype(np.int32)
    q, k, v = split(x)
    q1, k1 = api.rope(q, k, dev(pos), tab, status=st)
    qo, ko, vo = oracle(x, pos, table, ctx, cu)
    assert (np.abs(f64(k1) - ko) <= 2.0 ** -7 * np.abs(ko) + 1e-6).all()
    api.append_to_cache_f8(k1, v, pool, dev(table[:2]), dev(ctx), cu_new=dev(cu), max_new=50, status=st)
    ref.append(f64(k1), vo, table, ctx, cu)
    out = api.paged_attention_prefill_f8(q1, dev(cu), pool, dev(table[:2]), dev(ctx), d ** -0.5, max_new=50, status=st)
    check(st)
    assert_pool(pool, ref)
    assert_attention(out, *C.attention_f8(f64(q1), ref, table, ctx, cu, d ** -0.5), d)
    # sequence 2 forks from sequence 0: full blocks shared, the last one copied
    table[2, :4] = [30, 7, 39, 17]
    api.copy_blocks(blocks, dev([[2, 17]]), status=st)
    for t in (ref.k, ref.v, ref.k_scale, ref.v_scale):
        t[17] = t[2]
    table[0, 4], table[1, 3], table[2, 4] = 5, 19, 33
    ctx = [50, 33, 50]
    # decode steps: one graph, replayed with new inputs
    xs, ctx_d, pos_d, table_d = inputs(3), dev(ctx), dev(ctx), dev(table)
    ws = torch.empty(api.attention_decode_f8_workspace_size(3, H, Hkv, d), dtype=torch.uint8, device="cuda")
    y = torch.empty(3, H, d, dtype=torch.bfloat16, device="cuda")
    qd, kd = torch.empty(3, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(3, Hkv, d, dtype=torch.bfloat16, device="cuda")

    def step():
        q, k, v = split(xs)
        api.rope(q, k, pos_d, tab, q_out=qd, k_out=kd, status=st)
        api.append_to_cache_f8(kd, v, pool, table_d, ctx_d, status=st)
        api.paged_attention_decode_f8(qd, pool, table_d, ctx_d, d ** -0.5, out=y, workspace=ws, status=st)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    for i in range(20):
        xn = inputs(3)
        ctx = [c + 1 for c in ctx]
        xs.copy_(xn)
        ctx_d.copy_(dev(ctx))
        pos_d.copy_(dev([c - 1 for c in ctx]))
        g.replay()
        check(st)
        _, _, vo = oracle(xn, np.array(ctx) - 1, table, ctx, None)
        ref.append(f64(kd), vo, table, ctx, [0, 1, 2, 3])
        assert_attention(y, *C.attention_f8(f64(qd), ref, table, ctx, [0, 1, 2, 3], d ** -0.5), d)
    assert_pool(pool, ref)
    # sequence 1 ends: its blocks are free; the rest is packed
    y0 = y.clone()
    table[1] = -1
    table_d.copy_(dev(table))
    new_table, pairs, counts, _ = api.compact_blocks(table_d, nb, status=st)
    api.copy_blocks(blocks, pairs, n_pairs=counts[1:], status=st)
    want, moves, U, _ = C.compact(table, nb)
    check(st)
    assert counts.tolist() == [U, len(moves)] and (new_table.cpu().numpy() == want).all() and want.max() == U - 1
    ctx_d[1] = 0
    z = api.paged_attention_decode_f8(qd, pool, new_table, ctx_d, d ** -0.5, status=st)
    check(st)
    for b, w in ((0, y0[0]), (2, y0[2])):
        assert (np.abs(f64(z[b]) - f64(w)) <= 2.0 ** -7 * np.abs(f64(w)) + 1e-3).all()
    assert (z[1] == 0).all()


# ---------------------------------------------------------------- the layer and the stack over it

DIMS_128 = synth.LayerDims(512, 8, 2, 128, 1024, 32)


@pytest.mark.parametrize("d", [synth.DIMS_TINY, DIMS_128])
def test_layer_over_an_e4m3_pool(d):
    """A prompt, a chunk behind it and decode steps: codes and scales exact for the layer's own K and V (a BF16
    pool fed the same tokens holds them), the attention within its bound of the definition on the layer's q and
    codes, the output within the layer's bound of the definition from there."""
    B, nb, mb = 3, 40, 8
    W = synth.make_weights(d, 0.02, seed=11)
    Wn = {k: f64(v) for k, v in W.items()}
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = api.pack_weights(cfg, {k: v.cuda() for k, v in W.items()})
    table = np.random.default_rng(5).permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32)
    pool = api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim)
    kp, vp = (t.cuda() for t in synth.make_pool(nb, d, seed=3))
    ref = C.PoolF8(*(np.zeros(tuple(pool.k.shape), np.uint8) for _ in range(2)),
                   *(np.zeros(tuple(pool.k_scale.shape)) for _ in range(2)))
    st, done = status(), 0
    for n in (37, 20, 1, 1):
        ctx = [done + n] * B
        T = B * n
        x = synth.make_x(T, d.hidden, seed=100 + done).cuda()
        pos = np.tile(np.arange(done, done + n), B)
        api.layer_prefill(cfg, packed, x, dev(pos), B, n, kp, vp, dev(table), status=st)
        ws = api.new_workspace_f8(cfg, T, mb)
        if n == 1:
            y = api.layer_decode_step_f8(cfg, packed, x, pool, dev(table), dev(ctx), workspace=ws, status=st)
        else:
            y = api.layer_prefill_f8(cfg, packed, x, pool, dev(table), dev(ctx), n, workspace=ws, status=st)
        check(st)
        cp = api.checkpoints(cfg, ws, T, mb, T)
        cu = np.arange(B + 1) * n
        at = table[np.repeat(np.arange(B), n), pos // d.block_size]
        k, v = (f64(t)[at, :, pos % d.block_size] for t in (kp, vp))
        ref.append(k, v, table, ctx, cu)
        assert_pool(pool, ref)
        q = f64(cp["q"]).reshape(T, d.n_heads, d.head_dim)
        assert_attention(cp["o"].view(T, d.n_heads, d.head_dim), *C.attention_f8(q, ref, table, ctx, cu, d.head_dim ** -0.5),
                         d.head_dim)
        h = f64(x) + f64(cp["o"]) @ Wn["w_o"].T
        hh = O.bf16_round(O.rmsnorm(h, Wn["g_ffn"], d.rms_eps))
        a = O.bf16_round(O.silu(hh @ Wn["w_gate"].T) * (hh @ Wn["w_up"].T))
        assert_close(f64(y), h + a @ Wn["w_down"].T, f"after {done + n} tokens")
        done += n


def test_layer_f8_flags_contexts_shorter_than_the_new_tokens():
    d, B = synth.DIMS_TINY, 2
    cfg = api.make_config(d, max_position=64)
    packed = api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=1).items()})
    pool = api.PoolF8.empty(8, d.n_kv_heads, d.block_size, d.head_dim)
    before = pool.k.view(torch.uint8).clone()
    x = synth.make_x(B * 4, d.hidden, seed=2).cuda()
    st = status()
    api.layer_prefill_f8(cfg, packed, x, pool, dev([[0, 1], [2, 3]]), dev([3, 4]), 4, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & api.LL_DEV_BAD_POSITION
    assert torch.equal(pool.k.view(torch.uint8)[:2], before[:2]) and (pool.k_scale[2] > 0).all()
    # a context beyond the RoPE table is not written either
    st = status()
    api.layer_decode_step_f8(cfg, packed, x[:2], pool, dev([[4, 5, 6, 7, 0], [4, 5, 6, 7, 1]]), dev([65, 0]), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & api.LL_DEV_BAD_POSITION and (pool.k_scale[:2] == 0).all()
    with pytest.raises(ValueError):
        api.layer_prefill_f8(cfg, packed, x, api.PoolF8.empty(8, d.n_kv_heads, 32, d.head_dim), dev([[0, 1], [2, 3]]), dev([4, 4]), 4)


@pytest.mark.parametrize("f8", [False, True])
def test_stack_forks_and_compacts(f8):
    """A two-layer stack: a forked request answers as its parent does, and packing the pools changes no answer."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, L, nb, mb, slots, prompt = synth.DIMS_TINY, 2, 40, 8, 3, 24
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = [api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=100 + l).items()}) for l in range(L)]
    pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim) if f8 else
             tuple(t.cuda() for t in synth.make_pool(nb, d, seed=l)) for l in range(L)]
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
    eng = StackEngine(api, [cfg] * L, packed, pools, slots, mb, slots * prompt)
    stream = torch.cuda.Stream()
    torch.cuda.set_stream(stream)
    try:
        for s in (0, 1):
            sch.start_resident(s, prompt)
        eng.pf_table[:2].copy_(torch.from_numpy(sch.table[:2]))
        eng.pf_ctx[:2].copy_(dev([prompt, prompt]))
        eng.pf_pos[:2 * prompt].copy_(dev(np.tile(np.arange(prompt), 2)))
        eng.pf_x[:2 * prompt].copy_(synth.make_x(2 * prompt, d.hidden, seed=1))
        eng.prefill(2, prompt, stream)
        eng.copy_blocks(sch.fork(0, 2), stream)

        def step(seed):
            ctx = sch.grow_for_decode()
            x = synth.make_x(slots, d.hidden, seed=seed)
            x[2] = x[0]
            eng.table.copy_(torch.from_numpy(sch.table))
            eng.ctx.copy_(torch.from_numpy(ctx))
            eng.x.copy_(x)
            return eng.decode(stream).clone()

        for i in range(12):                   # over a block's end
            y = step(10 + i)
            assert torch.equal(y[0], y[2]) and not torch.equal(y[0], y[1])
        sch.retire(1)
        sch.start_resident(1, 5)              # leaves holes behind
        sch.retire(1)
        moved = eng.compact(sch, stream)
        sch.start_resident(1, 1)
        live = [b for s in (0, 2) for b in sch.slots[s].blocks]
        assert moved > 0 and max(live) < len(set(live)) and sorted(set(live)) == list(range(len(set(live))))
        eng.table.copy_(torch.from_numpy(sch.table))
        eng.ctx[1] = 1
        again = eng.decode(stream)            # the same step once more, from the packed pool
        assert torch.equal(again[0], y[0]) and torch.equal(again[2], y[2])
        torch.cuda.synchronize()
        assert int(eng.status.item()) == 0
    finally:
        torch.cuda.set_stream(torch.cuda.default_stream())


@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_zero_keys_and_a_zero_scale(d):
    """Blocks whose keys are all zeros (scale 0) that end inside a tile, or whose last keys the causal mask hides;
    scale 0: every visible key counts alike."""
    rng = np.random.default_rng(3 * d)
    ctx, bs, H, Hkv = [5, 150, 40], 16, 6, 2
    ref_pool, table = make_cache(rng, ctx, Hkv, d, bs)
    for blk in (table[0][0], table[1][8], table[1][9], table[2][1]):     # the last blocks of each
        ref_pool.k[blk], ref_pool.k_scale[blk] = 0, 0.0
    pool = to_gpu(ref_pool)
    new = [5, 60, 1]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.normal(size=(int(cu[-1]), H, d))).bfloat16()
    st = status()
    for scale in (d ** -0.5, 0.0):
        want = C.attention_f8(f64(q), ref_pool, table, ctx, cu, scale)
        assert_attention(api.paged_attention_prefill_f8(q.cuda(), dev(cu), pool, dev(table), dev(ctx), scale, max_new=60,
                                                        status=st), *want, d)
        want = C.attention_f8(f64(q[:3]), ref_pool, table, ctx, np.arange(4), scale)
        assert_attention(api.paged_attention_decode_f8(q[:3].cuda(), pool, dev(table), dev(ctx), scale, status=st), *want, d)
    check(st)


def test_rope_into_columns_of_one_buffer():
    """q, k, v and the rotated q and k all in one buffer: rows interleave, columns do not."""
    T, H, Hkv, d = 37, 4, 2, 64
    rng = np.random.default_rng(4)
    w = (2 * H + 3 * Hkv) * d
    x = torch.from_numpy(rng.normal(size=(T, w))).bfloat16().cuda()
    col = lambda at, n: x[:, at * d:(at + n) * d].view(T, n, d)  # noqa: E731
    q, k, v, q1, k1 = col(0, H), col(H, Hkv), col(H + Hkv, Hkv), col(H + 2 * Hkv, H), col(2 * H + 2 * Hkv, Hkv)
    tab = api.rope_table(api.make_rope_config(d), 64)
    pos = dev(np.arange(T))
    want = api.rope(q.contiguous(), k.contiguous(), pos, tab)
    kept = [t.clone() for t in (q, k, v)]
    api.rope(q, k, pos, tab, q_out=q1, k_out=k1)
    assert torch.equal(q1, want[0]) and torch.equal(k1, want[1])
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), kept))
    api.rope(q, k, pos, tab, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept[2])


# ---------------------------------------------------------------- many sequences, other streams, graphs

def test_many_sequences():
    """More sequences than the lanes of a warp (40) and than CTAs of a wave (700): prompts, then single tokens."""
    rng = np.random.default_rng(9)
    bs, H, Hkv, d = 16, 8, 2, 64
    before, new = rng.integers(0, 60, 40), rng.integers(0, 70, 40)
    new[[0, 7, 39]], before[[3, 7]] = 0, 0
    ctx = before + new
    ref, table = make_cache(rng, list(ctx), Hkv, d, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.normal(size=(int(cu[-1]) + 2, H, d))).bfloat16()
    st = status()
    out = torch.full(tuple(q.shape), 5.0, dtype=torch.bfloat16, device="cuda")
    api.paged_attention_prefill_f8(q.cuda(), dev(cu), to_gpu(ref), dev(table), dev(ctx), d ** -0.5, max_new=int(new.max()),
                                   out=out, status=st)
    check(st)
    assert_attention(out[:cu[-1]], *C.attention_f8(f64(q[:cu[-1]]), ref, table, ctx, cu, d ** -0.5), d)
    assert (out[cu[-1]:] == 5).all()
    B = 700
    ctx = rng.integers(0, 50, B)
    ctx[[1, 699]] = 0
    ref, table = make_cache(rng, list(ctx), Hkv, d, bs, extra=B + 2)
    free = iter(np.setdiff1d(np.arange(len(ref.k)), table[table >= 0]))
    table = np.concatenate([table, np.full((B, 1), -1, np.int32)], 1)
    for b in range(B):                        # a block for the token that starts one
        if ctx[b] % bs == 0:
            table[b, ctx[b] // bs] = next(free)
    gpu, ctx = to_gpu(ref), ctx + 1
    k, v = (bf16(rng.normal(size=(B, Hkv, d))) for _ in range(2))
    ref.append(k, v, table, ctx, np.arange(B + 1))
    api.append_to_cache_f8(*(torch.from_numpy(t).bfloat16().cuda() for t in (k, v)), gpu, dev(table), dev(ctx), status=st)
    q = torch.from_numpy(rng.normal(size=(B, H, d))).bfloat16()
    out = api.paged_attention_decode_f8(q.cuda(), gpu, dev(table), dev(ctx), d ** -0.5, status=st)
    check(st)
    assert_pool(gpu, ref)
    assert_attention(out, *C.attention_f8(f64(q), ref, table, ctx, np.arange(B + 1), d ** -0.5), d)


def small_batch(seed, d=64, bs=16, H=4, Hkv=2):
    """Inputs of one run of the cache operators, and the run: name -> result.  Three sequences, 40 new tokens."""
    rng = np.random.default_rng(seed)
    ctx, new = [50, 20, 33], [20, 20, 0]
    ref, table = make_cache(rng, ctx, Hkv, d, bs, poison=False)
    cu = np.array([0, 20, 40, 40], np.int32)
    x = dict(q=torch.from_numpy(rng.normal(size=(40, H, d))).bfloat16().cuda(), pool=to_gpu(ref),
             k=torch.from_numpy(rng.normal(size=(40, Hkv, d))).bfloat16().cuda(), table=dev(table), ctx=dev(ctx), cu=dev(cu),
             pos=dev(np.concatenate([np.arange(30, 50), np.arange(20)])), rope=api.rope_table(api.make_rope_config(d), 64),
             pairs=dev([[int(table[0, 0]), len(ref.k) - 1]]), spare=api.PoolF8.empty(len(ref.k), Hkv, bs, d))
    return x


def run_small(x, **kw):
    """Every operator once, everything that may be left out left out."""
    q, k = api.rope(x["q"], x["k"], x["pos"], x["rope"], **kw)
    yield api.append_to_cache_f8(k, x["k"], x["pool"], x["table"], x["ctx"], cu_new=x["cu"], max_new=20, **kw)
    yield q
    yield api.paged_attention_prefill_f8(q, x["cu"], x["pool"], x["table"], x["ctx"], 0.125, max_new=20, **kw)
    yield api.paged_attention_decode_f8(q[:3], x["pool"], x["table"], x["ctx"], 0.125, **kw)
    yield api.copy_blocks(api.BlockSet(x["pool"].tensors()), x["pairs"], **kw)
    new_table, _, counts, block_map = api.compact_blocks(x["table"], len(x["pool"].k), **kw)
    yield from (new_table, counts, block_map)
    yield from (t.view(torch.uint8) for t in (x["pool"].k, x["pool"].v))


def test_calls_on_a_stream_that_is_not_the_current_one():
    """What a call makes itself is made on the current stream, which is busy here; the call's stream waits for it."""
    want = [t.clone() for t in run_small(small_batch(1))]
    x = small_batch(1)
    bad = dev([[99, 0]])
    blocks = api.BlockSet(x["spare"].tensors())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)                                       # about 50 ms
    got = list(run_small(x, stream=stream))
    st = api.copy_blocks(blocks, bad, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(st.item()) == api.LL_DEV_BAD_BLOCK                        # not cleared behind the kernel that set it
    torch.cuda.synchronize()


def test_captured_runs_replayed_side_by_side():
    """Two captured runs of all operators, each with its own memory, replayed at once on two streams and with new
    inputs: the results of the plain calls."""
    sets, graphs, outs, streams = [small_batch(1), small_batch(2)], [], [], [torch.cuda.Stream() for _ in range(2)]
    first = [{n: t.clone() for n, t in zip("kv", (x["pool"].k.view(torch.uint8), x["pool"].v.view(torch.uint8)))} for x in sets]
    scales = [[x["pool"].k_scale.clone(), x["pool"].v_scale.clone()] for x in sets]
    for x, s in zip(sets, streams):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(list(run_small(x)))
        graphs.append(g)

    def reset():
        for x, f, sc in zip(sets, first, scales):
            x["pool"].k.view(torch.uint8).copy_(f["k"])
            x["pool"].v.view(torch.uint8).copy_(f["v"])
            x["pool"].k_scale.copy_(sc[0])
            x["pool"].v_scale.copy_(sc[1])

    for turn in range(3):
        if turn:
            for x in sets:
                x["q"].mul_(-0.5)
                x["k"].mul_(1.5)
        reset()
        want = [[t.clone() for t in run_small(x)] for x in sets]
        reset()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_stack_compaction_waits_for_the_step_that_reads_the_table():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, nb, mb, slots = synth.DIMS_TINY, 24, 4, 2
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = [api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=7).items()})]
    pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim)]
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=9)
    eng = StackEngine(api, [cfg], packed, pools, slots, mb, slots * 9)
    stream = torch.cuda.Stream()
    for s in range(slots):
        sch.start_resident(s, 9)
    eng.pf_table.copy_(torch.from_numpy(sch.table))
    eng.pf_ctx.fill_(9)
    eng.pf_x.copy_(synth.make_x(slots * 9, d.hidden, seed=1))
    torch.cuda.synchronize()
    eng.prefill(slots, 9, stream)
    eng.ctx.fill_(9)                          # the last position once more: the same codes and the same answer
    eng.x.copy_(synth.make_x(slots, d.hidden, seed=2))
    eng.table.copy_(torch.from_numpy(sch.table))
    torch.cuda.synchronize()
    eng.decode(stream)
    stream.synchronize()
    want = eng.decode(stream)
    stream.synchronize()
    want = want.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)
    y = eng.decode(stream)
    sch.retire(1)
    eng.compact(sch, stream)                  # returns when the stream is done
    assert torch.equal(y, want)
    assert int(eng.status.item()) == 0


@pytest.mark.parametrize("case", [(16, 14, 2, 64, [129], [255]), (16, 7, 7, 128, [129], [255]), (128, 8, 2, 128, [300, 0], [100, 257])])
def test_prefill_gives_the_same_bits_every_time(case):
    """Items of a few key tiles, whose codes follow each other into the same shared memory, 300 times."""
    bs, H, Hkv, d, before, new = case
    ctx = [b + n for b, n in zip(before, new)]
    rng = np.random.default_rng(sum(ctx))
    ref_pool, table = make_cache(rng, ctx, Hkv, d, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.normal(size=(int(cu[-1]), H, d))).bfloat16()
    pool, st = to_gpu(ref_pool), status()
    args = (q.cuda(), dev(cu), pool, dev(table), dev(ctx), d ** -0.5)
    first = api.paged_attention_prefill_f8(*args, max_new=max(new), status=st)
    assert_attention(first, *C.attention_f8(f64(q), ref_pool, table, ctx, cu, d ** -0.5), d)
    out, differ = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        out.fill_(5.0)
        api.paged_attention_prefill_f8(*args, max_new=max(new), out=out, status=st)
        differ += (out != first).any()
    check(st)
    assert int(differ.item()) == 0


def test_stack_over_e4m3_pools_replays_its_captured_step():
    """The captured all-layer step, replayed with other tables, contexts and inputs, against the plain calls."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, L, nb, mb, slots, prompt = synth.DIMS_TINY, 2, 40, 8, 3, 20
    cfg = api.make_config(d, max_position=mb * d.block_size)
    packed = [api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(d, 0.02, seed=50 + l).items()}) for l in range(L)]
    results, stream = [], torch.cuda.Stream()
    for captured in (False, True):
        pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim) for _ in range(L)]
        sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
        eng = StackEngine(api, [cfg] * L, packed, pools, slots, mb, slots * prompt)
        for s in range(slots):
            sch.start_resident(s, prompt)
        if captured:                          # with every slot empty: nothing is written
            torch.cuda.synchronize()
            eng.capture_decode(stream)
            stream.synchronize()
            eng.status.zero_()                # an empty context holds no room for the step's token: flagged
            assert all((p.k_scale == 0).all() and (p.v_scale == 0).all() for p in pools)
        eng.pf_table.copy_(torch.from_numpy(sch.table))
        eng.pf_ctx.fill_(prompt)
        eng.pf_x.copy_(synth.make_x(slots * prompt, d.hidden, seed=1))
        torch.cuda.synchronize()
        eng.prefill(slots, prompt, stream)
        ys = []
        for i in range(20):
            stream.synchronize()
            ctx = sch.grow_for_decode()
            eng.table.copy_(torch.from_numpy(sch.table))
            eng.ctx.copy_(torch.from_numpy(ctx))
            eng.x.copy_(synth.make_x(slots, d.hidden, seed=10 + i))
            torch.cuda.synchronize()
            y = eng.decode(stream)
            stream.synchronize()
            ys.append(y.clone())
        torch.cuda.synchronize()
        assert int(eng.status.item()) == 0
        results.append(ys + [t.view(torch.uint8) for p in pools for t in (p.k, p.v)] + [t for p in pools for t in (p.k_scale, p.v_scale)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_largest_batch():
    """65535 sequences of one token: the answer is the cached V row itself."""
    B, Hkv, d, bs = 65535, 1, 64, 16
    pool, st = api.PoolF8.empty(B, Hkv, bs, d), status()
    table = torch.randperm(B, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.int32).view(B, 1)
    ctx, cu = torch.ones(B, dtype=torch.int32, device="cuda"), torch.arange(B + 1, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    k, v = (torch.randn(B, Hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(B, 2, d, device="cuda", generator=g).bfloat16()
    api.append_to_cache_f8(k, v, pool, table, ctx, status=st)
    row = pool.v[table[:, 0].long(), :, 0].float() * pool.v_scale[table[:, 0].long()][..., None]
    want = row.expand(B, 2, d)                                           # codes times powers of two: exact in BF16
    assert (want - v.float()).abs().max() <= 2.0 ** -4 * v.float().abs().max()
    for out in (api.paged_attention_decode_f8(q, pool, table, ctx, 0.125, status=st),
                api.paged_attention_prefill_f8(q, cu, pool, table, ctx, 0.125, max_new=1, status=st)):
        assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs()).all()
    check(st)
    with pytest.raises(api.LayerError):
        api.append_to_cache_f8(torch.cat([k, k[:1]]), torch.cat([v, v[:1]]), pool, torch.cat([table, table[:1]]),
                               torch.ones(B + 1, dtype=torch.int32, device="cuda"), status=st)
