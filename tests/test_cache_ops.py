"""Host side of the operators around the cache: the oracle's pins, and what the library and the
binding refuse (CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from transformer_decoder_layer_llama_gb300 import api, synth

NULL = ctypes.c_void_p(0)
FAKE = 1 << 20                      # a non-null, 256-byte-aligned address that nothing on the host reads
INVALID, UNSUPPORTED, WORKSPACE = api.LL_ERR_INVALID_ARG, api.LL_ERR_UNSUPPORTED, api.LL_ERR_WORKSPACE


# ---------------------------------------------------------------- oracle pins

def test_e4m3_codes_against_torch():
    x = np.concatenate([np.linspace(-500, 500, 4001), np.linspace(-0.1, 0.1, 4001), C.E4M3[:127]])
    t = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float32)
    want = t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (C.e4m3_codes(t.double().numpy()) == want).all()
    assert C.e4m3_codes(np.array([np.inf, -np.inf, 449.0])).tolist() == [0x7E, 0xFE, 0x7E]
    assert C.E4M3[C.e4m3_codes(np.array([np.nan]))[0]] != C.E4M3[C.e4m3_codes(np.array([np.nan]))[0]]


def test_block_scale_is_the_smallest_power_of_two():
    for amax in (448.0, 448.1, 1e-30, 1.0, 3.0e38, 1e-45):
        s = C.block_scale(amax)
        assert amax <= 448 * s and (s == 2.0 ** -117 or amax > 448 * s / 2)
        assert math.frexp(s)[0] == 0.5
    assert C.block_scale(0.0) == 0.0


def test_append_in_steps_and_at_once_agree_up_to_subnormals():
    rng = np.random.default_rng(3)
    n, H, bs, d = 37, 2, 16, 8
    k, v = rng.normal(size=(2, n, H, d))
    table = np.array([[2, 0, 1]])
    mk = lambda: C.PoolF8(np.full((3, H, bs, d), 0x7F, np.uint8), np.full((3, H, bs, d), 0x7F, np.uint8),  # noqa: E731
                          np.full((3, H), np.nan), np.full((3, H), np.nan))
    a, b = mk(), mk()
    a.append(k, v, table, [n], [0, n])
    for i in range(n):
        b.append(k[i:i + 1], v[i:i + 1], table, [i + 1], [0, 1])
    for h in range(H):
        ka, va, _ = a.rows(table[0], n, h)
        kb, vb, _ = b.rows(table[0], n, h)
        assert (a.k_scale[2] == b.k_scale[2]).all()
        # a code is off by at most half a step, 2^-4 of the value; at most twice in two roundings
        assert (np.abs(ka - k[:, h]) <= 2 ** -4 * np.abs(k[:, h]) + 2.0 ** -10 * a.k_scale.max()).all()
        assert (np.abs(kb - k[:, h]) <= 2 ** -4 * np.abs(k[:, h]) + 2.0 ** -9 * b.k_scale.max()).all()
        assert np.isfinite(va).all() and np.isfinite(vb).all()
    assert (a.k[1, :, n - 32:] == 0x7F).all()          # rows behind the last token keep their bytes


def test_oracle_rope_turns_keep_lengths_and_transpose():
    rng = np.random.default_rng(1)
    x, y = rng.normal(size=(2, 5, 3, 12))
    pos = np.array([0, 1, 7, 100, 131071])
    for layout in ("half", "interleaved"):
        f, m = C.inv_freq(8)
        r = C.rope(x, pos, f, m, layout)
        assert np.allclose(np.linalg.norm(r, axis=-1), np.linalg.norm(x, axis=-1))
        assert (r[0] == x[0]).all() and (r[..., 8:] == x[..., 8:]).all()
        assert np.isclose((r * y).sum(), (x * C.rope(y, pos, f, m, layout, backward=True)).sum())
    for scaling in ("linear", "ntk", "banded", "yarn"):
        f, m = C.inv_freq(128, scaling=scaling, factor=8.0, original=4096)
        w, _ = C.inv_freq(128)
        assert (f <= w * (1 + 1e-12)).all() and (f >= w / 8 * (1 - 1e-12)).all()
        assert np.isclose(f[-1], w[-1] / 8) and (scaling == "linear" or np.isclose(f[0], w[0]))


def test_oracle_attention_is_the_plain_softmax():
    rng = np.random.default_rng(2)
    H, Hkv, d, bs, ctx = 4, 2, 8, 16, 21
    pool = C.PoolF8(*(np.zeros((4, Hkv, bs, d), np.uint8) for _ in range(2)), *(np.zeros((4, Hkv)) for _ in range(2)))
    k, v = rng.normal(size=(2, ctx, Hkv, d))
    pool.append(k, v, [[3, 1]], [ctx], [0, ctx])
    q = rng.normal(size=(2, H, d))
    out, _, _ = C.attention_f8(q, pool, [[3, 1]], [ctx], [0, 2], 0.3)
    for t in range(2):
        for h in range(H):
            kk, vv, _ = pool.rows([3, 1], ctx - 1 + t, h // 2)
            s = kk @ q[t, h] * 0.3
            p = np.exp(s - s.max())
            assert np.allclose(out[t, h], p @ vv / p.sum())


def test_oracle_compaction_is_minimal():
    new, moves, U, m = C.compact(np.array([[7, 2, -1], [9, 7, 0]]), 12)
    assert U == 4 and moves == [(7, 1), (9, 3)]
    assert new.tolist() == [[1, 2, -1], [3, 1, 0]]
    assert m.tolist() == [0, -1, 2, -1, -1, -1, -1, 1, -1, 3, -1, -1]


# ---------------------------------------------------------------- refusals of the library

def rope_cfg(**kw):
    return api.make_rope_config(**{"rotary_dim": 64, **kw})


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=7), dict(theta=1.0), dict(theta=math.inf),
                                 dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan),
                                 dict(scaling="ntk", factor=2.0, rotary_dim=2),
                                 dict(scaling="banded", factor=2.0),
                                 dict(scaling="yarn", factor=2.0, original_max_position=4096, low_turns=8, high_turns=8),
                                 dict(scaling="yarn", factor=2.0, original_max_position=4096, attention_factor=-1.0)])
def test_rope_config_refusals(bad):
    c = rope_cfg(**bad)
    assert api.lib.ll_rope_table_size(ctypes.byref(c), 16) == 0
    assert api.lib.ll_rope_table(ctypes.byref(c), 16, FAKE, 1 << 20, NULL) == INVALID


def test_rope_table_sizes_and_refusals():
    c = rope_cfg()
    assert api.lib.ll_rope_table_size(ctypes.byref(c), 100) == 100 * 32 * 8
    assert api.lib.ll_rope_table_size(ctypes.byref(c), 0) == 0
    f = lambda *a: api.lib.ll_rope_table(ctypes.byref(c), *a, NULL)  # noqa: E731
    assert f(100, NULL, 1 << 20) == INVALID and f(100, FAKE + 4, 1 << 20) == INVALID
    assert f(100, FAKE, 100 * 32 * 8 - 1) == INVALID
    big = rope_cfg(rotary_dim=2048)
    assert api.lib.ll_rope_table(ctypes.byref(big), 1, FAKE, 1 << 20, NULL) == UNSUPPORTED
    layer = api.make_config(synth.DIMS_7B, 128)
    n = api.packed_weights_size(layer)
    assert api.lib.ll_pack_rope(ctypes.byref(layer), ctypes.byref(c), FAKE, n, NULL) == INVALID   # 64 of 128
    whole = rope_cfg(rotary_dim=128)
    assert api.lib.ll_pack_rope(ctypes.byref(layer), ctypes.byref(whole), FAKE, n - 1, NULL) == INVALID
    with pytest.raises(ValueError):
        rope_cfg(scaling="cubic")


ROPE = dict(q=FAKE, k=2 * FAKE, dtype=0, positions=FAKE, tokens=4, n_heads=2, n_kv_heads=1, head_dim=64, rotary_dim=64,
            layout=0, direction=0, q_stride=128, k_stride=64, table=FAKE, max_position=16, q_out=3 * FAKE,
            k_out=4 * FAKE, q_out_stride=128, k_out_stride=64, status=FAKE)


@pytest.mark.parametrize("bad,code", [(dict(dtype=2), INVALID), (dict(layout=2), INVALID), (dict(direction=2), INVALID),
                                      (dict(positions=0), INVALID), (dict(table=0), INVALID), (dict(table=FAKE + 8), INVALID),
                                      (dict(status=0), INVALID), (dict(tokens=-1), INVALID),
                                      (dict(n_heads=0, n_kv_heads=0), INVALID), (dict(n_heads=-1), INVALID),
                                      (dict(rotary_dim=66), INVALID), (dict(rotary_dim=63), INVALID),
                                      (dict(rotary_dim=0), INVALID), (dict(q=0), INVALID), (dict(k_out=0), INVALID),
                                      (dict(q_stride=127), INVALID), (dict(k_out_stride=63), INVALID),
                                      (dict(q=FAKE + 1), INVALID), (dict(max_position=0), INVALID),
                                      (dict(head_dim=2048, q_stride=4096, k_stride=2048, q_out_stride=4096,
                                            k_out_stride=2048), UNSUPPORTED),
                                      (dict(q_out=FAKE + 128), INVALID), (dict(q_out=2 * FAKE + 2), INVALID),
                                      (dict(k_out=FAKE + 64), INVALID), (dict(tokens=1 << 25), UNSUPPORTED),
                                      (dict(q_out=FAKE, q_out_stride=256), INVALID)])
def test_rope_refusals(bad, code):
    assert api.lib.ll_rope(*{**ROPE, **bad}.values(), NULL) == code


# q and k as the columns of one buffer of 384-element rows: 0 .. 127 and 128 .. 191
MERGED = dict(q=FAKE, k=FAKE + 256, q_stride=384, k_stride=384, q_out_stride=384, k_out_stride=384)


@pytest.mark.parametrize("out", [dict(q_out=FAKE, k_out=FAKE),                       # k over q, which is rotated in place
                                 dict(q_out=FAKE, k_out=FAKE + 254),
                                 dict(q_out=FAKE + 200, k_out=FAKE + 256),           # q over its own columns
                                 dict(q_out=FAKE + 512, k_out=FAKE + 512 + 128),     # the outputs over each other
                                 dict(q_out=FAKE + 384, k_out=FAKE + 384 + 768),     # a row later is the same columns
                                 dict(q_out=FAKE + 640, k_out=FAKE + 256),           # q over the next row's start
                                 dict(q_out=8 * FAKE, k_out=8 * FAKE + 255 * 2, q_out_stride=256),   # strides that differ
                                 dict(q_out=8 * FAKE, k_out=8 * FAKE),
                                 dict(k=FAKE, q_out=FAKE, k_out=8 * FAKE)])          # k is read while q is rotated
def test_rope_refuses_outputs_that_share_memory(out):
    assert api.lib.ll_rope(*{**ROPE, **MERGED, **out}.values(), NULL) == INVALID


def test_rope_without_tokens_launches_nothing():
    assert api.lib.ll_rope(*{**ROPE, "tokens": 0}.values(), NULL) == api.LL_OK


def pool_f8(**kw):
    return api.ll_kv_pool_f8(*{**dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_blocks=8), **kw}.values())


SHAPES = [(dict(head_dim=96), UNSUPPORTED), (dict(block_size=24), UNSUPPORTED), (dict(block_size=8), UNSUPPORTED),
          (dict(block_size=512), UNSUPPORTED), (dict(batch=0), INVALID), (dict(max_blocks=0), INVALID),
          (dict(n_kv_heads=0), INVALID), (dict(block_table=0), INVALID), (dict(context_lens=0), INVALID),
          (dict(status=0), INVALID), (dict(max_blocks=1 << 27), UNSUPPORTED),
          (dict(pool=pool_f8(k=0)), INVALID), (dict(pool=pool_f8(v_scale=0)), INVALID),
          (dict(pool=pool_f8(num_blocks=0)), INVALID), (dict(pool=pool_f8(k=FAKE + 8)), INVALID),
          (dict(pool=pool_f8(k_scale=FAKE + 2)), INVALID), (dict(pool=pool_f8(num_blocks=1 << 27)), UNSUPPORTED)]

APPEND = dict(k=FAKE, v=FAKE, k_stride=256, v_stride=256, cu_new=FAKE, tokens=4, context_lens=FAKE, batch=2, max_new=4,
              n_kv_heads=2, head_dim=128, block_size=16, pool=pool_f8(), block_table=FAKE, max_blocks=4, status=FAKE)


@pytest.mark.parametrize("bad,code", SHAPES + [(dict(k=0), INVALID), (dict(v=FAKE + 8), INVALID), (dict(k_stride=252), INVALID),
                                               (dict(v_stride=248), INVALID), (dict(max_new=0), INVALID),
                                               (dict(cu_new=0), INVALID), (dict(cu_new=0, max_new=1), INVALID),
                                               (dict(tokens=-1), INVALID), (dict(batch=1 << 17), UNSUPPORTED)])
def test_append_refusals(bad, code):
    a = {**APPEND, **bad}
    a["pool"] = ctypes.byref(a["pool"])
    assert api.lib.ll_append_to_cache_f8(*a.values(), NULL) == code


DECODE = dict(q=FAKE, pool=pool_f8(), block_table=FAKE, max_blocks=4, context_lens=FAKE, batch=2, n_heads=4, n_kv_heads=2,
              head_dim=128, block_size=16, scale=0.1, out=FAKE, workspace=FAKE, workspace_bytes=1 << 30, status=FAKE)
PREFILL = dict(q=FAKE, cu_new=FAKE, tokens=4, pool=pool_f8(), block_table=FAKE, max_blocks=4, context_lens=FAKE, batch=2,
               max_new=4, n_heads=4, n_kv_heads=2, head_dim=128, block_size=16, scale=0.1, out=FAKE, workspace=FAKE,
               workspace_bytes=1 << 40, status=FAKE)
ATTN = SHAPES + [(dict(q=0), INVALID), (dict(q=FAKE + 2), INVALID), (dict(out=0), INVALID), (dict(scale=-1.0), INVALID),
                 (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(n_heads=5), UNSUPPORTED),
                 (dict(n_heads=34), UNSUPPORTED), (dict(workspace=0), WORKSPACE), (dict(workspace=FAKE + 8), WORKSPACE),
                 (dict(workspace_bytes=0), WORKSPACE)]


@pytest.mark.parametrize("bad,code", ATTN)
def test_decode_f8_refusals(bad, code):
    a = {**DECODE, **bad}
    a["pool"] = ctypes.byref(a["pool"])
    assert api.lib.ll_paged_attention_decode_f8(*a.values(), NULL) == code


@pytest.mark.parametrize("bad,code", ATTN + [(dict(cu_new=0), INVALID), (dict(max_new=0), INVALID), (dict(tokens=-1), INVALID)])
def test_prefill_f8_refusals(bad, code):
    a = {**PREFILL, **bad}
    a["pool"] = ctypes.byref(a["pool"])
    assert api.lib.ll_paged_attention_prefill_f8(*a.values(), NULL) == code


def test_f8_workspace_sizes():
    assert api.attention_decode_f8_workspace_size(4, 32, 8, 128) > 0
    assert api.attention_decode_f8_workspace_size(4, 32, 5, 128) == 0
    assert api.attention_decode_f8_workspace_size(4, 32, 8, 96) == 0
    assert api.attention_decode_f8_workspace_size(0, 32, 8, 128) == 0
    assert api.attention_prefill_f8_workspace_size(4, 100, 50, 32, 8, 128) > 0
    assert api.attention_prefill_f8_workspace_size(4, 100, 0, 32, 8, 128) == 0


def test_copy_blocks_refusals():
    def call(tensors, nb=8, pairs=FAKE, n=4, status=FAKE):
        arr = (api.ll_block_tensor * max(len(tensors), 1))(*tensors)
        return api.lib.ll_copy_blocks(arr, len(tensors), nb, pairs, n, NULL, status, NULL)
    ok = (FAKE, 64)
    assert call([]) == INVALID and call([ok], nb=0) == INVALID and call([ok], pairs=0) == INVALID
    assert call([ok], n=-1) == INVALID and call([ok], status=0) == INVALID and call([ok], pairs=FAKE + 4) == INVALID
    assert call([(0, 64)]) == INVALID and call([(FAKE, 0)]) == INVALID and call([(FAKE, 6)]) == INVALID
    assert call([(FAKE + 2, 64)]) == INVALID and call([ok, (FAKE, 1 << 31)]) == UNSUPPORTED
    assert call([ok], n=0) == api.LL_OK
    assert api.lib.ll_copy_blocks(None, 1, 8, FAKE, 1, NULL, FAKE, NULL) == INVALID


def test_compact_blocks_refusals():
    base = dict(table=FAKE, rows=4, max_blocks=8, nb=16, new=FAKE, pairs=FAKE, counts=FAKE, map=FAKE, status=FAKE)
    call = lambda **kw: api.lib.ll_compact_blocks(*{**base, **kw}.values(), NULL)  # noqa: E731
    for bad in (dict(table=0), dict(rows=-1), dict(max_blocks=-1), dict(nb=0), dict(new=0), dict(pairs=0), dict(counts=0),
                dict(map=0), dict(status=0), dict(pairs=FAKE + 4), dict(new=FAKE + 8)):
        assert call(**bad) == INVALID, bad
    assert call(nb=(1 << 19) + 1) == UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    tab = torch.zeros(8, 32, 2)
    with pytest.raises(ValueError, match="GPU"):
        api.rope(x, x, pos, tab)
    with pytest.raises(TypeError):
        api.rope(x.half(), None, pos, tab)
    with pytest.raises(ValueError, match="layout"):
        api.rope(x, None, pos, tab, layout="other")
    with pytest.raises(ValueError):
        api.rope(None, None, pos, tab)
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        api.PoolF8(codes, codes, torch.zeros(4, 2), torch.zeros(4, 2))
    f8 = codes.view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="GPU"):
        api.PoolF8(f8, f8, torch.zeros(4, 2), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        api.BlockSet([])
    with pytest.raises(ValueError):
        api.BlockSet([codes])
    with pytest.raises(ValueError, match="GPU"):
        api.compact_blocks(torch.zeros(2, 2, dtype=torch.int32), 8)


# ---------------------------------------------------------------- the serving side

def test_shared_blocks_are_freed_with_their_last_holder():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator
    a = BlockAllocator(8, seed=1)
    x = a.alloc(3)
    a.share(x[:2])
    assert [a.holders(b) for b in x] == [2, 2, 1]
    a.free(x)
    assert a.free_count() == 6 and a.holders(x[0]) == 1
    a.free(x[:2])
    assert a.free_count() == 8
    with pytest.raises(ValueError):
        a.share([x[0]])
    with pytest.raises(ValueError):
        a.free([x[0]])


def test_fork_retire_and_compaction_keep_the_books():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    nb, bs = 30, 16
    sch = Scheduler(4, bs, 6, BlockAllocator(nb, seed=3), seed=1)
    sch.start_resident(0, 40)
    sch.start_resident(1, 32)
    pairs = sch.fork(0, 2)                   # 2 full blocks shared, the third copied
    r0, r2 = sch.slots[0], sch.slots[2]
    assert r2.blocks[:2] == r0.blocks[:2] and pairs == [(r0.blocks[2], r2.blocks[2])] and r2.ctx == 40
    assert sch.fork(1, 3) == []              # 32 = 2 full blocks: nothing is filling
    assert sch.alloc.free_count() == nb - 6
    with pytest.raises(ValueError):
        sch.fork(0, 1)
    sch.retire(0)
    assert sch.alloc.free_count() == nb - 5 and sch.alloc.holders(r2.blocks[0]) == 1 and (sch.table[0] == -1).all()
    with pytest.raises(ValueError):
        sch.fork(0, 0)
    new, moves, U, block_map = C.compact(sch.table, nb)
    sch.apply_map(block_map)
    assert (sch.table == new).all() and U == 5
    used = {b for r in sch.slots if r is not None for b in r.blocks}
    assert used == set(range(5)) and sch.alloc.alloc(1) == [5]
    assert sch.alloc.holders(sch.slots[1].blocks[0]) == 2


LAYER_F8 = dict(cfg=None, packed=FAKE, x=FAKE, ctx=FAKE, batch=2, seq_len=4, pool=pool_f8(), table=FAKE, max_blocks=4,
                y=2 * FAKE, ws=FAKE, ws_bytes=1 << 40, status=FAKE)


@pytest.mark.parametrize("bad,code", [(dict(packed=0), INVALID), (dict(x=0), INVALID), (dict(ctx=0), INVALID),
                                      (dict(table=0), INVALID), (dict(y=0), INVALID), (dict(y=FAKE), INVALID),
                                      (dict(status=0), INVALID), (dict(batch=0), INVALID), (dict(seq_len=0), INVALID),
                                      (dict(pool=pool_f8(k_scale=0)), INVALID), (dict(pool=pool_f8(v=FAKE + 4)), INVALID),
                                      (dict(batch=70000), UNSUPPORTED), (dict(max_blocks=1 << 27), UNSUPPORTED),
                                      (dict(seq_len=1 << 24), UNSUPPORTED), (dict(ws=0), WORKSPACE), (dict(ws_bytes=100), WORKSPACE)])
def test_layer_f8_refusals(bad, code):
    cfg = api.make_config(synth.DIMS_TINY, 128)
    a = {**LAYER_F8, **bad, "cfg": ctypes.byref(cfg)}
    a["pool"] = ctypes.byref(a["pool"])
    assert api.lib.ll_layer_prefill_f8(*a.values(), NULL) == code
    if "seq_len" not in bad:
        order = ("cfg", "packed", "x", "pool", "table", "max_blocks", "ctx", "batch", "y", "ws", "ws_bytes", "status")
        assert api.lib.ll_layer_decode_step_f8(*(a[k] for k in order), NULL) == code


def test_layer_f8_workspace_holds_the_fused_one():
    cfg = api.make_config(synth.DIMS_70B, 4096)
    assert api.lib.ll_workspace_size_f8(ctypes.byref(cfg), 64, 16) > api.workspace_size(cfg, 64, 16)
    assert api.lib.ll_workspace_size_f8(ctypes.byref(cfg), 0, 16) == 0


def engine_without_a_gpu(nb):
    """A StackEngine whose every GPU call fails the test."""
    from transformer_decoder_layer_llama_gb300.serving import StackEngine
    eng = StackEngine.__new__(StackEngine)
    for name in ("api", "pools", "_blocks", "table", "pf_table", "status"):
        setattr(eng, name, None)                       # (any use of them raises AttributeError)
    return eng


@pytest.mark.parametrize("how", ["a prefix of a request that is gone", "a prefix of one that runs", "blocks of no request"])
def test_compaction_refuses_blocks_held_outside_the_requests_before_it_moves_any(how):
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    sch = Scheduler(3, 16, 6, BlockAllocator(30, seed=3), seed=1)
    for s in range(3):
        sch.start_resident(s, 40)
    if how == "blocks of no request":
        kept = sch.alloc.alloc(2)
    else:
        kept = sch.slots[0].blocks[:2]
        sch.alloc.share(kept)
        if how == "a prefix of a request that is gone":
            sch.retire(0)
    assert sch.held_outside() == sorted(kept)
    before = sch.table.copy(), [list(r.blocks) if r else None for r in sch.slots], dict(sch.alloc._used), list(sch.alloc._free)
    stream = None                                      # (waiting on it raises AttributeError)
    with pytest.raises(ValueError, match="held outside"):
        engine_without_a_gpu(30).compact(sch, stream)
    after = sch.table.copy(), [list(r.blocks) if r else None for r in sch.slots], dict(sch.alloc._used), list(sch.alloc._free)
    assert (before[0] == after[0]).all() and before[1:] == after[1:]
    sch.alloc.free(kept)
    assert sch.held_outside() == []
    sch.fork(1, 0) if sch.slots[0] is None else None   # shared between requests: theirs
    assert sch.held_outside() == []


def test_a_step_with_an_empty_slot_changes_no_request():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    sch = Scheduler(3, 16, 6, BlockAllocator(30, seed=3), seed=1, prompt_len=20)
    for s in range(3):
        sch.start_resident(s, 32)                      # the next token starts a block
    sch.retire(1)
    books = lambda: [(r.ctx, r.budget, list(r.blocks)) if r else None for r in sch.slots]  # noqa: E731
    before, free, table = books(), sch.alloc.free_count(), sch.table.copy()
    with pytest.raises(ValueError, match="empty"):
        sch.grow_for_decode()
    assert books() == before and sch.alloc.free_count() == free and (sch.table == table).all()
    sch.fork(2, 1)
    assert sch.grow_for_decode().tolist() == [33, 33, 33]
    sch.retire(0)
    assert sch.retire_and_admit() == [0]               # an empty slot takes the next request
    assert sch.grow_for_decode().tolist() == [21, 34, 34]


@pytest.mark.parametrize("nb,width,error", [(7, 6, MemoryError), (30, 2, ValueError)])
def test_a_step_without_room_changes_no_request(nb, width, error):
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    sch = Scheduler(3, 16, width, BlockAllocator(nb, seed=3), seed=1)
    for s in range(3):
        sch.start_resident(s, 32)                      # two blocks each; the next token starts another
    books = lambda: [(r.ctx, r.budget, list(r.blocks)) for r in sch.slots]  # noqa: E731
    before, free, table = books(), sch.alloc.free_count(), sch.table.copy()
    with pytest.raises(error):
        sch.grow_for_decode()
    assert books() == before and sch.alloc.free_count() == free and (sch.table == table).all()


@pytest.mark.parametrize("cls,names", [("PoolF8", ("k", "v", "k_scale", "v_scale", "device")), ("BlockSet", ("tensors", "device", "num_blocks"))])
def test_the_tensors_of_a_pool_cannot_be_replaced(cls, names):
    """The library is given the addresses that were checked; a tensor put in their place would pass the checks and
    not be used."""
    obj = object.__new__(getattr(api, cls))
    for name in names:
        with pytest.raises(AttributeError):
            setattr(obj, name, torch.zeros(2))


def test_the_stack_waits_for_the_stream_of_its_own_device(monkeypatch):
    """copy_blocks and compact wait for the current stream of the tables' device, whichever device is current."""
    from types import SimpleNamespace

    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    eng = engine_without_a_gpu(8)
    eng.table, eng.pf_table = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    eng._blocks = SimpleNamespace(num_blocks=8)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("the stream of", device))

    class Waited(Exception):
        pass

    class Stream:
        def wait_stream(self, other):
            raise Waited(other)

    for call in (lambda: eng.copy_blocks([(0, 1)], Stream()),
                 lambda: eng.compact(Scheduler(2, 16, 2, BlockAllocator(8, seed=1), seed=1), Stream())):
        with pytest.raises(Waited) as e:
            call()
        assert e.value.args == (("the stream of", eng.table.device),)


def test_rope_refuses_to_lose_a_gradient():
    x, pos, tab = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(8, 32, 2)
    g = x.clone().requires_grad_()
    for q, k in ((g, None), (None, g), (x, g), (g * 2, x)):
        with pytest.raises(ValueError, match="autograd"):
            api.rope(q, k, pos, tab)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):      # as for any other tensor
            api.rope(q, k, pos, tab)


def test_a_banded_table_does_not_look_at_the_attention_factor():
    kw = dict(factor=2.0, original_max_position=4096, high_turns=4.0)
    for factor in (-1.0, math.nan, math.inf):
        assert api.lib.ll_rope_table_size(ctypes.byref(rope_cfg(scaling="banded", attention_factor=factor, **kw)), 16) == 16 * 32 * 8
        assert api.lib.ll_rope_table_size(ctypes.byref(rope_cfg(scaling="yarn", attention_factor=factor, **kw)), 16) == 0


def test_sizes_beyond_the_grids_are_refused_as_such():
    a = {**PREFILL, **dict(n_heads=128, n_kv_heads=128, batch=65535, tokens=1 << 24, max_new=65535)}   # 128 * 256 * 65535 items
    a["pool"] = ctypes.byref(pool_f8())
    assert api.lib.ll_paged_attention_prefill_f8(*a.values(), NULL) == UNSUPPORTED
    a["max_new"] = (1 << 31) - 1                       # an upper bound, cut to the tokens
    assert api.lib.ll_paged_attention_prefill_f8(*a.values(), NULL) == UNSUPPORTED
    w = 32767 * 128
    b = {**APPEND, **dict(n_kv_heads=32767, k_stride=w, v_stride=w, tokens=(1 << 31) - 1, max_new=(1 << 31) - 1, max_blocks=1 << 16)}
    b["pool"] = ctypes.byref(pool_f8())
    assert api.lib.ll_append_to_cache_f8(*b.values(), NULL) == UNSUPPORTED


def test_binding_refuses_status_words_of_other_types():
    for bad in (torch.zeros(1, dtype=torch.int64), torch.zeros(4, dtype=torch.uint8)[1:], torch.zeros(1)):
        with pytest.raises(TypeError, match="status"):
            api._status(bad)
    with pytest.raises(ValueError, match="GPU"):
        api._status(torch.zeros(1, dtype=torch.int32))
