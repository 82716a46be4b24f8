"""Attention weights and evictions, without a GPU: the oracle's pins and what the library refuses."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import weight_ops as W
from transformer_decoder_layer_llama_gb300 import api

FAKE = 1 << 20
NULL = None
OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)


def test_probabilities():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(3, 2, 8)), rng.normal(size=(5, 8))
    p = W.probabilities(q, k, 0.3, 2)
    assert np.allclose(p.sum(-1), 1) and (p[0, :, 3:] == 0).all() and (p[1, :, 4:] == 0).all() and (p[2] > 0).all()
    one = np.exp(0.3 * q[0] @ k[:3].T)
    assert np.allclose(p[0, :, :3], one / one.sum(-1, keepdims=True))
    assert (W.probabilities(q, k[:0], 0.3, -1).shape == (3, 2, 0))
    assert (W.probabilities(q, k, 0.3, -4) == 0).all()


def test_kept_rows_by_hand():
    w = np.array([5, 1, 9, 1, 0, 1, 2, 0.5])
    assert W.keep_rows(w, 8, 0, 0).tolist() == list(range(8))
    assert W.keep_rows(w, 3, 0, 0).tolist() == [0, 2, 6]
    assert W.keep_rows(w, 4, 0, 0).tolist() == [0, 1, 2, 6]          # of the ones the first
    assert W.keep_rows(w, 4, 1, 2).tolist() == [0, 2, 6, 7]
    assert W.keep_rows(w, 2, 5, 1).tolist() == [0, 7] and W.keep_rows(w, 2, 5, 3).tolist() == [6, 7]
    assert W.keep_rows(w, 0, 5, 3).tolist() == []
    assert W.keep_rows(np.array([np.nan, -np.inf, 1, np.nan]), 3, 0, 0).tolist() == [0, 1, 2]


def pool(**kw):
    return api.ll_kv_pool(*{**dict(k=FAKE, v=FAKE, num_blocks=8), **kw}.values())


def pool_q8(**kw):
    return api.ll_kv_pool_q8(*{**dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_blocks=8), **kw}.values())


DECODE = dict(q=FAKE, pool=pool(), table=FAKE, max_blocks=8, ctx=FAKE, batch=2, n_heads=4, n_kv_heads=2, head_dim=128, block=16,
              scale=0.1, weights=FAKE, width=128, out=FAKE, ws=FAKE, ws_bytes=1 << 40, status=FAKE)
DECODE_BAD = [(dict(q=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(table=0), INVALID), (dict(ctx=0), INVALID), (dict(batch=0), INVALID),
              (dict(n_heads=5), UNSUPPORTED), (dict(n_heads=34), UNSUPPORTED), (dict(n_kv_heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
              (dict(block=24), UNSUPPORTED), (dict(block=8), UNSUPPORTED), (dict(block=512), UNSUPPORTED), (dict(scale=-1.0), INVALID),
              (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(weights=0), INVALID), (dict(weights=FAKE + 2), INVALID),
              (dict(width=0), INVALID), (dict(out=0), INVALID), (dict(out=FAKE + 4), INVALID), (dict(ws=0), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
              (dict(ws=FAKE + 8), WORKSPACE), (dict(status=0), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(max_blocks=1 << 27), UNSUPPORTED),
              (dict(max_blocks=0), INVALID)]


@pytest.mark.parametrize("bad,code", DECODE_BAD + [(dict(pool=pool(k=0)), INVALID), (dict(pool=pool(v=FAKE + 8)), INVALID),
                                                   (dict(pool=pool(num_blocks=0)), INVALID), (dict(pool=pool(num_blocks=1 << 26)), UNSUPPORTED)])
def test_decode_refusals(bad, code):
    a = {**DECODE, **bad}
    assert api.lib.ll_paged_attention_decode_weights(*a.values(), NULL) == code


@pytest.mark.parametrize("bad,code", DECODE_BAD + [(dict(pool=pool_q8(k_scale=0)), INVALID), (dict(pool=pool_q8(v_scale=FAKE + 4)), INVALID),
                                                   (dict(head_dim=64), UNSUPPORTED)])
def test_decode_q8_refusals(bad, code):
    a = {**DECODE, "pool": pool_q8(), **bad}
    assert api.lib.ll_paged_attention_decode_weights_q8(*a.values(), NULL) == code


def test_decode_workspace():
    n = api.attention_decode_weights_workspace_size(2, 4, 2, 128, 8, 16)
    assert n >= api.attention_workspace_size(2, 4, 128, 8, 16) + 2 * 4 * 8 * 16 * 4
    assert api.attention_decode_weights_workspace_size(2, 4, 2, 96, 8, 16) == 0
    assert api.attention_decode_weights_workspace_size(0, 4, 2, 128, 8, 16) == 0


def rows(*pairs):
    return (api.ll_row_tensor * max(len(pairs), 1))(*pairs)


EVICT = dict(tensors=rows((6 * FAKE, 256), (5 * FAKE, 256)), n=2, num_blocks=8, n_kv_heads=2, block=16, table=FAKE, max_blocks=8, ctx=FAKE,
             batch=2, weights=2 * FAKE, width=128, keep=0, max_keep=64, sinks=1, recent=2, weights_out=2 * FAKE, kept=3 * FAKE,
             new_lens=4 * FAKE, status=FAKE)


@pytest.mark.parametrize("bad,code", [
    (dict(tensors=None), INVALID), (dict(n=0), INVALID), (dict(n=9), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(block=24), UNSUPPORTED), (dict(table=0), INVALID), (dict(max_blocks=0), INVALID), (dict(ctx=0), INVALID), (dict(batch=0), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(weights=0), INVALID), (dict(weights=2 * FAKE + 1), INVALID), (dict(width=0), INVALID),
    (dict(max_keep=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(weights_out=0), INVALID),
    (dict(weights_out=2 * FAKE + 128), INVALID), (dict(kept=0), INVALID), (dict(kept=2 * FAKE + 256), INVALID), (dict(new_lens=0), INVALID),
    (dict(new_lens=FAKE + 4), INVALID), (dict(new_lens=3 * FAKE + 16), INVALID), (dict(keep=4 * FAKE), INVALID), (dict(status=0), INVALID),
    (dict(tensors=rows((6 * FAKE, 256), (5 * FAKE, 6))), INVALID), (dict(tensors=rows((6 * FAKE, 256), (5 * FAKE, 0))), INVALID),
    (dict(tensors=rows((6 * FAKE, 256), (0, 256))), INVALID), (dict(tensors=rows((6 * FAKE, 256), (5 * FAKE + 2, 256))), INVALID),
    (dict(tensors=rows((6 * FAKE, 256), (5 * FAKE, 4100))), UNSUPPORTED), (dict(num_blocks=1 << 26), UNSUPPORTED), (dict(max_blocks=1 << 27), UNSUPPORTED),
    (dict(n_kv_heads=40000), UNSUPPORTED), (dict(tensors=rows((6 * FAKE, 256), (6 * FAKE, 256))), INVALID),
    (dict(tensors=rows((6 * FAKE, 256), (6 * FAKE + 8 * 2 * 16 * 256 - 4, 4))), INVALID), (dict(tensors=rows((6 * FAKE, 256), (2 * FAKE, 256))), INVALID),
    (dict(new_lens=2 * FAKE + 64), INVALID), (dict(kept=5 * FAKE), INVALID)])
def test_evict_refusals(bad, code):
    assert api.lib.ll_evict_rows(*{**EVICT, **bad}.values(), NULL) == code


def test_binding_refusals():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="pool"):
        api.evict_rows(k, i(1, 2), i(1), torch.zeros(1, 2, 32), 4)
    with pytest.raises(ValueError, match="GPU"):
        api.evict_rows((k, k), i(1, 2), i(1), torch.zeros(1, 2, 32), 4)


OBSERVE = dict(q=FAKE, cu=FAKE, tokens=16, k=FAKE, num_blocks=8, table=FAKE, max_blocks=8, ctx=FAKE, batch=2, max_new=8, n_heads=4,
               n_kv_heads=2, head_dim=128, block=16, scale=0.1, weights=FAKE, width=128, ws=FAKE, ws_bytes=1 << 40, status=FAKE)


@pytest.mark.parametrize("bad,code", [
    (dict(q=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(cu=0), INVALID), (dict(tokens=-1), INVALID), (dict(k=0), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(num_blocks=0), INVALID), (dict(num_blocks=1 << 26), UNSUPPORTED), (dict(table=0), INVALID),
    (dict(max_blocks=0), INVALID), (dict(max_blocks=1 << 27), UNSUPPORTED), (dict(ctx=0), INVALID), (dict(batch=0), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(max_new=0), INVALID), (dict(n_heads=6, n_kv_heads=4), UNSUPPORTED), (dict(n_heads=34), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(block=48), UNSUPPORTED), (dict(scale=-0.1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(weights=0), INVALID), (dict(weights=FAKE + 1), INVALID), (dict(width=0), INVALID), (dict(ws=0), WORKSPACE),
    (dict(ws_bytes=16), WORKSPACE), (dict(status=0), INVALID),
    (dict(batch=65535, n_kv_heads=128, n_heads=128, tokens=1 << 24, max_new=1 << 24), UNSUPPORTED)])
def test_observe_refusals(bad, code):
    assert api.lib.ll_paged_attention_weights(*{**OBSERVE, **bad}.values(), NULL) == code


STEP = dict(packed=FAKE, x=FAKE, pool=pool(), table=FAKE, max_blocks=8, ctx=FAKE, positions=0, batch=2, weights=FAKE, width=128,
            y=2 * FAKE, ws=FAKE, ws_bytes=1 << 40, status=FAKE)


@pytest.mark.parametrize("bad,code", [
    (dict(packed=0), INVALID), (dict(x=0), INVALID), (dict(table=0), INVALID), (dict(max_blocks=0), INVALID), (dict(ctx=0), INVALID),
    (dict(batch=0), INVALID), (dict(batch=70000), UNSUPPORTED), (dict(weights=0), INVALID), (dict(weights=FAKE + 2), INVALID),
    (dict(width=0), INVALID), (dict(y=0), INVALID), (dict(y=FAKE), INVALID), (dict(ws=0), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE),
    (dict(status=0), INVALID), (dict(pool=pool(v=0)), INVALID), (dict(max_blocks=1 << 27), UNSUPPORTED),
    (dict(pool=pool(num_blocks=1 << 28)), UNSUPPORTED)])
def test_layer_step_refusals(bad, code):
    from transformer_decoder_layer_llama_gb300 import synth
    cfg = api.make_config(synth.DIMS_TINY, 128)
    a = {**STEP, **bad}
    assert api.lib.ll_layer_decode_step_weights(ctypes.byref(cfg), *a.values(), NULL) == code
    c7 = api.make_config(synth.DIMS_7B, 128)
    if "pool" not in bad:
        assert api.lib.ll_layer_decode_step_weights_q8(ctypes.byref(c7), *{**a, "pool": pool_q8()}.values(), NULL) == code
    assert api.lib.ll_layer_decode_step_weights_q8(ctypes.byref(cfg), *{**STEP, "pool": pool_q8()}.values(), NULL) == UNSUPPORTED
    n = api.lib.ll_workspace_size_weights(ctypes.byref(c7), 4, 16)
    assert n >= api.workspace_size(c7, 4, 16) + 4 * 32 * 16 * 128 * 4
    assert api.lib.ll_workspace_size_weights(ctypes.byref(c7), 0, 16) == 0


def test_the_scheduler_cuts_a_request():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    sch = Scheduler(3, 16, 8, BlockAllocator(30, seed=3), seed=1)
    for s in range(2):
        sch.start_resident(s, 70 + s)
    free = sch.alloc.free_count()
    assert sch.positions().tolist() == [69, 70, -1]
    blocks = list(sch.slots[0].blocks)
    sch.cut(0, 33)
    assert sch.slots[0].blocks == blocks[:3] and sch.alloc.free_count() == free + 2
    assert sch.table[0].tolist() == blocks[:3] + [-1] * 5 and sch.positions().tolist() == [69, 70, -1]
    sch.fork(0, 2)
    assert sch.positions().tolist() == [69, 70, 69]
    assert sch.grow_for_decode().tolist() == [34, 72, 34] and sch.positions().tolist() == [70, 71, 70]
    with pytest.raises(ValueError, match="shared"):
        sch.own_blocks(0)
    sch.own_blocks(1)
    for bad in ((0, 35), (0, -1)):
        with pytest.raises(ValueError):
            sch.cut(*bad)
    sch.retire(2)
    sch.own_blocks(0)
    for call in (lambda: sch.own_blocks(2), lambda: sch.cut(2, 0)):
        with pytest.raises(ValueError):
            call()
    sch.cut(1, 0)
    assert sch.slots[1].blocks == [] and sch.held_outside() == []


def test_a_workspace_is_enough_for_smaller_calls():
    """One workspace, of the largest call, for calls of fewer rows, tokens, sequences and blocks (which are cut into more pieces)."""
    size = api.attention_weights_workspace_size
    for heads, kv in ((64, 8), (32, 32), (16, 1), (7, 7)):
        most = size(8, 2048, 2048, heads, kv, 128, 256, 128)
        assert most >= 2048 * heads * 4
        for batch, tokens, new, blocks in ((8, 2048, 256, 256), (8, 2048, 32, 256), (8, 2048, 1, 256), (1, 2048, 2048, 256), (1, 33, 33, 256),
                                           (3, 2000, 700, 8), (8, 0, 5, 1)):
            assert 0 < size(batch, tokens, new, heads, kv, 128, blocks, 128) <= most


def test_the_scheduler_unshares_a_request():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler
    sch = Scheduler(3, 16, 8, BlockAllocator(14, seed=3), seed=1)
    sch.start_resident(0, 70)
    sch.start_resident(1, 20)
    sch.fork(0, 2)
    first, second, free = list(sch.slots[0].blocks), list(sch.slots[2].blocks), sch.alloc.free_count()
    assert sch.unshare(1) == [] and first[:4] == second[:4]
    pairs = sch.unshare(2)
    assert [a for a, _ in pairs] == first[:4] and sch.slots[2].blocks == [b for _, b in pairs] + second[4:]
    assert sch.table[2].tolist() == sch.slots[2].blocks + [-1] * 3 and sch.slots[0].blocks == first
    assert not set(sch.slots[2].blocks) & set(first) and sch.alloc.free_count() == free - 4
    for s in range(3):
        sch.own_blocks(s)
        assert sch.unshare(s) == []
    sch.retire(1)
    sch.fork(0, 1)
    held, free = list(sch.slots[1].blocks), sch.alloc.free_count()
    with pytest.raises(MemoryError):
        sch.unshare(1)
    assert held == sch.slots[1].blocks and sch.alloc.free_count() == free and sch.held_outside() == []
    sch.retire(1)
    with pytest.raises(ValueError):
        sch.unshare(1)
