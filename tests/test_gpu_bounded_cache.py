"""Normed heads, cache, attention weights and evictions together, as a server with a bounded cache uses them."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import weight_ops as W
from tests.helpers import bits, f64
from transformer_decoder_layer_llama_gb300 import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api

DIMS = synth.LayerDims(512, 8, 2, 128, 688, 16)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def check_status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


@pytest.mark.parametrize("int8", [False, True])
def test_a_served_batch_with_a_bounded_cache(int8):
    """Prompts: norm and rotate, write, weigh the rows; steps: norm and rotate at the uncut position, write, attend and
    weigh; whenever a sequence passes the bound, evict.  The reference keeps its own list of rows for each head and
    sequence; weights and outputs within 2^-6 of the largest value (BF16 heads and cache rows, 2^-8 each, and INT8 codes
    are taken from the library's own; what is compared is attention over the same rows)."""
    H, Hkv, d, bs, B, bound, sinks, recent = 8, 2, 128, 16, 3, 48, 2, 8
    G, mb, nb = H // Hkv, 6, 20
    g = torch.Generator().manual_seed(4)
    perm = torch.randperm(nb, generator=g).tolist()
    table = np.array([[perm.pop() for _ in range(mb)] for _ in range(B)])
    dt = i32(table)
    k_pool, v_pool = (torch.full((nb, Hkv, bs, d), math.nan).bfloat16().cuda() for _ in range(2))
    q8 = api.PoolQ8.empty(nb, Hkv, bs, d)
    gains = [(1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    rope = api.rope_table(api.make_rope_config(d), 256)
    freq, _ = C.inv_freq(d)
    weights, st, scale = torch.zeros(B, Hkv, mb * bs).cuda(), api.new_status(), 1 / math.sqrt(d)
    ref_w = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]
    lens, seen = [40, 33, 47], [40, 33, 47]                     # rows in the cache, tokens so far

    def heads(tokens, pos):
        x = torch.randn(tokens, (H + 2 * Hkv) * d, generator=g).bfloat16().cuda()
        q, k, v = x[:, :H * d].view(tokens, H, d), x[:, H * d:(H + Hkv) * d].view(tokens, Hkv, d), x[:, (H + Hkv) * d:].view(tokens, Hkv, d)
        q1, k1 = api.norm_rope(q, k, *gains, i32(pos), rope, status=st)
        ref = W.norm_rope(f64(k), f64(gains[1]), np.asarray(pos), freq, 1e-5, "half")
        assert (np.abs(f64(k1) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12).all()
        return q1, k1, v.contiguous()

    def write(k, v, seqs, places):
        slots = i32([table[b, p // bs] * bs + p % bs for b, p in zip(seqs, places)])
        if int8:
            api.reshape_and_cache_q8(k, v, slots, q8, status=st)
        api.reshape_and_cache(k, v, slots, k_pool, v_pool, status=st)      # (the prompts are weighed over BF16 keys)

    def rows(b, h, n):
        at = np.arange(n)
        blk = table[b, at // bs]
        if int8:
            codes, s = (t.cpu().numpy()[blk, h, at % bs] for t in (q8.k, q8.k_scale))
            vc, vs = (t.cpu().numpy()[blk, h, at % bs] for t in (q8.v, q8.v_scale))
            return codes.astype(np.float64) * s[:, None], vc.astype(np.float64) * vs[:, None]
        return f64(k_pool)[blk, h, at % bs], f64(v_pool)[blk, h, at % bs]

    def compare():
        for b in range(B):
            for h in range(Hkv):
                got = f64(weights[b, h])
                assert np.abs(got[:lens[b]] - ref_w[b][h]).max() <= 2.0 ** -6 * ref_w[b][h].max()
                assert (got[lens[b]:] == 0).all()

    # the prompts
    cu = np.cumsum([0] + lens)
    q, k, v = heads(cu[-1], np.concatenate([np.arange(n) for n in lens]))
    write(k, v, np.repeat(np.arange(B), lens), np.concatenate([np.arange(n) for n in lens]))
    api.paged_attention_weights(q, i32(cu), k_pool, dt, i32(lens), scale, weights, max(lens), status=st)
    for b in range(B):
        for h in range(Hkv):
            keys = f64(k_pool)[table[b, np.arange(lens[b]) // bs], h, np.arange(lens[b]) % bs]
            ref_w[b][h] = W.probabilities(f64(q[cu[b]:cu[b + 1], h * G:(h + 1) * G]), keys, scale, 0).sum((0, 1))
    check_status(st)
    compare()
    # steps, with evictions on the way
    for step in range(20):
        q, k, v = heads(B, seen)
        write(k, v, range(B), lens)
        lens, seen = [n + 1 for n in lens], [n + 1 for n in seen]
        if int8:
            out = api.paged_attention_decode_weights_q8(q, q8, dt, i32(lens), scale, weights, status=st)
        else:
            out = api.paged_attention_decode_weights(q, k_pool, v_pool, dt, i32(lens), scale, weights, status=st)
        check_status(st)
        for b in range(B):
            for h in range(Hkv):
                kk, vv = rows(b, h, lens[b])
                p = W.probabilities(f64(q[b, h * G:(h + 1) * G])[None], kk, scale, lens[b] - 1)[0]
                ref_w[b][h] = np.append(ref_w[b][h], 0.0) + p.sum(0)
                ref = p @ vv
                assert np.abs(f64(out[b, h * G:(h + 1) * G]) - ref).max() <= 2.0 ** -6 * np.abs(vv).max()
        compare()
        if max(lens) > bound:
            held = [[rows(b, h, lens[b]) for h in range(Hkv)] for b in range(B)]
            before = weights.clone()
            pool = q8 if int8 else (k_pool, v_pool)
            kept, new = api.evict_rows(pool, dt, i32(lens), weights, bound - 8, sinks=sinks, recent=recent, status=st)
            check_status(st)
            assert new.tolist() == [min(n, bound - 8) for n in lens]
            for b in range(B):
                for h in range(Hkv):
                    keep = W.keep_rows(before[b, h, :lens[b]].cpu().numpy(), bound - 8, sinks, recent)
                    assert (kept[b, h, :len(keep)].cpu().numpy() == keep).all()
                    ref_w[b][h] = ref_w[b][h][keep]
                    for a, o in zip(rows(b, h, len(keep)), held[b][h]):
                        assert (a == o[keep]).all()
            lens = new.tolist()
            compare()
    assert max(seen) > max(lens) and lens[0] <= bound


def layer(dims, seed, max_position=512):
    cfg = api.make_config(dims, max_position=max_position)
    return cfg, api.pack_weights(cfg, {k: v.cuda() for k, v in synth.make_weights(dims, 0.02, seed=seed).items()})


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B", [3, 40, 300])
def test_layer_step_with_weights(B, int8):
    """The step's output and cache are those of the plain step; its weights those of the attention over its own queries;
    other rotary positions are those of a step at that place.  (300 sequences take the prefill's form of the products.)"""
    dims, mb = DIMS, 5
    cfg, packed = layer(dims, 3)
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(1, mb * 16 + 1, (B,), generator=g).tolist()
    table, nb = synth.make_block_table([mb * 16] * B, 16, seed=1)
    table = table.cuda()
    x = synth.make_x(B, dims.hidden, seed=2).cuda()

    def pool():
        k, v = (t.cuda() for t in synth.make_pool(nb, dims, seed=5))
        if not int8:
            return k, v
        p = api.PoolQ8.empty(nb, 2, 16, 128)
        slots = torch.arange(nb * 16, dtype=torch.int32).cuda()
        flat = [t.transpose(1, 2).reshape(nb * 16, 2, 128).contiguous() for t in (k, v)]
        api.reshape_and_cache_q8(*flat, slots, p)
        return p
    tensors = lambda p: [p.k, p.v, p.k_scale, p.v_scale] if int8 else list(p)  # noqa: E731
    base = torch.rand(B, 2, mb * 16 + 7, generator=g).cuda()
    a, b, st = pool(), pool(), api.new_status()
    w, ws = base.clone(), api.new_workspace_weights(cfg, B, mb)
    y = api.layer_decode_step_weights(cfg, packed, x, a, table, i32(ctx), w, workspace=ws, status=st)
    if int8:
        want = api.layer_decode_step_q8(cfg, packed, x, b, table, i32(ctx))
    else:
        want = api.layer_decode_step(cfg, packed, x, *b, table, i32(ctx))
    check_status(st)
    assert torch.equal(y, want) and all(torch.equal(s, t) for s, t in zip(tensors(a), tensors(b)))
    q = api.checkpoints(cfg, ws, B, mb, B)["q"].view(B, 8, 128).clone()
    again = base.clone()
    if int8:
        api.paged_attention_decode_weights_q8(q, a, table, i32(ctx), 1 / math.sqrt(128), again)
    else:
        api.paged_attention_decode_weights(q, *a, table, i32(ctx), 1 / math.sqrt(128), again)
    assert torch.equal(again, w)
    # other positions: q and the new K are those of a step that stands there
    pos = [(c - 1 + 17) % (mb * 16) for c in ctx]
    a, b, w = pool(), pool(), base.clone()
    api.layer_decode_step_weights(cfg, packed, x, a, table, i32(ctx), w, positions=i32(pos), workspace=ws, status=st)
    q = api.checkpoints(cfg, ws, B, mb, B)["q"].clone()
    ws2 = api.new_workspace_weights(cfg, B, mb)
    api.layer_decode_step_weights(cfg, packed, x, b, table, i32([p + 1 for p in pos]), base.clone(), workspace=ws2, status=st)
    check_status(st)
    assert torch.equal(q, api.checkpoints(cfg, ws2, B, mb, B)["q"])
    place = lambda p, at: [t[table[torch.arange(B), torch.tensor(at) // 16].long(), :, torch.tensor(at) % 16] for t in tensors(p)]  # noqa: E731
    assert all(torch.equal(s, t) for s, t in zip(place(a, [c - 1 for c in ctx]), place(b, pos)))
    # a position beyond the table is flagged
    st = api.new_status()
    api.layer_decode_step_weights(cfg, packed, x, a, table, i32(ctx), w, positions=i32([512] + pos[1:]), workspace=ws, status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)


@pytest.mark.parametrize("captured", [False, True])
def test_stack_with_a_bounded_cache(captured):
    """A two-layer stack that evicts, against the same layer calls and evictions by hand."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, L, nb, mb, slots, prompt, keep = synth.DIMS_TINY, 2, 40, 5, 3, 40, 48
    layers = [layer(d, 60 + l) for l in range(L)]
    cfg, packed = layers[0][0], [p for _, p in layers]
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
    pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=l)) for l in range(L)]
    own = [tuple(t.clone() for t in p) for p in pools]
    eng = StackEngine(api, [cfg] * L, packed, pools, slots, mb, slots * prompt, track_weights=True)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    if captured:
        eng.ctx.fill_(1)
        torch.cuda.synchronize()
        eng.capture_decode(stream)                            # (table of -1: flagged, nothing is written)
        stream.synchronize()
        eng.status.zero_()
        eng.start_weights(range(slots), stream)
    for s in range(slots):
        sch.start_resident(s, prompt + s)
    weights = [torch.zeros(slots, d.n_kv_heads, mb * d.block_size).cuda() for _ in range(L)]
    st, cuts = api.new_status(), 0
    stream.synchronize()
    for i in range(30):
        ctx = sch.grow_for_decode()
        eng.table.copy_(torch.from_numpy(sch.table))
        eng.ctx.copy_(torch.from_numpy(ctx))
        eng.pos.copy_(torch.from_numpy(sch.positions()))
        assert sch.positions().tolist() == [prompt + s + i for s in range(slots)]
        x = synth.make_x(slots, d.hidden, seed=i)
        eng.x.copy_(x)
        torch.cuda.synchronize()
        y = eng.decode(stream)
        stream.synchronize()
        h = x.cuda()
        for l in range(L):
            h = api.layer_decode_step_weights(cfg, packed[l], h, own[l], i32(sch.table), i32(ctx), weights[l],
                                              positions=i32(sch.positions()), status=st)
        check_status(st)
        assert torch.equal(h, y) and all(torch.equal(a, b) for a, b in zip(weights, eng.weights))
        if max(r.ctx for r in sch.slots) > keep:
            table, lens = i32(sch.table), [r.ctx for r in sch.slots]
            done = eng.evict(sch, keep - 10, stream, sinks=2, recent=5)
            stream.synchronize()
            assert done == list(range(slots)) and [r.ctx for r in sch.slots] == [min(n, keep - 10) for n in lens]
            for l in range(L):
                api.evict_rows(own[l], table, i32(lens), weights[l], keep - 10, sinks=2, recent=5, status=st)
            check_status(st)
            assert all(torch.equal(a, b) for p, o in zip(pools, own) for a, b in zip(p, o))
            assert all(torch.equal(a, b) for a, b in zip(weights, eng.weights))
            assert all(len(r.blocks) == -(-r.ctx // d.block_size) for r in sch.slots)
            cuts += 1
    assert cuts >= 2 and int(eng.status.item()) == 0
    assert eng.evict(sch, 10 ** 6, stream) == []
    eng.start_weights([1], stream)
    eng.copy_weights(0, 2, stream)
    stream.synchronize()
    assert all((w[1] == 0).all() and torch.equal(w[0], w[2]) for w in eng.weights)


def test_a_shared_block_is_not_moved_into():
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, nb, mb, slots = synth.DIMS_TINY, 40, 5, 3
    cfg, packed = layer(d, 9)
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6)
    pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=1))]
    eng = StackEngine(api, [cfg], [packed], pools, slots, mb, 64, track_weights=True)
    sch.start_resident(0, 60)
    sch.start_resident(1, 60)
    sch.fork(0, 2)
    before, held = [bits(t) for t in pools[0]], [list(r.blocks) for r in sch.slots]
    stream = torch.cuda.Stream()
    with pytest.raises(ValueError, match="shared"):
        eng.evict(sch, 32, stream)
    stream.synchronize()
    assert all((a == bits(t)).all() for a, t in zip(before, pools[0])) and held == [list(r.blocks) for r in sch.slots]
    with pytest.raises(ValueError, match="track_weights"):
        StackEngine(api, [cfg], [packed], pools, slots, mb, 64).evict(sch, 32, stream)


@pytest.mark.parametrize("observe", [None, 0, 1, 7, 33])
def test_stack_prompts_start_the_weights(observe):
    """The weights after a prefill are those of the prompts' last queries over the keys the layers wrote, within 2^-6 of the
    largest (rows of BF16 queries and keys as they are); other slots keep theirs."""
    from transformer_decoder_layer_llama_gb300.serving import StackEngine
    d, L, nb, mb, S, T = synth.DIMS_TINY, 2, 30, 5, 4, 33
    layers = [layer(d, 70 + l) for l in range(L)]
    cfg, packed = layers[0][0], [p for _, p in layers]
    pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=l)) for l in range(L)]
    plain = [tuple(t.clone() for t in p) for p in pools]
    eng = StackEngine(api, [cfg] * L, packed, pools, S, mb, 2 * T, track_weights=True)
    ref = StackEngine(api, [cfg] * L, packed, plain, S, mb, 2 * T)
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(1))[:2 * mb].view(2, mb)
    stream = torch.cuda.Stream()
    for e in (eng, ref):
        e.pf_table[:2] = i32(table)
        e.pf_pos[:2 * T] = torch.arange(T, dtype=torch.int32).repeat(2).cuda()
        e.pf_x[:2 * T] = synth.make_x(2 * T, d.hidden, seed=3).cuda()
    for w in eng.weights:
        w.fill_(3.0)
    torch.cuda.synchronize()
    y = eng.prefill(2, T, stream, slots=[2, 0], observe=observe)
    want = ref.prefill(2, T, stream)
    stream.synchronize()
    assert torch.equal(y, want) and int(eng.status.item()) == 0
    assert all(torch.equal(a, b) for p, o in zip(pools, plain) for a, b in zip(p, o))
    n = T if observe is None else observe
    G = d.n_heads // d.n_kv_heads
    for l in range(L):
        got = f64(eng.weights[l])
        assert (got[[1, 3]] == 3).all() and (got[[0, 2]][:, :, T:] == 0).all()
        if l == L - 1 and n:
            q = f64(api.checkpoints(cfg, eng.ws, 2 * T, mb, 2 * T)["q"]).reshape(2, T, d.n_heads, d.head_dim)
            for i, s in enumerate((2, 0)):
                for h in range(d.n_kv_heads):
                    keys = f64(pools[l][0])[table[i].numpy()[np.arange(T) // d.block_size], h, np.arange(T) % d.block_size]
                    p = W.probabilities(q[i, T - n:, h * G:(h + 1) * G], keys, d.head_dim ** -0.5, T - n).sum((0, 1))
                    assert np.abs(got[s, h, :T] - p).max() <= 2.0 ** -6 * p.max()
        total = got[[0, 2]].sum(-1)
        assert (np.abs(total - n * G) <= 1e-4 * n * G).all()
    for bad in (dict(slots=[0]), dict(slots=[0, 0]), dict(slots=[0, S]), dict(slots=[0, 1], observe=T + 1)):
        with pytest.raises(ValueError):
            eng.prefill(2, T, stream, **bad)
    with pytest.raises(ValueError, match="track_weights"):
        ref.prefill(2, T, stream, slots=[0, 1])


def test_weights_beyond_32_bits():
    """Weights of 2.7e9 elements: the last sequences' lie behind 2^31.  The same bits as with narrow ones."""
    B, H, Hkv, d, bs, n, wide = 40, 16, 8, 64, 16, 300, 1 << 23
    g = torch.Generator().manual_seed(2)
    mb = -(-n // bs)
    table = i32(torch.randperm(B * mb, generator=g).view(B, mb))
    pools = [tuple(torch.randn(B * mb, Hkv, bs, d, generator=g).bfloat16().cuda() for _ in range(2))]
    pools.append(tuple(t.clone() for t in pools[0]))
    q, rows = torch.randn(B, H, d, generator=g).bfloat16().cuda(), torch.randn(B * 5, H, d, generator=g).bfloat16().cuda()
    ctx, cu, st = i32([n] * B), i32(range(0, 5 * B + 1, 5)), api.new_status()
    out = []
    for pool, width in zip(pools, (mb * bs, wide)):
        w = torch.zeros(B, Hkv, width, device="cuda")
        api.paged_attention_weights(rows, cu, pool[0], table, ctx, 0.125, w, 5, status=st)
        o = api.paged_attention_decode_weights(q, *pool, table, ctx, 0.125, w, status=st)
        kept, lens = api.evict_rows(pool, table, ctx, w, 200, sinks=2, recent=20, status=st)
        check_status(st)
        assert width < wide or (w[::13, :, mb * bs:] == 0).all()
        out.append((o, kept, lens, w[:, :, :mb * bs].clone()))
        del w
    assert all(torch.equal(a, b) for a, b in zip(*out)) and all(torch.equal(a, b) for a, b in zip(*pools))
    assert (out[0][3][-1, -1, :200] > 0).all()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["weights", "bf16", "e4m3"])
def test_capturing_between_steps_changes_nothing(kind):
    """Prompts, steps, the capture, steps: pools, weights, status and the last outputs are the same bits before and after
    capture_decode, whatever lies in x by then, and the replayed steps are those of an engine that captures nothing."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, L, nb, mb, slots, prompt = synth.DIMS_TINY, 2, 40, 5, 3, 21
    layers = [layer(d, 80 + l) for l in range(L)]
    cfg, packed = layers[0][0], [p for _, p in layers]
    results = []
    for captured in (False, True):
        sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
        if kind == "e4m3":
            pools = [api.PoolF8.empty(nb, d.n_kv_heads, d.block_size, d.head_dim) for _ in range(L)]
            parts = [t.view(torch.uint8) for p in pools for t in (p.k, p.v)] + [t for p in pools for t in (p.k_scale, p.v_scale)]
        else:
            pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=l)) for l in range(L)]
            parts = [t for p in pools for t in p]
        eng = StackEngine(api, [cfg] * L, packed, pools, slots, mb, slots * prompt, track_weights=kind == "weights")
        state = parts + (eng.weights or []) + [eng.status]
        for s in range(slots):
            sch.start_resident(s, prompt)
        eng.pf_table.copy_(torch.from_numpy(sch.table))
        eng.pf_ctx.fill_(prompt)
        eng.pf_pos.copy_(torch.arange(prompt, dtype=torch.int32).repeat(slots))
        eng.pf_x.copy_(synth.make_x(slots * prompt, d.hidden, seed=1))
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        eng.prefill(slots, prompt, stream, **({"slots": [0, 1, 2]} if kind == "weights" else {}))
        ys = []
        for i in range(6):
            stream.synchronize()
            if captured and i in (0, 3):
                eng.x.copy_(synth.make_x(slots, d.hidden, seed=99))
                torch.cuda.synchronize()
                before, y = [t.clone() for t in state], None if i == 0 else eng.y.clone()
                torch.cuda.synchronize()
                eng.capture_decode(stream)
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(before, state))
                assert y is None or torch.equal(y, eng.y)
                if i == 0:
                    eng.graph = None                          # (the next steps as plain calls)
            ctx = sch.grow_for_decode()
            eng.table.copy_(torch.from_numpy(sch.table))
            eng.ctx.copy_(torch.from_numpy(ctx))
            if kind == "weights":
                eng.pos.copy_(torch.from_numpy(sch.positions()))
            eng.x.copy_(synth.make_x(slots, d.hidden, seed=10 + i))
            torch.cuda.synchronize()
            eng.decode(stream)
            stream.synchronize()
            ys.append(eng.y.clone())
        torch.cuda.synchronize()
        assert int(eng.status.item()) == 0
        results.append(ys + [t.clone() for t in state])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_slot_starts_anew():
    """A request in the slot of one that has ended: its sums are those of a fresh engine's, and a prefill that does not say
    whose slots it fills is refused before anything is written; so are steps whose positions were never given."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, nb, mb, slots, prompt = synth.DIMS_TINY, 40, 5, 2, 25
    cfg, packed = layer(d, 90)
    stream = torch.cuda.Stream()

    def serve(before):
        """Weights and kept rows of the second request of slot 0; `before`: there was a first one."""
        pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=3))]
        sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
        eng = StackEngine(api, [cfg], [packed], pools, slots, mb, slots * prompt, track_weights=True)
        sch.start_resident(1, 3)
        for turn in range(2 if before else 1):
            sch.start_resident(0, prompt)
            eng.pf_table[:1].copy_(torch.from_numpy(sch.table[:1]))
            eng.pf_pos[:prompt].copy_(torch.arange(prompt, dtype=torch.int32))
            eng.pf_x[:prompt].copy_(synth.make_x(prompt, d.hidden, seed=7 + (before and turn == 0)))
            torch.cuda.synchronize()
            held = [t.clone() for t in (*pools[0], *eng.weights)]
            with pytest.raises(ValueError, match="slots"):
                eng.prefill(1, prompt, stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, (*pools[0], *eng.weights)))
            eng.prefill(1, prompt, stream, slots=[0], observe=9)
            kept = eng.weights[0].clone()
            eng.prefill(1, prompt, stream, slots=[])          # (leaves the weights)
            stream.synchronize()
            assert torch.equal(kept[0], eng.weights[0][0])
            for i in range(7):
                ctx = sch.grow_for_decode()
                eng.table.copy_(torch.from_numpy(sch.table))
                eng.ctx.copy_(torch.from_numpy(ctx))
                eng.pos.copy_(torch.from_numpy(sch.positions()))
                eng.x.copy_(synth.make_x(slots, d.hidden, seed=30 + i))
                torch.cuda.synchronize()
                eng.decode(stream)
                stream.synchronize()
            w = eng.weights[0][0].clone()
            assert eng.evict(sch, 20, stream, sinks=1, recent=3) == [0]
            stream.synchronize()
            rows = [t[torch.tensor(sch.slots[0].blocks).cuda()].transpose(1, 2).flatten(0, 1)[:20].clone() for t in pools[0]]
            if turn + 1 < (2 if before else 1):
                sch.retire(0)
        return [w, eng.weights[0][0].clone(), *rows]

    assert all(torch.equal(a, b) for a, b in zip(serve(True), serve(False)))
    # positions that nobody gave
    pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=3))]
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6, prompt_len=prompt)
    eng = StackEngine(api, [cfg], [packed], pools, slots, mb, slots * prompt, track_weights=True)
    for s in range(slots):
        sch.start_resident(s, prompt)
    eng.table.copy_(torch.from_numpy(sch.table))
    eng.ctx.copy_(torch.from_numpy(sch.grow_for_decode()))
    torch.cuda.synchronize()
    eng.decode(stream)
    stream.synchronize()
    assert int(eng.status.item()) == api.LL_DEV_BAD_POSITION


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("why", ["too far", "negative", "cache"])
def test_a_refused_token_leaves_its_row(why, kind):
    """A step whose token has no rotary position (behind the table, negative, or its place in the cache behind the table with
    none given): flagged, and codes, scales and rows of that place stay byte for byte, whatever an earlier call has left in the
    workspace; the other sequences' rows and outputs are those of a step without it."""
    dims, mb, B, far = DIMS, 5, 6, 2
    cfg, packed = layer(dims, 3, max_position=64)              # (the table of blocks reaches to 80)
    table, nb = synth.make_block_table([mb * 16] * B, 16, seed=1)
    table = table.cuda()
    ctx = [9, 64, 50, 17, 33, 1]
    if why == "cache":
        ctx[far] = 70
    pos = {"too far": 64, "negative": -1}
    positions = None if why == "cache" else i32([pos[why] if b == far else c - 1 for b, c in enumerate(ctx)])

    def pool():
        k, v = (t.cuda() for t in synth.make_pool(nb, dims, seed=5))
        if kind == "bf16":
            return k, v
        p = api.PoolQ8.empty(nb, 2, 16, 128)
        api.reshape_and_cache_q8(*(t.transpose(1, 2).reshape(nb * 16, 2, 128).contiguous() for t in (k, v)),
                                 torch.arange(nb * 16, dtype=torch.int32).cuda(), p)
        return p
    tensors = lambda p: [p.k, p.v, p.k_scale, p.v_scale] if kind == "int8" else list(p)  # noqa: E731
    ws = api.new_workspace_weights(cfg, B, mb)
    w = torch.zeros(B, 2, mb * 16, device="cuda")
    x, other = (synth.make_x(B, dims.hidden, seed=s).cuda() for s in (2, 3))
    # the workspace holds another step's rows
    api.layer_decode_step_weights(cfg, packed, other, pool(), table, i32([5] * B), w, workspace=ws)
    p, want, st = pool(), pool(), api.new_status()
    before = [t.clone() for t in tensors(p)]
    y = api.layer_decode_step_weights(cfg, packed, x, p, table, i32(ctx), w.zero_(), positions=positions, workspace=ws, status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    good = api.new_status()
    ref = api.layer_decode_step_weights(cfg, packed, x, want, table, i32([5 if b == far else c for b, c in enumerate(ctx)]),
                                        torch.zeros_like(w), status=good)
    check_status(good)
    rest = [b for b in range(B) if b != far]
    assert torch.equal(y[rest], ref[rest])
    for a, old, new in zip(tensors(p), before, tensors(want)):
        assert torch.equal(a[table[far].long()], old[table[far].long()])
        assert torch.equal(a[table[rest].long()], new[table[rest].long()])
    if why == "cache":                                         # the step without weights likewise
        p, st = pool(), api.new_status()
        if kind == "int8":
            api.layer_decode_step_q8(cfg, packed, x, p, table, i32(ctx), workspace=ws, status=st)
        else:
            api.layer_decode_step(cfg, packed, x, *p, table, i32(ctx), workspace=ws, status=st)
        check_status(st, api.LL_DEV_BAD_POSITION)
        for a, old in zip(tensors(p), before):
            assert torch.equal(a[table[far].long()], old[table[far].long()])


def test_a_forked_request_is_cut_once_it_has_its_own_blocks():
    """A fork: the other requests can still be cut, by name; with its blocks copied it can be, too, and the request that it
    shared them with keeps every byte."""
    from transformer_decoder_layer_llama_gb300.serving import BlockAllocator, Scheduler, StackEngine
    d, L, nb, mb, slots = synth.DIMS_TINY, 2, 40, 5, 3
    cfg, packed = layer(d, 9)
    sch = Scheduler(slots, d.block_size, mb, BlockAllocator(nb, seed=5), seed=6)
    pools = [tuple(t.cuda() for t in synth.make_pool(nb, d, seed=l)) for l in range(L)]
    eng = StackEngine(api, [cfg] * L, [packed] * L, pools, slots, mb, 64, track_weights=True)
    g = torch.Generator().manual_seed(1)
    for w in eng.weights:
        w.copy_(torch.rand(w.shape, generator=g))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    sch.start_resident(0, 60)
    sch.start_resident(1, 60)
    eng.copy_blocks(sch.fork(0, 2), stream)
    eng.copy_weights(0, 2, stream)

    def rows(slot, n):
        stream.synchronize()
        return [t[torch.tensor(sch.slots[slot].blocks).cuda()].transpose(1, 2).flatten(0, 1)[:n].clone() for p in pools for t in p]
    first, other = rows(0, 60), [w.clone() for w in eng.weights]
    assert all(torch.equal(a, b) for a, b in zip(first, rows(2, 60)))
    with pytest.raises(ValueError, match="shared"):
        eng.evict(sch, 32, stream, sinks=2, recent=5)
    assert eng.evict(sch, 32, stream, sinks=2, recent=5, slots=[1]) == [1] and [r.ctx for r in sch.slots] == [60, 32, 60]
    assert all(torch.equal(a, b) for s in (0, 2) for a, b in zip(first, rows(s, 60)))
    eng.copy_blocks(sch.unshare(2), stream)
    assert all(torch.equal(a, b) for s in (0, 2) for a, b in zip(first, rows(s, 60)))
    assert eng.evict(sch, 32, stream, sinks=2, recent=5, slots=[1, 2]) == [2] and [r.ctx for r in sch.slots] == [60, 32, 32]
    assert all(torch.equal(a, b) for a, b in zip(first, rows(0, 60)))
    got = rows(2, 32)
    for l in range(L):
        for h in range(d.n_kv_heads):
            keep = torch.from_numpy(W.keep_rows(other[l][2, h, :60].cpu().numpy(), 32, 2, 5)).cuda()
            for i in range(2):
                assert torch.equal(got[2 * l + i][:, h], first[2 * l + i][keep, h])
            assert torch.equal(eng.weights[l][2, h, :32], other[l][2, h, keep]) and (eng.weights[l][2, h, 32:60] == 0).all()
        assert torch.equal(eng.weights[l][0], other[l][0])
    assert eng.evict(sch, 32, stream, sinks=2, recent=5) == [0] and int(eng.status.item()) == 0
