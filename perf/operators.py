"""The operators around a paged KV cache, measured as a serving program calls them.

* ``rope``      rotary positions of the Q and K heads of a merged QKV output (half or
                interleaved pairs, part of the head, scaled frequencies, forward and gradient);
* ``append``    new tokens' K and V into a cache of e4m3 codes with one power-of-two scale per
                block of tokens and KV head;
* ``decode``    attention of one new token per sequence over that cache;
* ``prefill``   attention of a ragged batch of new tokens over it, causal at the end;
* ``copy``      copying blocks in the pools of every layer at once (forked sequences);
* ``compact``   the plan that packs the blocks in use to the front, with the moves it asks for.

``run`` computes them in plain torch (``own`` false) or by the library's calls (``own`` true).
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
PHI = 0.6180339887498949

# Shapes: the 7B layer has 32 query and 32 KV heads of 128 in blocks of 128 tokens, the 70B-shaped
# layer 64 and 8, the tiny layer 4 and 2 heads of 64 in blocks of 16.


def listed():
    return [
        # the Q and K heads of one decode step of 64 sequences (7B): the smallest call, latency counts
        dict(name="rope step", op="rope", tokens=64, heads=32, kv_heads=32, dim=128, rot=128, layout="half",
             scaling="plain", factor=1.0, original=4096, max_position=4096, dtype="bf16", backward=False),
        # a long prompt of the 70B-shaped layer, frequencies scaled in bands for 131072 positions
        dict(name="rope long prompt", op="rope", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="banded", factor=16.0, original=8192, max_position=131072, dtype="bf16", backward=False),
        # the gradient through interleaved pairs in half of each head, float32, an odd token count
        dict(name="rope gradient", op="rope", tokens=5003, heads=32, kv_heads=4, dim=128, rot=64,
             layout="interleaved", scaling="yarn", factor=8.0, original=4096, max_position=32768, dtype="f32",
             backward=True),
        # the cache write of one decode step of 64 sequences (7B)
        dict(name="append step", op="append", batch=64, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=512, heads=32,
             kv_heads=32, dim=128, block=128),
        # the cache write of a ragged batch of prompt chunks (70B shape), some behind a cached prefix
        dict(name="append chunks", op="append", batch=8, new_lo=777, new_hi=4096, ctx_lo=4096, ctx_hi=6000, heads=64,
             kv_heads=8, dim=128, block=128),
        # two short conversations of the tiny layer: nothing but latency
        dict(name="decode tiny", op="decode", batch=2, ctx_lo=65, ctx_hi=333, heads=4, kv_heads=2, dim=64, block=16),
        # the 7B decode workload: 64 sequences, contexts of 512 to 4096 tokens
        dict(name="decode 7B", op="decode", batch=64, ctx_lo=512, ctx_hi=4096, heads=32, kv_heads=32, dim=128,
             block=128),
        # the 70B-shaped decode workload: 16 sequences, contexts of 4096 to 32768 tokens
        dict(name="decode 70B", op="decode", batch=16, ctx_lo=4096, ctx_hi=32768, heads=64, kv_heads=8, dim=128,
             block=128),
        # the 7B prefill workload: one prompt of 2048 tokens
        dict(name="prefill 7B", op="prefill", batch=1, new_lo=2048, new_hi=2048, ctx_lo=2048, ctx_hi=2048, heads=32,
             kv_heads=32, dim=128, block=128),
        # a ragged batch of prompt chunks behind cached prefixes (70B shape)
        dict(name="prefill chunks", op="prefill", batch=4, new_lo=511, new_hi=1024, ctx_lo=4096, ctx_hi=8192,
             heads=64, kv_heads=8, dim=128, block=64),
        # 64 forked sequences copy their last block in 8 layers of a BF16 cache (7B blocks of 1 MB a tensor)
        dict(name="copy forks", op="copy", kind="bf16", layers=8, blocks=160, pairs=64, kv_heads=32, dim=128,
             block=128),
        # 64 sequences of a 32-layer e4m3 cache (70B shape) are packed to the front of the pool
        dict(name="compact", op="compact", kind="f8", layers=32, blocks=512, used=320, moves=96, rows=64, kv_heads=8,
             dim=128, block=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefill", "copy", "compact"])
    dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 16, 32])
    heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if kv * g <= 64])
    if op == "rope":
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(4, dim // 2)])
        tokens = _log(rng, 1, max(2, 150_000_000 // ((heads + kv) * dim * 4)))
        return dict(op=op, tokens=min(tokens, 16384), heads=heads, kv_heads=kv, dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "banded", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([2048, 4096, 8192]),
                    max_position=_log(rng, 512, 131072), dtype=rng.choice(["bf16", "f32"]),
                    backward=rng.random() < 0.4)
    if op == "append":
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(3, min(4096, 16_000_000 // (batch * kv * dim))))
        lo = rng.randint(1, new)
        ctx = new + _log(rng, 1, 512)
        return dict(op=op, batch=batch, new_lo=lo, new_hi=new, ctx_lo=new, ctx_hi=ctx, heads=heads, kv_heads=kv,
                    dim=dim, block=block)
    if op == "decode":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 2, max(3, min(32768, 400_000_000 // (batch * kv * dim))))
        return dict(op=op, batch=batch, ctx_lo=rng.randint(1, hi), ctx_hi=hi, heads=heads, kv_heads=kv, dim=dim,
                    block=block)
    if op == "prefill":
        batch = _log(rng, 1, 8)
        new = _log(rng, 2, 2048 // batch)
        hi = new + _log(rng, 1, max(2, min(16384, 500_000_000 // (batch * new * heads))))
        return dict(op=op, batch=batch, new_lo=rng.randint(1, new), new_hi=new, ctx_lo=rng.randint(new, hi),
                    ctx_hi=hi, heads=heads, kv_heads=kv, dim=dim, block=block)
    kind = rng.choice(["bf16", "f8"])
    layers = _log(rng, 1, 32)
    each = 2 * layers * kv * block * dim * (2 if kind == "bf16" else 1)
    blocks = max(8, min(2048, _log(rng, 64, 4096), 2_000_000_000 // each))
    if op == "copy":
        return dict(op=op, kind=kind, layers=layers, blocks=blocks, pairs=rng.randint(1, blocks // 2), kv_heads=kv,
                    dim=dim, block=block)
    used = rng.randint(2, blocks - 1)
    moves = rng.randint(1, min(used, blocks - used))
    return dict(op=op, kind=kind, layers=layers, blocks=blocks, used=used, moves=moves, rows=rng.randint(1, used),
                kv_heads=kv, dim=dim, block=block)


# ---------------------------------------------------------------- sizes that follow from a case alone

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the largest among them."""
    v = [lo + int((hi - lo) * ((i * PHI) % 1.0) + 0.5) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(c):
    """(context lengths, new tokens) of the sequences of a case; a context counts its new tokens."""
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
    new = _spread(c["new_lo"], c["new_hi"], c["batch"]) if "new_lo" in c else [1] * c["batch"]
    return [max(a, n) for a, n in zip(ctx, new)], new


def _block_bytes(c):
    """Bytes of one block in all tensors of a copy or compact case."""
    code = c["kv_heads"] * c["block"] * c["dim"] * (2 if c["kind"] == "bf16" else 1)
    return 2 * c["layers"] * (code + (4 * c["kv_heads"] if c["kind"] == "f8" else 0))


def work(c):
    d, hq, hk = c["dim"], c.get("heads", 0), c["kv_heads"]
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["tokens"] * (hq + hk)
        table = min(c["tokens"], c["max_position"]) * c["rot"] * 4
        return {"bytes": 2 * rows * d * size + table + 4 * c["tokens"], "flops": 3 * rows * c["rot"]}
    if c["op"] == "copy":
        return {"bytes": 2 * c["pairs"] * _block_bytes(c) + 8 * c["pairs"], "flops": 0}
    if c["op"] == "compact":
        table = c["rows"] * -(-c["used"] // c["rows"]) * 4
        return {"bytes": 2 * c["moves"] * _block_bytes(c) + 2 * table + 4 * c["blocks"] + 16 * c["moves"], "flops": 0}
    ctx, new = _lengths(c)
    cache = sum(ctx) * hk * d * 2 + sum(-(-n // c["block"]) for n in ctx) * hk * 8
    if c["op"] == "append":
        return {"bytes": sum(new) * hk * d * 2 * 3 + c["batch"] * hk * 16, "flops": sum(new) * hk * d * 4}
    pairs = sum(n * a - n * (n - 1) // 2 for a, n in zip(ctx, new))
    return {"bytes": cache + 2 * sum(new) * hq * d * 2, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _scale_of(amax):
    """The smallest power of two s, at least 2^-117, with amax <= 448 s (0 for 0): float32."""
    mant, ex = torch.frexp(amax.float())
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(min=-117)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(mant))


def _codes_of(x, scale):
    """float32 values as e4m3 codes of x / scale (nearest even, saturating); codes 0 where the scale is 0."""
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    return q.clamp(-448.0, 448.0).to(F8)


def _cache(c, ctx, g):
    """An e4m3 pool as serving leaves it and the block tables of its sequences: heads differ in size, a few
    channels of K are large, the pool's blocks lie in random order."""
    bs, hk, d = c["block"], c["kv_heads"], c["dim"]
    need = [-(-n // bs) for n in ctx]
    wide = max(need) + 1
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(ctx), wide), -1, dtype=torch.int32)
    spots, at = [], 0
    for b, n in enumerate(need):
        spots += [b * wide + j for j in range(n)]
        at += n
    table = table.cuda().view(-1)
    table[torch.tensor(spots, device="cuda")] = perm[:at]
    pools = []
    for which in range(2):
        x = torch.randn(nb, hk, bs, d, generator=g, device="cuda", dtype=torch.bfloat16)
        x *= torch.exp(0.5 * torch.randn(1, hk, 1, 1, generator=g, device="cuda")).bfloat16()
        if which == 0:
            x[..., :: max(d // 4, 1)] *= 4
        s = _scale_of(x.abs().amax(dim=(2, 3)))
        codes = torch.empty(nb, hk, bs, d, dtype=F8, device="cuda")
        for i in range(0, nb, 64):
            codes[i:i + 64] = _codes_of(x[i:i + 64].float(), s[i:i + 64, :, None, None])
        pools += [codes, s]
    return dict(k=pools[0], k_scale=pools[1], v=pools[2], v_scale=pools[3], table=table.view(len(ctx), wide),
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"))


def _inv_freq(c):
    """(inverse frequencies in 64 bits, factor on cos and sin) of a rope case."""
    theta, rot, f, orig = 10000.0, c["rot"], c["factor"], c["original"]
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        theta *= f ** (rot / (rot - 2.0))
    w = theta ** (-i / rot)
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] == "banded":     # bands between 1 and 4 turns over the original context
        turns = orig * w / (2 * math.pi)
        t = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - t) * w / f + t * w, 1.0
    if c["scaling"] == "yarn":       # ramp between 32 turns and 1 turn over the original context
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


LAYERS = ("k", "v", "k_scale", "v_scale")


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c, "scale": 1.0 / math.sqrt(c["dim"])}
    if c["op"] == "rope":
        hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
        x = torch.randn(c["tokens"], (hq + 2 * hk) * d, generator=g, device="cuda")
        x = x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["q"] = x[:, :hq * d].view(-1, hq, d)               # views of the merged QKV rows
        s["k"] = x[:, hq * d:(hq + hk) * d].view(-1, hk, d)
        s["pos"] = torch.randint(0, c["max_position"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        w, m = _inv_freq(c)
        a = torch.arange(c["max_position"], device="cuda", dtype=torch.float64)[:, None] * w.cuda()
        s["table"] = (torch.stack((a.cos(), a.sin()), -1) * m).float().contiguous()   # kept by the program
        if own:
            from transformer_decoder_layer_llama_gb300 import api
            s["status"] = api.new_status()
        return s
    if c["op"] in ("copy", "compact"):
        nb, hk = c["blocks"], c["kv_heads"]
        n = 2 * c["layers"] * nb * hk * c["block"] * c["dim"]
        if c["kind"] == "bf16":
            pool = torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            pool = torch.randint(0, 127, (n,), generator=g, device="cuda", dtype=torch.uint8).view(F8)
            s["scales"] = torch.rand(2 * c["layers"], nb, hk, generator=g, device="cuda") + 0.01
        s["pool"] = pool.view(2 * c["layers"], nb, hk, c["block"], c["dim"])
        if c["op"] == "copy":        # the sources are in use, the destinations fresh
            p = torch.randperm(nb, generator=g, device="cuda")[:2 * c["pairs"]].to(torch.int32)
            s["pairs"] = p.view(-1, 2).contiguous()
        else:                        # `used` blocks are in the tables, `moves` of them behind the first `used`
            u, m, r = c["used"], c["moves"], c["rows"]
            low = torch.randperm(u, generator=g, device="cuda")[:u - m]
            high = u + torch.randperm(nb - u, generator=g, device="cuda")[:m]
            ids = torch.cat((low, high))
            ids = ids[torch.randperm(u, generator=g, device="cuda")].to(torch.int32)
            wide = -(-u // r)
            s["table"] = torch.full((r * wide,), -1, dtype=torch.int32, device="cuda")
            s["table"][:u] = ids
            s["table"] = s["table"].view(wide, r).t().contiguous()
        if own:
            from transformer_decoder_layer_llama_gb300 import api
            s["set"] = api.BlockSet(list(s["pool"]) + (list(s["scales"]) if "scales" in s else []))
            s["status"] = api.new_status()
        return s
    ctx, new = _lengths(c)
    s.update(_cache(c, ctx, g))
    s["new_hi"] = max(new)
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    s["one"] = s["new_hi"] == 1 and min(new) == 1
    t, hq, hk, d = sum(new), c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        x = torch.randn(t, (hq + 2 * hk) * d, generator=g, device="cuda").bfloat16()
        s["k_new"] = x[:, hq * d:(hq + hk) * d].view(t, hk, d)   # views of the merged QKV rows
        s["v_new"] = x[:, (hq + hk) * d:].view(t, hk, d)
    else:
        s["q"] = torch.randn(t, hq, d, generator=g, device="cuda").bfloat16()
    if own:
        from transformer_decoder_layer_llama_gb300 import api
        s["status"] = api.new_status()
        s["cache"] = api.PoolF8(s["k"], s["v"], s["k_scale"], s["v_scale"])
        size = 0
        if c["op"] == "decode":
            size = api.attention_decode_f8_workspace_size(c["batch"], hq, hk, d)
        elif c["op"] == "prefill":
            size = api.attention_prefill_f8_workspace_size(c["batch"], t, s["new_hi"], hq, hk, d)
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def _rope(s):
    c = s["c"]
    rot, sign = c["rot"], -1.0 if c["backward"] else 1.0
    cs = s["table"][s["pos"].long()]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1] * sign
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        out.append(torch.cat((r, y[..., rot:]), -1).to(x.dtype))
    return out


def _append(s):
    bs = s["c"]["block"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    t = s["k_new"].shape[0]
    seq = torch.searchsorted(cu, torch.arange(t, device="cuda"), right=True) - 1
    pos = ctx[seq] - (cu[seq + 1] - torch.arange(t, device="cuda"))
    blk = s["table"].long()[seq, pos // bs]
    # the block that holds each sequence's first new token keeps its earlier rows
    p0 = ctx - (cu[1:] - cu[:-1])
    first = s["table"].long().gather(1, (p0 // bs).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    keep = (p0 % bs > 0) & (cu[1:] > cu[:-1])
    head = first[keep]
    rows = torch.arange(bs, device="cuda")[None, :] < (p0 % bs)[keep][:, None]
    for x, pool, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        x = x.float()
        mag = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
        old = torch.zeros_like(scale)
        old[head] = scale[head]
        want = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand_as(mag), mag, "amax")
        new = torch.maximum(old, _scale_of(want))
        was = pool[head].float()
        again = _codes_of(was * old[head][:, :, None, None], new[head][:, :, None, None]).float()
        pool[head] = torch.where(rows[:, None, :, None], again, was).to(F8)
        pool.view(torch.uint8)[blk, :, pos % bs] = _codes_of(x, new[blk][:, :, None]).view(torch.uint8)
        scale[blk] = new[blk]
    return [s[n] for n in LAYERS]


def _rows(codes, scale, table):
    """The cached rows of every sequence, float32 [batch, kv_heads, positions, dim]."""
    at = table.clamp(min=0).long()
    x = codes.view(torch.uint8)[at].view(F8).float() * scale[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, live, scale):
    """softmax(q k^T scale) v over the live keys of each row (float32); rows without one give 0."""
    a = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~live, -math.inf)
    m = a.amax(-1, keepdim=True)
    a = a.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = a.sum(-1, keepdim=True)
    return (a @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _decode(s):
    c = s["c"]
    k, v = _rows(s["k"], s["k_scale"], s["table"]), _rows(s["v"], s["v_scale"], s["table"])
    live = torch.arange(k.shape[2], device="cuda") < s["ctx"][:, None]
    q = s["q"].float().view(c["batch"], c["kv_heads"], -1, c["dim"])
    return _attend(q, k, v, live[:, None, None, :], s["scale"]).view(s["q"].shape).bfloat16()


def _prefill(s):
    c = s["c"]
    k, v = _rows(s["k"], s["k_scale"], s["table"]), _rows(s["v"], s["v_scale"], s["table"])
    cu, b, n, hk, d = s["cu"].long(), c["batch"], s["new_hi"], c["kv_heads"], c["dim"]
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    real = i < count[:, None]                                              # [batch, n]
    q = s["q"][(cu[:-1, None] + i).clamp(max=int(s["q"].shape[0]) - 1)]    # padded [batch, n, heads, dim]
    q = q.float().view(b, n, hk, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    pos = s["ctx"][:, None] - count[:, None] + i
    live = (torch.arange(k.shape[2], device="cuda") <= pos[..., None]) & real[..., None]
    live = live[:, None, None].expand(b, 1, c["heads"] // hk, n, -1).flatten(2, 3)
    o = _attend(q, k, v, live, s["scale"]).view(b, c["heads"], n, d).transpose(1, 2)
    return o[real].bfloat16()


def _copy(s, src, dst):
    raw = s["pool"].view(torch.int16 if s["c"]["kind"] == "bf16" else torch.uint8)
    raw[:, dst] = raw[:, src]
    if "scales" in s:
        s["scales"][:, dst] = s["scales"][:, src]
    return [s[n] for n in ("pool", "scales") if n in s]


def _compact(s):
    """Blocks in use move to the free places before them: the k-th used block at or behind place `used` to the
    k-th free place before it."""
    nb, table = s["c"]["blocks"], s["table"].long()
    used = torch.zeros(nb + 1, dtype=torch.bool, device="cuda")
    used[torch.where(table >= 0, table, nb)] = True
    used = used[:nb]
    at = torch.arange(nb, device="cuda")
    total = used.sum()
    src, dst = torch.nonzero(used & (at >= total))[:, 0], torch.nonzero(~used & (at < total))[:, 0]
    where = torch.where(used, at, -1)
    where[src] = dst
    pairs = torch.full((nb // 2, 2), -1, dtype=torch.int32, device="cuda")
    pairs[:src.shape[0]] = torch.stack((src, dst), 1).int()
    moved = torch.where(table >= 0, where[table.clamp(min=0)], table).int()
    counts = torch.stack((total, torch.full_like(total, src.shape[0]))).int()
    return [moved, pairs, counts, where.int()] + _copy(s, src, dst)


def run(s):
    c = s["c"]
    if not own:
        if c["op"] == "rope":
            return _rope(s)
        if c["op"] == "append":
            return _append(s)
        if c["op"] == "decode":
            return _decode(s)
        if c["op"] == "prefill":
            return _prefill(s)
        if c["op"] == "copy":
            p = s["pairs"].long()
            return _copy(s, p[:, 0], p[:, 1])
        return _compact(s)
    from transformer_decoder_layer_llama_gb300 import api
    if c["op"] == "rope":
        return list(api.rope(s["q"], s["k"], s["pos"], s["table"], layout=c["layout"], backward=c["backward"],
                             status=s["status"]))
    if c["op"] == "append":
        api.append_to_cache_f8(s["k_new"], s["v_new"], s["cache"], s["table"], s["ctx"],
                               cu_new=None if s["one"] else s["cu"], max_new=s["new_hi"], status=s["status"])
        return [s[n] for n in LAYERS]
    if c["op"] == "decode":
        return api.paged_attention_decode_f8(s["q"], s["cache"], s["table"], s["ctx"], s["scale"],
                                             workspace=s["ws"], status=s["status"])
    if c["op"] == "prefill":
        return api.paged_attention_prefill_f8(s["q"], s["cu"], s["cache"], s["table"], s["ctx"], s["scale"],
                                              max_new=s["new_hi"], workspace=s["ws"], status=s["status"])
    if c["op"] == "copy":
        api.copy_blocks(s["set"], s["pairs"], status=s["status"])
        return [s[n] for n in ("pool", "scales") if n in s]
    moved, pairs, counts, where = api.compact_blocks(s["table"], c["blocks"], status=s["status"])
    api.copy_blocks(s["set"], pairs, n_pairs=counts[1:], status=s["status"])
    return [moved, pairs, counts, where] + [s[n] for n in ("pool", "scales") if n in s]


# ---------------------------------------------------------------- the definitions, in 64 bits

def _e4m3(x):
    """float64 values rounded to e4m3 (nearest even, saturating), as float64."""
    a = x.abs().clamp(max=448.0)
    step = ((torch.frexp(a.clamp(min=2.0 ** -6))[1].long() + (1023 - 4)) << 52).view(torch.float64)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        w, m = _inv_freq(c)
        a = s["pos"].double()[:, None] * w.cuda()
        turn = torch.polar(torch.full_like(a, m), -a if c["backward"] else a)[:, None]
        out, rot = [], c["rot"]
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            if c["layout"] == "half":
                z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
                y[..., :rot] = torch.cat((z.real, z.imag), -1)
            else:
                z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
            out.append(y)
        return out
    if c["op"] == "copy":
        n = [s["pool"]] + ([s["scales"]] if "scales" in s else [])
        for a, b in s["pairs"].tolist():
            for t in n:
                t[:, b] = t[:, a]
        return n
    if c["op"] == "compact":
        names = [s["pool"]] + ([s["scales"]] if "scales" in s else [])
        ids = sorted({v for row in s["table"].tolist() for v in row if v >= 0})
        total = len(ids)
        holes = sorted(set(range(total)) - set(ids))
        for a, b in zip([v for v in ids if v >= total], holes):
            for t in names:
                t[:, b] = t[:, a]
        return [None, None, None, None] + names
    ctx, new = _lengths(c)
    table = s["table"].tolist()
    bs, hk = c["block"], c["kv_heads"]
    if c["op"] == "append":
        got = {n: s[n].double() for n in LAYERS}
        start = s["cu"].tolist()
        for b in range(c["batch"]):
            p, end = ctx[b] - new[b], ctx[b]
            while p < end:
                stop = min((p // bs + 1) * bs, end)
                blk, lo, hi = table[b][p // bs], p % bs, p % bs + stop - p
                t0 = start[b] + p - (ctx[b] - new[b])
                for n in ("k", "v"):
                    x = s[n + "_new"][t0:t0 + stop - p].double().transpose(0, 1)
                    top = x.abs().amax(dim=(1, 2))
                    f = (torch.arange(1023 - 117, 1023 + 121, device="cuda") << 52).view(torch.float64)  # every scale
                    f = f[torch.searchsorted(448.0 * f, top)] * (top > 0)  # the first with top <= 448 f
                    if lo:
                        f = torch.maximum(f, got[n + "_scale"][blk])
                        got[n][blk][:, :lo] = _e4m3(got[n][blk][:, :lo] * (got[n + "_scale"][blk] / f)[:, None, None])
                    got[n][blk][:, lo:hi] = _e4m3(x / f[:, None, None])
                    got[n + "_scale"][blk] = f
                p = stop
        return [got[n] for n in LAYERS]
    out, at, g = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0, c["heads"] // hk
    for b in range(c["batch"]):
        ids = torch.tensor(table[b][:-(-ctx[b] // bs)], device="cuda")
        k, v = ((s[n].view(torch.uint8)[ids].view(F8).double() * s[n + "_scale"][ids].double()[..., None, None])
                .transpose(0, 1).flatten(1, 2)[:, :ctx[b]] for n in ("k", "v"))
        past = torch.arange(ctx[b], device="cuda") > torch.arange(ctx[b] - new[b], ctx[b], device="cuda")[:, None]
        for h in range(hk):
            q = s["q"][at:at + new[b], h * g:(h + 1) * g].double().transpose(0, 1)      # [g, n, d]
            a = ((q @ k[h].t()) / math.sqrt(c["dim"])).masked_fill_(past, -math.inf)
            out[at:at + new[b], h * g:(h + 1) * g] = (torch.softmax(a, -1) @ v[h]).transpose(0, 1)
        at += new[b]
    return out
