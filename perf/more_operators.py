"""Normed heads in front of the cache, and which of its rows stay, measured as a serving program calls them.

* ``norm``     RMS norm of every Q and K head with its gain, and the rotary positions, in one pass;
* ``grad``     its gradient: of the heads before it and of the gains;
* ``weigh``    attention of one new token per sequence over a paged cache (BF16, or INT8 with a scale
               for each token and head) that also adds every cached token's attention weight to a sum;
* ``observe``  the same sums for a ragged batch of prompt rows (whole prompts, chunks, the last rows);
* ``evict``    each sequence and KV head keeps its first and last rows and those of the largest sums,
               moved to the front of the sequence's blocks.

``run`` computes them in plain torch (``own`` false) or by the library's calls (``own`` true).
"""
import math

import torch

own = False

PHI = 0.6180339887498949
EPS = 1e-5

# Shapes: the 7B layer has 32 query and 32 KV heads of 128 in blocks of 128 tokens, the 70B-shaped
# layer 64 and 8, the tiny layer 4 and 2 heads of 64 in blocks of 16.


def listed():
    return [
        # the heads of one decode step of 64 sequences (7B): the smallest call, latency counts
        dict(name="norm step", op="norm", tokens=64, heads=32, kv_heads=32, dim=128, rot=128, layout="half",
             max_position=4096, dtype="bf16"),
        # a long prompt of the 70B-shaped layer
        dict(name="norm long prompt", op="norm", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, layout="half",
             max_position=131072, dtype="bf16"),
        # a training step's sequence of 4096 tokens, grouped heads
        dict(name="grad sequence", op="grad", tokens=4096, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             max_position=8192, dtype="bf16"),
        # an odd count of tokens in float32, interleaved pairs in half of each head
        dict(name="grad float", op="grad", tokens=1777, heads=16, kv_heads=4, dim=64, rot=32, layout="interleaved",
             max_position=32768, dtype="f32"),
        # two short conversations of the tiny layer: nothing but latency
        dict(name="weigh tiny", op="weigh", kind="bf16", batch=2, ctx_lo=65, ctx_hi=333, heads=4, kv_heads=2, dim=64,
             block=16),
        # the 7B decode workload: 64 sequences, contexts of 512 to 4096 tokens
        dict(name="weigh 7B", op="weigh", kind="bf16", batch=64, ctx_lo=512, ctx_hi=4096, heads=32, kv_heads=32,
             dim=128, block=128),
        # the 70B-shaped decode workload over an INT8 cache: 16 sequences, contexts of 4096 to 32768 tokens
        dict(name="weigh 70B", op="weigh", kind="int8", batch=16, ctx_lo=4096, ctx_hi=32768, heads=64, kv_heads=8,
             dim=128, block=128),
        # the 7B prefill workload: every row of one prompt of 2048 tokens
        dict(name="observe prompt", op="observe", batch=1, new_lo=2048, new_hi=2048, ctx_lo=2048, ctx_hi=2048,
             heads=32, kv_heads=32, dim=128, block=128),
        # the last 32 rows of eight long prompts (70B shape) say what their caches keep
        dict(name="observe windows", op="observe", batch=8, new_lo=32, new_hi=32, ctx_lo=4096, ctx_hi=16384,
             heads=64, kv_heads=8, dim=128, block=64),
        # 64 sequences (7B) that have grown a little beyond 1024 tokens, as between decode steps
        dict(name="evict steps", op="evict", kind="bf16", batch=64, ctx_lo=1025, ctx_hi=1280, keep=1024, spread=False,
             sinks=4, recent=64, kv_heads=32, dim=128, block=128),
        # 16 prompts (70B shape) of 4096 to 32768 tokens keep 4096 rows each
        dict(name="evict prompts", op="evict", kind="bf16", batch=16, ctx_lo=4096, ctx_hi=32768, keep=4096,
             spread=False, sinks=4, recent=512, kv_heads=8, dim=128, block=128),
        # one long document in an INT8 cache keeps an eighth of its 65536 tokens: few rows of weights, long ones
        dict(name="evict document", op="evict", kind="int8", batch=1, ctx_lo=65536, ctx_hi=65536, keep=8192,
             spread=False, sinks=16, recent=1024, kv_heads=8, dim=128, block=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "grad", "weigh", "observe", "evict"])
    dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 16, 32])
    heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if kv * g <= 64])
    if op in ("norm", "grad"):
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(4, dim // 2)])
        most = (150_000_000 if op == "norm" else 25_000_000) // ((heads + kv) * dim)
        return dict(op=op, tokens=min(_log(rng, 1, max(2, most)), 16384), heads=heads, kv_heads=kv, dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), max_position=_log(rng, 512, 131072),
                    dtype=rng.choice(["bf16", "f32"]) if op == "grad" or dim < 256 else "bf16")
    if op == "weigh":
        kind = rng.choice(["bf16", "int8"])
        dim = 128 if kind == "int8" else dim
        batch = _log(rng, 1, 64)
        hi = _log(rng, 2, max(3, min(32768, 400_000_000 // (batch * kv * dim))))
        return dict(op=op, kind=kind, batch=batch, ctx_lo=rng.randint(1, hi), ctx_hi=hi, heads=heads, kv_heads=kv,
                    dim=dim, block=block)
    if op == "observe":
        batch = _log(rng, 1, 8)
        new = _log(rng, 1, 2048 // batch)
        hi = new + _log(rng, 1, max(2, min(16384, 130_000_000 // (batch * new * heads))))
        return dict(op=op, batch=batch, new_lo=rng.randint(1, new), new_hi=new, ctx_lo=rng.randint(new, hi),
                    ctx_hi=hi, heads=heads, kv_heads=kv, dim=dim, block=block)
    kind = rng.choice(["bf16", "int8"])
    dim = 128 if kind == "int8" else dim
    batch = _log(rng, 1, 64)
    hi = _log(rng, 8, max(9, min(65536, 250_000_000 // (batch * kv * dim))))
    keep = rng.randint(1, hi)
    recent = rng.randint(0, keep)
    return dict(op=op, kind=kind, batch=batch, ctx_lo=rng.randint(1, hi), ctx_hi=hi, keep=keep,
                spread=rng.random() < 0.5, sinks=rng.randint(0, min(keep - recent, 32)), recent=recent, kv_heads=kv,
                dim=dim, block=block)


# ---------------------------------------------------------------- sizes that follow from a case alone

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the largest among them."""
    v = [lo + int((hi - lo) * ((i * PHI) % 1.0) + 0.5) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(c):
    """(context lengths, new rows) of the sequences of a case; a context counts its new rows."""
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"])
    new = _spread(c["new_lo"], c["new_hi"], c["batch"]) if "new_lo" in c else [1] * c["batch"]
    return [max(a, n) for a, n in zip(ctx, new)], new


def _keep(c):
    """Rows that each sequence of an evict case keeps at most."""
    return _spread(max(c["keep"] // 2, 1), c["keep"], c["batch"]) if c["spread"] else [c["keep"]] * c["batch"]


def _row_bytes(c):
    """Bytes of one cached token and KV head, K and V together."""
    return 2 * (c["dim"] + 4 if c.get("kind") == "int8" else 2 * c["dim"])


def work(c):
    d, hq, hk = c["dim"], c.get("heads", 0), c["kv_heads"]
    if c["op"] in ("norm", "grad"):
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["tokens"] * (hq + hk)
        table = min(c["tokens"], c["max_position"]) * c["rot"] * 4
        if c["op"] == "norm":
            return {"bytes": 2 * rows * d * size + table + 4 * c["tokens"] + 8 * d, "flops": rows * (4 * d + 3 * c["rot"])}
        return {"bytes": 3 * rows * d * size + table + 4 * c["tokens"] + 16 * d, "flops": rows * (12 * d + 3 * c["rot"])}
    ctx, new = _lengths(c)
    if c["op"] == "weigh":
        return {"bytes": sum(ctx) * hk * (_row_bytes(c) + 8) + 2 * c["batch"] * hq * d * 2,
                "flops": 4 * sum(ctx) * hq * d}
    if c["op"] == "observe":
        pairs = sum(n * a - n * (n - 1) // 2 for a, n in zip(ctx, new))
        return {"bytes": sum(ctx) * hk * (2 * d + 8) + sum(new) * hq * d * 2, "flops": 2 * pairs * hq * d}
    left = [min(n, k) for n, k in zip(ctx, _keep(c))]
    moved = sum(max(m - c["sinks"], 0) for m, n in zip(left, ctx) if m < n)
    return {"bytes": hk * (8 * sum(ctx) + 4 * sum(left) + 2 * moved * _row_bytes(c)), "flops": 0}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tables(c, ctx, g):
    """Block tables of the sequences over a pool whose blocks lie in random order; -1 behind a sequence's blocks."""
    bs = c["block"]
    need = [-(-n // bs) for n in ctx]
    wide = max(need) + 1
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(ctx) * wide,), -1, dtype=torch.int32, device="cuda")
    table[torch.tensor([b * wide + j for b, n in enumerate(need) for j in range(n)], device="cuda")] = perm[:sum(need)]
    return table.view(len(ctx), wide), nb


def _rows_of(c, nb, which, g):
    """Cached rows: heads differ in size, a few channels of K are large."""
    hk, bs, d = c["kv_heads"], c["block"], c["dim"]
    x = torch.randn(nb, hk, bs, d, generator=g, device="cuda", dtype=torch.bfloat16)
    x *= torch.exp(0.5 * torch.randn(1, hk, 1, 1, generator=g, device="cuda")).bfloat16()
    if which == 0:
        x[..., :: max(d // 4, 1)] *= 4
    return x


def _pool(c, nb, g):
    """K and V (BF16), or codes and scales (INT8: scale = largest / 127 of a token and head)."""
    out = {}
    for which, n in enumerate(("k", "v")):
        x = _rows_of(c, nb, which, g)
        if c.get("kind") != "int8":
            out[n] = x
            continue
        out[n] = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        out[n + "_scale"] = torch.empty(x.shape[:3], dtype=torch.float32, device="cuda")
        for i in range(0, nb, 64):
            y = x[i:i + 64].float()
            s = y.abs().amax(-1) / 127
            out[n][i:i + 64] = torch.round(y / torch.where(s > 0, s, 1.0)[..., None]).to(torch.int8)
            out[n + "_scale"][i:i + 64] = s
    return out


NAMES = ("k", "v", "k_scale", "v_scale")


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if own:
        from transformer_decoder_layer_llama_gb300 import api
        s["status"] = api.new_status()
    hq, hk, d = c.get("heads", 0), c["kv_heads"], c["dim"]
    if c["op"] in ("norm", "grad"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        x = torch.randn(c["tokens"], (hq + 2 * hk) * d, generator=g, device="cuda").to(dt)
        s["q"] = x[:, :hq * d].view(-1, hq, d)               # views of the merged QKV rows
        s["k"] = x[:, hq * d:(hq + hk) * d].view(-1, hk, d)
        s["q_gain"], s["k_gain"] = (1 + 0.1 * torch.randn(2, d, generator=g, device="cuda")).unbind(0)
        s["pos"] = torch.randint(0, c["max_position"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        w = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        a = torch.arange(c["max_position"], device="cuda", dtype=torch.float64)[:, None] * w
        s["table"] = torch.stack((a.cos(), a.sin()), -1).float().contiguous()        # kept by the program
        if c["op"] == "grad":
            s["dq"], s["dk"] = (torch.randn(t.shape, generator=g, device="cuda").to(dt) for t in (s["q"], s["k"]))
            if own:
                s["ws"] = torch.empty(api.norm_rope_backward_workspace_size(d), dtype=torch.uint8, device="cuda")
        return s
    ctx, new = _lengths(c)
    s["scale"] = 1.0 / math.sqrt(d)
    s["table"], nb = _tables(c, ctx, g)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    batch, wide = s["table"].shape
    # sums of earlier steps: most tokens little, some much, a few that no query has looked at
    past = torch.exp(1.5 * torch.randn(batch, hk, wide * c["block"], generator=g, device="cuda"))
    past *= torch.rand(past.shape, generator=g, device="cuda") >= 0.02
    past *= torch.arange(past.shape[2], device="cuda") < s["ctx"][:, None, None]
    s["weights"] = past
    if c["op"] == "observe":
        s["k"] = _rows_of(c, nb, 0, g)
        s["max_new"] = max(new)
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(sum(new), hq, d, generator=g, device="cuda").bfloat16()
        if own:
            s["ws"] = torch.empty(api.attention_weights_workspace_size(batch, sum(new), s["max_new"], hq, hk, d, wide,
                                                                       c["block"]), dtype=torch.uint8, device="cuda")
        return s
    s.update(_pool(c, nb, g))
    if c["op"] == "weigh":
        s["q"] = torch.randn(batch, hq, d, generator=g, device="cuda").bfloat16()
        if own:
            s["ws"] = torch.empty(api.attention_decode_weights_workspace_size(batch, hq, hk, d, wide, c["block"]),
                                  dtype=torch.uint8, device="cuda")
    else:
        s["keep"] = torch.tensor(_keep(c), dtype=torch.int32, device="cuda")
        s["weights_out"] = torch.zeros_like(s["weights"])
    if own:
        s["pool"] = api.PoolQ8(*(s[n] for n in NAMES)) if c["kind"] == "int8" else (s["k"], s["v"])
    return s


# ---------------------------------------------------------------- the plain forms

def _turn(y, cos, sin, layout, rot):
    """The rotation of the first `rot` elements of float32 heads."""
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, y[..., rot:]), -1)


def _norm(s):
    c = s["c"]
    cs = s["table"][s["pos"].long()]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    out = []
    for n in ("q", "k"):
        x = s[n].float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[n + "_gain"]
        out.append(_turn(y, cos, sin, c["layout"], c["rot"]).to(s[n].dtype))
    return out


def _grad(s):
    c = s["c"]
    cs = s["table"][s["pos"].long()]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    heads, gains = [], []
    for n in ("q", "k"):
        x = s[n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        dn = _turn(s["d" + n].float(), cos, -sin, c["layout"], c["rot"])
        x = x * r
        gains.append((dn * x).sum((0, 1), dtype=torch.float64).float())
        dn = dn * s[n + "_gain"]
        heads.append((r * (dn - x * (dn * x).mean(-1, keepdim=True))).to(s[n].dtype))
    return heads + gains


def _cached(s, n):
    """The cached rows of every sequence, float32 [batch, kv_heads, positions, dim]."""
    at = s["table"].clamp(min=0).long()
    x = s[n][at].float()
    if n + "_scale" in s:
        x = x * s[n + "_scale"][at][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _softmax(a, live):
    a = a.masked_fill_(~live, -math.inf)
    m = a.amax(-1, keepdim=True)
    a = a.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = a.sum(-1, keepdim=True)
    return a.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _weigh(s):
    c = s["c"]
    k, v = _cached(s, "k"), _cached(s, "v")
    live = torch.arange(k.shape[2], device="cuda") < s["ctx"][:, None]
    q = s["q"].float().view(c["batch"], c["kv_heads"], -1, c["dim"])
    p = _softmax((q @ k.transpose(-1, -2)).mul_(s["scale"]), live[:, None, None, :])
    s["weights"] += p.sum(2)
    return [(p @ v).view(s["q"].shape).bfloat16(), s["weights"]]


def _observe(s):
    c = s["c"]
    k = _cached(s, "k")
    cu, b, n, hk = s["cu"].long(), c["batch"], s["max_new"], c["kv_heads"]
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    q = s["q"][(cu[:-1, None] + i).clamp(max=int(s["q"].shape[0]) - 1)]    # padded [batch, n, heads, dim]
    q = q.float().view(b, n, hk, -1, c["dim"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    pos = s["ctx"][:, None] - count[:, None] + i
    live = (torch.arange(k.shape[2], device="cuda") <= pos[..., None]) & (i < count[:, None])[..., None]
    live = live[:, None, None].expand(b, 1, c["heads"] // hk, n, -1).flatten(2, 3)
    s["weights"] += _softmax((q @ k.transpose(-1, -2)).mul_(s["scale"]), live).sum(2)
    return [s["weights"]]


def _evict(s):
    c = s["c"]
    bs, wide, top = c["block"], s["weights"].shape[2], c["keep"]
    at = torch.arange(wide, device="cuda")
    ctx, keep = s["ctx"].long()[:, None, None], s["keep"].long()[:, None, None]
    left = torch.minimum(ctx, keep)
    recent = left.clamp(max=c["recent"])
    sinks = (left - recent).clamp(max=c["sinks"])
    # first and last rows before all others, rows behind the context behind them; equal weights by position
    rank = torch.where((at < sinks) | (at >= ctx - recent), math.inf, s["weights"])
    rank = torch.where(at < ctx, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(rank.shape, dtype=torch.bool, device="cuda").scatter_(2, order, (at < left).expand_as(rank))
    kept = torch.where(chosen, at, wide).sort(-1).values[..., :min(top, wide)]
    real = kept < wide
    from_ = kept.clamp(max=wide - 1)
    moved = torch.where(real, s["weights"].gather(2, from_), 0.0)
    inside = at < ctx
    full = torch.zeros_like(s["weights"])
    full[..., :kept.shape[2]] = moved
    s["weights_out"].copy_(torch.where(inside, full, s["weights_out"]))
    b, h, j = torch.nonzero(real & (left < ctx), as_tuple=True)
    src, dst = from_[b, h, j], j
    tab = s["table"].long()
    sb, db = tab[b, src // bs], tab[b, dst // bs]
    for n in NAMES:
        if n in s:
            s[n][db, h, dst % bs] = s[n][sb, h, src % bs]
    out = torch.full((c["batch"], c["kv_heads"], top), -1, dtype=torch.int32, device="cuda")
    out[..., :kept.shape[2]] = torch.where(real, kept, -1).int()
    return [out, left.view(-1).int(), s["weights_out"]] + [s[n] for n in NAMES if n in s]


PLAIN = {"norm": _norm, "grad": _grad, "weigh": _weigh, "observe": _observe, "evict": _evict}


def run(s):
    c = s["c"]
    if not own:
        return PLAIN[c["op"]](s)
    from transformer_decoder_layer_llama_gb300 import api
    if c["op"] == "norm":
        return list(api.norm_rope(s["q"], s["k"], s["q_gain"], s["k_gain"], s["pos"], s["table"], eps=EPS,
                                  layout=c["layout"], status=s["status"]))
    if c["op"] == "grad":
        return list(api.norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["q_gain"], s["k_gain"], s["pos"],
                                           s["table"], eps=EPS, layout=c["layout"], workspace=s["ws"],
                                           status=s["status"]))
    if c["op"] == "weigh":
        if c["kind"] == "int8":
            o = api.paged_attention_decode_weights_q8(s["q"], s["pool"], s["table"], s["ctx"], s["scale"], s["weights"],
                                                      workspace=s["ws"], status=s["status"])
        else:
            o = api.paged_attention_decode_weights(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["scale"],
                                                   s["weights"], workspace=s["ws"], status=s["status"])
        return [o, s["weights"]]
    if c["op"] == "observe":
        return [api.paged_attention_weights(s["q"], s["cu"], s["k"], s["table"], s["ctx"], s["scale"], s["weights"],
                                            max_new=s["max_new"], workspace=s["ws"], status=s["status"])]
    kept, left = api.evict_rows(s["pool"], s["table"], s["ctx"], s["weights"], s["keep"] if c["spread"] else c["keep"],
                                max_keep=c["keep"], sinks=c["sinks"], recent=c["recent"], weights_out=s["weights_out"],
                                status=s["status"])
    return [kept, left, s["weights_out"]] + [s[n] for n in NAMES if n in s]


# ---------------------------------------------------------------- the definitions, in 64 bits

def _sequence(s, n, b, length):
    """The first `length` cached rows of sequence b, float64 [kv_heads, length, dim]."""
    bs = s["c"]["block"]
    ids = s["table"][b, :-(-length // bs)].long()
    x = s[n][ids].double()
    if n + "_scale" in s:
        x = x * s[n + "_scale"][ids].double().unsqueeze(-1)
    return torch.cat(tuple(x), 1)[:, :length]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("norm", "grad"):
        rot, half = c["rot"], c["layout"] == "half"
        w = torch.exp(-math.log(10000.0) * torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * w)[:, None]

        def rotate(x, turn):
            y = x.clone()
            if half:
                z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
                y[..., :rot] = torch.cat((z.real, z.imag), -1)
            else:
                z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
            return y

        first, second = [], []
        for n in ("q", "k"):
            x, g = s[n].double(), s[n + "_gain"].double()
            length = torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + EPS)
            if c["op"] == "norm":
                first.append(rotate(x / length * g, turn))
                continue
            up = rotate(s["d" + n].double(), turn.conj())
            second.append(torch.einsum("thd,thd->d", up, x / length))
            up = up * g
            first.append(up / length - x * (up * x).sum(-1, keepdim=True) / (c["dim"] * length ** 3))
        return first + second
    ctx, new = _lengths(c)
    hk = c["kv_heads"]
    if c["op"] == "evict":
        keep = _keep(c)
        bs, kept_rows = c["block"], []
        weights = s["weights"].cpu()
        out = s["weights_out"].double()
        table = s["table"].cpu()
        for b in range(c["batch"]):
            n, m = ctx[b], min(ctx[b], keep[b])
            last = min(c["recent"], m)
            front = min(c["sinks"], m - last)
            middle = weights[b, :, front:n - last].double()
            # the middle rows before which fewer than the rest are larger, or equal and earlier
            rest = m - last - front
            order = torch.argsort(-middle, dim=-1, stable=True)[:, :rest].sort(-1).values + front
            rows = torch.cat((torch.arange(front).expand(hk, -1), order, torch.arange(n - last, n).expand(hk, -1)), 1)
            for h in range(hk):
                out[b, h, :n] = 0
                out[b, h, :m] = weights[b, h, rows[h]].double().cuda()
            kept_rows.append(rows)
            if m < n:
                blocks = table[b, torch.arange(n) // bs].long()
                off = torch.arange(n) % bs
                for t in NAMES:
                    if t in s:
                        for h in range(hk):
                            old = s[t][blocks.cuda(), h, off.cuda()]
                            s[t][blocks[:m].cuda(), h, off[:m].cuda()] = old[rows[h].cuda()]
        return [None, None, out] + [s[t] for t in NAMES if t in s]
    total = s["weights"].double()
    at, g, outs = 0, c["heads"] // hk, []
    for b in range(c["batch"]):
        k = _sequence(s, "k", b, ctx[b])
        v = _sequence(s, "v", b, ctx[b]) if c["op"] == "weigh" else None
        past = torch.arange(ctx[b], device="cuda") > torch.arange(ctx[b] - new[b], ctx[b], device="cuda")[:, None]
        for h in range(hk):
            q = s["q"][at:at + new[b], h * g:(h + 1) * g].double().transpose(0, 1)      # [g, n, d]
            p = torch.softmax(((q @ k[h].t()) / math.sqrt(c["dim"])).masked_fill_(past, -math.inf), -1)
            total[b, h, :ctx[b]] += p.sum((0, 1))
            if v is not None:
                outs.append((p @ v[h]).squeeze(1))
        at += new[b]
    if c["op"] == "observe":
        return [total]
    return [torch.stack(outs).view(s["q"].shape), total]
