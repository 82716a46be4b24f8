"""Normed heads with rotary positions against their float64 definition on a GPU.

Tolerances, in units of u = 2^-24 (half a float32 step relative to the value):
* r = 1 / sqrt(mean + eps): the mean of squares is a sum of d positive terms; a thread adds at most 32 of them in a
  chain (a product's rounding goes into the fused add), then five shuffles, a division and eps: 40 u, of which the
  root takes half; rsqrtf itself 4 u (two steps): 24 u on r.
* normed and turned: two products and r 26 u on each normed element, a table entry 1 u, the products and the sum of the
  rotation 2 u: 30 u (|a| + |b|) of the pair's normed elements, then one rounding to the output's type.
* gradient: a turned dy is off by 4 u (|a| + |b|) of its pair; the sum of dy g x over a head adds 40 u of the sum of
  magnitudes, r^2 / d of it 50 u more; outside it r, the products and the difference 30 u of the two terms.
* gains: each term 34 u, and the chain of additions: a thread's rows, the groups of a CTA, the CTAs: below 200 at
  these sizes, so 240 u of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import weight_ops as W
from tests.helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from transformer_decoder_layer_llama_gb300 import api

U = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}     # (float32: within the terms above)
EPS = 1e-5
TINY = 2.0 ** -126

CASES = [  # tokens, heads, kv_heads, dim, rot
    (1, 1, 1, 64, 64), (7, 4, 2, 128, 128), (33, 5, 1, 128, 64), (3, 8, 8, 64, 10), (64, 32, 32, 128, 128), (5, 3, 2, 96, 32),
    (129, 64, 8, 128, 128), (2, 2, 0, 24, 8), (1025, 64, 8, 128, 32), (9, 0, 3, 256, 256), (4, 2, 1, 80, 2), (3, 1, 1, 1024, 512),
    (2, 3, 1, 512, 256), (1, 200, 3, 64, 48), (11, 4, 1, 16, 16), (3, 2, 2, 2, 2), (300, 16, 4, 96, 96)]


def setup(case, dtype, seed=0):
    T, H, Hk, d, rot = case
    g = torch.Generator().manual_seed(seed + T * 1000 + rot)
    qkv = (torch.randn(T, (H + 2 * Hk) * d + 8, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dtype).cuda()
    q = qkv[:, :H * d].view(T, H, d) if H else None
    k = qkv[:, H * d:(H + Hk) * d].view(T, Hk, d) if Hk else None
    gains = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    table = api.rope_table(api.make_rope_config(rot), 5000)
    freq, _ = C.inv_freq(rot)
    return g, qkv, q, k, gains, pos, table, freq


def pair_sum(x, rot, layout):
    """|a| + |b| of each element's pair; |x| behind the rotated part."""
    out, half = np.abs(x), rot // 2
    i0 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i1 = i0 + half if layout == "half" else i0 + 1
    s = np.abs(x[..., i0]) + np.abs(x[..., i1])
    out[..., i0] = out[..., i1] = s
    return out


def check_status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, layout, dtype):
    T, H, Hk, d, rot = case
    _, qkv, q, k, gains, pos, table, freq = setup(case, dtype)
    before, st = qkv.clone(), api.new_status()
    outs = api.norm_rope(q, k, *gains, pos.cuda(), table, eps=EPS, layout=layout, status=st)
    check_status(st)
    for x, gain, got in zip((q, k), gains, outs):
        if x is None:
            assert got is None
            continue
        xn, g = f64(x), f64(gain)
        ref = W.norm_rope(xn, g, pos.numpy(), freq, EPS, layout)
        n = xn / np.sqrt((xn * xn).mean(-1, keepdims=True) + EPS) * g
        assert got.is_contiguous() and got.dtype == dtype and got.shape == x.shape
        assert (np.abs(f64(got) - ref) <= 30 * U * pair_sum(n, rot, layout) + UNIT[dtype] * np.abs(ref) + TINY).all()
    assert torch.equal(qkv, before)
    # in place, through the views: the same bits, and nothing else of the merged rows changes
    again = api.norm_rope(q, k, *gains, pos.cuda(), table, eps=EPS, layout=layout, q_out=q, k_out=k, status=st)
    check_status(st)
    assert all(a is x for a, x in zip(again, (q, k)))
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, outs))
    assert torch.equal(qkv[:, (H + Hk) * d:], before[:, (H + Hk) * d:])


def gradient_bounds(dy, x, g, pos, freq, rot, layout):
    d = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    dn, mag = C.rope(dy, pos, freq, 1.0, layout, True), pair_sum(dy, rot, layout)
    dot = (np.abs(mag * g * x)).sum(-1, keepdims=True) * r * r / d
    bound = U * r * (4 * mag * np.abs(g) + 94 * np.abs(x) * dot + 30 * (np.abs(dn * g) + np.abs(x) * dot))
    return bound, 240 * U * (mag * np.abs(x) * r).sum((0, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", CASES)
def test_gradient(case, layout, dtype):
    T, H, Hk, d, rot = case
    gen, _, q, k, gains, pos, table, freq = setup(case, dtype)
    dq, dk = (None if x is None else torch.randn(x.shape, generator=gen).to(dtype).cuda() for x in (q, k))
    st = api.new_status()
    call = lambda **kw: api.norm_rope_backward(dq, dk, q, k, *gains, pos.cuda(), table, eps=EPS, layout=layout, status=st, **kw)  # noqa: E731
    outs = call()
    check_status(st)
    for x, dy, gain, dx, dg in zip((q, k), (dq, dk), gains, outs[:2], outs[2:]):
        if x is None:
            assert dx is None and dg is None
            continue
        xn, dn, g = f64(x), f64(dy), f64(gain)
        rx, rg = W.norm_rope_backward(dn, xn, g, pos.numpy(), freq, EPS, layout)
        bx, bg = gradient_bounds(dn, xn, g, pos.numpy(), freq, rot, layout)
        assert (np.abs(f64(dx) - rx) <= bx + UNIT[dtype] * np.abs(rx) + TINY).all()
        assert dg.dtype == torch.float32 and (np.abs(f64(dg) - rg) <= bg + TINY).all()
    # the same bits again, and over the gradients that came in
    again = call(workspace=torch.full((api.norm_rope_backward_workspace_size(d),), 255, dtype=torch.uint8, device="cuda"))
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, outs))
    over = call(q_grad=dq, k_grad=dk)
    check_status(st)
    assert all(a is None or torch.equal(a, b) for a, b in zip(over, outs))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_is_the_difference_quotient(layout):
    """float32: f(x + h) - f(x - h) over 2 h along a direction is <gradient, direction> but for h^2 and rounding."""
    case = (6, 3, 2, 64, 48)
    gen, _, q, k, gains, pos, table, _ = setup(case, torch.float32)
    dq, dk = (torch.randn(x.shape, generator=gen).cuda() for x in (q, k))
    grads = api.norm_rope_backward(dq, dk, q, k, *gains, pos.cuda(), table, eps=EPS, layout=layout)
    inputs = [q, k, *gains]
    for i, (x, grad) in enumerate(zip(inputs, grads)):
        step = torch.randn(x.shape, generator=gen).cuda() * (x.abs().mean(-1, keepdim=True) if i < 2 else 1.0)

        def value(h):
            t = list(inputs)
            t[i] = x + h * step
            out = api.norm_rope(*t, pos.cuda(), table, eps=EPS, layout=layout)
            return sum((f64(a) * f64(b)).sum() for a, b in zip(out, (dq, dk)))

        h = 2.0 ** -7
        want = (f64(grad) * f64(step)).sum()
        size = sum(np.abs(f64(b)).sum() for b in (dq, dk)) * 4          # |normed| stays below 4 in effect
        assert abs((value(h) - value(-h)) / (2 * h) - want) <= size * (h * h + 64 * U / h)


@pytest.mark.parametrize("case", [(5, 4, 2, 64, 64), (5, 4, 2, 66, 10)])
def test_bad_positions_are_left_out(case):
    T, H, Hk, d, rot = case
    gen, _, q, k, gains, _, table, freq = setup(case, torch.bfloat16)
    pos = torch.tensor([3, -1, 4999, 5000, 0], dtype=torch.int32)
    good = [0, 2, 4]
    dq, dk = (torch.randn(x.shape, generator=gen).bfloat16().cuda() for x in (q, k))
    st = api.new_status()
    outs = api.norm_rope(q, k, *gains, pos.cuda(), table, q_out=torch.full_like(dq, 7.0), k_out=torch.full_like(dk, 7.0), status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    st = api.new_status()
    grads = api.norm_rope_backward(dq, dk, q, k, *gains, pos.cuda(), table, q_grad=torch.full_like(dq, 7.0),
                                   k_grad=torch.full_like(dk, 7.0), status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    part = [t[good].contiguous() for t in (dq, dk, q, k)]
    ok = api.norm_rope(*part[2:], *gains, pos[good].cuda(), table)
    ok_grads = api.norm_rope_backward(*part, *gains, pos[good].cuda(), table)
    for a, b in zip(outs + grads[:2], ok + ok_grads[:2]):
        assert torch.equal(a[good], b) and (a[[1, 3]] == 7).all()
    for a, x, dy, gain, b in zip(grads[2:], part[2:], part[:2], gains, ok_grads[2:]):
        _, bg = gradient_bounds(f64(dy), f64(x), f64(gain), pos[good].numpy(), freq, rot, "half")
        assert (np.abs(f64(a) - f64(b)) <= 2 * bg + TINY).all()         # (other orders of the sum)


def test_zeros_large_values_and_no_tokens():
    d = 128
    table, pos, g = api.rope_table(api.make_rope_config(d), 16), torch.zeros(3, dtype=torch.int32).cuda(), torch.ones(d).cuda()
    x = torch.zeros(3, 2, d)
    x[1] = 2.0 ** 50                                             # squares of 2^100, their sum 2^107
    x[2] = 2.0 ** -90                                            # squares below float32's range: eps alone
    for dtype in (torch.bfloat16, torch.float32):
        y, _ = api.norm_rope(x.to(dtype).cuda(), None, g, None, pos, table, eps=2.0 ** -20)
        y = f64(y)
        assert (y[0] == 0).all() and np.allclose(y[1], 1.0, rtol=2.0 ** -8) and np.allclose(y[2], 2.0 ** -80, rtol=2.0 ** -8)
        dx, _, dg, _ = api.norm_rope_backward(torch.ones(3, 2, d).to(dtype).cuda(), None, x.to(dtype).cuda(), None, g, None, pos,
                                              table, eps=2.0 ** -20)
        assert np.isfinite(f64(dx)).all() and np.allclose(f64(dx)[0], 2.0 ** 10, rtol=2.0 ** -8)
        assert np.allclose(f64(dg), 2.0, rtol=2.0 ** -8)
        e = torch.empty(0, 2, d, dtype=dtype).cuda()
        out = api.norm_rope_backward(e, e, e, e, g, g, pos[:0], table)
        assert out[0].shape == e.shape and (out[2] == 0).all() and (out[3] == 0).all()
        assert api.norm_rope(e, None, g, None, pos[:0], table)[0].shape == e.shape


def test_unaligned_and_wide_rows_take_the_same_values():
    """Element-aligned views take the kernel for any shape: within the bounds of two evaluations."""
    T, H, d = 9, 3, 64
    _, _, q, _, gains, pos, table, freq = setup((T, H, 0, d, d), torch.bfloat16)
    wide = torch.zeros(T, H * d + 13, dtype=torch.bfloat16).cuda()
    view = wide[:, 5:5 + H * d].view(T, H, d)
    view.copy_(q)
    a, _ = api.norm_rope(q.contiguous(), None, gains[0], None, pos.cuda(), table)
    b, _ = api.norm_rope(view, None, gains[0], None, pos.cuda(), table, q_out=view)
    assert b is view and (wide[:, :5] == 0).all() and (wide[:, 5 + H * d:] == 0).all()
    ref = W.norm_rope(f64(q), f64(gains[0]), pos.numpy(), freq, 1e-5, "half")
    assert (np.abs(f64(a) - f64(b)) <= 2 * (2.0 ** -8 * np.abs(ref) + 2.0 ** -18)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case,pad", [((3001, 32, 8, 128, 128), 0), ((3001, 32, 8, 128, 64), 4), ((2500, 70, 3, 64, 32), 0), ((2500, 3, 40, 256, 64), 0),
                                      ((901, 5, 2, 128, 128), 4), ((901, 5, 2, 64, 64), 3),
                                      ((901, 5, 2, 128, 128), 2), ((700, 6, 2, 96, 36), 2), ((700, 6, 2, 256, 128), 2)])
def test_gradient_of_many_tokens(case, pad, layout, dtype):
    """Many turns of a CTA; rows on 16 bytes, on 8 and on an element's (pad: elements before and between rows).  A chain
    of a gain's sum: 3001 tokens x 40 heads over 600 CTAs, with the joins below 200."""
    T, H, Hk, d, rot = case
    gen, _, q, k, gains, pos, table, freq = setup(case, dtype, seed=5)

    def place(x):
        wide = torch.zeros(T, x.shape[1] * d + 8 + pad, dtype=dtype).cuda()
        view = wide[:, pad:pad + x.shape[1] * d].view(T, x.shape[1], d)
        view.copy_(x)
        return view

    q, k = place(q), place(k)
    dq, dk = (place(torch.randn(x.shape, generator=gen).to(dtype).cuda()) for x in (q, k))
    st = api.new_status()
    outs = api.norm_rope_backward(dq, dk, q, k, *gains, pos.cuda(), table, eps=EPS, layout=layout, status=st)
    check_status(st)
    for x, dy, gain, dx, dg in zip((q, k), (dq, dk), gains, outs[:2], outs[2:]):
        xn, dn, g = f64(x), f64(dy), f64(gain)
        rx, rg = W.norm_rope_backward(dn, xn, g, pos.numpy(), freq, EPS, layout)
        bx, bg = gradient_bounds(dn, xn, g, pos.numpy(), freq, rot, layout)
        assert (np.abs(f64(dx) - rx) <= bx + UNIT[dtype] * np.abs(rx) + TINY).all()
        assert (np.abs(f64(dg) - rg) <= bg + TINY).all()
    bad = pos.clone()
    bad[::7] = -1                                             # their rows stay as they were, the others do not change
    over = api.norm_rope_backward(dq, dk, q, k, *gains, bad.cuda(), table, eps=EPS, layout=layout, q_grad=dq.clone(), k_grad=dk.clone(), status=st)
    check_status(st, api.LL_DEV_BAD_POSITION)
    for got, dx, dy in zip(over[:2], outs[:2], (dq, dk)):
        assert torch.equal(got[::7], dy[::7])
        keep = torch.ones(T, dtype=torch.bool)
        keep[::7] = False
        assert torch.equal(got[keep.cuda()], dx[keep.cuda()])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("pad", [1, 2, 4, 6, 8])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 100), (128, 98), (256, 64), (66, 36), (1024, 16)])
def test_rows_on_any_element(d, rot, pad, layout, dtype):
    """Rows on one, two, four or eight elements, gains on one: what is loaded at a time goes by that."""
    T, H, Hk = 37, 3, 2
    _, _, q, k, gains, pos, table, freq = setup((T, H, Hk, d, rot), dtype)
    wide = torch.zeros(T, (H + Hk) * d + 2 * pad, dtype=dtype).cuda()
    views = [wide[:, pad:pad + H * d].view(T, H, d), wide[:, pad + H * d:pad + (H + Hk) * d].view(T, Hk, d)]
    moved = torch.zeros(2, 2 * d).cuda()
    for v, x in zip(views, (q, k)):
        v.copy_(x)
    odd = [moved[i, pad:pad + d].copy_(gain) for i, gain in enumerate(gains)]
    st = api.new_status()
    out = api.norm_rope(*views, *odd, pos.cuda(), table, eps=EPS, layout=layout, q_out=views[0], k_out=views[1], status=st)
    check_status(st)
    for x, gain, got in zip((q, k), gains, out):
        xn, g = f64(x), f64(gain)
        ref = W.norm_rope(xn, g, pos.numpy(), freq, EPS, layout)
        n = xn / np.sqrt((xn * xn).mean(-1, keepdims=True) + EPS) * g
        assert (np.abs(f64(got) - ref) <= 30 * U * pair_sum(n, rot, layout) + UNIT[dtype] * np.abs(ref) + TINY).all()
    assert (wide[:, :pad] == 0).all() and (wide[:, pad + (H + Hk) * d:] == 0).all()


def test_streams_and_graphs():
    case = (40, 8, 2, 128, 128)
    gen, _, q, k, gains, pos, table, _ = setup(case, torch.bfloat16)
    dq, dk = (torch.randn(x.shape, generator=gen).bfloat16().cuda() for x in (q, k))
    pos = pos.cuda()
    want = api.norm_rope(q, k, *gains, pos, table) + api.norm_rope_backward(dq, dk, q, k, *gains, pos, table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.norm_rope(q, k, *gains, pos, table, stream=side) + api.norm_rope_backward(dq, dk, q, k, *gains, pos, table, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(t) for t in want]
    st, ws = api.new_status(), torch.empty(api.norm_rope_backward_workspace_size(128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.norm_rope(q, k, *gains, pos, table, q_out=outs[0], k_out=outs[1], status=st)
        api.norm_rope_backward(dq, dk, q, k, *gains, pos, table, q_grad=outs[2], k_grad=outs[3], q_gain_grad=outs[4],
                               k_gain_grad=outs[5], workspace=ws, status=st)
    for scale in (1.0, 0.5):
        for x in (q, dq):
            x.mul_(scale)
        want = api.norm_rope(q, k, *gains, pos, table) + api.norm_rope_backward(dq, dk, q, k, *gains, pos, table)
        graph.replay()
        check_status(st)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_what_the_binding_refuses():
    """One thing wrong at a time, with all that a usual call has."""
    T, H, Hk, d = 6, 4, 2, 64
    ok = dict(q=torch.ones(T, H, d).bfloat16(), k=torch.ones(T, Hk, d).bfloat16(), q_gain=torch.ones(d), k_gain=torch.ones(d),
              positions=torch.zeros(T, dtype=torch.int32), table=torch.zeros(8, d // 2, 2), status=torch.zeros(1, dtype=torch.int32))
    ok = {n: t.cuda() for n, t in ok.items()}
    ws = torch.empty(api.norm_rope_backward_workspace_size(d), dtype=torch.uint8, device="cuda")
    wide = torch.ones(T, H, 2 * d).bfloat16().cuda()
    bad = [dict(q=ok["q"].half()), dict(k=ok["k"].float()), dict(q=ok["q"][0]), dict(k=ok["k"][:5]), dict(k=wide[..., :d // 2]), dict(q=wide[..., :d]),
           dict(q=wide[..., ::2]), dict(q=ok["q"].transpose(0, 1)), dict(q_gain=ok["q_gain"][:60]), dict(k_gain=ok["k_gain"].bfloat16()),
           dict(q_gain=torch.ones(2 * d).cuda()[::2]), dict(positions=ok["positions"].long()), dict(positions=ok["positions"][:5]),
           dict(positions=ok["positions"].cpu()), dict(table=ok["table"][..., 0]), dict(table=torch.zeros(8, d, 2).cuda()), dict(table=ok["table"].cpu()),
           dict(table=torch.zeros(8, d // 2, 4).cuda()[..., ::2]), dict(status=torch.zeros(1).cuda()), dict(status=ok["status"][:0]),
           dict(layout="quarter"), dict(q=ok["q"].clone().requires_grad_()), dict(k_gain=ok["k_gain"].clone().requires_grad_()), dict(q=None, k=None)]
    for change in bad:
        a = {**ok, **change}
        with pytest.raises((ValueError, TypeError)):
            api.norm_rope(**a)
        dq, dk = (torch.ones(T, n, d).bfloat16().cuda() for n in (H, Hk))
        with pytest.raises((ValueError, TypeError)):
            api.norm_rope_backward(dq, dk, workspace=ws, **a)
    dq, dk = torch.ones_like(ok["q"]), torch.ones_like(ok["k"])
    for change in (dict(dq=dq.float()), dict(dk=dk[:5]), dict(dq=wide[..., :d]), dict(dq=None), dict(dk=dk.cpu()), dict(workspace=ws.float()),
                   dict(workspace=ws.cpu())):
        with pytest.raises((ValueError, TypeError)):
            api.norm_rope_backward(**{**dict(dq=dq, dk=dk, workspace=ws), **ok, **change})
    with pytest.raises(api.LayerError):
        api.norm_rope_backward(dq, dk, workspace=ws[:64], **ok)
    with pytest.raises(api.LayerError):
        api.norm_rope(**ok, eps=0.0)
    check_status(ok["status"])
    with torch.no_grad():                                     # a leaf that wants a gradient, where none is recorded
        api.norm_rope(**{**ok, "q": ok["q"].clone().requires_grad_()})
    one = {n: t if n in ("q_gain", "k_gain", "table", "status") else t[:1] for n, t in ok.items()}
    assert torch.equal(api.norm_rope(**one)[0], api.norm_rope(**ok)[0][:1])


# Q alone with so many heads that the last turn of a token has groups without one (the smallest such sizes of their forms:
# float32 or loads of two elements with a head in 32 and in 16 lanes, whole BF16 columns likewise), and K alone.
ALONE = [(3, 127, 0, 256, 256), (2, 541, 0, 128, 100), (2, 295, 0, 256, 256), (1, 1261, 0, 128, 128), (3, 0, 127, 256, 256),
         (2, 0, 541, 128, 98), (1, 1400, 0, 80, 50), (2, 126, 1, 256, 10), (2, 127, 1, 256, 256), (2, 300, 0, 33, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", ALONE)
def test_many_heads_of_one_kind(case, layout, dtype):
    test_forward(case, layout, dtype)
    test_gradient(case, layout, dtype)
