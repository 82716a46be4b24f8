"""Normed heads with rotary positions, without a GPU: the oracle's pins and what the library refuses."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from oracle import weight_ops as W
from transformer_decoder_layer_llama_gb300 import api

FAKE = 1 << 20                          # an aligned address that nothing reads on the host
NULL = None
OK, INVALID, UNSUPPORTED, WORKSPACE = range(4)


def test_the_definition_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])                  # mean of squares 25 / 4
    freq = np.array([0.0, 0.0])                             # no turn
    y = W.norm_rope(x, np.array([1.0, 2.0, 3.0, 4.0]), np.array([5]), freq, 0.0, "half")
    assert np.allclose(y, [[[1.2, 3.2, 0.0, 0.0]]])
    y = W.norm_rope(x, np.ones(4), np.array([1]), np.array([np.pi / 2, 0.0]), 0.0, "half")      # pair (0, 2) by 90 degrees
    assert np.allclose(y, [[[0.0, 1.6, 1.2, 0.0]]])
    y = W.norm_rope(x, np.ones(4), np.array([1]), np.array([np.pi / 2]), 0.0, "interleaved")    # pair (0, 1)
    assert np.allclose(y, [[[-1.6, 1.2, 0.0, 0.0]]])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_gradient_is_the_difference_quotient(layout):
    rng = np.random.default_rng(2)
    T, H, d, rot, eps = 3, 2, 10, 6, 0.1
    x, dy, g = rng.normal(size=(T, H, d)), rng.normal(size=(T, H, d)), 1 + 0.3 * rng.normal(size=d)
    pos, freq = np.array([0, 7, 100]), rng.uniform(0.01, 1.0, rot // 2)
    f = lambda x, g: (dy * W.norm_rope(x, g, pos, freq, eps, layout)).sum()  # noqa: E731
    dx, dg = W.norm_rope_backward(dy, x, g, pos, freq, eps, layout)
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, g) - f(x - e, g)) / (2 * h) - dx[i]) < 1e-8
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(x, g + e) - f(x, g - e)) / (2 * h) - dg[i]) < 1e-8


def heads(data=FAKE, stride=512, n=4):
    return api.ll_head_rows(data, stride, n)


FORWARD = dict(q=heads(), k=heads(FAKE + 256 * 2, 512, 2), dtype=0, q_gain=FAKE, k_gain=FAKE, eps=1e-5, positions=FAKE, tokens=8,
               head_dim=64, rotary_dim=64, layout=0, table=FAKE, max_position=16, q_out=heads(2 * FAKE, 256, 4),
               k_out=heads(3 * FAKE, 128, 2), status=FAKE)
BACKWARD = dict(dq=heads(4 * FAKE, 256, 4), dk=heads(5 * FAKE, 128, 2), q=heads(), k=heads(FAKE + 256 * 2, 512, 2), dtype=0,
                q_gain=FAKE, k_gain=FAKE, eps=1e-5, positions=FAKE, tokens=8, head_dim=64, rotary_dim=64, layout=0, table=FAKE,
                max_position=16, q_grad=heads(2 * FAKE, 256, 4), k_grad=heads(3 * FAKE, 128, 2), dg_q=6 * FAKE, dg_k=7 * FAKE,
                ws=8 * FAKE, ws_bytes=1 << 30, status=FAKE)

SHARED = [(dict(dtype=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
          (dict(eps=float("inf")), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED),
          (dict(head_dim=0), INVALID), (dict(rotary_dim=0), INVALID), (dict(rotary_dim=3), INVALID), (dict(rotary_dim=66), INVALID),
          (dict(layout=2), INVALID), (dict(table=0), INVALID), (dict(table=FAKE + 8), INVALID), (dict(max_position=0), INVALID),
          (dict(status=0), INVALID), (dict(positions=0), INVALID), (dict(q_gain=0), INVALID), (dict(k_gain=0), INVALID),
          (dict(q_gain=FAKE + 2), INVALID), (dict(q=heads(0)), INVALID), (dict(q=heads(FAKE + 1)), INVALID),
          (dict(q=heads(stride=255)), INVALID), (dict(q=heads(stride=(1 << 34) + 1)), UNSUPPORTED), (dict(q=heads(n=-1)), INVALID),
          (dict(q=heads(n=5)), INVALID)]        # other head counts than its output


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(q_out=heads(FAKE, 256, 4)), INVALID),                       # over its input, another stride
    (dict(q_out=heads(2 * FAKE, 256, 3)), INVALID), (dict(k_out=heads(2 * FAKE + 512, 128, 2)), INVALID),
    (dict(q_out=heads(FAKE + 256 * 2, 512, 4)), INVALID),             # over k
    (dict(head_dim=1026, rotary_dim=2, q=heads(stride=8192), q_out=heads(2 * FAKE, 8192)), UNSUPPORTED)])
def test_forward_refusals(bad, code):
    assert api.lib.ll_norm_rope(*{**FORWARD, **bad}.values(), NULL) == code


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(dq=heads(0, 256, 4)), INVALID), (dict(dq=heads(4 * FAKE, 256, 3)), INVALID), (dict(q_grad=heads(2 * FAKE, 256, 3)), INVALID),
    (dict(q_grad=heads()), INVALID),                                   # over q: it is still read
    (dict(q_grad=heads(4 * FAKE, 512, 4)), INVALID),                   # over dq, another stride
    (dict(k_grad=heads(2 * FAKE, 128, 2)), INVALID), (dict(dg_q=0), INVALID), (dict(dg_k=6 * FAKE + 128), INVALID),
    (dict(dg_q=FAKE), INVALID),                                        # over a gain
    (dict(ws=0), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=8 * FAKE + 8), WORKSPACE)])
def test_backward_refusals(bad, code):
    assert api.lib.ll_norm_rope_backward(*{**BACKWARD, **bad}.values(), NULL) == code


def test_no_tokens_is_no_work():
    assert api.lib.ll_norm_rope(*{**FORWARD, "tokens": 0}.values(), NULL) == OK
    assert api.lib.ll_norm_rope_backward_workspace_size(0) == api.lib.ll_norm_rope_backward_workspace_size(1025) == 0
    assert api.norm_rope_backward_workspace_size(128) >= 2 * 152 * 2 * 128 * 4


def test_binding_refusals():
    x, g, pos, tab = torch.zeros(2, 4, 64), torch.ones(64), torch.zeros(2, dtype=torch.int32), torch.zeros(8, 32, 2)
    for q, k, gq in ((x.clone().requires_grad_(), None, g), (x, None, g.clone().requires_grad_())):
        with pytest.raises(ValueError, match="autograd"):
            api.norm_rope(q, k, gq, None, pos, tab)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            api.norm_rope(q, k, gq, None, pos, tab)
    with pytest.raises(ValueError, match="both None"):
        api.norm_rope(None, None, g, g, pos, tab)
    with pytest.raises(TypeError):
        api.norm_rope(x.half(), None, g, None, pos, tab)
    with pytest.raises(ValueError, match="layout"):
        api.norm_rope(x, None, g, None, pos, tab, layout="quarter")
    status, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        api.norm_rope(x, x, g, g, pos, tab, status=status)
    with pytest.raises(ValueError, match="GPU"):
        api.norm_rope_backward(x, x, x, x, g, g, pos, tab, workspace=ws, status=status)
