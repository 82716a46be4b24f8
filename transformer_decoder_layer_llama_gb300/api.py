"""ctypes binding of libllamalayer.so (include/llama_layer.h), names as in the C ABI.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, then their device pointers go to the library; every step of the
layer runs in the library's CUDA kernels.  Importing this module loads the
library and fails loudly if it has not been built (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

LL_OK = 0
LL_ERR_INVALID_ARG = 1
LL_ERR_UNSUPPORTED = 2
LL_ERR_WORKSPACE = 3
LL_ERR_CUDA = 4

LL_MODE_FUSED = 0
LL_MODE_STEP_BY_STEP = 1

LL_BF16 = 0
LL_F32 = 1

LL_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
LL_ROPE_FORWARD = 0
LL_ROPE_BACKWARD = 1
LL_ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "banded": 3, "yarn": 4}

LL_DEV_BAD_BLOCK = 1
LL_DEV_BAD_SLOT = 2
LL_DEV_BAD_POSITION = 4
LL_DEV_TIMEOUT = 8

EXPORTED = [
    "ll_strerror", "ll_last_error", "ll_packed_weights_size", "ll_pack_weights", "ll_workspace_size",
    "ll_layer_prefill", "ll_layer_decode_step", "ll_reshape_and_cache",
    "ll_attention_workspace_size", "ll_paged_attention_decode", "ll_linear_workspace_size",
    "ll_linear", "ll_device_sm_count", "ll_trace_begin", "ll_trace_end", "ll_trace_elapsed_ms",
    "ll_trace_name", "ll_paged_attention_decode_noalloc", "ll_selftest_bounded_wait",
    "ll_workspace_checkpoints", "ll_reshape_and_cache_q8", "ll_paged_attention_decode_q8",
    "ll_layer_decode_step_q8", "ll_workspace_size_mode", "ll_workspace_step_checkpoints",
    "ll_layer_prefill_mode", "ll_layer_decode_step_mode", "ll_set_prefill_attention_ctas",
    "ll_rope_table_size", "ll_rope_table", "ll_pack_rope", "ll_rope", "ll_append_to_cache_f8",
    "ll_attention_decode_f8_workspace_size", "ll_paged_attention_decode_f8",
    "ll_attention_prefill_f8_workspace_size", "ll_paged_attention_prefill_f8", "ll_copy_blocks",
    "ll_compact_blocks", "ll_workspace_size_f8", "ll_layer_prefill_f8", "ll_layer_decode_step_f8",
    "ll_norm_rope", "ll_norm_rope_backward_workspace_size", "ll_norm_rope_backward",
    "ll_attention_decode_weights_workspace_size", "ll_paged_attention_decode_weights",
    "ll_paged_attention_decode_weights_q8", "ll_evict_rows", "ll_attention_weights_workspace_size",
    "ll_paged_attention_weights", "ll_workspace_size_weights", "ll_layer_decode_step_weights",
    "ll_layer_decode_step_weights_q8",
]


class ll_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("intermediate", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("max_position", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float)]


class ll_weights(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("w_o", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("g_attn", ctypes.c_void_p), ("g_ffn", ctypes.c_void_p)]


class ll_kv_pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


class ll_kv_pool_q8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


class ll_rope_config(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("theta", ctypes.c_float),
                ("factor", ctypes.c_float), ("original_max_position", ctypes.c_int32),
                ("low_turns", ctypes.c_float), ("high_turns", ctypes.c_float),
                ("attention_factor", ctypes.c_float)]


class ll_head_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("n_heads", ctypes.c_int32)]


class ll_row_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


class ll_kv_pool_f8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


class ll_block_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_bytes", ctypes.c_int64)]


class ll_checkpoints(ctypes.Structure):
    _fields_ = [("x_hat", ctypes.c_size_t), ("q", ctypes.c_size_t), ("o", ctypes.c_size_t),
                ("h", ctypes.c_size_t), ("h_hat", ctypes.c_size_t), ("a", ctypes.c_size_t)]


class ll_step_checkpoints(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("qkv", "k", "v", "slots", "o_proj", "gate_up", "down")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, S, I32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    cfgp = ctypes.POINTER(ll_config)
    poolp = ctypes.POINTER(ll_kv_pool)
    poolf8 = ctypes.POINTER(ll_kv_pool_f8)
    ropep = ctypes.POINTER(ll_rope_config)
    I64, F32 = ctypes.c_int64, ctypes.c_float
    headp = ctypes.POINTER(ll_head_rows)
    sig = {
        "ll_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "ll_last_error": (ctypes.c_char_p, []),
        "ll_packed_weights_size": (S, [cfgp]),
        "ll_pack_weights": (ctypes.c_int, [cfgp, ctypes.POINTER(ll_weights), P, S, P]),
        "ll_workspace_size": (S, [cfgp, I32, I32]),
        "ll_layer_prefill": (ctypes.c_int, [cfgp, P, P, P, I32, I32, poolp, P, I32, P, P, S, P, P]),
        "ll_layer_decode_step": (ctypes.c_int, [cfgp, P, P, poolp, P, I32, P, I32, P, P, S, P, P]),
        "ll_reshape_and_cache": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, poolp, P, P]),
        "ll_attention_workspace_size": (S, [I32, I32, I32, I32, I32]),
        "ll_paged_attention_decode": (ctypes.c_int, [P, poolp, P, I32, P, I32, I32, I32, I32, I32,
                                                     ctypes.c_float, P, P, S, P, P]),
        "ll_paged_attention_decode_noalloc": (ctypes.c_int, [P, poolp, P, I32, P, I32, I32, I32, I32,
                                                             I32, ctypes.c_float, P, P, P]),
        "ll_linear_workspace_size": (S, [I32, I32, I32]),
        "ll_linear": (ctypes.c_int, [P, P, P, I32, I32, I32, P, S, P, P]),
        "ll_device_sm_count": (ctypes.c_int, []),
        "ll_set_prefill_attention_ctas": (ctypes.c_int, [I32]),
        "ll_trace_begin": (ctypes.c_int, [I32]),
        "ll_trace_end": (I32, []),
        "ll_trace_elapsed_ms": (ctypes.c_float, [I32]),
        "ll_trace_name": (ctypes.c_char_p, [I32]),
        "ll_selftest_bounded_wait": (ctypes.c_int, [I32, P, P, P]),
        "ll_workspace_checkpoints": (ctypes.c_int, [cfgp, I32, I32, ctypes.POINTER(ll_checkpoints)]),
        "ll_reshape_and_cache_q8": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, ctypes.POINTER(ll_kv_pool_q8),
                                                   P, P]),
        "ll_paged_attention_decode_q8": (ctypes.c_int, [P, ctypes.POINTER(ll_kv_pool_q8), P, I32, P, I32, I32, I32,
                                                        I32, I32, ctypes.c_float, P, P, S, P, P]),
        "ll_layer_decode_step_q8": (ctypes.c_int, [cfgp, P, P, ctypes.POINTER(ll_kv_pool_q8), P, I32, P, I32, P, P,
                                                   S, P, P]),
        "ll_workspace_size_mode": (S, [cfgp, I32, I32, I32]),
        "ll_workspace_step_checkpoints": (ctypes.c_int, [cfgp, I32, I32, ctypes.POINTER(ll_step_checkpoints)]),
        "ll_layer_prefill_mode": (ctypes.c_int, [cfgp, P, P, P, I32, I32, poolp, P, I32, P, P, S, P, I32, P]),
        "ll_layer_decode_step_mode": (ctypes.c_int, [cfgp, P, P, poolp, P, I32, P, I32, P, P, S, P, I32, P]),
        "ll_rope_table_size": (S, [ropep, I32]),
        "ll_rope_table": (ctypes.c_int, [ropep, I32, P, S, P]),
        "ll_pack_rope": (ctypes.c_int, [cfgp, ropep, P, S, P]),
        "ll_rope": (ctypes.c_int, [P, P, I32, P, I32, I32, I32, I32, I32, I32, I32, I64, I64, P, I32, P, P, I64, I64,
                                   P, P]),
        "ll_norm_rope": (ctypes.c_int, [headp, headp, I32, P, P, F32, P, I32, I32, I32, I32, P, I32, headp, headp, P, P]),
        "ll_norm_rope_backward_workspace_size": (S, [I32]),
        "ll_norm_rope_backward": (ctypes.c_int, [headp, headp, headp, headp, I32, P, P, F32, P, I32, I32, I32, I32, P, I32,
                                                 headp, headp, P, P, P, S, P, P]),
        "ll_attention_decode_weights_workspace_size": (S, [I32, I32, I32, I32, I32, I32]),
        "ll_paged_attention_decode_weights": (ctypes.c_int, [P, poolp, P, I32, P, I32, I32, I32, I32, I32, F32, P, I32, P, P,
                                                             S, P, P]),
        "ll_paged_attention_decode_weights_q8": (ctypes.c_int, [P, ctypes.POINTER(ll_kv_pool_q8), P, I32, P, I32, I32, I32,
                                                                I32, I32, F32, P, I32, P, P, S, P, P]),
        "ll_attention_weights_workspace_size": (S, [I32, I32, I32, I32, I32, I32, I32, I32]),
        "ll_paged_attention_weights": (ctypes.c_int, [P, P, I32, P, I32, P, I32, P, I32, I32, I32, I32, I32, I32, F32, P, I32, P,
                                                      S, P, P]),
        "ll_workspace_size_weights": (S, [cfgp, I32, I32]),
        "ll_layer_decode_step_weights": (ctypes.c_int, [cfgp, P, P, poolp, P, I32, P, P, I32, P, I32, P, P, S, P, P]),
        "ll_layer_decode_step_weights_q8": (ctypes.c_int, [cfgp, P, P, ctypes.POINTER(ll_kv_pool_q8), P, I32, P, P, I32, P, I32,
                                                           P, P, S, P, P]),
        "ll_evict_rows": (ctypes.c_int, [ctypes.POINTER(ll_row_tensor), I32, I32, I32, I32, P, I32, P, I32, P, I32, P, I32, I32,
                                         I32, P, P, P, P, P]),
        "ll_append_to_cache_f8": (ctypes.c_int, [P, P, I64, I64, P, I32, P, I32, I32, I32, I32, I32, poolf8, P, I32,
                                                 P, P]),
        "ll_attention_decode_f8_workspace_size": (S, [I32, I32, I32, I32]),
        "ll_paged_attention_decode_f8": (ctypes.c_int, [P, poolf8, P, I32, P, I32, I32, I32, I32, I32,
                                                        ctypes.c_float, P, P, S, P, P]),
        "ll_attention_prefill_f8_workspace_size": (S, [I32, I32, I32, I32, I32, I32]),
        "ll_paged_attention_prefill_f8": (ctypes.c_int, [P, P, I32, poolf8, P, I32, P, I32, I32, I32, I32, I32, I32,
                                                         ctypes.c_float, P, P, S, P, P]),
        "ll_workspace_size_f8": (S, [cfgp, I32, I32]),
        "ll_layer_prefill_f8": (ctypes.c_int, [cfgp, P, P, P, I32, I32, poolf8, P, I32, P, P, S, P, P]),
        "ll_layer_decode_step_f8": (ctypes.c_int, [cfgp, P, P, poolf8, P, I32, P, I32, P, P, S, P, P]),
        "ll_copy_blocks": (ctypes.c_int, [ctypes.POINTER(ll_block_tensor), I32, I32, P, I32, P, P, P]),
        "ll_compact_blocks": (ctypes.c_int, [P, I32, I32, I32, P, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class LayerError(RuntimeError):
    def __init__(self, name, code):
        detail = lib.ll_last_error().decode()
        super().__init__(f"{name}: {lib.ll_strerror(code).decode()} (code {code})"
                         + (f" -- {detail}" if detail else ""))
        self.code = code


def _check(name, rc):
    if rc != LL_OK:
        raise LayerError(name, rc)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_Tensor = torch.Tensor


def _need(t, name, dtype, device=True, shape=None):
    # (what holds in nearly every call first: the checks of a call of few tokens take as long as its kernels)
    if isinstance(t, _Tensor) and t.dtype is dtype and t.is_contiguous() and (t.is_cuda or not device) and \
            (shape is None or t.shape == shape):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def make_config(dims, max_position: int) -> ll_config:
    """ll_config from any object with the layer's dimension attributes."""
    return ll_config(dims.hidden, dims.n_heads, dims.n_kv_heads, dims.head_dim, dims.intermediate,
                     dims.block_size, int(max_position), float(dims.rms_eps), float(dims.rope_theta))


def new_status(device=None):
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def packed_weights_size(cfg: ll_config) -> int:
    return lib.ll_packed_weights_size(ctypes.byref(cfg))


def pack_weights(cfg: ll_config, W: dict, stream=None) -> torch.Tensor:
    """Packs canonical weights (dict of CUDA tensors, see include/llama_layer.h) into a new
    uint8 CUDA buffer and returns it."""
    H, I, d = cfg.hidden, cfg.intermediate, cfg.head_dim
    _need(W["w_qkv"], "w_qkv", torch.bfloat16, shape=((cfg.n_heads + 2 * cfg.n_kv_heads) * d, H))
    _need(W["w_o"], "w_o", torch.bfloat16, shape=(H, cfg.n_heads * d))
    _need(W["w_gate"], "w_gate", torch.bfloat16, shape=(I, H))
    _need(W["w_up"], "w_up", torch.bfloat16, shape=(I, H))
    _need(W["w_down"], "w_down", torch.bfloat16, shape=(H, I))
    _need(W["g_attn"], "g_attn", torch.float32, shape=(H,))
    _need(W["g_ffn"], "g_ffn", torch.float32, shape=(H,))
    n = packed_weights_size(cfg)
    if n == 0:
        raise LayerError("ll_packed_weights_size", LL_ERR_UNSUPPORTED)
    packed = torch.empty(n, dtype=torch.uint8, device=W["w_qkv"].device)
    w = ll_weights(W["w_qkv"].data_ptr(), W["w_o"].data_ptr(), W["w_gate"].data_ptr(),
                   W["w_up"].data_ptr(), W["w_down"].data_ptr(), W["g_attn"].data_ptr(),
                   W["g_ffn"].data_ptr())
    _check("ll_pack_weights", lib.ll_pack_weights(ctypes.byref(cfg), ctypes.byref(w), _ptr(packed),
                                                  n, _stream(stream)))
    return packed


def workspace_size(cfg: ll_config, max_tokens: int, max_blocks: int, mode: int = LL_MODE_FUSED) -> int:
    if mode == LL_MODE_FUSED:
        return lib.ll_workspace_size(ctypes.byref(cfg), int(max_tokens), int(max_blocks))
    return lib.ll_workspace_size_mode(ctypes.byref(cfg), int(max_tokens), int(max_blocks), int(mode))


def new_workspace(cfg, max_tokens, max_blocks, device=None, mode=LL_MODE_FUSED):
    n = workspace_size(cfg, max_tokens, max_blocks, mode)
    if n == 0:
        raise LayerError("ll_workspace_size", LL_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def checkpoints(cfg: ll_config, workspace: torch.Tensor, max_tokens: int, max_blocks: int, tokens: int) -> dict:
    """Views into `workspace` (allocated by new_workspace(cfg, max_tokens, max_blocks)) of the
    intermediates the last layer call over `tokens` tokens left there: x_hat, q, o, h_hat, a
    (BF16) and h (float32), each [tokens, features].  Read them after the call has finished
    on its stream; the next call on the workspace overwrites them."""
    out = ll_checkpoints()
    rc = lib.ll_workspace_checkpoints(ctypes.byref(cfg), int(max_tokens), int(max_blocks), ctypes.byref(out))
    if rc != 0:
        raise LayerError("ll_workspace_checkpoints", rc)
    if not 0 < tokens <= max_tokens:
        raise ValueError("tokens must be in 1..max_tokens")
    nq = cfg.n_heads * cfg.head_dim
    shapes = {"x_hat": (cfg.hidden, torch.bfloat16), "q": (nq, torch.bfloat16), "o": (nq, torch.bfloat16),
              "h": (cfg.hidden, torch.float32), "h_hat": (cfg.hidden, torch.bfloat16),
              "a": (cfg.intermediate, torch.bfloat16)}
    views = {}
    for name, (width, dt) in shapes.items():
        off = getattr(out, name)
        nbytes = tokens * width * torch.finfo(dt).bits // 8
        views[name] = workspace[off:off + nbytes].view(dt).view(tokens, width)
    return views


def step_checkpoints(cfg: ll_config, workspace: torch.Tensor, max_tokens: int, max_blocks: int,
                     tokens: int) -> dict:
    """Views into a step-by-step workspace (new_workspace(..., mode=LL_MODE_STEP_BY_STEP)) of
    the intermediates that mode adds, after a call over `tokens` tokens: qkv (float32, packed
    column order), k, v (BF16), slots (int32), o_proj, gate_up (interleaved), down (float32)."""
    out = ll_step_checkpoints()
    rc = lib.ll_workspace_step_checkpoints(ctypes.byref(cfg), int(max_tokens), int(max_blocks), ctypes.byref(out))
    if rc != 0:
        raise LayerError("ll_workspace_step_checkpoints", rc)
    if not 0 < tokens <= max_tokens:
        raise ValueError("tokens must be in 1..max_tokens")
    nqkv = (cfg.n_heads + 2 * cfg.n_kv_heads) * cfg.head_dim
    nkv = cfg.n_kv_heads * cfg.head_dim
    shapes = {"qkv": ((nqkv,), torch.float32), "k": ((nkv,), torch.bfloat16), "v": ((nkv,), torch.bfloat16),
              "slots": ((), torch.int32), "o_proj": ((cfg.hidden,), torch.float32),
              "gate_up": ((2 * cfg.intermediate,), torch.float32), "down": ((cfg.hidden,), torch.float32)}
    views = {}
    for name, (width, dt) in shapes.items():
        off = getattr(out, name)
        count = tokens * (width[0] if width else 1)
        nbytes = count * (torch.finfo(dt).bits if dt.is_floating_point else torch.iinfo(dt).bits) // 8
        views[name] = workspace[off:off + nbytes].view(dt).view(tokens, *width)
    return views


def _pool(k_pool, v_pool):
    _need(k_pool, "k_pool", torch.bfloat16)
    _need(v_pool, "v_pool", torch.bfloat16)
    if k_pool.shape != v_pool.shape or k_pool.dim() != 4:
        raise ValueError("k_pool and v_pool must both be [num_blocks, n_kv_heads, block_size, head_dim]")
    return ll_kv_pool(k_pool.data_ptr(), v_pool.data_ptr(), k_pool.shape[0])


def layer_prefill(cfg, packed, x, positions, batch, seq_len, k_pool, v_pool, block_table,
                  y=None, workspace=None, status=None, stream=None, mode=LL_MODE_FUSED):
    """ll_layer_prefill (ll_layer_prefill_mode for another mode).  Returns y (BF16
    [batch*seq_len, hidden])."""
    T = int(batch) * int(seq_len)
    _need(x, "x", torch.bfloat16, shape=(T, cfg.hidden))
    _need(positions, "positions", torch.int32, shape=(T,))
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] < batch:
        raise ValueError("block_table must be [batch, max_blocks]")
    pool = _pool(k_pool, v_pool)
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = new_workspace(cfg, T, block_table.shape[1], x.device, mode)
    if status is None:
        status = new_status(x.device)
    args = (ctypes.byref(cfg), _ptr(packed), _ptr(x), _ptr(positions), int(batch), int(seq_len),
            ctypes.byref(pool), _ptr(block_table), block_table.shape[1], _ptr(y), _ptr(workspace),
            workspace.numel(), _ptr(status))
    if mode == LL_MODE_FUSED:
        _check("ll_layer_prefill", lib.ll_layer_prefill(*args, _stream(stream)))
    else:
        _check("ll_layer_prefill_mode", lib.ll_layer_prefill_mode(*args, int(mode), _stream(stream)))
    return y


def layer_decode_step(cfg, packed, x, k_pool, v_pool, block_table, context_lens, y=None,
                      workspace=None, status=None, stream=None, mode=LL_MODE_FUSED):
    """ll_layer_decode_step (ll_layer_decode_step_mode for another mode).  Returns y (BF16
    [batch, hidden])."""
    B = x.shape[0]
    _need(x, "x", torch.bfloat16, shape=(B, cfg.hidden))
    _need(context_lens, "context_lens", torch.int32, shape=(B,))
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] < B:
        raise ValueError("block_table must be [batch, max_blocks]")
    pool = _pool(k_pool, v_pool)
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = new_workspace(cfg, B, block_table.shape[1], x.device, mode)
    if status is None:
        status = new_status(x.device)
    args = (ctypes.byref(cfg), _ptr(packed), _ptr(x), ctypes.byref(pool), _ptr(block_table),
            block_table.shape[1], _ptr(context_lens), B, _ptr(y), _ptr(workspace), workspace.numel(),
            _ptr(status))
    if mode == LL_MODE_FUSED:
        _check("ll_layer_decode_step", lib.ll_layer_decode_step(*args, _stream(stream)))
    else:
        _check("ll_layer_decode_step_mode", lib.ll_layer_decode_step_mode(*args, int(mode), _stream(stream)))
    return y


def layer_decode_step_q8(cfg, packed, x, pool, block_table, context_lens, y=None, workspace=None, status=None,
                         stream=None):
    """ll_layer_decode_step_q8 over an INT8 pool (PoolQ8).  Returns y (BF16 [batch, hidden])."""
    B = x.shape[0]
    _need(x, "x", torch.bfloat16, shape=(B, cfg.hidden))
    _need(context_lens, "context_lens", torch.int32, shape=(B,))
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] < B:
        raise ValueError("block_table must be [batch, max_blocks]")
    cp = pool.c()
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = new_workspace(cfg, B, block_table.shape[1], x.device)
    if status is None:
        status = new_status(x.device)
    _check("ll_layer_decode_step_q8", lib.ll_layer_decode_step_q8(
        ctypes.byref(cfg), _ptr(packed), _ptr(x), ctypes.byref(cp), _ptr(block_table), block_table.shape[1],
        _ptr(context_lens), B, _ptr(y), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return y


def reshape_and_cache(k, v, slot_mapping, k_pool, v_pool, status=None, stream=None):
    """ll_reshape_and_cache: k, v BF16 [tokens, n_kv_heads, head_dim]."""
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16, shape=tuple(k.shape))
    T, Hkv, d = k.shape
    _need(slot_mapping, "slot_mapping", torch.int32, shape=(T,))
    pool = _pool(k_pool, v_pool)
    if status is None:
        status = new_status(k.device)
    _check("ll_reshape_and_cache", lib.ll_reshape_and_cache(
        _ptr(k), _ptr(v), _ptr(slot_mapping), T, Hkv, d, k_pool.shape[2], ctypes.byref(pool),
        _ptr(status), _stream(stream)))
    return status


class PoolQ8:
    """An INT8 KV pool on the GPU: codes k, v int8 [num_blocks, n_kv_heads, block_size,
    head_dim] and float32 scales k_scale, v_scale [num_blocks, n_kv_heads, block_size]."""

    def __init__(self, k, v, k_scale, v_scale):
        _need(k, "k codes", torch.int8)
        _need(v, "v codes", torch.int8, shape=tuple(k.shape))
        _need(k_scale, "k_scale", torch.float32, shape=tuple(k.shape[:3]))
        _need(v_scale, "v_scale", torch.float32, shape=tuple(k.shape[:3]))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @classmethod
    def empty(cls, num_blocks, n_kv_heads, block_size, head_dim, device="cuda"):
        shape = (num_blocks, n_kv_heads, block_size, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:3], dtype=torch.float32, device=device),
                   torch.zeros(shape[:3], dtype=torch.float32, device=device))

    @property
    def block_size(self):
        return self.k.shape[2]

    def c(self):
        return ll_kv_pool_q8(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                             self.v_scale.data_ptr(), self.k.shape[0])


def reshape_and_cache_q8(k, v, slot_mapping, pool: PoolQ8, status=None, stream=None):
    """ll_reshape_and_cache_q8: k, v BF16 [tokens, n_kv_heads, head_dim] quantised into pool."""
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16, shape=tuple(k.shape))
    T, Hkv, d = k.shape
    _need(slot_mapping, "slot_mapping", torch.int32, shape=(T,))
    cp = pool.c()
    if status is None:
        status = new_status(k.device)
    _check("ll_reshape_and_cache_q8", lib.ll_reshape_and_cache_q8(
        _ptr(k), _ptr(v), _ptr(slot_mapping), T, Hkv, d, pool.block_size, ctypes.byref(cp),
        _ptr(status), _stream(stream)))
    return status


def paged_attention_decode_q8(q, pool: PoolQ8, block_table, context_lens, scale, out=None, workspace=None,
                              status=None, stream=None):
    """ll_paged_attention_decode_q8: q BF16 [batch, n_heads, 128] over an INT8 pool."""
    _need(q, "q", torch.bfloat16)
    B, Hq, d = q.shape
    _need(block_table, "block_table", torch.int32)
    _need(context_lens, "context_lens", torch.int32, shape=(B,))
    Hkv, bs = pool.k.shape[1], pool.block_size
    mb = block_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.empty(max(attention_workspace_size(B, Hq, d, mb, bs), 16), dtype=torch.uint8,
                                device=q.device)
    if status is None:
        status = new_status(q.device)
    cp = pool.c()
    _check("ll_paged_attention_decode_q8", lib.ll_paged_attention_decode_q8(
        _ptr(q), ctypes.byref(cp), _ptr(block_table), mb, _ptr(context_lens), B, Hq, Hkv, d, bs,
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return out


def attention_workspace_size(batch, n_heads, head_dim, max_blocks, block_size):
    return lib.ll_attention_workspace_size(batch, n_heads, head_dim, max_blocks, block_size)


def paged_attention_decode(q, k_pool, v_pool, block_table, context_lens, scale, out=None,
                           workspace=None, status=None, stream=None):
    """ll_paged_attention_decode: q BF16 [batch, n_heads, head_dim]."""
    _need(q, "q", torch.bfloat16)
    B, Hq, d = q.shape
    _need(block_table, "block_table", torch.int32)
    _need(context_lens, "context_lens", torch.int32, shape=(B,))
    pool = _pool(k_pool, v_pool)
    bs = k_pool.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        n = attention_workspace_size(B, Hq, d, block_table.shape[1], bs)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    _check("ll_paged_attention_decode", lib.ll_paged_attention_decode(
        _ptr(q), ctypes.byref(pool), _ptr(block_table), block_table.shape[1], _ptr(context_lens), B,
        Hq, k_pool.shape[1], d, bs, float(scale), _ptr(out), _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(stream)))
    return out


def paged_attention_decode_noalloc(q, k_pool, v_pool, block_table, context_lens, scale, out=None,
                                   status=None, stream=None):
    """ll_paged_attention_decode_noalloc: as paged_attention_decode, but the library keeps
    the split partials in its own fixed device array, so no workspace is passed or made."""
    _need(q, "q", torch.bfloat16)
    B, Hq, d = q.shape
    _need(block_table, "block_table", torch.int32)
    _need(context_lens, "context_lens", torch.int32, shape=(B,))
    pool = _pool(k_pool, v_pool)
    if out is None:
        out = torch.empty_like(q)
    if status is None:
        status = new_status(q.device)
    _check("ll_paged_attention_decode_noalloc", lib.ll_paged_attention_decode_noalloc(
        _ptr(q), ctypes.byref(pool), _ptr(block_table), block_table.shape[1], _ptr(context_lens), B,
        Hq, k_pool.shape[1], d, k_pool.shape[2], float(scale), _ptr(out), _ptr(status),
        _stream(stream)))
    return out


# ---------------------------------------------------------------- operators around the cache

def _rows3(t, name, dtype):
    """Checks a [tokens, heads, head_dim] tensor whose heads are contiguous within a token; returns the
    elements between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    T, H, d = shape
    if T == 0:
        return H * d
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (T > 1 and st < H * d):
        raise ValueError(f"{name} must hold each token's heads contiguously")
    return st if T > 1 else H * d


def _status(t):
    """A status word that the caller passed: the kernels set its bits as an int32."""
    _need(t, "status", torch.int32)
    if not t.numel():
        raise ValueError("status must hold one number")
    return t


def _on(first, *tensors):
    """The index of the device that all the tensors share (None among them is passed over)."""
    dev = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device is needed")
    return dev


# the current stream of a device as a number, without the Stream object around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name, fn, dev, stream, *args):
    """Calls the library on `stream` (default: the device's current one) with device index `dev` current."""
    if dev == torch.cuda.current_device():
        rc = fn(*args, stream.cuda_stream if stream is not None else _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream.cuda_stream if stream is not None else _raw_stream(dev))
    if rc != LL_OK:
        raise LayerError(name, rc)


def _made(stream, dev, *tensors):
    """Tensors made here, on the device's current stream, for a call on `stream`: it waits for that stream, and
    their memory is not handed out again before the call is done.  (None among them is passed over.)"""
    current = torch.cuda.current_stream(dev)
    tensors = [t for t in tensors if t is not None]
    if tensors and stream != current:
        stream.wait_stream(current)
        for t in tensors:
            t.record_stream(stream)


def make_rope_config(rotary_dim, theta=10000.0, scaling="plain", factor=1.0, original_max_position=0, low_turns=1.0,
                     high_turns=None, attention_factor=0.0) -> ll_rope_config:
    """ll_rope_config.  scaling: "plain", "linear", "ntk", "banded" or "yarn"; high_turns defaults to 4
    (banded) or 32 (yarn), attention_factor 0 to 0.1 ln(factor) + 1 (yarn)."""
    if scaling not in LL_ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(LL_ROPE_SCALINGS)}, got {scaling!r}")
    if high_turns is None:
        high_turns = 32.0 if scaling == "yarn" else 4.0
    return ll_rope_config(int(rotary_dim), LL_ROPE_SCALINGS[scaling], float(theta), float(factor),
                          int(original_max_position), float(low_turns), float(high_turns), float(attention_factor))


def rope_table(rope: ll_rope_config, max_position: int, device=None, stream=None) -> torch.Tensor:
    """ll_rope_table: a new float32 table [max_position, rotary_dim / 2, 2] of (cos, sin)."""
    n = lib.ll_rope_table_size(ctypes.byref(rope), int(max_position))
    if n == 0:
        raise LayerError("ll_rope_table_size", LL_ERR_INVALID_ARG)
    table = torch.empty(int(max_position), rope.rotary_dim // 2, 2, dtype=torch.float32, device=device or "cuda")
    if stream is not None:
        _made(stream, table.get_device(), table)
    _call("ll_rope_table", lib.ll_rope_table, table.get_device(), stream, ctypes.byref(rope), int(max_position), table.data_ptr(), n)
    return table


def pack_rope(cfg: ll_config, rope: ll_rope_config, packed: torch.Tensor, stream=None) -> None:
    """ll_pack_rope: the layer calls with `packed` rotate by the scaled frequencies from here on."""
    _need(packed, "packed", torch.uint8)
    _call("ll_pack_rope", lib.ll_pack_rope, packed.get_device(), stream, ctypes.byref(cfg), ctypes.byref(rope), packed.data_ptr(),
          packed.numel())


def rope(q, k, positions, table, layout="half", backward=False, q_out=None, k_out=None, status=None, stream=None):
    """ll_rope: q [tokens, n_heads, head_dim] and k [tokens, n_kv_heads, head_dim], BF16 or float32, heads
    contiguous within a token (views of a merged QKV output will do); either may be None.  `table` is
    rope_table()'s.  Pass q_out=q (k_out=k) to rotate in place.  The call is not recorded by autograd: the
    gradient is the call with backward=True, and a tensor that requires one is refused unless gradients are
    off (torch.no_grad()).  Returns (q_out, k_out)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q and k must be bfloat16 or float32 tensors")
    if layout not in LL_ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LL_ROPE_LAYOUTS)}, got {layout!r}")
    if torch.is_grad_enabled() and (getattr(q, "requires_grad", False) or getattr(k, "requires_grad", False)):
        raise ValueError("rope is not recorded by autograd: use torch.no_grad(), and backward=True for the gradient")
    T = d = None
    ends = []                      # per tensor: data, heads, stride, output data, output stride
    outs = []
    for t, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if t is None:
            ends.append((None, 0, 0, None, 0))
            outs.append(None)
            continue
        stride = _rows3(t, name, x.dtype)
        shape = t.shape
        if T is None:
            T, _, d = shape
        elif shape[0] != T or shape[2] != d:
            raise ValueError(f"k must be [{T}, n_kv_heads, {d}], got {tuple(shape)}")
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=x.device)     # (half the time of new_empty)
            out_stride = shape[1] * d
        else:
            out_stride = _rows3(out, name + "_out", x.dtype)
            if out.shape != shape:
                raise ValueError(f"{name}_out must have shape {tuple(shape)}, got {tuple(out.shape)}")
        ends.append((t.data_ptr(), shape[1], stride, out.data_ptr(), out_stride))
        outs.append(out)
    _need(positions, "positions", torch.int32, shape=(T,))
    _need(table, "table", torch.float32)
    rows = table.shape
    if len(rows) != 3 or rows[2] != 2 or not 2 <= 2 * rows[1] <= d:
        raise ValueError("table must be [max_position, rotary_dim / 2, 2] with rotary_dim <= head_dim")
    own_status = status is None
    status = new_status(x.device) if own_status else _status(status)
    dev = _on(x, k, outs[0], outs[1], positions, table, status)
    if stream is not None:
        _made(stream, dev, outs[0] if q_out is None else None, outs[1] if k_out is None else None,
              status if own_status else None)
    (qp, n_heads, qs, qo, qos), (kp, n_kv_heads, ks, ko, kos) = ends
    _call("ll_rope", lib.ll_rope, dev, stream, qp, kp, LL_F32 if x.dtype == torch.float32 else LL_BF16,
          positions.data_ptr(), T, n_heads, n_kv_heads, d, 2 * rows[1], LL_ROPE_LAYOUTS[layout],
          LL_ROPE_BACKWARD if backward else LL_ROPE_FORWARD, qs, ks, table.data_ptr(), rows[0], qo, ko, qos, kos,
          status.data_ptr())
    return outs[0], outs[1]


def _heads(t, name, dtype, shape=None):
    """ll_head_rows of a [tokens, heads, head_dim] tensor (None: no heads)."""
    if t is None:
        return ll_head_rows(None, 0, 0)
    stride = _rows3(t, name, dtype)
    own = t.shape
    if shape is not None and own != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(own)}")
    return ll_head_rows(t.data_ptr(), stride, own[1])


_NORM_DTYPES = {torch.bfloat16: LL_BF16, torch.float32: LL_F32}


def _norm_args(q, k, q_gain, k_gain, positions, table, layout, name):
    """Checks what norm_rope and its gradient share; returns (dtype, tokens, head_dim, ll_head_rows of q and k)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if not isinstance(x, _Tensor) or x.dtype not in _NORM_DTYPES:
        raise TypeError("q and k must be bfloat16 or float32 tensors")
    if layout not in LL_ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LL_ROPE_LAYOUTS)}, got {layout!r}")
    if torch.is_grad_enabled():
        for t in (q, k, q_gain, k_gain):
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} is not recorded by autograd: use torch.no_grad(), and norm_rope_backward for "
                                 "the gradient")
    dtype = x.dtype
    qh, kh = _heads(q, "q", dtype), _heads(k, "k", dtype)
    T, _, d = x.shape
    if q is not None:
        _need(q_gain, "q_gain", torch.float32, True, (d,))
    if k is not None:
        if q is not None:
            Tk, _, dk = k.shape
            if Tk != T or dk != d:
                raise ValueError(f"k must be [{T}, n_kv_heads, {d}], got {tuple(k.shape)}")
        _need(k_gain, "k_gain", torch.float32, True, (d,))
    _need(positions, "positions", torch.int32, True, (T,))
    _need(table, "table", torch.float32)
    rows = table.shape
    if len(rows) != 3 or rows[2] != 2 or not 2 <= 2 * rows[1] <= d:
        raise ValueError("table must be [max_position, rotary_dim / 2, 2] with rotary_dim <= head_dim")
    return dtype, T, d, qh, kh


def _head_out(t, out, name):
    """(`out`, or a new contiguous tensor of t's shape, and its ll_head_rows); None for None."""
    if t is None:
        return None, ll_head_rows(None, 0, 0)
    if out is not None:
        return out, _heads(out, name, t.dtype, t.shape)
    shape = t.shape
    out = torch.empty(shape, dtype=t.dtype, device=t.device)
    return out, ll_head_rows(out.data_ptr(), shape[1] * shape[2], shape[1])


def _norm_usual(q, k, q_gain, k_gain, positions, table, layout, status):
    """What nearly every call of norm_rope and its gradient is, in one look: q and k with their gains, rows, a status word,
    all on the current device.  Returns (device index, tokens, n_heads, n_kv_heads, head_dim, strides of q and k), or None:
    then the checks below say what is wrong, or do what is unusual.  (A call of few tokens takes 15.4 us so, 18.6 without; the gradient 24.7, 32.)"""
    for t in (q, k, q_gain, k_gain, positions, table, status):
        if not isinstance(t, _Tensor):
            return None
    if not q.is_cuda:
        return None
    dtype, dev = q.dtype, torch.cuda.current_device()
    if dtype not in _NORM_DTYPES or k.dtype is not dtype or q.dim() != 3 or k.dim() != 3 or layout not in LL_ROPE_LAYOUTS:
        return None
    T, H, d = q.shape
    Tk, Hk, dk = k.shape
    st, sh, sd = q.stride()
    kt, kh, kd = k.stride()
    if T == 1:
        st, kt = H * d, Hk * d
    if T < 1 or Tk != T or dk != d or sd != 1 or kd != 1 or sh != d or kh != d or st < H * d or kt < Hk * d or \
            q_gain.dtype is not torch.float32 or k_gain.dtype is not torch.float32 or table.dtype is not torch.float32 or \
            positions.dtype is not torch.int32 or status.dtype is not torch.int32 or q_gain.shape != (d,) or \
            k_gain.shape != (d,) or positions.shape != (T,) or table.dim() != 3 or not status.numel():
        return None
    if not (q.get_device() == dev and k.get_device() == dev and q_gain.get_device() == dev and k_gain.get_device() == dev and
            positions.get_device() == dev and table.get_device() == dev and status.get_device() == dev and
            q_gain.is_contiguous() and k_gain.is_contiguous() and positions.is_contiguous() and table.is_contiguous() and
            status.is_contiguous()):
        return None
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or q_gain.requires_grad or k_gain.requires_grad):
        return None
    _, half, two = table.shape
    return (dev, T, H, Hk, d, st, kt) if two == 2 and 2 <= 2 * half <= d else None


def norm_rope(q, k, q_gain, k_gain, positions, table, eps=1e-5, layout="half", q_out=None, k_out=None, status=None,
              stream=None):
    """ll_norm_rope: RMS norm of every head of q [tokens, n_heads, head_dim] and k [tokens, n_kv_heads, head_dim] with
    the gains (float32 [head_dim]), then the rotary positions of rope(), in one pass.  q and k are BF16 or float32,
    heads contiguous within a token; either may be None (its gain too).  Pass q_out=q (k_out=k) to work in place.
    Not recorded by autograd: norm_rope_backward is the gradient.  Returns (q_out, k_out)."""
    usual = _norm_usual(q, k, q_gain, k_gain, positions, table, layout, status) if stream is None and q_out is None and \
        k_out is None else None
    if usual is not None:
        dev, T, H, Hk, d, st, kt = usual
        dtype, device = q.dtype, q.device
        q_out = torch.empty((T, H, d), dtype=dtype, device=device)
        k_out = torch.empty((T, Hk, d), dtype=dtype, device=device)
        rc = lib.ll_norm_rope(ll_head_rows(q.data_ptr(), st, H), ll_head_rows(k.data_ptr(), kt, Hk), _NORM_DTYPES[dtype],
                              q_gain.data_ptr(), k_gain.data_ptr(), eps, positions.data_ptr(), T, d, 2 * table.shape[1],
                              LL_ROPE_LAYOUTS[layout], table.data_ptr(), table.shape[0], ll_head_rows(q_out.data_ptr(), H * d, H),
                              ll_head_rows(k_out.data_ptr(), Hk * d, Hk), status.data_ptr(), _raw_stream(dev))
        if rc != LL_OK:
            raise LayerError("ll_norm_rope", rc)
        return q_out, k_out
    dtype, T, d, qh, kh = _norm_args(q, k, q_gain, k_gain, positions, table, layout, "norm_rope")
    given = q_out, k_out, status
    q_out, qo = _head_out(q, q_out, "q_out")
    k_out, ko = _head_out(k, k_out, "k_out")
    x = q if q is not None else k
    status = new_status(x.device) if status is None else _status(status)
    if q is None:
        q_gain = None
    if k is None:
        k_gain = None
    dev = _on(x, k, q_out, k_out, q_gain, k_gain, positions, table, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (q_out, k_out, status))))
    _call("ll_norm_rope", lib.ll_norm_rope, dev, stream, qh, kh, _NORM_DTYPES[dtype],
          q_gain.data_ptr() if q is not None else None, k_gain.data_ptr() if k is not None else None, eps,
          positions.data_ptr(), T, d, 2 * table.shape[1], LL_ROPE_LAYOUTS[layout], table.data_ptr(), table.shape[0], qo, ko,
          status.data_ptr())
    return q_out, k_out


def norm_rope_backward_workspace_size(head_dim: int) -> int:
    return lib.ll_norm_rope_backward_workspace_size(int(head_dim))


def norm_rope_backward(dq, dk, q, k, q_gain, k_gain, positions, table, eps=1e-5, layout="half", q_grad=None, k_grad=None,
                       q_gain_grad=None, k_gain_grad=None, workspace=None, status=None, stream=None):
    """ll_norm_rope_backward: the gradients of norm_rope's inputs q, k and gains, from the gradients dq, dk of its
    outputs.  Pass q_grad=dq (k_grad=dk) to overwrite those.  Returns (q_grad, k_grad, q_gain_grad, k_gain_grad), the
    gains' in float32; None for a tensor that is None."""
    usual = _norm_usual(q, k, q_gain, k_gain, positions, table, layout, status) if stream is None and q_grad is None and \
        k_grad is None and q_gain_grad is None and k_gain_grad is None and isinstance(dq, _Tensor) and \
        isinstance(dk, _Tensor) and isinstance(workspace, _Tensor) else None
    if usual is not None:
        dev, T, H, Hk, d, st, kt = usual
        dtype, device = q.dtype, q.device
        if dq.dtype is dtype and dk.dtype is dtype and dq.shape == q.shape and dk.shape == k.shape and \
                workspace.dtype is torch.uint8 and workspace.is_contiguous() and dq.get_device() == dev and \
                dk.get_device() == dev and workspace.get_device() == dev:
            dst, dsh, dsd = dq.stride()
            dkt, dkh, dkd = dk.stride()
            if T == 1:
                dst, dkt = H * d, Hk * d
            if dsd == 1 and dkd == 1 and dsh == d and dkh == d and dst >= H * d and dkt >= Hk * d:
                q_grad = torch.empty((T, H, d), dtype=dtype, device=device)
                k_grad = torch.empty((T, Hk, d), dtype=dtype, device=device)
                q_gain_grad = torch.empty((d,), dtype=torch.float32, device=device)
                k_gain_grad = torch.empty((d,), dtype=torch.float32, device=device)
                rc = lib.ll_norm_rope_backward(
                    ll_head_rows(dq.data_ptr(), dst, H), ll_head_rows(dk.data_ptr(), dkt, Hk), ll_head_rows(q.data_ptr(), st, H),
                    ll_head_rows(k.data_ptr(), kt, Hk), _NORM_DTYPES[dtype], q_gain.data_ptr(), k_gain.data_ptr(), eps,
                    positions.data_ptr(), T, d, 2 * table.shape[1], LL_ROPE_LAYOUTS[layout], table.data_ptr(), table.shape[0],
                    ll_head_rows(q_grad.data_ptr(), H * d, H), ll_head_rows(k_grad.data_ptr(), Hk * d, Hk),
                    q_gain_grad.data_ptr(), k_gain_grad.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr(),
                    _raw_stream(dev))
                if rc != LL_OK:
                    raise LayerError("ll_norm_rope_backward", rc)
                return q_grad, k_grad, q_gain_grad, k_gain_grad
    dtype, T, d, qh, kh = _norm_args(q, k, q_gain, k_gain, positions, table, layout, "norm_rope_backward")
    if (dq is None) != (q is None) or (dk is None) != (k is None):
        raise ValueError("dq and dk go with q and k")
    given = q_grad, k_grad, q_gain_grad, k_gain_grad, workspace, status
    x = q if q is not None else k
    dqh = _heads(dq, "dq", dtype, q.shape if q is not None else None)
    dkh = _heads(dk, "dk", dtype, k.shape if k is not None else None)
    q_grad, qo = _head_out(q, q_grad, "q_grad")
    k_grad, ko = _head_out(k, k_grad, "k_grad")
    if q is None:
        q_gain = q_gain_grad = None
    elif q_gain_grad is None:
        q_gain_grad = torch.empty((d,), dtype=torch.float32, device=x.device)
    else:
        _need(q_gain_grad, "q_gain_grad", torch.float32, shape=(d,))
    if k is None:
        k_gain = k_gain_grad = None
    elif k_gain_grad is None:
        k_gain_grad = torch.empty((d,), dtype=torch.float32, device=x.device)
    else:
        _need(k_gain_grad, "k_gain_grad", torch.float32, shape=(d,))
    if workspace is None:
        workspace = torch.empty(max(norm_rope_backward_workspace_size(d), 16), dtype=torch.uint8, device=x.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(x.device) if status is None else _status(status)
    outs = q_grad, k_grad, q_gain_grad, k_gain_grad
    dev = _on(x, k, dq, dk, *outs, q_gain, k_gain, positions, table, workspace, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (*outs, workspace, status))))
    _call("ll_norm_rope_backward", lib.ll_norm_rope_backward, dev, stream, dqh, dkh, qh, kh, _NORM_DTYPES[dtype],
          q_gain.data_ptr() if q is not None else None,
          k_gain.data_ptr() if k is not None else None, eps, positions.data_ptr(), T, d, 2 * table.shape[1],
          LL_ROPE_LAYOUTS[layout], table.data_ptr(), table.shape[0], qo, ko,
          q_gain_grad.data_ptr() if q is not None else None, k_gain_grad.data_ptr() if k is not None else None,
          workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return outs


class PoolF8:
    """An e4m3 KV pool on the GPU: codes k, v float8_e4m3fn [num_blocks, n_kv_heads, block_size, head_dim]
    and float32 scales k_scale, v_scale [num_blocks, n_kv_heads].  The tensors were checked together: they
    cannot be replaced (another set is another pool)."""

    def __init__(self, k, v, k_scale, v_scale):
        _need(k, "k codes", torch.float8_e4m3fn)
        _need(v, "v codes", torch.float8_e4m3fn, shape=tuple(k.shape))
        if k.dim() != 4:
            raise ValueError("codes must be [num_blocks, n_kv_heads, block_size, head_dim]")
        _need(k_scale, "k_scale", torch.float32, shape=tuple(k.shape[:2]))
        _need(v_scale, "v_scale", torch.float32, shape=tuple(k.shape[:2]))
        _on(k, v, k_scale, v_scale)
        self._tensors = k, v, k_scale, v_scale
        self._c = ll_kv_pool_f8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.shape[0])

    @classmethod
    def empty(cls, num_blocks, n_kv_heads, block_size, head_dim, device="cuda"):
        shape = (num_blocks, n_kv_heads, block_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        return cls(*codes, *(torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @property
    def device(self):
        return self.k.device

    @property
    def block_size(self):
        return self.k.shape[2]

    def tensors(self):
        """The pool's tensors, block first, as a BlockSet takes them."""
        return list(self._tensors)

    def c(self):
        return self._c


def _f8_batch(pool, block_table, context_lens):
    _need(context_lens, "context_lens", torch.int32)
    if context_lens.dim() != 1:
        raise ValueError("context_lens must be [batch]")
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] < context_lens.shape[0]:
        raise ValueError("block_table must be [batch, max_blocks]")
    return context_lens.shape[0]


def append_to_cache_f8(k, v, pool: PoolF8, block_table, context_lens, cu_new=None, max_new=1, status=None, stream=None):
    """ll_append_to_cache_f8: k, v BF16 [tokens, n_kv_heads, head_dim] (heads contiguous within a token)
    into `pool` at the last positions of each sequence.  cu_new int32 [batch + 1] with at most max_new
    tokens per sequence; None: one token each.  Returns the status word."""
    ks, vs = _rows3(k, "k", torch.bfloat16), _rows3(v, "v", torch.bfloat16)
    if v.shape != k.shape or k.shape[1] != pool.k.shape[1] or k.shape[2] != pool.k.shape[3]:
        raise ValueError(f"k and v must both be [tokens, {pool.k.shape[1]}, {pool.k.shape[3]}]")
    B = _f8_batch(pool, block_table, context_lens)
    if cu_new is not None:
        _need(cu_new, "cu_new", torch.int32, shape=(B + 1,))
    own_status = status is None
    status = new_status(k.device) if own_status else _status(status)
    dev = _on(k, v, pool.k, block_table, context_lens, cu_new, status)
    if stream is not None and own_status:
        _made(stream, dev, status)
    _call("ll_append_to_cache_f8", lib.ll_append_to_cache_f8, dev, stream, k.data_ptr(), v.data_ptr(), ks, vs,
          cu_new.data_ptr() if cu_new is not None else None, k.shape[0], context_lens.data_ptr(), B, int(max_new),
          k.shape[1], k.shape[2], pool.block_size, ctypes.byref(pool.c()), block_table.data_ptr(),
          block_table.shape[1], status.data_ptr())
    return status


def attention_decode_f8_workspace_size(batch, n_heads, n_kv_heads, head_dim):
    return lib.ll_attention_decode_f8_workspace_size(int(batch), int(n_heads), int(n_kv_heads), int(head_dim))


def attention_prefill_f8_workspace_size(batch, tokens, max_new, n_heads, n_kv_heads, head_dim):
    return lib.ll_attention_prefill_f8_workspace_size(int(batch), int(tokens), int(max_new), int(n_heads),
                                                      int(n_kv_heads), int(head_dim))


def _f8_attention(q, pool, out, workspace, status, size, stream):
    """Checks q, out and the workspace of an attention call; makes what was not passed."""
    given = out, workspace, status
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[2] != pool.k.shape[3]:
        raise ValueError(f"q must be [rows, n_heads, {pool.k.shape[3]}], got {tuple(q.shape)}")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, shape=tuple(q.shape))
    if workspace is None:
        workspace = torch.empty(max(size(), 16), dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(q.device) if status is None else _status(status)
    if stream is not None:
        _made(stream, q.get_device(), *(t if g is None else None for g, t in zip(given, (out, workspace, status))))
    return out, workspace, status


def paged_attention_decode_f8(q, pool: PoolF8, block_table, context_lens, scale, out=None, workspace=None, status=None,
                              stream=None):
    """ll_paged_attention_decode_f8: q BF16 [batch, n_heads, head_dim] over an e4m3 pool.  Returns out."""
    B = _f8_batch(pool, block_table, context_lens)
    Hkv = pool.k.shape[1]
    out, workspace, status = _f8_attention(
        q, pool, out, workspace, status, lambda: attention_decode_f8_workspace_size(B, q.shape[1], Hkv, q.shape[2]),
        stream)
    if q.shape[0] != B:
        raise ValueError(f"q must have {B} rows, one per sequence")
    dev = _on(q, pool.k, block_table, context_lens, out, workspace, status)
    _call("ll_paged_attention_decode_f8", lib.ll_paged_attention_decode_f8, dev, stream, q.data_ptr(), ctypes.byref(pool.c()), block_table.data_ptr(),
          block_table.shape[1], context_lens.data_ptr(), B, q.shape[1], Hkv, q.shape[2], pool.block_size, float(scale),
          out.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return out


def paged_attention_prefill_f8(q, cu_new, pool: PoolF8, block_table, context_lens, scale, max_new, out=None,
                               workspace=None, status=None, stream=None):
    """ll_paged_attention_prefill_f8: q BF16 [tokens, n_heads, head_dim], sequence b's new tokens in rows
    cu_new[b] .. cu_new[b + 1] - 1 (at most max_new), already in the pool.  Returns out."""
    B = _f8_batch(pool, block_table, context_lens)
    _need(cu_new, "cu_new", torch.int32, shape=(B + 1,))
    Hkv = pool.k.shape[1]
    out, workspace, status = _f8_attention(
        q, pool, out, workspace, status,
        lambda: attention_prefill_f8_workspace_size(B, q.shape[0], max_new, q.shape[1], Hkv, q.shape[2]), stream)
    dev = _on(q, pool.k, cu_new, block_table, context_lens, out, workspace, status)
    _call("ll_paged_attention_prefill_f8", lib.ll_paged_attention_prefill_f8, dev, stream, q.data_ptr(), cu_new.data_ptr(), q.shape[0],
          ctypes.byref(pool.c()), block_table.data_ptr(), block_table.shape[1], context_lens.data_ptr(), B,
          int(max_new), q.shape[1], Hkv, q.shape[2], pool.block_size, float(scale), out.data_ptr(),
          workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return out


def new_workspace_f8(cfg, max_tokens, max_blocks, device=None):
    """A workspace for layer calls over an e4m3 pool of up to max_tokens tokens."""
    n = lib.ll_workspace_size_f8(ctypes.byref(cfg), int(max_tokens), int(max_blocks))
    if n == 0:
        raise LayerError("ll_workspace_size_f8", LL_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _layer_f8(cfg, packed, x, pool, block_table, context_lens, tokens, y, workspace, status, stream):
    given = y, workspace, status
    _need(packed, "packed", torch.uint8)
    _need(x, "x", torch.bfloat16, shape=(tokens, cfg.hidden))
    if tuple(pool.k.shape[1:]) != (cfg.n_kv_heads, cfg.block_size, cfg.head_dim):
        raise ValueError(f"the pool must be [num_blocks, {cfg.n_kv_heads}, {cfg.block_size}, {cfg.head_dim}]")
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", torch.bfloat16, shape=(tokens, cfg.hidden))
    if workspace is None:
        workspace = new_workspace_f8(cfg, tokens, block_table.shape[1], x.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(x.device) if status is None else _status(status)
    dev = _on(x, packed, pool.k, block_table, context_lens, y, workspace, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (y, workspace, status))))
    return y, workspace, status, dev


def layer_prefill_f8(cfg, packed, x, pool: PoolF8, block_table, context_lens, seq_len, y=None, workspace=None,
                     status=None, stream=None):
    """ll_layer_prefill_f8: x BF16 [batch * seq_len, hidden], each sequence's seq_len new tokens at its last
    positions.  Returns y."""
    B = _f8_batch(pool, block_table, context_lens)
    y, workspace, status, dev = _layer_f8(cfg, packed, x, pool, block_table, context_lens, B * int(seq_len), y,
                                          workspace, status, stream)
    _call("ll_layer_prefill_f8", lib.ll_layer_prefill_f8, dev, stream, ctypes.byref(cfg), packed.data_ptr(),
          x.data_ptr(), context_lens.data_ptr(), B, int(seq_len), ctypes.byref(pool.c()), block_table.data_ptr(),
          block_table.shape[1], y.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return y


def layer_decode_step_f8(cfg, packed, x, pool: PoolF8, block_table, context_lens, y=None, workspace=None, status=None,
                         stream=None):
    """ll_layer_decode_step_f8: x BF16 [batch, hidden], one new token per sequence.  Returns y."""
    B = _f8_batch(pool, block_table, context_lens)
    y, workspace, status, dev = _layer_f8(cfg, packed, x, pool, block_table, context_lens, B, y, workspace, status,
                                          stream)
    _call("ll_layer_decode_step_f8", lib.ll_layer_decode_step_f8, dev, stream, ctypes.byref(cfg), packed.data_ptr(),
          x.data_ptr(), ctypes.byref(pool.c()), block_table.data_ptr(), block_table.shape[1], context_lens.data_ptr(),
          B, y.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return y


# ---------------------------------------------------------------- attention weights

def _paged_batch(block_table, context_lens):
    """Checks a batch over a paged cache; returns its size."""
    _need(context_lens, "context_lens", torch.int32)
    _need(block_table, "block_table", torch.int32)
    if context_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != context_lens.shape[0]:
        raise ValueError("context_lens must be [batch] and block_table [batch, max_blocks]")
    return context_lens.shape[0]


def _weights(weights, batch, n_kv_heads):
    _need(weights, "weights", torch.float32)
    if weights.dim() != 3 or weights.shape[0] != batch or weights.shape[1] != n_kv_heads:
        raise ValueError(f"weights must be [{batch}, {n_kv_heads}, width], got {tuple(weights.shape)}")
    return weights.shape[2]


def attention_decode_weights_workspace_size(batch, n_heads, n_kv_heads, head_dim, max_blocks, block_size):
    return lib.ll_attention_decode_weights_workspace_size(int(batch), int(n_heads), int(n_kv_heads), int(head_dim),
                                                          int(max_blocks), int(block_size))


def _decode_weights(name, fn, cpool, pool_tensors, q, block_table, context_lens, scale, weights, out, workspace, status, stream):
    given = out, workspace, status
    k = pool_tensors[0]
    _, Hkv, bs, d = k.shape
    B = _paged_batch(block_table, context_lens)
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != d:
        raise ValueError(f"q must be [{B}, n_heads, {d}], got {tuple(q.shape)}")
    width = _weights(weights, B, Hkv)
    Hq, mb = q.shape[1], block_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, shape=tuple(q.shape))
    if workspace is None:
        workspace = torch.empty(max(attention_decode_weights_workspace_size(B, Hq, Hkv, d, mb, bs), 16), dtype=torch.uint8,
                                device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(q.device) if status is None else _status(status)
    dev = _on(q, *pool_tensors, block_table, context_lens, weights, out, workspace, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (out, workspace, status))))
    _call(name, fn, dev, stream, q.data_ptr(), cpool, block_table.data_ptr(), mb, context_lens.data_ptr(), B, Hq, Hkv, d, bs,
          float(scale), weights.data_ptr(), width, out.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return out


def paged_attention_decode_weights(q, k_pool, v_pool, block_table, context_lens, scale, weights, out=None, workspace=None,
                                   status=None, stream=None):
    """ll_paged_attention_decode_weights: paged_attention_decode that also adds every cached position's attention
    weight to `weights` (float32 [batch, n_kv_heads, width], in place).  Returns out."""
    return _decode_weights("ll_paged_attention_decode_weights", lib.ll_paged_attention_decode_weights, _pool(k_pool, v_pool),
                           (k_pool, v_pool), q, block_table, context_lens, scale, weights, out, workspace, status, stream)


def paged_attention_decode_weights_q8(q, pool: PoolQ8, block_table, context_lens, scale, weights, out=None, workspace=None,
                                      status=None, stream=None):
    """ll_paged_attention_decode_weights_q8: the same over an INT8 pool.  Returns out."""
    return _decode_weights("ll_paged_attention_decode_weights_q8", lib.ll_paged_attention_decode_weights_q8, pool.c(),
                           (pool.k, pool.v, pool.k_scale, pool.v_scale), q, block_table, context_lens, scale, weights, out,
                           workspace, status, stream)


def attention_weights_workspace_size(batch, tokens, max_new, n_heads, n_kv_heads, head_dim, max_blocks, block_size):
    return lib.ll_attention_weights_workspace_size(int(batch), int(tokens), int(max_new), int(n_heads), int(n_kv_heads),
                                                   int(head_dim), int(max_blocks), int(block_size))


def paged_attention_weights(q, cu_new, k_pool, block_table, context_lens, scale, weights, max_new, workspace=None, status=None,
                            stream=None):
    """ll_paged_attention_weights: adds the attention weights of query rows q BF16 [tokens, n_heads, head_dim] (sequence b's
    in rows cu_new[b] .. cu_new[b + 1] - 1, at most max_new, at the end of its context; whole prompts, chunks or the last
    rows) to `weights` (float32 [batch, n_kv_heads, width], in place).  k_pool BF16 [num_blocks, n_kv_heads, block_size,
    head_dim] already holds the keys.  Returns weights."""
    given = workspace, status
    _need(k_pool, "k_pool", torch.bfloat16)
    if k_pool.dim() != 4:
        raise ValueError("k_pool must be [num_blocks, n_kv_heads, block_size, head_dim]")
    nb, Hkv, bs, d = k_pool.shape
    B = _paged_batch(block_table, context_lens)
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [tokens, n_heads, {d}], got {tuple(q.shape)}")
    _need(cu_new, "cu_new", torch.int32, shape=(B + 1,))
    width = _weights(weights, B, Hkv)
    T, Hq, mb = q.shape[0], q.shape[1], block_table.shape[1]
    if workspace is None:
        workspace = torch.empty(max(attention_weights_workspace_size(B, T, max_new, Hq, Hkv, d, mb, bs), 16), dtype=torch.uint8,
                                device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(q.device) if status is None else _status(status)
    dev = _on(q, k_pool, cu_new, block_table, context_lens, weights, workspace, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (workspace, status))))
    _call("ll_paged_attention_weights", lib.ll_paged_attention_weights, dev, stream, q.data_ptr(), cu_new.data_ptr(), T,
          k_pool.data_ptr(), nb, block_table.data_ptr(), mb, context_lens.data_ptr(), B, int(max_new), Hq, Hkv, d, bs,
          float(scale), weights.data_ptr(), width, workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return weights


def new_workspace_weights(cfg, batch, max_blocks, device=None):
    """A workspace for layer_decode_step_weights of up to `batch` sequences."""
    n = lib.ll_workspace_size_weights(ctypes.byref(cfg), int(batch), int(max_blocks))
    if n == 0:
        raise LayerError("ll_workspace_size_weights", LL_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def layer_decode_step_weights(cfg, packed, x, pool, block_table, context_lens, weights, positions=None, y=None, workspace=None,
                              status=None, stream=None):
    """ll_layer_decode_step_weights (_q8 where `pool` is a PoolQ8; else a (K, V) pair of BF16 pools): the layer's decode
    step that adds its attention weights to `weights` (float32 [batch, n_kv_heads, width], in place).  positions int32
    [batch]: the new tokens' rotary positions where the cache has been cut (None: context_lens - 1).  Returns y."""
    given = y, workspace, status
    q8 = isinstance(pool, PoolQ8)
    if q8:
        k, cpool = pool.k, pool.c()
    else:
        cpool = _pool(*pool)
        k = pool[0]
    B = _paged_batch(block_table, context_lens)
    _need(packed, "packed", torch.uint8)
    _need(x, "x", torch.bfloat16, shape=(B, cfg.hidden))
    if tuple(k.shape[1:]) != (cfg.n_kv_heads, cfg.block_size, cfg.head_dim):
        raise ValueError(f"the pool must be [num_blocks, {cfg.n_kv_heads}, {cfg.block_size}, {cfg.head_dim}]")
    width = _weights(weights, B, cfg.n_kv_heads)
    if positions is not None:
        _need(positions, "positions", torch.int32, shape=(B,))
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", torch.bfloat16, shape=(B, cfg.hidden))
    mb = block_table.shape[1]
    if workspace is None:
        workspace = new_workspace_weights(cfg, B, mb, x.device)
    else:
        _need(workspace, "workspace", torch.uint8)
    status = new_status(x.device) if status is None else _status(status)
    dev = _on(x, packed, k, block_table, context_lens, weights, positions, y, workspace, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (y, workspace, status))))
    name = "ll_layer_decode_step_weights_q8" if q8 else "ll_layer_decode_step_weights"
    _call(name, getattr(lib, name), dev, stream, ctypes.byref(cfg), packed.data_ptr(), x.data_ptr(), cpool,
          block_table.data_ptr(), mb, context_lens.data_ptr(), positions.data_ptr() if positions is not None else None, B,
          weights.data_ptr(), width, y.data_ptr(), workspace.data_ptr(), workspace.numel(), status.data_ptr())
    return y


def evict_rows(pool, block_table, context_lens, weights, keep, max_keep=None, sinks=0, recent=0, weights_out=None,
               kept=None, new_lens=None, status=None, stream=None):
    """ll_evict_rows: every sequence keeps at most `keep` cached rows for each KV head (the first `sinks`, the last
    `recent`, and between them those of the largest weights), moved to the front of its blocks in place.

    pool: a (K, V) pair of BF16 pools or a PoolQ8.  keep: a number, or an int32 tensor [batch] with max_keep the
    largest of them.  weights float32 [batch, n_kv_heads, width] move along, in place or to weights_out.  Returns
    (kept, new_lens): int32 [batch, n_kv_heads, max_keep], the position that each row had (-1 behind the last), and
    int32 [batch], the new context lengths."""
    if isinstance(pool, PoolQ8):
        tensors = pool.k, pool.v, pool.k_scale, pool.v_scale
    elif isinstance(pool, (tuple, list)) and len(pool) == 2:
        _pool(*pool)
        tensors = tuple(pool)
    else:
        raise TypeError("pool must be a (K, V) pair of BF16 pools or a PoolQ8")
    nb, Hkv, bs = tensors[0].shape[:3]
    B = _paged_batch(block_table, context_lens)
    width = _weights(weights, B, Hkv)
    given = kept, new_lens, status
    if isinstance(keep, torch.Tensor):
        _need(keep, "keep", torch.int32, shape=(B,))
        if max_keep is None:
            raise ValueError("a keep of each sequence needs max_keep")
        per = keep
    else:
        if max_keep is not None and int(max_keep) != int(keep):
            raise ValueError("max_keep is keep where that is a number")
        max_keep, per = int(keep), None
    max_keep = int(max_keep)
    if max_keep < 1:
        raise ValueError("keep (max_keep) must be at least 1")
    if weights_out is None:
        weights_out = weights
    else:
        _need(weights_out, "weights_out", torch.float32, shape=tuple(weights.shape))
    if kept is None:
        kept = torch.empty((B, Hkv, max_keep), dtype=torch.int32, device=weights.device)
    else:
        _need(kept, "kept", torch.int32, shape=(B, Hkv, max_keep))
    if new_lens is None:
        new_lens = torch.empty((B,), dtype=torch.int32, device=weights.device)
    else:
        _need(new_lens, "new_lens", torch.int32, shape=(B,))
    status = new_status(weights.device) if status is None else _status(status)
    dev = _on(weights, *tensors, block_table, context_lens, per, weights_out, kept, new_lens, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (kept, new_lens, status))))
    rows = (ll_row_tensor * len(tensors))(
        *[(t.data_ptr(), t.element_size() * (t.shape[3] if t.dim() == 4 else 1)) for t in tensors])
    _call("ll_evict_rows", lib.ll_evict_rows, dev, stream, rows, len(tensors), nb, Hkv, bs, block_table.data_ptr(),
          block_table.shape[1], context_lens.data_ptr(), B, weights.data_ptr(), width,
          per.data_ptr() if per is not None else None, max_keep, int(sinks), int(recent), weights_out.data_ptr(),
          kept.data_ptr(), new_lens.data_ptr(), status.data_ptr())
    return kept, new_lens


class BlockSet:
    """Tensors [num_blocks, ...] that share their block ids (K and V pools of every layer, and their
    scales), for copy_blocks.  Keeps the tensors and the array that the library reads; they cannot be
    replaced (another set of tensors is another BlockSet)."""

    tensors = property(lambda self: self._tensors)
    device = property(lambda self: self._tensors[0].device)
    num_blocks = property(lambda self: self._tensors[0].shape[0])

    def __init__(self, tensors):
        self._tensors = tuple(tensors)
        if not self.tensors:
            raise ValueError("a BlockSet needs a tensor")
        for t in self.tensors:
            if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dim() < 1:
                raise ValueError("a BlockSet takes contiguous GPU tensors [num_blocks, ...]")
            if t.shape[0] != self.tensors[0].shape[0]:
                raise ValueError("the tensors of a BlockSet have the same number of blocks")
        _on(*self.tensors)
        self._c = (ll_block_tensor * len(self.tensors))(
            *((t.data_ptr(), t.numel() // max(self.num_blocks, 1) * t.element_size()) for t in self.tensors))


def copy_blocks(blocks: BlockSet, pairs, n_pairs=None, status=None, stream=None):
    """ll_copy_blocks: block pairs[i, 0] to block pairs[i, 1] (int32 [n, 2], on the GPU) in every tensor of
    the set; n_pairs: a GPU int32 tensor of one element with the number of pairs, None for all.  Returns
    the status word."""
    _need(pairs, "pairs", torch.int32)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    if n_pairs is not None:
        _need(n_pairs, "n_pairs", torch.int32)
        if n_pairs.numel() != 1:
            raise ValueError("n_pairs must hold one number")
    own_status = status is None
    status = new_status(blocks.device) if own_status else _status(status)
    dev = _on(blocks.tensors[0], pairs, n_pairs, status)
    if stream is not None and own_status:
        _made(stream, dev, status)
    _call("ll_copy_blocks", lib.ll_copy_blocks, dev, stream, blocks._c, len(blocks.tensors), blocks.num_blocks, pairs.data_ptr(),
          pairs.shape[0], n_pairs.data_ptr() if n_pairs is not None else None, status.data_ptr())
    return status


def compact_blocks(block_table, num_blocks, new_table=None, pairs=None, counts=None, block_map=None, status=None,
                   stream=None):
    """ll_compact_blocks: the plan that packs the blocks of block_table to the front of a pool of num_blocks.
    Returns (new_table, pairs [num_blocks // 2, 2], counts [2], block_map [num_blocks]); move the
    contents with copy_blocks(blocks, pairs, n_pairs=counts[1:])."""
    num_blocks = int(num_blocks)
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_blocks]")
    dev = block_table.device
    new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
    given = new_table, pairs, counts, block_map, status
    new_table = new(*block_table.shape) if new_table is None else new_table
    pairs = new(num_blocks // 2, 2) if pairs is None else pairs
    counts = new(2) if counts is None else counts
    block_map = new(num_blocks) if block_map is None else block_map
    _need(new_table, "new_table", torch.int32, shape=tuple(block_table.shape))
    _need(pairs, "pairs", torch.int32, shape=(num_blocks // 2, 2))
    _need(counts, "counts", torch.int32, shape=(2,))
    _need(block_map, "block_map", torch.int32, shape=(num_blocks,))
    status = new_status(dev) if status is None else _status(status)
    dev = _on(block_table, new_table, pairs, counts, block_map, status)
    if stream is not None:
        _made(stream, dev, *(t if g is None else None for g, t in zip(given, (new_table, pairs, counts, block_map, status))))
    _call("ll_compact_blocks", lib.ll_compact_blocks, dev, stream, block_table.data_ptr(), block_table.shape[0], block_table.shape[1],
          num_blocks, new_table.data_ptr(), pairs.data_ptr(), counts.data_ptr(), block_map.data_ptr(),
          status.data_ptr())
    return new_table, pairs, counts, block_map


def set_prefill_attention_ctas(n: int) -> None:
    """ll_set_prefill_attention_ctas: bound on the persistent prefill attention's CTAs
    (n <= 0: one per SM)."""
    lib.ll_set_prefill_attention_ctas(int(n))


def linear(x, w, y=None, workspace=None, status=None, stream=None):
    """ll_linear: y = x w^T, x BF16 [m, k], w BF16 [n, k]."""
    _need(x, "x", torch.bfloat16)
    _need(w, "w", torch.bfloat16)
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("w must be [n, k]")
    if y is None:
        y = torch.empty(m, n, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(lib.ll_linear_workspace_size(m, n, k), dtype=torch.uint8,
                                device=x.device)
    if status is None:
        status = new_status(x.device)
    _check("ll_linear", lib.ll_linear(_ptr(x), _ptr(w), _ptr(y), m, n, k, _ptr(workspace),
                                      workspace.numel(), _ptr(status), _stream(stream)))
    return y


class trace:
    """Context manager over ll_trace_begin/ll_trace_end: records every kernel launch the
    library makes inside the block.  After the stream is synchronised, `launches()`
    returns [(kernel name, milliseconds), ...] in launch order."""

    def __init__(self, capacity=4096):
        self.capacity = capacity
        self.count = 0

    def __enter__(self):
        _check("ll_trace_begin", lib.ll_trace_begin(self.capacity))
        return self

    def __exit__(self, *exc):
        self.count = lib.ll_trace_end()
        return False

    def launches(self):
        return [(lib.ll_trace_name(i).decode(), lib.ll_trace_elapsed_ms(i)) for i in range(self.count)]
