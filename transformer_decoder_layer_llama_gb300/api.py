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
    I64 = ctypes.c_int64
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


def _need(t, name, dtype, device=True, shape=None):
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
    if t.numel() < 1:
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
