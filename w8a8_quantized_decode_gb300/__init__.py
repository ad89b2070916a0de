"""Python binding of liba8w8.so, the GB300 A8W8 decode library.

Argument marshalling only: every operation runs in the CUDA kernels behind the
C ABI declared in include/a8w8.h, with the same entry-point names. PyTorch
supplies device memory and streams. BF16 tensors are passed as
``torch.bfloat16``; all tensors must be contiguous CUDA tensors. A call runs on
``stream`` (None: the current stream), in order with that stream's work only;
tensors that it shares with other streams are the caller's to order, as with
torch's own operators.

There is no CPU fallback: if the library is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liba8w8.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "a8w8.h")

_lock = threading.Lock()
_lib = None

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_BOUNDS, ERR_WORKSPACE, ERR_CUDA = 0, -1, -2, -3, -4, -5
FLAG_PERSISTENT_STEP = 0x1
DEVERR_SLOT, DEVERR_BLOCK, DEVERR_CTX, DEVERR_TOKEN, DEVERR_POS = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_ROW, DEVERR_PAGES, DEVERR_ALIAS = 0x40, 0x80, 0x100


class A8W8Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"a8w8 status {status}: {msg}")
        self.status = status


_p = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t


class Config(ctypes.Structure):
    _fields_ = [("hidden", _i), ("num_q_heads", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("intermediate", _i), ("num_layers", _i), ("vocab", _i), ("page_size", _i),
                ("down_k_splits", _i), ("rms_eps", _f), ("flags", _i)]


WEIGHT_FIELDS = ("input_norm_w", "w_qkv", "s_qkv", "q_norm_w", "k_norm_w", "w_o", "s_o",
                 "post_norm_w", "w_gate_up", "s_gate_up", "w_down", "s_down")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, _p) for n in WEIGHT_FIELDS]


BF16_WEIGHT_FIELDS = ("input_norm_w", "w_qkv", "q_norm_w", "k_norm_w", "w_o", "post_norm_w",
                      "w_gate_up", "w_down")


class Bf16LayerWeights(ctypes.Structure):
    _fields_ = [(n, _p) for n in BF16_WEIGHT_FIELDS]


class Model(ctypes.Structure):
    _fields_ = [("embed", _p), ("layers", _p), ("final_norm_w", _p), ("lm_head", _p)]


TAP_FIELDS = ("xn", "xq", "xs", "qkv", "q_rot", "k_rot", "attn", "aq", "as", "h1", "hn", "hq",
              "hs", "act", "actq", "acts")


class LayerTaps(ctypes.Structure):
    _fields_ = [(n, _p) for n in TAP_FIELDS]


_SIGNATURES = {
    "a8w8_last_error": (ctypes.c_char_p, []),
    "a8w8_version": (_i, []),
    "a8w8_read_device_errors": (_i, [ctypes.POINTER(ctypes.c_uint), _p]),
    "a8w8_quant_rows": (_i, [_p, _i, _i, _i, _p, _p, _p]),
    "a8w8_linear": (_i, [_p, _p, _i, _i, _p, _p, _i, _i, _p, _p, _p, _p]),
    "a8w8_gate_up_swiglu": (_i, [_p, _p, _i, _i, _p, _p, _i, _p, _p, _p]),
    "a8w8_matmul_i8": (_i, [_p, _i, _i, _p, _i, _i, _i, _p, _p, _p]),
    "a8w8_rmsnorm_gate_up_swiglu": (_i, [_p, _i, _i, _p, _f, _p, _p, _i, _p, _p]),
    "paged_kv_write": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _i, _i, _p]),
    "paged_decode_attention_bf16": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _p,
                                         _p, _sz, _p]),
    "a8w8_attention_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "paged_decode_attention_bf16_noalloc": (_i, [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                                 _f, _p, _p]),
    "paged_kv_write_i8": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _i, _i, _p]),
    "paged_decode_attention_i8kv": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                         _f, _p, _p, _sz, _p]),
    "a8w8_decode_layer_i8kv": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p, _i,
                                    _p, _sz, _p, _p]),
    "a8w8_prefill_layer_i8kv": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p, _i,
                                     _p, _sz, _p, _p]),
    "a8w8_decode_step_i8kv": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p, _i, _p,
                                   _p, _p, _p, _sz, _p]),
    "a8w8_prefill_step": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _i, _i, _p, _p, _p,
                               _p, _sz, _p]),
    "paged_kv_write_i4": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _p, _p, _i, _i, _p]),
    "paged_kv_read_i4": (_i, [_p, _p, _p, _p, _i, _i, _p, _i, _i, _i, _p, _p, _p]),
    "paged_decode_attention_i4kv": (_i, [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                         _f, _p, _p, _sz, _p]),
    "a8w8_attention_i4_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "paged_kv_append": (_i, [_p, _i, _i, _i, _i, _i, _p, _p, _f, _p, _p, _i, _p, _p, _p, _p, _i, _i,
                             _p]),
    "paged_kv_append_i8": (_i, [_p, _i, _i, _i, _i, _i, _p, _p, _f, _p, _p, _i, _p, _p, _p, _p, _p, _p,
                                _i, _i, _p]),
    "paged_kv_append_i4": (_i, [_p, _i, _i, _i, _i, _i, _p, _p, _f, _p, _p, _i, _p, _p, _p, _p, _p, _p,
                                _i, _i, _p]),
    "paged_chunk_attention_bf16": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                                        _p, _p, _sz, _p]),
    "paged_chunk_attention_i8kv": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                        _i, _f, _p, _p, _sz, _p]),
    "paged_chunk_attention_i4kv": (_i, [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                        _i, _f, _p, _p, _sz, _p]),
    "a8w8_chunk_attention_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "a8w8_pages_workspace_bytes": (_sz, [_i, _i, _i]),
    "paged_copy_pages": (_i, [_p, _p, _i, _i, _p, _p, _i, _p]),
    "paged_fork": (_i, [_p, _p, _i, _i, _i, _p, _p, _p, _i, _i, _p, _p, _i, _p, _sz, _p]),
    "paged_reserve": (_i, [_p, _p, _i, _i, _i, _i, _p, _p, _i, _p, _sz, _p]),
    "paged_free": (_i, [_p, _p, _p, _i, _i, _i, _p, _i, _p]),
    "paged_compact": (_i, [_p, _p, _i, _i, _p, _p, _i, _i, _p, _p, _sz, _p]),
    "bf16_linear": (_i, [_p, _i, _i, _p, _i, _p, _p, _p]),
    "bf16_gate_up_swiglu": (_i, [_p, _i, _i, _p, _i, _p, _p]),
    "bf16_decode_layer": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _i, _p, _sz, _p,
                               _p]),
    "a8w8_rope_table": (_i, [_p, _i, _i, ctypes.c_double, _p]),
    "a8w8_workspace_bytes": (_sz, [_p, _i, _i]),
    "a8w8_sample_workspace_bytes": (_sz, [_i, _i]),
    "a8w8_sample": (_i, [_p, _i, _i, _i, _f, _f, ctypes.c_uint64, ctypes.c_uint64, _p, _p, _sz,
                         _p]),
    "a8w8_decode_layer": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _i, _p, _sz, _p,
                               _p]),
    "a8w8_prefill_layer": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _i, _p, _sz, _p,
                                _p]),
    "a8w8_decode_step": (_i, [_p, _p, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _i, _p, _p, _p, _p,
                              _sz, _p]),
    "a8w8_step_graph_create": (_i, [ctypes.POINTER(_p), _p, _p, _i, _i, _i, _p, _p, _p, _i, _p,
                                    _p, _p, _p, _p, _p, _p, _i, _p, _sz, _p]),
    "a8w8_step_graph_create_sampled": (_i, [ctypes.POINTER(_p), _p, _p, _i, _i, _i, _p, _p, _p,
                                            _i, _p, _p, _p, _p, _p, _p, _p, _i, _f, _f,
                                            ctypes.c_uint64, _p, _p, _sz, _p, _sz, _p]),
    "a8w8_step_graph_launch": (_i, [_p, _p]),
    "a8w8_step_graph_run_host": (_i, [_p, _p, _p, _p, _p, _p, _p]),
    "a8w8_step_graph_destroy": (None, [_p]),
}


def header_functions() -> list[str]:
    """Names of the functions include/a8w8.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\**\s*([A-Za-z_][A-Za-z0-9_]*)\s*\(",
                       text, flags=re.M)
    return [n for n in names if n not in ("if", "while")]


def build(force: bool = False) -> str:
    from . import builder
    return builder.build(force=force)


def lib():
    """Load liba8w8.so (raises if it is missing; it is never bypassed)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise A8W8Error(ERR_CUDA, f"{LIB_PATH} is missing: run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def last_error() -> str:
    return lib().a8w8_last_error().decode()


def _check(status: int):
    if status != OK:
        raise A8W8Error(status, last_error())


# ---------------------------------------------------------------------------
# torch plumbing
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors"
    return t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _alloc(make, stream):
    """The tensor that make() allocates, for a call on `stream`. A given stream's memory comes from
    that stream's own pool: what the current stream gave back last may still be read or written by
    kernels queued there, for which `stream` does not wait. The current stream, where the caller goes
    on to use the tensor, is recorded as a user of it, so that its memory is not handed out again
    before that stream is done."""
    if stream is None:
        return make()
    torch = _torch()
    current = torch.cuda.current_stream()
    if stream.cuda_stream == current.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(current)
    return t


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor for a call on `stream`."""
    return _alloc(lambda: _torch().empty(shape, dtype=dtype, device=device), stream)


def make_config(cfg: dict) -> Config:
    return Config(cfg["hidden"], cfg["num_q_heads"], cfg["num_kv_heads"], cfg["head_dim"],
                  cfg["intermediate"], cfg.get("num_layers", 1), cfg.get("vocab", 0),
                  cfg["page_size"], cfg.get("down_k_splits", 2), cfg["rms_eps"],
                  cfg.get("flags", 0))


def layer_struct(w: dict) -> LayerWeights:
    s = LayerWeights()
    for n in WEIGHT_FIELDS:
        setattr(s, n, _ptr(w[n]))
    return s


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def version() -> int:
    return lib().a8w8_version()


def read_device_errors(stream=None) -> int:
    bits = ctypes.c_uint(0)
    _check(lib().a8w8_read_device_errors(ctypes.byref(bits), _stream(stream)))
    return bits.value


def a8w8_quant_rows(x, stream=None):
    torch = _torch()
    rows, cols = x.shape
    q = _empty((rows, cols), torch.int8, x.device, stream)
    s = _empty((rows,), torch.float32, x.device, stream)
    _check(lib().a8w8_quant_rows(_ptr(x), rows, cols, cols, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def a8w8_linear(xq, x_scale, W, w_scale, k_splits=1, residual=None, acc_out=False, out=None,
                stream=None):
    torch = _torch()
    M, K = xq.shape
    N = W.shape[0]
    y = out if out is not None else _empty((M, N), torch.bfloat16, xq.device, stream)
    acc = _empty((M, N), torch.int32, xq.device, stream) if acc_out else None
    _check(lib().a8w8_linear(_ptr(xq), _ptr(x_scale), M, K, _ptr(W), _ptr(w_scale), N, k_splits,
                             _ptr(residual), _ptr(y), _ptr(acc), _stream(stream)))
    return (y, acc) if acc_out else y


def a8w8_gate_up_swiglu(xq, x_scale, W_gu, s_gu, acc_out=False, stream=None):
    torch = _torch()
    M, K = xq.shape
    I = W_gu.shape[0] // 2
    act = _empty((M, I), torch.bfloat16, xq.device, stream)
    acc = _empty((M, 2 * I), torch.int32, xq.device, stream) if acc_out else None
    _check(lib().a8w8_gate_up_swiglu(_ptr(xq), _ptr(x_scale), M, K, _ptr(W_gu), _ptr(s_gu), I,
                                     _ptr(act), _ptr(acc), _stream(stream)))
    return (act, acc) if acc_out else act


def a8w8_matmul_i8(xq, W, k0=0, k1=None, out=None, scratch=None, stream=None):
    """Exact INT32 product on the tensor cores: xq [M, K] int8 . W [N, K]^T
    over K columns [k0, k1) -> [M, N] int32. `scratch` (>= 2 M K bytes on the
    device) receives the FP16 images of xq; allocated when not given."""
    torch = _torch()
    M, K = xq.shape
    N = W.shape[0]
    k1 = K if k1 is None else k1
    acc = out if out is not None else _empty((M, N), torch.int32, xq.device, stream)
    if scratch is None:
        scratch = _empty((max(M * K, 1),), torch.float16, xq.device, stream)
    _check(lib().a8w8_matmul_i8(_ptr(xq), M, K, _ptr(W), N, int(k0), int(k1), _ptr(acc),
                                _ptr(scratch), _stream(stream)))
    return acc


def a8w8_rmsnorm_gate_up_swiglu(x, norm_w, eps, W_gu, s_gu, out=None, stream=None):
    """Post-attention RMSNorm + per-row quantisation + fused Gate/Up + SwiGLU
    of x [M, K] bf16 in one kernel: W_gu [2I, K] int8 -> act [M, I] bf16."""
    torch = _torch()
    M, K = x.shape
    I = W_gu.shape[0] // 2
    act = out if out is not None else _empty((M, I), torch.bfloat16, x.device, stream)
    _check(lib().a8w8_rmsnorm_gate_up_swiglu(_ptr(x), M, K, _ptr(norm_w), float(eps), _ptr(W_gu),
                                             _ptr(s_gu), I, _ptr(act), _stream(stream)))
    return act


def paged_kv_write(k, v, slot_mapping, k_cache, v_cache, page_size, stream=None):
    T, Hkv, D = k.shape
    num_blocks = k_cache.numel() // (Hkv * D * page_size)
    _check(lib().paged_kv_write(_ptr(k), _ptr(v), T, Hkv, D, _ptr(slot_mapping), _ptr(k_cache),
                                _ptr(v_cache), num_blocks, page_size, _stream(stream)))


def attention_workspace_bytes(B, Hq, D, max_ctx) -> int:
    return lib().a8w8_attention_workspace_bytes(B, Hq, D, max_ctx)


def paged_decode_attention_bf16(q, k_cache, v_cache, block_table, ctx_lens, page_size,
                                softmax_scale=None, ws=None, out=None, stream=None):
    torch = _torch()
    B, Hq, D = q.shape
    Hkv = k_cache.shape[-2]
    num_blocks = k_cache.numel() // (Hkv * D * page_size)
    max_blocks = block_table.shape[1]
    scale = (1.0 / D ** 0.5) if softmax_scale is None else softmax_scale
    need = attention_workspace_bytes(B, Hq, D, max_blocks * page_size)
    if ws is None and need:
        ws = _empty(need, torch.uint8, q.device, stream)
    o = out if out is not None else _alloc(lambda: _torch().empty_like(q), stream)
    _check(lib().paged_decode_attention_bf16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), B, Hq, Hkv, D,
        page_size, max_blocks, num_blocks, scale, _ptr(o), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream)))
    return o


NOALLOC_SCRATCH_BYTES = 8 << 20


def paged_decode_attention_bf16_noalloc(q, k_cache, v_cache, block_table, ctx_lens, page_size,
                                        softmax_scale=None, out=None, stream=None):
    """Decode attention for callers that cannot allocate device memory.

    Same result as paged_decode_attention_bf16, with the split-KV partials in
    the library's built-in 8 MiB device scratch instead of a caller workspace.
    The first call on a device looks up that scratch's address (make it before
    any stream capture); calls that overlap on the GPU share the scratch and
    race, so serialise them."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[-2]
    num_blocks = k_cache.numel() // (Hkv * D * page_size)
    scale = (1.0 / D ** 0.5) if softmax_scale is None else softmax_scale
    o = out if out is not None else _alloc(lambda: _torch().empty_like(q), stream)
    _check(lib().paged_decode_attention_bf16_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), B, Hq, Hkv, D,
        page_size, block_table.shape[1], num_blocks, scale, _ptr(o), _stream(stream)))
    return o


def a8w8_rope_table(max_pos, D, theta, device="cuda", stream=None):
    torch = _torch()
    t = _empty((max_pos, 2 * D), torch.float32, device, stream)
    _check(lib().a8w8_rope_table(_ptr(t), max_pos, D, float(theta), _stream(stream)))
    return t


def a8w8_sample(logits, temperature: float, top_p: float, seed: int, step: int, out=None,
                ws=None, stream=None):
    """Next tokens [B] int32 from logits [B, V] float32 on the device:
    temperature <= 0 is greedy; otherwise a top-p nucleus draw by the
    Gumbel-max rule with Philox4x32-10 noise keyed by (seed, step)."""
    torch = _torch()
    B, V = logits.shape
    o = out if out is not None else _empty(B, torch.int32, logits.device, stream)
    need = lib().a8w8_sample_workspace_bytes(B, V)
    if ws is None:
        ws = _empty(need, torch.uint8, logits.device, stream)
    _check(lib().a8w8_sample(_ptr(logits), B, V, logits.stride(0), float(temperature), float(top_p),
                             int(seed) & (2 ** 64 - 1), int(step) & (2 ** 64 - 1), _ptr(o), _ptr(ws),
                             0 if ws is None else ws.numel(), _stream(stream)))
    return o


def workspace_bytes(cfg: dict, max_B: int, max_blocks: int) -> int:
    c = make_config(cfg)
    return lib().a8w8_workspace_bytes(ctypes.byref(c), max_B, max_blocks)


def alloc_workspace(cfg: dict, max_B: int, max_blocks: int, device="cuda"):
    torch = _torch()
    return torch.empty(workspace_bytes(cfg, max_B, max_blocks), dtype=torch.uint8, device=device)


def make_taps(cfg: dict, B: int, device="cuda") -> dict:
    torch = _torch()
    H, Hq, Hkv, D, I = (cfg["hidden"], cfg["num_q_heads"], cfg["num_kv_heads"], cfg["head_dim"],
                        cfg["intermediate"])
    bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    shapes = {"xn": (bf, (B, H)), "hn": (bf, (B, H)), "xq": (i8, (B, H)), "xs": (f32, (B,)), "qkv": (bf, (B, (Hq + 2 * Hkv) * D)),
              "q_rot": (bf, (B, Hq, D)), "k_rot": (bf, (B, Hkv, D)), "attn": (bf, (B, Hq * D)),
              "aq": (i8, (B, Hq * D)), "as": (f32, (B,)), "h1": (bf, (B, H)),
              "hq": (i8, (B, H)), "hs": (f32, (B,)), "act": (bf, (B, I)),
              "actq": (i8, (B, I)), "acts": (f32, (B,))}
    return {n: torch.zeros(s, dtype=dt, device=device) for n, (dt, s) in shapes.items()}


def a8w8_decode_layer(weights: dict, cfg: dict, hidden, slot_mapping, block_table, ctx_lens,
                      k_cache, v_cache, rope, ws, taps: dict | None = None, stream=None):
    """One decode layer; `hidden` [B, H] bf16 is updated in place."""
    B = hidden.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_cache.numel() // (Hkv * D * page)
    c = make_config(cfg)
    w = layer_struct(weights)
    t = None
    if taps is not None:
        t = LayerTaps()
        for n in TAP_FIELDS:
            setattr(t, n, _ptr(taps.get(n)))
    _check(lib().a8w8_decode_layer(
        ctypes.byref(w), ctypes.byref(c), B, _ptr(hidden), _ptr(slot_mapping), _ptr(block_table),
        block_table.shape[1], num_blocks, _ptr(ctx_lens), _ptr(k_cache), _ptr(v_cache),
        _ptr(rope), rope.shape[0], _ptr(ws), ws.numel(),
        None if t is None else ctypes.byref(t), _stream(stream)))


def paged_kv_write_i8(k, v, slot_mapping, k_codes, v_codes, k_scale, v_scale, page_size,
                      stream=None):
    """INT8 KV variant: quantise k, v [T, Hkv, D] bf16 row by row into codes
    [slots, Hkv, D] int8 and row scales [slots, Hkv] float32."""
    T, Hkv, D = k.shape
    num_blocks = k_codes.numel() // (Hkv * D * page_size)
    _check(lib().paged_kv_write_i8(_ptr(k), _ptr(v), T, Hkv, D, _ptr(slot_mapping),
                                   _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                                   num_blocks, page_size, _stream(stream)))


def paged_decode_attention_i8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, ctx_lens,
                                page_size, softmax_scale=None, ws=None, out=None, stream=None):
    """Decode attention over the INT8 KV cache (codes times row scales)."""
    torch = _torch()
    B, Hq, D = q.shape
    Hkv = k_codes.shape[-2]
    num_blocks = k_codes.numel() // (Hkv * D * page_size)
    max_blocks = block_table.shape[1]
    scale = (1.0 / D ** 0.5) if softmax_scale is None else softmax_scale
    need = attention_workspace_bytes(B, Hq, D, max_blocks * page_size)
    if ws is None and need:
        ws = _empty(need, torch.uint8, q.device, stream)
    o = out if out is not None else _alloc(lambda: _torch().empty_like(q), stream)
    _check(lib().paged_decode_attention_i8kv(
        _ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
        _ptr(ctx_lens), B, Hq, Hkv, D, page_size, max_blocks, num_blocks, scale, _ptr(o),
        _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return o


def a8w8_decode_layer_i8kv(weights: dict, cfg: dict, hidden, slot_mapping, block_table, ctx_lens,
                           k_codes, v_codes, k_scale, v_scale, rope, ws,
                           taps: dict | None = None, stream=None):
    """One decode layer over an INT8 KV cache; `hidden` [B, H] bf16 is updated
    in place, the codes and row scales at the rows' slots are written."""
    B = hidden.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_codes.numel() // (Hkv * D * page)
    c = make_config(cfg)
    w = layer_struct(weights)
    t = None
    if taps is not None:
        t = LayerTaps()
        for n in TAP_FIELDS:
            setattr(t, n, _ptr(taps.get(n)))
    _check(lib().a8w8_decode_layer_i8kv(
        ctypes.byref(w), ctypes.byref(c), B, _ptr(hidden), _ptr(slot_mapping), _ptr(block_table),
        block_table.shape[1], num_blocks, _ptr(ctx_lens), _ptr(k_codes), _ptr(v_codes),
        _ptr(k_scale), _ptr(v_scale), _ptr(rope), rope.shape[0], _ptr(ws), ws.numel(),
        None if t is None else ctypes.byref(t), _stream(stream)))


def a8w8_prefill_layer_i8kv(weights: dict, cfg: dict, hidden, slot_mapping, block_table, ctx_lens,
                            k_codes, v_codes, k_scale, v_scale, rope, ws,
                            taps: dict | None = None, stream=None):
    """One layer over a prefill chunk of M rows with the INT8 KV cache (rows as
    a8w8_prefill_layer); `hidden` [M, H] bf16 is updated in place."""
    M = hidden.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_codes.numel() // (Hkv * D * page)
    c = make_config(cfg)
    w = layer_struct(weights)
    t = None
    if taps is not None:
        t = LayerTaps()
        for n in TAP_FIELDS:
            setattr(t, n, _ptr(taps.get(n)))
    _check(lib().a8w8_prefill_layer_i8kv(
        ctypes.byref(w), ctypes.byref(c), M, _ptr(hidden), _ptr(slot_mapping), _ptr(block_table),
        block_table.shape[1], num_blocks, _ptr(ctx_lens), _ptr(k_codes), _ptr(v_codes),
        _ptr(k_scale), _ptr(v_scale), _ptr(rope), rope.shape[0], _ptr(ws), ws.numel(),
        None if t is None else ctypes.byref(t), _stream(stream)))


def _refuse(what, dtype, numel):
    raise A8W8Error(ERR_INVALID_ARG, f"{what}: need a contiguous {dtype} tensor on the current "
                    f"CUDA device" + (f" of {numel} elements" if numel is not None else ""))


def _typed(t, dtype, what, dev, numel=None):
    """Device pointer of t after checks of its type, device (the current one, by index) and,
    where given, size: the 4-bit and page entries index with these tensors, so a wrong one is
    refused here."""
    if t is None or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or \
            (numel is not None and t.numel() != numel):
        _refuse(what, dtype, numel)
    return t.data_ptr()


class _HostPath:
    """What a call of the 4-bit and page entries asks torch for between two kernel launches: the
    current device, its stream's handle, and uninitialised bf16 rows. torch's own generated code has
    entries for these that cost the host 0.1, 0.1 and 0.9 us where the public ones cost 0.2, 1.1 to
    2.9 and 1.3 to 3.3 (write and read of one token: 18.5 us a pass, 35 by the public ones). They are
    not part of its interface, so each is tried once, and the public way stands in where it is not
    what it was."""

    def __init__(self, torch):
        own = getattr(torch, "_C", None)

        def public_stream(dev):
            return torch.cuda.current_stream(dev).cuda_stream

        def public_rows(shape, strides, dtype):
            return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")

        self._rows = public_rows
        try:
            f = own._dynamo.guards._empty_strided_cuda
            t = f((2, 3, 4), (12, 4, 1), torch.bfloat16)
            if t.dtype is torch.bfloat16 and tuple(t.shape) == (2, 3, 4) and t.is_contiguous() and \
                    t.get_device() == torch.cuda.current_device():
                self._rows = f
        except Exception:
            pass
        self.stream = public_stream
        try:
            f = own._cuda_getCurrentRawStream
            if f(torch.cuda.current_device()) == torch.cuda.current_stream().cuda_stream:
                self.stream = f
        except Exception:
            pass
        self.device = torch.cuda.current_device
        try:
            f = own._cuda_getDevice
            if f() == torch.cuda.current_device():
                self.device = f
        except Exception:
            pass
        self._bf16 = torch.bfloat16

    def rows(self, a, b, c, stream):
        """An uninitialised bf16 tensor [a, b, c] on the current CUDA device, for a call on
        `stream`."""
        if stream is None:
            return self._rows((a, b, c), (b * c, c, 1), self._bf16)
        return _alloc(lambda: self._rows((a, b, c), (b * c, c, 1), self._bf16), stream)


_host_path = None


def _host():
    global _host_path
    if _host_path is None:
        _host_path = _HostPath(_torch())
    return _host_path


def _device() -> int:
    """Index of the current CUDA device."""
    return (_host_path or _host()).device()


def _raw_stream(stream, dev):
    """The cudaStream_t of `stream`, or of the current stream of device dev."""
    return (_host_path or _host()).stream(dev) if stream is None else stream.cuda_stream


def _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, D, page_size, what, dev):
    """Pointers and page count of a 4-bit cache: codes [slots, Hkv, D / 2] uint8 and (s, m)
    pairs [slots, Hkv, 2] bfloat16, in whole pages."""
    torch = _torch()
    u8, bf = torch.uint8, torch.bfloat16
    pairs = k_meta.numel()
    slots = pairs // (2 * Hkv) if Hkv > 0 else -1
    codes = slots * Hkv * D // 2
    if slots < 0 or page_size <= 0 or slots % page_size or pairs != slots * Hkv * 2 or \
            v_meta.numel() != pairs or k_codes.numel() != codes or v_codes.numel() != codes:
        raise A8W8Error(ERR_INVALID_ARG, f"{what}: codes [slots, {Hkv}, {D // 2}] and meta "
                        f"[slots, {Hkv}, 2] of whole pages of {page_size} tokens expected")
    if not (k_codes.dtype is v_codes.dtype is u8 and k_meta.dtype is v_meta.dtype is bf
            and k_codes.get_device() == v_codes.get_device() == dev
            and k_meta.get_device() == v_meta.get_device() == dev
            and k_codes.is_contiguous() and v_codes.is_contiguous()
            and k_meta.is_contiguous() and v_meta.is_contiguous()):
        _refuse(what, f"{u8} (codes), {bf} (meta)", None)
    return (k_codes.data_ptr(), v_codes.data_ptr(), k_meta.data_ptr(),
            v_meta.data_ptr()), slots // page_size


def paged_kv_write_i4(k, v, slot_mapping, k_codes, v_codes, k_meta, v_meta, page_size,
                      stream=None):
    """4-bit KV variant: quantise k, v [T, Hkv, D] bf16 row by row into codes
    [slots, Hkv, D / 2] uint8 and (s, m) pairs [slots, Hkv, 2] bf16."""
    torch = _torch()
    what, dev = "paged_kv_write_i4", _device()
    T, Hkv, D = k.shape
    ptrs, num_blocks = _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, D, page_size, what, dev)
    _check(lib().paged_kv_write_i4(
        _typed(k, torch.bfloat16, what, dev), _typed(v, torch.bfloat16, what, dev, T * Hkv * D), T,
        Hkv, D, _typed(slot_mapping, torch.int32, what, dev, T), *ptrs, num_blocks, page_size,
        _raw_stream(stream, dev)))


def paged_kv_read_i4(k_codes, v_codes, k_meta, v_meta, slot_mapping, page_size, out=None,
                     stream=None):
    """The rows at slot_mapping [T] of a 4-bit cache as k, v [T, Hkv, D] bf16 (zeros where the
    slot is negative); `out` may give the pair of tensors to fill."""
    torch = _torch()
    what, dev = "paged_kv_read_i4", _device()
    Hkv, D = k_codes.shape[-2], 2 * k_codes.shape[-1]
    T = slot_mapping.numel()
    ptrs, num_blocks = _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, D, page_size, what, dev)
    if out is None:
        h = _host()
        k, v = h.rows(T, Hkv, D, stream), h.rows(T, Hkv, D, stream)
        kv = k.data_ptr(), v.data_ptr()
    else:
        k, v = out
        kv = (_typed(k, torch.bfloat16, what, dev, T * Hkv * D),
              _typed(v, torch.bfloat16, what, dev, T * Hkv * D))
    _check(lib().paged_kv_read_i4(
        *ptrs, num_blocks, page_size, _typed(slot_mapping, torch.int32, what, dev, T), T, Hkv, D,
        *kv, _raw_stream(stream, dev)))
    return k, v


def attention_i4_workspace_bytes(B, Hq, Hkv, D, max_ctx) -> int:
    return lib().a8w8_attention_i4_workspace_bytes(B, Hq, Hkv, D, max_ctx)


def paged_decode_attention_i4kv(q, k_codes, v_codes, k_meta, v_meta, block_table, ctx_lens,
                                page_size, softmax_scale=None, ws=None, out=None, stream=None):
    """Decode attention over the 4-bit KV cache (codes [slots, Hkv, D / 2] uint8 and (s, m)
    pairs [slots, Hkv, 2] bf16), in float32, narrowed to bf16 once."""
    torch = _torch()
    what, dev = "paged_decode_attention_i4kv", _device()
    B, Hq, D = q.shape
    Hkv = k_codes.shape[-2]
    ptrs, num_blocks = _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, D, page_size, what, dev)
    max_blocks = block_table.shape[-1]
    scale = (1.0 / D ** 0.5) if softmax_scale is None else softmax_scale
    L = lib()
    if ws is None:
        need = L.a8w8_attention_i4_workspace_bytes(B, Hq, Hkv, D, max_blocks * page_size)
        if need:
            ws = _empty(need, torch.uint8, q.device, stream)
    qp = _typed(q, torch.bfloat16, what, dev)
    o = _host().rows(B, Hq, D, stream) if out is None else out
    _check(L.paged_decode_attention_i4kv(
        qp, *ptrs,
        _typed(block_table, torch.int32, what, dev, B * max_blocks),
        _typed(ctx_lens, torch.int32, what, dev, B), B, Hq, Hkv, D, page_size, max_blocks,
        num_blocks, scale,
        o.data_ptr() if out is None else _typed(o, torch.bfloat16, what, dev, B * Hq * D),
        None if ws is None else _typed(ws, torch.uint8, what, dev), 0 if ws is None else ws.numel(),
        _raw_stream(stream, dev)))
    return o


def chunk_attention_workspace_bytes(T, B, Hq, Hkv, D, max_ctx) -> int:
    return lib().a8w8_chunk_attention_workspace_bytes(T, B, Hq, Hkv, D, max_ctx)


def _cache_rows(data, dtype, Hkv, D, page_size, what, dev):
    """Pointers and page count of K and V rows [slots, Hkv, D] in whole pages."""
    n = data[0].numel()
    if Hkv <= 0 or D <= 0 or page_size <= 0 or n % (Hkv * D * page_size) or data[1].numel() != n or \
            any(t.shape[-1] != D for t in data):
        raise A8W8Error(ERR_INVALID_ARG, f"{what}: caches [slots, {Hkv}, {D}] of whole pages of "
                        f"{page_size} tokens expected")
    return [_typed(t, dtype, what, dev) for t in data], n // (Hkv * D * page_size)


def _chunk_attention(what, entry, q, ptrs, num_blocks, Hkv, dev, block_table, ctx_lens, q_starts,
                     page_size, softmax_scale, ws, out, stream):
    torch = _torch()
    i32 = torch.int32
    T, Hq, D = q.shape
    B, max_blocks = block_table.shape
    scale = (1.0 / D ** 0.5) if softmax_scale is None else softmax_scale
    L = lib()
    if ws is None:
        need = L.a8w8_chunk_attention_workspace_bytes(T, B, Hq, Hkv, D, max_blocks * page_size)
        ws = _empty(max(need, 16), torch.uint8, q.device, stream)
    qp = _typed(q, torch.bfloat16, what, dev)
    o = _host().rows(T, Hq, D, stream) if out is None else out
    _check(getattr(L, entry)(
        qp, *ptrs, _typed(block_table, i32, what, dev), _typed(ctx_lens, i32, what, dev, B),
        _typed(q_starts, i32, what, dev, B + 1), T, B, Hq, Hkv, D, page_size, max_blocks, num_blocks,
        scale, o.data_ptr() if out is None else _typed(o, torch.bfloat16, what, dev, T * Hq * D),
        _typed(ws, torch.uint8, what, dev), ws.numel(), _raw_stream(stream, dev)))
    return o


def _kv_append(what, qkv, positions, slot_mapping, rope, ptrs, num_blocks, page_size, Hkv, D, q_norm_w,
               k_norm_w, eps, q_out, stream, dev):
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    if qkv.dim() != 2 or qkv.dtype is not bf or qkv.get_device() != dev or qkv.stride(1) != 1:
        raise A8W8Error(ERR_INVALID_ARG, f"{what}: qkv is a [T, (Hq + 2 Hkv) D] {bf} tensor on the "
                        "current CUDA device, contiguous along its rows")
    T, cols = qkv.shape
    heads = cols // D
    Hq = heads - 2 * Hkv
    if cols % D or Hq < 0:
        raise A8W8Error(ERR_INVALID_ARG, f"{what}: rows of {cols} elements are not Hq + 2 x {Hkv} "
                        f"heads of {D}")
    ld = qkv.stride(0) if T > 1 else cols
    if ld >= 2 ** 31:
        raise A8W8Error(ERR_UNSUPPORTED_SHAPE, f"{what}: rows {ld} elements apart, 2^31 - 1 at most")
    if rope.dim() != 2 or rope.shape[1] != 2 * D:
        raise A8W8Error(ERR_INVALID_ARG, f"{what}: the rope table is [max_pos, {2 * D}]")
    if q_out is None:
        q_out = _host().rows(T, Hq, D, stream)
        qp = q_out.data_ptr()
    else:
        qp = _typed(q_out, bf, what, dev, T * Hq * D)
    norms = [None if w is None else _typed(w, bf, what, dev, D) for w in (q_norm_w, k_norm_w)]
    _check(getattr(lib(), what)(
        qkv.data_ptr(), T, Hq, Hkv, D, ld, *norms, eps, _typed(positions, i32, what, dev, T),
        _typed(rope, torch.float32, what, dev), rope.shape[0], _typed(slot_mapping, i32, what, dev, T),
        qp if T * Hq else None, *ptrs, num_blocks, page_size, _raw_stream(stream, dev)))
    return q_out


def paged_kv_append(qkv, positions, slot_mapping, rope, k_cache, v_cache, page_size, q_norm_w=None,
                    k_norm_w=None, eps=1e-6, q_out=None, stream=None):
    """A chunk's fused QKV rows [T, (Hq + 2 Hkv) D] bf16 (rows may be strided) past the per-head norm
    (where a weight is given) and the rotation at positions [T] int32: queries to the returned
    q_rot [T, Hq, D], keys and values to slot_mapping [T] int32 of the BF16 cache. `rope` is
    a8w8_rope_table's."""
    what, dev = "paged_kv_append", _device()
    Hkv, D = k_cache.shape[-2:]
    ptrs, num_blocks = _cache_rows((k_cache, v_cache), _torch().bfloat16, Hkv, D, page_size, what, dev)
    return _kv_append(what, qkv, positions, slot_mapping, rope, ptrs, num_blocks, page_size, Hkv, D,
                      q_norm_w, k_norm_w, eps, q_out, stream, dev)


def paged_kv_append_i8(qkv, positions, slot_mapping, rope, k_codes, v_codes, k_scale, v_scale, page_size,
                       q_norm_w=None, k_norm_w=None, eps=1e-6, q_out=None, stream=None):
    """paged_kv_append into the INT8 cache."""
    what, dev = "paged_kv_append_i8", _device()
    Hkv, D = k_codes.shape[-2:]
    ptrs, num_blocks = _cache_i8(k_codes, v_codes, k_scale, v_scale, Hkv, D, page_size, what, dev)
    return _kv_append(what, qkv, positions, slot_mapping, rope, ptrs, num_blocks, page_size, Hkv, D,
                      q_norm_w, k_norm_w, eps, q_out, stream, dev)


def paged_kv_append_i4(qkv, positions, slot_mapping, rope, k_codes, v_codes, k_meta, v_meta, page_size,
                       q_norm_w=None, k_norm_w=None, eps=1e-6, q_out=None, stream=None):
    """paged_kv_append into the 4-bit cache."""
    what, dev = "paged_kv_append_i4", _device()
    Hkv, D = k_codes.shape[-2], 2 * k_codes.shape[-1]
    ptrs, num_blocks = _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, D, page_size, what, dev)
    return _kv_append(what, qkv, positions, slot_mapping, rope, ptrs, num_blocks, page_size, Hkv, D,
                      q_norm_w, k_norm_w, eps, q_out, stream, dev)


def paged_chunk_attention_bf16(q, k_cache, v_cache, block_table, ctx_lens, q_starts, page_size,
                               softmax_scale=None, ws=None, out=None, stream=None):
    """Attention of a chunk over the paged BF16 cache: request b's rows q_starts[b] to
    q_starts[b + 1] - 1 of q [T, Hq, D] are the last tokens of its context, each seeing the tokens
    up to its own. Rows of no request are left as they are."""
    what, dev = "paged_chunk_attention_bf16", _device()
    Hkv = k_cache.shape[-2]
    ptrs, num_blocks = _cache_rows((k_cache, v_cache), _torch().bfloat16, Hkv, q.shape[-1],
                                   page_size, what, dev)
    return _chunk_attention(what, what, q, ptrs, num_blocks, Hkv, dev, block_table, ctx_lens,
                            q_starts, page_size, softmax_scale, ws, out, stream)


def _cache_i8(k_codes, v_codes, k_scale, v_scale, Hkv, D, page_size, what, dev):
    """Pointers and page count of an INT8 cache: codes [slots, Hkv, D] int8 and row scales
    [slots, Hkv] float32, in whole pages."""
    torch = _torch()
    ptrs, num_blocks = _cache_rows((k_codes, v_codes), torch.int8, Hkv, D, page_size, what, dev)
    n = num_blocks * page_size * Hkv
    return ptrs + [_typed(t, torch.float32, what, dev, n) for t in (k_scale, v_scale)], num_blocks


def paged_chunk_attention_i8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, ctx_lens, q_starts,
                               page_size, softmax_scale=None, ws=None, out=None, stream=None):
    """paged_chunk_attention_bf16 over the INT8 cache (codes times row scales)."""
    what, dev = "paged_chunk_attention_i8kv", _device()
    Hkv = k_codes.shape[-2]
    ptrs, num_blocks = _cache_i8(k_codes, v_codes, k_scale, v_scale, Hkv, q.shape[-1], page_size, what,
                                 dev)
    return _chunk_attention(what, what, q, ptrs, num_blocks, Hkv, dev, block_table, ctx_lens,
                            q_starts, page_size, softmax_scale, ws, out, stream)


def paged_chunk_attention_i4kv(q, k_codes, v_codes, k_meta, v_meta, block_table, ctx_lens, q_starts,
                               page_size, softmax_scale=None, ws=None, out=None, stream=None):
    """paged_chunk_attention_bf16 over the 4-bit cache (codes [slots, Hkv, D / 2] uint8 and (s, m)
    pairs [slots, Hkv, 2] bf16)."""
    what, dev = "paged_chunk_attention_i4kv", _device()
    Hkv = k_codes.shape[-2]
    ptrs, num_blocks = _cache_i4(k_codes, v_codes, k_meta, v_meta, Hkv, q.shape[-1], page_size, what,
                                 dev)
    return _chunk_attention(what, what, q, ptrs, num_blocks, Hkv, dev, block_table, ctx_lens,
                            q_starts, page_size, softmax_scale, ws, out, stream)


class PagePool:
    """The caches that share one page numbering (K and V of every layer, or codes and scales):
    each tensor of `caches` is num_blocks pages; at most 256 of them, each 16-byte aligned, with
    pages of a multiple of 4 bytes (for paged_fork of 4 bytes a token). Holds the caches and the
    arrays that the page operations take; pages and counts live in the caller's tensors:
    block_table [B, max_blocks], ctx_lens [B] and refcount [num_blocks], int32."""

    def __init__(self, caches, num_blocks: int, page_size: int):
        self.caches = list(caches)
        self.num_blocks, self.page_size = int(num_blocks), int(page_size)
        if self.num_blocks <= 0 or self.page_size <= 0 or not self.caches:
            raise A8W8Error(ERR_INVALID_ARG, "PagePool: caches, num_blocks and page_size expected")
        self.index = self.caches[0].get_device()
        ptrs, sizes = [], []
        for c in self.caches:
            size = c.numel() * c.element_size()
            if self.index < 0 or c.get_device() != self.index or not c.is_contiguous() or \
                    size % self.num_blocks:
                raise A8W8Error(ERR_INVALID_ARG, "PagePool: each cache is a contiguous CUDA tensor "
                                f"of {num_blocks} pages, all on one device")
            ptrs.append(c.data_ptr())
            sizes.append(size // self.num_blocks)
        self.device = self.caches[0].device
        n = len(ptrs)
        self._args = ((_p * n)(*ptrs), (_sz * n)(*sizes), n)
        # a copy of no pages: every rule that all page operations hold their caches to
        status = lib().paged_copy_pages(*self._args, self.num_blocks, None, None, 0, None)
        if status != OK:
            raise A8W8Error(status, last_error().replace("paged_copy_pages", "PagePool"))

    def _here(self, what) -> int:
        dev = _device()
        if dev != self.index:
            raise A8W8Error(ERR_INVALID_ARG, f"{what}: the pool is not on the current CUDA device")
        return dev

    def _tables(self, what, dev, block_table, refcount, ctx_lens=None):
        i32 = _torch().int32
        if block_table.dim() != 2:
            raise A8W8Error(ERR_INVALID_ARG, f"{what}: block_table is [B, max_blocks]")
        B, max_blocks = block_table.shape
        return (_typed(block_table, i32, what, dev),
                None if ctx_lens is None else _typed(ctx_lens, i32, what, dev, B),
                _typed(refcount, i32, what, dev, self.num_blocks), B, max_blocks)


def pages_workspace_bytes(num_blocks: int, B: int, n: int) -> int:
    return lib().a8w8_pages_workspace_bytes(num_blocks, B, n)


def _pages_ws(pool, B, n, ws, what, dev, stream):
    torch = _torch()
    if ws is None:
        need = pages_workspace_bytes(pool.num_blocks, B, n)
        ws = _empty(need, torch.uint8, pool.device, stream)
    return _typed(ws, torch.uint8, what, dev), ws.numel()


def paged_copy_pages(pool, src, dst, stream=None):
    """Copy page src[i] to page dst[i] (int32 [n] on the device) in every cache of the pool."""
    what = "paged_copy_pages"
    i32, dev, n = _torch().int32, pool._here(what), src.numel()
    _check(lib().paged_copy_pages(*pool._args, pool.num_blocks, _typed(src, i32, what, dev, n),
                                  _typed(dst, i32, what, dev, n), n, _raw_stream(stream, dev)))


def paged_fork(pool, block_table, ctx_lens, refcount, parents, children, ws=None, stream=None):
    """Fork row parents[i] into the free row children[i]: full pages shared, the page in
    progress copied. block_table, ctx_lens and refcount are updated in place."""
    what = "paged_fork"
    i32, dev, n = _torch().int32, pool._here(what), parents.numel()
    bt, cl, rc, B, max_blocks = pool._tables(what, dev, block_table, refcount, ctx_lens)
    _check(lib().paged_fork(*pool._args, pool.num_blocks, pool.page_size, bt, cl, rc, B,
                            max_blocks, _typed(parents, i32, what, dev, n),
                            _typed(children, i32, what, dev, n), n,
                            *_pages_ws(pool, B, n, ws, what, dev, stream), _raw_stream(stream, dev)))


def paged_reserve(pool, block_table, refcount, rows, tokens, ws=None, stream=None):
    """Give row rows[i] pages for tokens[i] tokens. block_table and refcount are updated in
    place."""
    what = "paged_reserve"
    i32, dev, n = _torch().int32, pool._here(what), rows.numel()
    bt, _, rc, B, max_blocks = pool._tables(what, dev, block_table, refcount)
    _check(lib().paged_reserve(bt, rc, B, max_blocks, pool.num_blocks, pool.page_size,
                               _typed(rows, i32, what, dev, n),
                               _typed(tokens, i32, what, dev, n), n,
                               *_pages_ws(pool, B, n, ws, what, dev, stream), _raw_stream(stream, dev)))


def paged_free(pool, block_table, ctx_lens, refcount, rows, stream=None):
    """Free the listed rows: their pages lose a reference, their table rows become -1, their
    contexts 0."""
    what = "paged_free"
    i32, dev, n = _torch().int32, pool._here(what), rows.numel()
    bt, cl, rc, B, max_blocks = pool._tables(what, dev, block_table, refcount, ctx_lens)
    _check(lib().paged_free(bt, cl, rc, B, max_blocks, pool.num_blocks,
                            _typed(rows, i32, what, dev, n), n, _raw_stream(stream, dev)))


def paged_compact(pool, block_table, refcount, num_live=None, ws=None, stream=None):
    """Move the live pages to the front of the pool; tables and counts follow. Returns num_live
    (int32 [1] on the device): pages from there on are free."""
    torch = _torch()
    what = "paged_compact"
    dev = pool._here(what)
    bt, _, rc, B, max_blocks = pool._tables(what, dev, block_table, refcount)
    if num_live is None:
        num_live = _empty(1, torch.int32, pool.device, stream)
    _check(lib().paged_compact(*pool._args, pool.num_blocks, bt, rc, B, max_blocks,
                               _typed(num_live, torch.int32, what, dev, 1),
                               *_pages_ws(pool, B, 0, ws, what, dev, stream), _raw_stream(stream, dev)))
    return num_live


def bf16_linear(x, W, residual=None, out=None, stream=None):
    """BF16 projection: bf16(x [M,K] . W [N,K]^T (+ residual)) -> [M, N]."""
    torch = _torch()
    M, K = x.shape
    N = W.shape[0]
    y = out if out is not None else _empty((M, N), torch.bfloat16, x.device, stream)
    _check(lib().bf16_linear(_ptr(x), M, K, _ptr(W), N, _ptr(residual), _ptr(y), _stream(stream)))
    return y


def bf16_gate_up_swiglu(x, W_gu, stream=None):
    """BF16 fused Gate/Up + SwiGLU: W_gu [2I, K] -> act [M, I]."""
    torch = _torch()
    M, K = x.shape
    I = W_gu.shape[0] // 2
    act = _empty((M, I), torch.bfloat16, x.device, stream)
    _check(lib().bf16_gate_up_swiglu(_ptr(x), M, K, _ptr(W_gu), I, _ptr(act), _stream(stream)))
    return act


def bf16_decode_layer(weights: dict, cfg: dict, hidden, slot_mapping, block_table, ctx_lens,
                      k_cache, v_cache, rope, ws, taps: dict | None = None, stream=None):
    """One BF16 (unquantised) decode layer; `hidden` [B, H] bf16 is updated in
    place; weights hold BF16_WEIGHT_FIELDS."""
    B = hidden.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_cache.numel() // (Hkv * D * page)
    c = make_config(cfg)
    w = Bf16LayerWeights()
    for n in BF16_WEIGHT_FIELDS:
        setattr(w, n, _ptr(weights[n]))
    t = None
    if taps is not None:
        t = LayerTaps()
        for n in TAP_FIELDS:
            setattr(t, n, _ptr(taps.get(n)))
    _check(lib().bf16_decode_layer(
        ctypes.byref(w), ctypes.byref(c), B, _ptr(hidden), _ptr(slot_mapping), _ptr(block_table),
        block_table.shape[1], num_blocks, _ptr(ctx_lens), _ptr(k_cache), _ptr(v_cache),
        _ptr(rope), rope.shape[0], _ptr(ws), ws.numel(),
        None if t is None else ctypes.byref(t), _stream(stream)))


def a8w8_prefill_layer(weights: dict, cfg: dict, hidden, slot_mapping, block_table, ctx_lens,
                       k_cache, v_cache, rope, ws, taps: dict | None = None, stream=None):
    """One layer over a prefill chunk of M token rows; `hidden` [M, H] bf16 is
    updated in place. Row r is the token at position ctx_lens[r] - 1 of the
    sequence whose block table row it carries; all rows' K/V are written
    before attention, so the chunk is causal."""
    M = hidden.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_cache.numel() // (Hkv * D * page)
    c = make_config(cfg)
    w = layer_struct(weights)
    t = None
    if taps is not None:
        t = LayerTaps()
        for n in TAP_FIELDS:
            setattr(t, n, _ptr(taps.get(n)))
    _check(lib().a8w8_prefill_layer(
        ctypes.byref(w), ctypes.byref(c), M, _ptr(hidden), _ptr(slot_mapping), _ptr(block_table),
        block_table.shape[1], num_blocks, _ptr(ctx_lens), _ptr(k_cache), _ptr(v_cache),
        _ptr(rope), rope.shape[0], _ptr(ws), ws.numel(),
        None if t is None else ctypes.byref(t), _stream(stream)))


class _ModelHandle:
    """Keeps the ctypes structs describing a model alive."""

    def __init__(self, model: dict, cfg: dict):
        L = cfg["num_layers"]
        self.layers = (LayerWeights * L)(*[layer_struct(model["layers"][i]) for i in range(L)])
        self.model = Model(_ptr(model["embed"]), ctypes.cast(self.layers, _p),
                           _ptr(model["final_norm_w"]), _ptr(model["lm_head"]))
        self.cfg = make_config(cfg)


def _cache_array(caches):
    return (_p * len(caches))(*[_ptr(c) for c in caches])


def a8w8_decode_step(model: dict, cfg: dict, token_ids, slot_mapping, block_table, ctx_lens,
                     k_caches, v_caches, rope, ws, next_tokens, logits=None, final_hidden=None,
                     stream=None):
    h = _ModelHandle(model, cfg)
    B = token_ids.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_caches[0].numel() // (Hkv * D * page)
    _check(lib().a8w8_decode_step(
        ctypes.byref(h.model), ctypes.byref(h.cfg), B, _ptr(token_ids), _ptr(slot_mapping),
        _ptr(block_table), block_table.shape[1], num_blocks, _ptr(ctx_lens),
        _cache_array(k_caches), _cache_array(v_caches), _ptr(rope), rope.shape[0],
        _ptr(next_tokens), _ptr(logits), _ptr(final_hidden), _ptr(ws), ws.numel(),
        _stream(stream)))


def a8w8_prefill_step(model: dict, cfg: dict, token_ids, slot_mapping, block_table, ctx_lens,
                      k_caches, v_caches, rope, ws, last_rows, next_tokens, logits=None,
                      stream=None):
    """The prompt rows (as a8w8_prefill_layer) through every layer, then the
    final norm, LM head and argmax on last_rows [S] -> next_tokens [S]."""
    h = _ModelHandle(model, cfg)
    M = token_ids.shape[0]
    S = last_rows.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_caches[0].numel() // (Hkv * D * page)
    _check(lib().a8w8_prefill_step(
        ctypes.byref(h.model), ctypes.byref(h.cfg), M, _ptr(token_ids), _ptr(slot_mapping),
        _ptr(block_table), block_table.shape[1], num_blocks, _ptr(ctx_lens),
        _cache_array(k_caches), _cache_array(v_caches), _ptr(rope), rope.shape[0], S,
        _ptr(last_rows), _ptr(next_tokens), _ptr(logits), _ptr(ws), ws.numel(), _stream(stream)))


def a8w8_decode_step_i8kv(model: dict, cfg: dict, token_ids, slot_mapping, block_table, ctx_lens,
                          k_codes, v_codes, k_scales, v_scales, rope, ws, next_tokens, logits=None,
                          final_hidden=None, stream=None):
    """One decode step over per-layer INT8 caches (lists of num_layers device
    tensors: codes [slots, Hkv, D] int8, row scales [slots, Hkv] float32)."""
    h = _ModelHandle(model, cfg)
    B = token_ids.shape[0]
    Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    num_blocks = k_codes[0].numel() // (Hkv * D * page)
    _check(lib().a8w8_decode_step_i8kv(
        ctypes.byref(h.model), ctypes.byref(h.cfg), B, _ptr(token_ids), _ptr(slot_mapping),
        _ptr(block_table), block_table.shape[1], num_blocks, _ptr(ctx_lens),
        _cache_array(k_codes), _cache_array(v_codes), _cache_array(k_scales),
        _cache_array(v_scales), _ptr(rope), rope.shape[0], _ptr(next_tokens), _ptr(logits),
        _ptr(final_hidden), _ptr(ws), ws.numel(), _stream(stream)))


class StepGraph:
    """A decode step captured once into a CUDA graph and replayed.

    The per-step inputs live in device tensors owned by this object:
    ``token_ids``, ``slot_mapping``, ``block_table``, ``ctx_lens`` (write them
    between replays) and ``next_tokens`` (read after a replay). With
    ``device_loop=True`` each replay also prepares the next step on the
    device (the drawn token fed back, context advanced by one token).

    ``sampling=dict(temperature=T, top_p=P, seed=S, step=s0)`` samples inside
    the graph (``a8w8_step_graph_create_sampled``): this object then owns the
    Philox step counter (``step_counter``, int64 [1], starting at s0 and
    advanced by each replay) and the sampling workspace, and ``logits`` is
    required."""

    def __init__(self, model: dict, cfg: dict, B: int, max_blocks: int, k_caches, v_caches, rope,
                 ws, logits=None, final_hidden=None, device_loop=False, stream=None,
                 sampling=None):
        torch = _torch()
        dev = k_caches[0].device
        self._h = _ModelHandle(model, cfg)
        self._keep = (model, k_caches, v_caches, rope, ws, logits, final_hidden)
        Hkv, D, page = cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
        num_blocks = k_caches[0].numel() // (Hkv * D * page)
        self.B, self.max_blocks = B, max_blocks
        i32 = torch.int32
        self.token_ids = torch.zeros(B, dtype=i32, device=dev)
        self.slot_mapping = torch.full((B,), -1, dtype=i32, device=dev)
        self.block_table = torch.zeros((B, max_blocks), dtype=i32, device=dev)
        self.ctx_lens = torch.zeros(B, dtype=i32, device=dev)
        self.next_tokens = torch.zeros(B, dtype=i32, device=dev)
        self._g = None
        g = _p()
        common = (ctypes.byref(g), ctypes.byref(self._h.model), ctypes.byref(self._h.cfg), B,
                  max_blocks, num_blocks, _cache_array(k_caches), _cache_array(v_caches),
                  _ptr(rope), rope.shape[0], _ptr(self.token_ids), _ptr(self.slot_mapping),
                  _ptr(self.block_table), _ptr(self.ctx_lens), _ptr(self.next_tokens),
                  _ptr(logits), _ptr(final_hidden), 1 if device_loop else 0)
        if sampling is None:
            _check(lib().a8w8_step_graph_create(*common, _ptr(ws), ws.numel(), _stream(stream)))
        else:
            if logits is None:
                raise ValueError("sampling inside the step needs a logits buffer")
            self.step_counter = torch.full((1,), int(sampling.get("step", 0)), dtype=torch.int64,
                                           device=dev)
            need = lib().a8w8_sample_workspace_bytes(B, cfg["vocab"])
            self._sample_ws = torch.empty(need, dtype=torch.uint8, device=dev)
            _check(lib().a8w8_step_graph_create_sampled(
                *common, float(sampling.get("temperature", 1.0)), float(sampling.get("top_p", 1.0)),
                int(sampling.get("seed", 0)) & (2 ** 64 - 1), _ptr(self.step_counter),
                _ptr(self._sample_ws),
                need, _ptr(ws), ws.numel(), _stream(stream)))
        self._g = g
        self._torch = torch

    def set_inputs(self, token_ids, slot_mapping, block_table, ctx_lens):
        self.token_ids.copy_(token_ids)
        self.slot_mapping.copy_(slot_mapping)
        self.block_table.copy_(block_table)
        self.ctx_lens.copy_(ctx_lens)

    def launch(self, stream=None):
        _check(lib().a8w8_step_graph_launch(self._g, _stream(stream)))

    def run_host(self, token_ids, slot_mapping, block_table, ctx_lens, next_tokens, stream=None):
        """Host (CPU, ideally pinned) int32 tensors in and out; synchronises."""
        for t in (token_ids, slot_mapping, block_table, ctx_lens, next_tokens):
            assert not t.is_cuda and t.is_contiguous() and t.dtype == self._torch.int32
        _check(lib().a8w8_step_graph_run_host(
            self._g, token_ids.data_ptr(), slot_mapping.data_ptr(), block_table.data_ptr(),
            ctx_lens.data_ptr(), next_tokens.data_ptr(), _stream(stream)))

    def close(self):
        if self._g:
            lib().a8w8_step_graph_destroy(self._g)
            self._g = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
