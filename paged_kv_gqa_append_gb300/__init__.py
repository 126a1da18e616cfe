"""Python binding of libpkv.so: paged GQA decode and fused RoPE + paged KV append.

The functions carry the C-ABI names and only marshal arguments: they check
dtypes, devices and shapes of torch tensors, pass raw pointers, sizes and the
current CUDA stream to the library, and raise ``PkvError`` on a non-zero
status.  Every step of the computation runs in the library's sm_103a kernels;
there is no fallback: the first call raises when libpkv.so is missing (build
it with ``python -m paged_kv_gqa_append_gb300.build``).  The calls that are
small enough for the host's time to count go through _calls.so first
(binding/calls.cpp), which does the same checks on the tensors in C++ and makes
the same C call; whatever it does not take as it is comes back to the functions
here, which say what is wrong or make the call.

Tensor layouts (see include/pkv.h):
    kv_pool       [num_pages, 2, 8, 16, 64] bf16   (K = 0, V = 1), 32 KiB/page
    block_tables  [num_seqs, >= max_blocks] int32  (-1 = no page)
    q / out       [num_seqs, 32, 64] bf16
    k / v         [T, 8, 64] bf16;  positions / token_seq [T] int32
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import re

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")
CALLS_PATH = os.path.join(_HERE, "_calls.so")

NUM_Q_HEADS = 32
NUM_KV_HEADS = 8
HEAD_DIM = 64
PAGE_TOKENS = 16
ROPE_PAIRS = 32

COMPUTE_TENSOR = 0
COMPUTE_FMA = 1
SCHEDULE_STATIC, SCHEDULE_DYNAMIC, SCHEDULE_AUTO = 0, 1, 2

STATUS = {
    0: "PKV_OK", 1: "PKV_ERR_INVALID_ARGUMENT", 2: "PKV_ERR_MISALIGNED",
    3: "PKV_ERR_UNSUPPORTED_SHAPE", 4: "PKV_ERR_WORKSPACE_TOO_SMALL", 5: "PKV_ERR_CUDA",
    6: "PKV_ERR_DEVICE_INDEX", 7: "PKV_ERR_POOL_EXHAUSTED", 8: "PKV_ERR_REQUEST_TOO_LARGE",
    9: "PKV_ERR_TIMEOUT",
}
OK, ERR_INVALID_ARGUMENT, ERR_DEVICE_INDEX, ERR_POOL_EXHAUSTED = 0, 1, 6, 7
ERR_REQUEST_TOO_LARGE, ERR_TIMEOUT = 8, 9


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


_p, _i, _f, _d, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
_ll = ctypes.c_longlong
_ip = ctypes.POINTER(ctypes.c_int)


class DecodeOpts(ctypes.Structure):
    _fields_ = [("compute", _i), ("min_units_per_warp", _i), ("ctas_per_sm", _i), ("stages", _i),
                ("warps_per_cta", _i), ("combine", _i), ("schedule", _i), ("early_kv", _i),
                ("wait_limit_ns", ctypes.c_longlong), ("expire_first_wait", _i)]


_SIGS = {
    "pkv_status_string": (ctypes.c_char_p, [_i]),
    "pkv_version": (_i, []),
    "pkv_last_error": (ctypes.c_char_p, []),
    "pkv_rope_inv_freq_plain": (_i, [_p, _d]),
    "pkv_rope_inv_freq_llama3": (_i, [_p, _d, _d, _d, _d, _i]),
    "pkv_rope_table_fill": (_i, [_p, _p, _i, _p]),
    "kv_append_rope": (_i, [_p, _p, _p, _p, _i, _p, _i, _i, _i, _p, _i, _p, _p, _i, _p, _p, _p, _p]),
    "paged_gqa_decode_workspace_bytes": (_sz, [_i]),
    "paged_gqa_prefill": (_i, [_p, _i, _p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _p]),
    "paged_gqa_prefill_ex": (_i, [_p, _i, _p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _p, _i]),
    "pkv_argmax_f32": (_i, [_p, _i, _i, ctypes.c_longlong, _p, _p]),
    "paged_gqa_decode": (_i, [_p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _sz, _p, _p]),
    "paged_gqa_decode_ex": (_i, [_p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _sz, _p, _p,
                                 ctypes.POINTER(DecodeOpts)]),
    "paged_gqa_decode_append": (_i, [_p, _p, _p, _p, _p, _i, _p, _i, _p, _i, _i, _p, _i, _i, _p, _p,
                                     _f, _p, _sz, _p, _p, ctypes.POINTER(DecodeOpts)]),
    "paged_gqa_decode_noalloc": (_i, [_p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _p]),
    "kv_append_rope_int8": (_i, [_p, _p, _p, _p, _i, _p, _i, _i, _i, _p, _i, _p, _p, _i, _p, _p, _p,
                                 _p]),
    "kv_append_rope_layers": (_i, [_p, _p, _i, _i, _p, _sz, _p, _p, _i, _p, ctypes.c_longlong, _i,
                                   _i, _i, _p, _i, _i, _p, _p, _i, _p, _p]),
    "paged_gqa_decode_int8": (_i, [_p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _sz, _p, _p]),
    "paged_gqa_decode_int8_ex": (_i, [_p, _p, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _sz, _p, _p,
                                      ctypes.POINTER(DecodeOpts)]),
    "paged_gqa_decode_append_int8": (_i, [_p, _p, _p, _p, _p, _i, _p, _i, _p, _i, _i, _p, _i, _i, _p,
                                          _p, _f, _p, _sz, _p, _p, ctypes.POINTER(DecodeOpts)]),
    "paged_gqa_decode_append_layers": (_i, [_p, _p, _p, _p, _p, _i, _i, _p, _p, _i, _p, _i, _i, _p,
                                            ctypes.c_longlong, _i, _i, _p, _i, _f, _p, _sz, _p, _p,
                                            _i, _p, _p, _sz]),
    "pkv_rope_inv_freq_scaled": (_i, [_p, _i, _d, _i, _d, _i, _d, _d, ctypes.POINTER(_d)]),
    "pkv_rope_table_fill_scaled": (_i, [_p, _p, _i, _i, _p, _d]),
    "kv_append_norm_rope": (_i, [_p, _ll, _p, _ll, _p, _ll, _p, _p, _i, _f, _p, _p, _i, _i, _i, _p,
                                 _p, _i, _p, _i, _i, _i, _p, _i, _p, _p, _p, _p]),
    "kv_append_rope_bs8": (_i, [_p, _ll, _p, _ll, _p, _p, _i, _p, _i, _i, _i, _p, _p, _i, _i, _p, _p,
                                _i, _p, _ll, _p, _p, _p]),
    "kv_read_bs8": (_i, [_p, _p, _i, _i, _p, _i, _p, _p, _p]),
    "paged_gqa_decode_bs8_workspace_bytes": (_sz, [_i]),
    "paged_gqa_decode_bs8": (_i, [_p, _p, _p, _i, _i, _p, _i, _i, _p, _i, _i, _p, _f, _p, _sz, _p,
                                  _p]),
    "pkv_process_logits": (_i, [_p, _i, _i, _i, _ll, _p, _ll, _p, _p, _ll, _p, _p, _p, _p, _p, _p,
                                _p, _i, _p, _ll, _p]),
    "pkv_read_device_error": (_i, [_p, _p, _i, _ip]),
    "pkv_credit_pages": (_i, [_i, _i, _i]),
    "pkv_sched_create": (_p, [_i, _i, _i, _i]),
    "pkv_sched_set_mode": (_i, [_p, _i]),
    "pkv_sched_destroy": (None, [_p]),
    "pkv_sched_submit": (_i, [_p, _i, _i, _ip]),
    "pkv_sched_admit": (_i, [_p, _p, _i, _ip]),
    "pkv_sched_grow": (_i, [_p, _i, _i]),
    "pkv_sched_finish": (_i, [_p, _i]),
    "pkv_sched_block_table": (_i, [_p, _i, _i, _p, _ip]),
    "pkv_sched_stats": (_i, [_p, _ip, _ip, _ip, _ip]),
    "pkv_sched_event_count": (_i, [_p]),
    "pkv_sched_event": (_i, [_p, _i, _ip, _ip, _ip, _ip]),
    "pkv_sched_begin_step": (_i, [_p, _p, _p, _i, _ip]),
    "pkv_sched_step_bytes": (_sz, [_p, _i, _i]),
    "pkv_sched_pack_step": (_i, [_p, _p, _i, _i, _p, _sz]),
}

_LIB = None


def _L():
    """The loaded libpkv.so; raises if it has not been built (no fallback exists)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpkv.so not found at {LIB_PATH}; build it with "
                               "`python -m paged_kv_gqa_append_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


_CALLS = None


def _load_calls():
    """The module of binding/calls.cpp (it needs the torch that is imported here)."""
    global _CALLS
    if not os.path.exists(CALLS_PATH):
        raise RuntimeError(f"_calls.so not found at {CALLS_PATH}; build it with "
                           "`python -m paged_kv_gqa_append_gb300.build`")
    _L()
    spec = importlib.util.spec_from_file_location(__name__ + "._calls", CALLS_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    built, here = module.torch_version, re.match(r"\d+\.\d+\.\d+", torch.__version__).group()
    if built != here:  # another layout of its tensors, perhaps
        raise RuntimeError(f"_calls.so was built against torch {built}, this is {here}; build it with "
                           "`python -m paged_kv_gqa_append_gb300.build`")
    _CALLS = module
    return module


def __getattr__(name):
    if name == "lib":
        return _L()
    raise AttributeError(name)


def _check(status: int, where: str):
    if status != OK:
        detail = _L().pkv_last_error().decode() if status == 5 else ""
        raise PkvError(status, where, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, device=None, shape_tail=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if shape_tail is not None and tuple(t.shape[-len(shape_tail):]) != tuple(shape_tail):
        raise ValueError(f"{name} must end in shape {shape_tail}, got {tuple(t.shape)}")


def status_string(status: int) -> str:
    return _L().pkv_status_string(status).decode()


# --------------------------------------------------------------- RoPE set-up --

def pkv_rope_inv_freq_plain(theta: float = 500000.0) -> np.ndarray:
    out = np.zeros(ROPE_PAIRS, np.float64)
    _check(_L().pkv_rope_inv_freq_plain(out.ctypes.data, theta), "pkv_rope_inv_freq_plain")
    return out


def pkv_rope_inv_freq_llama3(theta=500000.0, factor=32.0, low_freq_factor=1.0,
                             high_freq_factor=4.0, original_max_pos=8192) -> np.ndarray:
    out = np.zeros(ROPE_PAIRS, np.float64)
    _check(_L().pkv_rope_inv_freq_llama3(out.ctypes.data, theta, factor, low_freq_factor,
                                        high_freq_factor, original_max_pos),
           "pkv_rope_inv_freq_llama3")
    return out


def pkv_rope_table_fill(inv_freq, max_pos: int):
    """Host fp32 cos/sin tables [max_pos][32] (numpy)."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.shape != (ROPE_PAIRS,):
        raise ValueError("inv_freq must have 32 entries")
    cos = np.empty((max_pos, ROPE_PAIRS), np.float32)
    sin = np.empty_like(cos)
    _check(_L().pkv_rope_table_fill(cos.ctypes.data, sin.ctypes.data, max_pos, f.ctypes.data),
           "pkv_rope_table_fill")
    return cos, sin


def rope_tables_device(device, max_pos: int = 2048, inv_freq=None):
    """cos/sin tables on `device` (Llama-3.2 frequencies by default)."""
    if inv_freq is None:
        inv_freq = pkv_rope_inv_freq_llama3()
    cos, sin = pkv_rope_table_fill(inv_freq, max_pos)
    return torch.from_numpy(cos).to(device), torch.from_numpy(sin).to(device)


ROPE_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def pkv_rope_inv_freq_scaled(rotary_dim: int = HEAD_DIM, theta: float = 500000.0, scaling=None,
                             factor: float = 1.0, original_max_pos: int = 8192,
                             beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq [rotary_dim / 2], attention factor) of a head whose first
    rotary_dim dims are rotated; scaling: None, "linear", "ntk" or "yarn"
    (pkv.h gives the formulas)."""
    if rotary_dim % 2 or not 2 <= rotary_dim <= HEAD_DIM:
        raise ValueError("rotary_dim must be even and within the head")
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALING)}")
    out = np.zeros(rotary_dim // 2, np.float64)
    mul = ctypes.c_double(1.0)
    _check(_L().pkv_rope_inv_freq_scaled(out.ctypes.data, rotary_dim // 2, theta, ROPE_SCALING[scaling],
                                        factor, original_max_pos, beta_fast, beta_slow,
                                        ctypes.byref(mul)), "pkv_rope_inv_freq_scaled")
    return out, mul.value


def rope_tables_scaled_device(device, max_pos: int, inv_freq, attention_factor: float = 1.0):
    """cos/sin tables [max_pos, pairs] on `device` for kv_append_norm_rope."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.ndim != 1 or not 1 <= len(f) <= ROPE_PAIRS:
        raise ValueError("inv_freq must have 1 to 32 entries")
    cos = np.empty((max_pos, len(f)), np.float32)
    sin = np.empty_like(cos)
    _check(_L().pkv_rope_table_fill_scaled(cos.ctypes.data, sin.ctypes.data, max_pos, len(f), f.ctypes.data,
                                          attention_factor), "pkv_rope_table_fill_scaled")
    return torch.from_numpy(cos).to(device), torch.from_numpy(sin).to(device)


# ------------------------------------------------------------------- append --

def kv_append_rope(k, v, positions, block_tables, kv_pool, rope_cos, rope_sin,
                   token_seq=None, q_in=None, q_out=None, d_err=None, max_blocks=None,
                   stream=None):
    """Rotate K (and optionally q) at `positions` and write K/V into pool pages."""
    dev = kv_pool.device
    _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    _need(k, "k", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    _need(v, "v", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    T = k.numel() // (NUM_KV_HEADS * HEAD_DIM)
    if v.numel() != k.numel():
        raise ValueError("k and v must have the same shape")
    _need(positions, "positions", torch.int32, dev)
    if positions.numel() != T:
        raise ValueError("positions must have one entry per token")
    if token_seq is not None:
        _need(token_seq, "token_seq", torch.int32, dev)
        if token_seq.numel() != T:
            raise ValueError("token_seq must have one entry per token")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, row_stride]")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    if (q_in is None) != (q_out is None):
        raise ValueError("q_in and q_out go together")
    if q_in is not None:
        _need(q_in, "q_in", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        _need(q_out, "q_out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        if q_in.numel() != T * NUM_Q_HEADS * HEAD_DIM or q_out.numel() != q_in.numel():
            raise ValueError("q_in/q_out must be [T, 32, 64]")
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    S, stride = block_tables.shape
    mb = stride if max_blocks is None else max_blocks
    st = _L().kv_append_rope(_ptr(k), _ptr(v), _ptr(positions), _ptr(token_seq), T,
                            _ptr(block_tables), S, stride, mb, _ptr(kv_pool), kv_pool.shape[0],
                            _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0],
                            _ptr(q_in), _ptr(q_out), _ptr(d_err), _stream(stream))
    _check(st, "kv_append_rope")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_KV_ROW, _Q_ROW = (NUM_KV_HEADS, HEAD_DIM), (NUM_Q_HEADS, HEAD_DIM)
_KV_ROW_ELEMS, _Q_ROW_ELEMS = NUM_KV_HEADS * HEAD_DIM, NUM_Q_HEADS * HEAD_DIM
_PAGE = (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM)
_PAGE_ELEMS = 2 * NUM_KV_HEADS * PAGE_TOKENS * HEAD_DIM


# The checks of the calls that _calls.so did not take: each attribute of a
# tensor is read once (about 0.1 us each), and the error messages are made only
# when a check fails (_need says what is wrong).

def _on_device(t, name):
    """The CUDA device of `t`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _vec(t, name, dtype, dev, n):
    """`t` as a contiguous tensor of n elements; returns its address."""
    try:
        if t.dtype is dtype and t.device == dev and t.is_contiguous() and t.numel() == n:
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, dev)
    raise ValueError(f"{name} must have {n} elements, got {t.numel()}")


def _opt(t, name, dtype, dev, n):
    return None if t is None else _vec(t, name, dtype, dev, n)


def _rows(t, name, heads, dev, tokens=-1):
    """`t` as token rows [T, heads, 64] bf16 with contiguous heads and any
    token stride; returns (address, token stride, T)."""
    try:
        shape, stride = t.shape, t.stride()
        if (t.dtype is _BF16 and t.device == dev and len(shape) == 3 and shape[1] == heads
                and shape[2] == HEAD_DIM and stride[2] == 1 and stride[1] == HEAD_DIM
                and (tokens < 0 or shape[0] == tokens)):
            n = shape[0]
            return t.data_ptr(), stride[0] if n > 1 else heads * HEAD_DIM, n
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    want = "T" if tokens < 0 else tokens
    if len(shape) != 3 or tuple(shape[1:]) != (heads, HEAD_DIM) or (tokens >= 0 and shape[0] != tokens):
        raise ValueError(f"{name} must be [{want}, {heads}, {HEAD_DIM}], got {tuple(shape)}")
    raise ValueError(f"{name}: the heads of a token must be contiguous")


def _block_rows(t, dev, rows=0):
    """block_tables as (address, rows, row stride)."""
    try:
        shape = t.shape
        if t.dtype is _I32 and t.device == dev and t.is_contiguous() and len(shape) == 2 and shape[0] >= rows:
            return t.data_ptr(), shape[0], shape[1]
    except AttributeError:
        pass
    _need(t, "block_tables", _I32, dev)
    raise ValueError("block_tables must be [>= num_seqs, row_stride]")


def _device_error(t, dev):
    if t is None:
        return None
    try:
        if t.dtype is _I32 and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, "d_err", _I32, dev)


def _call(dev, stream, where, args):
    """The C call `where` of the tuple `args` with the stream appended: the
    given one, or the current one of the tensors' device (made current for the
    call)."""
    fn = getattr(_LIB or _L(), where)
    if stream is not None:
        st = fn(*args, stream.cuda_stream)
    else:
        index = dev.index
        raw = torch._C._cuda_getCurrentRawStream(index)
        if index == torch._C._cuda_getDevice():
            st = fn(*args, raw)
        else:
            with torch.cuda.device(dev):
                st = fn(*args, raw)
    if st != OK:
        _check(st, where)


def _empty(shape, dtype, dev, stream):
    """A new tensor for a call on `stream`: allocated there, so that the
    allocator neither hands out memory that another stream still uses nor
    reuses it before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _weight(w, name, dev):
    """(address, whether fp32) of a norm's weights."""
    if w is None:
        return None, None
    if getattr(w, "dtype", None) not in (_BF16, _F32):
        raise TypeError(f"{name} must be a bfloat16 or float32 tensor")
    return _vec(w, name, w.dtype, dev, HEAD_DIM), w.dtype is _F32


def _norm_rope(q, k, v, positions, token_seq, block_tables, kv_pool, rope_cos, rope_sin, q_out, k_out,
               q_weight, k_weight, eps, interleaved, d_err, max_blocks, stream):
    if stream is None:
        st = (_CALLS or _load_calls()).norm_rope(q, k, v, positions, token_seq, block_tables, kv_pool, rope_cos,
                                                 rope_sin, q_out, k_out, q_weight, k_weight, eps, interleaved, d_err,
                                                 max_blocks)
        if st >= 0:
            return _check(st, "kv_append_norm_rope")
    dev = _on_device(k, "k")
    k_ptr, k_stride, T = _rows(k, "k", NUM_KV_HEADS, dev)
    q_ptr = v_ptr = bt = pool = seq = None
    q_stride = v_stride = S = row = pages = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        q_ptr, q_stride, _ = _rows(q, "q", NUM_Q_HEADS, dev, T)
    elif q_weight is not None:
        raise ValueError("q_weight needs q")
    qo = None if q_out is None else _vec(q_out, "q_out", _BF16, dev, T * _Q_ROW_ELEMS)
    ko = None if k_out is None else _vec(k_out, "k_out", _BF16, dev, T * _KV_ROW_ELEMS)
    pos = _vec(positions, "positions", _I32, dev, T)
    if kv_pool is not None:
        page = kv_pool.shape
        if page[1:] != _PAGE:
            raise ValueError(f"kv_pool must be [num_pages, {', '.join(map(str, _PAGE))}], got {tuple(page)}")
        pages = page[0]
        pool = _vec(kv_pool, "kv_pool", _BF16, dev, pages * _PAGE_ELEMS)
        v_ptr, v_stride, _ = _rows(v, "v", NUM_KV_HEADS, dev, T)
        bt, S, row = _block_rows(block_tables, dev)
        seq = None if token_seq is None else _vec(token_seq, "token_seq", _I32, dev, T)
    shape = rope_cos.shape
    if len(shape) != 2 or not 1 <= shape[1] <= ROPE_PAIRS or rope_sin.shape != shape:
        raise ValueError("rope_cos and rope_sin must be [max_pos, pairs] with 1 to 32 pairs")
    n = shape[0] * shape[1]
    cos, sin = _vec(rope_cos, "rope_cos", _F32, dev, n), _vec(rope_sin, "rope_sin", _F32, dev, n)
    qw, q_f32 = _weight(q_weight, "q_weight", dev)
    kw, k_f32 = _weight(k_weight, "k_weight", dev)
    if q_f32 is not None and k_f32 is not None and q_f32 != k_f32:
        raise TypeError("q_weight and k_weight must have the same dtype")
    err = _device_error(d_err, dev)
    if T == 0:
        return
    _call(dev, stream, "kv_append_norm_rope", (q_ptr, q_stride, k_ptr, k_stride, v_ptr, v_stride, qw, kw,
          1 if q_f32 or k_f32 else 0, float(eps), cos, sin, shape[0], shape[1], 1 if interleaved else 0, pos, seq, T,
          bt, S, row, row if max_blocks is None else max_blocks, pool, pages, qo, ko, err))


def kv_append_norm_rope(k, v, positions, block_tables, kv_pool, rope_cos, rope_sin, token_seq=None,
                        q_in=None, q_out=None, k_out=None, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, d_err=None, max_blocks=None, stream=None):
    """kv_append_rope for models that normalise the heads of q and k (RMS over
    the 64 dims, then q_weight / k_weight), rotate only the first
    2 * rope_cos.shape[1] dims, or pair the dims (2 i, 2 i + 1)
    (interleaved=True): one pass from the projections' rows to the pages.

    k, v [T, 8, 64] and q_in [T, 32, 64] bf16 may be slices of one fused
    [T, 48, 64] projection (any token stride that is a multiple of 8).
    rope_cos/sin [max_pos, pairs] fp32 (rope_tables_scaled_device).  Weights
    [64] bf16 or fp32; None: not normalised.  Tokens and pages as for
    kv_append_rope; k_out [T, 8, 64], if given, gets the K rows as well."""
    if kv_pool is None:
        raise ValueError("kv_pool must be given")
    _norm_rope(q_in, k, v, positions, token_seq, block_tables, kv_pool, rope_cos, rope_sin, q_out, k_out,
               q_weight, k_weight, eps, interleaved, d_err, max_blocks, stream)


def qk_norm_rope(q, k, positions, rope_cos, rope_sin, q_out, k_out, q_weight=None, k_weight=None,
                 eps=1e-6, interleaved=False, d_err=None, stream=None):
    """The q and k heads normalised and rotated as kv_append_norm_rope does,
    into q_out and k_out, without an append (e.g. before kv_append_rope_bs8, or
    for a prompt's own attention)."""
    if k_out is None:
        raise ValueError("k_out must be given")
    _norm_rope(q, k, None, positions, None, None, None, rope_cos, rope_sin, q_out, k_out, q_weight,
               k_weight, eps, interleaved, d_err, None, stream)


# ------------------------------------------------------------------- decode --

def paged_gqa_decode_workspace_bytes(num_seqs: int) -> int:
    return int(_L().paged_gqa_decode_workspace_bytes(num_seqs))


def alloc_workspace(num_seqs: int, device) -> torch.Tensor:
    """Caller-owned workspace for paged_gqa_decode, zero-filled as the call requires."""
    with torch.cuda.device(device):
        n = paged_gqa_decode_workspace_bytes(num_seqs)
    if n <= 0:
        raise PkvError(5, "paged_gqa_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def paged_gqa_decode(q, kv_pool, block_tables, seq_lens, out, scale, workspace=None,
                     max_seq_len=None, d_err=None, max_blocks=None, compute=None,
                     min_units_per_warp=0, ctas_per_sm=0, stages=0, warps_per_cta=0,
                     combine=0, schedule=None, early_kv=0, stream=None, wait_limit_ns=0,
                     expire_first_wait=0):
    """out[s, h] = softmax(scale * q[s, h] . K) V over sequence s's own pages.

    early_kv=1 promises that the kernel enqueued just before this call on the
    stream writes neither block_tables, seq_lens nor the pages read here; the
    call then starts on them while that kernel finishes.  schedule: None or
    SCHEDULE_AUTO (by work per SM), SCHEDULE_STATIC or SCHEDULE_DYNAMIC.
    wait_limit_ns and expire_first_wait: the bounded-wait limit and its test
    (pkv_decode_opts).
    """
    dev = kv_pool.device
    _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    _need(q, "q", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    _need(out, "out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    S = q.numel() // (NUM_Q_HEADS * HEAD_DIM)
    if out.numel() != q.numel():
        raise ValueError("out must match q")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2 or block_tables.shape[0] < S:
        raise ValueError("block_tables must be [>= num_seqs, row_stride]")
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != S:
        raise ValueError("seq_lens must have num_seqs entries")
    stride = block_tables.shape[1]
    mb = stride if max_blocks is None else max_blocks
    if max_seq_len is None:
        max_seq_len = PAGE_TOKENS * mb
    if workspace is None:
        workspace = alloc_workspace(S, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    args = (_ptr(q), _ptr(kv_pool), kv_pool.shape[0], _ptr(block_tables), stride, mb,
            _ptr(seq_lens), S, int(max_seq_len), _ptr(out), float(scale), _ptr(workspace),
            workspace.numel(), _ptr(d_err), _stream(stream))
    if compute is None and not (min_units_per_warp or ctas_per_sm or stages or warps_per_cta
                                or combine or schedule is not None or early_kv
                                or wait_limit_ns or expire_first_wait):
        st = _L().paged_gqa_decode(*args)
    else:
        opts = DecodeOpts(COMPUTE_TENSOR if compute is None else compute,
                          min_units_per_warp, ctas_per_sm, stages, warps_per_cta, combine,
                          SCHEDULE_AUTO if schedule is None else schedule, early_kv,
                          wait_limit_ns, expire_first_wait)
        st = _L().paged_gqa_decode_ex(*args, ctypes.byref(opts))
    _check(st, "paged_gqa_decode")


# --------------------------------------------------------------- INT8 pages --

I8_BLOCK_BYTES = 2 * PAGE_TOKENS * HEAD_DIM + 2 * PAGE_TOKENS * 4   # 2176 per (page, KV head)


def new_int8_pool(num_pages: int, device) -> torch.Tensor:
    """An empty INT8 pool, uint8 [num_pages, 8, 2176]: every code 0 (stored as
    the byte 0x80) and every scale 0.  The block format is in pkv.h."""
    pool = torch.zeros((num_pages, NUM_KV_HEADS, I8_BLOCK_BYTES), dtype=torch.uint8, device=device)
    pool[:, :, :2 * 16 * 64] = 0x80
    return pool


def _need_i8_pool(kv_pool, dev):
    _need(kv_pool, "kv_pool", torch.uint8, dev, (NUM_KV_HEADS, I8_BLOCK_BYTES))
    if kv_pool.dim() != 3:
        raise ValueError("the INT8 pool must be [num_pages, 8, 2176] uint8")


def kv_append_rope_layers(k, v, positions, block_tables, kv_pool, rope_cos, rope_sin,
                          token_seq=None, stage=None, d_err=None, max_blocks=None, stream=None):
    """The same T tokens appended into every layer in one native call (a new
    request's prompt).  k, v: sequences of L tensors [T, 8, 64] bf16, all on
    the pool's device, or all in host memory (pinned for an asynchronous
    copy; each layer's rows then pass through `stage`, a device uint8 tensor
    of at least 2 * T * 1024 bytes).  block_tables: [L, num_seqs, >= max_blocks]
    int32 with unit stride in its last dimension (any layer and row strides,
    e.g. the one-row view of a request in a larger table).  kv_pool: a bf16
    pool or an INT8 pool (new_int8_pool).  No q rotation."""
    dev = kv_pool.device
    int8 = kv_pool.dtype == torch.uint8
    if int8:
        _need_i8_pool(kv_pool, dev)
    else:
        _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    L = len(k)
    if len(v) != L:
        raise ValueError("k and v must hold one tensor per layer each")
    if L == 0:
        return
    src_host = k[0].device.type == "cpu"
    where = torch.device("cpu") if src_host else dev
    T = k[0].numel() // (NUM_KV_HEADS * HEAD_DIM)
    for i, t in enumerate(list(k) + list(v)):
        _need(t, f"{'kv'[i // L]}[{i % L}]", torch.bfloat16, where, (NUM_KV_HEADS, HEAD_DIM))
        if t.numel() != T * NUM_KV_HEADS * HEAD_DIM:
            raise ValueError("every layer's k and v must be [T, 8, 64]")
    _need(positions, "positions", torch.int32, dev)
    if positions.numel() != T:
        raise ValueError("positions must have one entry per token")
    if token_seq is not None:
        _need(token_seq, "token_seq", torch.int32, dev)
        if token_seq.numel() != T:
            raise ValueError("token_seq must have one entry per token")
    if (not isinstance(block_tables, torch.Tensor) or block_tables.dtype != torch.int32 or
            block_tables.device != dev or block_tables.dim() != 3 or block_tables.stride(2) != 1):
        raise ValueError("block_tables must be an int32 [L, num_seqs, row] tensor on the pool's "
                         "device with unit stride in its last dimension")
    if block_tables.shape[0] < L:
        raise ValueError("block_tables must hold one table per layer")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    if src_host:
        _need(stage, "stage", torch.uint8, dev)
        if stage.numel() < 2 * T * NUM_KV_HEADS * HEAD_DIM * 2:
            raise ValueError("stage must hold 2 * T * 1024 bytes")
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    S, mb0 = block_tables.shape[1], block_tables.shape[2]
    ks = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k])
    vs = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v])
    st = _L().kv_append_rope_layers(
        ks, vs, L, int(src_host), _ptr(stage) if src_host else None,
        stage.numel() if src_host else 0, _ptr(positions), _ptr(token_seq), T,
        _ptr(block_tables), block_tables.stride(0), S, block_tables.stride(1),
        mb0 if max_blocks is None else max_blocks, _ptr(kv_pool), kv_pool.shape[0], int(int8),
        _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0], _ptr(d_err), _stream(stream))
    _check(st, "kv_append_rope_layers")


def kv_append_rope_int8(k, v, positions, block_tables, kv_pool, rope_cos, rope_sin,
                        token_seq=None, q_in=None, q_out=None, d_err=None, max_blocks=None,
                        stream=None):
    """kv_append_rope into INT8 pages: each (token, head) row of the rotated K
    and of V is stored as 64 int8 codes and one fp32 scale."""
    dev = kv_pool.device
    _need_i8_pool(kv_pool, dev)
    _need(k, "k", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    _need(v, "v", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    T = k.numel() // (NUM_KV_HEADS * HEAD_DIM)
    if v.numel() != k.numel():
        raise ValueError("k and v must have the same shape")
    _need(positions, "positions", torch.int32, dev)
    if positions.numel() != T:
        raise ValueError("positions must have one entry per token")
    if token_seq is not None:
        _need(token_seq, "token_seq", torch.int32, dev)
        if token_seq.numel() != T:
            raise ValueError("token_seq must have one entry per token")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, row_stride]")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    if (q_in is None) != (q_out is None):
        raise ValueError("q_in and q_out go together")
    if q_in is not None:
        _need(q_in, "q_in", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        _need(q_out, "q_out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        if q_in.numel() != T * NUM_Q_HEADS * HEAD_DIM or q_out.numel() != q_in.numel():
            raise ValueError("q_in/q_out must be [T, 32, 64]")
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    S, stride = block_tables.shape
    mb = stride if max_blocks is None else max_blocks
    st = _L().kv_append_rope_int8(_ptr(k), _ptr(v), _ptr(positions), _ptr(token_seq), T,
                                 _ptr(block_tables), S, stride, mb, _ptr(kv_pool), kv_pool.shape[0],
                                 _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0], _ptr(q_in),
                                 _ptr(q_out), _ptr(d_err), _stream(stream))
    _check(st, "kv_append_rope_int8")


def paged_gqa_decode_int8(q, kv_pool, block_tables, seq_lens, out, scale, workspace=None,
                          max_seq_len=None, d_err=None, max_blocks=None, min_units_per_warp=0,
                          ctas_per_sm=0, stages=0, warps_per_cta=0, early_kv=0, stream=None):
    """paged_gqa_decode over INT8 pages (early_kv as for paged_gqa_decode: the
    lengths, tables and first pages are read before the previous kernel on the
    stream has finished, which must not write them)."""
    dev = kv_pool.device
    _need_i8_pool(kv_pool, dev)
    _need(q, "q", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    _need(out, "out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    S = q.numel() // (NUM_Q_HEADS * HEAD_DIM)
    if out.numel() != q.numel():
        raise ValueError("out must match q")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2 or block_tables.shape[0] < S:
        raise ValueError("block_tables must be [>= num_seqs, row_stride]")
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != S:
        raise ValueError("seq_lens must have num_seqs entries")
    stride = block_tables.shape[1]
    mb = stride if max_blocks is None else max_blocks
    if max_seq_len is None:
        max_seq_len = PAGE_TOKENS * mb
    if workspace is None:
        workspace = alloc_workspace(S, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    args = (_ptr(q), _ptr(kv_pool), kv_pool.shape[0], _ptr(block_tables), stride, mb,
            _ptr(seq_lens), S, int(max_seq_len), _ptr(out), float(scale), _ptr(workspace),
            workspace.numel(), _ptr(d_err), _stream(stream))
    if not (min_units_per_warp or ctas_per_sm or stages or warps_per_cta or early_kv):
        st = _L().paged_gqa_decode_int8(*args)
    else:
        opts = DecodeOpts(COMPUTE_TENSOR, min_units_per_warp, ctas_per_sm, stages, warps_per_cta,
                          0, SCHEDULE_AUTO, int(bool(early_kv)))
        st = _L().paged_gqa_decode_int8_ex(*args, ctypes.byref(opts))
    _check(st, "paged_gqa_decode_int8")


def paged_gqa_decode_append_int8(q, k_new, v_new, kv_pool, block_tables, seq_lens, out, rope_cos,
                                 rope_sin, scale, q_out=None, workspace=None, max_seq_len=None,
                                 d_err=None, max_blocks=None, min_units_per_warp=0, early_kv=0,
                                 stream=None):
    """paged_gqa_decode_append on INT8 pages: sequence s's new token (k_new[s],
    v_new[s]) is quantised into its page at seq_lens[s] - 1 and q rotated
    there, then attention over seq_lens[s] tokens -- one kernel."""
    dev = kv_pool.device
    _need_i8_pool(kv_pool, dev)
    _need(q, "q", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    _need(out, "out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    S = q.numel() // (NUM_Q_HEADS * HEAD_DIM)
    if out.numel() != q.numel():
        raise ValueError("out must match q")
    _need(k_new, "k_new", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    _need(v_new, "v_new", torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
    if k_new.numel() != S * NUM_KV_HEADS * HEAD_DIM or v_new.numel() != k_new.numel():
        raise ValueError("k_new/v_new must be [num_seqs, 8, 64]")
    if q_out is not None:
        _need(q_out, "q_out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        if q_out.numel() != q.numel():
            raise ValueError("q_out must match q")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2 or block_tables.shape[0] < S:
        raise ValueError("block_tables must be [>= num_seqs, row_stride]")
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != S:
        raise ValueError("seq_lens must have num_seqs entries")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    stride = block_tables.shape[1]
    mb = stride if max_blocks is None else max_blocks
    if max_seq_len is None:
        max_seq_len = PAGE_TOKENS * mb
    if workspace is None:
        workspace = alloc_workspace(S, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    opts = DecodeOpts(COMPUTE_TENSOR, min_units_per_warp, 0, 0, 0, 0, SCHEDULE_AUTO, early_kv)
    st = _L().paged_gqa_decode_append_int8(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0],
        _ptr(kv_pool), kv_pool.shape[0], _ptr(block_tables), stride, mb, _ptr(seq_lens), S,
        int(max_seq_len), _ptr(q_out), _ptr(out), float(scale), _ptr(workspace), workspace.numel(),
        _ptr(d_err), _stream(stream), ctypes.byref(opts))
    _check(st, "paged_gqa_decode_append_int8")


# ------------------------------------------- block-scaled 8-bit pages (bs8) --

BS8_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}


def new_bs8_pool(num_pages: int, device, dtype=torch.int8):
    """An empty block-scaled pool: (codes [num_pages, 2, 8, 16, 64] int8 or
    float8_e4m3fn, scales [num_pages, 2, 8] fp32), all zero.  A code stands for
    code * scale of its (page, K|V, KV head)."""
    if dtype not in BS8_CODES:
        raise TypeError(f"dtype must be one of {list(BS8_CODES)}")
    codes = torch.zeros((num_pages, 2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM), dtype=torch.int8, device=device)
    return codes.view(dtype), torch.zeros((num_pages, 2, NUM_KV_HEADS), dtype=torch.float32, device=device)


def _bs8_pool(kv_pool, kv_scales):
    """Checks a pool and its scales; returns (device, pool address, scales
    address, pages, code type)."""
    dev = _on_device(kv_pool, "kv_pool")
    shape = kv_pool.shape
    code = BS8_CODES.get(kv_pool.dtype)
    if code is None:
        raise TypeError(f"kv_pool must be int8 or float8_e4m3fn, got {kv_pool.dtype}")
    if shape[1:] != _PAGE or not kv_pool.is_contiguous():
        raise ValueError("kv_pool must be a contiguous [num_pages, 2, 8, 16, 64]")
    return dev, kv_pool.data_ptr(), _vec(kv_scales, "kv_scales", _F32, dev, shape[0] * 2 * NUM_KV_HEADS), shape[0], code


def kv_append_rope_bs8(k, v, cu_new, seq_lens, block_tables, kv_pool, kv_scales, rope_cos=None,
                       rope_sin=None, q_in=None, q_out=None, d_err=None, max_blocks=None, stream=None):
    """The newest tokens of every sequence written into block-scaled 8-bit pages.

    Rows cu_new[s] .. cu_new[s + 1] - 1 of k and v are the last tokens of the
    seq_lens[s] that sequence s then holds (cu_new = arange for a decode step).
    With tables [max_pos, 32], K (and q_in into q_out) are rotated as in
    kv_append_rope; without, K is taken as it is.  The new tokens of a block
    set its scale together, and a block whose scale grows has its held codes
    written again (pkv.h).  k, v [T, 8, 64], q_in [T, 32, 64] bf16 with any
    token stride that is a multiple of 8."""
    if stream is None:
        st = (_CALLS or _load_calls()).append_bs8(kv_pool, kv_scales, k, v, cu_new, seq_lens, block_tables, rope_cos,
                                                  rope_sin, q_in, q_out, d_err, max_blocks)
        if st >= 0:
            return _check(st, "kv_append_rope_bs8")
    dev, pool, scales, pages, code = _bs8_pool(kv_pool, kv_scales)
    k_ptr, k_stride, T = _rows(k, "k", NUM_KV_HEADS, dev)
    v_ptr, v_stride, _ = _rows(v, "v", NUM_KV_HEADS, dev, T)
    S = seq_lens.numel()
    lens = _vec(seq_lens, "seq_lens", _I32, dev, S)
    cu = _vec(cu_new, "cu_new", _I32, dev, S + 1)
    bt, _, row = _block_rows(block_tables, dev, S)
    cos = sin = q_ptr = q_dst = None
    max_pos = q_stride = 0
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin go together")
    if rope_cos is not None:
        shape = rope_cos.shape
        if len(shape) != 2 or shape[1] != ROPE_PAIRS:
            raise ValueError("rope_cos and rope_sin must be [max_pos, 32]")
        max_pos = shape[0]
        cos = _vec(rope_cos, "rope_cos", _F32, dev, max_pos * ROPE_PAIRS)
        sin = _vec(rope_sin, "rope_sin", _F32, dev, max_pos * ROPE_PAIRS)
    if (q_in is None) != (q_out is None):
        raise ValueError("q_in and q_out go together")
    if q_in is not None:
        if rope_cos is None:
            raise ValueError("q_in needs rope_cos and rope_sin")
        q_ptr, q_stride, _ = _rows(q_in, "q_in", NUM_Q_HEADS, dev, T)
        q_dst = _vec(q_out, "q_out", _BF16, dev, T * _Q_ROW_ELEMS)
    err = _device_error(d_err, dev)
    if T == 0 or S == 0:
        return
    _call(dev, stream, "kv_append_rope_bs8", (k_ptr, k_stride, v_ptr, v_stride, cu, lens, T, bt, S, row,
          row if max_blocks is None else max_blocks, pool, scales, pages, code, cos, sin, max_pos, q_ptr,
          q_stride, q_dst, err))


def kv_read_bs8(kv_pool, kv_scales, page_ids, out=None, d_err=None, stream=None):
    """Pages page_ids of a block-scaled pool as bf16 pages
    [len(page_ids), 2, 8, 16, 64] (a bf16 pool, e.g. for paged_gqa_prefill over
    a cached prefix with block table 0 .. n - 1)."""
    if stream is None:
        st = (_CALLS or _load_calls()).read_bs8(kv_pool, kv_scales, page_ids, out, d_err)
        if st >= 0:
            _check(st, "kv_read_bs8")
            return out
    dev, pool, scales, pages, code = _bs8_pool(kv_pool, kv_scales)
    n = page_ids.numel()
    ids = _vec(page_ids, "page_ids", _I32, dev, n)
    if out is None:
        out = _empty((n, *_PAGE), _BF16, dev, stream)
    dst = _vec(out, "out", _BF16, dev, n * _PAGE_ELEMS)
    err = _device_error(d_err, dev)
    if n:
        _call(dev, stream, "kv_read_bs8", (pool, scales, pages, code, ids, n, dst, err))
    return out


def paged_gqa_decode_bs8_workspace_bytes(num_seqs: int) -> int:
    return int(_L().paged_gqa_decode_bs8_workspace_bytes(num_seqs))


def alloc_bs8_workspace(num_seqs: int, device, stream=None) -> torch.Tensor:
    """Caller-owned workspace for paged_gqa_decode_bs8 of up to num_seqs
    sequences (allocated on `stream`, default the current one)."""
    with torch.cuda.device(device):
        n = paged_gqa_decode_bs8_workspace_bytes(num_seqs)
    if n <= 0:
        raise PkvError(3 if num_seqs > 4096 else 5, "paged_gqa_decode_bs8_workspace_bytes")
    return _empty(n, torch.uint8, device, stream)


def paged_gqa_decode_bs8(q, kv_pool, kv_scales, block_tables, seq_lens, out, scale, workspace=None,
                         max_seq_len=None, d_err=None, max_blocks=None, stream=None):
    """paged_gqa_decode over block-scaled 8-bit pages (new_bs8_pool): q, out
    [num_seqs, 32, 64] bf16, q rotated.  workspace: alloc_bs8_workspace, one
    for each stream or captured graph that may run at the same time."""
    if stream is None:
        st = (_CALLS or _load_calls()).decode_bs8(kv_pool, kv_scales, q, block_tables, seq_lens, out, scale, workspace,
                                                  max_seq_len, d_err, max_blocks)
        if st >= 0:
            return _check(st, "paged_gqa_decode_bs8")
    dev, pool, scales, pages, code = _bs8_pool(kv_pool, kv_scales)
    shape = q.shape
    if shape[-2:] != _Q_ROW:
        raise ValueError(f"q must end in shape {_Q_ROW}, got {tuple(shape)}")
    n = q.numel()
    S = n // _Q_ROW_ELEMS
    q_ptr, dst = _vec(q, "q", _BF16, dev, n), _vec(out, "out", _BF16, dev, n)
    lens = _vec(seq_lens, "seq_lens", _I32, dev, S)
    bt, _, row = _block_rows(block_tables, dev, S)
    mb = row if max_blocks is None else max_blocks
    err = _device_error(d_err, dev)
    if S == 0:
        return
    if workspace is None:
        workspace = alloc_bs8_workspace(S, dev, stream)
    size = workspace.numel()
    _call(dev, stream, "paged_gqa_decode_bs8", (q_ptr, pool, scales, pages, code, bt, row, mb, lens, S,
          PAGE_TOKENS * mb if max_seq_len is None else int(max_seq_len), dst, float(scale),
          _vec(workspace, "workspace", torch.uint8, dev, size), size, err))


def paged_gqa_decode_append(q, k_new, v_new, kv_pool, block_tables, seq_lens, out, rope_cos,
                            rope_sin, scale, q_out=None, workspace=None, max_seq_len=None,
                            d_err=None, max_blocks=None, warps_per_cta=0, min_units_per_warp=0,
                            ctas_per_sm=0, schedule=None, early_kv=0, stream=None):
    """One decode step: append each sequence's new token at seq_lens-1, then attend.

    early_kv as for paged_gqa_decode (the pages meant are the ones this call
    reads and appends to).
    """
    dev = kv_pool.device
    _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    _need(q, "q", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    _need(out, "out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    S = q.numel() // (NUM_Q_HEADS * HEAD_DIM)
    if out.numel() != q.numel():
        raise ValueError("out must match q")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, name, torch.bfloat16, dev, (NUM_KV_HEADS, HEAD_DIM))
        if t.numel() != S * NUM_KV_HEADS * HEAD_DIM:
            raise ValueError(f"{name} must be [num_seqs, 8, 64]")
    if q_out is not None:
        _need(q_out, "q_out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        if q_out.numel() != q.numel():
            raise ValueError("q_out must match q")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2 or block_tables.shape[0] < S:
        raise ValueError("block_tables must be [>= num_seqs, row_stride]")
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != S:
        raise ValueError("seq_lens must have num_seqs entries")
    stride = block_tables.shape[1]
    mb = stride if max_blocks is None else max_blocks
    if max_seq_len is None:
        max_seq_len = PAGE_TOKENS * mb
    if workspace is None:
        workspace = alloc_workspace(S, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    opts = DecodeOpts(COMPUTE_TENSOR, min_units_per_warp, ctas_per_sm, 0, warps_per_cta, 0,
                      SCHEDULE_AUTO if schedule is None else schedule, early_kv)
    st = _L().paged_gqa_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(rope_cos), _ptr(rope_sin), rope_cos.shape[0],
        _ptr(kv_pool), kv_pool.shape[0], _ptr(block_tables), stride, mb, _ptr(seq_lens), S,
        int(max_seq_len), _ptr(q_out), _ptr(out), float(scale), _ptr(workspace),
        workspace.numel(), _ptr(d_err), _stream(stream), ctypes.byref(opts))
    _check(st, "paged_gqa_decode_append")


def paged_gqa_decode_append_layers(q, k_new, v_new, kv_pool, block_tables, seq_lens, out,
                                   rope_cos, rope_sin, scale, workspace, max_seq_len=None,
                                   d_err=None, stream=None, q_out=None, early_kv=1,
                                   host_stage=None, dev_stage=None, check=True):
    """A whole decode step: for every layer l, the fused append + decode of
    q[l], k_new[l], v_new[l] over block_tables[l] into out[l] on a bf16 pool
    (paged_gqa_decode_append) or an INT8 pool (paged_gqa_decode_append_int8),
    in layer order on one stream -- one call of the C function of the same
    name, which makes those per-layer calls.

    q, out (and q_out): [L, S, 32, 64] bf16; k_new, v_new: [L, S, 8, 64] bf16;
    block_tables: [L, S', row_stride] int32 with S' >= S; seq_lens: [S] int32,
    shared by the layers.  early_kv=1 lets layers >= 1 read their tables and
    stage their first pages while the previous layer's kernel finishes (the
    layers' pages must be disjoint).  host_stage (pinned uint8 host tensor) and
    dev_stage (uint8 device tensor of at least its size): one copy of the
    first into the second runs on the stream before the launches, e.g. the
    block of pkv_sched_pack_step that block_tables / seq_lens are views of.
    check=False skips the tensor checks below (the C call still checks sizes,
    pointers and alignment): for a caller that built the tensors itself and
    checked their shapes once, as ContinuousBatcher does every step.
    """
    dev = kv_pool.device
    int8 = kv_pool.dtype == torch.uint8
    if check:
        _check_layers_args(q, k_new, v_new, kv_pool, block_tables, seq_lens, out, rope_cos,
                           rope_sin, workspace, d_err, q_out, host_stage, dev_stage, int8, dev)
    L, S = q.shape[0], q.shape[1]
    if L == 0:
        return
    stage = 0 if host_stage is None else host_stage.numel()
    stride = block_tables.shape[2]
    if max_seq_len is None:
        max_seq_len = PAGE_TOKENS * stride
    st = _L().paged_gqa_decode_append_layers(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(q_out), _ptr(out), L, S, _ptr(rope_cos),
        _ptr(rope_sin), rope_cos.shape[0], _ptr(kv_pool), kv_pool.shape[0], int(int8),
        _ptr(block_tables), block_tables.shape[1] * stride, stride, stride, _ptr(seq_lens),
        int(max_seq_len), float(scale), _ptr(workspace), workspace.numel(), _ptr(d_err),
        _stream(stream), int(early_kv), _ptr(host_stage), _ptr(dev_stage), stage)
    _check(st, "paged_gqa_decode_append_layers")


def _check_layers_args(q, k_new, v_new, kv_pool, block_tables, seq_lens, out, rope_cos, rope_sin,
                       workspace, d_err, q_out, host_stage, dev_stage, int8, dev):
    if int8:
        _need_i8_pool(kv_pool, dev)
    else:
        _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    for t, name, heads in ((q, "q", NUM_Q_HEADS), (out, "out", NUM_Q_HEADS),
                           (k_new, "k_new", NUM_KV_HEADS), (v_new, "v_new", NUM_KV_HEADS)):
        _need(t, name, torch.bfloat16, dev, (heads, HEAD_DIM))
        if t.dim() != 4:
            raise ValueError(f"{name} must be [layers, num_seqs, {heads}, {HEAD_DIM}]")
    L, S = q.shape[0], q.shape[1]
    if out.shape != q.shape or k_new.shape[:2] != (L, S) or v_new.shape != k_new.shape:
        raise ValueError("q/out [L, S, 32, 64] and k_new/v_new [L, S, 8, 64] must agree")
    if q_out is not None:
        _need(q_out, "q_out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
        if q_out.shape != q.shape:
            raise ValueError("q_out must match q")
    if L == 0:
        return
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 3 or block_tables.shape[0] != L or block_tables.shape[1] < S:
        raise ValueError("block_tables must be [layers, >= num_seqs, row_stride]")
    _need(seq_lens, "seq_lens", torch.int32, dev)
    if seq_lens.numel() != S:
        raise ValueError("seq_lens must have num_seqs entries")
    _need(rope_cos, "rope_cos", torch.float32, dev, (ROPE_PAIRS,))
    _need(rope_sin, "rope_sin", torch.float32, dev, (ROPE_PAIRS,))
    _need(workspace, "workspace", torch.uint8, dev)
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    if (host_stage is None) != (dev_stage is None):
        raise ValueError("host_stage and dev_stage go together")
    if host_stage is not None:
        if host_stage.dtype != torch.uint8 or not host_stage.is_contiguous():
            raise TypeError("host_stage must be a contiguous uint8 host tensor")
        _need(dev_stage, "dev_stage", torch.uint8, dev)
        if dev_stage.numel() < host_stage.numel():
            raise ValueError("dev_stage is smaller than host_stage")


PREFILL_MMA_SYNC = 2  # comparison arm of paged_gqa_prefill (legacy bf16 mma.sync)


def paged_gqa_prefill(q, cu_q, kv_pool, block_tables, seq_lens, out, scale, max_q_len=None,
                      d_err=None, max_blocks=None, compute=None, stream=None):
    """Causal attention of each sequence's last q_len tokens over its own pages.

    q, out: [T, 32, 64] bf16 (q rotated); cu_q: [S + 1] int32 row offsets on
    the device; seq_lens: [S] int32 tokens held (the queries are the last
    cu_q[s+1] - cu_q[s] of them).  max_q_len: host bound of every q_len
    (default T).  compute: None / COMPUTE_TENSOR (tcgen05, tensor memory) or
    PREFILL_MMA_SYNC.
    """
    dev = kv_pool.device
    _need(kv_pool, "kv_pool", torch.bfloat16, dev, (2, NUM_KV_HEADS, PAGE_TOKENS, HEAD_DIM))
    _need(q, "q", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    _need(out, "out", torch.bfloat16, dev, (NUM_Q_HEADS, HEAD_DIM))
    T = q.numel() // (NUM_Q_HEADS * HEAD_DIM)
    if out.numel() != q.numel():
        raise ValueError("out must match q")
    _need(cu_q, "cu_q", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    S = seq_lens.numel()
    if cu_q.numel() != S + 1:
        raise ValueError("cu_q must have num_seqs + 1 entries")
    _need(block_tables, "block_tables", torch.int32, dev)
    if block_tables.dim() != 2 or block_tables.shape[0] < S:
        raise ValueError("block_tables must be [>= num_seqs, row_stride]")
    stride = block_tables.shape[1]
    mb = stride if max_blocks is None else max_blocks
    if d_err is not None:
        _need(d_err, "d_err", torch.int32, dev)
    st = _L().paged_gqa_prefill_ex(_ptr(q), T, _ptr(cu_q), _ptr(kv_pool), kv_pool.shape[0],
                                   _ptr(block_tables), stride, mb, _ptr(seq_lens), S,
                                   int(T if max_q_len is None else max_q_len), _ptr(out),
                                   float(scale), _ptr(d_err), _stream(stream),
                                   COMPUTE_TENSOR if compute is None else int(compute))
    _check(st, "paged_gqa_prefill")


def argmax_rows(logits, out=None, stream=None):
    """Next-token ids: per row of FP32 logits [rows, vocab] (row stride may
    exceed vocab), the first index of the largest non-NaN value."""
    if logits.dtype != torch.float32 or not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a 2-D float32 CUDA tensor")
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    rows, vocab = logits.shape
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    _need(out, "out", torch.int32, logits.device)
    _check(_L().pkv_argmax_f32(_ptr(logits), rows, vocab, logits.stride(0), _ptr(out),
                               _stream(stream)), "pkv_argmax_f32")
    return out


LOGITS_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def process_logits(logits, out=None, ids=None, history=None, history_lens=None, prompt_lens=None,
                   repetition=None, presence=None, frequency=None, bias_ids=None, bias_values=None,
                   allow_mask=None, stream=None):
    """Penalties, biases and a grammar's mask on next-token logits, and the next
    token of each row; returns ids ([rows] int32, -1 where nothing is allowed).

    logits [rows, vocab] fp32, bf16 or fp16 (row stride may exceed vocab).
    out [rows, vocab] fp32 gets the processed logits (None: ids only; logits
    itself for fp32: in place).  history [rows, H] int32: each row's prompt
    ids, then the generated ones, history_lens [rows] of them, the first
    prompt_lens [rows] from the prompt; repetition counts both, presence and
    frequency the generated ones ([rows] fp32 each, None: off).  bias_ids /
    bias_values [rows, B] int32 / fp32; ids outside the vocabulary are padding.
    allow_mask [rows, >= ceil(vocab / 32)] int32, bit i % 32 of word i / 32 set:
    token i is allowed."""
    if stream is None:
        if ids is None and isinstance(logits, torch.Tensor) and logits.is_cuda and logits.dim() == 2:
            ids = torch.empty(logits.shape[0], dtype=_I32, device=logits.device)
        st = (_CALLS or _load_calls()).process_logits(logits, out, ids, history, history_lens, prompt_lens, repetition,
                                                      presence, frequency, bias_ids, bias_values, allow_mask)
        if st >= 0:
            _check(st, "pkv_process_logits")
            return ids
    dev = _on_device(logits, "logits")
    shape, stride, dtype = logits.shape, logits.stride(), LOGITS_DTYPES.get(logits.dtype)
    if dtype is None or len(shape) != 2:
        raise TypeError("logits must be a 2-D float32, bfloat16 or float16 tensor")
    rows, vocab = shape
    if vocab < 1 or (stride[1] != 1 and vocab > 1):
        raise ValueError("logits rows must be contiguous and not empty")
    dst = hist = h_lens = p_lens = rep = pres = freq = b_ids = b_vals = mask = None
    out_stride = H = B = mask_stride = 0
    if out is not None:
        if getattr(out, "dtype", None) is not _F32:
            raise TypeError("out must be a float32 tensor")
        out_stride = out.stride()
        if out.device != dev or out.shape != shape or (out_stride[1] != 1 and vocab > 1):
            raise ValueError("out must be [rows, vocab] on the logits' device with contiguous rows")
        dst, out_stride = out.data_ptr(), out_stride[0] if rows > 1 else vocab
    if ids is None:
        ids = _empty(rows, _I32, dev, stream)
    id_ptr = _vec(ids, "ids", _I32, dev, rows)
    if history is None:
        if not (history_lens is prompt_lens is repetition is presence is frequency is None):
            raise ValueError("lengths and penalties need a history")
    else:
        h_shape = history.shape
        if len(h_shape) != 2 or h_shape[0] != rows:
            raise ValueError("history must be [rows, H]")
        if history_lens is None:
            raise ValueError("history needs history_lens")
        H = h_shape[1]
        hist = _vec(history, "history", _I32, dev, rows * H)
        h_lens = _vec(history_lens, "history_lens", _I32, dev, rows)
        p_lens = _opt(prompt_lens, "prompt_lens", _I32, dev, rows)
        rep = _opt(repetition, "repetition", _F32, dev, rows)
        pres = _opt(presence, "presence", _F32, dev, rows)
        freq = _opt(frequency, "frequency", _F32, dev, rows)
        if H == 0:  # nothing to count
            hist = h_lens = p_lens = rep = pres = freq = None
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        b_shape = bias_ids.shape
        if len(b_shape) != 2 or b_shape[0] != rows or bias_values.shape != b_shape:
            raise ValueError("bias_ids and bias_values must be [rows, B]")
        B = b_shape[1]
        b_ids = _vec(bias_ids, "bias_ids", _I32, dev, rows * B)
        b_vals = _vec(bias_values, "bias_values", _F32, dev, rows * B)
    if allow_mask is not None:
        m_shape = allow_mask.shape
        if len(m_shape) != 2 or m_shape[0] != rows or m_shape[1] < (vocab + 31) // 32:
            raise ValueError("allow_mask must be [rows, >= ceil(vocab / 32)]")
        mask_stride = m_shape[1]
        mask = _vec(allow_mask, "allow_mask", _I32, dev, rows * mask_stride)
    if rows == 0:
        return ids
    _call(dev, stream, "pkv_process_logits", (logits.data_ptr(), dtype, rows, vocab,
          stride[0] if rows > 1 else vocab, dst, out_stride, id_ptr, hist, H, h_lens, p_lens, rep, pres, freq,
          b_ids, b_vals, B, mask, mask_stride))
    return ids


def pkv_read_device_error(d_err, clear: bool = True, stream=None) -> int:
    """Synchronise the stream and return the device error word (optionally reset it)."""
    code = ctypes.c_int(0)
    _check(_L().pkv_read_device_error(_ptr(d_err), _stream(stream), int(clear), ctypes.byref(code)),
           "pkv_read_device_error")
    return code.value


# ---------------------------------------------------------------- scheduler --

def pkv_credit_pages(prompt_tokens: int, allowed_new_tokens: int, num_layers: int) -> int:
    return int(_L().pkv_credit_pages(prompt_tokens, allowed_new_tokens, num_layers))


class Scheduler:
    """Admission and page allocation (C++ pkv_sched): continuous batching, or
    static batching (static=True: a new group only once the current one has
    finished)."""

    def __init__(self, num_pages: int, num_layers: int, max_blocks: int = 128, max_slots: int = 256,
                 static: bool = False):
        self._h = _L().pkv_sched_create(num_pages, num_layers, max_blocks, max_slots)
        if not self._h:
            raise PkvError(1, "pkv_sched_create")
        self.num_layers, self.max_blocks, self.max_slots = num_layers, max_blocks, max_slots
        if static:
            _check(_L().pkv_sched_set_mode(self._h, 1), "pkv_sched_set_mode")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().pkv_sched_destroy(h)
            self._h = None

    def submit(self, prompt_tokens: int, allowed_new_tokens: int):
        """Returns (status, request id); oversize requests give ERR_REQUEST_TOO_LARGE."""
        rid = ctypes.c_int(-1)
        st = _L().pkv_sched_submit(self._h, prompt_tokens, allowed_new_tokens, ctypes.byref(rid))
        if st not in (OK, ERR_REQUEST_TOO_LARGE):
            raise PkvError(st, "pkv_sched_submit")
        return st, rid.value

    def admit(self):
        buf = (ctypes.c_int * self.max_slots)()
        n = ctypes.c_int(0)
        _check(_L().pkv_sched_admit(self._h, buf, self.max_slots, ctypes.byref(n)), "pkv_sched_admit")
        return list(buf[:n.value])

    def grow(self, rid: int, new_len: int) -> int:
        st = _L().pkv_sched_grow(self._h, rid, new_len)
        if st not in (OK, ERR_POOL_EXHAUSTED):
            raise PkvError(st, "pkv_sched_grow")
        return st

    def finish(self, rid: int):
        _check(_L().pkv_sched_finish(self._h, rid), "pkv_sched_finish")

    def block_table(self, rid: int, layer: int):
        row = np.empty(self.max_blocks, np.int32)
        slot = ctypes.c_int(-1)
        _check(_L().pkv_sched_block_table(self._h, rid, layer, row.ctypes.data, ctypes.byref(slot)),
               "pkv_sched_block_table")
        return row, slot.value

    def stats(self):
        v = [ctypes.c_int(0) for _ in range(4)]
        _check(_L().pkv_sched_stats(self._h, *[ctypes.byref(x) for x in v]), "pkv_sched_stats")
        return dict(free=v[0].value, reserved=v[1].value, queued=v[2].value, running=v[3].value)

    def begin_step(self):
        """Grow every running request by one token (admission order); returns
        (ids, lengths after the step) as int32 arrays."""
        ids = np.empty(self.max_slots, np.int32)
        lens = np.empty(self.max_slots, np.int32)
        n = ctypes.c_int(0)
        st = _L().pkv_sched_begin_step(self._h, ids.ctypes.data, lens.ctypes.data, self.max_slots,
                                       ctypes.byref(n))
        _check(st, "pkv_sched_begin_step")
        return ids[:n.value].copy(), lens[:n.value].copy()

    def step_bytes(self, batch: int, max_len: int) -> int:
        return int(_L().pkv_sched_step_bytes(self._h, batch, max_len))

    def pack_step(self, ids, max_len: int, block) -> int:
        """Write the step block (lengths, then tables [L][B][P]) of requests
        `ids` into `block` (a contiguous uint8 host tensor or array); returns P."""
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        ptr = block.data_ptr() if isinstance(block, torch.Tensor) else block.ctypes.data
        nbytes = block.numel() if isinstance(block, torch.Tensor) else block.nbytes
        _check(_L().pkv_sched_pack_step(self._h, ids.ctypes.data, len(ids), int(max_len), ptr,
                                        nbytes), "pkv_sched_pack_step")
        return max(1, (int(max_len) + PAGE_TOKENS - 1) // PAGE_TOKENS)

    def events(self):
        n = _L().pkv_sched_event_count(self._h)
        out = []
        v = [ctypes.c_int(0) for _ in range(4)]
        for i in range(n):
            _check(_L().pkv_sched_event(self._h, i, *[ctypes.byref(x) for x in v]), "pkv_sched_event")
            out.append(tuple(x.value for x in v))
        return out


# --------------------------------------------------------------- decode step --

class DecodeStep:
    """One decode step over every layer, captured once into a CUDA graph.

    Per layer l (in order, as a model runs them), by default one fused call
        paged_gqa_decode_append(q[l], k[l], v[l], pool, block_tables[l],
                                seq_lens, out[l], cos, sin, q_out=q_rot[l])
    which appends token s of layer l at position seq_lens[s] - 1 and attends
    over seq_lens[s] tokens; the rotated queries are written only when the
    caller passes a q_rot buffer (the attention itself keeps them in
    registers: leaving the copy out saves about 0.2 us per layer at batch 32
    x 2048 on GB300).  With fused=False the same step runs as
        kv_append_rope(k[l], v[l], positions, block_tables[l], pool, cos, sin,
                       q_in=q[l], q_out=q_rot[l])
        paged_gqa_decode(q_rot[l], pool, block_tables[l], seq_lens, out[l], scale)
    (token s written at positions[s]).  The tensors are bound at construction: refresh
    their contents in place (new K/V/q, positions, lengths, tables) and call
    run().  Replaying the graph removes the per-call host cost, and the
    kernels' programmatic-dependent-launch edges overlap each launch with
    the previous kernel's tail.  With overlap_layers (the default) the decode
    kernel of layer l >= 1 also reads its tables and stages its first pages
    before layer l - 1's kernel has finished (early_kv), which requires the
    layers' block tables to name disjoint pages, as separate layers' caches
    do.  Layer 0 always waits for whatever ran before the step.

        pool          [num_pages, 2, 8, 16, 64] bf16
        block_tables  [L, S, max_blocks] int32
        seq_lens      [S] int32;  positions [S] int32
        k, v          [L, S, 8, 64] bf16;  q, out [L, S, 32, 64] bf16
    """

    def __init__(self, pool, block_tables, seq_lens, positions, k, v, q, out, rope_cos, rope_sin,
                 scale, max_seq_len=None, workspace=None, d_err=None, q_rot=None, compute=None,
                 use_graph=True, stream=None, fused=True, overlap_layers=True, schedule=None):
        self.L, self.S = block_tables.shape[0], block_tables.shape[1]
        self.t = dict(pool=pool, bt=block_tables, lens=seq_lens, pos=positions, k=k, v=v, q=q,
                      out=out, cos=rope_cos, sin=rope_sin)
        dev = pool.device
        self.workspace = alloc_workspace(self.S, dev) if workspace is None else workspace
        self.d_err = torch.zeros(1, dtype=torch.int32, device=dev) if d_err is None else d_err
        self.scale = float(scale)
        self.max_seq_len = max_seq_len
        self.compute = compute
        self.overlap = bool(overlap_layers)
        self.schedule = None if schedule is None else int(schedule)   # None: automatic
        # the fused kernel places each new token at seq_lens - 1 (positions unused)
        self.fused = fused and compute in (None, COMPUTE_TENSOR)
        # the rotated queries: kept by the fused step only in a buffer of the
        # caller's; the two-kernel step needs them (its decode reads them)
        self.q_rot = q_rot if (q_rot is not None or self.fused) else torch.empty_like(q)
        self._q_scratch = None  # the two-kernel timing graphs' rotated q on a fused step without q_rot
        self.launches_per_step = (1 if self.fused else 2) * self.L
        self._launch()                      # eager run: sets up kernels and descriptors
        torch.cuda.synchronize(dev)
        self.graph = None
        if use_graph:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=stream):
                self._launch()

    def _launch(self, decode_only=False):
        t = self.t
        if self.fused and not decode_only:
            for l in range(self.L):
                paged_gqa_decode_append(t["q"][l], t["k"][l], t["v"][l], t["pool"], t["bt"][l],
                                        t["lens"], t["out"][l], t["cos"], t["sin"], self.scale,
                                        q_out=None if self.q_rot is None else self.q_rot[l],
                                        workspace=self.workspace,
                                        max_seq_len=self.max_seq_len, d_err=self.d_err,
                                        early_kv=int(self.overlap and l > 0),
                                        schedule=self.schedule)
            return
        q_rot = self._rotated()
        for l in range(self.L):
            if not decode_only:
                kv_append_rope(t["k"][l], t["v"][l], t["pos"], t["bt"][l], t["pool"], t["cos"],
                               t["sin"], q_in=t["q"][l], q_out=q_rot[l], d_err=self.d_err)
            # after kv_append_rope of the same layer the pages are not ready early
            paged_gqa_decode(q_rot[l], t["pool"], t["bt"][l], t["lens"], t["out"][l],
                             self.scale, workspace=self.workspace, max_seq_len=self.max_seq_len,
                             d_err=self.d_err, compute=self.compute,
                             early_kv=int(self.overlap and decode_only and l > 0),
                             schedule=self.schedule)

    def run(self):
        if self.graph is not None:
            self.graph.replay()
        else:
            self._launch()

    def _rotated(self):
        """The buffer the two-kernel form rotates q into: q_rot, else a
        scratch copy of q made on first use (outside any capture: the graph
        helpers below call this before capturing)."""
        if self.q_rot is not None:
            return self.q_rot
        if self._q_scratch is None:
            self._q_scratch = self.t["q"].clone()
        return self._q_scratch

    def append_only_graph(self):
        """A graph of just the L kv_append_rope calls of the step (tokens at
        `positions`, q rotated into the step's q_rot buffer, or a scratch one)."""
        t = self.t
        q_rot = self._rotated()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for l in range(self.L):
                kv_append_rope(t["k"][l], t["v"][l], t["pos"], t["bt"][l], t["pool"], t["cos"],
                               t["sin"], q_in=t["q"][l], q_out=q_rot[l], d_err=self.d_err)
        return g

    def decode_only_graph(self):
        """A graph of just the L decode calls (for timing the decode kernel)."""
        self._rotated()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self._launch(decode_only=True)
        return g

    def error(self) -> int:
        """Synchronise and return (and clear) the device error word."""
        return pkv_read_device_error(self.d_err)


class Int8DecodeStep:
    """One decode step over every layer on INT8 pages, captured into a CUDA graph.

    Per layer l:
        kv_append_rope_int8(k[l], v[l], positions, block_tables[l], kv_pool, cos, sin,
                            q_in=q[l], q_out=q_rot[l])
        paged_gqa_decode_int8(q_rot[l], kv_pool, block_tables[l], seq_lens, out[l], scale)
    (the fused form writes q_rot only when the caller passes one, as in DecodeStep)
    With fused=True each layer is one call
        paged_gqa_decode_append_int8(q[l], k[l], v[l], kv_pool, block_tables[l],
                                     seq_lens, out[l], cos, sin, q_out=q_rot[l])
    which places token s at seq_lens[s] - 1 (positions unused).  The default
    (fused=None) is the fused form, the faster one at every batch measured (on
    GB300 at 2048 tokens a sequence: 32 sequences 17.5 vs 23.1 us/layer, 256
    sequences 96.6 vs 108.4).  With
    overlap_layers (the default) layer l >= 1 reads its tables and stages its
    first pages before layer l - 1's kernel has finished, which requires the
    layers' block tables to name disjoint pages.  Tensors are bound at
    construction (refresh their contents in place and call run()), as for
    DecodeStep.

        kv_pool [num_pages, 8, 2176] uint8 (see new_int8_pool)
        block_tables [L, S, max_blocks] int32;  seq_lens, positions [S] int32
        k, v [L, S, 8, 64] bf16;  q, out [L, S, 32, 64] bf16
    """

    def __init__(self, kv_pool, block_tables, seq_lens, positions, k, v, q, out, rope_cos,
                 rope_sin, scale, max_seq_len=None, workspace=None, d_err=None, q_rot=None,
                 use_graph=True, stream=None, fused=None, overlap_layers=True):
        self.L, self.S = block_tables.shape[0], block_tables.shape[1]
        self.fused = True if fused is None else bool(fused)
        self.overlap = bool(overlap_layers)
        self.t = dict(pool=kv_pool, bt=block_tables, lens=seq_lens, pos=positions,
                      k=k, v=v, q=q, out=out, cos=rope_cos, sin=rope_sin)
        dev = kv_pool.device
        # the rotated queries, as for DecodeStep: kept by the fused step only
        # in a buffer of the caller's; the two-kernel step needs them
        self.q_rot = q_rot if (q_rot is not None or self.fused) else torch.empty_like(q)
        self._q_scratch = None  # the partial graphs' rotated q on a fused step without q_rot
        self.workspace = alloc_workspace(self.S, dev) if workspace is None else workspace
        self.d_err = torch.zeros(1, dtype=torch.int32, device=dev) if d_err is None else d_err
        self.scale = float(scale)
        self.max_seq_len = max_seq_len
        self.launches_per_step = (1 if self.fused else 2) * self.L
        self._launch()                      # eager run: sets up kernels and descriptors
        torch.cuda.synchronize(dev)
        self.graph = None
        if use_graph:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=stream):
                self._launch()

    def _launch(self, append=True, decode=True):
        t = self.t
        if self.fused and append and decode:
            for l in range(self.L):
                paged_gqa_decode_append_int8(t["q"][l], t["k"][l], t["v"][l], t["pool"], t["bt"][l],
                                             t["lens"], t["out"][l], t["cos"], t["sin"], self.scale,
                                             q_out=None if self.q_rot is None else self.q_rot[l],
                                             workspace=self.workspace,
                                             max_seq_len=self.max_seq_len, d_err=self.d_err,
                                             early_kv=int(self.overlap and l > 0))
            return
        q_rot = self._rotated()
        for l in range(self.L):
            if append:
                kv_append_rope_int8(t["k"][l], t["v"][l], t["pos"], t["bt"][l], t["pool"],
                                    t["cos"], t["sin"], q_in=t["q"][l], q_out=q_rot[l],
                                    d_err=self.d_err)
            if decode:
                # a decode-only graph (timing) has no append between the layers:
                # layers >= 1 may stage their pages early, as in DecodeStep
                paged_gqa_decode_int8(q_rot[l], t["pool"], t["bt"][l], t["lens"], t["out"][l],
                                      self.scale, workspace=self.workspace,
                                      max_seq_len=self.max_seq_len, d_err=self.d_err,
                                      early_kv=int(self.overlap and not append and l > 0))

    def run(self):
        if self.graph is not None:
            self.graph.replay()
        else:
            self._launch()

    def _rotated(self):
        """As DecodeStep._rotated."""
        if self.q_rot is not None:
            return self.q_rot
        if self._q_scratch is None:
            self._q_scratch = self.t["q"].clone()
        return self._q_scratch

    def partial_graph(self, append: bool, decode: bool):
        """A graph of only the append calls or only the decode calls (for timing)."""
        self._rotated()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self._launch(append=append, decode=decode)
        return g

    def error(self) -> int:
        """Synchronise and return (and clear) the device error word."""
        return pkv_read_device_error(self.d_err)
