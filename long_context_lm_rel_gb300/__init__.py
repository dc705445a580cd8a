"""Python binding of librxl (include/rxl.h): argument marshalling only.

Every function has the name and the argument order of its C entry point.
Tensors may be torch tensors (their data_ptr() is passed) or raw integer
device addresses. Each call raises RxlError on a non-OK status. The library
must have been built (``build()``); nothing here computes anything, and
there is no fallback when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

from .build import LIB, build  # noqa: F401

RXL_OK = 0
RXL_ERR_INVALID_ARGUMENT = 1
RXL_ERR_UNSUPPORTED = 2
RXL_ERR_MISALIGNED = 3
RXL_ERR_WORKSPACE_TOO_SMALL = 4
RXL_ERR_CUDA = 5
RXL_DTYPE_F32 = 0
RXL_DTYPE_BF16 = 1


class rxl_attn_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("dh", ctypes.c_int),
                ("mem_cap", ctypes.c_int), ("mem_len", ctypes.c_int), ("mem_head", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class rxl_ring(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("planes", ctypes.c_int), ("cap", ctypes.c_int),
                ("D", ctypes.c_int), ("plane_stride", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("head", ctypes.c_int), ("len", ctypes.c_int)]


class rxl_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_q", "w_k", "w_v", "w_o", "r", "u", "vbias", "ln1_gamma", "ln1_beta",
        "w_1", "b_1", "w_2", "b_2", "ln2_gamma", "ln2_beta")]


class rxl_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int)]


class rxl_logprob_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("V", ctypes.c_int), ("top_k", ctypes.c_int), ("dtype", ctypes.c_int)]


class rxl_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] \
        + [("n", ctypes.c_longlong), ("weight_decay", ctypes.c_float)]


class rxl_adamw_desc(ctypes.Structure):
    _fields_ = [("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("state_bits", ctypes.c_int),
                ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float)]


class rxl_adamw_scalars(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("m_correction", ctypes.c_float), ("v_correction", ctypes.c_float),
                ("grad_scale", ctypes.c_float), ("seed", ctypes.c_uint32)]


def make_layer_weights(**tensors) -> rxl_layer_weights:
    """rxl_layer_weights from tensors (or addresses) named as its fields."""
    return rxl_layer_weights(**{k: _ptr(v) for k, v in tensors.items()})


class RxlError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {rxl_status_string(status)}"
                         + (f" (cuda error {lib().rxl_last_cuda_error()})" if status == RXL_ERR_CUDA else ""))


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded librxl (ctypes). Raises if the library was not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB):
                raise RuntimeError(f"librxl.so is not built ({LIB}); call long_context_lm_rel_gb300.build()")
            L = ctypes.CDLL(LIB)
            P, vp = ctypes.POINTER, ctypes.c_void_p
            L.rxl_attn_fwd.argtypes = [P(rxl_attn_desc)] + [vp] * 8 + [vp]
            L.rxl_attn_fwd.restype = ctypes.c_int
            L.rxl_attn_bwd_workspace_bytes.argtypes = [P(rxl_attn_desc)]
            L.rxl_attn_bwd_workspace_bytes.restype = ctypes.c_size_t
            L.rxl_attn_bwd.argtypes = [P(rxl_attn_desc)] + [vp] * 16 + [ctypes.c_size_t, vp]
            L.rxl_attn_bwd.restype = ctypes.c_int
            L.rxl_mem_update.argtypes = [P(rxl_ring), vp, ctypes.c_longlong, ctypes.c_int, vp]
            L.rxl_mem_update.restype = ctypes.c_int
            L.rxl_mem_update_rings.argtypes = [P(P(rxl_ring)), P(vp), P(ctypes.c_longlong), ctypes.c_int,
                                               ctypes.c_int, vp]
            L.rxl_mem_update_rings.restype = ctypes.c_int
            L.rxl_status_string.argtypes = [ctypes.c_int]
            L.rxl_status_string.restype = ctypes.c_char_p
            L.rxl_last_cuda_error.argtypes = []
            L.rxl_last_cuda_error.restype = ctypes.c_int
            L.rxl_last_launch_count.argtypes = []
            L.rxl_last_launch_count.restype = ctypes.c_int
            L.rxl_device_error_flags.argtypes = []
            L.rxl_device_error_flags.restype = ctypes.c_int
            L.rxl_attn_fwd_ex.argtypes = [P(rxl_attn_desc)] + [vp] * 9 + [vp]
            L.rxl_attn_fwd_ex.restype = ctypes.c_int
            L.rxl_attn_bwd_ex.argtypes = [P(rxl_attn_desc)] + [vp] * 17 + [ctypes.c_size_t, vp]
            L.rxl_attn_bwd_ex.restype = ctypes.c_int
            L.rxl_attn_fwd_reset.argtypes = [P(rxl_attn_desc)] + [vp] * 10 + [vp]
            L.rxl_attn_fwd_reset.restype = ctypes.c_int
            L.rxl_attn_bwd_reset.argtypes = [P(rxl_attn_desc)] + [vp] * 18 + [ctypes.c_size_t, vp]
            L.rxl_attn_bwd_reset.restype = ctypes.c_int
            L.rxl_qkv_proj.argtypes = [P(rxl_attn_desc), ctypes.c_int] + [vp] * 8 + [vp]
            L.rxl_qkv_proj.restype = ctypes.c_int
            L.rxl_layer_fwd_workspace_bytes.argtypes = [P(rxl_attn_desc), ctypes.c_int, ctypes.c_int]
            L.rxl_layer_fwd_workspace_bytes.restype = ctypes.c_size_t
            L.rxl_layer_fwd.argtypes = [P(rxl_attn_desc), ctypes.c_int, ctypes.c_int, P(rxl_layer_weights)] \
                + [vp] * 4 + [ctypes.c_size_t, vp]
            L.rxl_layer_fwd.restype = ctypes.c_int
            ll = ctypes.c_longlong
            L.rxl_layernorm_fwd.argtypes = [P(rxl_norm_desc), vp, ll, vp, ll, vp, vp, vp, ll, vp, ll, vp, vp, vp]
            L.rxl_layernorm_fwd.restype = ctypes.c_int
            L.rxl_layernorm_bwd_workspace_bytes.argtypes = [P(rxl_norm_desc)]
            L.rxl_layernorm_bwd_workspace_bytes.restype = ctypes.c_size_t
            L.rxl_layernorm_bwd.argtypes = [P(rxl_norm_desc), vp, ll, vp, ll] + [vp] * 4 + [ll] + [vp] * 3 \
                + [ctypes.c_size_t, vp]
            L.rxl_layernorm_bwd.restype = ctypes.c_int
            L.rxl_token_logprob_fwd.argtypes = [P(rxl_logprob_desc), vp, ll] + [vp] * 7
            L.rxl_token_logprob_fwd.restype = ctypes.c_int
            L.rxl_token_logprob_bwd.argtypes = [P(rxl_logprob_desc), vp, ll] + [vp] * 6 + [ll, vp]
            L.rxl_token_logprob_bwd.restype = ctypes.c_int
            L.rxl_adamw_scalars_at.argtypes = [P(rxl_adamw_desc), ll, ctypes.c_float, ctypes.c_float,
                                               ctypes.c_uint32, P(rxl_adamw_scalars)]
            L.rxl_adamw_scalars_at.restype = ctypes.c_int
            L.rxl_adamw_step.argtypes = [P(rxl_adamw_desc), P(rxl_adamw_tensor), ctypes.c_int,
                                         P(rxl_adamw_scalars), vp, vp]
            L.rxl_adamw_step.restype = ctypes.c_int
            L.rxl_kernel_timing.argtypes = [ctypes.c_int]
            L.rxl_kernel_timing.restype = ctypes.c_int
            L.rxl_kernel_timing_read.argtypes = [ctypes.c_int, P(ctypes.c_double), P(ctypes.c_int)]
            L.rxl_kernel_timing_read.restype = ctypes.c_int
            L.rxl_test_fail_next_launch.argtypes = [ctypes.c_int]
            L.rxl_test_fail_next_launch.restype = None
            L.rxl_test_forward_wait_timeout.argtypes = [ctypes.c_longlong, ctypes.c_int]
            L.rxl_test_forward_wait_timeout.restype = ctypes.c_int
            L.rxl_attn_bwd_noalloc.argtypes = [P(rxl_attn_desc)] + [vp] * 15 + [vp]
            L.rxl_attn_bwd_noalloc.restype = ctypes.c_int
            L.rxl_attn_bwd_noalloc_max_scratch_bytes.argtypes = []
            L.rxl_attn_bwd_noalloc_max_scratch_bytes.restype = ctypes.c_size_t
            _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != RXL_OK:
        raise RxlError(status, where)


def make_desc(B, H, L, mem_cap, mem_len, mem_head=0, scale=0.125, dtype=RXL_DTYPE_BF16, dh=64):
    return rxl_attn_desc(B, H, L, dh, mem_cap, mem_len, mem_head, scale, dtype)


def rxl_attn_fwd(desc, q, k, v, r, u, vbias, o, lse, stream=None):
    _check(lib().rxl_attn_fwd(ctypes.byref(desc), *map(_ptr, (q, k, v, r, u, vbias, o, lse)),
                              _stream(stream)), "rxl_attn_fwd")


def rxl_attn_fwd_ex(desc, q, k, v, r, u, vbias, o, o_lo, lse, stream=None):
    _check(lib().rxl_attn_fwd_ex(ctypes.byref(desc), *map(_ptr, (q, k, v, r, u, vbias, o, o_lo, lse)),
                                 _stream(stream)), "rxl_attn_fwd_ex")


def rxl_attn_bwd_ex(desc, q, k, v, r, u, vbias, o, o_lo, lse, dout, dq, dk, dv, dr, du, dvbias,
                    workspace, workspace_bytes, stream=None):
    _check(lib().rxl_attn_bwd_ex(ctypes.byref(desc),
                                 *map(_ptr, (q, k, v, r, u, vbias, o, o_lo, lse, dout, dq, dk, dv, dr,
                                             du, dvbias, workspace)),
                                 int(workspace_bytes), _stream(stream)), "rxl_attn_bwd_ex")


def rxl_attn_fwd_reset(desc, mem_visible, q, k, v, r, u, vbias, o, o_lo, lse, stream=None):
    _check(lib().rxl_attn_fwd_reset(ctypes.byref(desc),
                                    *map(_ptr, (mem_visible, q, k, v, r, u, vbias, o, o_lo, lse)),
                                    _stream(stream)), "rxl_attn_fwd_reset")


def rxl_attn_bwd_reset(desc, mem_visible, q, k, v, r, u, vbias, o, o_lo, lse, dout, dq, dk, dv, dr,
                       du, dvbias, workspace, workspace_bytes, stream=None):
    _check(lib().rxl_attn_bwd_reset(ctypes.byref(desc),
                                    *map(_ptr, (mem_visible, q, k, v, r, u, vbias, o, o_lo, lse, dout,
                                                dq, dk, dv, dr, du, dvbias, workspace)),
                                    int(workspace_bytes), _stream(stream)), "rxl_attn_bwd_reset")


def rxl_qkv_proj(desc, d_model, h_mem, h_cur, w_q, w_k, w_v, q, k, v, stream=None):
    _check(lib().rxl_qkv_proj(ctypes.byref(desc), int(d_model),
                              *map(_ptr, (h_mem, h_cur, w_q, w_k, w_v, q, k, v)), _stream(stream)),
           "rxl_qkv_proj")


def rxl_layer_fwd_workspace_bytes(desc, d_model, d_ff) -> int:
    return int(lib().rxl_layer_fwd_workspace_bytes(ctypes.byref(desc), int(d_model), int(d_ff)))


def rxl_layer_fwd(desc, d_model, d_ff, weights, h_mem, h_in, h_out, workspace, workspace_bytes,
                  stream=None):
    _check(lib().rxl_layer_fwd(ctypes.byref(desc), int(d_model), int(d_ff), ctypes.byref(weights),
                               *map(_ptr, (h_mem, h_in, h_out, workspace)), int(workspace_bytes),
                               _stream(stream)), "rxl_layer_fwd")


def rxl_attn_bwd_workspace_bytes(desc) -> int:
    return int(lib().rxl_attn_bwd_workspace_bytes(ctypes.byref(desc)))


def rxl_attn_bwd(desc, q, k, v, r, u, vbias, o, lse, dout, dq, dk, dv, dr, du, dvbias,
                 workspace, workspace_bytes, stream=None):
    _check(lib().rxl_attn_bwd(ctypes.byref(desc),
                              *map(_ptr, (q, k, v, r, u, vbias, o, lse, dout, dq, dk, dv, dr, du,
                                          dvbias, workspace)),
                              int(workspace_bytes), _stream(stream)), "rxl_attn_bwd")


def rxl_attn_bwd_noalloc(desc, q, k, v, r, u, vbias, o, lse, dout, dq, dk, dv, dr, du, dvbias,
                         stream=None):
    """rxl_attn_bwd for callers that cannot allocate: the scratch is a fixed
    array inside the library (see include/rxl.h for its size and rules)."""
    _check(lib().rxl_attn_bwd_noalloc(ctypes.byref(desc),
                                      *map(_ptr, (q, k, v, r, u, vbias, o, lse, dout, dq, dk, dv,
                                                  dr, du, dvbias)),
                                      _stream(stream)), "rxl_attn_bwd_noalloc")


def rxl_attn_bwd_noalloc_max_scratch_bytes() -> int:
    return int(lib().rxl_attn_bwd_noalloc_max_scratch_bytes())


def rxl_mem_update(ring: rxl_ring, src, src_plane_stride: int, L: int, stream=None):
    _check(lib().rxl_mem_update(ctypes.byref(ring), _ptr(src), int(src_plane_stride), int(L),
                                _stream(stream)), "rxl_mem_update")


def rxl_mem_update_rings(rings, srcs, src_plane_strides, L: int, stream=None):
    """rxl_mem_update of several rings of one geometry in one launch; the
    rxl_ring structs in `rings` are advanced in place."""
    n = len(rings)
    ring_ptrs = (ctypes.POINTER(rxl_ring) * n)(*[ctypes.pointer(r) for r in rings])
    src_arr = (ctypes.c_void_p * n)(*[_ptr(x) for x in srcs])
    str_arr = (ctypes.c_longlong * n)(*[int(x) for x in src_plane_strides])
    _check(lib().rxl_mem_update_rings(ring_ptrs, src_arr, str_arr, n, int(L), _stream(stream)),
           "rxl_mem_update_rings")


# ---- the rest of a training step. A tensor given to these must live on the
# current device and have the element type its place asks for (ValueError):
# the kernels would read a host address or misread the elements.

class _Torch:
    """What the calls below look up in torch, once: these take about as long
    on the host as the launch itself, so their overhead is kept small."""
    kinds = None  # torch types of the library's dtypes and of "f32" and "i32" places

    @classmethod
    def bind(cls):
        import torch
        cls.tensor = torch.Tensor
        cls.device = staticmethod(torch._C._cuda_getDevice)
        cls.stream = staticmethod(torch._C._cuda_getCurrentRawStream)
        cls.kinds = {RXL_DTYPE_F32: torch.float32, RXL_DTYPE_BF16: torch.bfloat16, "f32": torch.float32,
                     "i32": torch.int32}


def _current_device():
    """The current CUDA device; -2, which no tensor is on, where there is none."""
    if _Torch.kinds is None:
        _Torch.bind()
    try:
        return _Torch.device()
    except RuntimeError:
        return -2


def _current_stream(stream, device):
    return _Torch.stream(device) if stream is None else _stream(stream)


def _addresses(device, kind, *tensors):
    """Addresses of tensors (or addresses, or None) that hold `kind`; a kind
    without a torch type (workspaces, a dtype the library will refuse) is any."""
    want, cls = _Torch.kinds.get(kind), _Torch.tensor
    return [t.data_ptr() if t.__class__ is cls and t.dtype is want and t.get_device() == device
            else _address(device, want, t) for t in tensors]


def _address(device, want, t):
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != device or (want is not None and t.dtype is not want):  # -1: a host tensor
        raise ValueError(f"a tensor of {t.dtype} on {t.device} was given where {want or 'any type'} on the current "
                         "CUDA device is read")
    return t.data_ptr()


def make_norm_desc(rows, D, eps=1e-5, dtype=RXL_DTYPE_BF16):
    return rxl_norm_desc(rows, D, eps, dtype)


def rxl_layernorm_fwd(desc, x, x_stride, residual, residual_stride, gamma, beta, y, y_stride, sum, sum_stride,
                      mean, rstd, stream=None):
    d = _current_device()
    x, residual, gamma, beta, y, sum = _addresses(d, desc.dtype, x, residual, gamma, beta, y, sum)
    mean, rstd = _addresses(d, "f32", mean, rstd)
    _check(lib().rxl_layernorm_fwd(ctypes.byref(desc), x, x_stride, residual, residual_stride, gamma, beta, y,
                                   y_stride, sum, sum_stride, mean, rstd, _current_stream(stream, d)),
           "rxl_layernorm_fwd")


def rxl_layernorm_bwd_workspace_bytes(desc) -> int:
    return int(lib().rxl_layernorm_bwd_workspace_bytes(ctypes.byref(desc)))


def rxl_layernorm_bwd(desc, dy, dy_stride, s, s_stride, gamma, mean, rstd, dx, dx_stride, dgamma, dbeta,
                      workspace, workspace_bytes, stream=None):
    d = _current_device()
    dy, s, gamma, dx = _addresses(d, desc.dtype, dy, s, gamma, dx)
    mean, rstd, dgamma, dbeta = _addresses(d, "f32", mean, rstd, dgamma, dbeta)
    _check(lib().rxl_layernorm_bwd(ctypes.byref(desc), dy, dy_stride, s, s_stride, gamma, mean, rstd, dx, dx_stride,
                                   dgamma, dbeta, _address(d, None, workspace), int(workspace_bytes),
                                   _current_stream(stream, d)), "rxl_layernorm_bwd")


def make_logprob_desc(rows, V, top_k=0, dtype=RXL_DTYPE_BF16):
    return rxl_logprob_desc(rows, V, top_k, dtype)


def rxl_token_logprob_fwd(desc, logits, logits_stride, tokens, logp, lse, entropy, top_ids, top_logp, stream=None):
    d = _current_device()
    logits, = _addresses(d, desc.dtype, logits)
    tokens, top_ids = _addresses(d, "i32", tokens, top_ids)
    logp, lse, entropy, top_logp = _addresses(d, "f32", logp, lse, entropy, top_logp)
    _check(lib().rxl_token_logprob_fwd(ctypes.byref(desc), logits, logits_stride, tokens, logp, lse, entropy,
                                       top_ids, top_logp, _current_stream(stream, d)), "rxl_token_logprob_fwd")


def rxl_token_logprob_bwd(desc, logits, logits_stride, tokens, lse, entropy, dlogp, dentropy, dlogits,
                          dlogits_stride, stream=None):
    d = _current_device()
    logits, dlogits = _addresses(d, desc.dtype, logits, dlogits)
    tokens, = _addresses(d, "i32", tokens)
    lse, entropy, dlogp, dentropy = _addresses(d, "f32", lse, entropy, dlogp, dentropy)
    _check(lib().rxl_token_logprob_bwd(ctypes.byref(desc), logits, logits_stride, tokens, lse, entropy, dlogp,
                                       dentropy, dlogits, dlogits_stride, _current_stream(stream, d)),
           "rxl_token_logprob_bwd")


def make_adamw_desc(param_dtype=RXL_DTYPE_BF16, grad_dtype=RXL_DTYPE_BF16, state_bits=32, beta1=0.9, beta2=0.999,
                    eps=1e-8):
    return rxl_adamw_desc(param_dtype, grad_dtype, state_bits, beta1, beta2, eps)


def _check_adamw_sizes(t):
    """ValueError unless the tensors of one entry hold its n elements in one
    order. The list is made once, so this costs a step nothing."""
    n = t["n"]
    held = {k: t.get(k) for k in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")}
    held = {k: x for k, x in held.items() if x is not None and not isinstance(x, int)}
    for k, x in held.items():
        need = -(-n // 128) if k.endswith("_scale") else n
        if x.numel() < need:
            raise ValueError(f"{k} has {x.numel()} elements where {need} are read")
    if n == 0 or all(x.is_contiguous() for x in held.values()):
        return
    full = [x for k, x in held.items() if not k.endswith("_scale")]
    alike = all(x.shape == full[0].shape and x.stride() == full[0].stride() for x in full)
    for k, x in held.items():
        # without gaps: the last element lies numel - 1 places behind the first
        dense = sum((s - 1) * d for s, d in zip(x.shape, x.stride())) == x.numel() - 1
        if not x.is_contiguous() and not (alike and dense and not k.endswith("_scale")):
            raise ValueError(f"{k} is not contiguous (nor without gaps and in one order with the entry's other tensors)")


def make_adamw_tensors(desc, tensors):
    """The list rxl_adamw_step takes, from dicts with the fields of
    rxl_adamw_tensor (master, m_scale, v_scale and weight_decay may be left
    out). An entry's tensors hold n elements or more (scales one for every
    128), contiguous, or all in one other order without gaps (ValueError). The
    list holds addresses only: keep it with the tensors, for as long as they
    stay where they are."""
    out, d = (rxl_adamw_tensor * max(len(tensors), 1))(), _current_device()
    state = None if desc.state_bits == 8 else "f32"
    for i, t in enumerate(tensors):
        _check_adamw_sizes(t)
        m, v = t.get("m"), t.get("v")
        if desc.state_bits == 8 and any(getattr(x, "itemsize", 1) != 1 for x in (m, v)):
            raise ValueError("8-bit states are tensors of one byte an element")
        param, = _addresses(d, desc.param_dtype, t.get("param"))
        grad, = _addresses(d, desc.grad_dtype, t.get("grad"))
        m, v = _addresses(d, state, m, v)
        master, m_scale, v_scale = _addresses(d, "f32", t.get("master"), t.get("m_scale"), t.get("v_scale"))
        out[i] = rxl_adamw_tensor(param, master, grad, m, v, m_scale, v_scale, t["n"], t.get("weight_decay", 0.0))
    return out


def rxl_adamw_scalars_at(desc, step, lr, grad_scale=1.0, seed=0) -> rxl_adamw_scalars:
    out = rxl_adamw_scalars()
    _check(lib().rxl_adamw_scalars_at(ctypes.byref(desc), step, lr, grad_scale, seed, ctypes.byref(out)),
           "rxl_adamw_scalars_at")
    return out


def rxl_adamw_step(desc, tensors, n, scalars, scalars_dev, stream=None):
    if n > (0 if tensors is None else len(tensors)):
        raise ValueError(f"{n} tensors of a list of {0 if tensors is None else len(tensors)}")
    d = _current_device()
    _check(lib().rxl_adamw_step(ctypes.byref(desc), tensors, n, None if scalars is None else ctypes.byref(scalars),
                                _address(d, None, scalars_dev), _current_stream(stream, d)), "rxl_adamw_step")


RXL_KERNEL_FWD, RXL_KERNEL_BWD_MAIN, RXL_KERNEL_BWD_PREP, RXL_KERNEL_BWD_FINISH = 0, 1, 2, 3


def rxl_kernel_timing(enable: bool):
    rc = lib().rxl_kernel_timing(1 if enable else 0)
    if rc:
        raise RuntimeError(f"rxl_kernel_timing: cuda error {rc}")


def rxl_kernel_timing_read(kernel: int):
    """(summed device ms, timed launches) of kernel since the last read."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int(0)
    rc = lib().rxl_kernel_timing_read(int(kernel), ctypes.byref(ms), ctypes.byref(n))
    if rc:
        raise RuntimeError(f"rxl_kernel_timing_read: cuda error {rc}")
    return ms.value, n.value


def rxl_status_string(status: int) -> str:
    return lib().rxl_status_string(int(status)).decode()


def rxl_last_launch_count() -> int:
    return int(lib().rxl_last_launch_count())


def rxl_device_error_flags() -> int:
    return int(lib().rxl_device_error_flags())
