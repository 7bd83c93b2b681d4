"""Python binding of the padding-removed encoder-layer library (include/rpp.h).

Each function here marshals torch CUDA tensors into the C ABI call of the same name
(``remove_padding`` -> ``rpp_remove_padding`` ...) on the current CUDA stream and
raises :class:`RppError` on a negative status.  Every step of the path runs in the
library's CUDA kernels; PyTorch only provides device memory and the stream.  The
library must have been built (``python -m remove_padding_prefix_gb300.build``); there
is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

import numpy as np
import torch

from . import _abi
from ._abi import (RPP_F32, RPP_F16, RPP_BF16, RPP_I8, RPP_E4M3, RPP_EPI_BIAS, RPP_EPI_BIAS_GELU,  # noqa: F401
                   RPP_EPI_BIAS_RESIDUAL, RPP_DERR_LENGTH, RPP_DERR_TIMEOUT, RPP_DERR_ROWS, RPP_DERR_TMEM,
                   RPP_DERR_SLOT, RPP_DERR_PAGE, RPP_DERR_FULL, EncoderCfg, LayerSrc, SwinCfg, SwinSrc, MergeCfg, KvCfg,
                   KvArrays, Kv8Cfg, Kv8Arrays)

__all__ = [
    "RppError", "lib", "torch_dtype", "dtype_code", "build_offsets", "remove_padding", "rebuild_padding", "linear",
    "layernorm", "attention_varlen", "attention_varlen_i8", "encoder_cfg", "EncoderLayer", "encoder_layer_forward",
    "encoder_layer_calibrate", "encoder_forward", "quantize_weight", "quantize_activation", "gemm_i8_i32",
    "swin_cfg", "SwinBlock", "swin_prepare_bias", "window_attention_forward", "swin_block_forward",
    "merge_cfg", "PatchMerge", "patch_merge_forward",
    "KvCache", "KvCache8", "kv_reserve", "kv_append", "kv_read", "kv_fork", "kv_free", "kv_compact",
    "attention_causal_varlen", "attention_decode_workspace", "attention_decode",
    "get_device_error", "new_error_word",
]

_DT = {"fp32": RPP_F32, "fp16": RPP_F16, "bf16": RPP_BF16, "int8": RPP_F16}
_TORCH = {RPP_F32: torch.float32, RPP_F16: torch.float16, RPP_BF16: torch.bfloat16, RPP_I8: torch.int8}


class RppError(RuntimeError):
    def __init__(self, name, status):
        msg = lib().rpp_status_string(status).decode()
        super().__init__(f"{name} failed: {msg} ({status})")
        self.status = status


def lib():
    return _abi.load()


_CODE = {t: code for code, t in _TORCH.items()}


def dtype_code(dt) -> int:
    if isinstance(dt, str):
        return _DT[dt]
    if dt in _CODE:
        return _CODE[dt]
    raise ValueError(dt)


def torch_dtype(dt) -> torch.dtype:
    return _TORCH[dtype_code(dt) if not isinstance(dt, int) else dt]


def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(name, status):
    if status != 0:
        raise RppError(name, status)


def new_error_word(device="cuda") -> torch.Tensor:
    """A zeroed int32 device error word."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def get_device_error(err: torch.Tensor, stream=None) -> int:
    code = C.c_int32(0)
    st = lib().rpp_get_device_error(_p(err), C.byref(code), _stream(stream))
    if st not in (0, _abi.RPP_EDEVICE):
        raise RppError("rpp_get_device_error", st)
    return code.value


# ---------------------------------------------------------------- padding removal
def build_offsets(lengths: torch.Tensor, L: int, cu_seqlens=None, padding_offset=None, err=None, stream=None):
    B = lengths.numel()
    dev = lengths.device
    cu = cu_seqlens if cu_seqlens is not None else torch.empty(B + 1, dtype=torch.int32, device=dev)
    po = padding_offset if padding_offset is not None else torch.zeros(B * L, dtype=torch.int32, device=dev)
    _check("rpp_build_offsets", lib().rpp_build_offsets(_p(lengths), B, L, _p(cu), _p(po), _p(err), _stream(stream)))
    return cu, po


def remove_padding(padded: torch.Tensor, padding_offset, cu_seqlens, B: int, L: int, packed=None, err=None,
                   stream=None):
    H = padded.shape[-1]
    out = packed if packed is not None else torch.empty(B * L, H, dtype=padded.dtype, device=padded.device)
    _check("rpp_remove_padding", lib().rpp_remove_padding(_p(padded), _p(padding_offset), _p(cu_seqlens), B, L, H,
                                                          dtype_code(padded.dtype), _p(out), _p(err),
                                                          _stream(stream)))
    return out


def rebuild_padding(packed: torch.Tensor, cu_seqlens, B: int, L: int, padded=None, err=None, stream=None):
    H = packed.shape[-1]
    out = padded if padded is not None else torch.empty(B * L, H, dtype=packed.dtype, device=packed.device)
    _check("rpp_rebuild_padding", lib().rpp_rebuild_padding(_p(packed), _p(cu_seqlens), B, L, H,
                                                            dtype_code(packed.dtype), _p(out), _p(err),
                                                            _stream(stream)))
    return out


# ---------------------------------------------------------------- building blocks
def linear(a, w_t, bias, epilogue=RPP_EPI_BIAS, residual=None, out=None, rows=None, err=None, stream=None):
    M, K = a.shape
    N = w_t.shape[0]
    o = out if out is not None else torch.empty(M, N, dtype=a.dtype, device=a.device)
    _check("rpp_linear", lib().rpp_linear(_p(a), _p(w_t), _p(bias), _p(residual), _p(o), M, _p(rows), N, K,
                                          dtype_code(a.dtype), epilogue, _p(err), _stream(stream)))
    return o


def layernorm(x, gamma, beta, eps, out=None, rows=None, err=None, stream=None):
    M, H = x.shape
    o = out if out is not None else torch.empty_like(x)
    _check("rpp_layernorm", lib().rpp_layernorm(_p(x), _p(gamma), _p(beta), _p(o), M, _p(rows), H, float(eps),
                                                dtype_code(x.dtype), _p(err), _stream(stream)))
    return o


def attention_varlen(qkv, cu_seqlens, B: int, max_len: int, nh: int, d: int = 64, out=None, err=None, stream=None):
    T_max = qkv.shape[0]
    o = out if out is not None else torch.empty(T_max, nh * d, dtype=qkv.dtype, device=qkv.device)
    _check("rpp_attention_varlen", lib().rpp_attention_varlen(_p(qkv), _p(cu_seqlens), B, T_max, max_len, nh, d,
                                                              dtype_code(qkv.dtype), _p(o), _p(err),
                                                              _stream(stream)))
    return o


def attention_varlen_i8(qkv_codes, qkv_scales, cu_seqlens, B: int, max_len: int, nh: int, d: int = 64, out=None,
                        err=None, stream=None):
    """Attention on int8 codes held in a bf16 [T_max, 3*nh*d] tensor; qkv_scales: device
    float32[3] (s_q, s_k, s_v); returns the fp16 [T_max, nh*d] output."""
    T_max = qkv_codes.shape[0]
    o = out if out is not None else torch.empty(T_max, nh * d, dtype=torch.float16, device=qkv_codes.device)
    _check("rpp_attention_varlen_i8", lib().rpp_attention_varlen_i8(_p(qkv_codes), _p(qkv_scales), _p(cu_seqlens), B,
                                                                    T_max, max_len, nh, d, _p(o), _p(err),
                                                                    _stream(stream)))
    return o


# ---------------------------------------------------------------- encoder layer
def encoder_cfg(H, nh, F, eps, dtype, int8=False, tokens_hint=0) -> EncoderCfg:
    code = dtype_code(dtype) if not isinstance(dtype, int) else dtype
    return EncoderCfg(H, nh, H // nh, F, float(eps), code, int(int8), int(tokens_hint))


class EncoderLayer:
    """One prepared layer: the library-private weight block in device memory."""

    def __init__(self, cfg: EncoderCfg, weights: dict, device="cuda", stream=None):
        self.cfg = cfg
        nbytes = lib().rpp_layer_bytes(C.byref(cfg))
        if nbytes == 0:
            raise RppError("rpp_layer_bytes", _abi.RPP_EINVAL)
        self.block = torch.empty(nbytes, dtype=torch.uint8, device=device)
        tdt = _TORCH[cfg.dtype]
        H = cfg.hidden
        up = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(device=device, dtype=tdt).contiguous()
        W = weights["Wqkv"]
        b = weights["bqkv"]
        tens = {
            "Wq": up(W[:, :H]), "Wk": up(W[:, H:2 * H]), "Wv": up(W[:, 2 * H:]),
            "bq": up(b[:H]), "bk": up(b[H:2 * H]), "bv": up(b[2 * H:]),
            "Wo": up(weights["Wo"]), "bo": up(weights["bo"]), "W1": up(weights["W1"]), "b1": up(weights["b1"]),
            "W2": up(weights["W2"]), "b2": up(weights["b2"]),
            "gamma1": up(weights["gamma1"]), "beta1": up(weights["beta1"]),
            "gamma2": up(weights["gamma2"]), "beta2": up(weights["beta2"]),
        }
        src = LayerSrc(**{k: v.data_ptr() for k, v in tens.items()})
        _check("rpp_prepare_layer", lib().rpp_prepare_layer(C.byref(cfg), C.byref(src), _p(self.block),
                                                            _stream(stream)))
        (stream or torch.cuda.current_stream()).synchronize()   # the source tensors die here
        del tens

    def workspace_bytes(self, T_max: int) -> int:
        return lib().rpp_encoder_workspace_bytes(C.byref(self.cfg), T_max)

    def workspace(self, T_max: int, device="cuda") -> torch.Tensor:
        return torch.empty(self.workspace_bytes(T_max), dtype=torch.uint8, device=device)


def encoder_layer_forward(layer: EncoderLayer, x, cu_seqlens, B: int, max_len: int, y=None, workspace=None,
                          act_scales=None, err=None, stream=None):
    T_max = x.shape[0]
    out = y if y is not None else torch.empty_like(x)
    ws = workspace if workspace is not None else layer.workspace(T_max, x.device)
    _check("rpp_encoder_layer_forward",
           lib().rpp_encoder_layer_forward(C.byref(layer.cfg), _p(layer.block), _p(act_scales), _p(x),
                                           _p(cu_seqlens), B, T_max, max_len, _p(out), _p(ws), ws.numel(), _p(err),
                                           _stream(stream)))
    return out


def encoder_layer_calibrate(layer: EncoderLayer, x, cu_seqlens, B: int, max_len: int, workspace=None, err=None,
                            stream=None):
    T_max = x.shape[0]
    amax = torch.empty(7, dtype=torch.float32, device=x.device)
    ws = workspace if workspace is not None else layer.workspace(T_max, x.device)
    _check("rpp_encoder_layer_calibrate",
           lib().rpp_encoder_layer_calibrate(C.byref(layer.cfg), _p(layer.block), _p(x), _p(cu_seqlens), B, T_max,
                                             max_len, _p(amax), _p(ws), ws.numel(), _p(err), _stream(stream)))
    return amax


def encoder_forward(layers: Sequence[EncoderLayer], lengths, x_padded, L: int, act_scales=None, y_padded=None,
                    cu_seqlens=None, padding_offset=None, packed=None, workspace=None, err=None, stream=None):
    """Offsets -> remove padding -> layers -> rebuild padding, one C ABI call."""
    B = lengths.numel()
    H = x_padded.shape[-1]
    dev = x_padded.device
    cfg = layers[0].cfg
    y = y_padded if y_padded is not None else torch.empty(B * L, H, dtype=x_padded.dtype, device=dev)
    cu = cu_seqlens if cu_seqlens is not None else torch.empty(B + 1, dtype=torch.int32, device=dev)
    po = padding_offset if padding_offset is not None else torch.zeros(B * L, dtype=torch.int32, device=dev)
    pk = packed if packed is not None else torch.empty(B * L, H, dtype=x_padded.dtype, device=dev)
    ws = workspace if workspace is not None else layers[0].workspace(B * L, dev)
    lp = (C.c_void_p * len(layers))(*[l.block.data_ptr() for l in layers])
    sp = None
    if act_scales is not None:
        sp = (C.c_void_p * len(layers))(*[s.data_ptr() for s in act_scales])
    _check("rpp_encoder_forward",
           lib().rpp_encoder_forward(C.byref(cfg), lp, sp, len(layers), _p(lengths), B, L, _p(x_padded), _p(y),
                                     _p(cu), _p(po), _p(pk), _p(ws), ws.numel(), _p(err), _stream(stream)))
    return y, cu, po


# ---------------------------------------------------------------- int8 pieces
def quantize_weight(w, stream=None):
    """w [K, N] (in, out) -> (codes int8 [N, K], s_w float32 [N])."""
    K, N = w.shape
    q = torch.empty(N, K, dtype=torch.int8, device=w.device)
    s = torch.empty(N, dtype=torch.float32, device=w.device)
    _check("rpp_quantize_weight", lib().rpp_quantize_weight(_p(w), K, N, dtype_code(w.dtype), _p(q), _p(s),
                                                            _stream(stream)))
    return q, s


def quantize_activation(x, scale, rows=None, err=None, stream=None):
    M, H = x.shape
    q = torch.empty(M, H, dtype=torch.int8, device=x.device)
    _check("rpp_quantize_activation", lib().rpp_quantize_activation(_p(x), _p(scale), _p(q), M, _p(rows), H,
                                                                    dtype_code(x.dtype), _p(err), _stream(stream)))
    return q


def gemm_i8_i32(aq, wq_t, workspace=None, err=None, stream=None):
    M, K = aq.shape
    N = wq_t.shape[0]
    acc = torch.empty(M, N, dtype=torch.int32, device=aq.device)
    nbytes = lib().rpp_gemm_i8_workspace_bytes(M, N, K)
    ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=aq.device)
    _check("rpp_gemm_i8_i32", lib().rpp_gemm_i8_i32(_p(aq), _p(wq_t), _p(acc), M, N, K, _p(ws), ws.numel(), _p(err),
                                                    _stream(stream)))
    return acc


# ---------------------------------------------------------------- Swin
def swin_cfg(I, C_, nh, w, s, mlp, eps, dtype) -> SwinCfg:
    code = dtype_code(dtype) if not isinstance(dtype, int) else dtype
    return SwinCfg(I, C_, nh, w, s, mlp, float(eps), code)


def swin_prepare_bias(cfg: SwinCfg, table, stream=None):
    N = cfg.window * cfg.window
    bias = torch.empty(cfg.heads, N, N, dtype=torch.float32, device=table.device)
    _check("rpp_swin_prepare_bias", lib().rpp_swin_prepare_bias(C.byref(cfg), _p(table), _p(bias), _stream(stream)))
    return bias


def window_attention_forward(cfg: SwinCfg, B: int, qkv, bias, out=None, err=None, stream=None):
    o = out if out is not None else torch.empty(qkv.shape[0], cfg.channels, dtype=qkv.dtype, device=qkv.device)
    _check("rpp_window_attention_forward",
           lib().rpp_window_attention_forward(C.byref(cfg), B, _p(qkv), _p(bias), _p(o), _p(err), _stream(stream)))
    return o


class SwinBlock:
    """One prepared Swin block (library-private weight block in device memory)."""

    def __init__(self, cfg: SwinCfg, weights: dict, device="cuda", stream=None):
        self.cfg = cfg
        nbytes = lib().rpp_swin_block_bytes(C.byref(cfg))
        if nbytes == 0:
            raise RppError("rpp_swin_block_bytes", _abi.RPP_EINVAL)
        self.block = torch.empty(nbytes, dtype=torch.uint8, device=device)
        tdt = _TORCH[cfg.dtype]
        up = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(device=device, dtype=tdt).contiguous()
        tens = {k: up(weights[k]) for k in ("gamma1", "beta1", "Wqkv", "bqkv", "table", "Wo", "bo", "gamma2",
                                            "beta2", "W1", "b1", "W2", "b2")}
        src = SwinSrc(**{k: v.data_ptr() for k, v in tens.items()})
        _check("rpp_swin_prepare_block", lib().rpp_swin_prepare_block(C.byref(cfg), C.byref(src), _p(self.block),
                                                                      _stream(stream)))
        (stream or torch.cuda.current_stream()).synchronize()
        del tens

    def workspace_bytes(self, B: int) -> int:
        return lib().rpp_swin_workspace_bytes(C.byref(self.cfg), B)

    def workspace(self, B: int, device="cuda") -> torch.Tensor:
        return torch.empty(self.workspace_bytes(B), dtype=torch.uint8, device=device)


def swin_block_forward(block: SwinBlock, x, B: int, y=None, workspace=None, err=None, stream=None):
    out = y if y is not None else torch.empty_like(x)
    ws = workspace if workspace is not None else block.workspace(B, x.device)
    _check("rpp_swin_block_forward",
           lib().rpp_swin_block_forward(C.byref(block.cfg), _p(block.block), B, _p(x), _p(out), _p(ws), ws.numel(),
                                        _p(err), _stream(stream)))
    return out


# ---------------------------------------------------------------- Swin patch merging
def merge_cfg(I, C_, eps, dtype) -> MergeCfg:
    code = dtype_code(dtype) if not isinstance(dtype, int) else dtype
    return MergeCfg(I, C_, float(eps), code)


class PatchMerge:
    """Prepared patch-merging weights (K-major reduction map, fp32 LayerNorm parameters)."""

    def __init__(self, cfg: MergeCfg, gamma, beta, W, device="cuda", stream=None):
        self.cfg = cfg
        nbytes = lib().rpp_patch_merge_bytes(C.byref(cfg))
        if nbytes == 0:
            raise RppError("rpp_patch_merge_bytes", _abi.RPP_EUNSUPPORTED)
        self.block = torch.empty(nbytes, dtype=torch.uint8, device=device)
        tdt = _TORCH[cfg.dtype]
        up = lambda a: torch.as_tensor(np.ascontiguousarray(a)).to(device=device, dtype=tdt).contiguous()
        g, b, w = up(gamma), up(beta), up(W)
        _check("rpp_patch_merge_prepare", lib().rpp_patch_merge_prepare(C.byref(cfg), _p(g), _p(b), _p(w),
                                                                        _p(self.block), _stream(stream)))
        (stream or torch.cuda.current_stream()).synchronize()

    def workspace(self, B: int, device="cuda") -> torch.Tensor:
        return torch.empty(lib().rpp_patch_merge_workspace_bytes(C.byref(self.cfg), B), dtype=torch.uint8,
                           device=device)


def patch_merge_forward(pm: PatchMerge, x, B: int, y=None, workspace=None, err=None, stream=None):
    I, C_ = pm.cfg.img, pm.cfg.channels
    out = y if y is not None else torch.empty(B * (I // 2) * (I // 2), 2 * C_, dtype=x.dtype, device=x.device)
    ws = workspace if workspace is not None else pm.workspace(B, x.device)
    _check("rpp_patch_merge_forward",
           lib().rpp_patch_merge_forward(C.byref(pm.cfg), _p(pm.block), B, _p(x), _p(out), _p(ws), ws.numel(),
                                         _p(err), _stream(stream)))
    return out


# ---------------------------------------------------------------- decoder serving: paged key-value cache
# These calls take a few microseconds on the GPU at their smallest, so their checks use the cheap
# accessors: get_device() (-1 off the GPU, so it also says whether there is one) and one
# reading each of shape and stride.
def _here(*tensors) -> int:
    """The current device's raw stream, once every tensor given is on that device."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected a tensor on the current device (cuda:{dev}), got one on {t.device}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _made(stream, make, *args, **kw):
    """make(*args, **kw), a tensor of the stream that the call runs on: memory of the current stream's could
    be in use by work queued there, or be given out there again while the call's stream still uses it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _ints(name, t, n=None):
    if t.dtype is not torch.int32 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name}: expected a contiguous int32 tensor" + (f" of {n}" if n is not None else ""))
    return t.data_ptr()


def _rows(name, t, width, dtype) -> int:
    """A 2D view of 16-bit rows whose columns are contiguous; returns the row stride in elements."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width or stride[1] != 1 or t.dtype is not dtype:
        raise ValueError(f"{name}: expected rows of {width} contiguous {dtype}")
    # the stride of a single row is whatever made the view: any valid one will do
    return stride[0] if shape[0] > 1 or (stride[0] >= width and stride[0] % 8 == 0) else width


class KvCache:
    """A paged key-value cache: the pool [layers, pages, 2, kv_heads, page_size, head_dim] and
    its table, lens and refs (include/rpp.h, "Decoder serving"), in device memory.

    ``err`` is the device error word that the calls use when none is given."""

    def __init__(self, layers, pages, page_size, kv_heads, head_dim, slots, max_pages, dtype="bf16", device="cuda"):
        self._bind(torch.empty(layers, pages, 2, kv_heads, page_size, head_dim, dtype=torch_dtype(dtype),
                               device=device),
                   torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device))
        self._own()

    @classmethod
    def from_tensors(cls, pool, table, lens, refs):
        """A cache over arrays that the caller holds already (kept, not copied)."""
        c = cls.__new__(cls)
        c._bind(pool, table, lens, refs)
        c._own()
        return c

    # the C calls of this kind of cache
    _calls = {name: f"rpp_kv_{name}" for name in ("reserve", "append", "read", "fork", "free", "compact",
                                                  "compact_workspace_bytes")}
    _calls |= {"decode": "rpp_attention_decode", "decode_workspace_bytes": "rpp_attention_decode_workspace_bytes"}

    def _call(self, name):
        """The C call, looked up once (a lookup costs a part of a launch)."""
        fn = self._fns.get(name)
        if fn is None:
            fn = self._fns[name] = getattr(lib(), self._calls[name])
        return fn

    _fns = {}

    def _rows_dtype(self, dtype):
        """The type of rows that go in and come out, given one, and how the C calls take it."""
        return self._dtype, ()

    def _own(self):
        self.err = new_error_word(self.pool.device)
        nbytes = self._call("compact_workspace_bytes")(self._cfg)
        # kv_compact's lists: of the cache, as the calls that change one are ordered anyway
        self._remap = torch.empty(self.cfg.pages, dtype=torch.int32, device=self.pool.device)
        self._lists = torch.empty(nbytes, dtype=torch.uint8, device=self.pool.device)

    def _bind(self, pool, table, lens, refs):
        if pool.dim() != 6 or pool.shape[2] != 2 or not pool.is_contiguous():
            raise ValueError("pool: expected a contiguous [layers, pages, 2, kv_heads, page_size, head_dim] tensor")
        if table.dim() != 2:
            raise ValueError("table: expected [slots, max_pages]")
        _ints("table", table)
        _ints("lens", lens, table.shape[0])
        _ints("refs", refs, pool.shape[1])
        if not all(t.is_cuda and t.device == pool.device for t in (pool, table, lens, refs)):
            raise ValueError("expected CUDA tensors on one device")
        self.pool, self.table, self.lens, self.refs = pool, table, lens, refs
        layers, pages, _, heads, rows, d = pool.shape
        self.cfg = KvCfg(layers, pages, rows, heads, d, table.shape[0], table.shape[1], self._pool_code())
        self._arrays = KvArrays(pool.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr())
        self._dtype, self._d, self._width = pool.dtype, d, heads * d
        self._bind_calls()

    def _pool_code(self):
        return dtype_code(self.pool.dtype)

    def _bind_calls(self):
        """What the C calls take."""
        self._cfg, self._cache = C.byref(self.cfg), C.byref(self._arrays)
        if lib().rpp_kv_pool_bytes(self._cfg) == 0:
            raise RppError("rpp_kv_pool_bytes", _abi.RPP_EUNSUPPORTED)

    def adopt(self, table, refs):
        """Take the table and counts that kv_compact wrote to arrays of their own."""
        self._bind(self.pool, table, self.lens, refs)


class KvCache8(KvCache):
    """A paged key-value cache held in 8 bits (include/rpp.h, "The same cache held in 8 bits"): the pool of int8 or e4m3
    codes and ``scales``, uint8 [layers, pages, 2, kv_heads, page_size // block], a scale byte for each ``block``
    tokens of a head.  Every call of a KvCache takes it: rows and queries are fp16 or bf16."""

    _calls = {name: call.replace("rpp_kv_", "rpp_kv8_").replace("decode", "decode8") for name, call in KvCache._calls.items()}
    _codes = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
    _fns = {}
    _row_types = {torch.float16: (torch.float16, (RPP_F16,)), torch.bfloat16: (torch.bfloat16, (RPP_BF16,))}

    def __init__(self, layers, pages, page_size, kv_heads, head_dim, slots, max_pages, dtype="e4m3", block=16,
                 device="cuda"):
        if dtype not in self._codes:
            raise ValueError(f"dtype: expected one of {sorted(self._codes)}")
        if block <= 0 or page_size % block:
            raise ValueError("block: expected a divisor of page_size")
        # (filled by the page: a byte of zeros is a scale, too)
        self.scales = torch.zeros(layers, pages, 2, kv_heads, page_size // block, dtype=torch.uint8, device=device)
        self._bind(torch.empty(layers, pages, 2, kv_heads, page_size, head_dim, dtype=self._codes[dtype], device=device),
                   torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device))
        self._own()

    @classmethod
    def from_tensors(cls, pool, scales, table, lens, refs):
        """A cache over arrays that the caller holds already (kept, not copied).

        scales: bytes 0 to 248, as rows of 16 bits give them, or 255 (NaN).  Those between stand for 2^122 to 2^127, but
        the attention takes K's of 254 for infinite."""
        c = cls.__new__(cls)
        c.scales = scales
        c._bind(pool, table, lens, refs)
        c._own()
        return c

    def _pool_code(self):
        if self.pool.dtype not in self._codes.values():
            raise ValueError("pool: expected int8 or float8_e4m3fn codes")
        return RPP_I8 if self.pool.dtype is torch.int8 else RPP_E4M3

    def _bind_calls(self):
        scales, pool = self.scales, self.pool
        if (scales.dim() != 5 or scales.shape[:4] != pool.shape[:4] or scales.dtype is not torch.uint8 or
                not scales.is_contiguous() or scales.device != pool.device or not scales.shape[4] or
                pool.shape[4] % scales.shape[4]):
            raise ValueError("scales: expected a contiguous uint8 [layers, pages, 2, kv_heads, page_size // block] tensor "
                             "beside the pool")
        self.block = pool.shape[4] // scales.shape[4]
        self._cfg8 = Kv8Cfg(self.cfg, self.block)
        self._arrays8 = Kv8Arrays(self._arrays, scales.data_ptr())
        self._cfg, self._cache = C.byref(self._cfg8), C.byref(self._arrays8)
        if lib().rpp_kv8_pool_bytes(self._cfg) == 0:
            raise RppError("rpp_kv8_pool_bytes", _abi.RPP_EUNSUPPORTED)

    def _rows_dtype(self, dtype):
        got = self._row_types.get(dtype)
        if got is None:
            raise ValueError(f"expected fp16 or bf16 rows, got {dtype}")
        return got


def kv_reserve(cache: KvCache, slots, counts, err=None, stream=None):
    """Room for counts[i] more tokens in slot slots[i] (both device int32[n])."""
    err = cache.err if err is None else err
    here = _here(cache.pool, slots, counts, err)
    n = slots.numel()
    _check(cache._calls["reserve"], cache._call("reserve")(cache._cfg, cache._cache, _ints("slots", slots),
                                                           _ints("counts", counts, n), n, err.data_ptr(),
                                                           here if stream is None else stream.cuda_stream))


def kv_append(cache: KvCache, layer: int, k, v, slots, cu_seqlens=None, err=None, stream=None):
    """Write the K and V rows of the last tokens of each sequence into one layer.

    k, v: [rows, kv_heads * head_dim] (column ranges of one QKV projection's output will
    do); rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 belong to slots[i], or row i without
    cu_seqlens."""
    err = cache.err if err is None else err
    here = _here(cache.pool, k, v, slots, cu_seqlens, err)
    n, rows = slots.numel(), k.shape[0]
    dtype, code = cache._rows_dtype(k.dtype)
    ld = _rows("k", k, cache._width, dtype)
    if _rows("v", v, cache._width, dtype) != ld or v.shape[0] != rows:
        raise ValueError("k and v: expected equal row counts and strides")
    _check(cache._calls["append"],
           cache._call("append")(cache._cfg, cache._cache, layer, k.data_ptr(), v.data_ptr(), *code, ld,
                                 _ints("slots", slots),
                                 None if cu_seqlens is None else _ints("cu_seqlens", cu_seqlens, n + 1), n, rows,
                                 err.data_ptr(), here if stream is None else stream.cuda_stream))


def kv_read(cache: KvCache, layer: int, slots, cu_seqlens=None, starts=None, rows=None, dtype=None, k=None, v=None,
            err=None, stream=None):
    """Rows of sequences read back from one layer, as kv_append takes them; returns (k, v).

    Rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 (row i without cu_seqlens) receive the tokens of slots[i] from position
    starts[i] on, or its last ones without starts.  k, v: where they go, [rows, kv_heads * head_dim]
    each (columns of one wider tensor will do; rows behind the last sequence stay as they are); without
    them a new tensor of ``rows`` rows (at least one; needed with cu_seqlens) and ``dtype`` (of a KvCache8: fp16 or bf16,
    bf16 by default) is made."""
    err = cache.err if err is None else err
    n, w = slots.numel(), cache._width
    if (k is None) != (v is None):
        raise ValueError("k and v: expected both or neither")
    if isinstance(dtype, str):
        dtype = torch_dtype(dtype)
    if k is None:
        if rows is None:
            if cu_seqlens is not None:
                raise ValueError("rows: needed with cu_seqlens where k and v are not given")
            rows = n
        if dtype is None:
            dtype = torch.bfloat16 if isinstance(cache, KvCache8) else cache._dtype
        got, code = cache._rows_dtype(dtype)
        if got is not dtype:
            raise ValueError(f"dtype: a cache of {got} has no rows of {dtype}")
        k, v = (_made(stream, torch.empty, (rows, w), dtype=dtype, device=cache.pool.device) for _ in range(2))
        ld = w
    else:
        if (rows is not None and rows != k.shape[0]) or (dtype is not None and dtype is not k.dtype):
            raise ValueError("rows and dtype: k and v, which are given, have their own")
        rows = k.shape[0]
        dtype, code = cache._rows_dtype(k.dtype)
        ld = _rows("k", k, w, dtype)
        if _rows("v", v, w, dtype) != ld or v.shape[0] != rows:
            raise ValueError("k and v: expected equal row counts and strides")
    here = _here(cache.pool, k, v, slots, cu_seqlens, starts, err)
    _check(cache._calls["read"],
           cache._call("read")(cache._cfg, cache._cache, layer, _ints("slots", slots),
                               None if starts is None else _ints("starts", starts, n),
                               None if cu_seqlens is None else _ints("cu_seqlens", cu_seqlens, n + 1), n, rows,
                               k.data_ptr(), v.data_ptr(), *code, ld, err.data_ptr(),
                               here if stream is None else stream.cuda_stream))
    return k, v


def kv_fork(cache: KvCache, src, dst, err=None, stream=None):
    """Slot dst[i] (empty) becomes a copy of slot src[i]; whole pages are shared."""
    err = cache.err if err is None else err
    here = _here(cache.pool, src, dst, err)
    n = src.numel()
    _check(cache._calls["fork"], cache._call("fork")(cache._cfg, cache._cache, _ints("src", src), _ints("dst", dst, n), n,
                                                     err.data_ptr(), here if stream is None else stream.cuda_stream))


def kv_free(cache: KvCache, slots, err=None, stream=None):
    """Empty the slots; pages that no sequence uses any more become free."""
    err = cache.err if err is None else err
    here = _here(cache.pool, slots, err)
    _check(cache._calls["free"], cache._call("free")(cache._cfg, cache._cache, _ints("slots", slots), slots.numel(),
                                                     err.data_ptr(), here if stream is None else stream.cuda_stream))


def kv_compact(cache: KvCache, table_out=None, refs_out=None, remap=None, live=None, err=None, stream=None):
    """Move the pages in use to the front of the pool; returns (table, refs, live).

    Without table_out and refs_out the cache's own arrays are rewritten; with both the old
    ones stay as they are (KvCache.adopt takes the new).  live: device int32[1]; remap:
    device int32[pages], each page's new number, for tables of the caller's own."""
    err = cache.err if err is None else err
    table = cache.table if table_out is None else table_out
    refs = cache.refs if refs_out is None else refs_out
    remap = cache._remap if remap is None else remap
    if live is None:
        live = _made(stream, torch.empty, 1, dtype=torch.int32, device=cache.pool.device)
    here = _here(cache.pool, table, refs, remap, live, err)
    cfg, lists = cache.cfg, cache._lists
    _check(cache._calls["compact"],
           cache._call("compact")(cache._cfg, cache._cache, _ints("table_out", table, cfg.slots * cfg.max_pages),
                                  _ints("refs_out", refs, cfg.pages), _ints("remap", remap, cfg.pages),
                                  _ints("live", live, 1), lists.data_ptr(), lists.numel(), err.data_ptr(),
                                  here if stream is None else stream.cuda_stream))
    return table, refs, live


def _out_like(q, out, rows, width, stream):
    if out is None:
        return _made(stream, torch.empty, (rows, width), dtype=q.dtype, device=q.device)
    if out.shape != (rows, width) or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError("out: expected a contiguous tensor like q")
    return out


def attention_causal_varlen(q, k, v, cu_seqlens, B: int, max_len: int, nh: int, nkv: int, d: int, scale=None, out=None,
                            err=None, stream=None):
    """Causal attention over packed prompts: q [T_max, nh * d], k and v [T_max, nkv * d] (column
    ranges of one QKV projection's output will do), scale 1 / sqrt(d) by default."""
    here = _here(q, k, v, cu_seqlens, out, err)
    T_max, dtype = q.shape[0], q.dtype
    ldq, ld = _rows("q", q, nh * d, dtype), _rows("k", k, nkv * d, dtype)
    if _rows("v", v, nkv * d, dtype) != ld or k.shape[0] != T_max or v.shape[0] != T_max:
        raise ValueError("q, k and v: expected equal row counts, k and v equal strides")
    o = _out_like(q, out, T_max, nh * d, stream)
    _check("rpp_attention_causal_varlen",
           lib().rpp_attention_causal_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), ldq, ld,
                                             _ints("cu_seqlens", cu_seqlens, B + 1), B, T_max, max_len, nh, nkv, d,
                                             dtype_code(dtype), d ** -0.5 if scale is None else scale, o.data_ptr(),
                                             None if err is None else err.data_ptr(),
                                             here if stream is None else stream.cuda_stream))
    return o


def attention_decode_workspace(cache: KvCache, n: int, nh: int) -> torch.Tensor:
    nbytes = cache._call("decode_workspace_bytes")(cache._cfg, n, nh)
    if nbytes == 0:
        raise RppError(cache._calls["decode_workspace_bytes"], _abi.RPP_EINVAL)
    return torch.empty(nbytes, dtype=torch.uint8, device=cache.pool.device)


def attention_decode(cache: KvCache, layer: int, q, slots=None, scale=None, out=None, workspace=None, err=None,
                     stream=None):
    """Attention of one new token per sequence over the cache (a KvCache or a KvCache8).

    q: [n, nh * head_dim] (a column range of a QKV projection's output will do); slots:
    device int32[n], or None for slots 0 .. n - 1; scale: 1 / sqrt(head_dim) by default."""
    err = cache.err if err is None else err
    d = cache._d
    n, width = q.shape
    nh = width // d
    ws = _made(stream, attention_decode_workspace, cache, n, nh) if workspace is None else workspace
    if not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    here = _here(cache.pool, q, slots, out, ws, err)
    dtype, code = cache._rows_dtype(q.dtype)
    ld = _rows("q", q, nh * d, dtype)
    o = _out_like(q, out, n, nh * d, stream)
    _check(cache._calls["decode"],
           cache._call("decode")(cache._cfg, cache._cache, layer, q.data_ptr(), *code, ld,
                                 None if slots is None else _ints("slots", slots, n), n, nh,
                                 d ** -0.5 if scale is None else scale, o.data_ptr(), ws.data_ptr(), ws.nbytes,
                                 err.data_ptr(), here if stream is None else stream.cuda_stream))
    return o
