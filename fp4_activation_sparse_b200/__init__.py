"""Python binding of libsharq: SharQ's online sparse-dense FP4 linear layer on B200.

Argument marshalling only (ctypes). Every computation runs in the library's CUDA
kernels; torch supplies device memory and streams. There is no CPU fallback: the
library is loaded on first use (so that ``fp4_activation_sparse_b200.build`` can run on
a fresh tree), and every call raises ImportError if ``libsharq.so`` is missing or does
not export what this binding expects.

The three calls of the method ("SharQ: Bridging Activation Sparsity and FP4
Quantization for LLM Inference", Abstract):
  sharq_pack_weight  - one FP4 weight payload with sparse-path and dense-path scale views
  sharq_prepare      - the fused preparation operator (RMSNorm, N:M mask, FP4 backbone,
                       residual against the quantized backbone, dense FP4 residual)
  sharq_prepare_swiglu - the same operator on a down projection's gated input SiLU(g)*u
  sharq_prepare_tensor_scale - the same operator with one NVFP4 second-level scale per tensor
  sharq_linear       - sparse FP4 GEMM + dense FP4 GEMM into one output
  sharq_linear_grouped - the same for many experts (mixture of experts) in one launch
and the library's dense FP4 baseline (the README's "NVFP4" mode):
  sharq_quantize_dense, sharq_linear_dense.

The attention side of a served transformer block, between those linear layers:
  sharq_kv_append    - per-head RMSNorm and rotation of q and k; k and v quantized into a paged
                       FP4 cache (KVCache, KVBatch; alloc_kv_cache)
  sharq_kv_read      - rows of that cache back as values
  sharq_attention    - attention over it: single tokens, several, whole prompts
  sharq_norm_residual - norms before and after a block, its gate, the scaled residual stream
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsharq.so")

SHARQ_NVFP4, SHARQ_MXFP4 = 0, 1
SHARQ_OUT_BF16, SHARQ_OUT_F32 = 0, 1
SHARQ_OK, SHARQ_ERR_INVALID_ARG, SHARQ_ERR_UNSUPPORTED, SHARQ_ERR_CUDA, SHARQ_ERR_TIMEOUT = range(5)
FMT = {"nvfp4": SHARQ_NVFP4, "mxfp4": SHARQ_MXFP4}
UNIT_ELEMENT, UNIT_PAIR = 1, 2


class SharqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"sharq status {status}: {message}")
        self.status = status


class _Prep(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("tokens", ctypes.c_int), ("k", ctypes.c_int), ("nm_n", ctypes.c_int),
                ("nm_m", ctypes.c_int), ("unit", ctypes.c_int), ("fmt", ctypes.c_int)]


class _WPack(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("n_out", ctypes.c_int), ("k", ctypes.c_int), ("fmt", ctypes.c_int)]


class _KVCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("fmt", ctypes.c_int)]


class _KVBatch(ctypes.Structure):
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_seq", ctypes.c_int), ("max_pages", ctypes.c_int), ("max_q", ctypes.c_int),
                ("tokens", ctypes.c_int)]


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m fp4_activation_sparse_b200.build`")
    lib = ctypes.CDLL(path)
    if not hasattr(lib, "sharq_dense_buffer_sizes") or not hasattr(lib, "sharq_norm_residual"):
        raise ImportError(f"{path} is stale (ABI older than this binding): rebuild it")
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L, KC, KB = ctypes.c_longlong, ctypes.POINTER(_KVCache), ctypes.POINTER(_KVBatch)
    sig = {
        "sharq_prep_buffer_sizes": (S, [I, I, I, I, I, I, ctypes.POINTER(S)]),
        "sharq_dense_buffer_sizes": (S, [I, I, I, ctypes.POINTER(S)]),
        "sharq_wpack_buffer_sizes": (S, [I, I, I, ctypes.POINTER(S)]),
        "sharq_pack_weight": (I, [P, I, I, I, ctypes.POINTER(_WPack), P]),
        "sharq_prepare": (I, [P, I, I, P, F, I, I, I, I, ctypes.POINTER(_Prep), P]),
        "sharq_prepare_tensor_scale_noalloc": (I, [P, I, I, P, F, I, I, I, I, ctypes.POINTER(_Prep), P]),
        "sharq_prepare_swiglu": (I, [P, I, I, I, I, I, I, ctypes.POINTER(_Prep), P]),
        "sharq_tensor_scale_workspace_size": (S, [I, I]),
        "sharq_prepare_tensor_scale": (I, [P, I, I, P, F, I, I, I, I, ctypes.POINTER(_Prep), P, P]),
        "sharq_linear": (I, [ctypes.POINTER(_Prep), ctypes.POINTER(_WPack), P, I, P]),
        "sharq_linear_workspace_size": (S, [I, I, I]),
        "sharq_linear_split": (I, [ctypes.POINTER(_Prep), ctypes.POINTER(_WPack), P, I, P, S, P]),
        "sharq_linear_grouped": (I, [ctypes.POINTER(_Prep), ctypes.POINTER(_WPack), ctypes.POINTER(P), I, I, P]),
        "sharq_quantize_dense": (I, [P, I, I, P, F, I, P, P, P]),
        "sharq_linear_dense": (I, [P, P, I, I, ctypes.POINTER(_WPack), P, I, P]),
        "sharq_rmsnorm": (I, [P, I, I, P, F, P, P]),
        "sharq_kv_page_bytes": (S, [I, I, I, I]),
        "sharq_kv_append": (I, [P, L, I, KC, KB, P, P, F, P, I, I, P, P]),
        "sharq_kv_read": (I, [KC, KB, P, P, I, P]),
        "sharq_attention_workspace_size": (S, [KC, KB, I]),
        "sharq_attention": (I, [P, L, I, KC, KB, I, I, F, P, P, P, S, P]),
        "sharq_norm_residual": (I, [P, P, I, I, P, P, I, I, F, P, F, P, P, P]),
        "sharq_mma_peak": (I, [I, I, I, I, P]),
        "sharq_device_status": (I, [P]),
        "sharq_set_wait_limit": (None, [ctypes.c_longlong]),
        "sharq_last_error": (ctypes.c_char_p, []),
        "sharq_version": (I, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


class _Lib:
    """The loaded libsharq.so, opened on first attribute access."""
    _cdll: ctypes.CDLL | None = None

    def __getattr__(self, name):
        if _Lib._cdll is None:
            _Lib._cdll = _load()
        return getattr(_Lib._cdll, name)


lib = _Lib()


def load() -> ctypes.CDLL:
    """Open libsharq.so now (raises ImportError if it is missing or stale)."""
    lib.sharq_version  # noqa: B018  (attribute access loads the library)
    return _Lib._cdll


def last_error() -> str:
    return lib.sharq_last_error().decode()


def _check(status: int):
    if status != SHARQ_OK:
        raise SharqError(status, last_error())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:  # the current stream's handle, without building a Stream object (3 us)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _fmt(fmt) -> int:
    return FMT[fmt] if isinstance(fmt, str) else int(fmt)


# ------------------------------------------------------------------ buffer holders
@dataclass
class Prep:
    """A prepared activation: the tiled operand, the row scales and the C struct."""
    tiles: torch.Tensor
    row_scale: torch.Tensor
    tokens: int
    k: int
    nm_n: int
    nm_m: int
    unit: int
    fmt: int
    c: _Prep = field(default=None, repr=False)

    def struct(self) -> _Prep:
        if self.c is None:
            self.c = _Prep(self.tiles.data_ptr(), self.row_scale.data_ptr(), self.tokens, self.k, self.nm_n,
                           self.nm_m, self.unit, self.fmt)
        return self.c


@dataclass
class WPack:
    """A packed weight: the tiled operand (codes and both scale views) and the tensor scale."""
    tiles: torch.Tensor
    tensor_scale: torch.Tensor
    n_out: int
    k: int
    fmt: int
    c: _WPack = field(default=None, repr=False)

    def struct(self) -> _WPack:
        if self.c is None:
            self.c = _WPack(self.tiles.data_ptr(), self.tensor_scale.data_ptr(), self.n_out, self.k, self.fmt)
        return self.c


def _sizes(fn, *args) -> list[int]:
    sizes = (ctypes.c_size_t * 2)()
    if fn(*args, sizes) == 0:
        raise SharqError(SHARQ_ERR_INVALID_ARG, last_error())
    return list(sizes)


def sharq_prep_buffer_sizes(tokens: int, k: int, nm_n: int, nm_m: int, unit: int, fmt) -> list[int]:
    return _sizes(lib.sharq_prep_buffer_sizes, tokens, k, nm_n, nm_m, unit, _fmt(fmt))


def sharq_dense_buffer_sizes(tokens: int, k: int, fmt) -> list[int]:
    return _sizes(lib.sharq_dense_buffer_sizes, tokens, k, _fmt(fmt))


def sharq_wpack_buffer_sizes(n_out: int, k: int, fmt) -> list[int]:
    return _sizes(lib.sharq_wpack_buffer_sizes, n_out, k, _fmt(fmt))


def _bytes(n: int, device) -> torch.Tensor:
    # 16-byte aligned (torch's caching allocator aligns to 512 bytes)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def alloc_prep(tokens: int, k: int, nm_n: int = 2, nm_m: int = 4, unit: int = UNIT_PAIR, fmt="nvfp4",
               device="cuda") -> Prep:
    s = sharq_prep_buffer_sizes(tokens, k, nm_n, nm_m, unit, fmt)
    return Prep(_bytes(s[0], device), torch.empty(tokens, dtype=torch.float32, device=device),
                tokens, k, nm_n, nm_m, unit, _fmt(fmt))


def alloc_wpack(n_out: int, k: int, fmt="nvfp4", device="cuda") -> WPack:
    s = sharq_wpack_buffer_sizes(n_out, k, fmt)
    return WPack(_bytes(s[0], device), torch.empty(4, dtype=torch.float32, device=device), n_out, k, _fmt(fmt))


# ------------------------------------------------------------------ the calls
def sharq_pack_weight(w: torch.Tensor, fmt="nvfp4", out: WPack | None = None, stream=None) -> WPack:
    """Pack a bf16 weight [n_out, k] (device) into one FP4 payload with two scale views."""
    assert w.dtype == torch.bfloat16 and w.is_cuda and w.is_contiguous()
    n_out, k = w.shape
    out = out or alloc_wpack(n_out, k, fmt, w.device)
    st = out.struct()
    _check(lib.sharq_pack_weight(_ptr(w), n_out, k, _fmt(fmt), ctypes.byref(st), _stream(stream)))
    return out


def sharq_prepare(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6, nm_n: int = 2,
                  nm_m: int = 4, unit: int = UNIT_PAIR, fmt="nvfp4", out: Prep | None = None, stream=None) -> Prep:
    """The fused preparation operator on bf16 activations [tokens, k] (device)."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous()
    tokens, k = x.shape
    if gamma is not None:
        assert gamma.dtype == torch.bfloat16 and gamma.is_cuda and gamma.numel() == k
    out = out or alloc_prep(tokens, k, nm_n, nm_m, unit, fmt, x.device)
    st = out.struct()
    _check(lib.sharq_prepare(_ptr(x), tokens, k, _ptr(gamma), ctypes.c_float(eps), nm_n, nm_m, unit, _fmt(fmt),
                             ctypes.byref(st), _stream(stream)))
    return out


def sharq_tensor_scale_workspace_size(tokens: int, k: int) -> int:
    n = lib.sharq_tensor_scale_workspace_size(tokens, k)
    if n == 0:
        raise SharqError(SHARQ_ERR_INVALID_ARG, last_error())
    return n


def sharq_prepare_tensor_scale(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6,
                               nm_n: int = 2, nm_m: int = 4, unit: int = UNIT_PAIR, fmt="nvfp4",
                               out: Prep | None = None, workspace: torch.Tensor | None = None,
                               stream=None) -> Prep:
    """sharq_prepare with one NVFP4 second-level scale for the whole tensor (every row_scale
    entry holds it). One cooperative launch; `workspace` carries its grid barrier: device bytes
    zeroed once before first use (allocated zeroed here if omitted), reusable afterwards."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous()
    tokens, k = x.shape
    if gamma is not None:
        assert gamma.dtype == torch.bfloat16 and gamma.is_cuda and gamma.numel() == k
    out = out or alloc_prep(tokens, k, nm_n, nm_m, unit, fmt, x.device)
    if workspace is None:
        workspace = torch.zeros(sharq_tensor_scale_workspace_size(tokens, k), dtype=torch.uint8, device=x.device)
    st = out.struct()
    _check(lib.sharq_prepare_tensor_scale(_ptr(x), tokens, k, _ptr(gamma), ctypes.c_float(eps), nm_n, nm_m, unit,
                                          _fmt(fmt), ctypes.byref(st), _ptr(workspace), _stream(stream)))
    return out


def sharq_prepare_tensor_scale_noalloc(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6,
                                       nm_n: int = 2, nm_m: int = 4, unit: int = UNIT_PAIR, fmt="nvfp4",
                                       out: Prep | None = None, stream=None) -> Prep:
    """sharq_prepare_tensor_scale without a workspace: for callers that may not allocate device
    memory, the library's own static scratch carries the grid barrier (calls that overlap on the
    GPU race on it). Only the output holder is allocated here, and only if `out` is omitted."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous()
    tokens, k = x.shape
    if gamma is not None:
        assert gamma.dtype == torch.bfloat16 and gamma.is_cuda and gamma.numel() == k
    out = out or alloc_prep(tokens, k, nm_n, nm_m, unit, fmt, x.device)
    st = out.struct()
    _check(lib.sharq_prepare_tensor_scale_noalloc(_ptr(x), tokens, k, _ptr(gamma), ctypes.c_float(eps), nm_n, nm_m,
                                                  unit, _fmt(fmt), ctypes.byref(st), _stream(stream)))
    return out


def sharq_prepare_swiglu(gate_up: torch.Tensor, nm_n: int = 2, nm_m: int = 4, unit: int = UNIT_PAIR,
                         fmt="nvfp4", out: Prep | None = None, stream=None) -> Prep:
    """The preparation operator on a down projection's gated input x = SiLU(g) * u, formed in
    registers from the gate/up output [tokens, 2k] = [g | u] (bf16, device)."""
    assert gate_up.dtype == torch.bfloat16 and gate_up.is_cuda and gate_up.is_contiguous()
    tokens, k2 = gate_up.shape
    assert k2 % 2 == 0
    k = k2 // 2
    out = out or alloc_prep(tokens, k, nm_n, nm_m, unit, fmt, gate_up.device)
    st = out.struct()
    _check(lib.sharq_prepare_swiglu(_ptr(gate_up), tokens, k, nm_n, nm_m, unit, _fmt(fmt), ctypes.byref(st),
                                    _stream(stream)))
    return out


def sharq_linear(prep: Prep, w: WPack, y: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                 stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Y [tokens, n_out] = sparse FP4 GEMM (backbone) + dense FP4 GEMM (residual), one output.
    With `workspace` (device bytes, sharq_linear_workspace_size) the split-K form runs where the
    shape calls for it (sharq_linear_split)."""
    if y is None:
        y = torch.empty(prep.tokens, w.n_out, dtype=out_dtype, device=prep.tiles.device)
    code = SHARQ_OUT_F32 if y.dtype == torch.float32 else SHARQ_OUT_BF16
    if workspace is not None:
        _check(lib.sharq_linear_split(ctypes.byref(prep.struct()), ctypes.byref(w.struct()), _ptr(y), code,
                                      _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    else:
        _check(lib.sharq_linear(ctypes.byref(prep.struct()), ctypes.byref(w.struct()), _ptr(y), code,
                                _stream(stream)))
    return y


def sharq_linear_workspace_size(tokens: int, n_out: int, k: int) -> int:
    """Bytes of workspace the split-K form of sharq_linear wants for this shape (0: none)."""
    return int(lib.sharq_linear_workspace_size(tokens, n_out, k))


def sharq_linear_grouped(preps: list[Prep], ws: list[WPack], ys: list[torch.Tensor] | None = None,
                         out_dtype=torch.bfloat16, stream=None) -> list[torch.Tensor]:
    """Mixture-of-experts form: Y_e = sharq_linear(preps[e], ws[e]) for every expert in one
    launch (per 64 experts). Every weight shares n_out and k."""
    n = len(preps)
    assert n == len(ws) and n >= 1
    if ys is None:
        ys = [torch.empty(p.tokens, w.n_out, dtype=out_dtype, device=p.tiles.device) for p, w in zip(preps, ws)]
    code = SHARQ_OUT_F32 if ys[0].dtype == torch.float32 else SHARQ_OUT_BF16
    a = (_Prep * n)(*[p.struct() for p in preps])
    w = (_WPack * n)(*[x.struct() for x in ws])
    y = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ys])
    _check(lib.sharq_linear_grouped(a, w, y, n, code, _stream(stream)))
    return ys


@dataclass
class DenseQ:
    """A dense-quantized activation: the tiled operand and the row scales."""
    tiles: torch.Tensor
    row_scale: torch.Tensor
    tokens: int
    k: int
    fmt: int


def sharq_quantize_dense(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-6, fmt="nvfp4",
                         out: DenseQ | None = None, stream=None) -> DenseQ:
    """The dense FP4 baseline quantizer (optional RMSNorm + block quantization of every element)."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous()
    tokens, k = x.shape
    if out is None:
        s = sharq_dense_buffer_sizes(tokens, k, fmt)
        out = DenseQ(_bytes(s[0], x.device), torch.empty(tokens, dtype=torch.float32, device=x.device), tokens, k,
                     _fmt(fmt))
    _check(lib.sharq_quantize_dense(_ptr(x), tokens, k, _ptr(gamma), ctypes.c_float(eps), _fmt(fmt),
                                    _ptr(out.tiles), _ptr(out.row_scale), _stream(stream)))
    return out


def sharq_linear_dense(q: DenseQ, w: WPack, y: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                       stream=None) -> torch.Tensor:
    """The dense FP4 baseline GEMM against the weight's dense-path scale view."""
    if y is None:
        y = torch.empty(q.tokens, w.n_out, dtype=out_dtype, device=q.tiles.device)
    code = SHARQ_OUT_F32 if y.dtype == torch.float32 else SHARQ_OUT_BF16
    _check(lib.sharq_linear_dense(_ptr(q.tiles), _ptr(q.row_scale), q.tokens, q.k, ctypes.byref(w.struct()),
                                  _ptr(y), code, _stream(stream)))
    return y


def sharq_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """The dense baseline's separate RMSNorm pass: y = bf16(fp32(fp32(x*rstd)*gamma))."""
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous() and gamma.dtype == torch.bfloat16
    tokens, k = x.shape
    out = torch.empty_like(x) if out is None else out
    _check(lib.sharq_rmsnorm(_ptr(x), tokens, k, _ptr(gamma), float(eps), _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------------------ the attention side of a block
def _reject(message: str):
    raise SharqError(SHARQ_ERR_INVALID_ARG, message)


def _tensor(t, name: str, dtype, device: int | None, shape=None, contiguous: bool = True):
    """Checks one device tensor argument (`device`: index, `shape`: entries of None are free)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape
            and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _reject(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        _reject(f"{name} must be {dtype} (got {t.dtype})")
    if device is not None and t.get_device() != device:
        _reject(f"{name} is on {t.device}, the call on cuda:{device}")
    if shape is not None and (t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape))):
        _reject(f"{name} must have shape {tuple('any' if n is None else n for n in shape)} (got {tuple(t.shape)})")
    if contiguous and not t.is_contiguous():
        _reject(f"{name} must be contiguous")


def _rows(t: torch.Tensor, name: str) -> int:
    """Distance in elements between the first-axis rows of `t`, which must itself be dense."""
    n = t.shape[1] if t.dim() == 2 else t.shape[1] * t.shape[2]
    if t.is_contiguous():
        return n
    dense = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != dense:
            _reject(f"{name} may be strided along its first axis only")
        dense *= size
    return t.stride(0) if t.shape[0] > 1 else n


def _address(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device: torch.device) -> int:
    """The raw handle of a stream: an object with `cuda_stream` (of the call's device, where it says) or an integer."""
    try:
        own = getattr(stream, "device", None)
        own = device if own is None else torch.device(own)
        handle = int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)
    except (TypeError, ValueError, RuntimeError):
        _reject(f"stream must be a stream or its handle (got {type(stream).__name__})")
    if own.type != device.type or own.index not in (None, device.index):
        _reject(f"the stream is of {own}, the call on {device}")
    return handle


def _on_stream(stream, device: torch.device):
    """`stream` as the current one: what a call allocates and clears, and what it launches, is then
    ordered on it. Handles 0 and 1 are the device's default stream."""
    handle = _stream_handle(stream, device)
    if device.type != "cuda":
        _reject(f"the call is on {device}, not on a CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=device)
    return torch.cuda.stream(stream)


def _launch(device: int, fn, *args):
    """The call on the tensors' device and its current stream."""
    handle = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, handle))


def sharq_kv_page_bytes(page_size: int, kv_heads: int, head_dim: int, fmt="nvfp4") -> int:
    """Bytes of one page of the cache (all key heads)."""
    n = lib.sharq_kv_page_bytes(page_size, kv_heads, head_dim, _fmt(fmt))
    if n == 0:
        raise SharqError(SHARQ_ERR_INVALID_ARG, last_error())
    return n


@dataclass(frozen=True, eq=False)
class KVCache:
    """A paged cache of FP4 keys and values: num_pages pages of page_size tokens in `pages`
    (device bytes, num_pages * sharq_kv_page_bytes). k_scale, v_scale: float32 NVFP4 second-level
    scales, one per key head (None: 1); MXFP4 has none."""
    pages: torch.Tensor
    num_pages: int
    page_size: int
    kv_heads: int
    head_dim: int
    fmt: int | str = "nvfp4"
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    c: _KVCache = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        need = self.num_pages * sharq_kv_page_bytes(self.page_size, self.kv_heads, self.head_dim, self.fmt)
        _tensor(self.pages, "pages", torch.uint8, None)
        if self.num_pages < 1 or self.pages.numel() < need:
            _reject(f"{self.num_pages} pages need {need} bytes (got {self.pages.numel()})")
        for name in ("k_scale", "v_scale"):
            t = getattr(self, name)
            if t is not None:
                _tensor(t, name, torch.float32, self.pages.get_device())
                if t.numel() != self.kv_heads:
                    _reject(f"{name} must have one value per key head ({self.kv_heads}, got {t.numel()})")
        if _fmt(self.fmt) == SHARQ_MXFP4 and (self.k_scale is not None or self.v_scale is not None):
            _reject("MXFP4 has no second-level scales")
        object.__setattr__(self, "c", _KVCache(
            self.pages.data_ptr(), 0 if self.k_scale is None else self.k_scale.data_ptr(),
            0 if self.v_scale is None else self.v_scale.data_ptr(), self.num_pages, self.page_size, self.kv_heads,
            self.head_dim, _fmt(self.fmt)))


@dataclass(frozen=True, eq=False)
class KVBatch:
    """One call's ragged batch (int32 device tensors): token rows [cu_q[b], cu_q[b+1]) are the
    newest of sequence b, which has kv_len[b] tokens in the cache with them; position x lives in
    page page_table[b, x // page_size]. max_q bounds the rows of one sequence; tokens is the row
    count of the call's tensors (rows at or behind cu_q[-1] belong to no sequence: they are left
    as they were). The tensors' contents are read when the kernels run and may change between
    calls."""
    cu_q: torch.Tensor
    kv_len: torch.Tensor
    page_table: torch.Tensor
    max_q: int
    tokens: int
    c: _KVBatch = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        _tensor(self.kv_len, "kv_len", torch.int32, None, (None,))
        n = self.kv_len.numel()
        _tensor(self.cu_q, "cu_q", torch.int32, self.kv_len.get_device(), (n + 1,))
        _tensor(self.page_table, "page_table", torch.int32, self.kv_len.get_device(), (n, None))
        object.__setattr__(self, "c", _KVBatch(self.cu_q.data_ptr(), self.kv_len.data_ptr(), self.page_table.data_ptr(),
                                               n, self.page_table.shape[1], self.max_q, self.tokens))


def alloc_kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt="nvfp4",
                   k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                   device="cuda") -> KVCache:
    """A cache whose every value is zero."""
    n = num_pages * sharq_kv_page_bytes(page_size, kv_heads, head_dim, fmt)
    return KVCache(torch.zeros(n, dtype=torch.uint8, device=device), num_pages, page_size, kv_heads, head_dim, fmt,
                   k_scale, v_scale)


def _same_device(cache: KVCache, batch: KVBatch) -> int:
    device = cache.pages.get_device()
    if batch.kv_len.get_device() != device:
        _reject(f"the batch is on {batch.kv_len.device}, the cache on {cache.pages.device}")
    return device


def sharq_kv_append(qkv: torch.Tensor, cache: KVCache, batch: KVBatch, q_heads: int,
                    inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                    q_gamma: torch.Tensor | None = None, k_gamma: torch.Tensor | None = None, eps: float = 1e-6,
                    q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Append a call's keys and values. qkv bf16 [tokens, (q_heads + 2 kv_heads) * head_dim] (a
    QKV projection's output; rows may be strided): q and k are normalized per head where gammas
    are given, rotated by position * inv_freq (float32 [rot_dim/2]; None: no rotation), k and v
    quantized into the cache. Returns the queries, bf16 [tokens, q_heads, head_dim]."""
    if stream is not None:
        with _on_stream(stream, cache.pages.device):
            return sharq_kv_append(qkv, cache, batch, q_heads, inv_freq, interleaved, q_gamma, k_gamma, eps, q_out)
    dev = _same_device(cache, batch)
    d, h = cache.head_dim, cache.kv_heads
    _tensor(qkv, "qkv", torch.bfloat16, dev, (batch.tokens, (q_heads + 2 * h) * d), contiguous=False)
    stride = _rows(qkv, "qkv")
    for name, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
        if g is not None:
            _tensor(g, name, torch.bfloat16, dev, (d,))
    if inv_freq is not None:
        _tensor(inv_freq, "inv_freq", torch.float32, dev, (None,))
    if q_out is None:
        q_out = torch.empty(batch.tokens, q_heads, d, dtype=torch.bfloat16, device=cache.pages.device)
    else:
        _tensor(q_out, "q_out", torch.bfloat16, dev, (batch.tokens, q_heads, d))
    _launch(dev, lib.sharq_kv_append, qkv.data_ptr(), stride, q_heads, ctypes.byref(cache.c),
            ctypes.byref(batch.c), _address(q_gamma), _address(k_gamma), eps, _address(inv_freq),
            0 if inv_freq is None else 2 * inv_freq.numel(), int(interleaved), q_out.data_ptr())
    return q_out


def sharq_kv_read(cache: KVCache, batch: KVBatch, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The batch's token rows of the cache as values: (k, v), [tokens, kv_heads, head_dim], bf16
    or float32."""
    if stream is not None:
        with _on_stream(stream, cache.pages.device):
            return sharq_kv_read(cache, batch, k_out, v_out, out_dtype)
    dev = _same_device(cache, batch)
    shape = (batch.tokens, cache.kv_heads, cache.head_dim)
    if k_out is not None:
        out_dtype = k_out.dtype
    elif v_out is not None:
        out_dtype = v_out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        _reject(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    k_out = torch.empty(shape, dtype=out_dtype, device=cache.pages.device) if k_out is None else k_out
    v_out = torch.empty(shape, dtype=out_dtype, device=cache.pages.device) if v_out is None else v_out
    _tensor(k_out, "k_out", out_dtype, dev, shape)
    _tensor(v_out, "v_out", out_dtype, dev, shape)
    _launch(dev, lib.sharq_kv_read, ctypes.byref(cache.c), ctypes.byref(batch.c), k_out.data_ptr(),
            v_out.data_ptr(), SHARQ_OUT_F32 if out_dtype == torch.float32 else SHARQ_OUT_BF16)
    return k_out, v_out


def sharq_attention_workspace_size(cache: KVCache, batch: KVBatch, q_heads: int) -> int:
    n = lib.sharq_attention_workspace_size(ctypes.byref(cache.c), ctypes.byref(batch.c), q_heads)
    if n == 0:
        raise SharqError(SHARQ_ERR_INVALID_ARG, last_error())
    return n


def alloc_attention_workspace(cache: KVCache, batch: KVBatch, q_heads: int) -> torch.Tensor:
    """A workspace for sharq_attention calls of this shape (zeroed once here; each call leaves it
    ready for the next). Calls that may overlap on the GPU need one each."""
    n = sharq_attention_workspace_size(cache, batch, q_heads)
    return torch.zeros(n, dtype=torch.uint8, device=cache.pages.device)


def sharq_attention(q: torch.Tensor, cache: KVCache, batch: KVBatch, causal: bool = True, window: int = 0,
                    scale: float | None = None, return_lse: bool = False, y: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q bf16 [tokens, q_heads, head_dim] (rows may be strided) over the cache:
    y bf16 of q's shape, or (y, lse) with return_lse or an `lse` given (float32
    [tokens, q_heads], the natural log of the sum of exponentials). `window` > 0 (causal only):
    the last `window` positions. scale defaults to head_dim ** -0.5. `workspace` as from
    alloc_attention_workspace (allocated here if omitted)."""
    if stream is not None:
        with _on_stream(stream, cache.pages.device):
            return sharq_attention(q, cache, batch, causal, window, scale, return_lse, y, lse, workspace)
    dev = _same_device(cache, batch)
    d = cache.head_dim
    hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    _tensor(q, "q", torch.bfloat16, dev, (batch.tokens, hq, d), contiguous=False)
    stride = _rows(q, "q")
    if y is None:
        y = torch.empty(batch.tokens, hq, d, dtype=torch.bfloat16, device=cache.pages.device)
    else:
        _tensor(y, "y", torch.bfloat16, dev, (batch.tokens, hq, d))
    if lse is not None:
        _tensor(lse, "lse", torch.float32, dev, (batch.tokens, hq))
    elif return_lse:
        lse = torch.empty(batch.tokens, hq, dtype=torch.float32, device=cache.pages.device)
    if workspace is None:
        workspace = alloc_attention_workspace(cache, batch, hq)
    else:
        _tensor(workspace, "workspace", torch.uint8, dev)
    _launch(dev, lib.sharq_attention, q.data_ptr(), stride, hq, ctypes.byref(cache.c), ctypes.byref(batch.c),
            int(causal), window, d ** -0.5 if scale is None else scale, y.data_ptr(), _address(lse),
            workspace.data_ptr(), workspace.numel())
    return y if lse is None else (y, lse)


def sharq_norm_residual(y: torch.Tensor, residual: torch.Tensor, post_gamma: torch.Tensor | None = None,
                        gate: torch.Tensor | None = None, rows_per_gate: int = 0, alpha: float = 1.0,
                        pre_gamma: torch.Tensor | None = None, eps: float = 1e-6,
                        residual_out: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                        stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """r' = bf16(alpha * residual + gate * norm(y)) and h = bf16(norm(r')): the norms after and
    before a block (each only where its gamma [k] is given) with the block's gate ([k] or
    [gate_rows, k]; token t uses row t // rows_per_gate, or row 0 when rows_per_gate is 0) and the
    scaled residual stream. y, residual bf16 [tokens, k]. Returns (r', h); h is None without
    pre_gamma. residual_out may be residual, h_out may be y."""
    if stream is not None and isinstance(y, torch.Tensor):
        with _on_stream(stream, y.device):
            return sharq_norm_residual(y, residual, post_gamma, gate, rows_per_gate, alpha, pre_gamma, eps, residual_out,
                                       h_out)
    shape = y.shape if isinstance(y, torch.Tensor) and y.dim() == 2 else (None, None)
    _tensor(y, "y", torch.bfloat16, y.get_device() if isinstance(y, torch.Tensor) and y.is_cuda else None, shape)
    tokens, k = shape
    dev = y.get_device()
    _tensor(residual, "residual", torch.bfloat16, dev, (tokens, k))
    for name, g in (("post_gamma", post_gamma), ("pre_gamma", pre_gamma)):
        if g is not None:
            _tensor(g, name, torch.bfloat16, dev, (k,))
    gate_rows = 0
    if gate is not None:
        _tensor(gate, "gate", torch.bfloat16, dev, (k,) if gate.dim() == 1 else (None, k))
        gate_rows = 1 if gate.dim() == 1 else gate.shape[0]
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    else:
        _tensor(residual_out, "residual_out", torch.bfloat16, dev, (tokens, k))
    if pre_gamma is None:
        if h_out is not None:
            _reject("h_out needs pre_gamma")
    elif h_out is None:
        h_out = torch.empty_like(residual)
    else:
        _tensor(h_out, "h_out", torch.bfloat16, dev, (tokens, k))
    _launch(dev, lib.sharq_norm_residual, y.data_ptr(), residual.data_ptr(), tokens, k, _address(post_gamma),
            _address(gate), gate_rows, rows_per_gate, alpha, _address(pre_gamma), eps, residual_out.data_ptr(),
            _address(h_out))
    return residual_out, h_out


# flops one K step of one CTA pair performs in sharq_mma_peak, per mode: dense; sparse (logical,
# counting the dropped half as NVIDIA's sparse peaks do); both, in sharq_linear's dense-equivalent
# units (3 * 256^3: the dense path over all of K plus the sparse path over its kept half)
MMA_PEAK_STEP_FLOPS = {0: 2.0 * 256 ** 3, 1: 2.0 * 256 ** 3, 2: 3.0 * 256 ** 3}


def sharq_mma_peak(mode: int, fmt="nvfp4", iters: int = 65536, clusters: int = 0, stream=None) -> None:
    """Launch the tensor-core peak loop (mode 0 dense, 1 sparse, 2 both); the caller times it."""
    _check(lib.sharq_mma_peak(int(mode), _fmt(fmt), int(iters), int(clusters), _stream(stream)))


def sharq_device_status(stream=None) -> int:
    """Synchronize the stream; return (and clear) the status of the bounded device waits."""
    return lib.sharq_device_status(_stream(stream))


def sharq_set_wait_limit(nanoseconds: int) -> None:
    """Test hook: time limit of the library's bounded device waits (0 restores the default of 4 s)."""
    lib.sharq_set_wait_limit(int(nanoseconds))
