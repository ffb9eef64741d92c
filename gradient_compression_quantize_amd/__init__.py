"""gradient_compression_quantize_amd -- gradient quantization kernels for MI355X.

Python binding of ``libgcq.so`` (HIP kernels for gfx950 behind the C ABI of
``include/gcq.h``). Each function has the name of the C entry point it calls
and only marshals arguments: torch tensors supply device memory and the
stream, and every step of the computation runs in the library's kernels.
There is no fallback: if ``libgcq.so`` is missing, ``load()`` raises.
Tensors must be contiguous, of the documented dtype, and on torch's current
device, which is where the library launches (an explicit ``stream`` must
belong to that device too); anything else is refused before the call.

Two method families (see include/gcq.h for exact semantics):
  * 2-bit threshold quantization with residual error feedback (apache MXNet
    pull request #8342): compress_2bit, decompress_2bit, decompress_2bit_sum,
    Plan2bitMulti / compress_2bit_multi, and the same codes packed five per
    byte: compress_ternary, decompress_ternary, decompress_ternary_sum;
  * QSGDMaxNorm stochastic quantization and GlobalRandK (vineeths96
    "Gradient-Compression"): qsgd_global_maxnorm (and qsgd_global_maxnorm_noalloc,
    which needs no workspace), qsgd_maxnorm_quantize,
    qsgd_dequant_sum, qsgd_quantize_sum (the W quantizes and the level sum fused),
    grandk_indices, gather_f32, and grandk_mn_step (the whole GRandK-MN step).

Training operators, whose gradients the two families compress (activations in
float32, bfloat16 or float16; gradients of parameters in float32):
  * dropout and dropout_backward, on the same counter-based generator, the
    mask drawn again where it is needed instead of stored;
  * norm_residual and norm_residual_grad: the norms around a block fused with
    its dropout, gate and residual scale;
  * layer_norm and layer_norm_grad: layer norm behind a block's dropout and
    residual sum;
  * linear_xent_loss and linear_xent_grad: softmax cross entropy of a linear
    layer over a large vocabulary, the logits never kept;
  * orthogonalize and muon_step: an update made nearly orthogonal by
    Newton-Schulz products, and the optimiser step from the reduced gradients
    to the new weights.
"""
from __future__ import annotations

import ctypes
import pathlib
from typing import Sequence

LIB_PATH = pathlib.Path(__file__).resolve().parent / "libgcq.so"

GC_OK = 0
GC_EINVAL = -1
GC_EHIP = -2
GC_EUNSUPPORTED = -3
GC_MAX_WORKERS = 64

GC_F32 = 0
GC_BF16 = 1
GC_F16 = 2


class GcqError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


_lib = None

_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f = ctypes.c_float
_i = ctypes.c_int


def load() -> ctypes.CDLL:
    """Load libgcq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "python gradient_compression_quantize_amd/build.py")
        _lib = _declare(ctypes.CDLL(str(LIB_PATH)))
    return _lib


def _declare(L):
    L.gc_last_error.argtypes = []
    L.gc_last_error.restype = ctypes.c_char_p
    L.gc_compressed_2bit_words.argtypes = [_sz]
    L.gc_compressed_2bit_words.restype = _sz
    L.compress_2bit.argtypes = [_vp, _vp, _sz, _f, _f, _vp, _vp]
    L.decompress_2bit.argtypes = [_vp, _sz, _vp, _i, _vp]
    L.decompress_2bit_sum.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _vp]
    L.gc_compressed_ternary_words.argtypes = [_sz]
    L.gc_compressed_ternary_words.restype = _sz
    L.compress_ternary.argtypes = [_vp, _vp, _sz, _f, _f, _vp, _vp]
    L.decompress_ternary.argtypes = [_vp, _sz, _vp, _i, _vp]
    L.decompress_ternary_sum.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _vp]
    L.gc_plan_2bit_multi_create.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                            ctypes.POINTER(_sz), _i, ctypes.POINTER(_vp)]
    L.gc_plan_compressed_words.argtypes = [_vp]
    L.gc_plan_compressed_words.restype = _sz
    L.gc_plan_block_offsets.argtypes = [_vp, ctypes.POINTER(_sz)]
    L.compress_2bit_multi.argtypes = [_vp, _f, _f, _vp, _vp]
    L.gc_plan_destroy.argtypes = [_vp]
    L.gc_plan_destroy.restype = None
    L.qsgd_global_maxnorm.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _vp,
                                      ctypes.POINTER(_sz), _vp]
    L.qsgd_global_maxnorm_noalloc.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _vp]
    L.qsgd_maxnorm_quantize.argtypes = [_vp, _sz, _vp, _i, ctypes.c_uint64, ctypes.c_uint32,
                                        _vp, _vp]
    L.qsgd_dequant_sum.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _i, _vp, _vp, _vp, _sz,
                                   _vp]
    L.qsgd_quantize_sum.argtypes = [ctypes.POINTER(_vp), _i, _sz, _vp, _i, ctypes.c_uint64,
                                    _vp, _vp, _vp]
    L.grandk_indices.argtypes = [_sz, ctypes.c_uint32, ctypes.c_uint64, _vp, _vp,
                                 ctypes.POINTER(_sz), _vp]
    L.gather_f32.argtypes = [_vp, _vp, _sz, _vp, _vp]
    L.grandk_mn_step.argtypes = [ctypes.POINTER(_vp), _i, _sz, ctypes.c_uint32, ctypes.c_uint64,
                                 _i, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_sz), _vp]
    u64, u32, dbl = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_double
    L.dropout.argtypes = [_vp, _vp, _sz, _i, dbl, u64, u32, u64, _vp, _vp, _vp]
    L.dropout_backward.argtypes = [_vp, _sz, _i, dbl, u64, u32, u64, _vp, _vp, _vp]
    L.norm_residual.argtypes = [_vp, _vp, _i, _sz, _sz, _vp, _vp, _sz, _vp, _f, _f, dbl, u64, u32,
                                _vp, _vp, _vp, _vp, _vp, _vp]
    L.norm_residual_grad.argtypes = [_vp, _vp, _i, _sz, _sz, _vp, _vp, _sz, _vp, _f, dbl, u64, u32,
                                     _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(_sz), _vp]
    L.layer_norm.argtypes = [_vp, _vp, _i, _sz, _sz, _vp, _vp, _f, dbl, u64, u32, _vp, _vp, _vp,
                             _vp, _vp, _vp]
    L.layer_norm_grad.argtypes = [_vp, _vp, _vp, _i, _sz, _sz, _vp, dbl, u64, u32, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_sz), _vp]
    i64 = ctypes.c_int64
    L.linear_xent_loss.argtypes = [_vp, _vp, _i, _sz, _sz, _sz, _vp, i64, _vp, _vp, _vp,
                                   ctypes.POINTER(_sz), _vp]
    L.linear_xent_grad.argtypes = [_vp, _vp, _i, _sz, _sz, _sz, _vp, i64, _vp, _vp, _vp, _i, _vp,
                                   _i, _vp, ctypes.POINTER(_sz), _vp]
    pp = ctypes.POINTER(_vp)
    L.orthogonalize.argtypes = [pp, _i, _sz, _sz, _i, _vp, _i, _f, _f, pp, _i, _vp,
                                ctypes.POINTER(_sz), _vp]
    L.muon_step.argtypes = [pp, _i, _sz, _sz, pp, pp, _i, _i, _vp, _i, _f, _f, dbl, _i, _f, _vp, _f,
                            _f, pp, pp, _vp, ctypes.POINTER(_sz), _vp]
    for name in ("compress_2bit", "decompress_2bit", "decompress_2bit_sum",
                 "compress_ternary", "decompress_ternary", "decompress_ternary_sum",
                 "gc_plan_2bit_multi_create", "gc_plan_block_offsets", "compress_2bit_multi",
                 "qsgd_global_maxnorm", "qsgd_global_maxnorm_noalloc",
                 "qsgd_maxnorm_quantize", "qsgd_dequant_sum",
                 "qsgd_quantize_sum",
                 "grandk_indices", "gather_f32", "grandk_mn_step",
                 "dropout", "dropout_backward", "norm_residual", "norm_residual_grad",
                 "layer_norm", "layer_norm_grad", "orthogonalize", "muon_step",
                 "linear_xent_loss", "linear_xent_grad"):
        getattr(L, name).restype = _i
    return L


def last_error() -> str:
    return load().gc_last_error().decode()


def _check(rc: int) -> None:
    if rc != GC_OK:
        raise GcqError(rc, last_error())


# ---- marshalling helpers -------------------------------------------------

def _torch():
    import torch
    return torch


_gpu_present = None
_get_device = None
_raw_stream = None


def _current_device():
    """Index of torch's current device, or None when torch sees no GPU (then
    there is nothing to compare against: every call fails validation or its
    device-tensor checks first). Once torch's device state is set up, this
    reads the device straight from torch's C layer (every call of the
    binding asks once per tensor, so it is worth a few microseconds a call)."""
    global _gpu_present, _get_device, _raw_stream
    if _gpu_present is None:
        torch = _torch()
        present = bool(torch.cuda.is_available())
        if present:
            torch.cuda.current_device()  # sets up torch's device state
            _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _gpu_present = present
    if not _gpu_present:
        return None
    return _get_device() if _get_device is not None else _torch().cuda.current_device()


def _stream(stream) -> ctypes.c_void_p:
    torch = _torch()
    if stream is None:
        cur = _current_device()
        if cur is not None and _raw_stream is not None:
            # the same handle as torch.cuda.current_stream().cuda_stream,
            # without building a Stream object
            return _vp(_raw_stream(cur))
        s = torch.cuda.current_stream()
    else:
        s = stream
        dev = getattr(s, "device", None)
        cur = _current_device()
        if dev is not None and cur is not None and dev.index != cur:
            raise ValueError(f"stream is on cuda:{dev.index} but the current device is "
                             f"cuda:{cur}; the library launches on the current device")
    return _vp(s.cuda_stream)


def _refuse(t, dtype, what: str, cur) -> None:
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous tensor")
    raise ValueError(f"{what}: on cuda:{t.get_device()} but the current device is "
                     f"cuda:{cur}; the library launches on the current device")


def _ptr(t, dtype, what: str, cur, k=None) -> int:
    """Device address of a contiguous tensor of the given dtype on device
    `cur` (the current device, which the library launches on; None when
    torch sees no GPU). The error names `what`, or `what[k]`."""
    if (not t.is_cuda or t.dtype != dtype or not t.is_contiguous()
            or (cur is not None and t.get_device() != cur)):
        _refuse(t, dtype, what if k is None else f"{what}[{k}]", cur)
    return t.data_ptr()


def _dev(t, dtype, what: str) -> ctypes.c_void_p:
    """Device pointer of a contiguous tensor of the given dtype on the current
    device (the device the library launches on)."""
    if t is None:
        return _vp(None)
    return _vp(_ptr(t, dtype, what, _current_device()))


def _need_norm(norm, what: str) -> None:
    """The shared max-norm is one fp32 device scalar: refuse an empty tensor
    (the kernels read element 0, and qsgd_global_maxnorm writes it)."""
    if norm is not None and norm.numel() < 1:
        raise ValueError(f"{what}: norm must hold at least one element")


def _ptr_array(ts, dtype, what: str):
    arr = (_vp * len(ts))()
    cur = _current_device()
    for k, t in enumerate(ts):
        arr[k] = None if t is None else _ptr(t, dtype, what, cur, k)
    return arr


# ---- 2-bit threshold quantization -----------------------------------------

def gc_compressed_2bit_words(n: int) -> int:
    return int(load().gc_compressed_2bit_words(n))


compressed_2bit_words = gc_compressed_2bit_words


def compress_2bit(grad, residual, neg_threshold: float, pos_threshold: float, compr,
                  stream=None) -> None:
    torch = _torch()
    n = grad.numel()
    if residual.numel() != n:
        raise ValueError("compress_2bit: grad and residual differ in size")
    if compr.numel() < gc_compressed_2bit_words(n):
        raise ValueError("compress_2bit: compr too small")
    _check(load().compress_2bit(_dev(grad, torch.float32, "grad"),
                                _dev(residual, torch.float32, "residual"), n,
                                float(neg_threshold), float(pos_threshold),
                                _dev(compr, torch.int32, "compr"), _stream(stream)))


def decompress_2bit(compr, n: int, out, accumulate: bool = False, stream=None) -> None:
    torch = _torch()
    if compr.numel() < gc_compressed_2bit_words(n) or out.numel() < n:
        raise ValueError("decompress_2bit: buffer too small")
    _check(load().decompress_2bit(_dev(compr, torch.int32, "compr"), n,
                                  _dev(out, torch.float32, "out"), int(bool(accumulate)),
                                  _stream(stream)))


def decompress_2bit_sum(comprs: Sequence, n: int, out, stream=None) -> None:
    torch = _torch()
    for c in comprs:
        if c.numel() < gc_compressed_2bit_words(n):
            raise ValueError("decompress_2bit_sum: compr too small")
    if out.numel() < n:
        raise ValueError("decompress_2bit_sum: out too small")
    arr = _ptr_array(comprs, torch.int32, "compr")
    _check(load().decompress_2bit_sum(arr, len(comprs), n, _dev(out, torch.float32, "out"),
                                      _stream(stream)))


# ---- the same codes, five per byte ------------------------------------------

def gc_compressed_ternary_words(n: int) -> int:
    return int(load().gc_compressed_ternary_words(n))


compressed_ternary_words = gc_compressed_ternary_words


def compress_ternary(grad, residual, neg_threshold: float, pos_threshold: float, compr,
                     stream=None) -> None:
    torch = _torch()
    n = grad.numel()
    if residual.numel() != n:
        raise ValueError("compress_ternary: grad and residual differ in size")
    if compr.numel() < gc_compressed_ternary_words(n):
        raise ValueError("compress_ternary: compr too small")
    _check(load().compress_ternary(_dev(grad, torch.float32, "grad"),
                                   _dev(residual, torch.float32, "residual"), n,
                                   float(neg_threshold), float(pos_threshold),
                                   _dev(compr, torch.int32, "compr"), _stream(stream)))


def decompress_ternary(compr, n: int, out, accumulate: bool = False, stream=None) -> None:
    torch = _torch()
    if compr.numel() < gc_compressed_ternary_words(n) or out.numel() < n:
        raise ValueError("decompress_ternary: buffer too small")
    _check(load().decompress_ternary(_dev(compr, torch.int32, "compr"), n,
                                     _dev(out, torch.float32, "out"), int(bool(accumulate)),
                                     _stream(stream)))


def decompress_ternary_sum(comprs: Sequence, n: int, out, stream=None) -> None:
    torch = _torch()
    for c in comprs:
        if c.numel() < gc_compressed_ternary_words(n):
            raise ValueError("decompress_ternary_sum: compr too small")
    if out.numel() < n:
        raise ValueError("decompress_ternary_sum: out too small")
    arr = _ptr_array(comprs, torch.int32, "compr")
    _check(load().decompress_ternary_sum(arr, len(comprs), n, _dev(out, torch.float32, "out"),
                                         _stream(stream)))


class Plan2bitMulti:
    """gc_plan_2bit_multi_create / compress_2bit_multi / gc_plan_destroy.
    Holds references to the tensors so their memory outlives the plan."""

    def __init__(self, grads: Sequence, residuals: Sequence):
        torch = _torch()
        if len(grads) != len(residuals) or not grads:
            raise ValueError("Plan2bitMulti: need matching, non-empty tensor lists")
        T = len(grads)
        ns = (_sz * T)(*[g.numel() for g in grads])
        for g, r in zip(grads, residuals):
            if g.numel() != r.numel():
                raise ValueError("Plan2bitMulti: grad and residual differ in size")
        self._keep = (list(grads), list(residuals))
        self.sizes = [g.numel() for g in grads]
        handle = _vp()
        _check(load().gc_plan_2bit_multi_create(_ptr_array(grads, torch.float32, "grads"),
                                                _ptr_array(residuals, torch.float32, "residuals"),
                                                ns, T, ctypes.byref(handle)))
        self._handle = handle

    @property
    def compressed_words(self) -> int:
        return int(load().gc_plan_compressed_words(self._handle))

    def block_offsets(self) -> list[int]:
        T = len(self.sizes)
        out = (_sz * T)()
        _check(load().gc_plan_block_offsets(self._handle, out))
        return list(out)

    def compress(self, neg_threshold: float, pos_threshold: float, compr_base,
                 stream=None) -> None:
        torch = _torch()
        if compr_base.numel() < self.compressed_words:
            raise ValueError("compress_2bit_multi: compr_base too small")
        _check(load().compress_2bit_multi(self._handle, float(neg_threshold),
                                          float(pos_threshold),
                                          _dev(compr_base, torch.int32, "compr_base"),
                                          _stream(stream)))

    def destroy(self) -> None:
        if getattr(self, "_handle", None) is not None and self._handle.value:
            load().gc_plan_destroy(self._handle)
        self._handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def compress_2bit_multi(plan: Plan2bitMulti, neg_threshold: float, pos_threshold: float,
                        compr_base, stream=None) -> None:
    plan.compress(neg_threshold, pos_threshold, compr_base, stream)


# ---- QSGDMaxNorm ----------------------------------------------------------

def qsgd_maxnorm_ws_bytes(W: int, n: int) -> int:
    size = _sz(0)
    _check(load().qsgd_global_maxnorm(None, W, n, None, None, ctypes.byref(size), None))
    return int(size.value)


def qsgd_global_maxnorm(grads: Sequence, norm, ws, stream=None) -> None:
    """norm: 1-element float32 device tensor; ws: uint8 device tensor of at
    least qsgd_maxnorm_ws_bytes(W, n) bytes."""
    torch = _torch()
    n = grads[0].numel()
    for g in grads:
        if g.numel() != n:
            raise ValueError("qsgd_global_maxnorm: gradients differ in size")
    _need_norm(norm, "qsgd_global_maxnorm")
    size = _sz(ws.numel())
    _check(load().qsgd_global_maxnorm(_ptr_array(grads, torch.float32, "grads"), len(grads), n,
                                      _dev(norm, torch.float32, "norm"),
                                      _dev(ws, torch.uint8, "ws"), ctypes.byref(size),
                                      _stream(stream)))


def qsgd_global_maxnorm_noalloc(grads: Sequence, norm, stream=None) -> None:
    """qsgd_global_maxnorm without a workspace: the partial maxima go to the
    library's fixed device array. Calls that overlap on one device race."""
    torch = _torch()
    n = grads[0].numel()
    for g in grads:
        if g.numel() != n:
            raise ValueError("qsgd_global_maxnorm_noalloc: gradients differ in size")
    _need_norm(norm, "qsgd_global_maxnorm_noalloc")
    _check(load().qsgd_global_maxnorm_noalloc(_ptr_array(grads, torch.float32, "grads"),
                                              len(grads), n, _dev(norm, torch.float32, "norm"),
                                              _stream(stream)))


def qsgd_maxnorm_quantize(grad, norm, s: int, seed: int, worker: int, levels,
                          stream=None) -> None:
    torch = _torch()
    n = grad.numel()
    if levels.numel() < n:
        raise ValueError("qsgd_maxnorm_quantize: levels too small")
    _need_norm(norm, "qsgd_maxnorm_quantize")
    _check(load().qsgd_maxnorm_quantize(_dev(grad, torch.float32, "grad"), n,
                                        _dev(norm, torch.float32, "norm"), int(s), int(seed),
                                        int(worker), _dev(levels, torch.int8, "levels"),
                                        _stream(stream)))


def qsgd_dequant_sum(levels: Sequence, norm, s: int, out, sums=None, scatter_idx=None,
                     dense_n: int = 0, stream=None) -> None:
    torch = _torch()
    n = levels[0].numel()
    for q in levels:
        if q.numel() != n:
            raise ValueError("qsgd_dequant_sum: level arrays differ in size")
    if scatter_idx is None:
        if out.numel() < n or (sums is not None and sums.numel() < n):
            raise ValueError("qsgd_dequant_sum: output too small")
    else:
        if scatter_idx.numel() != n or out.numel() < dense_n:
            raise ValueError("qsgd_dequant_sum: scatter_idx / out size mismatch")
        if sums is not None and sums.numel() < n:
            raise ValueError("qsgd_dequant_sum: sums too small")
    _need_norm(norm, "qsgd_dequant_sum")
    _check(load().qsgd_dequant_sum(_ptr_array(levels, torch.int8, "levels"), len(levels), n,
                                   _dev(norm, torch.float32, "norm"), int(s),
                                   _dev(sums, torch.int32, "sums"),
                                   _dev(out, torch.float32, "out"),
                                   _dev(scatter_idx, torch.int32, "scatter_idx"),
                                   int(dense_n), _stream(stream)))


# ---- GlobalRandK ------------------------------------------------------------

def qsgd_quantize_sum(grads: Sequence, norm, s: int, seed: int, out, sums=None,
                      stream=None) -> None:
    torch = _torch()
    n = grads[0].numel()
    if any(g.numel() != n for g in grads):
        raise ValueError("qsgd_quantize_sum: gradients differ in size")
    if out.numel() < n or (sums is not None and sums.numel() < n):
        raise ValueError("qsgd_quantize_sum: out or sums too small")
    _need_norm(norm, "qsgd_quantize_sum")
    arr = _ptr_array(grads, torch.float32, "grads")
    _check(load().qsgd_quantize_sum(arr, len(grads), n, _dev(norm, torch.float32, "norm"),
                                    int(s), int(seed) & (2 ** 64 - 1),
                                    _dev(sums, torch.int32, "sums"),
                                    _dev(out, torch.float32, "out"), _stream(stream)))


def grandk_ws_bytes(n: int, K: int) -> int:
    size = _sz(0)
    _check(load().grandk_indices(n, K, 0, None, None, ctypes.byref(size), None))
    return int(size.value)


def grandk_indices(n: int, K: int, seed: int, idx, ws, stream=None) -> None:
    """idx: int32 device tensor of K elements (holding uint32 values < 2^31
    for any n a torch int32 tensor can index); ws: uint8 device tensor."""
    torch = _torch()
    if idx.numel() < K:
        raise ValueError("grandk_indices: idx too small")
    size = _sz(ws.numel())
    _check(load().grandk_indices(n, K, int(seed), _dev(idx, torch.int32, "idx"),
                                 _dev(ws, torch.uint8, "ws"), ctypes.byref(size),
                                 _stream(stream)))


def gather_f32(x, idx, out, stream=None) -> None:
    torch = _torch()
    K = idx.numel()
    if out.numel() < K:
        raise ValueError("gather_f32: out too small")
    _check(load().gather_f32(_dev(x, torch.float32, "x"), _dev(idx, torch.int32, "idx"), K,
                             _dev(out, torch.float32, "out"), _stream(stream)))


def grandk_mn_step_ws_bytes(W: int, n: int, K: int) -> int:
    size = _sz(0)
    arr = (_vp * W)()
    _check(load().grandk_mn_step(arr, W, n, K, 0, 7, None, None, None, None, None,
                                 ctypes.byref(size), None))
    return size.value


def grandk_mn_step(grads: Sequence, K: int, seed: int, s: int, idx, dense, ws, sums=None,
                   norm=None, stream=None) -> None:
    torch = _torch()
    n = grads[0].numel()
    if any(g.numel() != n for g in grads):
        raise ValueError("grandk_mn_step: gradients differ in size")
    if idx.numel() < K or dense.numel() < n or (sums is not None and sums.numel() < K):
        raise ValueError("grandk_mn_step: idx, sums or dense too small")
    _need_norm(norm, "grandk_mn_step")
    arr = _ptr_array(grads, torch.float32, "grads")
    size = _sz(ws.numel() * ws.element_size())
    _check(load().grandk_mn_step(arr, len(grads), n, K, int(seed) & (2 ** 64 - 1), int(s),
                                 _dev(idx, torch.int32, "idx"), _dev(sums, torch.int32, "sums"),
                                 _dev(dense, torch.float32, "dense"),
                                 _dev(norm, torch.float32, "norm"), _dev(ws, torch.uint8, "ws"),
                                 ctypes.byref(size), _stream(stream)))


# ---- training operators -------------------------------------------------------

_dtypes = {}


def _dtype(t, what: str) -> int:
    """gc_dtype of a tensor of activations."""
    code = _dtypes.get(t.dtype)
    if code is None:
        torch = _torch()
        _dtypes.update({torch.float32: GC_F32, torch.bfloat16: GC_BF16, torch.float16: GC_F16})
        code = _dtypes.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: expected float32, bfloat16 or float16, got {t.dtype}")
    return code


def _at(t, dtype, what: str, cur):
    """Device address of a tensor (see _ptr), or None of None."""
    return None if t is None else _ptr(t, dtype, what, cur)


def _ats(cur, dtype, names: str, *ts) -> list:
    """_at of several tensors of one dtype; `names` holds theirs, in order. One
    loop for them all, since a small call is mostly marshalling."""
    out = []
    for k, t in enumerate(ts):
        if t is None:
            out.append(None)
        elif (not t.is_cuda or t.dtype != dtype or not t.is_contiguous()
              or (cur is not None and t.get_device() != cur)):
            _refuse(t, dtype, names.split()[k], cur)
        else:
            out.append(t.data_ptr())
    return out


def _ws(ws, what: str):
    """The size of a workspace; one of no bytes would read as a query."""
    if ws.numel() == 0:
        raise ValueError(f"{what}: ws too small")
    return _sz(ws.numel())


def _step(step, cur):
    """A device counter added to the seed: an int64 tensor of one element."""
    if step is None:
        return None
    if step.numel() != 1:
        raise ValueError("step must hold one element")
    return _ptr(step, _torch().int64, "step", cur)


def _u64(v: int) -> int:
    return int(v) & (2 ** 64 - 1)


def _worker(worker: int) -> int:
    if not 0 <= int(worker) < 2 ** 32:
        raise ValueError("worker must lie in 0 .. 2^32 - 1")
    return int(worker)


def _offset(offset: int) -> int:
    if not 0 <= int(offset) < 2 ** 64:
        raise ValueError("offset must lie in 0 .. 2^64 - 1")
    return int(offset)


def dropout(x, p: float, seed: int, worker: int, out, residual=None, offset: int = 0, step=None,
            stream=None) -> None:
    """out = dropout(x) (+ residual). out may be x or residual itself; step:
    one-element int64 device tensor added to the seed on the device."""
    n = x.numel()
    if out.numel() != n or (residual is not None and residual.numel() != n):
        raise ValueError("dropout: x, out and residual differ in size")
    cur = _current_device()
    _check(load().dropout(_at(x, x.dtype, "x", cur), _at(residual, x.dtype, "residual", cur), n,
                          _dtype(x, "x"), float(p), _u64(seed), _worker(worker), _offset(offset),
                          _step(step, cur), _at(out, x.dtype, "out", cur), _stream(stream)))


def dropout_backward(grad_out, p: float, seed: int, worker: int, grad_in, offset: int = 0,
                     step=None, stream=None) -> None:
    n = grad_out.numel()
    if grad_in.numel() != n:
        raise ValueError("dropout_backward: grad_out and grad_in differ in size")
    cur = _current_device()
    _check(load().dropout_backward(_at(grad_out, grad_out.dtype, "grad_out", cur), n,
                                   _dtype(grad_out, "grad_out"), float(p), _u64(seed),
                                   _worker(worker), _offset(offset), _step(step, cur),
                                   _at(grad_in, grad_out.dtype, "grad_in", cur), _stream(stream)))


def _norm_shape(y, what: str, same, gate, columns, per_row):
    """(rows, d, gates) of y [..., d], after the sizes of everything else:
    `same` like y, `columns` of d values, `per_row` of one value a row."""
    if y.dim() < 1 or y.shape[-1] == 0:
        raise ValueError(f"{what}: a row must hold at least one value")
    d = y.shape[-1]
    rows = y.numel() // d
    n = rows * d
    for t in same:
        if t is not None and t.numel() != n:
            raise ValueError(f"{what}: the activations differ in size")
    for t in columns:
        if t is not None and t.numel() != d:
            raise ValueError(f"{what}: a gain must hold one value a column")
    for t in per_row:
        if t is not None and t.numel() != rows:
            raise ValueError(f"{what}: rstd_post and rstd_pre must hold one value a row")
    if gate is None:
        return rows, d, 1
    gates = gate.numel() // d
    if gates == 0 or gate.numel() != gates * d or rows % gates:
        raise ValueError(f"{what}: gate must be [gates, d], gates dividing the rows")
    return rows, d, gates


def norm_residual(x, y, z, h=None, post_gain=None, gate=None, pre_gain=None,
                  residual_scale: float = 1.0, eps: float = 1e-6, p: float = 0.0, seed: int = 0,
                  worker: int = 0, step=None, rstd_post=None, rstd_pre=None, stream=None) -> None:
    """z = residual_scale * x + gate * dropout(norm(y) * post_gain) and
    h = norm(z) * pre_gain. x, y, z, h: [..., d] of one dtype; gains [d], gate
    [gates, d] or [d], rstd_post and rstd_pre (one value a row) float32."""
    rows, d, gates = _norm_shape(y, "norm_residual", (x, z, h), gate, (post_gain, pre_gain),
                                 (rstd_post, rstd_pre))
    cur = _current_device()
    code = _dtype(y, "y")
    xp, yp, zp, hp = _ats(cur, y.dtype, "x y z h", x, y, z, h)
    post, gp, pre, rp, rz = _ats(cur, _torch().float32, "post_gain gate pre_gain rstd_post rstd_pre",
                                 post_gain, gate, pre_gain, rstd_post, rstd_pre)
    _check(load().norm_residual(xp, yp, code, rows, d, post, gp, gates, pre, residual_scale, eps, p,
                                _u64(seed), _worker(worker), _step(step, cur), zp, hp, rp, rz,
                                _stream(stream)))


def norm_residual_grad_ws_bytes(rows: int, d: int, gates: int = 1) -> int:
    size = _sz(0)
    null = [None] * 11
    _check(load().norm_residual_grad(None, None, GC_F32, rows, d, None, None, gates, None, 1.0,
                                     0.0, 0, 0, None, *null[:10], ctypes.byref(size), None))
    return int(size.value)


def norm_residual_grad(z, y, dx, dy, ws, dz=None, dh=None, post_gain=None, gate=None,
                       pre_gain=None, residual_scale: float = 1.0, p: float = 0.0, seed: int = 0,
                       worker: int = 0, step=None, rstd_post=None, rstd_pre=None, dpost_gain=None,
                       dgate=None, dpre_gain=None, stream=None) -> None:
    """The gradient of norm_residual, from its z, y, arguments and rstd. ws:
    uint8 device tensor of at least norm_residual_grad_ws_bytes(rows, d,
    gates) bytes. The gains' and gate's gradients are float32, or None."""
    torch = _torch()
    rows, d, gates = _norm_shape(y, "norm_residual_grad", (z, dx, dy, dz, dh), gate,
                                 (post_gain, pre_gain, dpost_gain, dpre_gain),
                                 (rstd_post, rstd_pre))
    if dgate is not None and (gate is None or dgate.numel() != gate.numel()):
        raise ValueError("norm_residual_grad: dgate differs from gate in size")
    size = _ws(ws, "norm_residual_grad")
    cur = _current_device()
    code = _dtype(y, "y")
    zp, yp, dzp, dhp, dxp, dyp = _ats(cur, y.dtype, "z y dz dh dx dy", z, y, dz, dh, dx, dy)
    post, gp, pre, rp, rz, dpost, dgp, dpre = _ats(
        cur, torch.float32,
        "post_gain gate pre_gain rstd_post rstd_pre dpost_gain dgate dpre_gain", post_gain, gate,
        pre_gain, rstd_post, rstd_pre, dpost_gain, dgate, dpre_gain)
    _check(load().norm_residual_grad(
        zp, yp, code, rows, d, post, gp, gates, pre, residual_scale, p, _u64(seed),
        _worker(worker), _step(step, cur), rp, rz, dzp, dhp, dxp, dyp, dpost, dgp, dpre,
        _at(ws, torch.uint8, "ws", cur), ctypes.byref(size), _stream(stream)))


def _row_shape(x, what: str, same, columns, per_row):
    """(rows, d) of x [..., d], after the sizes of everything else: `same`
    like x, `columns` of d values, `per_row` of one value a row."""
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"{what}: a row must hold at least one value")
    d = x.shape[-1]
    n = x.numel()
    for t in same:
        if t is not None and t.numel() != n:
            raise ValueError(f"{what}: the activations differ in size")
    for t in columns:
        if t is not None and t.numel() != d:
            raise ValueError(f"{what}: gain, bias and their gradients must hold one value a column")
    for t in per_row:
        if t is not None and t.numel() != n // d:
            raise ValueError(f"{what}: mean and rstd must hold one value a row")
    return n // d, d


def layer_norm(x, h, y=None, z=None, gain=None, bias=None, eps: float = 1e-5, p: float = 0.0,
               seed: int = 0, worker: int = 0, step=None, mean=None, rstd=None, stream=None) -> None:
    """z = x + dropout(y) and h = (z - mean) * rstd * gain + bias. x, y, z, h:
    [..., d] of one dtype; gain and bias [d], mean and rstd (one value a row)
    float32. Without y, z is x and is not written."""
    rows, d = _row_shape(x, "layer_norm", (h, y, z), (gain, bias), (mean, rstd))
    cur = _current_device()
    code = _dtype(x, "x")
    xp, yp, zp, hp = _ats(cur, x.dtype, "x y z h", x, y, z, h)
    gp, bp, mp, rp = _ats(cur, _torch().float32, "gain bias mean rstd", gain, bias, mean, rstd)
    _check(load().layer_norm(xp, yp, code, rows, d, gp, bp, eps, p, _u64(seed), _worker(worker),
                             _step(step, cur), zp, hp, mp, rp, _stream(stream)))


def layer_norm_grad_ws_bytes(rows: int, d: int) -> int:
    size = _sz(0)
    _check(load().layer_norm_grad(None, None, None, GC_F32, rows, d, None, 0.0, 0, 0, None, None,
                                  None, None, None, None, None, None, ctypes.byref(size), None))
    return int(size.value)


def layer_norm_grad(z, dh, dx, ws, dz=None, dy=None, gain=None, p: float = 0.0, seed: int = 0,
                    worker: int = 0, step=None, mean=None, rstd=None, dgain=None, dbias=None,
                    stream=None) -> None:
    """The gradient of layer_norm, from its z (without y: its x), arguments,
    mean and rstd; dz is what reaches z by another way. ws: uint8 device
    tensor of at least layer_norm_grad_ws_bytes(rows, d) bytes. dgain and
    dbias are float32, or None."""
    torch = _torch()
    rows, d = _row_shape(z, "layer_norm_grad", (dh, dx, dz, dy), (gain, dgain, dbias), (mean, rstd))
    size = _ws(ws, "layer_norm_grad")
    cur = _current_device()
    code = _dtype(z, "z")
    zp, dhp, dxp, dzp, dyp = _ats(cur, z.dtype, "z dh dx dz dy", z, dh, dx, dz, dy)
    gp, mp, rp, dgp, dbp = _ats(cur, torch.float32, "gain mean rstd dgain dbias", gain, mean, rstd,
                                dgain, dbias)
    _check(load().layer_norm_grad(zp, dhp, dzp, code, rows, d, gp, p, _u64(seed), _worker(worker),
                                  _step(step, cur), mp, rp, dxp, dyp, dgp, dbp,
                                  _at(ws, torch.uint8, "ws", cur), ctypes.byref(size),
                                  _stream(stream)))


def _dtype_code(dtype) -> int:
    """gc_dtype of a torch dtype."""
    torch = _torch()
    return _dtype(torch.empty(0, dtype=dtype), "dtype")


def linear_xent_loss_ws_bytes(N: int, V: int, D: int, dtype) -> int:
    """dtype: the torch dtype of hidden and weight."""
    size = _sz(0)
    _check(load().linear_xent_loss(None, None, _dtype_code(dtype), N, V, D, None, 0, None, None,
                                   None, ctypes.byref(size), None))
    return int(size.value)


def linear_xent_grad_ws_bytes(N: int, V: int, D: int, dtype, dhidden_dtype=None,
                              dweight_dtype=None) -> int:
    """The gradients' dtypes default to that of hidden and weight."""
    size = _sz(0)
    code = _dtype_code(dtype)
    _check(load().linear_xent_grad(
        None, None, code, N, V, D, None, 0, None, None, None,
        code if dhidden_dtype is None else _dtype_code(dhidden_dtype), None,
        code if dweight_dtype is None else _dtype_code(dweight_dtype), None, ctypes.byref(size),
        None))
    return int(size.value)


def _xent_sizes(hidden, weight, what: str):
    """(N, V, D) of hidden [..., D] and weight [V, D]."""
    if weight.dim() != 2 or hidden.dim() < 1 or hidden.shape[-1] != weight.shape[1]:
        raise ValueError(f"{what}: hidden must be [..., D] and weight [V, D]")
    V, D = weight.shape
    if D == 0:
        raise ValueError(f"{what}: the hidden size must be at least 1")
    return hidden.numel() // D, V, D


def linear_xent_loss(hidden, weight, target, loss, lse, ws, ignore_index: int = -100,
                     stream=None) -> None:
    """hidden [..., D] and weight [V, D] of one dtype; target int64, loss and
    lse float32, one value a token; ws: uint8 device tensor of at least
    linear_xent_loss_ws_bytes(N, V, D, dtype) bytes."""
    torch = _torch()
    N, V, D = _xent_sizes(hidden, weight, "linear_xent_loss")
    if target.numel() != N or loss.numel() != N or lse.numel() != N:
        raise ValueError("linear_xent_loss: target, loss and lse must hold one value a token")
    size = _ws(ws, "linear_xent_loss")
    cur = _current_device()
    _check(load().linear_xent_loss(
        _at(hidden, hidden.dtype, "hidden", cur), _at(weight, hidden.dtype, "weight", cur),
        _dtype(hidden, "hidden"), N, V, D, _at(target, torch.int64, "target", cur), int(ignore_index),
        _at(loss, torch.float32, "loss", cur), _at(lse, torch.float32, "lse", cur),
        _at(ws, torch.uint8, "ws", cur), ctypes.byref(size), _stream(stream)))


def linear_xent_grad(hidden, weight, target, lse, dloss, dhidden, dweight, ws,
                     ignore_index: int = -100, stream=None) -> None:
    """The gradient of (dloss * loss).sum(); dhidden or dweight may be None.
    Each has the dtype of hidden and weight, or float32. ws: uint8 device
    tensor of at least linear_xent_grad_ws_bytes(...) bytes for these dtypes
    (a gradient left out counts as one of the inputs' dtype)."""
    torch = _torch()
    N, V, D = _xent_sizes(hidden, weight, "linear_xent_grad")
    if target.numel() != N or dloss.numel() != N or lse.numel() != N:
        raise ValueError("linear_xent_grad: target, lse and dloss must hold one value a token")
    if dhidden is not None and dhidden.numel() != N * D:
        raise ValueError("linear_xent_grad: dhidden differs from hidden in size")
    if dweight is not None and dweight.numel() != V * D:
        raise ValueError("linear_xent_grad: dweight differs from weight in size")
    code = _dtype(hidden, "hidden")
    h_code = code if dhidden is None else _dtype(dhidden, "dhidden")
    w_code = code if dweight is None else _dtype(dweight, "dweight")
    size = _ws(ws, "linear_xent_grad")
    cur = _current_device()
    _check(load().linear_xent_grad(
        _at(hidden, hidden.dtype, "hidden", cur), _at(weight, hidden.dtype, "weight", cur), code, N, V, D,
        _at(target, torch.int64, "target", cur), int(ignore_index), _at(lse, torch.float32, "lse", cur),
        _at(dloss, torch.float32, "dloss", cur),
        _at(dhidden, None if dhidden is None else dhidden.dtype, "dhidden", cur), h_code,
        _at(dweight, None if dweight is None else dweight.dtype, "dweight", cur), w_code,
        _at(ws, torch.uint8, "ws", cur), ctypes.byref(size), _stream(stream)))


# ---- orthogonalised updates ---------------------------------------------------

# (a, b, c) of each step: brings the singular values that are not far below the
# largest one near 1.
NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5


def _coefficients(coefficients):
    """fp32 array of the steps' triples, and their number."""
    flat = []
    for triple in coefficients:
        if len(triple) != 3:
            raise ValueError("coefficients must hold three numbers a step")
        flat += triple
    return (_f * max(len(flat), 1))(*flat), len(flat) // 3


def _matrices(what: str, names, *lists):
    """(count, m, n) of lists of matrices of one size."""
    first = lists[0]
    if len(first) < 1 or len(first) > GC_MAX_WORKERS:
        raise ValueError(f"{what}: the number of matrices must lie in 1 .. {GC_MAX_WORKERS}")
    if first[0].dim() != 2:
        raise ValueError(f"{what}: {names.split()[0]} must be matrices [m, n]")
    shape = tuple(first[0].shape)
    for name, ts in zip(names.split(), lists):
        if len(ts) != len(first):
            raise ValueError(f"{what}: {name} differ in number")
        for t in ts:
            if tuple(t.shape) != shape:
                raise ValueError(f"{what}: {name} differ in size")
    return len(first), shape[0], shape[1]


def orthogonalize_ws_bytes(count: int, m: int, n: int, out_dtype) -> int:
    size = _sz(0)
    _check(load().orthogonalize(None, count, m, n, GC_F32, None, 0, 0.0, 1.0, None,
                                _dtype_code(out_dtype), None, ctypes.byref(size), None))
    return int(size.value)


def orthogonalize(xs: Sequence, outs: Sequence, ws, coefficients=NEWTON_SCHULZ,
                  scale: float = 1.0, eps: float = 1e-7, stream=None) -> None:
    """outs[k] = scale * (xs[k] / (its norm + eps) after a step a X + b (X X') X
    + c (X X')^2 X for each triple of `coefficients`). xs and outs: up to 64
    matrices [m, n], the xs of one dtype and the outs of one; the dtype of the
    outs says how exactly they are computed. outs[k] may be xs[k] itself, but
    overlap no other matrix of the call. ws: uint8 device tensor of at least
    orthogonalize_ws_bytes(count, m, n, out_dtype) bytes."""
    count, m, n = _matrices("orthogonalize", "xs outs", xs, outs)
    coef, steps = _coefficients(coefficients)
    size = _ws(ws, "orthogonalize")
    code, out_code = _dtype(xs[0], "xs"), _dtype(outs[0], "outs")
    _check(load().orthogonalize(
        _ptr_array(xs, xs[0].dtype, "xs"), count, m, n, code, coef, steps, eps, scale,
        _ptr_array(outs, outs[0].dtype, "outs"), out_code,
        _at(ws, _torch().uint8, "ws", _current_device()), ctypes.byref(size), _stream(stream)))


def muon_step_ws_bytes(count: int, m: int, n: int, update_dtype) -> int:
    """update_dtype: as in muon_step (by default the weights' dtype)."""
    size = _sz(0)
    _check(load().muon_step(None, count, m, n, None, None, GC_F32, _dtype_code(update_dtype), None,
                            0, 0.0, 1.0, 0.0, 0, 0.0, None, 0.0, 1.0, None, None, None,
                            ctypes.byref(size), None))
    return int(size.value)


def muon_step(grads: Sequence, momenta: Sequence, weights: Sequence, ws,
              coefficients=NEWTON_SCHULZ, eps: float = 1e-7, momentum: float = 0.95,
              nesterov: bool = True, grad_scale: float = 1.0, lr: float = 0.02, lr_scale=None,
              weight_decay: float = 0.0, update_scale: float = 1.0, update_dtype=None,
              new_momenta=None, new_weights=None, stream=None) -> None:
    """Moves the momenta along the gradients, and the weights along the
    orthogonalised momenta. Up to 64 matrices [m, n]: grads and momenta
    float32, weights of one dtype; new_momenta and new_weights default to the
    tensors themselves, and overlap no other matrix of the call. update_dtype
    (by default the weights' dtype) says how exactly the update is computed:
    bfloat16 is a third of the products of float32. lr_scale: one-element
    float32 device tensor multiplied to lr on the device. ws: uint8 device
    tensor of at least muon_step_ws_bytes(count, m, n, update_dtype) bytes."""
    torch = _torch()
    new_momenta = momenta if new_momenta is None else new_momenta
    new_weights = weights if new_weights is None else new_weights
    count, m, n = _matrices("muon_step", "grads momenta weights new_momenta new_weights", grads,
                            momenta, weights, new_momenta, new_weights)
    coef, steps = _coefficients(coefficients)
    size = _ws(ws, "muon_step")
    cur = _current_device()
    code = _dtype(weights[0], "weights")
    if lr_scale is not None and lr_scale.numel() != 1:
        raise ValueError("muon_step: lr_scale must hold one element")
    f32 = torch.float32
    _check(load().muon_step(
        _ptr_array(grads, f32, "grads"), count, m, n, _ptr_array(momenta, f32, "momenta"),
        _ptr_array(weights, weights[0].dtype, "weights"), code,
        code if update_dtype is None else _dtype_code(update_dtype), coef, steps, eps, grad_scale,
        momentum, int(bool(nesterov)), lr, _at(lr_scale, f32, "lr_scale", cur), weight_decay,
        update_scale, _ptr_array(new_momenta, f32, "new_momenta"),
        _ptr_array(new_weights, weights[0].dtype, "new_weights"),
        _at(ws, torch.uint8, "ws", cur), ctypes.byref(size), _stream(stream)))
