"""ctypes binding of libsbn (include/sbn.h): argument marshalling only.

Every step of the BitLinear forward runs in libsbn's CUDA kernels; PyTorch
only supplies device memory and the current stream. There is no CPU
fallback: if ``libsbn.so`` is missing, loading it raises.

    packed = quantize_weights(w_bf16, n=6, m=8)       # dynamic N:M mask + ternary + pack
    xq, s = quantize_acts(x_bf16)                      # per-token absmax INT8
    y = bitlinear(xq, s, packed)                       # INT8 x ternary -> bf16
"""

from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsbn.so")

SBN_STATUS = {
    0: "SBN_OK", 1: "SBN_ERR_NULL", 2: "SBN_ERR_SHAPE", 3: "SBN_ERR_PATTERN",
    4: "SBN_ERR_ALIGN", 5: "SBN_ERR_WORKSPACE", 6: "SBN_ERR_CUDA",
    7: "SBN_ERR_TIMEOUT", 8: "SBN_ERR_DEVICE",
}

_c_i32, _c_sz, _c_p = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p

# name -> (restype, argtypes), mirroring include/sbn.h
PROTOTYPES = {
    "sbn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sbn_version": (ctypes.c_int, []),
    "sbn_codes_row_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "sbn_codes_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "sbn_meta_row_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "sbn_meta_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "sbn_quantize_weights_workspace_bytes": (_c_sz, [_c_i32, _c_i32]),
    "sbn_quantize_weights": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p,
                                            _c_p, _c_p, _c_sz, _c_p]),
    "sbn_quantize_weights_noalloc": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                                    _c_p, _c_p, _c_p]),
    "sbn_gamma_bins": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_p, _c_p]),
    "sbn_quantize_weights_from_bins": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                                      ctypes.c_int64, _c_p, _c_p, _c_p, _c_p]),
    "sbn_quantize_acts": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_p, _c_p, _c_p]),
    "sbn_bitlinear": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                     _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "sbn_bitlinear_acc32": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                           _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_x": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p,
                                       _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_x_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "sbn_mask_flips": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p]),
    "sbn_entropy_row_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "sbn_entropy_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "sbn_pack_entropy": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p]),
    "sbn_bitlinear_entropy": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                             _c_p, _c_p, _c_p, _c_p]),
    "sbn_bitlinear_entropy_acc32": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                   _c_p, _c_p, _c_p]),
    "sbn_bitlinear_entropy_x": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                               _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_entropy_x_workspace_bytes": (_c_sz, [_c_i32, _c_i32]),
    "sbn_bitlinear_grad_x": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p,
                                            _c_p, _c_p]),
    "sbn_bitlinear_grad_w": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_p]),
    "sbn_bitlinear_act": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p,
                                         _c_p, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_x_act": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_p,
                                           _c_i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_act_grad": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p]),
    "sbn_bitlinear_grouped": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                             _c_p, _c_p, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_p]),
    "sbn_bitlinear_grouped_x": (ctypes.c_int, [_c_p, _c_i32, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_p,
                                               _c_p, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz,
                                               _c_p]),
    "sbn_bitlinear_grouped_x_workspace_bytes": (_c_sz, [_c_i32, _c_i32]),
    "sbn_bitlinear_grouped_grad_x": (ctypes.c_int, [_c_p, _c_i32, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                    _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_grouped_grad_x_workspace_bytes": (_c_sz, [_c_i32, _c_i32]),
    "sbn_bitlinear_grouped_grad_w": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i32, _c_p, _c_i32, _c_i32, _c_i32, _c_p,
                                                    _c_p, _c_sz, _c_p]),
    "sbn_bitlinear_grouped_grad_w_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "sbn_bitlinear_grouped_grad_w2_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32]),
    "sbn_adamw": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_p, ctypes.c_double, _c_p,
                                 ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double, _c_p,
                                 ctypes.c_uint32, _c_p]),
    "sbn_probe_i8_mma": (ctypes.c_int, [_c_i32, ctypes.POINTER(ctypes.c_int32), _c_p]),
    "sbn_probe_i8_sparse_mma": (ctypes.c_int, [_c_i32, ctypes.POINTER(ctypes.c_int32), _c_p]),
    "sbn_selftest_wait_timeout": (ctypes.c_int, [_c_i32, ctypes.c_int64, _c_p]),
    "sbn_set_programmatic_launch": (_c_i32, [_c_i32]),
    "sbn_get_device_error": (ctypes.c_int, [_c_p]),
}

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libsbn.so (once). Raises ImportError if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m sparse_linear_layers_fwd_b200.build` (needs nvcc)")
        cdll = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in PROTOTYPES.items():
            fn = getattr(cdll, name)
            fn.restype = res
            fn.argtypes = args
        _lib = cdll
    return _lib


class SbnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().sbn_status_string(status).decode()
        super().__init__(f"{where}: {msg}")


def _check(status: int, where: str):
    if status != 0:
        raise SbnError(status, where)


def _stream_ptr(stream) -> int:
    if stream is None:
        # the handle alone: building a Stream object takes several microseconds
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _one_device(*tensors) -> torch.device:
    """The device of the tensors (None entries skipped); all must share it."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev


def _run_on(dev: torch.device, name: str, stream, *args):
    """Call entry point `name` with the stream appended, on the device of its
    tensors (made current for the call when another one is)."""
    st = _status_on(dev, name, stream, *args)
    if st != 0:
        raise SbnError(st, name)


def _status_on(dev: torch.device, name: str, stream, *args) -> int:
    fn = getattr(_lib or lib(), name)
    current = torch.cuda.current_device()
    if dev.index != current:
        with torch.cuda.device(dev):
            return fn(*args, _stream_ptr(stream))
    if stream is None:
        return fn(*args, torch._C._cuda_getCurrentRawStream(current))
    return fn(*args, _stream_ptr(stream))


def _alloc_on(dev: torch.device, stream):
    """Scope in which outputs and workspaces of a call on `stream` are allocated:
    memory belongs to the stream that uses it, so that it is not handed out
    again while the call still runs."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


@dataclass
class Pattern:
    n: int
    m: int


@dataclass
class PackedWeights:
    """Packed ternary weights in the canonical format of include/sbn.h."""
    codes: torch.Tensor            # uint8 [n_out, codes_row_bytes]
    meta: Optional[torch.Tensor]   # uint8 [n_out, meta_row_bytes] or None (n == m)
    gamma: torch.Tensor            # float32 [1]
    n_out: int
    k: int
    n: int
    m: int


def codes_row_bytes(k: int, n: int, m: int) -> int:
    return int(lib().sbn_codes_row_bytes(k, n, m))


def meta_row_bytes(k: int, n: int, m: int) -> int:
    return int(lib().sbn_meta_row_bytes(k, n, m))


def workspace_bytes(n_out: int, k: int) -> int:
    return int(lib().sbn_quantize_weights_workspace_bytes(n_out, k))


def alloc_packed(n_out: int, k: int, n: int, m: int, device) -> PackedWeights:
    cr, mr = codes_row_bytes(k, n, m), meta_row_bytes(k, n, m)
    if cr == 0:
        raise SbnError(3, "alloc_packed")
    codes = torch.empty((n_out, cr), dtype=torch.uint8, device=device)
    meta = torch.empty((n_out, mr), dtype=torch.uint8, device=device) if mr else None
    gamma = torch.empty((1,), dtype=torch.float32, device=device)
    return PackedWeights(codes, meta, gamma, n_out, k, n, m)


def quantize_weights(w: torch.Tensor, n: int, m: int, out: Optional[PackedWeights] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> PackedWeights:
    """sbn_quantize_weights: N:M magnitude mask, absmean ternary codes, packing."""
    _need(w, torch.bfloat16, "w")
    n_out, k = w.shape
    if out is None:
        out = alloc_packed(n_out, k, n, m, w.device)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(n_out, k), dtype=torch.uint8, device=w.device)
    st = lib().sbn_quantize_weights(_ptr(w), n_out, k, n, m, _ptr(out.codes), _ptr(out.meta),
                                    _ptr(out.gamma), _ptr(workspace), workspace.numel(),
                                    _stream_ptr(stream))
    _check(st, "sbn_quantize_weights")
    return out


def quantize_weights_noalloc(w: torch.Tensor, n: int, m: int, out: PackedWeights,
                             stream=None) -> PackedWeights:
    """sbn_quantize_weights_noalloc: like quantize_weights, with the library's
    fixed internal scratch instead of a caller workspace (no allocation)."""
    _need(w, torch.bfloat16, "w")
    n_out, k = w.shape
    st = lib().sbn_quantize_weights_noalloc(_ptr(w), n_out, k, n, m, _ptr(out.codes),
                                            _ptr(out.meta), _ptr(out.gamma), _stream_ptr(stream))
    _check(st, "sbn_quantize_weights_noalloc")
    return out


GAMMA_BINS = 256   # SBN_GAMMA_BINS


def gamma_bins(w: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_gamma_bins: the exact gamma bins of one shard of rows, as int64 [256]
    (the bit patterns of the library's uint64 bins; every value stays below
    2^63). Bins of several shards add up to the bins of their union, so a
    column-parallel layer sums them with an all-reduce before quantizing."""
    _need(w, torch.bfloat16, "w")
    n_out, k = w.shape
    if out is None:
        out = torch.empty((GAMMA_BINS,), dtype=torch.int64, device=w.device)
    _need(out, torch.int64, "bins")
    st = lib().sbn_gamma_bins(_ptr(w), n_out, k, _ptr(out), _stream_ptr(stream))
    _check(st, "sbn_gamma_bins")
    return out


def quantize_weights_from_bins(w: torch.Tensor, n: int, m: int, bins: torch.Tensor, total_elems: int,
                               out: Optional[PackedWeights] = None, stream=None) -> PackedWeights:
    """sbn_quantize_weights_from_bins: mask, codes and packing of one shard of
    rows with the gamma of the whole tensor (bins summed over all shards,
    total_elems the element count of the whole tensor)."""
    _need(w, torch.bfloat16, "w")
    _need(bins, torch.int64, "bins")
    n_out, k = w.shape
    if out is None:
        out = alloc_packed(n_out, k, n, m, w.device)
    st = lib().sbn_quantize_weights_from_bins(_ptr(w), n_out, k, n, m, _ptr(bins), int(total_elems),
                                              _ptr(out.codes), _ptr(out.meta), _ptr(out.gamma),
                                              _stream_ptr(stream))
    _check(st, "sbn_quantize_weights_from_bins")
    return out


def quantize_acts(x: torch.Tensor, out_q: Optional[torch.Tensor] = None,
                  out_s: Optional[torch.Tensor] = None, stream=None):
    """sbn_quantize_acts: per-token absmax INT8. Returns (xq int8 [T,K], s fp32 [T])."""
    _need(x, torch.bfloat16, "x")
    t, k = x.shape
    if out_q is None:
        out_q = torch.empty((t, k), dtype=torch.int8, device=x.device)
    if out_s is None:
        out_s = torch.empty((t,), dtype=torch.float32, device=x.device)
    if t == 0:
        return out_q, out_s
    st = lib().sbn_quantize_acts(_ptr(x), t, k, _ptr(out_q), _ptr(out_s), _stream_ptr(stream))
    _check(st, "sbn_quantize_acts")
    return out_q, out_s


def bitlinear_workspace_bytes(t: int, k: int, n_out: int) -> int:
    """Bytes of the contraction's optional workspace (0 when T <= 16)."""
    return int(lib().sbn_bitlinear_workspace_bytes(t, k, n_out))


def _bitlinear_ws(workspace, t: int, k: int, n_out: int, device):
    """None: allocate the workspace (expanded-weights route); False: no
    workspace (weights expanded inside the kernel); else the given tensor."""
    if workspace is False:
        return None
    if workspace is None:
        nb = bitlinear_workspace_bytes(t, k, n_out)
        return torch.empty((nb,), dtype=torch.uint8, device=device) if nb else None
    return workspace


def bitlinear(xq: torch.Tensor, s: torch.Tensor, w: PackedWeights,
              out: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """sbn_bitlinear: y[t, o] = bf16(acc * gamma * s_t / 127)."""
    _need(xq, torch.int8, "xq")
    _need(s, torch.float32, "s")
    t, k = xq.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.bfloat16, device=xq.device)
    ws = _bitlinear_ws(workspace, t, k, w.n_out, xq.device)
    st = lib().sbn_bitlinear(_ptr(xq), _ptr(s), t, k, w.n_out, w.n, w.m, _ptr(w.codes),
                             _ptr(w.meta), _ptr(w.gamma), _ptr(out), _ptr(ws),
                             0 if ws is None else ws.numel(), _stream_ptr(stream))
    _check(st, "sbn_bitlinear")
    return out


def bitlinear_acc32(xq: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None,
                    workspace=None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_acc32: the exact int32 accumulators [T, N_out]."""
    _need(xq, torch.int8, "xq")
    t, k = xq.shape
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.int32, device=xq.device)
    ws = _bitlinear_ws(workspace, t, k, w.n_out, xq.device)
    st = lib().sbn_bitlinear_acc32(_ptr(xq), t, k, w.n_out, w.n, w.m, _ptr(w.codes),
                                   _ptr(w.meta), _ptr(out), _ptr(ws),
                                   0 if ws is None else ws.numel(), _stream_ptr(stream))
    _check(st, "sbn_bitlinear_acc32")
    return out


def bitlinear_x_workspace_bytes(t: int, k: int, n_out: int) -> int:
    return int(lib().sbn_bitlinear_x_workspace_bytes(t, k, n_out))


def bitlinear_x(x: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None,
                out_q: Optional[torch.Tensor] = None, out_s: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_x: y = bitlinear(quantize_acts(x)) in one call (one kernel
    for T <= 16). out_q / out_s, if given, receive Xq and s."""
    _need(x, torch.bfloat16, "x")
    t, k = x.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty((bitlinear_x_workspace_bytes(t, k, w.n_out),), dtype=torch.uint8,
                                device=x.device)
    st = lib().sbn_bitlinear_x(_ptr(x), t, k, w.n_out, w.n, w.m, _ptr(w.codes), _ptr(w.meta),
                               _ptr(w.gamma), _ptr(out), _ptr(out_q), _ptr(out_s), _ptr(workspace),
                               workspace.numel(), _stream_ptr(stream))
    _check(st, "sbn_bitlinear_x")
    return out


def mask_flips(a: PackedWeights, b: PackedWeights, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """sbn_mask_flips: positions whose keep bit differs between two packed
    versions of one layer (device int64 scalar); flip rate = count / (N_out*K)."""
    if (a.n_out, a.k, a.n, a.m) != (b.n_out, b.k, b.n, b.m):
        raise ValueError("the two packed weights describe different layers")
    if out is None:
        out = torch.empty((1,), dtype=torch.int64, device=a.codes.device)
    st = lib().sbn_mask_flips(_ptr(a.meta), _ptr(b.meta), a.n_out, a.k, a.n, a.m, _ptr(out),
                              _stream_ptr(stream))
    _check(st, "sbn_mask_flips")
    return out


def entropy_row_bytes(k: int, n: int, m: int) -> int:
    return int(lib().sbn_entropy_row_bytes(k, n, m))


def pack_entropy(w: PackedWeights, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_pack_entropy: the entropy-tight format [N_out, entropy_row_bytes] (uint8)."""
    if out is None:
        out = torch.empty((w.n_out, entropy_row_bytes(w.k, w.n, w.m)), dtype=torch.uint8,
                          device=w.codes.device)
    st = lib().sbn_pack_entropy(_ptr(w.codes), _ptr(w.meta), w.n_out, w.k, w.n, w.m, _ptr(out),
                                _stream_ptr(stream))
    _check(st, "sbn_pack_entropy")
    return out


def bitlinear_entropy(xq: torch.Tensor, s: torch.Tensor, ent: torch.Tensor, w: PackedWeights,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_entropy: decode contraction over entropy-tight weights
    (shape, pattern and gamma from the PackedWeights they were packed from)."""
    _need(xq, torch.int8, "xq")
    _need(s, torch.float32, "s")
    t, k = xq.shape
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.bfloat16, device=xq.device)
    st = lib().sbn_bitlinear_entropy(_ptr(xq), _ptr(s), t, k, w.n_out, w.n, w.m, _ptr(ent),
                                     _ptr(w.gamma), _ptr(out), _stream_ptr(stream))
    _check(st, "sbn_bitlinear_entropy")
    return out


def bitlinear_entropy_acc32(xq: torch.Tensor, ent: torch.Tensor, w: PackedWeights,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _need(xq, torch.int8, "xq")
    t, k = xq.shape
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.int32, device=xq.device)
    st = lib().sbn_bitlinear_entropy_acc32(_ptr(xq), t, k, w.n_out, w.n, w.m, _ptr(ent), _ptr(out),
                                           _stream_ptr(stream))
    _check(st, "sbn_bitlinear_entropy_acc32")
    return out


def bitlinear_entropy_x(x: torch.Tensor, ent: torch.Tensor, w: PackedWeights,
                        out: Optional[torch.Tensor] = None, out_q: Optional[torch.Tensor] = None,
                        out_s: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_entropy_x: y = bitlinear_entropy(quantize_acts(x)) in one
    call (one kernel when the bf16 rows fit in shared memory). out_q / out_s,
    if given, receive Xq and s. workspace: None allocates the two-step route's
    scratch, False passes none."""
    _need(x, torch.bfloat16, "x")
    t, k = x.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    if out is None:
        out = torch.empty((t, w.n_out), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty((int(lib().sbn_bitlinear_entropy_x_workspace_bytes(t, k)),),
                                dtype=torch.uint8, device=x.device)
    ws_ptr, ws_n = (None, 0) if workspace is False else (_ptr(workspace), workspace.numel())
    st = lib().sbn_bitlinear_entropy_x(_ptr(x), t, k, w.n_out, w.n, w.m, _ptr(ent), _ptr(w.gamma),
                                       _ptr(out), _ptr(out_q), _ptr(out_s), ws_ptr, ws_n,
                                       _stream_ptr(stream))
    _check(st, "sbn_bitlinear_entropy_x")
    return out


def bitlinear_grad_x(dy: torch.Tensor, w: PackedWeights, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """sbn_bitlinear_grad_x: dX = dY (gamma C) under the straight-through estimator."""
    _need(dy, torch.bfloat16, "dy")
    t, n_out = dy.shape
    if n_out != w.n_out:
        raise ValueError("N_out mismatch between dY and the weights")
    if out is None:
        out = torch.empty((t, w.k), dtype=torch.bfloat16, device=dy.device)
    st = lib().sbn_bitlinear_grad_x(_ptr(dy), t, w.k, w.n_out, w.n, w.m, _ptr(w.codes), _ptr(w.meta),
                                    _ptr(w.gamma), _ptr(out), _stream_ptr(stream))
    _check(st, "sbn_bitlinear_grad_x")
    return out


def bitlinear_grad_w(dy: torch.Tensor, xq: torch.Tensor, s: torch.Tensor,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_grad_w: dW = dY^T (Xq s / 127) under the straight-through
    estimator (every latent weight, pruned ones included)."""
    _need(dy, torch.bfloat16, "dy")
    _need(xq, torch.int8, "xq")
    _need(s, torch.float32, "s")
    t, n_out = dy.shape
    if xq.shape[0] != t:
        raise ValueError("T mismatch between dY and Xq")
    k = xq.shape[1]
    if out is None:
        out = torch.empty((n_out, k), dtype=torch.bfloat16, device=dy.device)
    st = lib().sbn_bitlinear_grad_w(_ptr(dy), _ptr(xq), _ptr(s), t, k, n_out, _ptr(out), _stream_ptr(stream))
    _check(st, "sbn_bitlinear_grad_w")
    return out


ACTS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4}   # SBN_ACT_*


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _need_shape(t: Optional[torch.Tensor], dtype, shape, what: str):
    """The checks of an optional tensor argument of a given shape."""
    if t is None:
        return
    _need(t, dtype, what)
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _apart(z: Optional[torch.Tensor], *others: Optional[torch.Tensor]):
    if z is not None and z.numel() and any(o is not None and o.data_ptr() == z.data_ptr() for o in others):
        raise ValueError("out_z must not be another tensor of the call")


@functools.lru_cache(maxsize=256)
def _row_bytes(k: int, n: int, m: int):
    return codes_row_bytes(k, n, m), meta_row_bytes(k, n, m)


def _need_packed(w, layers: int, dev: torch.device):
    """The packed arrays of `layers` layers are as large as the sizes beside them say."""
    c, m, g = w.codes, w.meta, w.gamma
    cr, mr = _row_bytes(w.k, w.n, w.m)
    rows = layers * w.n_out
    if c.nbytes != rows * cr or g.nbytes != 4 * layers or (m is not None and mr and m.nbytes != rows * mr):
        raise ValueError(f"the packed arrays are not those of {layers} layer(s) of {w.n_out} x {w.k} at {w.n}:{w.m}")
    if c.device != dev or g.device != dev or (m is not None and m.device != dev):
        raise ValueError(f"the packed weights must be on {dev}")
    if not (c.is_contiguous() and g.is_contiguous() and (m is None or m.is_contiguous())):
        raise ValueError("the packed weights must be contiguous")


def _act_buffers(x, rows: int, w, lead, bias, residual, out, out_z, stream):
    """Checks of the epilogue's tensors; the output, allocated if not given."""
    _need_packed(w, lead[0] if lead else 1, x.device)
    _need_shape(bias, torch.float32, lead + (w.n_out,), "bias")
    _need_shape(residual, torch.bfloat16, (rows, w.n_out), "residual")
    _need_shape(out, torch.bfloat16, (rows, w.n_out), "out")
    _need_shape(out_z, torch.bfloat16, (rows, w.n_out), "out_z")
    _one_device(x, bias, residual, out, out_z)
    _apart(out_z, out, residual)
    return _new((rows, w.n_out), torch.bfloat16, x, stream) if out is None else out


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An uninitialized tensor on the device of `like` that belongs to the call's stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _alloc_on(like.device, stream):
        return like.new_empty(shape, dtype=dtype)


def _zero(t: torch.Tensor, stream) -> torch.Tensor:
    """Zeros in `t` on the call's stream: the gradient of no rows."""
    with _alloc_on(t.device, stream):
        return t.zero_()


def _scratch(need: int, workspace, like: torch.Tensor, stream):
    if workspace is None:
        return _new((need,), torch.uint8, like, stream) if need else None
    _need(workspace, torch.uint8, "workspace")
    if workspace.device != like.device:
        raise ValueError(f"workspace must be on {like.device}")
    return workspace


def _run_with_scratch(like: torch.Tensor, name: str, stream, try_without: bool, workspace, need, args) -> None:
    """A call whose workspace is last among its arguments. A decode call mostly
    needs none: it is tried without one first (the library refuses it before
    anything is enqueued) when the caller gave none."""
    if workspace is None and try_without:
        st = _status_on(like.device, name, stream, *args, None, 0)
        if st == 0:
            return
        if SBN_STATUS[st] != "SBN_ERR_WORKSPACE":
            raise SbnError(st, name)
    ws = _scratch(need(), workspace, like, stream)
    _run_on(like.device, name, stream, *args, _ptr(ws), ws.numel())


def bitlinear_act(xq: torch.Tensor, s: torch.Tensor, w: PackedWeights, bias: Optional[torch.Tensor] = None,
                  act: str = "none", residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  out_z: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_act: y = f(z) + residual with z = acc gamma s_t / 127 + bias.
    T may be 0 in this and the following calls (nothing is enqueued, sums and
    weight gradients are zeros).

    act: "none", "relu", "relu2", "silu" or "gelu". bias: fp32 [N_out];
    residual: bf16 [T, N_out], may be `out` itself. out_z, if given, receives z
    in bf16 (the input of act_grad). workspace: as for bitlinear."""
    _need(xq, torch.int8, "xq")
    t, k = xq.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    _need_shape(s, torch.float32, (t,), "s")
    _one_device(xq, s)
    code = _act(act)
    out = _act_buffers(xq, t, w, (), bias, residual, out, out_z, stream)
    if t == 0:
        return out
    ws = None
    if workspace is not False:
        ws = _scratch(bitlinear_workspace_bytes(t, k, w.n_out), workspace, xq, stream)
    _run_on(xq.device, "sbn_bitlinear_act", stream, _ptr(xq), _ptr(s), t, k, w.n_out, w.n, w.m, _ptr(w.codes),
            _ptr(w.meta), _ptr(w.gamma), _ptr(bias), code, _ptr(residual), _ptr(out_z), _ptr(out), _ptr(ws),
            0 if ws is None else ws.numel())
    return out


def bitlinear_x_act(x: torch.Tensor, w: PackedWeights, bias: Optional[torch.Tensor] = None, act: str = "none",
                    residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    out_z: Optional[torch.Tensor] = None, out_q: Optional[torch.Tensor] = None,
                    out_s: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """sbn_bitlinear_x_act: bitlinear_act from bf16 activations (one kernel for
    T <= 16). out_q / out_s, if given, receive Xq and s."""
    _need(x, torch.bfloat16, "x")
    t, k = x.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    code = _act(act)
    _need_shape(out_q, torch.int8, (t, k), "out_q")
    _need_shape(out_s, torch.float32, (t,), "out_s")
    _one_device(x, out_q, out_s)
    out = _act_buffers(x, t, w, (), bias, residual, out, out_z, stream)
    if t == 0:
        return out
    args = (_ptr(x), t, k, w.n_out, w.n, w.m, _ptr(w.codes), _ptr(w.meta), _ptr(w.gamma), _ptr(bias), code,
            _ptr(residual), _ptr(out_z), _ptr(out), _ptr(out_q), _ptr(out_s))
    _run_with_scratch(x, "sbn_bitlinear_x_act", stream, t <= 16, workspace,
                      lambda: bitlinear_x_workspace_bytes(t, k, w.n_out), args)
    return out


def act_grad(dy: torch.Tensor, z: torch.Tensor, act: str, offsets: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, out_bias: Optional[torch.Tensor] = None, stream=None):
    """sbn_act_grad: (dz, dbias) of the epilogue, dz = dy f'(z) in bf16 and dbias
    its column sums in fp32: [N_out], or [E, N_out] for rows grouped by the
    int32 offsets [E + 1]. out may be dy itself; out_bias=False leaves the
    sums out (dbias is None). The residual's gradient is dy."""
    _need(dy, torch.bfloat16, "dy")
    rows, n_out = dy.shape
    _need_shape(z, torch.bfloat16, (rows, n_out), "z")
    _need_shape(out, torch.bfloat16, (rows, n_out), "out")
    code = _act(act)
    experts, lead = 1, ()
    if offsets is not None:
        experts = _experts_of(offsets)
        lead = (experts,)
    if out is None:
        out = _new((rows, n_out), torch.bfloat16, dy, stream)
    if out_bias is None:
        out_bias = _new(lead + (n_out,), torch.float32, dy, stream)
    dbias = None if out_bias is False else out_bias
    _need_shape(dbias, torch.float32, lead + (n_out,), "out_bias")
    _one_device(dy, z, offsets, out, dbias)
    if rows == 0:
        if dbias is not None:
            _zero(dbias, stream)
        return out, dbias
    if out.data_ptr() == z.data_ptr():
        raise ValueError("out must not be z")
    _run_on(dy.device, "sbn_act_grad", stream, _ptr(dy), _ptr(z), rows, _ptr(offsets), experts, n_out, code, _ptr(out),
            _ptr(dbias))
    return out, dbias


@dataclass
class PackedExperts:
    """Packed ternary weights of a set of layers of one shape, stacked."""
    codes: torch.Tensor            # uint8 [E, n_out, codes_row_bytes]
    meta: Optional[torch.Tensor]   # uint8 [E, n_out, meta_row_bytes] or None (n == m)
    gamma: torch.Tensor            # float32 [E]
    n_out: int
    k: int
    n: int
    m: int
    experts: int

    def expert(self, e: int) -> PackedWeights:
        """The packed weights of one expert (views)."""
        return PackedWeights(self.codes[e], None if self.meta is None else self.meta[e], self.gamma[e:e + 1],
                             self.n_out, self.k, self.n, self.m)


def alloc_experts(experts: int, n_out: int, k: int, n: int, m: int, device) -> PackedExperts:
    cr, mr = codes_row_bytes(k, n, m), meta_row_bytes(k, n, m)
    if cr == 0:
        raise SbnError(3, "alloc_experts")
    codes = torch.empty((experts, n_out, cr), dtype=torch.uint8, device=device)
    meta = torch.empty((experts, n_out, mr), dtype=torch.uint8, device=device) if mr else None
    gamma = torch.empty((experts,), dtype=torch.float32, device=device)
    return PackedExperts(codes, meta, gamma, n_out, k, n, m, experts)


def quantize_experts(w: torch.Tensor, n: int, m: int, out: Optional[PackedExperts] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> PackedExperts:
    """quantize_weights of every expert of w [E, N_out, K], each with its own gamma."""
    _need(w, torch.bfloat16, "w")
    experts, n_out, k = w.shape
    with _alloc_on(w.device, stream):
        if out is None:
            out = alloc_experts(experts, n_out, k, n, m, w.device)
        if workspace is None:
            workspace = torch.empty(workspace_bytes(n_out, k), dtype=torch.uint8, device=w.device)
    if (out.experts, out.n_out, out.k, out.n, out.m) != (experts, n_out, k, n, m):
        raise ValueError("out describes other experts")
    _need_packed(out, experts, w.device)
    _need(workspace, torch.uint8, "workspace")
    _one_device(w, workspace)
    for e in range(experts):
        p = out.expert(e)
        _run_on(w.device, "sbn_quantize_weights", stream, _ptr(w[e]), n_out, k, n, m, _ptr(p.codes), _ptr(p.meta),
                _ptr(p.gamma), _ptr(workspace), workspace.numel())
    return out


def _experts_of(offsets: torch.Tensor) -> int:
    _need(offsets, torch.int32, "offsets")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must have shape (experts + 1,)")
    return offsets.numel() - 1


def bitlinear_grouped(xq: torch.Tensor, s: torch.Tensor, offsets: torch.Tensor, w: PackedExperts,
                      bias: Optional[torch.Tensor] = None, act: str = "none",
                      residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      out_z: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sbn_bitlinear_grouped: bitlinear_act of every expert on its rows, rows
    sorted by expert, expert e owning rows offsets[e] .. offsets[e + 1] - 1
    (int32 [E + 1] on the device). bias: fp32 [E, N_out]. Rows outside
    [offsets[0], offsets[E]) of `out` keep their values."""
    _need(xq, torch.int8, "xq")
    rows, k = xq.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    if _experts_of(offsets) != w.experts:
        raise ValueError("offsets and weights differ in experts")
    _need_shape(s, torch.float32, (rows,), "s")
    _one_device(xq, s, offsets)
    code = _act(act)
    out = _act_buffers(xq, rows, w, (w.experts,), bias, residual, out, out_z, stream)
    if rows == 0:
        return out
    _run_on(xq.device, "sbn_bitlinear_grouped", stream, _ptr(xq), _ptr(s), rows, _ptr(offsets), w.experts, k, w.n_out,
            w.n, w.m, _ptr(w.codes), _ptr(w.meta), _ptr(w.gamma), _ptr(bias), code, _ptr(residual), _ptr(out_z),
            _ptr(out))
    return out


def bitlinear_grouped_x(x: torch.Tensor, offsets: torch.Tensor, w: PackedExperts,
                        bias: Optional[torch.Tensor] = None, act: str = "none",
                        residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        out_z: Optional[torch.Tensor] = None, out_q: Optional[torch.Tensor] = None,
                        out_s: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """sbn_bitlinear_grouped_x: bitlinear_grouped from bf16 activations (one
    kernel for up to 16 rows). out_q / out_s, if given, receive Xq and s of
    every row."""
    _need(x, torch.bfloat16, "x")
    rows, k = x.shape
    if k != w.k:
        raise ValueError("K mismatch between activations and weights")
    if _experts_of(offsets) != w.experts:
        raise ValueError("offsets and weights differ in experts")
    _need_shape(out_q, torch.int8, (rows, k), "out_q")
    _need_shape(out_s, torch.float32, (rows,), "out_s")
    _one_device(x, offsets, out_q, out_s)
    code = _act(act)
    out = _act_buffers(x, rows, w, (w.experts,), bias, residual, out, out_z, stream)
    if rows == 0:
        return out
    args = (_ptr(x), rows, _ptr(offsets), w.experts, k, w.n_out, w.n, w.m, _ptr(w.codes), _ptr(w.meta),
            _ptr(w.gamma), _ptr(bias), code, _ptr(residual), _ptr(out_z), _ptr(out), _ptr(out_q), _ptr(out_s))
    _run_with_scratch(x, "sbn_bitlinear_grouped_x", stream, rows <= 16, workspace,
                      lambda: int(lib().sbn_bitlinear_grouped_x_workspace_bytes(rows, k)), args)
    return out


def bitlinear_grouped_grad_x(dy: torch.Tensor, offsets: torch.Tensor, w: PackedExperts,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """sbn_bitlinear_grouped_grad_x: dX of every expert's rows (bf16 [R, K])."""
    _need(dy, torch.bfloat16, "dy")
    rows, n_out = dy.shape
    if n_out != w.n_out:
        raise ValueError("N_out mismatch between dY and the weights")
    if _experts_of(offsets) != w.experts:
        raise ValueError("offsets and weights differ in experts")
    _need_shape(out, torch.bfloat16, (rows, w.k), "out")
    _need_packed(w, w.experts, dy.device)
    _one_device(dy, offsets, out)
    if out is None:
        out = _new((rows, w.k), torch.bfloat16, dy, stream)
    if rows == 0:
        return out
    ws = _scratch(int(lib().sbn_bitlinear_grouped_grad_x_workspace_bytes(rows, n_out)), workspace, dy, stream)
    _run_on(dy.device, "sbn_bitlinear_grouped_grad_x", stream, _ptr(dy), rows, _ptr(offsets), w.experts, w.k, n_out,
            w.n, w.m, _ptr(w.codes), _ptr(w.meta), _ptr(w.gamma), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel())
    return out


def bitlinear_grouped_grad_w(dy: torch.Tensor, xq: torch.Tensor, s: torch.Tensor, offsets: torch.Tensor,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """sbn_bitlinear_grouped_grad_w: dW of every expert (bf16 [E, N_out, K]),
    zero for an expert without rows. A workspace given by the caller decides
    between two parts of dY s / 127 (22 bits of every term, as without one) and
    one (11 bits, half the MMAs), by its size."""
    _need(dy, torch.bfloat16, "dy")
    _need(xq, torch.int8, "xq")
    rows, n_out = dy.shape
    if xq.shape[0] != rows:
        raise ValueError("row mismatch between dY and Xq")
    k = xq.shape[1]
    experts = _experts_of(offsets)
    _need_shape(s, torch.float32, (rows,), "s")
    _need_shape(out, torch.bfloat16, (experts, n_out, k), "out")
    _one_device(dy, xq, s, offsets, out)
    if out is None:
        out = _new((experts, n_out, k), torch.bfloat16, dy, stream)
    if rows == 0:
        return _zero(out, stream)
    need = int(lib().sbn_bitlinear_grouped_grad_w2_workspace_bytes(rows, experts, k, n_out))
    ws = _scratch(need, workspace, dy, stream)
    _run_on(dy.device, "sbn_bitlinear_grouped_grad_w", stream, _ptr(dy), _ptr(xq), _ptr(s), rows, _ptr(offsets),
            experts, k, n_out, _ptr(out), _ptr(ws), 0 if ws is None else ws.numel())
    return out


_nbytes, _dtype_of = torch.Tensor.nbytes.__get__, torch.Tensor.dtype.__get__

ADAMW_BLOCK = 256   # SBN_ADAMW_BLOCK: elements that share a scale in the 8-bit states


class AdamW:
    """sbn_adamw: AdamW over a list of tensors, one launch per step.

        opt = AdamW(masters, lr=1e-3, state_bits=8, copies=latent_bf16)
        opt.step(grads)

    params: contiguous CUDA tensors, all fp32 or all bf16. copies (fp32
    parameters only): bf16 tensors that receive the updated parameters, the
    latent weights quantize_weights reads. state_bits: 32 keeps m and v in
    fp32; 8 keeps m and sqrt(v) as float8_e4m3fn codes with one power of two
    per 256 elements, rounded stochastically from `seed`, the step, the position
    of the tensor in the list and the index of the element.

    The state lives in m, v, m_scales, v_scales (tuples, in the order of
    params; assigning a sequence replaces them) and step_state (int32 [2] on the
    device: completed steps and a word of the library); state_dict() and
    load_state_dict() copy it. lr is a float, or
    an fp32 device tensor of one element that a captured graph reads anew at
    every replay.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr=1e-3, betas=(0.9, 0.95), eps: float = 1e-5,
                 weight_decay: float = 0.1, state_bits: int = 32,
                 copies: Optional[Sequence[torch.Tensor]] = None, seed: int = 0):
        self.params = list(params)
        self.copies = None if copies is None else list(copies)
        if not self.params:
            raise ValueError("no parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits, self.seed = state_bits, seed
        dt = self.params[0].dtype
        if dt not in (torch.float32, torch.bfloat16):
            raise TypeError(f"parameters must be float32 or bfloat16, got {dt}")
        for p in self.params:
            _need(p, dt, "params")
        self.device = _one_device(*self.params)
        if self.copies is not None:
            if dt != torch.float32:
                raise TypeError("copies go with float32 parameters")
            if len(self.copies) != len(self.params):
                raise ValueError("copies and params differ in length")
            for p, c in zip(self.params, self.copies):
                _need(c, torch.bfloat16, "copies")
                if c.numel() != p.numel():
                    raise ValueError("a copy and its parameter differ in size")
            _one_device(self.params[0], *self.copies)
        self._sizes = [p.numel() for p in self.params]
        self._kept = self.params + (self.copies or [])
        self._bytes, self._dtypes = [t.nbytes for t in self._kept], [t.dtype for t in self._kept]
        self._at = array.array("q", map(torch.Tensor.data_ptr, self._kept))   # their addresses at the last step
        self._need_apart(self._at)
        # entries of sbn_adamw_tensor: eight 64-bit words each
        self._table = array.array("q", bytes(64 * len(self.params)))
        self._table[7::8] = array.array("q", self._sizes)
        st = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        like = self.params[0]
        self.m, self.v = (self._filled(like.new_zeros, st, self._sizes) for _ in "mv")
        if state_bits == 8:
            self.m_scales, self.v_scales = (self._filled(like.new_ones, torch.float32, self._scale_sizes()) for _ in "mv")
        self.step_state = like.new_zeros(2, dtype=torch.int32)

    def _need_apart(self, at) -> None:
        spans = sorted((a, a + n) for a, n in zip(at, self._bytes) if n)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("parameters or copies overlap, or one appears twice")

    @staticmethod
    def _filled(new, dtype, sizes) -> list:
        """A tensor of every size, parts of one buffer from `new` (one fill for
        all of them) that start on multiples of ADAMW_BLOCK elements."""
        cuts = [c for n in sizes for c in (n, -n % ADAMW_BLOCK)]
        return list(torch.split_with_sizes(new(sum(cuts), dtype=dtype), cuts)[::2])

    def _own(self, column: int, tensors, dtype, sizes) -> tuple:
        """State tensors of one kind, checked, their addresses put into the table."""
        tensors = tuple(tensors)
        self._need_like_params(tensors, dtype, sizes, "state")
        self._table[column::8] = array.array("q", map(torch.Tensor.data_ptr, tensors))
        return tensors

    def _need_like_params(self, tensors, dtype, sizes, what: str):
        """Checks of one contiguous tensor for every parameter, all at once."""
        if (list(map(torch.Tensor.numel, tensors)) != sizes or not all(map(torch.Tensor.is_contiguous, tensors))
                or set(map(_dtype_of, tensors)) != {dtype}
                or set(map(torch.Tensor.get_device, tensors)) != {self.device.index}):
            for t in tensors:
                _need(t, dtype, what)
            raise ValueError(f"a {what} differs from its parameter in size or device")

    def _state_dtype(self):
        return torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn

    def _scale_sizes(self):
        if self.state_bits != 8:
            raise ValueError("scales go with 8-bit states")
        return [-(-n // ADAMW_BLOCK) for n in self._sizes]

    step_state = property(lambda self: self._step_state)

    @step_state.setter
    def step_state(self, t):
        _need(t, torch.int32, "step_state")
        if t.numel() != 2:
            raise ValueError("step_state must have two elements")
        _one_device(self.params[0], t)
        self._step_state = t

    m = property(lambda self: self._m)
    v = property(lambda self: self._v)
    m_scales = property(lambda self: self._ms)
    v_scales = property(lambda self: self._vs)
    _ms = _vs = None

    @m.setter
    def m(self, tensors):
        self._m = self._own(2, tensors, self._state_dtype(), self._sizes)

    @v.setter
    def v(self, tensors):
        self._v = self._own(3, tensors, self._state_dtype(), self._sizes)

    @m_scales.setter
    def m_scales(self, tensors):
        if tensors is not None or self.state_bits == 8:
            self._ms = self._own(4, tensors, torch.float32, self._scale_sizes())

    @v_scales.setter
    def v_scales(self, tensors):
        if tensors is not None or self.state_bits == 8:
            self._vs = self._own(5, tensors, torch.float32, self._scale_sizes())

    def step(self, grads: Sequence[torch.Tensor], grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
        """One step with the gradients of params (same order and sizes, all
        bf16 or all fp32, contiguous). grad_scale: fp32 device tensor of one
        element that multiplies every gradient first."""
        if len(grads) != len(self.params):
            raise ValueError("grads and params differ in length")
        gd = grads[0].dtype
        if gd not in (torch.float32, torch.bfloat16):
            raise TypeError(f"grads must be float32 or bfloat16, got {gd}")
        self._need_like_params(grads, gd, self._sizes, "gradient")
        lr_dev = None
        lr = self.lr
        for t, what in ((lr if isinstance(lr, torch.Tensor) else None, "lr"), (grad_scale, "grad_scale")):
            if t is not None:
                _need(t, torch.float32, what)
                if t.numel() != 1:
                    raise ValueError(f"{what} must have one element")
                _one_device(self.params[0], t)
        if isinstance(lr, torch.Tensor):
            lr_dev, lr = lr, 0.0
        # the parameters' own storage may have been exchanged since the last step
        # (an address belongs to one device, so only a new one can be elsewhere)
        table, ptr, kept = self._table, torch.Tensor.data_ptr, self._kept
        at = array.array("q", map(ptr, kept))
        if (list(map(_nbytes, kept)) != self._bytes or not all(map(torch.Tensor.is_contiguous, kept))
                or at != self._at and any((t.device, t.dtype) != (self.device, d) for t, d in zip(kept, self._dtypes))):
            raise ValueError("a parameter or a copy changed its size, type, layout or device")
        if at != self._at:
            self._need_apart(at)
            self._at = at
        n = len(self.params)
        table[0::8] = at[:n]
        table[1::8] = array.array("q", map(ptr, grads))
        if self.copies is not None:
            table[6::8] = at[n:]
        _run_on(self.device, "sbn_adamw", stream, table.buffer_info()[0], len(self.params),
                int(self.params[0].dtype == torch.bfloat16), int(gd == torch.bfloat16), self.state_bits,
                _ptr(self.step_state), float(lr), _ptr(lr_dev), float(self.betas[0]), float(self.betas[1]),
                float(self.eps), float(self.weight_decay), _ptr(grad_scale), int(self.seed) & 0xFFFFFFFF)

    def _state(self):
        names = ("m", "v") + (("m_scales", "v_scales") if self.state_bits == 8 else ())
        return {n: getattr(self, n) for n in names}

    def state_dict(self) -> dict:
        """Copies of the state (the parameters and their copies are the caller's)."""
        d = {n: [t.clone() for t in ts] for n, ts in self._state().items()}
        d["step"] = self.step_state.clone()
        d["state_bits"] = self.state_bits
        return d

    def load_state_dict(self, d: dict) -> None:
        if d["state_bits"] != self.state_bits:
            raise ValueError("the state has other state_bits")
        for n, ts in self._state().items():
            if [t.shape for t in d[n]] != [t.shape for t in ts]:
                raise ValueError("the state belongs to other parameters")
        for n, ts in self._state().items():
            for t, src in zip(ts, d[n]):
                t.copy_(src)
        self.step_state.copy_(d["step"])


def set_programmatic_launch(enable: bool) -> bool:
    """sbn_set_programmatic_launch: switch programmatic dependent launch of
    the library's kernels on or off; returns the previous setting."""
    return bool(lib().sbn_set_programmatic_launch(1 if enable else 0))


def get_device_error(stream=None) -> int:
    """sbn_get_device_error: sync the stream, read and clear the device error word."""
    return int(lib().sbn_get_device_error(_stream_ptr(stream)))


class BitLinear(torch.nn.Module):
    """BitLinear layer with a dynamic N:M mask on latent bf16 weights.

    Every forward re-derives the packed ternary weights from the latent
    weights (the mask is dynamic), quantizes the activations per token and
    runs the integer contraction. No bias. Inference only (no autograd).
    """

    def __init__(self, in_features: int, out_features: int, n: int = 6, m: int = 8,
                 device=None, weight: Optional[torch.Tensor] = None):
        super().__init__()
        if weight is None:
            weight = torch.empty((out_features, in_features), dtype=torch.bfloat16, device=device)
            torch.nn.init.normal_(weight, std=0.02)
        self.weight = torch.nn.Parameter(weight, requires_grad=False)
        self.n, self.m = n, m
        self._ws = None
        self._packed = None

    def pack(self) -> PackedWeights:
        w = self.weight.data
        if self._packed is None or self._packed.codes.device != w.device:
            self._packed = alloc_packed(w.shape[0], w.shape[1], self.n, self.m, w.device)
            self._ws = torch.empty(workspace_bytes(*w.shape), dtype=torch.uint8, device=w.device)
        return quantize_weights(w, self.n, self.m, out=self._packed, workspace=self._ws)

    @torch.no_grad()
    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        packed = self.pack()
        y = bitlinear_x(x2, packed)   # activation quantization fused for T <= 16
        return y.reshape(*lead, packed.n_out)


def probe_i8_mma(iters: int, stream=None) -> int:
    """sbn_probe_i8_mma: launches the tensor-pipe INT8 probe; returns the
    number of CTAs (each issued `iters` MMAs of 2*128*256*32 operations)."""
    ctas = ctypes.c_int32(0)
    _check(lib().sbn_probe_i8_mma(int(iters), ctypes.byref(ctas), _stream_ptr(stream)), "sbn_probe_i8_mma")
    return int(ctas.value)


def probe_i8_sparse_mma(iters: int, stream=None) -> int:
    """sbn_probe_i8_sparse_mma: launches the sparse INT8 probe on CTA pairs;
    returns the number of pairs (each issued `iters` MMAs of 2*256*224*64
    logical operations)."""
    pairs = ctypes.c_int32(0)
    _check(lib().sbn_probe_i8_sparse_mma(int(iters), ctypes.byref(pairs), _stream_ptr(stream)),
           "sbn_probe_i8_sparse_mma")
    return int(pairs.value)


def selftest_wait_timeout(which: int, limit_ns: int, stream=None) -> None:
    """sbn_selftest_wait_timeout: one bounded device wait that runs out (test hook)."""
    _check(lib().sbn_selftest_wait_timeout(int(which), int(limit_ns), _stream_ptr(stream)),
           "sbn_selftest_wait_timeout")
