"""Python binding of the B200 exact-attention C library (``libattn.so``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI of ``include/attn.h``.  PyTorch provides device
memory and the stream.  There is no CPU or library fallback: if the compiled
library is missing, every call raises.

The functions carry the C entry points' names:

* ``attn_fwd(Q, K, V, ...) -> (O, LSE)``
* ``attn_fwd_varlen(Q, K, V, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, ...) -> (O, LSE)``
* ``attn_fwd_splitkv_decode(Q, Kcache, Vcache, k_lens, ...) -> (O, LSE)``
* ``attn_fwd_splitkv_decode_paged(Q, Kpages, Vpages, block_table, k_lens, ...) -> (O, LSE)``
* ``attn_bwd(Q, K, V, O, dO, LSE, ...) -> (dQ, dK, dV)``
* ``attn_fwd_sliding`` / ``attn_bwd_sliding``: the same with a sliding-window causal mask
* ``attn_fwd_fp8(Q8, K8, V8, q_scale, k_scale, v_scale, ...) -> (O, LSE)``: E4M3 inputs with
  one scale per 128-row tile
* ``attn_fwd_splitkv_decode_noalloc``: the split decode without a workspace (a fixed
  device array of ``ATTN_NOALLOC_SCRATCH_BYTES``)
* ``attn_fwd_merge``, ``attn_merge_partial``, ``attn_accumulate``: the folds of ring
  attention's partial results (``exact_io_aware_46_b200.ring`` drives them)
* ``attn_fwd_diff(Q, K, V, lam, ...) -> (O, O2, LSE)``: differential attention (two softmax
  maps a head, subtracted with a learned weight)
* ``attn_bwd_diff(Q, K, V, lam, O, O2, dO, LSE, ...) -> (dQ, dK, dV, dlam)``: its gradients
* ``attn_fwd_splitkv_decode_diff`` / ``attn_fwd_splitkv_decode_diff_paged(...) -> (O, LSE)``: the
  same for one new token per sequence over a cache
* ``attn_kv_append_paged(K, V, Kpages, Vpages, block_table, k_lens, ...)``: new tokens' keys and
  values into a paged cache, with the position rotation applied on the way
* the ``*_workspace_size`` queries and the device-status helpers.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

#: what the compiled binding was built against: it uses torch's C++ classes, whose layout may
#: change without any symbol missing
BINDING_TAG = (f"exact_io_aware_46_b200 binding for torch {torch.__version__}, "
               f"C++11 ABI {int(torch.compiled_with_cxx11_abi())}")


def _load_binding(load):
    """The compiled checks and marshalling of the differential calls' common form; None, with a
    warning if the library itself is built, where it is missing or was built for another torch
    (the same then runs in Python)."""
    try:
        module = load()
        if getattr(module, "BUILT_FOR", None) == BINDING_TAG:
            return module
        why = f"it was built for {getattr(module, 'BUILT_FOR', 'something else')}"
    except ImportError as e:
        why = str(e)
    if os.path.exists(LIB_PATH):
        warnings.warn(f"the compiled binding is not used, small calls cost more on the host: {why}; "
                      "run `python -m exact_io_aware_46_b200.build`", RuntimeWarning, stacklevel=3)
    return None


def _import_binding():
    from . import _binding

    return _binding


_binding = _load_binding(_import_binding)

(ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT,
 ATTN_ERR_CAPACITY) = range(6)
#: size of the fixed device scratch used by attn_fwd_splitkv_decode_noalloc
ATTN_NOALLOC_SCRATCH_BYTES = 16 << 20
ATTN_MASK_NONE, ATTN_MASK_CAUSAL = 0, 1
ATTN_DEV_BAD_KLEN, ATTN_DEV_TIMEOUT, ATTN_DEV_BAD_PAGE, ATTN_DEV_BAD_SCALE = 1, 2, 4, 8

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_f = ctypes.c_float
_ll = ctypes.c_longlong

#: exported symbol -> (restype, argtypes); mirrors include/attn.h
SIGNATURES = {
    "attn_status_string": (ctypes.c_char_p, [_i]),
    "attn_num_sms": (_i, []),
    "attn_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _sz,
                      _vp]),
    "attn_fwd_sliding": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp,
                              _sz, _vp]),
    "attn_fwd_merge": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                            _vp, _sz, _vp]),
    "attn_accumulate": (_i, [_vp, _vp, _vp, ctypes.c_longlong, _i, _vp]),
    "attn_merge_partial": (_i, [_vp, _vp, _vp, _vp, _vp, ctypes.c_longlong, _i, _i, _vp]),
    "attn_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i,
                          _vp, _vp, _sz, _vp]),
    "attn_bwd_sliding": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                              _f, _i, _vp, _vp, _sz, _vp]),
    "attn_fwd_varlen_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_fwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                             _f, _i, _vp, _sz, _vp]),
    "attn_decode_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "attn_fwd_splitkv_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp,
                                     _sz, _vp]),
    "attn_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f,
                      _i, _vp, _vp, _sz, _vp]),
    "attn_fwd_splitkv_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                                             _vp, _vp]),
    "attn_fwd_splitkv_decode_paged": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i,
                                           _i, _f, _vp, _vp, _sz, _vp]),
    "attn_fwd_diff_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_fwd_diff": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i,
                           _vp, _vp, _sz, _vp]),
    "attn_bwd_diff_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_bwd_diff": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                           _i, _i, _i, _i, _f, _i, _vp, _vp, _sz, _vp]),
    "attn_decode_diff_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "attn_fwd_splitkv_decode_diff": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i,
                                          _f, _vp, _vp, _sz, _vp]),
    "attn_fwd_splitkv_decode_diff_paged": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _vp,
                                                _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp]),
    "attn_kv_append_paged_workspace_size": (_sz, []),
    "attn_kv_append_paged": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _i, _i, _i,
                                  _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _i, _i, _i, _i, _vp, _sz,
                                  _vp]),
    "attn_read_device_status": (_i, [_vp, _vp, ctypes.POINTER(ctypes.c_int32)]),
    "attn_clear_device_status": (_i, [_vp, _vp]),
}


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


#: the entry points that _binding calls, in the order that its bind() takes
_BOUND = ("attn_fwd_diff", "attn_bwd_diff", "attn_fwd_splitkv_decode_diff",
          "attn_fwd_splitkv_decode_diff_paged", "attn_kv_append_paged",
          "attn_fwd_diff_workspace_size", "attn_bwd_diff_workspace_size",
          "attn_decode_diff_workspace_size", "attn_kv_append_paged_workspace_size",
          "attn_clear_device_status", "attn_num_sms")


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library not built: {LIB_PATH} is missing "
                    "(run `python -m exact_io_aware_46_b200.build`); there is no fallback")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            if _binding is not None:
                _binding.bind(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value
                                for n in _BOUND))
            _lib = L
    return _lib


def status_string(code: int) -> str:
    try:
        return lib().attn_status_string(int(code)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(code: int, where: str) -> None:
    if code != ATTN_OK:
        raise AttnError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------------ argument validation
# Every tensor handed to the library is checked here first: a host tensor, a
# tensor on another GPU, a wrong dtype or a shape smaller than the one the
# library derives from Q and K would otherwise reach the kernels as a raw
# pointer (an illegal address, or reads and writes past an allocation).  The
# checks use only shape, dtype, device and contiguity.

_DTYPE_NAMES = {torch.bfloat16: "bfloat16", torch.float32: "float32", torch.int32: "int32",
                torch.uint8: "uint8"}


def _need(t, name, dtype, shape=None, device=None):
    """``t`` must be a contiguous CUDA tensor of ``dtype`` (and ``shape`` and
    ``device`` when given)."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape) and (device is None or t.device == device)):
        return t  # a small call costs about as much as its checks: the sound case first
    if t is None:
        raise ValueError(f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor (host memory is not accepted; "
                         f"there is no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {_DTYPE_NAMES.get(dtype, dtype)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    return t


def _opt(t, name, dtype, shape, device):
    """An optional tensor: None, or as ``_need``."""
    return None if t is None else _need(t, name, dtype, shape, device)


def _heads(Hq, Hkv):
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"query heads ({Hq}) must be a multiple of key/value heads ({Hkv})")


def _qkv(Q, K, V, dtype=torch.bfloat16, names=("Q", "K", "V")):
    """Q [B,Hq,Lq,d], K and V [B,Hkv,Lk,d] of one dtype on one device.
    Returns (B, Hq, Hkv, Lq, Lk, d, device)."""
    _need(Q, names[0], dtype)
    if Q.dim() != 4:
        raise ValueError(f"{names[0]} must be [B, H, L, d], got {tuple(Q.shape)}")
    B, Hq, Lq, d = Q.shape
    dev = Q.device
    _need(K, names[1], dtype, device=dev)
    kv = K.shape
    if len(kv) != 4 or kv[0] != B or kv[3] != d:
        raise ValueError(f"{names[1]} must be [{B}, Hkv, Lk, {d}], got {tuple(kv)}")
    _need(V, names[2], dtype, kv, dev)
    Hkv, Lk = kv[1], kv[2]
    _heads(Hq, Hkv)
    return B, Hq, Hkv, Lq, Lk, d, dev


def _klens(k_lens, B, dev, required=False):
    if k_lens is None:
        if required:
            raise ValueError("k_lens is required")
        return None
    return _need(k_lens, "k_lens", torch.int32, (B,), dev)


def _ws_check(ws, nbytes, dev):
    _need(ws, "workspace", torch.uint8, device=dev)
    if ws.numel() < nbytes:
        raise ValueError(f"workspace holds {ws.numel()} bytes, the call needs {nbytes}")
    return ws


def _bf16(t, name):
    _need(t, name, torch.bfloat16)


def _u8(t, name):
    _need(t, name, torch.uint8)


def _f32(t, name):
    _need(t, name, torch.float32)


def _workspace(nbytes: int, device, stream):
    ws = torch.empty(max(256, int(nbytes)), dtype=torch.uint8, device=device)
    _check(lib().attn_clear_device_status(_ptr(ws), _stream(stream)), "attn_clear_device_status")
    return ws


def _ws_or_new(workspace, nbytes, dev, stream):
    if workspace is None:
        return _workspace(nbytes, dev, stream)
    return _ws_check(workspace, nbytes, dev)


def attn_num_sms() -> int:
    return int(lib().attn_num_sms())


def attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d) -> int:
    return int(lib().attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d))


def attn_fwd_varlen_workspace_size(B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d) -> int:
    return int(lib().attn_fwd_varlen_workspace_size(B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d))


def attn_decode_workspace_size(B, Hq, Hkv, Lmax, d) -> int:
    return int(lib().attn_decode_workspace_size(B, Hq, Hkv, Lmax, d))


def attn_bwd_workspace_size(B, Hq, Hkv, Lq, Lk, d) -> int:
    return int(lib().attn_bwd_workspace_size(B, Hq, Hkv, Lq, Lk, d))


def attn_read_device_status(workspace, stream=None) -> tuple[int, int]:
    bits = ctypes.c_int32(0)
    code = lib().attn_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(bits))
    return int(code), int(bits.value)


def attn_clear_device_status(workspace, stream=None) -> None:
    _check(lib().attn_clear_device_status(_ptr(workspace), _stream(stream)),
           "attn_clear_device_status")


def _mask(causal):
    return ATTN_MASK_CAUSAL if causal else ATTN_MASK_NONE


def attn_fwd(Q, K, V, scale=None, causal=False, k_lens=None, O=None, lse=None, workspace=None,
             stream=None, want_lse=True):
    """Forward attention.  Q [B,Hq,Lq,d], K/V [B,Hkv,Lk,d] bf16 on the GPU.

    Returns (O, LSE) with O bf16 [B,Hq,Lq,d] and LSE fp32 [B,Hq,Lq] (None if
    ``want_lse`` is False)."""
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    _klens(k_lens, B, dev)
    _opt(O, "O", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(lse, "lse", torch.float32, (B, Hq, Lq), dev)
    workspace = _ws_or_new(workspace, attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), B, Hq, Hkv, Lq, Lk, d,
                          float(scale), _mask(causal), _ptr(k_lens), _ptr(workspace),
                          workspace.numel(), _stream(stream))
    _check(code, "attn_fwd")
    return O, lse


def attn_fwd_fp8(Q8, K8, V8, q_scale, k_scale, v_scale, scale=None, causal=False, k_lens=None,
                 O=None, lse=None, workspace=None, stream=None, want_lse=True):
    """Forward of E4M3 inputs.  Q8 [B,Hq,Lq,d], K8/V8 [B,Hkv,Lk,d] uint8 codes;
    q_scale [B,Hq,ceil(Lq/128)], k_scale/v_scale [B,Hkv,ceil(Lk/128)] fp32 (one
    scale per 128-row tile).  Returns (O bf16 [B,Hq,Lq,d], LSE fp32 [B,Hq,Lq])."""
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q8, K8, V8, torch.uint8, ("Q8", "K8", "V8"))
    _need(q_scale, "q_scale", torch.float32, (B, Hq, (Lq + 127) // 128), dev)
    _need(k_scale, "k_scale", torch.float32, (B, Hkv, (Lk + 127) // 128), dev)
    _need(v_scale, "v_scale", torch.float32, (B, Hkv, (Lk + 127) // 128), dev)
    _klens(k_lens, B, dev)
    _opt(O, "O", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(lse, "lse", torch.float32, (B, Hq, Lq), dev)
    workspace = _ws_or_new(workspace, attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty((B, Hq, Lq, d), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_fp8(_ptr(Q8), _ptr(K8), _ptr(V8), _ptr(q_scale), _ptr(k_scale),
                              _ptr(v_scale), _ptr(O), _ptr(lse), B, Hq, Hkv, Lq, Lk, d,
                              float(scale), _mask(causal), _ptr(k_lens), _ptr(workspace),
                              workspace.numel(), _stream(stream))
    _check(code, "attn_fwd_fp8")
    return O, lse


def attn_fwd_merge(Q, K, V, O_acc, lse_acc, init, O_out=None, scale=None, causal=False,
                   k_lens=None, workspace=None, stream=None):
    """attn_fwd over K/V (a subset of the keys), folded into the fp32 accumulator
    (O_acc [B,Hq,Lq,d], lse_acc [B,Hq,Lq]) in place with the normalised merge
    rule (``init``: overwrite it instead); ``O_out`` (bf16, optional) receives
    the merged O."""
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    _need(O_acc, "O_acc", torch.float32, (B, Hq, Lq, d), dev)
    _need(lse_acc, "lse_acc", torch.float32, (B, Hq, Lq), dev)
    _opt(O_out, "O_out", torch.bfloat16, (B, Hq, Lq, d), dev)
    _klens(k_lens, B, dev)
    workspace = _ws_or_new(workspace, attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    code = lib().attn_fwd_merge(_ptr(Q), _ptr(K), _ptr(V), _ptr(O_acc), _ptr(lse_acc),
                                _ptr(O_out), 1 if init else 0, B, Hq, Hkv, Lq, Lk, d,
                                float(scale), _mask(causal), _ptr(k_lens), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(code, "attn_fwd_merge")


def attn_accumulate(part, acc, init, out=None, stream=None):
    """acc (fp32) += part (bf16), or acc = part with ``init``; ``part`` None adds
    nothing; ``out`` (bf16, optional) receives the sum."""
    _need(acc, "acc", torch.float32)
    _opt(part, "part", torch.bfloat16, tuple(acc.shape), acc.device)
    _opt(out, "out", torch.bfloat16, tuple(acc.shape), acc.device)
    code = lib().attn_accumulate(_ptr(part), _ptr(acc), _ptr(out), acc.numel(),
                                 1 if init else 0, _stream(stream))
    _check(code, "attn_accumulate")


def attn_merge_partial(O_part, lse_part, O_acc, lse_acc, init, O_out=None, stream=None):
    """Fold a partial result (O_part bf16 [..., d], lse_part fp32 [...]) into the
    fp32 accumulator (O_acc, lse_acc) in place (``init``: overwrite it instead);
    ``O_out`` (bf16, optional) also receives the merged O."""
    _need(O_part, "O_part", torch.bfloat16)
    if O_part.dim() < 1:
        raise ValueError("O_part must have a trailing head dimension")
    dev = O_part.device
    rows_shape = tuple(O_part.shape[:-1])
    _need(lse_part, "lse_part", torch.float32, rows_shape, dev)
    _need(O_acc, "O_acc", torch.float32, tuple(O_part.shape), dev)
    _need(lse_acc, "lse_acc", torch.float32, rows_shape, dev)
    _opt(O_out, "O_out", torch.bfloat16, tuple(O_part.shape), dev)
    d = int(O_part.shape[-1])
    rows = O_part.numel() // d if d else 0
    code = lib().attn_merge_partial(_ptr(O_part), _ptr(lse_part), _ptr(O_acc), _ptr(lse_acc),
                                    _ptr(O_out), rows, d, 1 if init else 0, _stream(stream))
    _check(code, "attn_merge_partial")


def attn_fwd_sliding(Q, K, V, window, scale=None, k_lens=None, O=None, lse=None, workspace=None,
                     stream=None, want_lse=True):
    """Sliding-window causal forward: row i sees its ``window`` latest keys."""
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    _klens(k_lens, B, dev)
    _opt(O, "O", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(lse, "lse", torch.float32, (B, Hq, Lq), dev)
    workspace = _ws_or_new(workspace, attn_fwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_sliding(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), B, Hq, Hkv, Lq,
                                  Lk, d, float(scale), int(window), _ptr(k_lens), _ptr(workspace),
                                  workspace.numel(), _stream(stream))
    _check(code, "attn_fwd_sliding")
    return O, lse


def _bwd_args(Q, K, V, O, dO, lse, k_lens, dQ, dK, dV):
    """Validation shared by the backward entry points."""
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    _need(O, "O", torch.bfloat16, (B, Hq, Lq, d), dev)
    _need(dO, "dO", torch.bfloat16, (B, Hq, Lq, d), dev)
    _need(lse, "lse", torch.float32, (B, Hq, Lq), dev)
    _klens(k_lens, B, dev)
    _opt(dQ, "dQ", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(dK, "dK", torch.bfloat16, (B, Hkv, Lk, d), dev)
    _opt(dV, "dV", torch.bfloat16, (B, Hkv, Lk, d), dev)
    return B, Hq, Hkv, Lq, Lk, d, dev


def attn_bwd_sliding(Q, K, V, O, dO, lse, window, scale=None, k_lens=None, dQ=None, dK=None,
                     dV=None, workspace=None, stream=None):
    """Backward of attn_fwd_sliding.  Returns (dQ, dK, dV) bf16."""
    B, Hq, Hkv, Lq, Lk, d, dev = _bwd_args(Q, K, V, O, dO, lse, k_lens, dQ, dK, dV)
    workspace = _ws_or_new(workspace, attn_bwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    code = lib().attn_bwd_sliding(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse),
                                  _ptr(dQ), _ptr(dK), _ptr(dV), B, Hq, Hkv, Lq, Lk, d,
                                  float(scale), int(window), _ptr(k_lens), _ptr(workspace),
                                  workspace.numel(), _stream(stream))
    _check(code, "attn_bwd_sliding")
    return dQ, dK, dV


def attn_fwd_varlen(Q, K, V, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                    scale=None, causal=False, O=None, lse=None, workspace=None, stream=None,
                    want_lse=True):
    """Forward over packed sequences.  Q [total_q,Hq,d], K/V [total_k,Hkv,d] bf16;
    cu_seqlens_q / cu_seqlens_k int32 [B+1] on the device.  LSE is [Hq, total_q]."""
    _need(Q, "Q", torch.bfloat16)
    if Q.dim() != 3:
        raise ValueError(f"Q must be [total_q, Hq, d], got {tuple(Q.shape)}")
    total_q, Hq, d = (int(x) for x in Q.shape)
    dev = Q.device
    _need(K, "K", torch.bfloat16, device=dev)
    if K.dim() != 3 or int(K.shape[2]) != d:
        raise ValueError(f"K must be [total_k, Hkv, {d}], got {tuple(K.shape)}")
    _need(V, "V", torch.bfloat16, tuple(K.shape), dev)
    total_k, Hkv = int(K.shape[0]), int(K.shape[1])
    _heads(Hq, Hkv)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, device=dev)
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q must be a 1-D int32 tensor of B + 1 offsets")
    B = cu_seqlens_q.numel() - 1
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, (B + 1,), dev)
    _opt(O, "O", torch.bfloat16, (total_q, Hq, d), dev)
    _opt(lse, "lse", torch.float32, (Hq, total_q), dev)
    workspace = _ws_or_new(workspace, attn_fwd_varlen_workspace_size(
        B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_varlen(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                 _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, Hq, Hkv,
                                 int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, d,
                                 float(scale), _mask(causal), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(code, "attn_fwd_varlen")
    return O, lse


def _decode_args(Q, Kc, Vc, k_lens, O, lse, kv_names=("Kcache", "Vcache")):
    """Validation shared by the decode entry points: Q [B,Hq,1,d], the cache
    [X,Hkv,Y,d] (contiguous [B,Hkv,Lmax,d] or pages [n_pages,Hkv,page,d])."""
    _need(Q, "Q", torch.bfloat16)
    if Q.dim() != 4 or int(Q.shape[2]) != 1:
        raise ValueError(f"Q must be [B, Hq, 1, d], got {tuple(Q.shape)}")
    B, Hq, _, d = Q.shape
    dev = Q.device
    _need(Kc, kv_names[0], torch.bfloat16, device=dev)
    kv = Kc.shape
    if len(kv) != 4 or kv[3] != d:
        raise ValueError(f"{kv_names[0]} must be [*, Hkv, *, {d}], got {tuple(kv)}")
    _need(Vc, kv_names[1], torch.bfloat16, kv, dev)
    Hkv = kv[1]
    _heads(Hq, Hkv)
    _klens(k_lens, B, dev, required=True)
    _opt(O, "O", torch.bfloat16, (B, Hq, 1, d), dev)
    _opt(lse, "lse", torch.float32, (B, Hq), dev)
    return B, Hq, Hkv, d, dev


def attn_fwd_splitkv_decode(Q, Kc, Vc, k_lens, scale=None, O=None, lse=None, workspace=None,
                            stream=None, want_lse=True):
    """Split-KV decode.  Q [B,Hq,1,d]; Kc/Vc [B,Hkv,Lmax,d] bf16; k_lens int32 [B] (device)."""
    B, Hq, Hkv, d, dev = _decode_args(Q, Kc, Vc, k_lens, O, lse)
    if int(Kc.shape[0]) != B:
        raise ValueError(f"Kcache must be [{B}, Hkv, Lmax, {d}], got {tuple(Kc.shape)}")
    Lmax = int(Kc.shape[2])
    workspace = _ws_or_new(workspace, attn_decode_workspace_size(B, Hq, Hkv, Lmax, d), dev,
                           stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_splitkv_decode(_ptr(Q), _ptr(Kc), _ptr(Vc), _ptr(O), _ptr(lse), B, Hq,
                                         Hkv, Lmax, d, float(scale), _ptr(k_lens),
                                         _ptr(workspace), workspace.numel(), _stream(stream))
    _check(code, "attn_fwd_splitkv_decode")
    return O, lse


def attn_fwd_splitkv_decode_paged(Q, Kp, Vp, block_table, k_lens, scale=None, O=None, lse=None,
                                  workspace=None, stream=None, want_lse=True):
    """Split-KV decode over a paged cache.  Q [B,Hq,1,d]; Kp/Vp [n_pages,Hkv,page,d] bf16;
    block_table int32 [B,max_blocks] and k_lens int32 [B] on the device."""
    B, Hq, Hkv, d, dev = _decode_args(Q, Kp, Vp, k_lens, O, lse, ("Kpages", "Vpages"))
    _need(block_table, "block_table", torch.int32, device=dev)
    if block_table.dim() != 2 or int(block_table.shape[0]) != B:
        raise ValueError(f"block_table must be [{B}, max_blocks], got {tuple(block_table.shape)}")
    n_pages, page = int(Kp.shape[0]), int(Kp.shape[2])
    max_blocks = int(block_table.shape[1])
    workspace = _ws_or_new(workspace, attn_decode_workspace_size(B, Hq, Hkv, max_blocks * page, d),
                           dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_splitkv_decode_paged(_ptr(Q), _ptr(Kp), _ptr(Vp), _ptr(block_table),
                                               max_blocks, page, n_pages, _ptr(O), _ptr(lse), B,
                                               Hq, Hkv, d, float(scale), _ptr(k_lens),
                                               _ptr(workspace), workspace.numel(),
                                               _stream(stream))
    _check(code, "attn_fwd_splitkv_decode_paged")
    return O, lse


def attn_fwd_splitkv_decode_noalloc(Q, Kc, Vc, k_lens, scale=None, O=None, lse=None,
                                    stream=None, want_lse=True):
    """Split-KV decode without a workspace, for callers that cannot allocate
    device memory (the library call itself allocates nothing; this wrapper only
    creates O / LSE when they are not passed in).  Calls that overlap on the
    GPU share one fixed scratch array and race: serialise them."""
    B, Hq, Hkv, d, dev = _decode_args(Q, Kc, Vc, k_lens, O, lse)
    if int(Kc.shape[0]) != B:
        raise ValueError(f"Kcache must be [{B}, Hkv, Lmax, {d}], got {tuple(Kc.shape)}")
    Lmax = int(Kc.shape[2])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    code = lib().attn_fwd_splitkv_decode_noalloc(_ptr(Q), _ptr(Kc), _ptr(Vc), _ptr(O), _ptr(lse),
                                                 B, Hq, Hkv, Lmax, d, float(scale),
                                                 _ptr(k_lens), _stream(stream))
    _check(code, "attn_fwd_splitkv_decode_noalloc")
    return O, lse


def attn_bwd(Q, K, V, O, dO, lse, scale=None, causal=False, k_lens=None, dQ=None, dK=None,
             dV=None, workspace=None, stream=None):
    """Backward.  Returns (dQ, dK, dV) bf16."""
    B, Hq, Hkv, Lq, Lk, d, dev = _bwd_args(Q, K, V, O, dO, lse, k_lens, dQ, dK, dV)
    workspace = _ws_or_new(workspace, attn_bwd_workspace_size(B, Hq, Hkv, Lq, Lk, d), dev, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    code = lib().attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse), _ptr(dQ),
                          _ptr(dK), _ptr(dV), B, Hq, Hkv, Lq, Lk, d, float(scale),
                          _mask(causal), _ptr(k_lens), _ptr(workspace), workspace.numel(),
                          _stream(stream))
    _check(code, "attn_bwd")
    return dQ, dK, dV


# ------------------------------------------------------------------ differential attention


# Each of these functions hands sound arguments to _binding, which answers None to anything
# else (before any launch), to a stream argument, to another device than the current one and
# before the library is loaded; the Python code after it is for those.


def _done(result, where):
    if type(result) is int:  # a status that is not a refusal
        _check(result, where)
    return result


def _launch(dev, stream, call):
    """``call(handle)`` on ``stream`` (default: the current stream of the tensors' device):
    what it allocates belongs to that stream, and the tensors' device is current meanwhile."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return call(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_raw_stream(dev.index))
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


try:  # the same handle without a Stream object around it (a microsecond of a small call)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream  # noqa: F811
except ImportError:
    pass


def _own_workspace(like, nbytes, handle, clear):
    """A workspace for one call, from a bf16 tensor on its device: (tensor, bytes).  Nobody reads
    its status word, so it is cleared only where the call needs its counters at zero."""
    ws = like.new_empty(nbytes // 2)
    if clear:
        _check(lib().attn_clear_device_status(ws.data_ptr(), handle), "attn_clear_device_status")
    return ws, nbytes


@functools.lru_cache(maxsize=None)
def _sms(index):
    with torch.cuda.device(index):
        return attn_num_sms()


def _lam(lam, Hq, dev):
    _need(lam, "lam", torch.float32, device=dev)
    if lam.dim() != 1 or lam.numel() not in (1, Hq):
        raise ValueError(f"lam must be [{Hq}] or [1], got {tuple(lam.shape)}")
    return int(lam.numel())


@functools.lru_cache(maxsize=256)
def attn_fwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d) -> int:
    return int(lib().attn_fwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d))


@functools.lru_cache(maxsize=256)
def attn_decode_diff_workspace_size(B, Hq, Hkv, Lmax, d) -> int:
    return int(lib().attn_decode_diff_workspace_size(B, Hq, Hkv, Lmax, d))


def attn_fwd_diff(Q, K, V, lam, scale=None, causal=False, k_lens=None, O=None, O2=None, lse=None,
                  workspace=None, stream=None, want_aux=True):
    """Differential attention: each head row holds two maps' halves, Q = [q1 q2] and
    K = [k1 k2], and O = softmax(scale q1 k1^T) V - lam softmax(scale q2 k2^T) V.

    Q [B,Hq,Lq,d], K/V [B,Hkv,Lk,d] bf16; lam fp32 [Hq] or [1]; scale defaults to
    1/sqrt(d / 2).  Returns (O, O2, LSE): O2 [B,Hq,Lq,d] bf16, the second map's output, and
    LSE fp32 [B,Hq,2,Lq] are what attn_bwd_diff needs (None if ``want_aux`` is False and they
    are not passed in)."""
    if stream is None and _binding is not None:
        done = _binding.fwd_diff(Q, K, V, lam, scale, causal, k_lens, O, O2, lse, workspace,
                                 want_aux)
        if done is not None:
            return _done(done, "attn_fwd_diff")
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    n_lam = _lam(lam, Hq, dev)
    _klens(k_lens, B, dev)
    _opt(O, "O", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(O2, "O2", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(lse, "lse", torch.float32, (B, Hq, 2, Lq), dev)
    nbytes = attn_fwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d)
    if workspace is not None:
        _ws_check(workspace, nbytes, dev)
    scale = 1.0 / math.sqrt(d / 2) if scale is None else float(scale)

    def call(handle):
        ws, room = (workspace, workspace.numel()) if workspace is not None else _own_workspace(
            Q, nbytes, handle, B * Hq * ((Lq + 127) // 128) > _sms(dev.index))
        o = torch.empty_like(Q) if O is None else O
        o2 = torch.empty_like(Q) if want_aux and O2 is None else O2
        ls = lse
        if want_aux and ls is None:
            ls = lam.new_empty((B, Hq, 2, Lq))
        _check(lib().attn_fwd_diff(Q.data_ptr(), K.data_ptr(), V.data_ptr(), lam.data_ptr(), n_lam,
                                   o.data_ptr(), _addr(o2), _addr(ls), B, Hq, Hkv, Lq, Lk, d,
                                   scale, _mask(causal), _addr(k_lens), ws.data_ptr(), room,
                                   handle), "attn_fwd_diff")
        return o, o2, ls

    return _launch(dev, stream, call)


@functools.lru_cache(maxsize=256)
def attn_bwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d) -> int:
    return int(lib().attn_bwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d))


def attn_bwd_diff(Q, K, V, lam, O, O2, dO, lse, scale=None, causal=False, k_lens=None, dQ=None,
                  dK=None, dV=None, dlam=None, workspace=None, stream=None):
    """Backward of attn_fwd_diff, from its O, O2 and LSE.  Returns (dQ, dK, dV, dlam), bf16
    like every gradient here; dlam has lam's shape (one shared weight gets the heads' sum)."""
    if stream is None and _binding is not None:
        done = _binding.bwd_diff(Q, K, V, lam, O, O2, dO, lse, scale, causal, k_lens, dQ, dK, dV,
                                 dlam, workspace)
        if done is not None:
            return _done(done, "attn_bwd_diff")
    B, Hq, Hkv, Lq, Lk, d, dev = _qkv(Q, K, V)
    n_lam = _lam(lam, Hq, dev)
    for t, name in ((O, "O"), (O2, "O2"), (dO, "dO")):
        _need(t, name, torch.bfloat16, (B, Hq, Lq, d), dev)
    _need(lse, "lse", torch.float32, (B, Hq, 2, Lq), dev)
    _klens(k_lens, B, dev)
    _opt(dQ, "dQ", torch.bfloat16, (B, Hq, Lq, d), dev)
    _opt(dK, "dK", torch.bfloat16, (B, Hkv, Lk, d), dev)
    _opt(dV, "dV", torch.bfloat16, (B, Hkv, Lk, d), dev)
    _opt(dlam, "dlam", torch.bfloat16, (n_lam,), dev)
    nbytes = attn_bwd_diff_workspace_size(B, Hq, Hkv, Lq, Lk, d)
    if workspace is not None:
        _ws_check(workspace, nbytes, dev)
    scale = 1.0 / math.sqrt(d / 2) if scale is None else float(scale)

    def call(handle):
        ws, room = (workspace, workspace.numel()) if workspace is not None else _own_workspace(
            Q, nbytes, handle, Lq == 0)
        dq = torch.empty_like(Q) if dQ is None else dQ
        dk = torch.empty_like(K) if dK is None else dK
        dv = torch.empty_like(V) if dV is None else dV
        dl = Q.new_empty(n_lam) if dlam is None else dlam
        _check(lib().attn_bwd_diff(Q.data_ptr(), K.data_ptr(), V.data_ptr(), lam.data_ptr(), n_lam,
                                   O.data_ptr(), O2.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                                   dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dl.data_ptr(), B,
                                   Hq, Hkv, Lq, Lk, d, scale, _mask(causal), _addr(k_lens),
                                   ws.data_ptr(), room, handle), "attn_bwd_diff")
        return dq, dk, dv, dl

    return _launch(dev, stream, call)


def _decode_diff(Q, Kc, Vc, block_table, lam, k_lens, scale, O, lse, workspace, stream, want_lse):
    """Both differential decodes: contiguous cache (``block_table`` None) or pages."""
    if stream is None and _binding is not None:
        done = _binding.decode_diff(Q, Kc, Vc, block_table, lam, k_lens, scale, O, lse, workspace,
                                    want_lse)
        if done is not None:
            return _done(done, "attn_fwd_splitkv_decode_diff")
    paged = block_table is not None
    names = ("Kpages", "Vpages") if paged else ("Kcache", "Vcache")
    B, Hq, Hkv, d, dev = _decode_args(Q, Kc, Vc, k_lens, O, None, names)
    n_lam = _lam(lam, Hq, dev)
    _opt(lse, "lse", torch.float32, (B, Hq, 2), dev)
    rows = int(Kc.shape[2])
    if paged:
        _need(block_table, "block_table", torch.int32, device=dev)
        if block_table.dim() != 2 or int(block_table.shape[0]) != B:
            raise ValueError(f"block_table must be [{B}, max_blocks], "
                             f"got {tuple(block_table.shape)}")
        max_blocks = int(block_table.shape[1])
        Lmax = max_blocks * rows
    else:
        if int(Kc.shape[0]) != B:
            raise ValueError(f"Kcache must be [{B}, Hkv, Lmax, {d}], got {tuple(Kc.shape)}")
        Lmax = rows
    if Lmax > 1 << 30:
        raise ValueError(f"a cache of {Lmax} rows a sequence is past the limit of 2^30")
    nbytes = attn_decode_diff_workspace_size(B, Hq, Hkv, Lmax, d)
    if workspace is not None:
        _ws_check(workspace, nbytes, dev)
    scale = 1.0 / math.sqrt(d / 2) if scale is None else float(scale)

    def call(handle):
        ws, room = (workspace, workspace.numel()) if workspace is not None else _own_workspace(
            Q, nbytes, handle, False)
        o = torch.empty_like(Q) if O is None else O
        ls = lse
        if ls is None and want_lse:
            ls = lam.new_empty((B, Hq, 2))
        tail = (d, scale, k_lens.data_ptr(), ws.data_ptr(), room, handle)
        if paged:
            _check(lib().attn_fwd_splitkv_decode_diff_paged(
                Q.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), block_table.data_ptr(), max_blocks,
                rows, Kc.shape[0], lam.data_ptr(), n_lam, o.data_ptr(), _addr(ls), B, Hq, Hkv,
                *tail), "attn_fwd_splitkv_decode_diff_paged")
        else:
            _check(lib().attn_fwd_splitkv_decode_diff(
                Q.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), lam.data_ptr(), n_lam, o.data_ptr(),
                _addr(ls), B, Hq, Hkv, Lmax, *tail), "attn_fwd_splitkv_decode_diff")
        return o, ls

    return _launch(dev, stream, call)


def attn_fwd_splitkv_decode_diff(Q, Kc, Vc, lam, k_lens, scale=None, O=None, lse=None,
                                 workspace=None, stream=None, want_lse=True):
    """attn_fwd_diff of one new token per sequence over a cache.  Q [B,Hq,1,d]; Kc/Vc
    [B,Hkv,Lmax,d] bf16; lam fp32 [Hq] or [1]; k_lens int32 [B].  Returns (O [B,Hq,1,d] bf16,
    LSE [B,Hq,2] fp32)."""
    return _decode_diff(Q, Kc, Vc, None, lam, k_lens, scale, O, lse, workspace, stream, want_lse)


def attn_fwd_splitkv_decode_diff_paged(Q, Kp, Vp, block_table, lam, k_lens, scale=None, O=None,
                                       lse=None, workspace=None, stream=None, want_lse=True):
    """The same over a paged cache: Kp/Vp [n_pages,Hkv,page,d] bf16; block_table int32
    [B,max_blocks]."""
    if block_table is None:
        raise ValueError("block_table is required")
    return _decode_diff(Q, Kp, Vp, block_table, lam, k_lens, scale, O, lse, workspace, stream,
                        want_lse)


# ------------------------------------------------------------------ append to a paged cache


@functools.lru_cache(maxsize=1)
def attn_kv_append_paged_workspace_size() -> int:
    return int(lib().attn_kv_append_paged_workspace_size())


def _tokens(t, name, d, dev, heads=None, T=None):
    """New tokens [T, H, d] bf16 whose head rows are contiguous within a token (any token
    stride that is a multiple of 8: views of a fused projection).  Returns (T, H, stride)."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.bfloat16 and t.dim() == 3 \
            and t.device == dev:
        (t0, h0, d0), (s0, s1, s2) = t.shape, t.stride()
        if d0 == d and s2 == 1 and s1 == d and s0 % 8 == 0 and s0 >= h0 * d and t0 > 0 \
                and (heads is None or h0 == heads) and (T is None or t0 == T):
            return t0, h0, s0  # the sound case first
    if t is None:
        raise ValueError(f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor (host memory is not accepted; "
                         f"there is no CPU path)")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 3 or int(t.shape[2]) != d or (heads is not None and int(t.shape[1]) != heads) \
            or (T is not None and int(t.shape[0]) != T):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"[{'T' if T is None else T}, {'H' if heads is None else heads}, {d}]")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    T, H = int(t.shape[0]), int(t.shape[1])
    stride = H * d
    if not t.is_contiguous():
        s0, s1, s2 = (int(x) for x in t.stride())
        if s2 != 1 or (H > 1 and s1 != d) or (T > 1 and (s0 % 8 != 0 or s0 < H * d)):
            raise ValueError(f"{name} has strides {(s0, s1, s2)}: a token's rows must be "
                             f"contiguous, its tokens a multiple of 8 elements apart")
        stride = s0 if T > 1 else H * d
    return T, H, stride


def attn_kv_append_paged(K, V, Kp, Vp, block_table, k_lens, cu_seqlens=None, Q=None, Q_out=None,
                         cos=None, sin=None, maps=1, interleaved=False, workspace=None,
                         stream=None):
    """Appends new tokens to a paged cache, rotating K (and Q) by position on the way.

    K/V [T,Hkv,d] and Q [T,Hq,d] bf16, packed; tokens may be strided (views of a fused
    projection).  Kp/Vp [n_pages,Hkv,page,d]; block_table int32 [B,max_blocks]; k_lens int32 [B],
    the lengths AFTER the append (those of the decode that follows); cu_seqlens int32 [B+1]
    gives each sequence's new tokens (None: one token per sequence).  cos/sin fp32
    [n_pos, rope_dim/2] or both None (no rotation); maps = 2 rotates each half of a
    differential head by itself.  Returns the rotated Q [T,Hq,d] (None without Q); rows behind
    the last sequence are left as they were.  For attn_fwd_splitkv_decode_paged allocate the pages
    zeroed: it wants finite values behind a sequence's end (the differential decode does not)."""
    if stream is None and _binding is not None:
        done = _binding.append(K, V, Kp, Vp, block_table, k_lens, cu_seqlens, Q, Q_out, cos, sin,
                               maps, interleaved, workspace)
        if done is not None:
            return _done(done, "attn_kv_append_paged")[0]
    _need(Kp, "Kpages", torch.bfloat16)
    if Kp.dim() != 4:
        raise ValueError(f"Kpages must be [n_pages, Hkv, page, d], got {tuple(Kp.shape)}")
    n_pages, Hkv, page, d = Kp.shape
    dev = Kp.device
    _need(Vp, "Vpages", torch.bfloat16, Kp.shape, dev)
    T, _, ks = _tokens(K, "K", d, dev, Hkv)
    _, _, vs = _tokens(V, "V", d, dev, Hkv, T)
    _need(k_lens, "k_lens", torch.int32, device=dev)
    if k_lens.dim() != 1 or k_lens.numel() < 1:
        raise ValueError("k_lens must be a 1-D int32 tensor of B lengths")
    B = int(k_lens.numel())
    if cu_seqlens is None:
        if T != B:
            raise ValueError(f"{T} tokens for {B} sequences: pass cu_seqlens unless every "
                             f"sequence has one new token")
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), dev)
    _need(block_table, "block_table", torch.int32, device=dev)
    if block_table.dim() != 2 or int(block_table.shape[0]) != B:
        raise ValueError(f"block_table must be [{B}, max_blocks], got {tuple(block_table.shape)}")
    Hq, qs = Hkv, 0
    if Q is not None:
        _, Hq, qs = _tokens(Q, "Q", d, dev, None, T)
        _heads(Hq, Hkv)
        _opt(Q_out, "Q_out", torch.bfloat16, (T, Hq, d), dev)
    elif Q_out is not None:
        raise ValueError("Q_out without Q")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    n_pos = rope = 0
    if cos is not None:
        _need(cos, "cos", torch.float32, device=dev)
        if cos.dim() != 2:
            raise ValueError(f"cos must be [n_pos, rope_dim / 2], got {tuple(cos.shape)}")
        n_pos, rope = int(cos.shape[0]), 2 * int(cos.shape[1])
        _need(sin, "sin", torch.float32, cos.shape, dev)
    # the library takes these as 32-bit numbers
    for n, what in ((B, "sequences"), (block_table.shape[1], "blocks a sequence"),
                    (n_pos, "positions")):
        if n > 0x7fffffff:
            raise ValueError(f"{n} {what} are past the limit of 2^31 - 1")
    nbytes = attn_kv_append_paged_workspace_size()
    if workspace is not None:
        _ws_check(workspace, nbytes, dev)

    def call(handle):
        ws, room = (workspace, workspace.numel()) if workspace is not None else _own_workspace(
            Kp, nbytes, handle, False)
        qo = Q_out
        if Q is not None and qo is None:
            qo = Kp.new_empty((T, Hq, d))
        _check(lib().attn_kv_append_paged(
            _addr(Q), qs, K.data_ptr(), ks, V.data_ptr(), vs, _addr(qo), Kp.data_ptr(),
            Vp.data_ptr(), block_table.data_ptr(), block_table.shape[1], page, n_pages,
            _addr(cu_seqlens), k_lens.data_ptr(), B, T, Hq, Hkv, d, _addr(cos), _addr(sin), n_pos,
            rope, maps, 1 if interleaved else 0, ws.data_ptr(), room, handle),
            "attn_kv_append_paged")
        return qo

    return _launch(dev, stream, call)
