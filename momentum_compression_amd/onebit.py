"""ctypes binding of libonebit.so (the C ABI declared in include/onebit.h).

Argument marshalling only: tensors become device pointers, the stream
defaults to torch's current HIP stream, and a nonzero status raises
``OnebitError``.  Every step of the compression stage runs in the library's
HIP kernels; nothing here computes.  The library must have been built
(``python -m momentum_compression_amd.build``); a missing library is an
error, never a fallback.
"""

from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libonebit.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "onebit.h")

ONEBIT_OK = 0
ONEBIT_E_NULL = -1
ONEBIT_E_SIZE = -2
ONEBIT_E_ALIGN = -3
ONEBIT_E_WORKSPACE = -4
ONEBIT_E_ARG = -5
ONEBIT_E_HIP = -6
ONEBIT_UNIT_SCALE = 1
ONEBIT_KEEP_PREV = 2
ONEBIT_F32 = 0
ONEBIT_BF16 = 1
ONEBIT_F16 = 2

_c_i32, _c_i64, _c_u32, _c_u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
_c_f, _c_p, _c_sz = ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class FrozenVArgs(ctypes.Structure):
    """Mirror of onebit_frozen_v_args."""

    _fields_ = [
        ("mode", _c_i32), ("use_c_t", _c_i32), ("N", _c_i64),
        ("lr", _c_f), ("eps", _c_f), ("beta1", _c_f), ("beta2", _c_f),
        ("r_threshold", _c_f), ("r_min", _c_f), ("r_max", _c_f),
        ("n_seg", _c_i32),
        ("x", _c_p), ("m", _c_p), ("v", _c_p), ("m_prev", _c_p), ("v_fresh", _c_p),
        ("seg_off", _c_p), ("c_avg", _c_p), ("r_prev", _c_p), ("c_prev", _c_p),
        ("ratio_max", _c_p),
        ("m_bits", _c_p), ("m_scales", _c_p), ("m_chunks", _c_i32),
        ("err_ratio", _c_p),
        ("m_out", _c_p), ("m_seg_k", _c_p),
        ("mp_bits", _c_p), ("mp_scales", _c_p),
    ]


class RelAttentionArgs(ctypes.Structure):
    """Mirror of rel_attention_args."""

    _fields_ = [
        ("dtype", _c_i32), ("B", _c_i32), ("H", _c_i32), ("Hkv", _c_i32), ("Tq", _c_i32),
        ("Tk", _c_i32), ("D", _c_i32), ("causal", _c_i32), ("q_pos", _c_i32),
        ("n_buckets", _c_i32), ("radius", _c_i32), ("scale", _c_f), ("p", _c_f),
        ("step", _c_u32), ("seed", _c_u64), ("step_dev", _c_p), ("q_pos_of", _c_p),
        ("k_len", _c_p), ("table", _c_p), ("map", _c_p), ("q", _c_p), ("k", _c_p), ("v", _c_p),
        ("o", _c_p), ("lse", _c_p), ("q_stride", _c_i64 * 3), ("k_stride", _c_i64 * 3),
        ("v_stride", _c_i64 * 3), ("o_stride", _c_i64 * 3), ("d_o", _c_p), ("dq", _c_p),
        ("dk", _c_p), ("dv", _c_p), ("do_stride", _c_i64 * 3), ("dq_stride", _c_i64 * 3),
        ("dk_stride", _c_i64 * 3), ("dv_stride", _c_i64 * 3), ("dtable", _c_p),
        ("accumulate", _c_i32),
    ]


_SIGNATURES = {
    "onebit_compress": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_f, _c_i32, _c_p, _c_p,
                                 _c_i32, _c_p, _c_sz, _c_p]),
    "onebit_compress_grad": (_c_i32, [_c_p, _c_p, _c_p, _c_f, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_f,
                                      _c_i32, _c_p, _c_p, _c_i32, _c_p, _c_sz, _c_p]),
    "onebit_compress_ex": (_c_i32, [_c_p, _c_p, _c_p, _c_f, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_f,
                                    _c_i32, _c_p, _c_p, _c_p, _c_i32, _c_u32, _c_p, _c_sz, _c_p]),
    "onebit_server_reduce_ex": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                         _c_i32, _c_i64, _c_i32, _c_i32, _c_u32, _c_p, _c_sz,
                                         _c_p]),
    "onebit_server_reduce_noalloc": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                              _c_p, _c_i32, _c_i64, _c_i32, _c_i32, _c_u32, _c_p]),
    "int8_quantize": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_i32, _c_u64, _c_u32,
                               _c_p, _c_sz, _c_p]),
    "onebit_server_reduce": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_i64,
                                      _c_i32, _c_i32, _c_p, _c_sz, _c_p]),
    "onebit_decompress": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_i64, _c_i32, _c_p]),
    "onebit_error_materialize": (_c_i32, [_c_p, _c_p, _c_p, _c_i64, _c_i32, _c_i32, _c_p]),
    "lamb_layer_scale": (_c_i32, [_c_p, _c_i64, _c_i32, _c_p, _c_p, _c_i32, _c_i32, _c_p]),
    "frozen_v_step": (_c_i32, [ctypes.POINTER(FrozenVArgs), _c_p, _c_sz, _c_p]),
    "int8_sr_quantize": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i32, _c_u64, _c_u32, _c_p]),
    "onebit_workspace_bytes": (_c_sz, [_c_i64, _c_i32, _c_i32]),
    "frozen_v_workspace_bytes": (_c_sz, [_c_i64, _c_i32]),
    "warmup_adam_step": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_f, _c_f, _c_f, _c_f, _c_p]),
    "warmup_lamb_step": (_c_i32, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_i32, _c_f, _c_f, _c_f,
                                  _c_f, _c_f, _c_i32, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "lamb_momentum_scale": (_c_i32, [_c_p, _c_i64, _c_p, _c_i32, _c_p, _c_p, _c_sz, _c_p]),
    "warmup_workspace_bytes": (_c_sz, [_c_i64, _c_i32]),
    "dropout_apply": (_c_i32, [_c_p, _c_p, _c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64,
                               _c_f, _c_u64, _c_u32, _c_p, _c_i64, _c_p]),
    "rel_bias_expand": (_c_i32, [_c_p, _c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                 _c_i32, _c_p]),
    "rel_bias_grad": (_c_i32, [_c_p, _c_i32, _c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                               _c_i32, _c_i32, _c_i32, _c_p, _c_sz, _c_p]),
    "rel_bias_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32]),
    # the struct by reference, or its bytes as the binding packs them
    "rel_attention_forward": (_c_i32, [_c_p, _c_p, _c_sz, _c_p]),
    "rel_attention_backward": (_c_i32, [_c_p, _c_p, _c_sz, _c_p]),
    "rel_attention_workspace_bytes": (_c_sz, [_c_i32] * 8),
    "onebit_strerror": (ctypes.c_char_p, [_c_i32]),
}

_lib: Optional[ctypes.CDLL] = None


class OnebitError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({strerror(status)})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libonebit.so (raises if it has not been built).

    torch is imported first.  Its wheel carries its own HIP runtime, whose
    soname (libamdhip64.so.7) the library's dependency then resolves to, so
    the process holds one runtime, the one torch's tensors and streams
    belong to.  Loaded before torch, the library would bind to the system's
    runtime and torch would then load its own beside it: two runtimes, and
    the library's calls fail (a runtime that finds the device already taken
    reports no device)."""
    global _lib
    if _lib is None:
        import torch  # noqa: F401  (before the library: one HIP runtime)

        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m momentum_compression_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def declared_functions() -> list:
    """Function names declared in include/onebit.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\**(\w+)\s*\(", text, flags=re.M)))


def strerror(status: int) -> str:
    return load().onebit_strerror(status).decode()


def _on_gpu(t) -> bool:
    return t.is_cuda


# element kinds of the C ABI's buffers and the tensor dtypes that carry them
_KINDS = {"f32": ("float32",), "u32": ("int32", "uint32"), "i64": ("int64",),
          "i8": ("int8",), "u8": ("uint8",), "i32": ("int32",),
          "bf16": ("bfloat16",), "f16": ("float16",)}

# element types of the training operators
_DTYPES = {"float32": ("f32", ONEBIT_F32), "bfloat16": ("bf16", ONEBIT_BF16),
           "float16": ("f16", ONEBIT_F16)}


_CARRIES = set()  # (dtype object, kind) that go together, as calls meet them


def _name(dtype) -> str:
    return str(dtype).replace("torch.", "")


def _buf(x, count: int, kind: str, name: str) -> Optional[int]:
    """Device pointer of a tensor argument that must hold at least ``count``
    elements of ``kind``.  Plain integers (raw device addresses) pass as they
    are; a host tensor, a wrong dtype or a short buffer raises ValueError
    before the library sees the call (the C ABI cannot check sizes)."""
    if x is None or isinstance(x, int):
        return x
    if not _on_gpu(x):
        raise ValueError(f"{name} must be a device tensor (got {x.device})")
    if (x.dtype, kind) not in _CARRIES:
        if _name(x.dtype) not in _KINDS[kind]:
            raise ValueError(f"{name} must be {' or '.join(_KINDS[kind])} (got {x.dtype})")
        _CARRIES.add((x.dtype, kind))
    if x.numel() < count:
        raise ValueError(f"{name} holds {x.numel()} elements, the call needs {count}")
    if not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch

        # the raw handle: building a Stream object around it costs 2.7 us
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int) -> None:
    if st != ONEBIT_OK:
        raise OnebitError(fn, st)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def workspace_bytes(N: int, n: int, n_seg: int = 0) -> int:
    return int(load().onebit_workspace_bytes(N, n, n_seg))


def frozen_v_workspace_bytes(N: int, n_seg: int) -> int:
    return int(load().frozen_v_workspace_bytes(N, n_seg))


def onebit_compress(m, ef, scales, bits, N: int, n: int, clip: float = 0.0, reset: bool = False,
                    seg_off=None, seg_k=None, n_seg: int = 0, ws=None, stream=None) -> None:
    _check("onebit_compress", load().onebit_compress(
        _buf(m, n * N, "f32", "m"), _buf(ef, n * N, "f32", "ef"), _buf(scales, n * n, "f32", "scales"),
        _buf(bits, n * N // 32, "u32", "bits"), N, n, clip, int(bool(reset)),
        _buf(seg_off, n_seg + 1, "i64", "seg_off"), _buf(seg_k, n_seg, "f32", "seg_k"), n_seg,
        _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0, _stream(stream)))


def onebit_compress_grad(g, mb_bits, mb_scales, beta1: float, ef, scales, bits, N: int, n: int,
                         clip: float = 0.0, reset: bool = False, seg_off=None, seg_k=None,
                         n_seg: int = 0, ws=None, stream=None) -> None:
    _check("onebit_compress_grad", load().onebit_compress_grad(
        _buf(g, n * N, "f32", "g"), _buf(mb_bits, N // 32, "u32", "mb_bits"),
        _buf(mb_scales, n, "f32", "mb_scales"), beta1, _buf(ef, n * N, "f32", "ef"),
        _buf(scales, n * n, "f32", "scales"), _buf(bits, n * N // 32, "u32", "bits"), N, n,
        clip, int(bool(reset)), _buf(seg_off, n_seg + 1, "i64", "seg_off"),
        _buf(seg_k, n_seg, "f32", "seg_k"), n_seg, _buf(ws, 0, "u8", "ws"),
        _nbytes(ws) if ws is not None else 0, _stream(stream)))


def onebit_compress_ex(m, ef, scales, bits, N: int, n: int, mb_bits=None, mb_scales=None,
                       beta1: float = 0.0, clip: float = 0.0, reset: bool = False, seg_off=None,
                       seg_k=None, seg_err_ratio=None, n_seg: int = 0, flags: int = 0, ws=None,
                       stream=None) -> None:
    _check("onebit_compress_ex", load().onebit_compress_ex(
        _buf(m, n * N, "f32", "m"), _buf(mb_bits, N // 32, "u32", "mb_bits"),
        _buf(mb_scales, n, "f32", "mb_scales"), beta1, _buf(ef, n * N, "f32", "ef"),
        _buf(scales, n * n, "f32", "scales"), _buf(bits, n * N // 32, "u32", "bits"), N, n,
        clip, int(bool(reset)), _buf(seg_off, n_seg + 1, "i64", "seg_off"),
        _buf(seg_k, n_seg, "f32", "seg_k"), _buf(seg_err_ratio, n_seg, "f32", "seg_err_ratio"),
        n_seg, flags, _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0,
        _stream(stream)))


def onebit_server_reduce_ex(bits, scales, ef, sv_scales, sv_bits, m_out, N: int, n: int,
                            reset: bool = False, seg_off=None, seg_k=None, seg_err_ratio=None,
                            n_seg: int = 0, flags: int = 0, ws=None, stream=None) -> None:
    _check("onebit_server_reduce_ex", load().onebit_server_reduce_ex(
        _buf(bits, n * N // 32, "u32", "bits"), _buf(scales, n * n, "f32", "scales"),
        _buf(ef, N, "f32", "ef"),
        _buf(sv_scales, 2 * n if flags & ONEBIT_KEEP_PREV else n, "f32", "sv_scales"),
        _buf(sv_bits, N // 32, "u32", "sv_bits"), _buf(m_out, N, "f32", "m_out"),
        _buf(seg_off, n_seg + 1, "i64", "seg_off"), _buf(seg_k, n_seg, "f32", "seg_k"),
        _buf(seg_err_ratio, n_seg, "f32", "seg_err_ratio"), n_seg, N, n, int(bool(reset)), flags,
        _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0, _stream(stream)))


def onebit_server_reduce_noalloc(bits, scales, ef, sv_scales, sv_bits, m_out, N: int, n: int,
                                 reset: bool = False, seg_off=None, seg_k=None,
                                 seg_err_ratio=None, n_seg: int = 0, flags: int = 0,
                                 stream=None) -> None:
    """``onebit_server_reduce_ex`` without a workspace (the library's fixed
    per-device scratch)."""
    _check("onebit_server_reduce_noalloc", load().onebit_server_reduce_noalloc(
        _buf(bits, n * N // 32, "u32", "bits"), _buf(scales, n * n, "f32", "scales"),
        _buf(ef, N, "f32", "ef"),
        _buf(sv_scales, 2 * n if flags & ONEBIT_KEEP_PREV else n, "f32", "sv_scales"),
        _buf(sv_bits, N // 32, "u32", "sv_bits"), _buf(m_out, N, "f32", "m_out"),
        _buf(seg_off, n_seg + 1, "i64", "seg_off"), _buf(seg_k, n_seg, "f32", "seg_k"),
        _buf(seg_err_ratio, n_seg, "f32", "seg_err_ratio"), n_seg, N, n, int(bool(reset)), flags,
        _stream(stream)))


def onebit_server_reduce(bits, scales, ef, sv_scales, sv_bits, m_out, N: int, n: int,
                         reset: bool = False, seg_off=None, seg_k=None, n_seg: int = 0, ws=None,
                         stream=None) -> None:
    _check("onebit_server_reduce", load().onebit_server_reduce(
        _buf(bits, n * N // 32, "u32", "bits"), _buf(scales, n * n, "f32", "scales"),
        _buf(ef, N, "f32", "ef"), _buf(sv_scales, n, "f32", "sv_scales"),
        _buf(sv_bits, N // 32, "u32", "sv_bits"), _buf(m_out, N, "f32", "m_out"),
        _buf(seg_off, n_seg + 1, "i64", "seg_off"), _buf(seg_k, n_seg, "f32", "seg_k"), n_seg, N,
        n, int(bool(reset)), _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0,
        _stream(stream)))


def onebit_decompress(sv_bits, sv_scales, m_out, N: int, n: int, seg_off=None, seg_k=None,
                      n_seg: int = 0, stream=None) -> None:
    _check("onebit_decompress", load().onebit_decompress(
        _buf(sv_bits, N // 32, "u32", "sv_bits"), _buf(sv_scales, n, "f32", "sv_scales"),
        _buf(m_out, N, "f32", "m_out"), _buf(seg_off, n_seg + 1, "i64", "seg_off"),
        _buf(seg_k, n_seg, "f32", "seg_k"), n_seg, N, n, _stream(stream)))


def onebit_error_materialize(ef, scales, e_out, N: int, rows: int, n: int, stream=None) -> None:
    _check("onebit_error_materialize", load().onebit_error_materialize(
        _buf(ef, rows * N, "f32", "ef"), _buf(scales, rows * n, "f32", "scales"),
        _buf(e_out, rows * N, "f32", "e_out"), N, rows, n, _stream(stream)))


def lamb_layer_scale(buf, N: int, batch: int, seg_off, seg_k, n_seg: int, divide: bool,
                     stream=None) -> None:
    _check("lamb_layer_scale", load().lamb_layer_scale(
        _buf(buf, batch * N, "f32", "buf"), N, batch, _buf(seg_off, n_seg + 1, "i64", "seg_off"),
        _buf(seg_k, n_seg, "f32", "seg_k"), n_seg, int(bool(divide)), _stream(stream)))


def frozen_v_step(*, mode: int, N: int, x, m, v, lr: float, eps: float, beta1: float = 0.9,
                  beta2: float = 0.999, m_prev=None, v_fresh=None, seg_off=None, n_seg: int = 0,
                  c_avg=None, r_prev=None, c_prev=None, ratio_max=None, r_threshold: float = 0.1,
                  r_min: float = 0.5, r_max: float = 4.0, use_c_t: bool = False, m_bits=None,
                  m_scales=None, m_chunks: int = 0, err_ratio=None, m_out=None, m_seg_k=None,
                  mp_bits=None, mp_scales=None, ws=None, stream=None) -> None:
    a = FrozenVArgs(mode=mode, use_c_t=int(bool(use_c_t)), N=N, lr=lr, eps=eps, beta1=beta1,
                    beta2=beta2, r_threshold=r_threshold, r_min=r_min, r_max=r_max, n_seg=n_seg,
                    x=_buf(x, N, "f32", "x"), m=_buf(m, N, "f32", "m"), v=_buf(v, N, "f32", "v"),
                    m_prev=_buf(m_prev, N, "f32", "m_prev"),
                    v_fresh=_buf(v_fresh, N, "f32", "v_fresh"),
                    seg_off=_buf(seg_off, n_seg + 1, "i64", "seg_off"),
                    c_avg=_buf(c_avg, n_seg, "f32", "c_avg"), r_prev=_buf(r_prev, n_seg, "f32", "r_prev"),
                    c_prev=_buf(c_prev, n_seg, "f32", "c_prev"),
                    ratio_max=_buf(ratio_max, n_seg, "f32", "ratio_max"),
                    m_bits=_buf(m_bits, N // 32, "u32", "m_bits"),
                    m_scales=_buf(m_scales, m_chunks, "f32", "m_scales"), m_chunks=m_chunks,
                    err_ratio=_buf(err_ratio, n_seg, "f32", "err_ratio"),
                    m_out=_buf(m_out, N, "f32", "m_out"), m_seg_k=_buf(m_seg_k, n_seg, "f32", "m_seg_k"),
                    mp_bits=_buf(mp_bits, N // 32, "u32", "mp_bits"),
                    mp_scales=_buf(mp_scales, m_chunks, "f32", "mp_scales"))
    _check("frozen_v_step", load().frozen_v_step(
        ctypes.byref(a), _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0,
        _stream(stream)))


def int8_sr_quantize(g, err, codes, block_scales, deq, N: int, block: int, seed: int, step: int,
                     stream=None) -> None:
    nsc = N // block if block > 0 else 1
    _check("int8_sr_quantize", load().int8_sr_quantize(
        _buf(g, N, "f32", "g"), _buf(err, N, "f32", "err"), _buf(codes, N, "i8", "codes"),
        _buf(block_scales, nsc, "f32", "block_scales"), _buf(deq, N, "f32", "deq"), N, block,
        seed & 0xFFFFFFFFFFFFFFFF, step & 0xFFFFFFFF, _stream(stream)))


def int8_quantize(g, err, codes, block_scales, deq, N: int, block: int, rounding: int, seed: int,
                  step: int, ws=None, stream=None) -> None:
    nsc = N // block if block > 0 else 1
    _check("int8_quantize", load().int8_quantize(
        _buf(g, N, "f32", "g"), _buf(err, N, "f32", "err"), _buf(codes, N, "i8", "codes"),
        _buf(block_scales, nsc, "f32", "block_scales"), _buf(deq, N, "f32", "deq"), N, block,
        rounding, seed & 0xFFFFFFFFFFFFFFFF, step & 0xFFFFFFFF, _buf(ws, 0, "u8", "ws"),
        _nbytes(ws) if ws is not None else 0, _stream(stream)))


def warmup_workspace_bytes(N: int, n_seg: int) -> int:
    return int(load().warmup_workspace_bytes(N, n_seg))


def warmup_adam_step(x, m, v, g, N: int, lr: float, eps: float, beta1: float, beta2: float,
                     stream=None) -> None:
    _check("warmup_adam_step", load().warmup_adam_step(
        _buf(x, N, "f32", "x"), _buf(m, N, "f32", "m"), _buf(v, N, "f32", "v"),
        _buf(g, N, "f32", "g"), N, lr, eps, beta1, beta2, _stream(stream)))


def warmup_lamb_step(x, m, v, g, N: int, seg_off, n_seg: int, lr: float, eps: float, beta1: float,
                     beta2: float, beta_c: float, first: bool, c, c_avg, ws, stream=None) -> None:
    _check("warmup_lamb_step", load().warmup_lamb_step(
        _buf(x, N, "f32", "x"), _buf(m, N, "f32", "m"), _buf(v, N, "f32", "v"),
        _buf(g, N, "f32", "g"), N, _buf(seg_off, n_seg + 1, "i64", "seg_off"), n_seg, lr, eps,
        beta1, beta2, beta_c, 1 if first else 0, _buf(c, n_seg, "f32", "c"),
        _buf(c_avg, n_seg, "f32", "c_avg"), _buf(ws, 0, "u8", "ws"), _nbytes(ws), _stream(stream)))


def lamb_momentum_scale(m, N: int, seg_off, n_seg: int, k, ws, stream=None) -> None:
    _check("lamb_momentum_scale", load().lamb_momentum_scale(
        _buf(m, N, "f32", "m"), N, _buf(seg_off, n_seg + 1, "i64", "seg_off"), n_seg,
        _buf(k, n_seg, "f32", "k"), _buf(ws, 0, "u8", "ws"), _nbytes(ws), _stream(stream)))


# ---------------------------------------------------------------- training operators


def _dtype(t, name: str):
    """(element kind, C ABI type) of a training operator's tensor."""
    found = _BY_DTYPE.get(t.dtype)
    if found is None:
        found = _DTYPES.get(str(t.dtype).replace("torch.", ""))
        if found is None:
            raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
        _BY_DTYPE[t.dtype] = found
    return found


_BY_DTYPE = {}  # _DTYPES by the dtype object, as calls meet them


def _stream_of(stream, *tensors) -> Optional[int]:
    """The call's stream; its tensors must live on the device that it launches
    on (None and raw addresses are passed over)."""
    import torch

    current = torch.cuda.current_device()
    for x in tensors:
        if x is not None and type(x) is not int and x.get_device() != current:
            raise ValueError(f"a tensor is on {x.device}, the current device is cuda:{current}")
    if stream is None:
        # the raw handle: building a Stream object around it costs 2.7 us
        return torch._C._cuda_getCurrentRawStream(current)
    return _stream(stream)


def _i32(x, name: str) -> int:
    """A number that the C ABI takes in 32 bits, which would wrap silently."""
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name} = {x} does not fit in 32 bits")
    return x


def _rows(x, rows: int, cols: int, kind: str, name: str):
    """(device pointer, elements between rows) of a matrix argument: a
    contiguous buffer of at least rows * cols elements, or a 2-D view of that
    shape whose rows are contiguous."""
    if x is None:
        return None, cols
    if x.is_contiguous():
        found = _BY_DTYPE.get(x.dtype)
        if found is not None and found[0] == kind and x.numel() >= rows * cols and _on_gpu(x):
            return x.data_ptr(), cols
        return _buf(x, rows * cols, kind, name), cols
    if x.dim() != 2 or rows <= 1 and x.shape != (rows, cols):
        return _buf(x, rows * cols, kind, name), cols
    if tuple(x.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, the call needs {(rows, cols)}")
    if (x.stride(1) != 1 and cols > 1) or (x.stride(0) < cols and rows > 1):
        raise ValueError(f"{name} must have contiguous, disjoint rows")
    if not _on_gpu(x):
        raise ValueError(f"{name} must be a device tensor (got {x.device})")
    if str(x.dtype).replace("torch.", "") not in _KINDS[kind]:
        raise ValueError(f"{name} must be {' or '.join(_KINDS[kind])} (got {x.dtype})")
    return x.data_ptr(), x.stride(0) if rows > 1 else cols


def dropout_apply(x, y, rows: int, cols: int, p: float, seed: int, step: int, residual=None,
                  row0: int = 0, step_dev=None, stream=None) -> None:
    """y = [residual +] dropout(x); on the gradient, its backward pass."""
    kind, code = _dtype(x, "x")
    xp, ld_x = _rows(x, rows, cols, kind, "x")
    rp, ld_r = _rows(residual, rows, cols, kind, "residual")
    yp, ld_y = _rows(y, rows, cols, kind, "y")
    _check("dropout_apply", load().dropout_apply(
        xp, rp, yp, code, rows, cols, ld_x, ld_r, ld_y, p, seed & 0xFFFFFFFFFFFFFFFF,
        step & 0xFFFFFFFF, _buf(step_dev, 1, "u32", "step_dev"), row0,
        _stream_of(stream, x, y, residual, step_dev)))


def _shape(t, dims: int, name: str):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {t.dim()})")
    return tuple(t.shape)


def _radius(bucket_map) -> int:
    """Largest distance of a bucket map of 2 radius + 1 entries."""
    if bucket_map.dim() != 1 or bucket_map.numel() % 2 == 0:
        raise ValueError("bucket_map must hold 2 * radius + 1 buckets")
    return bucket_map.numel() // 2


def rel_bias_expand(table, bucket_map, out, q_pos: int = 0, stream=None) -> None:
    """out [H, Tq, Tk] from table [n_buckets, H]."""
    n_buckets, H = _shape(table, 2, "table")
    h, Tq, Tk = _shape(out, 3, "out")
    if h != H:
        raise ValueError(f"out has {h} heads, table has {H}")
    kind, code = _dtype(out, "out")
    radius = _radius(bucket_map)
    _check("rel_bias_expand", load().rel_bias_expand(
        _buf(table, n_buckets * H, "f32", "table"), _buf(bucket_map, 2 * radius + 1, "i32",
                                                         "bucket_map"),
        _buf(out, H * Tq * Tk, kind, "out"), code, _i32(H, "H"), _i32(n_buckets, "n_buckets"),
        _i32(radius, "radius"), _i32(Tq, "Tq"), _i32(Tk, "Tk"), _i32(q_pos, "q_pos"),
        _stream_of(stream, table, bucket_map, out)))


def rel_bias_workspace_bytes(B: int, H: int, Tq: int, Tk: int, radius: int) -> int:
    return int(load().rel_bias_workspace_bytes(_i32(B, "B"), _i32(H, "H"), _i32(Tq, "Tq"),
                                               _i32(Tk, "Tk"), _i32(radius, "radius")))


def rel_bias_grad(ds, bucket_map, dtable, q_pos: int = 0, accumulate: bool = False, ws=None,
                  stream=None) -> None:
    """dtable [n_buckets, H] from the scores' gradient ds [B, H, Tq, Tk]."""
    n_buckets, H = _shape(dtable, 2, "dtable")
    B, h, Tq, Tk = _shape(ds, 4, "ds")
    if h != H:
        raise ValueError(f"ds has {h} heads, dtable has {H}")
    kind, code = _dtype(ds, "ds")
    radius = _radius(bucket_map)
    _check("rel_bias_grad", load().rel_bias_grad(
        _buf(ds, B * H * Tq * Tk, kind, "ds"), code, _buf(bucket_map, 2 * radius + 1, "i32",
                                                          "bucket_map"),
        _buf(dtable, n_buckets * H, "f32", "dtable"), _i32(B, "B"), _i32(H, "H"),
        _i32(n_buckets, "n_buckets"), _i32(radius, "radius"), _i32(Tq, "Tq"), _i32(Tk, "Tk"),
        _i32(q_pos, "q_pos"), int(bool(accumulate)), _buf(ws, 0, "u8", "ws"),
        _nbytes(ws) if ws is not None else 0, _stream_of(stream, ds, bucket_map, dtable, ws)))


def rel_attention_workspace_bytes(B: int, H: int, Hkv: int, Tq: int, Tk: int, D: int,
                                  radius: int = 0, backward: bool = False) -> int:
    return int(load().rel_attention_workspace_bytes(
        _i32(B, "B"), _i32(H, "H"), _i32(Hkv, "Hkv"), _i32(Tq, "Tq"), _i32(Tk, "Tk"), _i32(D, "D"),
        _i32(radius, "radius"), int(bool(backward))))


def _heads(x, shape, dtype, device: int, name: str):
    """(device pointer, strides of sequences, tokens and heads) of a
    [B, T, heads, D] tensor of any strides, D side by side, on the device of
    the call's others."""
    st = x.stride()
    if x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, the call needs {tuple(shape)}")
    if x.get_device() != device:
        raise ValueError(f"{name} is on {x.device}, not with q")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {str(dtype).replace('torch.', '')} (got {x.dtype})")
    if st[3] != 1 and shape[3] > 1 and x.numel():
        raise ValueError(f"{name}: the elements of a head must lie side by side")
    # a dimension of one element has no stride of its own
    return (x.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0,
            st[2] if shape[2] > 1 else 0)


# rel_attention_args as one packing: the struct's fields in order (its size and
# offsets are checked against the declaration by the tests)
_ATTENTION = struct.Struct("<11i2fIQ10q12q4q12qqi4x")
_NONE = (0, 0, 0, 0)


def _attention_args(q, k, v, o, lse, scale, causal, q_pos, k_len, table, bucket_map, p, seed, step,
                    step_dev, do=None, dq=None, dk=None, dv=None, dtable=None, accumulate=False):
    q_shape, k_shape = q.shape, k.shape
    if len(q_shape) != 4 or len(k_shape) != 4:
        raise ValueError("q and k must have 4 dimensions")
    B, Tq, H, D = q_shape
    _, Tk, Hkv, _ = k_shape
    kind, code = _dtype(q, "q")
    if kind == "f32":
        raise ValueError("attention takes bfloat16 or float16 (got torch.float32)")
    if not _on_gpu(q):
        raise ValueError(f"q must be a device tensor (got {q.device})")
    dt, dev = q.dtype, q.get_device()
    kv_shape = (B, Tk, Hkv, D)
    qp, kp = _heads(q, q_shape, dt, dev, "q"), _heads(k, kv_shape, dt, dev, "k")
    vp, op = _heads(v, kv_shape, dt, dev, "v"), _heads(o, q_shape, dt, dev, "o")
    n_buckets = radius = tp = mp = pos = 0
    pos_of = None
    if isinstance(q_pos, int):
        pos = q_pos
    else:
        pos_of = _buf(q_pos, B, "i32", "q_pos")
    if (table is None) != (bucket_map is None):
        raise ValueError("a bias needs its table and its bucket map")
    if table is not None:
        n_buckets, heads = _shape(table, 2, "table")
        if heads != H:
            raise ValueError(f"table has {heads} heads, q has {H}")
        radius = _radius(bucket_map)
        tp = _buf(table, n_buckets * H, "f32", "table")
        mp = _buf(bucket_map, 2 * radius + 1, "i32", "bucket_map")
    gp = dqp = dkp = dvp = _NONE
    if do is not None:
        gp, dqp = _heads(do, q_shape, dt, dev, "do"), _heads(dq, q_shape, dt, dev, "dq")
        dkp, dvp = _heads(dk, k_shape, dt, dev, "dk"), _heads(dv, k_shape, dt, dev, "dv")
        if dtable is not None and table is not None and dtable.shape != table.shape:
            raise ValueError(f"dtable has shape {tuple(dtable.shape)}, table {tuple(table.shape)}")
    lens = _buf(k_len, B, "i32", "k_len") or 0
    lse_p = _buf(lse, B * H * Tq, "f32", "lse") or 0
    dtp = _buf(dtable, n_buckets * H, "f32", "dtable") or 0
    step_p = _buf(step_dev, 1, "u32", "step_dev") or 0
    try:
        return _ATTENTION.pack(
            code, B, H, Hkv, Tq, Tk, D, 1 if causal else 0, pos, n_buckets, radius,
            D ** -0.5 if scale is None else scale, p, step & 0xFFFFFFFF, seed & 0xFFFFFFFFFFFFFFFF,
            step_p, pos_of or 0, lens, tp, mp, qp[0], kp[0], vp[0], op[0], lse_p,
            *qp[1:], *kp[1:], *vp[1:], *op[1:], gp[0], dqp[0], dkp[0], dvp[0],
            *gp[1:], *dqp[1:], *dkp[1:], *dvp[1:], dtp, 1 if accumulate else 0)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"a size, position, scale or p is not a number of 32 bits: {e}") from None


def rel_attention_forward(q, k, v, o, lse=None, scale: Optional[float] = None,
                          causal: bool = False, q_pos=0, k_len=None, table=None, bucket_map=None,
                          p: float = 0.0, seed: int = 0, step: int = 0, step_dev=None, ws=None,
                          stream=None) -> None:
    """o [B, Tq, H, D] (and lse [B, H, Tq]) from q [B, Tq, H, D] and k, v
    [B, Tk, Hkv, D]; scale is D ** -0.5 unless given, q_pos a number or an
    int32 tensor [B]."""
    a = _attention_args(q, k, v, o, lse, scale, causal, q_pos, k_len, table, bucket_map, p, seed,
                        step, step_dev)
    _check("rel_attention_forward", load().rel_attention_forward(
        a, _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0,
        _stream_of(stream, q, lse, q_pos, k_len, table, bucket_map, step_dev, ws)))


def rel_attention_backward(q, k, v, o, lse, do, dq, dk, dv, dtable=None, accumulate: bool = False,
                           scale: Optional[float] = None, causal: bool = False, q_pos=0,
                           k_len=None, table=None, bucket_map=None, p: float = 0.0, seed: int = 0,
                           step: int = 0, step_dev=None, ws=None, stream=None) -> None:
    """dq, dk, dv (and dtable) from the forward call's arguments, its o and lse
    and the gradient do."""
    a = _attention_args(q, k, v, o, lse, scale, causal, q_pos, k_len, table, bucket_map, p, seed,
                        step, step_dev, do, dq, dk, dv, dtable, accumulate)
    _check("rel_attention_backward", load().rel_attention_backward(
        a, _buf(ws, 0, "u8", "ws"), _nbytes(ws) if ws is not None else 0,
        _stream_of(stream, q, lse, dtable, q_pos, k_len, table, bucket_map, step_dev, ws)))
