"""Python binding of libaq (include/aq.h): affine group-64 3/4-bit matmul on GB300.

Argument marshalling only.  Every function has the name of the C entry point
it calls; tensors are torch tensors (device memory for ``*_dev`` arguments),
``stream`` defaults to torch's current CUDA stream.  All the work runs in the
library's CUDA kernels; there is no Python or CPU compute path, and importing
this package fails if libaq.so cannot be loaded.

    y = aq_matmul(x, Wq, scales, biases, bits)        # fp16 x -> fp16 y
    y = aq_matmul_bf16(x, Wq, scales, biases, bits)   # bf16 x -> bf16 y
    Wq = aq_pack(codes, bits)                         # uint8 codes -> uint32 words
    y, ids, weights = aq_moe(x, AqRouter(...), AqExperts(...))  # experts' layer
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, Optional, Union

import torch

from . import build as _build

__all__ = [
    "AqError", "AQ_F16", "AQ_BF16", "AQ_VARIANT_AUTO", "AQ_VARIANT_GENERIC", "AQ_VARIANT_QMV",
    "AQ_VARIANT_TC", "AQ_VARIANT_GEMV", "AQ_VARIANT_TCW", "AQ_NUM_VARIANTS", "aq_pack", "aq_quantize",
    "aq_quantize_bf16", "aq_matmul", "aq_matmul_bf16", "aq_matmul_multi", "aq_matmul_gate_up",
    "aq_matmul_ex", "aq_quantize_ex", "aq_attention_decode", "aq_attention_describe",
    "aq_attention_workspace_bytes", "aq_attention_decode_ws", "aq_attention_describe_ws",
    "aq_attention_decode_static", "AqCache", "aq_cache_record_bytes", "aq_cache_append",
    "aq_cache_read", "aq_cache_copy", "aq_cache_fork", "aq_cache_trim", "aq_cache_grow",
    "aq_cache_compact", "aq_cache_workspace_bytes", "aq_attention_batch",
    "aq_attention_batch_workspace_bytes",
    "AQ_SCORE_SOFTMAX", "AQ_SCORE_SIGMOID", "AqRouter", "AqExperts", "aq_moe_route",
    "aq_moe_experts", "aq_moe", "aq_moe_workspace_bytes", "aq_embed",
    "aq_matmul_variant", "aq_matmul_host", "aq_select", "aq_describe", "aq_stats", "aq_stats_reset",
    "aq_device_error",
    "aq_free", "aq_status_string", "aq_variant_name", "aq_version", "lib_path", "load",
]

AQ_OK = 0
AQ_F16, AQ_BF16 = 0, 1
AQ_VARIANT_AUTO, AQ_VARIANT_GENERIC, AQ_VARIANT_QMV, AQ_VARIANT_TC = -1, 0, 1, 2
AQ_VARIANT_GEMV = 3
AQ_VARIANT_TCW = 4
AQ_NUM_VARIANTS = 5
AQ_SCORE_SOFTMAX, AQ_SCORE_SIGMOID = 0, 1

_lib: Optional[ctypes.CDLL] = None


class AqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {aq_status_string(status)} (status {status})")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libaq.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(path):
        raise ImportError(f"libaq.so not built at {path}")
    lib = ctypes.CDLL(path)
    p, i64, i32, u32p = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    sz, f32 = ctypes.c_size_t, ctypes.c_float
    sig = {
        "aq_pack": ([p, i64, i64, i32, p, p], i32),
        "aq_quantize": ([p, i64, i64, i32, p, p, p, p], i32),
        "aq_matmul_multi": ([i32, p, i32, p, p, p, p, i64, i64, i32, p, p], i32),
        "aq_matmul_ex": ([i32, p, p, p, p, i64, i64, i64, i32, i32, p, p], i32),
        "aq_attention_decode": ([i32, p, p, p, p, p, p, p, i64, i64, i64, i64, i32, i32, p, p],
                                i32),
        "aq_quantize_ex": ([i32, p, i64, i64, i32, i32, p, p, p, p], i32),
        "aq_matmul_gate_up": ([i32, p, p, p, p, p, p, p, i64, i64, i64, i32, p, p], i32),
        "aq_quantize_bf16": ([p, i64, i64, i32, p, p, p, p], i32),
        "aq_matmul": ([p, p, p, p, i64, i64, i64, i32, p, p], i32),
        "aq_matmul_bf16": ([p, p, p, p, i64, i64, i64, i32, p, p], i32),
        "aq_matmul_variant": ([i32, i32, p, p, p, p, i64, i64, i64, i32, p, p], i32),
        "aq_matmul_host": ([i32, p, p, p, p, i64, i64, i64, i32, p, p, p, p], i32),
        "aq_select": ([i64, i64, i64, i32, i32], i32),
        "aq_describe": ([i64, i64, i64, i32, i32, p, i32], i32),
        "aq_attention_describe": ([i64, i64, i64, i64, i32, i32, p, i32], i32),
        "aq_attention_workspace_bytes": ([i64, i64, i64, i64, i32, i32], sz),
        "aq_attention_decode_ws": ([i32, p, p, p, p, p, p, p, i64, i64, i64, i64, i32, i32, p, p,
                                    sz, p], i32),
        "aq_attention_describe_ws": ([i64, i64, i64, i64, i32, i32, sz, p, i32], i32),
        "aq_attention_decode_static": ([i32, p, p, p, p, p, p, p, i64, i64, i64, i64, i32, i32, p,
                                        p], i32),
        "aq_cache_record_bytes": ([i64, i32, i32, i32], sz),
        "aq_cache_append": ([p, i64, i32, p, i64, p, i64, i64, p, p, p, i64, i64, p], i32),
        "aq_cache_read": ([p, i64, i32, p, p, i64, p, p, p, i64, i64, p], i32),
        "aq_cache_copy": ([p, p, p, i64, p], i32),
        "aq_cache_workspace_bytes": ([i64, i64], sz),
        "aq_cache_fork": ([p, p, p, p, p, p, i64, i64, p, p, p, p, p], i32),
        "aq_cache_trim": ([p, p, p, p, p, i64, i64, p, p, p, p, p], i32),
        "aq_cache_grow": ([p, p, p, p, p, i64, i64, p, p, p, p, p, sz, p], i32),
        "aq_cache_compact": ([p, p, p, p, i64, i64, p, p, p, p, sz, p], i32),
        "aq_attention_batch_workspace_bytes": ([p, i64, i64, i64, i64], sz),
        "aq_attention_batch": ([p, i64, i32, p, i64, p, p, p, p, i64, i64, i64, i64, i64, f32, p,
                                p, sz, p], i32),
        "aq_moe_route": ([p, p, i64, p, p, p], i32),
        "aq_moe_workspace_bytes": ([p, i64, i32], sz),
        "aq_moe_experts": ([p, i32, p, i64, i32, p, p, p, p, sz, p], i32),
        "aq_moe": ([p, p, p, i64, p, p, p, p, sz, p], i32),
        "aq_embed": ([i32, p, i32, i64, p, p, p, i64, i64, i32, i32, f32, p, p], i32),
        "aq_stats": ([p, i32], i32),
        "aq_stats_reset": ([], None),
        "aq_device_error": ([u32p, i32], i32),
        "aq_free": ([], None),
        "aq_status_string": ([i32], ctypes.c_char_p),
        "aq_variant_name": ([i32], ctypes.c_char_p),
        "aq_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _stream(stream) -> int:
    if stream is None:
        # the handle alone: a Stream object costs microseconds a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _side(stream, device):
    """The torch stream of a call that is not on the current one, else None."""
    if stream is None or device.type != "cuda":
        return None
    if _stream(stream) == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _on(side, device, make):
    """make() with the stream `side` as the current one (torch.cuda.stream's
    work without its second look at everything: 1 us, not 7)."""
    if side is None:
        return make()
    sid, index, kind = torch._C._cuda_getCurrentStream(device.index)
    torch._C._cuda_setStream(stream_id=side.stream_id, device_index=side.device_index,
                             device_type=side.device_type)
    try:
        return make()
    finally:
        torch._C._cuda_setStream(stream_id=sid, device_index=index, device_type=kind)


def _empty(shape, dtype, device, stream, result=True) -> torch.Tensor:
    """Memory that a call writes, of the call's stream: a block of the current
    stream's may still be in use by kernels that wait there, and would return
    there while this call's run.  A result is also known to the current
    stream, where the caller may drop it while kernels there read it."""
    side = _side(stream, device)
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    t = _on(side, device, lambda: torch.empty(shape, dtype=dtype, device=device))
    if result:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace for one call, handed back to its stream's memory on return."""
    return _empty(nbytes, torch.uint8, device, stream, result=False)


def _check(status: int, what: str) -> None:
    if status != AQ_OK:
        raise AqError(status, what)


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _sized(t: torch.Tensor, name: str, nbytes: int, dtype=None) -> None:
    """The library reads or writes exactly nbytes through t's pointer: a
    buffer of another size (or dtype) is refused here, before any launch."""
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if _nbytes(t) != nbytes:
        raise ValueError(f"{name} holds {_nbytes(t)} bytes; this call uses {nbytes}")


_ACT = (torch.float16, torch.bfloat16)


def _check_weights(Wq, scales, biases, N: int, K: int, bits: int, group: int,
                   tag: str = "") -> None:
    """Sizes of one packed weight matrix; checked only when the arguments are
    otherwise valid (the library reports invalid ones with its own status)."""
    if bits not in (2, 3, 4, 5, 6, 8) or group not in (32, 64, 128) or K <= 0 or N <= 0:
        return
    if K % group or (K * bits) % 32:
        return
    _sized(Wq, f"Wq{tag}", N * K * bits // 8)
    _sized(scales, f"scales{tag}", 2 * N * (K // group), torch.float16)
    _sized(biases, f"biases{tag}", 2 * N * (K // group), torch.float16)


def _check_out(out, name: str, numel: int, dtype) -> None:
    if out.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {out.dtype}")
    _sized(out, name, numel * out.element_size())


def aq_status_string(status: int) -> str:
    return load().aq_status_string(status).decode()


def aq_variant_name(variant: int) -> str:
    return load().aq_variant_name(variant).decode()


def aq_version() -> str:
    return load().aq_version().decode()


def aq_pack(codes: torch.Tensor, bits: int, words: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """codes uint8 [N, K] (device) -> words uint32-as-int32 [N, K*bits/32]."""
    N, K = codes.shape
    if codes.dtype != torch.uint8:
        raise ValueError("codes must be uint8")
    if words is None:
        words = _empty((N, K * bits // 32), torch.int32, codes.device, stream)
    elif bits in (2, 3, 4, 5, 6, 8) and K % 32 == 0:
        _sized(words, "words", N * K * bits // 8)
    _check(load().aq_pack(_dev(codes, "codes"), N, K, bits, _dev(words, "words"),
                          _stream(stream)), "aq_pack")
    return words


def _quantize(dtype, w: torch.Tensor, bits: int, stream) -> tuple:
    want = torch.float16 if dtype == AQ_F16 else torch.bfloat16
    if w.dtype != want:
        raise ValueError(f"w must be {want}")
    N, K = w.shape
    Wq = _empty((N, K * bits // 32), torch.int32, w.device, stream)
    scales = _empty((N, K // 64), torch.float16, w.device, stream)
    biases = _empty((N, K // 64), torch.float16, w.device, stream)
    f = load().aq_quantize if dtype == AQ_F16 else load().aq_quantize_bf16
    _check(f(_dev(w, "w"), N, K, bits, _dev(Wq, "Wq"), _dev(scales, "scales"),
             _dev(biases, "biases"), _stream(stream)), "aq_quantize")
    return Wq, scales, biases


def aq_quantize(w: torch.Tensor, bits: int, stream=None) -> tuple:
    """fp16 weights [N, K] (device) -> (Wq uint32-as-int32 [N, K*bits/32],
    scales fp16 [N, K/64], biases fp16 [N, K/64])."""
    return _quantize(AQ_F16, w, bits, stream)


def aq_quantize_bf16(w: torch.Tensor, bits: int, stream=None) -> tuple:
    """aq_quantize for bf16 weights."""
    return _quantize(AQ_BF16, w, bits, stream)


def _mm(variant: int, dtype: int, x, Wq, scales, biases, bits, out, stream) -> torch.Tensor:
    want = torch.float16 if dtype == AQ_F16 else torch.bfloat16
    if x.dtype != want:
        raise ValueError(f"x must be {want}")
    if scales.dtype != torch.float16 or biases.dtype != torch.float16:
        raise ValueError("scales and biases must be float16")
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    N = scales.shape[0]
    if bits in (3, 4):
        _check_weights(Wq, scales, biases, N, K, bits, 64)
    if out is None:
        out = _empty((*x.shape[:-1], N), x.dtype, x.device, stream)
    _check_out(out, "out", M * N, x.dtype)
    _check(load().aq_matmul_variant(variant, dtype, _dev(x, "x"), _dev(Wq, "Wq"),
                                    _dev(scales, "scales"), _dev(biases, "biases"), M, N, K,
                                    bits, _dev(out, "out"), _stream(stream)), "aq_matmul")
    return out


def aq_matmul(x, Wq, scales, biases, bits, out=None, stream=None) -> torch.Tensor:
    """y = x . dequant(W)^T for fp16 x [..., K]; returns fp16 [..., N]."""
    return _mm(AQ_VARIANT_AUTO, AQ_F16, x, Wq, scales, biases, bits, out, stream)


def aq_matmul_bf16(x, Wq, scales, biases, bits, out=None, stream=None) -> torch.Tensor:
    """y = x . dequant(W)^T for bf16 x [..., K]; returns bf16 [..., N]."""
    return _mm(AQ_VARIANT_AUTO, AQ_BF16, x, Wq, scales, biases, bits, out, stream)


def aq_matmul_ex(x, Wq, scales, biases, bits, group_size, out=None, stream=None):
    """Any code width of 2/3/4/5/6/8 bits and group size of 32/64/128; the
    dtype follows x (fp16 or bf16)."""
    if x.dtype not in _ACT:
        raise ValueError("x must be float16 or bfloat16")
    dtype = AQ_BF16 if x.dtype == torch.bfloat16 else AQ_F16
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    N = scales.shape[0]
    _check_weights(Wq, scales, biases, N, K, bits, group_size)
    if out is None:
        out = _empty((*x.shape[:-1], N), x.dtype, x.device, stream)
    _check_out(out, "out", M * N, x.dtype)
    _check(load().aq_matmul_ex(dtype, _dev(x, "x"), _dev(Wq, "Wq"), _dev(scales, "scales"),
                               _dev(biases, "biases"), M, N, K, bits, group_size,
                               _dev(out, "out"), _stream(stream)), "aq_matmul_ex")
    return out


def _attention_args(q, k, v, bits, group_size, out, stream):
    if q.dtype not in _ACT:
        raise ValueError("q must be float16 or bfloat16")
    if q.dim() != 2 or len(k) != 3 or len(v) != 3 or any(t.dim() != 3 for t in (*k, *v)):
        raise ValueError("q must be [H, D]; k and v (words, scales, biases), each [KV, N, ...]")
    dtype = AQ_BF16 if q.dtype == torch.bfloat16 else AQ_F16
    H, D = q.shape
    KV, N = k[0].shape[0], k[0].shape[1]
    if bits in (4, 8) and group_size in (32, 64, 128) and D > 0 and D % group_size == 0:
        for side, (w, sc, bi) in (("k", k), ("v", v)):
            _sized(w, f"{side}_words", KV * N * D * bits // 8)
            _sized(sc, f"{side}_scales", 2 * KV * N * (D // group_size), torch.float16)
            _sized(bi, f"{side}_biases", 2 * KV * N * (D // group_size), torch.float16)
    if out is None:
        out = _empty((H, D), q.dtype, q.device, stream)
    _check_out(out, "out", H * D, q.dtype)
    ptrs = (_dev(q, "q"), _dev(k[0], "k_words"), _dev(k[1], "k_scales"), _dev(k[2], "k_biases"),
            _dev(v[0], "v_words"), _dev(v[1], "v_scales"), _dev(v[2], "v_biases"))
    return dtype, ptrs, (H, KV, N, D), out


def aq_attention_decode(q, k, v, bits, group_size, out=None, stream=None) -> torch.Tensor:
    """Decode attention over a quantised KV cache.  q [H, D] (fp16 or bf16);
    k and v are (words [KV, N, D*bits/32] int32, scales [KV, N, D/group] fp16,
    biases [KV, N, D/group] fp16).  Returns o [H, D] in q's dtype."""
    dtype, ptrs, (H, KV, N, D), out = _attention_args(q, k, v, bits, group_size, out, stream)
    _check(load().aq_attention_decode(dtype, *ptrs, H, KV, N, D, bits, group_size,
                                      _dev(out, "out"), _stream(stream)), "aq_attention_decode")
    return out


def aq_attention_decode_static(q, k, v, bits, group_size, out=None, stream=None) -> torch.Tensor:
    """aq_attention_decode_ws with the library's own fixed scratch instead of
    a workspace (nothing allocated per call); calls on one device must not
    overlap in time."""
    dtype, ptrs, (H, KV, N, D), out = _attention_args(q, k, v, bits, group_size, out, stream)
    _check(load().aq_attention_decode_static(dtype, *ptrs, H, KV, N, D, bits, group_size,
                                             _dev(out, "out"), _stream(stream)),
           "aq_attention_decode_static")
    return out


def aq_attention_workspace_bytes(H: int, KV: int, N: int, D: int, bits: int,
                                 group_size: int) -> int:
    """Workspace bytes for aq_attention_decode_ws's several-cluster plan (0:
    one cluster per KV head is best, or the sizes are refused)."""
    return int(load().aq_attention_workspace_bytes(H, KV, N, D, bits, group_size))


def aq_attention_decode_ws(q, k, v, bits, group_size, workspace=None, out=None,
                           stream=None) -> torch.Tensor:
    """aq_attention_decode with a workspace (a uint8 device tensor whose
    first KV 32-bit words are zero before the first call; every call leaves
    them zero).  workspace=None allocates a zeroed one of the size the plan
    needs for this call."""
    dtype, ptrs, (H, KV, N, D), out = _attention_args(q, k, v, bits, group_size, out, stream)
    if workspace is None:
        n = aq_attention_workspace_bytes(H, KV, N, D, bits, group_size)
        workspace = _on(_side(stream, q.device), q.device,  # zeroed in the call's order
                        lambda: torch.zeros(max(n, 1), dtype=torch.uint8, device=q.device))
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _check(load().aq_attention_decode_ws(dtype, *ptrs, H, KV, N, D, bits, group_size,
                                         _dev(out, "out"), _dev(workspace, "workspace"),
                                         workspace.numel(), _stream(stream)),
           "aq_attention_decode_ws")
    return out


def aq_quantize_ex(w: torch.Tensor, bits: int, group_size: int, stream=None) -> tuple:
    """aq_quantize for any code width and group size; w fp16 or bf16 [N, K]."""
    dtype = AQ_BF16 if w.dtype == torch.bfloat16 else AQ_F16
    N, K = w.shape
    Wq = _empty((N, K * bits // 32), torch.int32, w.device, stream)
    scales = _empty((N, K // group_size), torch.float16, w.device, stream)
    biases = _empty((N, K // group_size), torch.float16, w.device, stream)
    _check(load().aq_quantize_ex(dtype, _dev(w, "w"), N, K, bits, group_size, _dev(Wq, "Wq"),
                                 _dev(scales, "scales"), _dev(biases, "biases"), _stream(stream)),
           "aq_quantize_ex")
    return Wq, scales, biases


class _CacheStruct(ctypes.Structure):
    _fields_ = [("pool_dev", ctypes.c_void_p), ("layers", ctypes.c_int64),
                ("n_pages", ctypes.c_int64), ("KV", ctypes.c_int64), ("D", ctypes.c_int64),
                ("page", ctypes.c_int), ("bits", ctypes.c_int), ("group_size", ctypes.c_int)]


class AqCache:
    """A paged KV cache (struct aq_cache): pool is a uint8 device tensor
    [layers, n_pages, KV, record], record = aq_cache_record_bytes(head_dim,
    page, bits, group_size).  The tensor stays the caller's; this object only
    names its geometry and may be made anew for every call."""

    __slots__ = ("pool", "page", "head_dim", "bits", "group_size", "layers", "n_pages", "kv_heads",
                 "_struct", "_ref")

    def __init__(self, pool: torch.Tensor, page: int, head_dim: int, bits: int, group_size: int):
        shape = pool.shape
        if pool.dtype != torch.uint8 or len(shape) != 4:
            raise ValueError("pool must be uint8 [layers, n_pages, KV, record]")
        want = aq_cache_record_bytes(head_dim, page, bits, group_size)
        if want == 0:
            raise ValueError("head_dim 64/128/256/512, page 16/32/64/128, bits 4/8 and group_size "
                             "32/64/128 are served")
        if shape[3] != want:
            raise ValueError(f"pool's records hold {shape[3]} bytes; this geometry uses {want}")
        self.pool, self.page, self.head_dim = pool, page, head_dim
        self.bits, self.group_size = bits, group_size
        self.layers, self.n_pages, self.kv_heads = shape[0], shape[1], shape[2]
        self._struct = _CacheStruct(_dev(pool, "pool"), shape[0], shape[1], shape[2], head_dim, page,
                                    bits, group_size)
        self._ref = ctypes.addressof(self._struct)

    @staticmethod
    def empty(layers: int, n_pages: int, kv_heads: int, head_dim: int, page: int, bits: int,
              group_size: int, device="cuda") -> "AqCache":
        """A cache over a pool allocated here (its pages need no initial value)."""
        rec = aq_cache_record_bytes(head_dim, page, bits, group_size)
        pool = torch.empty((layers, n_pages, kv_heads, rec), dtype=torch.uint8, device=device)
        return AqCache(pool, page, head_dim, bits, group_size)


@functools.lru_cache(maxsize=256)
def aq_cache_record_bytes(D: int, page: int, bits: int, group_size: int) -> int:
    """Bytes of one page's record of one KV head (0: sizes not served)."""
    return int(load().aq_cache_record_bytes(D, page, bits, group_size))


@functools.lru_cache(maxsize=256)
def aq_cache_workspace_bytes(n_pages: int, B: int) -> int:
    """Workspace bytes of aq_cache_grow and aq_cache_compact."""
    return int(load().aq_cache_workspace_bytes(n_pages, B))


_I32, _F32 = torch.int32, torch.float32


def _ints(t: torch.Tensor, name: str, *shape) -> int:
    """The address of a dense int32 device tensor of this shape."""
    if t.dtype is not _I32 or t.shape != shape:
        raise ValueError(f"{name} must be int32 {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        return _dev(t, name)  # says which
    return t.data_ptr()


def _table_shape(table: torch.Tensor) -> tuple:
    if table.dim() != 2:
        raise ValueError("table must be [B, max_pages]")
    return tuple(table.shape)


def _token_rows(t: torch.Tensor, name: str, heads: int, D: int) -> tuple:
    """(address, elements between tokens) of [T, heads, D] with dense heads."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != D:
        raise ValueError(f"{name} must be [T, {heads}, {D}], got {list(t.shape)}")
    if t.numel() and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != D)):
        raise ValueError(f"{name}: a token's heads must be dense")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else heads * D


def aq_cache_append(cache: AqCache, layer: int, k, v, cu, start, table, stream=None) -> None:
    """Quantise the rows k, v [T, KV, D] (fp16 or bf16; a slice of a fused
    projection's output will do) into their pages: tokens cu[b] .. cu[b+1]-1
    go to row b from position start[b] on.  cu int32 [B + 1], start int32 [B],
    table int32 [B, max_pages]."""
    if k.dtype not in _ACT or v.dtype != k.dtype:
        raise ValueError("k and v must both be float16 or both bfloat16")
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    B, width = _table_shape(table)
    kp, ks = _token_rows(k, "k", cache.kv_heads, cache.head_dim)
    vp, vs = _token_rows(v, "v", cache.kv_heads, cache.head_dim)
    _check(load().aq_cache_append(cache._ref, layer, AQ_BF16 if k.dtype == torch.bfloat16 else AQ_F16,
                                  kp, ks, vp, vs, k.shape[0], _ints(cu, "cu", B + 1),
                                  _ints(start, "start", B), _ints(table, "table", B, width), B,
                                  width, _stream(stream)), "aq_cache_append")


def aq_cache_read(cache: AqCache, layer: int, cu, start, table, total: int, dtype, out=None,
                  stream=None) -> tuple:
    """The cached rows of the same tokens as floats: (k, v), each
    [total, KV, D] of dtype (zeros for tokens outside every sequence)."""
    if dtype not in _ACT:
        raise ValueError("dtype must be float16 or bfloat16")
    B, width = _table_shape(table)
    shape = (total, cache.kv_heads, cache.head_dim)
    if out is None:
        if total < 0:
            raise ValueError("total must not be negative")
        k, v = (_empty(shape, dtype, cache.pool.device, stream) for _ in range(2))
        kp, vp = k.data_ptr(), v.data_ptr()
    else:
        k, v = out
        for name, t in (("k", k), ("v", v)):
            if t.dtype != dtype or tuple(t.shape) != shape:
                raise ValueError(f"out {name} must be {dtype} {list(shape)}")
        kp, vp = _dev(k, "out k"), _dev(v, "out v")
    st = load().aq_cache_read(cache._ref, layer, AQ_BF16 if dtype is torch.bfloat16 else AQ_F16, kp, vp,
                              total, _ints(cu, "cu", B + 1), _ints(start, "start", B),
                              _ints(table, "table", B, width), B, width, _stream(stream))
    if st:
        _check(st, "aq_cache_read")
    return k, v


def aq_cache_copy(cache: AqCache, src, dst, stream=None) -> None:
    """Page src[i] onto page dst[i] in every layer; src, dst int32 [n]."""
    n = src.numel()
    _check(load().aq_cache_copy(cache._ref, _ints(src, "src", n), _ints(dst, "dst", n), n,
                                _stream(stream)), "aq_cache_copy")


def _tables(f, cache, refs, table, lens, args, in_place, out, workspace, stream, with_lens=True):
    """Calls a page-table operation f: the checks and the outputs that they
    share.  args: (name, tensor) of its other inputs; workspace: None where it
    takes none, else a list with the caller's tensor or None."""
    B, width = _table_shape(table)
    r, t, n = (_ints(refs, "refs", cache.n_pages), _ints(table, "table", B, width),
               _ints(lens, "lens", B))
    more = [_ints(x, name, B) for name, x in args]
    status = _empty(4, _I32, refs.device, stream)
    if out is None and in_place:
        res, outs = [refs, table, lens], [r, t, n]
    elif out is None:
        res = [_empty(x.shape, _I32, refs.device, stream)
               for x in ((refs, table, lens) if with_lens else (refs, table))]
        outs = [o.data_ptr() for o in res]
    else:
        res = list(out)
        given = (refs, table, lens) if with_lens else (refs, table)
        if len(res) != len(given):
            raise ValueError(f"out must be {len(given)} tensors")
        outs = [_ints(o, f"out[{i}]", *g.shape) for i, (o, g) in enumerate(zip(res, given))]
    if not with_lens:
        del res[2:], outs[2:]
    if workspace is None:
        st = f(cache._ref, r, t, n, *more, B, width, *outs, status.data_ptr(), _stream(stream))
    else:
        ws = workspace[0]
        if ws is None:
            ws = _scratch(aq_cache_workspace_bytes(cache.n_pages, B), cache.pool.device, stream)
        if ws.dtype != torch.uint8:
            raise ValueError("workspace must be a contiguous uint8 tensor")
        st = f(cache._ref, r, t, n, *more, B, width, *outs, status.data_ptr(),
               _dev(ws, "workspace"), ws.numel(), _stream(stream))
    if st:
        _check(st, f.__name__)
    res.append(status)
    return tuple(res)


def aq_cache_fork(cache, refs, table, lens, parent, keep, in_place=True, out=None,
                  stream=None) -> tuple:
    """Row b with parent[b] >= 0 becomes a copy of that row's first keep[b]
    tokens (keep[b] < 0: all).  refs int32 [n_pages], table int32
    [B, max_pages], lens, parent, keep int32 [B].  Returns (refs, table, lens,
    status): the same tensors, or new ones with in_place=False (or out)."""
    return _tables(load().aq_cache_fork, cache, refs, table, lens,
                   (("parent", parent), ("keep", keep)), in_place, out, None, stream)


def aq_cache_trim(cache, refs, table, lens, keep, in_place=True, out=None, stream=None) -> tuple:
    """Row b with 0 <= keep[b] < lens[b] is cut to keep[b] tokens (0 frees
    it).  Arguments and results as aq_cache_fork."""
    return _tables(load().aq_cache_trim, cache, refs, table, lens, (("keep", keep),), in_place, out,
                   None, stream)


def aq_cache_grow(cache, refs, table, lens, add, in_place=True, out=None, workspace=None,
                  stream=None) -> tuple:
    """Pages for add[b] more tokens of every row, with copy on write of shared
    partial pages.  Arguments and results as aq_cache_fork."""
    return _tables(load().aq_cache_grow, cache, refs, table, lens, (("add", add),), in_place, out,
                   [workspace], stream)


def aq_cache_compact(cache, refs, table, lens, in_place=True, out=None, workspace=None,
                     stream=None) -> tuple:
    """Moves the live pages to the front of the pool.  Returns (refs, table,
    status); lens is only read."""
    return _tables(load().aq_cache_compact, cache, refs, table, lens, (), in_place, out, [workspace],
                   stream, False)


@functools.lru_cache(maxsize=1024)
def _batch_workspace(device: int, n_pages: int, KV: int, D: int, page: int, bits: int, group_size: int,
                     B: int, L: int, H: int, G: int) -> int:
    # a function of sizes and of the device's SMs only; the pool is not read
    c = _CacheStruct(256, 1, n_pages, KV, D, page, bits, group_size)
    return int(load().aq_attention_batch_workspace_bytes(ctypes.addressof(c), B, L, H, G))


def aq_attention_batch_workspace_bytes(cache: AqCache, B: int, L: int, H: int, G: int = 0) -> int:
    """Workspace bytes of aq_attention_batch (0: sizes that it refuses)."""
    return _batch_workspace(cache.pool.get_device(), cache.n_pages, cache.kv_heads, cache.head_dim,
                            cache.page, cache.bits, cache.group_size, B, L, H, G)


def aq_attention_batch(q, cache: AqCache, layer: int, table, lens, scale: float, group_start=None,
                       shared=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of the last L tokens of each of B sequences over one layer of
    the paged cache, the keys that a group of sequences shares read once.
    q [B, L, H, D] (fp16 or bf16, a token's heads dense); table int32
    [B, max_pages]; lens int32 [B] counts the L new tokens; group_start int32
    [G + 1] and shared int32 [G] name the groups and how many first tokens
    each shares.  Returns o [B, L, H, D] in q's dtype."""
    if q.dtype not in _ACT:
        raise ValueError("q must be float16 or bfloat16")
    if q.dim() != 4 or q.shape[3] != cache.head_dim:
        raise ValueError(f"q must be [B, L, H, {cache.head_dim}], got {list(q.shape)}")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    B, L, H, D = q.shape
    step = H * D
    stride = step
    if not q.is_contiguous():
        sb, sl, sh, sd = q.stride()
        if B * L > 1:
            stride = sl if L > 1 else sb
        if (L > 1 and B > 1 and sb != L * stride) or sd != 1 or (H > 1 and sh != D):
            raise ValueError("q: a token's heads must be dense, and tokens a fixed step apart")
    rows, width = _table_shape(table)
    if rows != B:
        raise ValueError(f"table has {rows} rows for {B} sequences")
    G = 0
    gs = sh = None
    if shared is not None and group_start is not None:
        G = shared.numel()
        gs, sh = _ints(group_start, "group_start", G + 1), _ints(shared, "shared", G)
    elif shared is not None or group_start is not None:
        raise ValueError("group_start and shared go together")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
        to = out.data_ptr()
    else:
        _check_out(out, "out", B * L * step, q.dtype)
        to = _dev(out, "out")
    if workspace is None:
        n = aq_attention_batch_workspace_bytes(cache, B, L, H, G)
        n = n or 256  # so that refused sizes reach the library's checks
        workspace = _scratch(n, q.device, stream)
        ws = workspace.data_ptr()
    else:
        if workspace.dtype != torch.uint8:
            raise ValueError("workspace must be a contiguous uint8 tensor")
        n, ws = workspace.numel(), _dev(workspace, "workspace")
    st = load().aq_attention_batch(cache._ref, layer, AQ_F16 if q.dtype is torch.float16 else AQ_BF16,
                                   q.data_ptr(), stride, _ints(table, "table", B, width),
                                   _ints(lens, "lens", B), gs, sh, B, L, H, G, width, scale, to, ws,
                                   n, _stream(stream))
    if st:
        _check(st, "aq_attention_batch")
    return out


class _RouterStruct(ctypes.Structure):
    _fields_ = [("weight_dev", ctypes.c_void_p), ("bias_dev", ctypes.c_void_p),
                ("E", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("top_k", ctypes.c_int), ("score", ctypes.c_int), ("normalize", ctypes.c_int),
                ("scale", ctypes.c_float)]


class _ExpertsStruct(ctypes.Structure):
    _fields_ = [(f"{m}_{part}_dev", ctypes.c_void_p) for m in ("gate", "up", "down")
                for part in ("words", "scales", "biases")] + \
               [("E", ctypes.c_int64), ("K", ctypes.c_int64), ("I", ctypes.c_int64),
                ("bits", ctypes.c_int), ("group_size", ctypes.c_int)]


_SCORES = {"softmax": AQ_SCORE_SOFTMAX, "sigmoid": AQ_SCORE_SIGMOID}


class _Fixed:
    """An object whose attributes are those its struct was made of: the library
    reads the struct, the binding's checks the attributes.  (What a subclass adds
    is its own.)"""

    __slots__ = ()
    _names = frozenset()

    def _fix(self, **kw):
        for name, value in kw.items():
            object.__setattr__(self, name, value)

    def _check_name(self, name):
        if name in self._names:
            raise AttributeError(f"{name} is fixed: make another {type(self).__name__}")

    def __setattr__(self, name, value):
        self._check_name(name)
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        self._check_name(name)
        object.__delattr__(self, name)

    def __copy__(self):
        return self


class AqRouter(_Fixed):
    """A router (struct aq_router): weight [E, K] fp16 or bf16, bias float32
    [E] or None (sigmoid scores only), score "softmax" or "sigmoid".  The
    tensors stay the caller's; this object holds them and is kept for a layer.
    Its attributes do not change."""

    __slots__ = ("weight", "bias", "top_k", "_struct", "_ref", "_index", "_dtype", "_shape")
    _names = frozenset(__slots__)

    def __init__(self, weight, top_k: int, bias=None, score: str = "softmax",
                 normalize: bool = True, scale: float = 1.0):
        if weight.dtype not in _ACT or weight.dim() != 2:
            raise ValueError("weight must be float16 or bfloat16 [E, K]")
        if score not in _SCORES:
            raise ValueError(f"score must be one of {sorted(_SCORES)}")
        E, K = weight.shape
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (E,)):
            raise ValueError(f"bias must be float32 [{E}]")
        if bias is not None and bias.device != weight.device:
            raise ValueError("bias must be on weight's device")
        struct = _RouterStruct(_dev(weight, "weight"), None if bias is None else _dev(bias, "bias"), E, K,
                               AQ_BF16 if weight.dtype == torch.bfloat16 else AQ_F16, top_k,
                               _SCORES[score], int(normalize), scale)
        self._fix(weight=weight, bias=bias, top_k=top_k, _index=weight.get_device(), _dtype=weight.dtype,
                  _shape=(E, K), _struct=struct, _ref=ctypes.addressof(struct))


class AqExperts(_Fixed):
    """The experts of a layer (struct aq_experts): gate and up are (words
    [E, I, K*bits/32] int32, scales [E, I, K/group] fp16, biases), down the
    same with [E, K, I]; bits 2/3/4/5/6/8, groups of 32/64/128.  The tensors
    stay the caller's; this object holds them and is kept for a layer.  Its
    attributes do not change."""

    __slots__ = ("gate", "up", "down", "bits", "group_size", "count", "hidden", "inner", "_struct",
                 "_ref", "_workspaces", "_index")
    _names = frozenset(__slots__)

    def __init__(self, gate, up, down, bits: int, group_size: int):
        if bits not in (2, 3, 4, 5, 6, 8) or group_size not in (32, 64, 128):
            raise ValueError("bits 2/3/4/5/6/8 and group_size 32/64/128 are served")
        if any(t.dim() != 3 for m in (gate, up, down) for t in m):
            raise ValueError("gate, up and down must be (words, scales, biases), each [E, rows, ...]")
        E, inner, hidden = gate[1].shape[0], gate[1].shape[1], down[1].shape[1]
        if hidden % group_size or inner % group_size or hidden % 64 or inner % 64:
            raise ValueError(f"hidden and inner size must be multiples of 64 and of the group size, "
                             f"got {hidden} and {inner}")
        parts = []
        for name, m, rows, cols in (("gate", gate, inner, hidden), ("up", up, inner, hidden),
                                    ("down", down, hidden, inner)):
            for part, t, last in (("words", m[0], cols * bits // 32),
                                  ("scales", m[1], cols // group_size),
                                  ("biases", m[2], cols // group_size)):
                if tuple(t.shape) != (E, rows, last):
                    raise ValueError(f"{name} {part} must be {[E, rows, last]}, got {list(t.shape)}")
                if part != "words" and t.dtype != torch.float16:
                    raise ValueError(f"{name} {part} must be {torch.float16}, got {t.dtype}")
                if part == "words" and t.element_size() != 4:
                    raise ValueError(f"{name} words must be of 32 bits, got {t.dtype}")
                if t.device != gate[0].device:
                    raise ValueError("gate, up and down must be on one device")
                parts.append((t, f"{name} {part}"))
        struct = _ExpertsStruct(*(_dev(t, name) for t, name in parts), E, hidden, inner, bits, group_size)
        self._fix(gate=tuple(gate), up=tuple(up), down=tuple(down), bits=bits, group_size=group_size, count=E,
                  hidden=hidden, inner=inner, _index=gate[0].get_device(), _struct=struct,
                  _ref=ctypes.addressof(struct), _workspaces={})


def _moe_tokens(x, K: int, index: int, dtype=None) -> int:
    """Checks x [T, K] on the weights' device; returns T."""
    if x.dtype not in _ACT or (dtype is not None and x.dtype is not dtype):
        raise ValueError(f"x must be {dtype or 'float16 or bfloat16'}, got {x.dtype}")
    shape = x.shape
    if len(shape) != 2 or shape[1] != K:
        raise ValueError(f"x must be [T, {K}], got {list(shape)}")
    if x.get_device() != index:
        raise ValueError("x must be on the weights' device")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return shape[0]


def _moe_given(t, name: str, dtype, T: int, top_k: int, index: int) -> int:
    """The address of the experts' ids or weights, [T, top_k]."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (T, top_k):
        raise ValueError(f"{name} must be {[T, top_k]}, got {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on x's device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _moe_pair(routed, T: int, top_k: int, x, stream) -> tuple:
    if routed is None:
        shape, dev = (T, top_k), x.device
        if stream is None:
            ids, weights = torch.empty(shape, dtype=_I32, device=dev), torch.empty(shape, dtype=_F32, device=dev)
        else:
            ids, weights = _empty(shape, _I32, dev, stream), _empty(shape, _F32, dev, stream)
        return ids, weights, ids.data_ptr(), weights.data_ptr()
    ids, weights = routed
    index = x.get_device()
    return (ids, weights, _moe_given(ids, "experts", _I32, T, top_k, index),
            _moe_given(weights, "weights", _F32, T, top_k, index))


def _moe_out(x, out, workspace, experts: AqExperts, T: int, top_k: int, stream) -> tuple:
    if out is None:
        out = torch.empty_like(x) if stream is None else _empty(x.shape, x.dtype, x.device, stream)
        to = out.data_ptr()
    else:
        if out.shape != x.shape or out.get_device() != x.get_device():
            raise ValueError(f"out must be {list(x.shape)} on x's device")
        _check_out(out, "out", x.numel(), x.dtype)
        to = _dev(out, "out")
    if workspace is None:
        # refused sizes reach the library's checks
        n = aq_moe_workspace_bytes(experts, T, top_k) or 256
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device) if stream is None else \
            _scratch(n, x.device, stream)
        return out, to, workspace.data_ptr(), n, workspace
    if workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a contiguous uint8 tensor")
    if workspace.get_device() != x.get_device():
        raise ValueError("workspace must be on x's device")
    return out, to, _dev(workspace, "workspace"), workspace.numel(), workspace


def aq_moe_workspace_bytes(experts: AqExperts, T: int, top_k: int) -> int:
    """Workspace bytes of aq_moe and aq_moe_experts (0: sizes that they refuse)."""
    n = experts._workspaces.get((T, top_k))
    if n is None:
        n = int(load().aq_moe_workspace_bytes(experts._ref, T, top_k))
        experts._workspaces[(T, top_k)] = n
    return n


def aq_moe_route(x, router: AqRouter, out=None,
                 stream: Union[torch.cuda.Stream, int, None] = None) -> tuple:
    """The experts of each token of x [T, K]: (experts int32 [T, top_k], each
    row ascending, weights float32 [T, top_k])."""
    T = _moe_tokens(x, router._shape[1], router._index, router._dtype)
    ids, weights, ip, wp = _moe_pair(out, T, router.top_k, x, stream)
    st = load().aq_moe_route(router._ref, x.data_ptr(), T, ip, wp, _stream(stream))
    if st:
        _check(st, "aq_moe_route")
    return ids, weights


def aq_moe_experts(x, experts: AqExperts, ids, weights, out=None, workspace=None,
                   stream: Union[torch.cuda.Stream, int, None] = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * expert ids[t, j] of x[t]; ids int32
    [T, top_k] (outside 0..E-1: none), weights float32 [T, top_k]."""
    index = experts._index
    T = _moe_tokens(x, experts.hidden, index)
    if ids.dim() != 2:
        raise ValueError("experts must be [T, top_k]")
    top_k = ids.shape[1]
    ip = _moe_given(ids, "experts", _I32, T, top_k, index)
    wp = _moe_given(weights, "weights", _F32, T, top_k, index)
    out, op, ws, n, hold = _moe_out(x, out, workspace, experts, T, top_k, stream)
    st = load().aq_moe_experts(experts._ref, AQ_BF16 if x.dtype is torch.bfloat16 else AQ_F16,
                             x.data_ptr(), T, top_k, ip, wp, op, ws, n, _stream(stream))
    if st:
        _check(st, "aq_moe_experts")
    return out


def aq_moe(x, router: AqRouter, experts: AqExperts, out=None, routed=None, workspace=None,
           stream: Union[torch.cuda.Stream, int, None] = None) -> tuple:
    """The whole layer: routes x [T, K] and runs the chosen experts.  Returns
    (y [T, K], experts int32 [T, top_k], weights float32 [T, top_k]); routed:
    tensors for the last two."""
    T = _moe_tokens(x, experts.hidden, experts._index, router._dtype)
    if router._shape != (experts.count, experts.hidden):
        raise ValueError(f"the router is {list(router._shape)}, the experts "
                         f"{[experts.count, experts.hidden]}")
    if router._index != experts._index:
        raise ValueError("router and experts must be on one device")
    ids, weights, ip, wp = _moe_pair(routed, T, router.top_k, x, stream)
    out, op, ws, n, hold = _moe_out(x, out, workspace, experts, T, router.top_k, stream)
    st = load().aq_moe(router._ref, experts._ref, x.data_ptr(), T, ip, wp, op, ws, n, _stream(stream))
    if st:
        _check(st, "aq_moe")
    return out, ids, weights


def aq_embed(ids, Wq, scales, biases, bits: int, group_size: int, dtype, scale: float = 1.0,
             out=None, stream: Union[torch.cuda.Stream, int, None] = None) -> torch.Tensor:
    """Rows of a quantised table by token: scale * row ids[...] as dtype (fp16
    or bf16) [..., K]; ids int32 or int64, outside 0..N-1 a row of zeros.  Wq
    [N, K*bits/32], scales and biases fp16 [N, K/group_size]."""
    if dtype not in _ACT:
        raise ValueError("dtype must be float16 or bfloat16")
    wide = ids.dtype is torch.int64
    if not wide and ids.dtype is not _I32:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    shape = scales.shape
    if len(shape) != 2:
        raise ValueError("scales must be [N, K/group_size]")
    N, K = shape[0], shape[1] * group_size
    if Wq.numel() * Wq.element_size() * 8 != N * K * bits or biases.shape != shape or \
            scales.dtype is not torch.float16 or biases.dtype is not torch.float16:
        _check_weights(Wq, scales, biases, N, K, bits, group_size)  # says which
        if biases.shape != shape:
            raise ValueError(f"biases must be {list(shape)}, got {list(biases.shape)}")
    index = ids.get_device()
    if index < 0:
        raise ValueError("ids must be a CUDA tensor")
    if Wq.get_device() != index or scales.get_device() != index or biases.get_device() != index:
        raise ValueError("ids and the table must be on one device")
    if not (ids.is_contiguous() and Wq.is_contiguous() and scales.is_contiguous() and biases.is_contiguous()):
        raise ValueError("ids and the table must be contiguous")
    T = ids.numel()
    if out is None:
        shape = (*ids.shape, K)
        out = torch.empty(shape, dtype=dtype, device=ids.device) if stream is None else \
            _empty(shape, dtype, ids.device, stream)
    else:
        if out.get_device() != index:
            raise ValueError("out must be on ids' device")
        _check_out(out, "out", T * K, dtype)
        _dev(out, "out")
    st = load().aq_embed(AQ_BF16 if dtype is torch.bfloat16 else AQ_F16, ids.data_ptr(), 8 if wide else 4, T,
                       Wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), N, K, bits, group_size, scale,
                       out.data_ptr(), _stream(stream))
    if st:
        _check(st, "aq_embed")
    return out


def aq_matmul_multi(x, weights, bits, outs=None, stream=None) -> list:
    """Several projections of the same x in one call: weights is a list of
    (Wq, scales, biases) triples (1..4); returns [y_j] in x's dtype."""
    dtype = AQ_BF16 if x.dtype == torch.bfloat16 else AQ_F16
    P = len(weights)
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    Ns = [w[1].shape[0] for w in weights]
    if bits in (3, 4):
        for j, (w, n) in enumerate(zip(weights, Ns)):
            _check_weights(w[0], w[1], w[2], n, K, bits, 64, f"[{j}]")
    if outs is None:
        outs = [_empty((*x.shape[:-1], n), x.dtype, x.device, stream) for n in Ns]
    if len(outs) != P:
        raise ValueError("one output per projection")
    for j, (o, n) in enumerate(zip(outs, Ns)):
        _check_out(o, f"outs[{j}]", M * n, x.dtype)
    ptr_arr = ctypes.c_void_p * max(P, 1)
    Wp = ptr_arr(*[_dev(w[0], "Wq") for w in weights])
    Sp = ptr_arr(*[_dev(w[1], "scales") for w in weights])
    Bp = ptr_arr(*[_dev(w[2], "biases") for w in weights])
    Op = ptr_arr(*[_dev(o, "out") for o in outs])
    Na = (ctypes.c_int64 * max(P, 1))(*Ns)
    _check(load().aq_matmul_multi(dtype, _dev(x, "x"), P, ctypes.cast(Wp, ctypes.c_void_p),
                                  ctypes.cast(Sp, ctypes.c_void_p), ctypes.cast(Bp, ctypes.c_void_p),
                                  ctypes.cast(Na, ctypes.c_void_p), M, K, bits,
                                  ctypes.cast(Op, ctypes.c_void_p), _stream(stream)),
           "aq_matmul_multi")
    return outs


def aq_matmul_gate_up(x, gate, up, bits, out=None, stream=None) -> torch.Tensor:
    """h = silu(x . W_gate^T) * (x . W_up^T); gate and up are (Wq, scales,
    biases) triples with the same N."""
    dtype = AQ_BF16 if x.dtype == torch.bfloat16 else AQ_F16
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    N = gate[1].shape[0]
    if bits in (3, 4):
        _check_weights(gate[0], gate[1], gate[2], N, K, bits, 64, " (gate)")
        _check_weights(up[0], up[1], up[2], N, K, bits, 64, " (up)")
    if out is None:
        out = _empty((*x.shape[:-1], N), x.dtype, x.device, stream)
    _check_out(out, "out", M * N, x.dtype)
    _check(load().aq_matmul_gate_up(dtype, _dev(x, "x"), _dev(gate[0], "Wq"),
                                    _dev(gate[1], "scales"), _dev(gate[2], "biases"),
                                    _dev(up[0], "Wq"), _dev(up[1], "scales"),
                                    _dev(up[2], "biases"), M, N, K, bits, _dev(out, "out"),
                                    _stream(stream)), "aq_matmul_gate_up")
    return out


def aq_matmul_variant(variant, x, Wq, scales, biases, bits, out=None, stream=None):
    """Explicit kernel variant; the dtype follows x (fp16 or bf16)."""
    dtype = AQ_BF16 if x.dtype == torch.bfloat16 else AQ_F16
    return _mm(variant, dtype, x, Wq, scales, biases, bits, out, stream)


def aq_matmul_host(x_host: torch.Tensor, Wq, scales, biases, bits, out_host: torch.Tensor,
                   x_dev: torch.Tensor, out_dev: torch.Tensor, stream=None) -> torch.Tensor:
    """Host x in, host y out (device staging buffers supplied); synchronises."""
    dtype = AQ_BF16 if x_host.dtype == torch.bfloat16 else AQ_F16
    if x_host.is_cuda or out_host.is_cuda:
        raise ValueError("x_host and out_host must be host tensors")
    K = x_host.shape[-1]
    M = x_host.numel() // K
    N = scales.shape[0]
    if bits in (3, 4):
        _check_weights(Wq, scales, biases, N, K, bits, 64)
    _check_out(out_host, "out_host", M * N, x_host.dtype)
    _check_out(x_dev, "x_dev", M * K, x_host.dtype)
    _check_out(out_dev, "out_dev", M * N, x_host.dtype)
    _check(load().aq_matmul_host(dtype, x_host.data_ptr(), _dev(Wq, "Wq"),
                                 _dev(scales, "scales"), _dev(biases, "biases"), M, N, K, bits,
                                 out_host.data_ptr(), _dev(x_dev, "x_dev"),
                                 _dev(out_dev, "out_dev"), _stream(stream)), "aq_matmul_host")
    return out_host


def aq_select(M: int, N: int, K: int, bits: int, dtype: int = AQ_F16) -> int:
    return load().aq_select(M, N, K, bits, dtype)


def aq_describe(M: int, N: int, K: int, bits: int, dtype: int = AQ_F16) -> str:
    buf = ctypes.create_string_buffer(256)
    load().aq_describe(M, N, K, bits, dtype, ctypes.addressof(buf), 256)
    return buf.value.decode()


def aq_attention_describe(H: int, KV: int, N: int, D: int, bits: int, group_size: int) -> str:
    """The launch geometry of aq_attention_decode for these sizes (needs the
    device for its count of co-resident clusters)."""
    buf = ctypes.create_string_buffer(256)
    load().aq_attention_describe(H, KV, N, D, bits, group_size, ctypes.addressof(buf), 256)
    return buf.value.decode()


def aq_attention_describe_ws(H: int, KV: int, N: int, D: int, bits: int, group_size: int,
                             workspace_bytes: int) -> str:
    """The launch geometry of aq_attention_decode_ws with a workspace of
    workspace_bytes."""
    buf = ctypes.create_string_buffer(256)
    load().aq_attention_describe_ws(H, KV, N, D, bits, group_size, workspace_bytes,
                                    ctypes.addressof(buf), 256)
    return buf.value.decode()


def aq_stats(reset: bool = False) -> List[int]:
    """Calls per variant (aq_stats); reset=True also calls aq_stats_reset."""
    buf = (ctypes.c_uint64 * AQ_NUM_VARIANTS)()
    _check(load().aq_stats(ctypes.cast(buf, ctypes.c_void_p), AQ_NUM_VARIANTS), "aq_stats")
    if reset:
        aq_stats_reset()
    return list(buf)


def aq_stats_reset() -> None:
    load().aq_stats_reset()


def aq_device_error(clear: bool = False) -> int:
    code = ctypes.c_uint32(0)
    _check(load().aq_device_error(ctypes.addressof(code), int(clear)), "aq_device_error")
    return code.value


def aq_free() -> None:
    load().aq_free()


load()
