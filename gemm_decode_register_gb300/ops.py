"""Python binding of the C ABI in include/mx.h (argument marshalling only).

Each function takes torch CUDA tensors, passes their device pointers and
the current torch stream to libmxgemm.so, and raises MxError on a non-zero
status.  Every step of the computation runs in the library's kernels; there
is no fallback path: if the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import threading
from typing import NamedTuple

import torch

from .synth import FMT_MXFP4, FMT_MXFP8, FMT_NVFP4, block_of  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmxgemm.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "mx.h")

_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


class MxError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libmxgemm.so (built by ``gemm_decode_register_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} is missing "
                               "(run __graft_entry__.build() or python -m "
                               "gemm_decode_register_gb300.build)")
        lib = ctypes.CDLL(p)
        P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        sig = {
            "mx_qmv": [I, P, P, P, P, I, I, I],
            "mx_qmv_noalloc": [I, P, P, P, P, I, I, I],
            "mx_moe_qmv": [I, P, P, P, P, P, I, I, I, I, I],
            "mx_moe_gate_up_swiglu": [I, P, P, P, P, P, I, I, I, I, I],
            "mx_moe_down_combine": [I, P, P, P, P, P, P, I, I, I, I, I],
            "mx_qmm": [I, P, P, P, P, I, I, I],
            "mx_set_stream": [P],
            "mx_dequant": [I, P, P, P, I, I],
            "mx_swiglu": [P, P, I, I],
            "mx_moe_combine": [P, P, P, I, I, I],
            "mx_device_error": [],
            "mx_debug_qmm_stall": [I, ctypes.c_ulonglong],
            "mx_qmm_qx": [I, P, P, P, P, P, I, I, I],
            "mx_mma_peak": [I, I, P],
            "mx_moe_qmm": [I, P, P, P, P, P, I, I, I, I, I, P, Z],
            "mx_quantize": [I, P, P, P, I, I],
            "mx_moe_ffn_prefill": [I, P, P, P, P, P, P, P, P, I, I, I, I, I, P, Z],
            "mx_rope_table": [P, ctypes.c_double, P, L, I, I],
            "mx_rope": [P, P, I, P, P, I, I, I, I, I, L, L, L, L, I],
            "mx_kv_append": [P, P, I, L, P, P, P, I, I, P, I, I, I, I],
            "mx_paged_attn": [P, P, L, L, P, P, ctypes.c_float, I, I, P, P, P, I, I, I, P, Z],
            "mx_beam_select": [P, I, L, P, P, L, I, I, I, I, I, P, P, P, P, P, P, P, Z],
            "mx_kv_remap": [P, I, P, I, I, P, I, P, I, I, P, I, P, P, P, I, P],
            "mx_kv_compact": [P, I, P, I, I, P, I, P],
            "mx_kv_copy_pages": [P, I, P, I],
            "mx_i8_quantize": [P, I, P, P, I, I],
            "mx_i8_mm": [P, I, P, P, P, P, I, I, I, I, P, Z],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = I
        for name, args in {"mx_moe_qmm_workspace_size": [I, I, I, I],
                           "mx_moe_ffn_prefill_workspace_size": [I, I, I, I, I],
                           "mx_paged_attn_workspace_size": [I, I, I, I, I],
                           "mx_beam_select_workspace_size": [I, I, I, I],
                           "mx_page_pool_work_size": [I],
                           "mx_i8_mm_workspace_size": [I, I]}.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = Z
        lib.mx_strerror.argtypes = [I]
        lib.mx_strerror.restype = ctypes.c_char_p
        _lib = lib
        return lib


def header_symbols() -> list[str]:
    """Names of the functions include/mx.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^\s*(?:const\s+char\s*\*|int|size_t)\s*(mx_\w+)\s*\(", text, flags=re.M)


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MxError(fn, status, load().mx_strerror(status).decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (3 us of a small call's 13): torch's own accessors where
# they exist.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream() -> None:
    if _raw_stream is not None and _raw_device is not None:
        load().mx_set_stream(_raw_stream(_raw_device()))
    else:
        load().mx_set_stream(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


def qmv(fmt: int, codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, N: int,
        y: torch.Tensor | None = None) -> torch.Tensor:
    """y[M][N] fp32 = x (bf16 [M][K]) . W^T, W block-float [N][K]."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _stream()
    _check("mx_qmv", load().mx_qmv(fmt, _ptr(codes), _ptr(scales), _ptr(x), _ptr(y), M, N, K))
    return y


def qmv_noalloc(fmt: int, codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, N: int,
                y: torch.Tensor | None = None) -> torch.Tensor:
    """mx_qmv_noalloc: the same product, with no device allocation."""
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _stream()
    _check("mx_qmv_noalloc", load().mx_qmv_noalloc(fmt, _ptr(codes), _ptr(scales), _ptr(x), _ptr(y), M, N, K))
    return y


def moe_qmv(fmt: int, codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
            expert_ids: torch.Tensor, E: int, N: int, y: torch.Tensor | None = None) -> torch.Tensor:
    """y[T][topk][N] fp32 over the routed experts of each token."""
    T, K = x.shape
    topk = expert_ids.shape[1]
    if y is None:
        y = torch.empty((T, topk, N), dtype=torch.float32, device=x.device)
    _stream()
    _check("mx_moe_qmv", load().mx_moe_qmv(fmt, _ptr(codes), _ptr(scales), _ptr(x),
                                           _ptr(expert_ids), _ptr(y), T, E, topk, N, K))
    return y


def moe_gate_up_swiglu(fmt: int, codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                       expert_ids: torch.Tensor, E: int, I: int, h: torch.Tensor | None = None) -> torch.Tensor:
    """h[T][topk][I] bf16 = SwiGLU of the routed experts' gate and up rows."""
    T, K = x.shape
    topk = expert_ids.shape[1]
    if h is None:
        h = torch.empty((T, topk, I), dtype=torch.bfloat16, device=x.device)
    _stream()
    _check("mx_moe_gate_up_swiglu", load().mx_moe_gate_up_swiglu(fmt, _ptr(codes), _ptr(scales), _ptr(x),
                                                                 _ptr(expert_ids), _ptr(h), T, E, topk, I, K))
    return h


def moe_down_combine(fmt: int, codes: torch.Tensor, scales: torch.Tensor, h: torch.Tensor,
                     expert_ids: torch.Tensor, router_weights: torch.Tensor, E: int, N: int,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """out[T][N] fp32 = router-weighted sum of the routed experts' down rows."""
    T, topk = expert_ids.shape
    K = h.shape[-1]
    if out is None:
        out = torch.empty((T, N), dtype=torch.float32, device=h.device)
    _stream()
    _check("mx_moe_down_combine", load().mx_moe_down_combine(fmt, _ptr(codes), _ptr(scales), _ptr(h),
                                                             _ptr(expert_ids), _ptr(router_weights), _ptr(out),
                                                             T, E, topk, N, K))
    return out


def qmm(fmt: int, codes: torch.Tensor, scales: torch.Tensor, X: torch.Tensor, N: int,
        Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[M][N] bf16 = X (bf16 [M][K]) . W^T with fp32 accumulation."""
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _stream()
    _check("mx_qmm", load().mx_qmm(fmt, _ptr(codes), _ptr(scales), _ptr(X), _ptr(Y), M, N, K))
    return Y


def qmm_qx(fmt: int, codes: torch.Tensor, scales: torch.Tensor, xcodes: torch.Tensor, xscales: torch.Tensor,
           M: int, N: int, K: int, Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[M][N] bf16 = Xq . W^T on the block-scaled tensor cores, Xq given as
    block-float codes and scales in the weights' format."""
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=codes.device)
    _stream()
    _check("mx_qmm_qx", load().mx_qmm_qx(fmt, _ptr(codes), _ptr(scales), _ptr(xcodes), _ptr(xscales), _ptr(Y),
                                         M, N, K))
    return Y


MMA_KINDS = {"bf16": (0, 16), "e4m3": (1, 32), "mxfp8": (2, 32), "mxfp4": (3, 64), "nvfp4": (4, 64)}


PEAK_FILLED, PEAK_ROTATE, PEAK_SMEM_STORES, PEAK_TMEM_STORES = 0x100, 0x200, 0x400, 0x800


def mma_peak_tflops(kind: str, iters: int = 8192, reps: int = 5, filled: bool = False, flags: int = 0) -> float:
    """Best of `reps` mx_mma_peak runs, as dense TFLOP/s of the whole GPU
    (filled: random finite operands instead of zeros; flags: the other
    MX_PEAK_* bits)."""
    code, k = MMA_KINDS[kind]
    code |= flags
    if filled:
        code |= PEAK_FILLED
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    best = 0.0
    ms = ctypes.c_float()
    for _ in range(reps):
        _stream()
        _check("mx_mma_peak", load().mx_mma_peak(code, iters, ctypes.byref(ms)))
        best = max(best, 2.0 * 128 * 256 * k * 4 * iters * sms / (ms.value * 1e-3) / 1e12)
    return best


def _workspace(nbytes: int, ws: torch.Tensor | None, device) -> torch.Tensor:
    if nbytes == 0:
        raise ValueError("sizes outside the library's limits")
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def moe_qmm(fmt: int, codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, expert_ids: torch.Tensor,
            E: int, N: int, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[t][j] bf16 = W_{expert_ids[t][j]} x[t] for many tokens (grouped tensor-core GEMM)."""
    T, K = x.shape
    topk = expert_ids.shape[1]
    if y is None:
        y = torch.empty((T, topk, N), dtype=torch.bfloat16, device=x.device)
    lib = load()
    ws = _workspace(lib.mx_moe_qmm_workspace_size(T, E, topk, K), workspace, x.device)
    _stream()
    _check("mx_moe_qmm", lib.mx_moe_qmm(fmt, _ptr(codes), _ptr(scales), _ptr(x), _ptr(expert_ids), _ptr(y),
                                        T, E, topk, N, K, _ptr(ws), ws.numel()))
    return y


def moe_ffn_prefill_workspace(T: int, E: int, topk: int, H: int, I: int, device="cuda") -> torch.Tensor:
    return _workspace(load().mx_moe_ffn_prefill_workspace_size(T, E, topk, H, I), None, device)


def moe_ffn_prefill(fmt: int, gu_codes: torch.Tensor, gu_scales: torch.Tensor, dn_codes: torch.Tensor,
                    dn_scales: torch.Tensor, x: torch.Tensor, expert_ids: torch.Tensor,
                    router_weights: torch.Tensor, E: int, I: int, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] fp32 = sum_j r[t][j] down_e(SwiGLU(gate_up_e x[t])) over many tokens."""
    T, H = x.shape
    topk = expert_ids.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=x.device)
    lib = load()
    ws = _workspace(lib.mx_moe_ffn_prefill_workspace_size(T, E, topk, H, I), workspace, x.device)
    _stream()
    _check("mx_moe_ffn_prefill", lib.mx_moe_ffn_prefill(fmt, _ptr(gu_codes), _ptr(gu_scales), _ptr(dn_codes),
                                                        _ptr(dn_scales), _ptr(x), _ptr(expert_ids),
                                                        _ptr(router_weights), _ptr(out), T, E, topk, H, I,
                                                        _ptr(ws), ws.numel()))
    return out


def quantize(fmt: int, x: torch.Tensor, codes: torch.Tensor | None = None,
             scales: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 x [M][K] -> (codes, scales) uint8 in the decode's layouts (NVFP4:
    the fp32 tensor scale appended to the scales)."""
    M, K = x.shape
    blk = block_of(fmt)
    if codes is None:
        codes = torch.empty(M * K if fmt == FMT_MXFP8 else M * K // 2, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(M * K // blk + (4 if fmt == FMT_NVFP4 else 0), dtype=torch.uint8, device=x.device)
    _stream()
    _check("mx_quantize", load().mx_quantize(fmt, _ptr(x), _ptr(codes), _ptr(scales), M, K))
    return codes, scales


def dequant(fmt: int, codes: torch.Tensor, scales: torch.Tensor, N: int, K: int,
            W: torch.Tensor | None = None) -> torch.Tensor:
    if W is None:
        W = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    _stream()
    _check("mx_dequant", load().mx_dequant(fmt, _ptr(codes), _ptr(scales), _ptr(W), N, K))
    return W


def swiglu(gu: torch.Tensor, I: int, h: torch.Tensor | None = None) -> torch.Tensor:
    Q = gu.numel() // (2 * I)
    if h is None:
        h = torch.empty((Q, I), dtype=torch.bfloat16, device=gu.device)
    _stream()
    _check("mx_swiglu", load().mx_swiglu(_ptr(gu), _ptr(h), Q, I))
    return h


def moe_combine(yd: torch.Tensor, r: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    T, topk = r.shape
    N = yd.numel() // (T * topk)
    if out is None:
        out = torch.empty((T, N), dtype=torch.float32, device=yd.device)
    _stream()
    _check("mx_moe_combine", load().mx_moe_combine(_ptr(yd), _ptr(r), _ptr(out), T, topk, N))
    return out


# ---- rotary positions, paged key/value cache, attention

KV_BF16, KV_MXFP8 = 0, 1
ROPE_INTERLEAVED, ROPE_INVERSE = 0x1, 0x2
ATTN_CAUSAL = 0x1
WORKSPACE_SLOT_BYTES = 16 << 20  # the library's own workspace of a stream
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _cuda(name: str, t: torch.Tensor, dtype, dim: int) -> int:
    """Device pointer of a tensor of the type, its last dimension contiguous."""
    if t.dtype is dtype and t.is_cuda and t.dim() == dim and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name}: expected {dim} dimensions, got {t.dim()}")
    raise ValueError(f"{name}: the last dimension must be contiguous")


def _whole(name: str, t: torch.Tensor, dtype, shape: tuple) -> int:
    """Device pointer of a contiguous tensor of the type and shape."""
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtype}, shape {tuple(shape)}; got {t.dtype}, "
                     f"{tuple(t.shape)} on {t.device}")


def _strides(t: torch.Tensor) -> tuple:
    """Strides; of a dimension of length one, where they may be anything, those of a tensor whose elements lie together."""
    if 1 not in t.shape:
        return t.stride()
    s = list(t.stride())
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] == 1:
            s[i] = t.shape[i + 1] * s[i + 1]
    return tuple(s)


class _PagedKV(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales", "block_table")]
    _fields_ += [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride", "scale_page_stride",
                                               "scale_head_stride", "scale_token_stride")]
    _fields_ += [(n, ctypes.c_int32) for n in ("kv_fmt", "num_pages", "page_size", "Hkv", "D", "table_stride",
                                               "table_pages")]


class PagedKV:
    """A paged key/value cache and a batch's block table, as mx_kv_append and
    mx_paged_attn take them (mx_paged_kv).

    k, v         [num_pages][Hkv][page_size][D], any strides with the last
                 dimension contiguous (a transposed view of tokens-major pages
                 works), the same for both: bf16, or uint8 E4M3 codes with
    k_scales, v_scales  uint8 E8M0 [num_pages][Hkv][page_size][D/32]
    block_table  int32 [B][pages], the last dimension contiguous (the first
                 columns of a wider table work; the columns past them are not read)

    The object keeps the tensors alive and may be kept and reused while the
    table's contents change."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
        if (k_scales is None) != (v_scales is None):
            raise ValueError("k_scales and v_scales come together")
        mx8 = k_scales is not None
        dtype = torch.uint8 if mx8 else torch.bfloat16
        c = _PagedKV()
        c.k, c.v = _cuda("k", k, dtype, 4), _cuda("v", v, dtype, 4)
        if k.shape != v.shape or _strides(k) != _strides(v):
            raise ValueError("k and v: expected the same shape and strides")
        c.num_pages, c.Hkv, c.page_size, c.D = k.shape
        c.page_stride, c.head_stride, c.token_stride, _ = _strides(k)
        if mx8:
            c.k_scales, c.v_scales = (_cuda("scales", t, torch.uint8, 4) for t in (k_scales, v_scales))
            want = (*k.shape[:3], k.shape[3] // 32)
            if k_scales.shape != want or v_scales.shape != want or _strides(k_scales) != _strides(v_scales):
                raise ValueError(f"scales: expected shape {want} and the same strides")
            c.scale_page_stride, c.scale_head_stride, c.scale_token_stride, _ = _strides(k_scales)
        c.kv_fmt = KV_MXFP8 if mx8 else KV_BF16
        c.block_table = _cuda("block_table", block_table, torch.int32, 2)
        self.B, c.table_pages = block_table.shape
        stride = c.table_pages if self.B == 1 else block_table.stride(0)  # (one row may have any stride)
        if not c.table_pages <= stride < 1 << 31:
            raise ValueError("block_table: expected rows that do not overlap")
        c.table_stride = stride
        self.k, self.v, self.k_scales, self.v_scales, self.block_table = k, v, k_scales, v_scales, block_table
        self.Hkv, self.D = c.Hkv, c.D
        self._c = c
        self._ref = ctypes.byref(c)

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, D: int, block_table: torch.Tensor,
              kv_fmt: int = KV_BF16) -> "PagedKV":
        """A new cache of heads-major pages (contents undefined)."""
        mx8 = kv_fmt == KV_MXFP8
        kv = [torch.empty((num_pages, Hkv, page_size, D), dtype=torch.uint8 if mx8 else torch.bfloat16,
                          device=block_table.device) for _ in "kv"]
        sc = [torch.empty((num_pages, Hkv, page_size, D // 32), dtype=torch.uint8, device=block_table.device)
              for _ in "kv"] if mx8 else [None, None]
        return cls(*kv, block_table, *sc)


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 8192, low: float = 1.0, high: float | None = None) -> tuple[torch.Tensor, float]:
    """Radians per position of the rot/2 pairs (fp64) and the factor on the
    cosines and sines, base^(-2i/rot) and 1 unless a scaling for contexts
    longer than the trained `original_len` changes them:

    "linear"  every frequency over `factor`;
    "base"    the base times factor^(rot/(rot-2)): the slowest pair turns
              `factor` times slower, the fastest as before;
    "banded"  by the turns a pair makes over original_len: above `high` (4)
              unchanged, below `low` (1) over `factor`, blended between;
    "yarn"    the blend runs over the pair's number, between those that turn
              `high` (32) and `low` (1) times, and cosines and sines grow by
              0.1 ln(factor) + 1.

    In brackets what `high` and `low` are where they are left out, as published.
    """
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if rot <= 0 or rot % 2 or base <= 1.0 or factor < 1.0:
        raise ValueError("rope_frequencies: rot even and positive, base > 1, factor >= 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "base":
        return (base * factor ** (rot / (rot - 2.0))) ** (-i / rot) if rot > 2 else f, 1.0
    if scaling == "banded":
        turns = original_len * f / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 1.0
    if scaling == "yarn":
        def dim(turns: float) -> float:
            return rot * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        first, last = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        slow = ((i / 2 - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"rope_frequencies: unknown scaling {scaling!r}")


def rope_table(inv_freq: torch.Tensor, n: int, factor: float = 1.0, pos0: int = 0, device="cuda") -> torch.Tensor:
    """fp32 [n][half][2] cosines and sines (times factor) of positions pos0 .. pos0 + n - 1."""
    f = inv_freq.to(device=device, dtype=torch.float64).contiguous()
    table = torch.empty((n, f.numel(), 2), dtype=torch.float32, device=f.device)
    _stream()
    _check("mx_rope_table", load().mx_rope_table(_ptr(f), factor, _ptr(table), pos0, n, f.numel()))
    return table


def _table_arg(table: torch.Tensor | None) -> tuple[int | None, int, int]:
    """Pointer, positions and rotating dimensions of a rotation table."""
    if table is None:
        return None, 0, 0
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table: expected [positions][rot / 2][2]")
    n, half, _ = shape = table.shape
    return _whole("table", table, torch.float32, shape), n, 2 * half


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor | None, interleaved: bool = False,
         inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate the first 2 * table.shape[1] dimensions of each head of x [T][H][D]
    (bf16 or fp32, the last dimension contiguous) by the angles of its token's position
    (positions int32 [T]); inverse: rotate back (the gradient); table None: a copy.  out may be x."""
    if x.dtype not in _DTYPES:
        raise ValueError(f"x: expected bf16 or fp32, got {x.dtype}")
    xp = _cuda("x", x, x.dtype, 3)
    T, H, D = x.shape
    xt, xh, _ = x.stride()
    if H == 1:  # (as _strides)
        xh = D
    if T == 1:
        xt = H * xh
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
        op, yt, yh = out.data_ptr(), H * D, D
    else:
        if out.shape != x.shape:
            raise ValueError("out: expected the shape of x")
        op = _cuda("out", out, x.dtype, 3)
        yt, yh, _ = _strides(out)
    tp, n, rot = _table_arg(table)
    pp = _whole("positions", positions, torch.int32, (T,))
    if T == 0:
        return out
    _stream()
    _check("mx_rope", load().mx_rope(xp, op, _DTYPES[x.dtype], pp, tp, n, T, H, D, rot, xt, xh, yt, yh,
                                     (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0)))
    return out


def kv_append(kv: PagedKV, rows: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, Hq: int,
              table: torch.Tensor | None, interleaved: bool = False, q: torch.Tensor | None = None) -> torch.Tensor:
    """Split the fused QKV rows [T][(Hq + 2 Hkv) D] (bf16 or fp32): rotate queries
    and keys at their places in the contexts, write keys and values to the
    cache and return the queries, bf16 [T][Hq][D].  q_start int32 [B+1], kv_len int32 [B] (new
    tokens included); table None: no rotation."""
    if rows.dtype not in _DTYPES:
        raise ValueError(f"rows: expected bf16 or fp32, got {rows.dtype}")
    rp = _cuda("rows", rows, rows.dtype, 2)
    T, D = rows.shape[0], kv.D
    if rows.shape[1] != (Hq + 2 * kv.Hkv) * D:
        raise ValueError(f"rows: expected (Hq + 2 Hkv) D = {(Hq + 2 * kv.Hkv) * D} elements per token")
    if q is None:
        q = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=rows.device)
        qp = q.data_ptr()
    else:
        qp = _whole("q", q, torch.bfloat16, (T, Hq, D))
    tp, n, rot = _table_arg(table)
    sp, lp = _whole("q_start", q_start, torch.int32, (kv.B + 1,)), _whole("kv_len", kv_len, torch.int32, (kv.B,))
    if T == 0:
        return q
    _stream()
    stride = rows.stride(0) if T > 1 else rows.shape[1]
    _check("mx_kv_append", load().mx_kv_append(kv._ref, rp, _DTYPES[rows.dtype], stride, sp, lp, tp, n, rot, qp, T, kv.B,
                                               Hq, ROPE_INTERLEAVED if interleaved else 0))
    return q


def paged_attn_workspace(T: int, B: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    return _workspace(load().mx_paged_attn_workspace_size(T, B, Hq, Hkv, D), None, device)


def paged_attn(kv: PagedKV, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               scale: float | None = None, causal: bool = True, window: int = 0, sinks: torch.Tensor | None = None,
               out: torch.Tensor | None = None, return_lse: bool = False, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """Attention of the new tokens' queries q [T][Hq][D] (bf16, the last dimension
    contiguous) over their contexts in the cache; out bf16 [T][Hq][D], and with
    return_lse (out, lse) with lse fp32 [T][Hq].  scale: 1/sqrt(D) by default; window > 0 (of any size): each token sees
    itself and the window - 1 tokens before it; sinks fp32 [Hq]."""
    qp = _cuda("q", q, torch.bfloat16, 3)
    T, Hq, D = q.shape
    if D != kv.D:
        raise ValueError(f"q: heads of {D}, the cache's have {kv.D}")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _whole("out", out, torch.bfloat16, (T, Hq, D))
    if lse is not None:
        ep = _whole("lse", lse, torch.float32, (T, Hq))
    elif return_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
        ep = lse.data_ptr()
    else:
        ep = None
    kp = None if sinks is None else _whole("sinks", sinks, torch.float32, (Hq,))
    B = kv.B
    sp, lp = _whole("q_start", q_start, torch.int32, (B + 1,)), _whole("kv_len", kv_len, torch.int32, (B,))
    if T > 0:
        lib = load()
        if workspace is None:
            need = lib.mx_paged_attn_workspace_size(T, B, Hq, kv.Hkv, D)
            if need == 0 or need > WORKSPACE_SLOT_BYTES:
                workspace = _workspace(need, None, q.device)
        wp, wn = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
        qt, qh, _ = q.stride()
        if Hq == 1:  # (as _strides)
            qh = D
        if T == 1:
            qt = Hq * qh
        _stream()
        _check("mx_paged_attn", lib.mx_paged_attn(kv._ref, qp, qt, qh, sp, lp,
                                                  1.0 / math.sqrt(D) if scale is None else scale,
                                                  ATTN_CAUSAL if causal else 0,
                                                  max(-1, min(window, 0x7FFFFFFF)), kp, op, ep, T, B, Hq, wp, wn))
    return (out, lse) if return_lse else out


# ---- decode loops: beams, and the pages of their contexts


class Beams(NamedTuple):
    """beam_select's result: the k best continuations of each batch entry [B][k] (score fp32, parent and token
    int32), and of those the first W that do not end [B][W]."""
    score: torch.Tensor
    parent: torch.Tensor
    token: torch.Tensor
    next_score: torch.Tensor
    next_parent: torch.Tensor
    next_token: torch.Tensor


def beam_select_workspace(B: int, W: int, V: int, k: int, device="cuda") -> torch.Tensor:
    return _workspace(load().mx_beam_select_workspace_size(B, W, V, k), None, device)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, k: int | None = None, eos: int = -1,
                mask: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> Beams:
    """The k (2 W by default) best continuations of each batch entry's beams: logits [B * W][V] (bf16 or fp32, the
    last dimension contiguous), scores fp32 [B][W] (logarithms of the beams' probabilities; -inf: no beam), key = score
    + log_softmax(logits).  Ordered by key, then beam, then logit, then the lower token.  parent is the row of
    `logits`, so it serves kv_remap as it is.  Places without a candidate hold -inf, -1, 0.  eos: the token that ends
    a beam; beams of that token are left out of next_*.  mask int32 [B * W][ceil(V / 32)]: bit v % 32 of word v // 32
    allows token v; the probabilities are those among the allowed tokens."""
    dt, dev = _DTYPES.get(logits.dtype), logits.device
    if dt is None:
        raise ValueError(f"logits: expected bf16 or fp32, got {logits.dtype}")
    xp = _cuda("logits", logits, logits.dtype, 2)
    rows, V = logits.shape
    shape = scores.shape
    if len(shape) != 2 or shape[0] * shape[1] != rows:
        raise ValueError("scores: expected [B][W] with a row of logits for each")
    B, W = shape
    sp = _whole("scores", scores, torch.float32, shape)
    if k is None:
        k = 2 * W
    mp, ms = None, 0
    if mask is not None:
        mp = _cuda("mask", mask, torch.int32, 2)
        if mask.shape != (rows, (V + 31) // 32):
            raise ValueError(f"mask: expected shape {(rows, (V + 31) // 32)}")
        ms = mask.stride(0) if rows > 1 else mask.shape[1]
    # (six allocations cost less than one and six views)
    empty, f32, i32, bk, bw = torch.empty, torch.float32, torch.int32, (B, k), (B, W)
    out = Beams(empty(bk, dtype=f32, device=dev), empty(bk, dtype=i32, device=dev), empty(bk, dtype=i32, device=dev),
                empty(bw, dtype=f32, device=dev), empty(bw, dtype=i32, device=dev), empty(bw, dtype=i32, device=dev))
    if rows > 0:
        lib = load()
        stride = logits.stride(0) if rows > 1 else V
        a, b, c, d, e, f = out
        op = (a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr(), e.data_ptr(), f.data_ptr())
        wp, wn = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
        _stream()
        s = lib.mx_beam_select(xp, dt, stride, sp, mp, ms, B, W, V, k, eos if eos >= 0 else -1, *op, wp, wn)
        if s == -1 and workspace is None:  # (the stream's own may be too small)
            need = lib.mx_beam_select_workspace_size(B, W, V, k)
            if need > WORKSPACE_SLOT_BYTES:
                workspace = _workspace(need, None, dev)
                s = lib.mx_beam_select(xp, dt, stride, sp, mp, ms, B, W, V, k, max(eos, -1), *op, workspace.data_ptr(), need)
        _check("mx_beam_select", s)
    return out


class _PagePool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("count", "refs", "free_pages", "work")] + [("num_pages", ctypes.c_int32)]


class PagePool:
    """Which of a cache's pages are in use, kept on the device (mx_page_pool): `count` int32 [1] free pages,
    `refs` int32 [num_pages] references of each page (one for each table entry, and those of other holders),
    `free_pages` int32 [num_pages] the stack of free pages.  All pages are free at first, page 0 is taken first.  The
    three are views of `state` int32 [4 + 2 num_pages], which may be given (a pool as it was saved)."""

    def __init__(self, num_pages: int, device="cuda", state: torch.Tensor | None = None):
        if state is None:
            state = torch.zeros(4 + 2 * num_pages, dtype=torch.int32, device=device)
            state[0] = num_pages
            state[4 + num_pages:] = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        sp = _whole("state", state, torch.int32, (4 + 2 * num_pages,))
        size = load().mx_page_pool_work_size(num_pages)
        if size == 0:
            raise ValueError("sizes outside the library's limits")
        self.work = torch.zeros(size, dtype=torch.uint8, device=state.device)
        self.num_pages, self.state = num_pages, state
        self.count, self.refs, self.free_pages = state[:1], state[4:4 + num_pages], state[4 + num_pages:]
        c = _PagePool(sp, sp + 16, sp + 16 + 4 * num_pages, self.work.data_ptr(), num_pages)
        self._c, self._ref = c, ctypes.byref(c)


def _table_of(name: str, table: torch.Tensor) -> tuple[int, int, int, int]:
    """Pointer, row stride, pages of a row and sequences of a block table."""
    p = _cuda(name, table, torch.int32, 2)
    S, n = table.shape
    return p, n if S == 1 else table.stride(0), n, S


def kv_remap(pool: PagePool, page_size: int, table: torch.Tensor, kv_len: torch.Tensor, parent: torch.Tensor,
             table_out: torch.Tensor, add: int | torch.Tensor = 1, keep: torch.Tensor | None = None,
             kv_len_out: torch.Tensor | None = None,
             copies: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """One step of the sequences' pages: forks, growth, cuts and releases at once (mx_kv_remap).

    New sequence s takes the first keep[s] tokens (int32 [S_out]; None: all) of sequence parent[s] (int32 [S_out], a
    row of `table` int32 [S_in][pages] and `kv_len` int32 [S_in]; negative: none) and grows by add (int32 [S_out], or one
    number for all sequences that have a parent).  `table_out` int32 [S_out][pages] receives its pages; sequences
    that are no one's parent release theirs.  Pages are shared; a sequence that grows in the middle of a page
    others hold too gets a page and a copy.  Returns the new lengths int32 [S_out] and the copies that
    kv_copy_pages has to make before the cache is used.  Where the pool cannot supply the step, or the arguments do
    not fit, nothing changes, the lengths are -1 and device_error() tells why."""
    i32 = torch.int32
    tp, ts, tn, S_in = _table_of("table", table)
    op, os_, on, S_out = _table_of("table_out", table_out)
    size = (S_out,)
    lp = _whole("kv_len", kv_len, i32, (S_in,))
    if parent.dim() != 1:
        parent = parent.reshape(-1)  # (a copy where its rows lie apart: kept until the call is made)
    pp = _whole("parent", parent, i32, size)
    kp = None if keep is None else _whole("keep", keep, i32, size)
    ap, each = (None, add) if isinstance(add, int) else (_whole("add", add, i32, size), 0)
    if kv_len_out is None:
        kv_len_out = torch.empty(size, dtype=i32, device=table.device)
        np_ = kv_len_out.data_ptr()
    else:
        np_ = _whole("kv_len_out", kv_len_out, i32, size)
    if copies is None:
        copies = torch.empty((1 + S_out, 4), dtype=i32, device=table.device)
        cp = copies.data_ptr()
    else:
        cp = _whole("copies", copies, i32, (1 + S_out, 4))
    _stream()
    _check("mx_kv_remap", load().mx_kv_remap(pool._ref, page_size, tp, ts, tn, lp, S_in, op, os_, on, np_, S_out, pp, kp,
                                             ap, each, cp))
    return kv_len_out, copies


def kv_compact(pool: PagePool, page_size: int, table: torch.Tensor, kv_len: torch.Tensor,
               copies: torch.Tensor | None = None) -> torch.Tensor:
    """Make the pool dense in place (mx_kv_compact): pages in use move to the lowest places, `table` follows.
    Pages with holders besides this table stay.  Returns the copies [1 + num_pages // 2][4] that kv_copy_pages has to
    make before the cache is used."""
    tp, ts, tn, S = _table_of("table", table)
    lp = _whole("kv_len", kv_len, torch.int32, (S,))
    rows = 1 + pool.num_pages // 2
    if copies is None:
        copies = torch.empty((rows, 4), dtype=torch.int32, device=table.device)
        cp = copies.data_ptr()
    else:
        cp = _whole("copies", copies, torch.int32, (rows, 4))
    _stream()
    _check("mx_kv_compact", load().mx_kv_compact(pool._ref, page_size, tp, ts, tn, lp, S, cp))
    return copies


class PagedKVLayers:
    """The caches of several layers that share a pool (the same format, sizes and strides), as kv_copy_pages takes
    them.  Keeps them alive."""

    def __init__(self, layers: list[PagedKV]):
        self.layers = list(layers)
        self._c = (_PagedKV * len(self.layers))(*(kv._c for kv in self.layers))


def kv_copy_pages(layers: PagedKVLayers | PagedKV, copies: torch.Tensor) -> None:
    """Copy pages in every layer's cache, by a list as kv_remap and kv_compact return it: int32 [1 + most][4], row 0
    {n, 0, 0, 0}, then n rows {source, destination, tokens, 0}."""
    c, n = (layers._ref, 1) if isinstance(layers, PagedKV) else (layers._c, len(layers.layers))
    most = copies.shape[0] - 1
    cp = _whole("copies", copies, torch.int32, (1 + most, 4))
    if most == 0:
        return
    _stream()
    _check("mx_kv_copy_pages", load().mx_kv_copy_pages(c, n, cp, most))


# ---- products of 8-bit integers


def i8_quantize(x: torch.Tensor, q: torch.Tensor | None = None,
                scales: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """x [M][K] (bf16 or fp32) -> (codes int8 [M][K], scales fp32 [M]): the scale max |x| / 127 of each token, codes
    x / scale to the nearest even integer."""
    if x.dtype not in _DTYPES:
        raise ValueError(f"x: expected bf16 or fp32, got {x.dtype}")
    M, K = x.shape
    xp = _whole("x", x, x.dtype, (M, K))
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    qp, sp = _whole("q", q, torch.int8, (M, K)), _whole("scales", scales, torch.float32, (M,))
    if M == 0:
        return q, scales
    _stream()
    _check("mx_i8_quantize", load().mx_i8_quantize(xp, _DTYPES[x.dtype], qp, sp, M, K))
    return q, scales


def i8_mm_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    return _workspace(load().mx_i8_mm_workspace_size(M, K), None, device)


def i8_mm(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, x_scales: torch.Tensor | None = None,
          out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[M][N] (bf16 or fp32) = (xq . w^T) * x_scales[m] * w_scales[n], w int8 [N][K], w_scales fp32 [N].  x: int8
    [M][K] with x_scales fp32 [M] (i8_quantize), or bf16 / fp32 [M][K], quantised on the way."""
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x and w: expected [M][K] and [N][K]")
    M, K = x.shape
    N = w.shape[0]
    if x.dtype is torch.int8:
        if x_scales is None:
            raise ValueError("x_scales: int8 codes come with their scales")
        xd, sp = 2, _whole("x_scales", x_scales, torch.float32, (M,))
    elif x.dtype in _DTYPES:
        if x_scales is not None:
            raise ValueError("x_scales: only with int8 codes")
        xd, sp = _DTYPES[x.dtype], None
    else:
        raise ValueError(f"x: expected int8, bf16 or fp32, got {x.dtype}")
    xp, wp = _whole("x", x, x.dtype, (M, K)), _whole("w", w, torch.int8, (N, K))
    cp = _whole("w_scales", w_scales, torch.float32, (N,))
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError(f"out_dtype: expected bf16 or fp32, got {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
        op = out.data_ptr()
    else:
        if out.dtype not in _DTYPES:
            raise ValueError(f"out: expected bf16 or fp32, got {out.dtype}")
        op = _whole("out", out, out.dtype, (M, N))
    if M == 0:
        return out
    lib = load()
    if workspace is None and M * K > WORKSPACE_SLOT_BYTES // 4:  # (2 bytes an element and 4 a row, rounded up)
        need = lib.mx_i8_mm_workspace_size(M, K)
        if need > WORKSPACE_SLOT_BYTES:
            workspace = _workspace(need, None, x.device)
    ap, an = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
    _stream()
    _check("mx_i8_mm", lib.mx_i8_mm(xp, xd, sp, wp, cp, op, _DTYPES[out.dtype], M, N, K, ap, an))
    return out


def debug_qmm_stall(stall: bool, wait_ns: int = 0) -> None:
    """Test hook: make later tensor-core GEMM launches withhold their
    activation loads so that their bounded waits time out (see mx.h)."""
    _check("mx_debug_qmm_stall", load().mx_debug_qmm_stall(1 if stall else 0, wait_ns))


def device_error() -> int:
    """Synchronise the current stream; return and clear the device error word."""
    _stream()
    s = load().mx_device_error()
    if s < 0:
        _check("mx_device_error", s)
    return s


def raw_call(name: str, *args) -> int:
    """Call an ABI function with raw integer/pointer arguments (tests)."""
    return getattr(load(), name)(*args)
