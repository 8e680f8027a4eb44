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
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = I
        for name, args in {"mx_moe_qmm_workspace_size": [I, I, I, I],
                           "mx_moe_ffn_prefill_workspace_size": [I, I, I, I, I],
                           "mx_paged_attn_workspace_size": [I, I, I, I, I]}.items():
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
