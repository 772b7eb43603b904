"""Python binding of libqaff (group-wise affine quantized matmul, MI355X / gfx950).

Argument marshalling only: every computation runs in the HIP kernels of
libqaff.so, reached through its C ABI (include/qaff.h).  PyTorch supplies
device memory and the current HIP stream; nothing here computes.  There is no
CPU fallback: if the library is missing this module raises on first use.

Functions mirror the C entry points:
    qmm_affine, qgemv_affine, qgemv_affine_grouped, qmm_gptq, qgemm_w4a8,
    gptq_to_affine_repack, quantize_pack_affine, rmsnorm, rmsnorm_w4a8,
    qgemm_w4a8_codes, kv_cache_append_affine, kv_cache_read_affine,
    paged_attention_affine, kv_pages_assign, kv_pages_trim, rotary,
    kv_cache_append_rotary_affine, qmoe_affine
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

__all__ = ["QaffError", "qmm_affine", "qmm_affine_noalloc", "qgemv_affine", "qgemv_affine_grouped", "GroupedGemv", "qmm_gptq", "qgemm_w4a8", "qgemm_w4a8_tiled", "gptq_to_affine_repack",
           "quantize_pack_affine", "dequantize_affine", "qgemv_affine_silu_gate", "smoothquant_factors",
           "w4a8_quantize_weights", "qgemm_w4a8_smooth", "qgemm_w4a8_codes", "rmsnorm", "rmsnorm_w4a8", "AffineKVCache",
           "kv_cache_append_affine", "kv_cache_read_affine", "paged_attention_affine", "KVPagePool", "kv_pages_assign",
           "kv_pages_trim", "Rotary", "rotary", "kv_cache_append_rotary_affine", "AffineExperts",
           "qmoe_affine",
           "release_workspaces", "GemvChain", "library_path", "lib",
           "STATUS", "DTYPE"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libqaff.so")

STATUS = {0: "QAFF_OK", 1: "QAFF_E_INVAL", 2: "QAFF_E_UNSUPPORTED", 3: "QAFF_E_ALIGN", 4: "QAFF_E_HIP"}
DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_I64, _I32, _VP = C.c_int64, C.c_int32, C.c_void_p

# argument type lists of the exported symbols (include/qaff.h)
_SIGS = {
    "qmm_affine": [_VP] * 6 + [_I64] * 3 + [_I32] * 5 + [_VP],
    "qgemv_affine": [_VP] * 6 + [_I64] * 3 + [_I32] * 5 + [_VP],
    "qmm_affine_noalloc": [_VP] * 6 + [_I64] * 3 + [_I32] * 5 + [_VP],
    "qmm_gptq": [_VP] * 6 + [_I64] * 3 + [_I32, _VP],
    "qgemm_w4a8": [_VP] * 7 + [_I64] * 3 + [_VP],
    "qgemm_w4a8_tiled": [_VP] * 7 + [_I64] * 3 + [_I32] * 3 + [_VP],
    "gptq_to_affine_repack": [_VP] * 7 + [_I32, _VP] + [_I64] * 2 + [_I32, _VP],
    "quantize_pack_affine": [_VP, _I32, _VP, _VP, _VP, _I32, _I64, _I64, _I32, _I32, _VP],
    "qgemv_affine_grouped": [_VP, _I32, _I64] + [_I32] * 5 + [_VP],
    "dequantize_affine": [_VP] * 4 + [_I64] * 2 + [_I32] * 5 + [_VP],
    "qgemv_affine_silu_gate": [_VP] * 7 + [_I64] * 3 + [_I32] * 5 + [_VP],
    "smoothquant_factors": [_VP, _VP, _I32, C.c_double, _VP, _I64, _I64, _VP],
    "w4a8_quantize_weights": [_VP, _I32, _VP, _VP, _VP, _I64, _I64, _VP],
    "qgemm_w4a8_smooth": [_VP] * 8 + [_I64] * 3 + [_VP],
    "qgemm_w4a8_codes": [_VP] * 6 + [_I64] * 3 + [_VP],
    "rmsnorm": [_VP] * 3 + [C.c_double] + [_VP] * 2 + [_I64] * 5 + [_I32] * 2 + [_VP],
    "rmsnorm_w4a8": [_VP] * 3 + [C.c_double] + [_VP] * 3 + [_I64] * 5 + [_I32] * 2 + [_VP],
    "kv_cache_append_affine": [_VP] * 3 + [_I64] * 4 + [_VP, _I64, _VP],
    "kv_cache_read_affine": [_VP] * 4 + [_I64, _VP],
    "paged_attention_affine": [_VP, _VP] + [_I64] * 2 + [_VP] + [_I64] * 2 + [_VP] * 2 + [_I64, _I32, C.c_double, _I64,
                                                                                       _VP],
    "kv_pages_assign": [_VP] + [_I64] * 2 + [_VP] * 5 + [_I64, _I32, _I64] + [_VP] * 3 + [_I64, _VP],
    "kv_pages_trim": [_VP] + [_I64] * 2 + [_VP] * 5 + [_I64, _I32, _I64, _VP],
    "rotary_frequencies": [_VP, _I32, C.c_double, _I32] + [C.c_double] * 4 + [_VP],
    "rotary": [_VP] + [_VP, _I64, _I64] * 4 + [_VP, _I64] + [_I32] * 4 + [_VP],
    "kv_cache_append_rotary_affine": [_VP] * 2 + [_VP, _I64, _I64] * 4 + [_VP] * 2 + [_I64, _I32, _VP],
    "qmoe_affine": [_VP] * 3 + [_I32] + [_VP] * 2 + [_I64, _I32, _I32, C.c_double, _VP],
    "qaff_stream_read": [_VP, C.c_uint64, _VP, _I32, _VP],
    "qgemv_affine_chain_plan": [_VP, _I32, _I32, _I32, _I32, C.POINTER(_VP)],
    "qgemv_affine_chain_run": [_VP, _VP],
    "qgemv_affine_chain_status": [_VP, C.POINTER(_I32)],
    "qgemv_affine_chain_free": [_VP],
}


class GemvProblem(C.Structure):
    """qaff_gemv_problem (include/qaff.h)."""
    _fields_ = [("x", _VP), ("w_packed", _VP), ("scales", _VP), ("biases", _VP), ("k_perm", _VP), ("y", _VP),
                ("N", _I64), ("K", _I64)]


class ChainLinear(C.Structure):
    """qaff_chain_linear (include/qaff.h)."""
    _fields_ = [("x", _VP), ("gate", _VP), ("resid", _VP), ("w_packed", _VP), ("scales", _VP), ("biases", _VP),
                ("y", _VP), ("N", _I64), ("K", _I64), ("stage", _I32)]


class KVCacheArrays(C.Structure):
    """qaff_kv_cache (include/qaff.h)."""
    _fields_ = [(n, _VP) for n in ("k_packed", "k_scales", "k_biases", "v_packed", "v_scales", "v_biases")] + \
               [("num_pages", _I64)] + \
               [(n, _I32) for n in ("page_size", "kv_heads", "head_dim", "group_size", "bits", "dtype")]


class RotarySpec(C.Structure):
    """qaff_rotary (include/qaff.h)."""
    _fields_ = [("inv_freq", _VP), ("rotary_dim", _I32), ("interleaved", _I32), ("magnitude", C.c_double)]


class ExpertArrays(C.Structure):
    """qaff_experts (include/qaff.h)."""
    _fields_ = [(n, _VP) for n in ("gate_up_packed", "gate_up_scales", "gate_up_biases", "down_packed", "down_scales",
                                   "down_biases")] + \
               [("hidden", _I64), ("inner", _I64)] + \
               [(n, _I32) for n in ("num_experts", "group_size", "bits", "dtype")]


class QaffError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None
# the current device, and the current stream's handle without making a torch.cuda.Stream (1.7 us of a 6 us call): set by
# lib(), None where torch is built without a GPU and has no such names
_current_device = _raw_stream = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libqaff.so (ctypes), with argument types declared."""
    global _lib, _current_device, _raw_stream
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")
        L = C.CDLL(_LIB_PATH)
        for name, argtypes in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = argtypes
            f.restype = C.c_int
        L.qaff_last_error.restype = C.c_char_p
        L.qaff_last_error.argtypes = []
        L.qaff_version.restype = C.c_int
        L.qaff_release_workspaces.restype = C.c_int
        L.qaff_release_workspaces.argtypes = [C.POINTER(C.c_uint64)]
        _current_device = getattr(torch._C, "_cuda_getDevice", None)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise QaffError(status, where, lib().qaff_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(device) -> int:
    return _raw_stream(device.index)


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return DTYPE[t.dtype]


def _u32(t: torch.Tensor) -> torch.Tensor:
    # packed words travel as int32 or uint32 tensors; only the bits matter
    if t.dtype not in (torch.int32, torch.uint32):
        raise ValueError("packed words must be an int32/uint32 tensor")
    return t


def _run(name: str, device, *args) -> None:
    """Calls an entry point on the current stream of `device`, with `device` the current one (a launch goes there)."""
    f = getattr(_lib or lib(), name)
    index = device.index
    if index == _current_device():
        st = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = f(*args, _raw_stream(index))
    if st != 0:
        _check(st, name)


def _check_shapes(first: torch.Tensor, **others):
    """Raises for the first of (tensor, shape) pairs that lacks its shape or lies on another device than `first`."""
    for name, (t, shape) in others.items():
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _out(out: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    """`out`, checked, or a new dense tensor of the shape and type of `like`."""
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
        raise ValueError(f"out must be a {tuple(like.shape)} tensor of {like.dtype} on {like.device}")
    return out


def _row_ptr(t: torch.Tensor) -> int:
    """Address of a tensor whose last dimension is dense; the others go by their strides."""
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError("the last dimension must be contiguous")
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return t.data_ptr()


def _rows(t: torch.Tensor, dense: bool = False):
    """Address and strides of rows [T, heads, D]; `dense`: the call has just made it."""
    if dense:
        _, m, d = t.shape
        return t.data_ptr(), m * d, d
    return (_row_ptr(t), *_strides(t))


def _strides(t: torch.Tensor):
    """Strides of the two leading dimensions; 0 where one has a single entry, whose stride means nothing."""
    a, b = t.stride()[:2]
    n, m = t.shape[:2]
    return a if n > 1 else 0, b if m > 1 else 0


def _affine(fn: str, x, w_packed, scales, biases, group_size, bits, k_perm, out):
    M, K = x.shape
    N = w_packed.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
    st = getattr(lib(), fn)(_ptr(x), _ptr(_u32(w_packed)), _ptr(scales), _ptr(biases), _ptr(k_perm), _ptr(y), M, N, K,
                            group_size, bits, _dt(x), _dt(scales), _dt(biases), _stream(x.device))
    _check(st, fn)
    return y


def qmm_affine(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
               group_size: int, bits: int, k_perm: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[M,N] = x[M,K] . W^T, W[n,k] = code*scale[n,k/G] + bias[n,k/G]."""
    return _affine("qmm_affine", x, w_packed, scales, biases, group_size, bits, k_perm, out)


def qmm_affine_noalloc(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                       group_size: int, bits: int, k_perm: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """As qmm_affine, with the library's fixed scratch array (no device allocation)."""
    return _affine("qmm_affine_noalloc", x, w_packed, scales, biases, group_size, bits, k_perm, out)


def qgemv_affine(x, w_packed, scales, biases, group_size: int, bits: int, k_perm=None, out=None) -> torch.Tensor:
    """As qmm_affine, always on the GEMV kernel (M <= 16)."""
    return _affine("qgemv_affine", x, w_packed, scales, biases, group_size, bits, k_perm, out)


def qgemv_affine_silu_gate(gate, up, w_packed, scales, biases, group_size: int, bits: int, resid=None,
                           out=None) -> torch.Tensor:
    """y = W (silu(gate) * up) [+ resid] in one launch; gate/up [M, K], M <= 16."""
    M, K = gate.shape
    N = w_packed.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=gate.dtype, device=gate.device)
    st = lib().qgemv_affine_silu_gate(_ptr(gate), _ptr(up), _ptr(resid), _ptr(_u32(w_packed)), _ptr(scales),
                                      _ptr(biases), _ptr(y), M, N, K, group_size, bits, _dt(gate), _dt(scales),
                                      _dt(biases), _stream(gate.device))
    _check(st, "qgemv_affine_silu_gate")
    return y


def qgemv_affine_grouped(problems, group_size: int, bits: int, outs=None):
    """Independent GEMVs in as few launches as possible.

    problems: sequence of (x, w_packed, scales, biases) or (..., k_perm)
    tuples sharing M, dtypes, group_size and bits; returns the list of y.
    """
    n = len(problems)
    arr = (GemvProblem * max(n, 1))()
    ys = []
    for i, p in enumerate(problems):
        x, w, sc, bi = p[:4]
        kp = p[4] if len(p) > 4 else None
        M, K = x.shape
        N = w.shape[0]
        y = outs[i] if outs is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
        ys.append(y)
        arr[i] = GemvProblem(_ptr(x), _ptr(_u32(w)), _ptr(sc), _ptr(bi), _ptr(kp), _ptr(y), N, K)
    if n == 0:
        return ys
    x0, w0, s0, b0 = problems[0][:4]
    st = lib().qgemv_affine_grouped(C.cast(arr, _VP), n, x0.shape[0], group_size, bits, _dt(x0), _dt(s0), _dt(b0),
                                    _stream(x0.device))
    _check(st, "qgemv_affine_grouped")
    return ys


class GroupedGemv:
    """qgemv_affine_grouped with the descriptor array marshalled once.

    Holds references to every tensor it points at; calling it enqueues the
    GEMVs on the current stream of the device of the first x.
    """

    def __init__(self, problems, group_size: int, bits: int, outs=None):
        self.problems = [tuple(p) for p in problems]
        self.ys = []
        self.arr = (GemvProblem * max(len(problems), 1))()
        for i, p in enumerate(self.problems):
            x, w, sc, bi = p[:4]
            kp = p[4] if len(p) > 4 else None
            M, K = x.shape
            N = w.shape[0]
            y = outs[i] if outs is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
            self.ys.append(y)
            self.arr[i] = GemvProblem(_ptr(x), _ptr(_u32(w)), _ptr(sc), _ptr(bi), _ptr(kp), _ptr(y), N, K)
        x0, _, s0, b0 = self.problems[0][:4]
        self.args = (len(self.problems), x0.shape[0], group_size, bits, _dt(x0), _dt(s0), _dt(b0))
        self.device = x0.device

    def __call__(self):
        st = lib().qgemv_affine_grouped(C.cast(self.arr, _VP), *self.args, _stream(self.device))
        _check(st, "qgemv_affine_grouped")
        return self.ys


class GemvChain:
    """qgemv_affine_chain_plan / _run / _status / _free: linears of a decode
    step (one x row, 4-bit codes) in dependency stages, one launch per run.

    `linears`: dicts with x, w, s, b, y, stage and optionally gate, resid
    (tensors; x, gate [1, K] or [K], y and resid [1, N] or [N]).  Holds
    references to every tensor it points at; calling it enqueues the chain
    on the current stream of the device of the first x.
    """

    def __init__(self, linears, group_size: int, bits: int = 4):
        self.linears = [dict(l) for l in linears]
        arr = (ChainLinear * max(len(self.linears), 1))()
        for i, l in enumerate(self.linears):
            N, K = l["w"].shape[0], l["x"].shape[-1]
            arr[i] = ChainLinear(_ptr(l["x"]), _ptr(l.get("gate")), _ptr(l.get("resid")), _ptr(_u32(l["w"])),
                                 _ptr(l["s"]), _ptr(l["b"]), _ptr(l["y"]), N, K, int(l["stage"]))
        x0 = self.linears[0]["x"]
        self.device = x0.device
        self.plan = None
        h = _VP()
        with torch.cuda.device(self.device):
            st = lib().qgemv_affine_chain_plan(C.cast(arr, _VP), len(self.linears), group_size, bits, _dt(x0),
                                               C.byref(h))
        _check(st, "qgemv_affine_chain_plan")
        self.plan = h.value

    def __call__(self):
        st = lib().qgemv_affine_chain_run(self.plan, _stream(self.device))
        _check(st, "qgemv_affine_chain_run")

    def timed_out(self) -> bool:
        v = _I32(0)
        with torch.cuda.device(self.device):
            st = lib().qgemv_affine_chain_status(self.plan, C.byref(v))
        _check(st, "qgemv_affine_chain_status")
        return bool(v.value)

    def close(self):
        if self.plan is not None:
            with torch.cuda.device(self.device):
                st = lib().qgemv_affine_chain_free(self.plan)
            self.plan = None
            _check(st, "qgemv_affine_chain_free")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qmm_gptq(x: torch.Tensor, qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
             g_idx: Optional[torch.Tensor], group_size: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x . W^T for a GPTQ layer (qweight [K/8,N], qzeros [K/G,N/8], scales f16 [K/G,N])."""
    M, K = x.shape
    N = qweight.shape[1]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=x.device)
    st = lib().qmm_gptq(_ptr(x), _ptr(qweight), _ptr(qzeros), _ptr(scales), _ptr(g_idx), _ptr(y), M, N, K,
                        group_size, _stream(x.device))
    _check(st, "qmm_gptq")
    return y


def qgemm_w4a8(x: torch.Tensor, w_q4: torch.Tensor, s_w: torch.Tensor, want_acc: bool = False):
    """Returns (y f16 [M,N], x_q int8 [M,K], s_x f32 [M], acc int32 [M,N] or None)."""
    M, K = x.shape
    N = w_q4.shape[0]
    dev = x.device
    y = torch.empty((M, N), dtype=torch.float16, device=dev)
    x_q = torch.empty((M, K), dtype=torch.int8, device=dev)
    s_x = torch.empty((M,), dtype=torch.float32, device=dev)
    acc = torch.empty((M, N), dtype=torch.int32, device=dev) if want_acc else None
    st = lib().qgemm_w4a8(_ptr(x), _ptr(_u32(w_q4)), _ptr(s_w), _ptr(y), _ptr(x_q), _ptr(s_x), _ptr(acc), M, N, K,
                          _stream(dev))
    _check(st, "qgemm_w4a8")
    return y, x_q, s_x, acc


def qgemm_w4a8_tiled(x: torch.Tensor, w_q4: torch.Tensor, s_w: torch.Tensor, staged: bool, bm: int, bn: int,
                     want_acc: bool = False):
    """qgemm_w4a8 (M > 16) with the lowering (staged or full-K) and the bm x bn tile chosen."""
    M, K = x.shape
    N = w_q4.shape[0]
    dev = x.device
    y = torch.empty((M, N), dtype=torch.float16, device=dev)
    x_q = torch.empty((M, K), dtype=torch.int8, device=dev)
    s_x = torch.empty((M,), dtype=torch.float32, device=dev)
    acc = torch.empty((M, N), dtype=torch.int32, device=dev) if want_acc else None
    st = lib().qgemm_w4a8_tiled(_ptr(x), _ptr(_u32(w_q4)), _ptr(s_w), _ptr(y), _ptr(x_q), _ptr(s_x), _ptr(acc), M, N,
                                K, int(bool(staged)), bm, bn, _stream(dev))
    _check(st, "qgemm_w4a8_tiled")
    return y, x_q, s_x, acc


def smoothquant_factors(act_absmax: torch.Tensor, w: torch.Tensor, alpha: float = 0.5) -> torch.Tensor:
    """Per-input-channel smoothing factors s [K] f32 from calibration maxima of x and the dense weight w [N, K]."""
    N, K = w.shape
    s = torch.empty((K,), dtype=torch.float32, device=w.device)
    st = lib().smoothquant_factors(_ptr(act_absmax), _ptr(w), _dt(w), float(alpha), _ptr(s), N, K, _stream(w.device))
    _check(st, "smoothquant_factors")
    return s


def w4a8_quantize_weights(w: torch.Tensor, smooth: Optional[torch.Tensor] = None):
    """(w_q4 [N, K/8] int32, s_w [N] f16): the per-channel int4 weight, smoothing folded in when given."""
    N, K = w.shape
    wq = torch.empty((N, K // 8), dtype=torch.int32, device=w.device)
    sw = torch.empty((N,), dtype=torch.float16, device=w.device)
    st = lib().w4a8_quantize_weights(_ptr(w), _dt(w), _ptr(smooth), _ptr(wq), _ptr(sw), N, K, _stream(w.device))
    _check(st, "w4a8_quantize_weights")
    return wq, sw


def qgemm_w4a8_smooth(x: torch.Tensor, smooth: torch.Tensor, w_q4: torch.Tensor, s_w: torch.Tensor,
                      want_acc: bool = False):
    """qgemm_w4a8 on x / smooth: (y, x_q, s_x, acc or None)."""
    M, K = x.shape
    N = w_q4.shape[0]
    dev = x.device
    y = torch.empty((M, N), dtype=torch.float16, device=dev)
    x_q = torch.empty((M, K), dtype=torch.int8, device=dev)
    s_x = torch.empty((M,), dtype=torch.float32, device=dev)
    acc = torch.empty((M, N), dtype=torch.int32, device=dev) if want_acc else None
    st = lib().qgemm_w4a8_smooth(_ptr(x), _ptr(smooth), _ptr(_u32(w_q4)), _ptr(s_w), _ptr(y), _ptr(x_q), _ptr(s_x),
                                 _ptr(acc), M, N, K, _stream(dev))
    _check(st, "qgemm_w4a8_smooth")
    return y, x_q, s_x, acc


def qgemm_w4a8_codes(x_q: torch.Tensor, s_x: torch.Tensor, w_q4: torch.Tensor, s_w: torch.Tensor,
                     want_acc: bool = False, out: Optional[torch.Tensor] = None):
    """qgemm_w4a8 from int8 codes x_q [M, K] and scales s_x [M] (rmsnorm_w4a8): (y f16 [M, N], acc int32 or None)."""
    M, K = x_q.shape
    N = w_q4.shape[0]
    dev = x_q.device
    if x_q.dtype != torch.int8 or s_x.dtype != torch.float32 or s_w.dtype != torch.float16:
        raise ValueError("x_q must be int8, s_x float32 and s_w float16")
    _check_shapes(x_q, s_x=(s_x, (M,)), w_q4=(w_q4, (N, K // 8)), s_w=(s_w, (N,)))
    y = torch.empty((M, N), dtype=torch.float16, device=dev)
    if out is not None:
        y = _out(out, y)
    acc = torch.empty((M, N), dtype=torch.int32, device=dev) if want_acc else None
    _run("qgemm_w4a8_codes", dev, _ptr(x_q), _ptr(s_x), _ptr(_u32(w_q4)), _ptr(s_w), _ptr(y), _ptr(acc), M, N, K)
    return y, acc


def _norm(fn: str, x, weight, eps, resid, resid_out, *outputs):
    shape, dev, dt = x.shape, x.device, x.dtype
    M, K = shape
    if weight.shape != (K,) or weight.device != dev:
        _check_shapes(x, weight=(weight, (K,)))
    h, hp, rp, ldr, ldh = x, None, None, K, K
    if resid is not None:
        if resid.shape != shape or resid.device != dev:
            _check_shapes(x, resid=(resid, shape))
        if resid.dtype != dt or (resid_out is not None and resid_out.dtype != dt):
            raise ValueError("x, resid and resid_out must have one dtype")
        rp, ldr = _row_ptr(resid), resid.stride(0)
        if resid_out is None:
            h = torch.empty_like(x, memory_format=torch.contiguous_format)
            hp = h.data_ptr()
        else:
            h = resid_out
            _check_shapes(x, resid_out=(h, shape))
            hp, ldh = _row_ptr(h), h.stride(0)
    elif resid_out is not None:
        raise ValueError("resid_out without resid")
    ldx = x.stride(0)
    if M == 1:  # the stride of a single row means nothing
        ldx = ldr = ldh = K
    _run(fn, dev, _row_ptr(x), rp, _ptr(weight), eps, hp, *outputs, M, K, ldx, ldr, ldh, _dt(x), _dt(weight))
    return h


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, resid: Optional[torch.Tensor] = None,
            resid_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """(y, h): h = x + resid (x without resid), y = h / rms(h) * weight; x, resid, resid_out [M, K] with dense rows."""
    y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else _out(out, x)
    return y, _norm("rmsnorm", x, weight, eps, resid, resid_out, _ptr(y))


def rmsnorm_w4a8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, resid: Optional[torch.Tensor] = None,
                 resid_out: Optional[torch.Tensor] = None):
    """(x_q int8 [M, K], s_x f32 [M], h): rmsnorm's value quantized per row, for qgemm_w4a8_codes."""
    x_q = torch.empty_like(x, dtype=torch.int8, memory_format=torch.contiguous_format)
    s_x = x.new_empty(x.shape[0], dtype=torch.float32)
    return x_q, s_x, _norm("rmsnorm_w4a8", x, weight, eps, resid, resid_out, x_q.data_ptr(), s_x.data_ptr())


class AffineKVCache:
    """A paged key-value cache in the affine layout (qaff_kv_cache).

    `k` and `v` are triples (packed, scales, biases) of the caller's tensors:
    packed [num_pages, kv_heads, page_size, head_dim * bits / 32] int32,
    scales and biases [num_pages, kv_heads, page_size, head_dim / group_size]
    in bf16 or f16, the type of the keys, values and queries.  Holds
    references to them.  `AffineKVCache.empty` allocates them.
    """

    def __init__(self, k, v, group_size: int, bits: int):
        self.k, self.v = tuple(k), tuple(v)
        packed, scales = self.k[:2]
        if bits not in (2, 4, 8) or group_size not in (32, 64, 128):
            raise ValueError("bits must be 2, 4 or 8 and group_size 32, 64 or 128")
        pages, heads, size, words = packed.shape
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, size, words * 32 // bits
        self.group_size, self.bits, self.dtype, self.device = group_size, bits, scales.dtype, packed.device
        if self.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("scales must be bfloat16 or float16")
        rows = (pages, heads, size)
        for name, (p, s, b) in (("k", self.k), ("v", self.v)):
            _check_shapes(packed, **{name + " packed": (_u32(p), (*rows, words)),
                                     name + " scales": (s, (*rows, self.head_dim // group_size)),
                                     name + " biases": (b, (*rows, self.head_dim // group_size))})
            if s.dtype != self.dtype or b.dtype != self.dtype:
                raise ValueError("scales and biases must have one dtype")
        self.arrays = KVCacheArrays(*[_ptr(t) for t in self.k + self.v], pages, size, heads, self.head_dim, group_size,
                                    bits, DTYPE[self.dtype])
        self.ref = C.addressof(self.arrays)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int = 64, bits: int = 4,
              dtype=torch.bfloat16, device="cuda") -> "AffineKVCache":
        """A cache of zeros."""
        rows = (num_pages, kv_heads, page_size)
        k, v = ((torch.zeros((*rows, head_dim * bits // 32), dtype=torch.int32, device=device),
                 torch.zeros((*rows, head_dim // group_size), dtype=dtype, device=device),
                 torch.zeros((*rows, head_dim // group_size), dtype=dtype, device=device)) for _ in range(2))
        return cls(k, v, group_size, bits)


def kv_cache_append_affine(cache: AffineKVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k, v [T, kv_heads, head_dim] (rows dense) into slots [T] int64 of the cache; a slot outside is skipped."""
    dev = cache.device
    T, = slots.shape
    shape = (T, cache.kv_heads, cache.head_dim)
    if k.shape != shape or v.shape != shape or k.device != dev or v.device != dev or slots.device != dev:
        _check_shapes(cache.k[0], k=(k, shape), v=(v, shape), slots=(slots, (T,)))
    if k.dtype != cache.dtype or v.dtype != cache.dtype or slots.dtype != torch.int64:
        raise ValueError(f"k and v must be {cache.dtype}, slots int64")
    _run("kv_cache_append_affine", dev, cache.ref, _row_ptr(k), _row_ptr(v), *_strides(k), *_strides(v), _ptr(slots), T)


def kv_cache_read_affine(cache: AffineKVCache, slots: torch.Tensor, out=None):
    """(k, v) [T, kv_heads, head_dim] of slots [T] int64; a slot outside the cache reads as zeros."""
    T, = slots.shape
    if slots.dtype != torch.int64:
        raise ValueError("slots must be int64")
    if slots.device != cache.device:
        _check_shapes(cache.k[0], slots=(slots, (T,)))
    shape = (T, cache.kv_heads, cache.head_dim)
    if out is None:
        k, v = cache.k[1].new_empty(shape), cache.k[1].new_empty(shape)
    else:
        k, v = out
        for t in out:
            if t.shape != shape or t.dtype != cache.dtype or t.device != cache.device:
                raise ValueError(f"out must be two {shape} tensors of {cache.dtype} on {cache.device}")
    _run("kv_cache_read_affine", cache.device, cache.ref, _ptr(slots), _ptr(k), _ptr(v), T)
    return k, v


def paged_attention_affine(q: torch.Tensor, cache: AffineKVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                           scale: Optional[float] = None, window: int = 0,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token a sequence, q [B, heads, head_dim] (rows dense), over the cached tokens.

    page_table [B, max_pages] int32 (rows dense), seq_lens [B] int32; scale
    defaults to head_dim ** -0.5; window > 0 keeps the last `window` tokens.
    """
    dev = cache.device
    B, heads, D = q.shape
    per = page_table.shape[-1]
    if (D != cache.head_dim or page_table.shape != (B, per) or seq_lens.shape != (B,) or q.device != dev
            or page_table.device != dev or seq_lens.device != dev):
        _check_shapes(cache.k[0], q=(q, (B, heads, cache.head_dim)), page_table=(page_table, (B, per)), seq_lens=(seq_lens, (B,)))
    if q.dtype != cache.dtype or page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError(f"q must be {cache.dtype}, page_table and seq_lens int32")
    o = _out(out, q)
    _run("paged_attention_affine", dev, cache.ref, _row_ptr(q), *_strides(q), _row_ptr(page_table),
         page_table.stride(0) if B > 1 else per, per, _ptr(seq_lens), _ptr(o), B, heads,
         D ** -0.5 if scale is None else scale, window)
    return o


class KVPagePool:
    """The free pages of a paged cache: a stack that kv_pages_assign takes from and kv_pages_trim returns to.

    free_pages [num_pages] int32, of which the first state[0] are free; state
    [4] int32: free pages, pages short at the last assign, the library's word.
    Made with every page free, page 0 on top.
    """

    def __init__(self, num_pages: int, page_size: int, device="cuda"):
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.free_pages = torch.arange(self.num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.state = torch.zeros(4, dtype=torch.int32, device=device)
        self.state[0] = self.num_pages
        self.device = self.free_pages.device


def _pages(fn: str, pool: KVPagePool, page_table, seq_lens, other, lens_out, *outputs):
    dev = pool.device
    B, per = page_table.shape
    if (page_table.device != dev or seq_lens.shape != (B,) or seq_lens.device != dev or other.shape != (B,)
            or other.device != dev):
        _check_shapes(pool.state, page_table=(page_table, (B, per)), lengths=(seq_lens, (B,)), new_or_kept=(other, (B,)))
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or other.dtype != torch.int32:
        raise ValueError("page_table and lengths must be int32")
    free, state = pool.free_pages, pool.state
    if (free.shape != (pool.num_pages,) or state.shape != (4,) or free.dtype != torch.int32 or state.dtype != torch.int32
            or free.device != dev or state.device != dev):
        raise ValueError("the pool's free_pages and state must stay as they were made")
    lens_out = _out(lens_out, seq_lens)
    _run(fn, dev, _row_ptr(page_table), page_table.stride(0) if B > 1 else per, per, _ptr(seq_lens), _ptr(other),
         _ptr(lens_out), _ptr(free), _ptr(state), pool.num_pages, pool.page_size, B, *outputs)
    return lens_out


def kv_pages_assign(pool: KVPagePool, page_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, rows: int,
                    lens_out: Optional[torch.Tensor] = None):
    """Pages for new_lens [B] int32 further tokens of every sequence: (slots int64, positions int32, seq_ids int32 [rows], lens).

    page_table [B, max_pages] int32 (rows dense) gets the new pages; lens [B]
    are the lengths with them (lens_out, which may be seq_lens itself).  Rows
    lists the new tokens sequence by sequence; the ones behind the last get
    slot -1, position 0 and sequence -1.
    """
    new = pool.state.new_empty
    slots, positions, seq_ids = new(rows, dtype=torch.int64), new(rows), new(rows)
    lens = _pages("kv_pages_assign", pool, page_table, seq_lens, new_lens, lens_out, slots.data_ptr(), positions.data_ptr(),
                  seq_ids.data_ptr(), rows)
    return slots, positions, seq_ids, lens


def kv_pages_trim(pool: KVPagePool, page_table: torch.Tensor, seq_lens: torch.Tensor, keep_lens: torch.Tensor,
                  lens_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every sequence keeps its first keep_lens [B] tokens (0: it ends); the pages behind them return to the pool."""
    return _pages("kv_pages_trim", pool, page_table, seq_lens, keep_lens, lens_out)


ROTARY_SCALINGS = {None: 0, "linear": 1, "base": 2, "bands": 3}


class Rotary:
    """Rotary positions (qaff_rotary): inv_freq [rotary_dim / 2] float64 on the GPU, radians a position of each pair.

    Pairs are columns (j, j + rotary_dim / 2), or (2j, 2j + 1) when
    interleaved; magnitude multiplies both turned tensors.  Holds a reference
    to inv_freq.  `Rotary.make` computes the frequencies.
    """

    def __init__(self, inv_freq: torch.Tensor, interleaved: bool = False, magnitude: float = 1.0):
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a vector of float64")
        self.inv_freq, self.interleaved, self.magnitude = inv_freq, bool(interleaved), float(magnitude)
        self.rotary_dim, self.device = 2 * inv_freq.shape[0], inv_freq.device
        self.spec = RotarySpec(_ptr(inv_freq), self.rotary_dim, int(self.interleaved), self.magnitude)
        self.ref = C.addressof(self.spec)

    @classmethod
    def make(cls, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: Optional[str] = None,
             factor: float = 1.0, original_len: float = 0.0, low: float = 1.0, high: float = 4.0, magnitude: float = 1.0,
             device="cuda") -> "Rotary":
        """base^(-2j / rotary_dim), scaled: None, "linear", "base" or "bands" (rotary_frequencies in include/qaff.h)."""
        if scaling not in ROTARY_SCALINGS:
            raise ValueError(f"unknown scaling {scaling!r}")
        f = torch.empty(rotary_dim // 2, dtype=torch.float64, device=device)
        _run("rotary_frequencies", f.device, _ptr(f), rotary_dim, base, ROTARY_SCALINGS[scaling], factor, original_len, low,
             high)
        return cls(f, interleaved, magnitude)


def _check_positions(first: torch.Tensor, rot: Rotary, positions: torch.Tensor):
    if positions.shape != first.shape[:1] or positions.device != first.device or rot.device != first.device:
        _check_shapes(first, positions=(positions, first.shape[:1]), inv_freq=(rot.inv_freq, rot.inv_freq.shape))
    if positions.dtype != torch.int32:
        raise ValueError("positions must be int32")


def rotary(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, rot: Rotary, q_out: Optional[torch.Tensor] = None,
           k_out: Optional[torch.Tensor] = None):
    """(q_out, k_out): q [T, heads, D] and k [T, kv_heads, D] (rows dense) turned by positions [T] int32.

    An output may be its input (turned in place); strides of both are free.
    """
    T, H, D = q.shape
    HK = k.shape[1]
    if k.shape != (T, HK, D) or k.device != q.device:
        _check_shapes(q, k=(k, (T, HK, D)))
    if k.dtype != q.dtype:
        raise ValueError("q and k must have one dtype")
    _check_positions(q, rot, positions)
    qo, ko = _out(q_out, q), _out(k_out, k)
    _run("rotary", q.device, rot.ref, *_rows(q), *_rows(k), *_rows(qo, q_out is None), *_rows(ko, k_out is None),
         _ptr(positions), T, H, HK, D, _dt(q))
    return qo, ko


def kv_cache_append_rotary_affine(cache: AffineKVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  positions: torch.Tensor, slots: torch.Tensor, rot: Rotary,
                                  q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rotary and kv_cache_append_affine in one launch: q turned (q_out), the turned k and v into slots [T] int64."""
    dev = cache.device
    T, H, D = q.shape
    shape = (T, cache.kv_heads, cache.head_dim)
    if (D != cache.head_dim or k.shape != shape or v.shape != shape or slots.shape != (T,) or q.device != dev
            or k.device != dev or v.device != dev or slots.device != dev):
        _check_shapes(cache.k[0], q=(q, (T, H, cache.head_dim)), k=(k, shape), v=(v, shape), slots=(slots, (T,)))
    if q.dtype != cache.dtype or k.dtype != cache.dtype or v.dtype != cache.dtype or slots.dtype != torch.int64:
        raise ValueError(f"q, k and v must be {cache.dtype}, slots int64")
    _check_positions(q, rot, positions)
    o = _out(q_out, q)
    _run("kv_cache_append_rotary_affine", dev, cache.ref, rot.ref, *_rows(q), *_rows(k), *_rows(v), *_rows(o, q_out is None),
         _ptr(positions), _ptr(slots), T, H)
    return o


class AffineExperts:
    """The experts of a mixture-of-experts block in the affine layout (qaff_experts).

    `gate_up` and `down` are triples (packed, scales, biases): packed
    [E, 2 * inner, hidden * bits / 32] (the gate's rows, then up's) and
    [E, hidden, inner * bits / 32] int32, scales and biases [.., columns /
    group_size] in bf16 or f16, the type of the activations.  Holds references
    to them.
    """

    def __init__(self, gate_up, down, group_size: int, bits: int):
        self.gate_up, self.down = tuple(gate_up), tuple(down)
        if bits not in (2, 4, 8) or group_size not in (32, 64, 128):
            raise ValueError("bits must be 2, 4 or 8 and group_size 32, 64 or 128")
        first = self.gate_up[0]
        E, rows, words = first.shape
        self.num_experts, self.hidden, self.inner = E, words * 32 // bits, rows // 2
        self.group_size, self.bits, self.dtype, self.device = group_size, bits, self.gate_up[1].dtype, first.device
        if self.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("scales must be bfloat16 or float16")
        if rows % 2:
            raise ValueError("gate_up must hold as many rows of up as of the gate")
        for name, (p, s, b), n, k in (("gate_up", self.gate_up, rows, self.hidden), ("down", self.down, self.hidden, self.inner)):
            _check_shapes(first, **{name + " packed": (_u32(p), (E, n, k * bits // 32)),
                                    name + " scales": (s, (E, n, k // group_size)),
                                    name + " biases": (b, (E, n, k // group_size))})
            if s.dtype != self.dtype or b.dtype != self.dtype:
                raise ValueError("scales and biases must have one dtype")
        self.arrays = ExpertArrays(*[_ptr(t) for t in self.gate_up + self.down], self.hidden, self.inner, E, group_size, bits,
                                   DTYPE[self.dtype])
        self.ref = C.addressof(self.arrays)


def qmoe_affine(x: torch.Tensor, logits: torch.Tensor, experts: AffineExperts, top_k: int, renormalize: bool = True,
                scale: float = 1.0, resid: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = resid + scale * sum_e p_e Down_e(silu(Gate_e x) * (Up_e x)) over the top_k experts of each row.

    x [M, hidden], logits [M, E] float32 or x's type (ties go to the lowest
    index, minus infinity is never chosen); p is the softmax over the chosen
    (renormalize) or over all experts.  M is at most 256.  out may be resid.
    """
    dev = experts.device
    M = x.shape[0]
    shape = (M, experts.hidden)
    if x.shape != shape or x.device != dev or logits.shape != (M, experts.num_experts) or logits.device != dev:
        _check_shapes(experts.down[0], x=(x, shape), logits=(logits, (M, experts.num_experts)))
    if x.dtype != experts.dtype or (resid is not None and resid.dtype != x.dtype):
        raise ValueError(f"x and resid must be {experts.dtype}")
    if resid is not None:
        _check_shapes(x, resid=(resid, shape))
    y = _out(out, x)
    _run("qmoe_affine", dev, experts.ref, _ptr(x), _ptr(logits), _dt(logits), _ptr(resid), _ptr(y), M, top_k,
         int(bool(renormalize)), scale)
    return y


def gptq_to_affine_repack(qweight: torch.Tensor, qzeros: torch.Tensor, scales: torch.Tensor,
                          g_idx: Optional[torch.Tensor], group_size: int, bias_dtype=torch.float32):
    """Returns (w_packed [N,K/8] int32, scales [N,K/G] f16, biases [N,K/G] bias_dtype, k_perm [K] int32)."""
    K = qweight.shape[0] * 8
    N = qweight.shape[1]
    dev = qweight.device
    w = torch.empty((N, K // 8), dtype=torch.int32, device=dev)
    s = torch.empty((N, K // group_size), dtype=torch.float16, device=dev)
    b = torch.empty((N, K // group_size), dtype=bias_dtype, device=dev)
    kp = torch.empty((K,), dtype=torch.int32, device=dev)
    st = lib().gptq_to_affine_repack(_ptr(qweight), _ptr(qzeros), _ptr(scales), _ptr(g_idx), _ptr(w), _ptr(s),
                                     _ptr(b), DTYPE[bias_dtype], _ptr(kp), K, N, group_size, _stream(dev))
    _check(st, "gptq_to_affine_repack")
    return w, s, b, kp


def dequantize_affine(w_packed: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, K: int, group_size: int,
                      bits: int, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The dense weight [N, K] in out_dtype: code*scale + bias, rounded once."""
    N = w_packed.shape[0]
    o = out if out is not None else torch.empty((N, K), dtype=out_dtype, device=w_packed.device)
    st = lib().dequantize_affine(_ptr(_u32(w_packed)), _ptr(scales), _ptr(biases), _ptr(o), N, K, group_size, bits,
                                 _dt(scales), _dt(biases), _dt(o), _stream(w_packed.device))
    _check(st, "dequantize_affine")
    return o


def stream_read(buf: torch.Tensor, sink: torch.Tensor, blocks: int) -> None:
    """Measurement helper: read all of `buf` once (qaff_stream_read)."""
    st = lib().qaff_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), blocks, _stream(buf.device))
    _check(st, "qaff_stream_read")


def release_workspaces() -> int:
    """Free the scratch the library holds (qaff_release_workspaces).  Call it
    only with no library work pending on any stream and no captured graph
    that will replay a library call.  Returns the bytes of the per-stream
    buffers that were cached."""
    freed = C.c_uint64(0)
    _check(lib().qaff_release_workspaces(C.byref(freed)), "qaff_release_workspaces")
    return int(freed.value)


def quantize_pack_affine(w: torch.Tensor, group_size: int, bits: int, sb_dtype=torch.bfloat16):
    """Returns (w_packed [N, K*bits/32] int32, scales [N,K/G], biases [N,K/G])."""
    N, K = w.shape
    dev = w.device
    packed = torch.empty((N, K * bits // 32), dtype=torch.int32, device=dev)
    s = torch.empty((N, K // group_size), dtype=sb_dtype, device=dev)
    b = torch.empty((N, K // group_size), dtype=sb_dtype, device=dev)
    st = lib().quantize_pack_affine(_ptr(w), _dt(w), _ptr(packed), _ptr(s), _ptr(b), DTYPE[sb_dtype], N, K,
                                    group_size, bits, _stream(dev))
    _check(st, "quantize_pack_affine")
    return packed, s, b
