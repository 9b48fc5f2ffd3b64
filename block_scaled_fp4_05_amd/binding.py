"""ctypes binding of libfp4q -- argument marshalling only.

Each ``fp4q_*`` function here has the name and argument order of the C entry point
in include/fp4q.h.  Device buffers are passed as torch CUDA tensors (or None for a
NULL pointer), the stream defaults to torch's current stream, and a non-OK status
raises :class:`Fp4qError`.  Every quantization step runs in the HIP library; if
libfp4q.so is missing, loading fails loudly -- there is no fallback.

The ``quantize_*`` / ``dequantize`` / ``rht`` helpers below only allocate the output
tensors with torch and call the same-name entry points.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp4q.so")

F32, BF16 = 0, 1
RTN, SR = 0, 1
FMT_NVFP4, FMT_NVFP4_2D, FMT_MXFP4, FMT_IF4 = 0, 1, 2, 3
ROWWISE, COLWISE = 1, 2
AMAX_COMPUTE, AMAX_GIVEN = 0, 1
STATUS = {0: "FP4Q_OK", 1: "FP4Q_E_NULL", 2: "FP4Q_E_SHAPE", 3: "FP4Q_E_ALIGN", 4: "FP4Q_E_ARG", 5: "FP4Q_E_HIP"}

EXPORTS = ["fp4q_workspace_create", "fp4q_workspace_destroy", "fp4q_workspace_set_wait", "fp4q_workspace_fallbacks",
           "fp4q_quantize_nvfp4", "fp4q_quantize_nvfp4_noalloc", "fp4q_quantize_nvfp4_2d", "fp4q_quantize_mxfp4", "fp4q_quantize_mxfp6",
           "fp4q_quantize_if4", "fp4q_quantize_variant", "fp4q_dequantize_variant", "fp4q_rht", "fp4q_gemm_mxfp4", "fp4q_gemm_nvfp4", "fp4q_dequantize", "fp4q_amax",
           "fp4q_rht_signs_from_seed", "fp4q_status_string", "fp4q_abi_version",
           "fp4q_quantize_mxfp8", "fp4q_dequantize_mxfp8", "fp4q_rmsnorm_mxfp8", "fp4q_rmsnorm_backward",
           "fp4q_rmsnorm_backward_scratch", "fp4q_gemm_mxfp8_mxfp4", "fp4q_moe_mxfp4",
           "fp4q_moe_scratch"]


class Fp4qError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


_lib = None
_P, _I64, _U64, _I, _U = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_uint
_F = ctypes.c_float


def lib() -> ctypes.CDLL:
    """Load libfp4q.so (built in-tree by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with block_scaled_fp4_05_amd/build.py "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "fp4q_workspace_create": [_P],
            "fp4q_workspace_destroy": [_P],
            "fp4q_workspace_set_wait": [_P, _U],
            "fp4q_workspace_fallbacks": [_P, _P, _P],
            "fp4q_quantize_nvfp4": [_P, _I, _I64, _I64, _U, _I, _U64, _P, _U, _P, _P, _P, _P, _P, _P, _P, _P],
            "fp4q_quantize_nvfp4_noalloc": [_P, _I, _I64, _I64, _U, _I, _U64, _P, _U, _P, _P, _P, _P, _P, _P, _P],
            "fp4q_quantize_nvfp4_2d": [_P, _I, _I64, _I64, _U, _P, _P, _P, _P, _P, _P, _P],
            "fp4q_quantize_mxfp4": [_P, _I, _I64, _I64, _I, _U64, _P, _P, _P, _P, _P],
            "fp4q_quantize_mxfp6": [_P, _I, _I64, _I64, _I, _P, _P, _P],
            "fp4q_quantize_if4": [_P, _I, _I64, _I64, _U, _P, _P, _P, _P, _P, _P],
            "fp4q_quantize_variant": [_P, _I, _I64, _I64, _I, _U, _P, _P, _P, _P, _P, _P],
            "fp4q_dequantize_variant": [_I, _P, _P, _P, _I64, _I64, _I, _P, _P],
            "fp4q_rht": [_P, _I, _I64, _I64, _P, _I, _P, _P],
            "fp4q_gemm_mxfp4": [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P],
            "fp4q_gemm_nvfp4": [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _U, _I, _P, _P, _P],
            "fp4q_dequantize": [_I, _P, _P, _P, _I64, _I64, _I, _P, _P],
            "fp4q_amax": [_P, _I, _I64, _I64, _P, _P],
            "fp4q_rht_signs_from_seed": [_U64, _P],
            "fp4q_status_string": [_I],
            "fp4q_abi_version": [],
            "fp4q_quantize_mxfp8": [_P, _I, _I64, _I64, _P, _P, _P],
            "fp4q_dequantize_mxfp8": [_P, _P, _I64, _I64, _I, _P, _P],
            "fp4q_rmsnorm_mxfp8": [_P, _P, _I, _I64, _I64, _P, _F, _P, _P, _P, _P, _P, _P],
            "fp4q_rmsnorm_backward": [_P, _P, _P, _I, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P],
            "fp4q_rmsnorm_backward_scratch": [_I64, _I64],
            "fp4q_gemm_mxfp8_mxfp4": [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P],
            "fp4q_moe_mxfp4": [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _U, _P, _P, _I, _P,
                               _P, _I64, _P],
            "fp4q_moe_scratch": [_I64, _I64, _I64, _I64, _I64],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _I
        L.fp4q_rht_signs_from_seed.restype = None
        L.fp4q_rmsnorm_backward_scratch.restype = _I64
        L.fp4q_moe_scratch.restype = _I64
        L.fp4q_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, Workspace):
        return t.handle
    return t.data_ptr()


def _s(stream) -> int | None:
    if stream is None:   # the handle alone, by torch's own call for it: a Stream object takes 2.6 us, a third of a small call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int) -> int:
    if status != 0:
        raise Fp4qError(fn, status)
    return status


def _signs_arg(signs):
    if signs is None:
        return None, None
    arr = (ctypes.c_uint32 * 4)(*[int(v) & 0xFFFFFFFF for v in signs])
    return ctypes.addressof(arr), arr


# --- workspaces ----------------------------------------------------------------------

class Workspace:
    """A libfp4q workspace (fp4q_workspace_create on the current device).  close()
    destroys it; the caller makes sure no enqueued work still uses it."""

    def __init__(self):
        h = ctypes.c_void_p(0)
        _check("fp4q_workspace_create", lib().fp4q_workspace_create(ctypes.addressof(h)))
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            _check("fp4q_workspace_destroy", lib().fp4q_workspace_destroy(self.handle))
            self.handle = None


_ws_cache: dict = {}


def stream_workspace(stream=None) -> Workspace:
    """The helpers' workspace for (current device, stream), created on first use and kept
    for the life of the process (create one yourself, or pass ws=None, where a call must
    not allocate, e.g. inside graph capture)."""
    key = (torch.cuda.current_device(), _s(stream))
    w = _ws_cache.get(key)
    if w is None:
        w = _ws_cache[key] = Workspace()
    return w


def _ws(ws, stream):
    return stream_workspace(stream) if isinstance(ws, str) and ws == "auto" else ws


# --- the C entry points, same names -----------------------------------------------

def fp4q_workspace_set_wait(ws: Workspace, microseconds: int) -> int:
    return _check("fp4q_workspace_set_wait", lib().fp4q_workspace_set_wait(_p(ws), microseconds))


def fp4q_workspace_fallbacks(ws: Workspace, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check("fp4q_workspace_fallbacks", lib().fp4q_workspace_fallbacks(_p(ws), _s(stream), ctypes.addressof(out)))
    return out.value


def fp4q_quantize_nvfp4(x, dt, rows, cols, layouts, rnd, sr_seed, rht_signs, amax_mode, amax, tensor_scale,
                        row_codes, row_scales, col_codes, col_scales, ws=None, stream=None) -> int:
    sp, _keep = _signs_arg(rht_signs)
    return _check("fp4q_quantize_nvfp4", lib().fp4q_quantize_nvfp4(
        _p(x), dt, rows, cols, layouts, rnd, sr_seed, sp, amax_mode, _p(amax), _p(tensor_scale),
        _p(row_codes), _p(row_scales), _p(col_codes), _p(col_scales), _p(ws), _s(stream)))


def fp4q_quantize_nvfp4_noalloc(x, dt, rows, cols, layouts, rnd, sr_seed, rht_signs, amax_mode, amax, tensor_scale,
                                row_codes, row_scales, col_codes, col_scales, stream=None) -> int:
    sp, _keep = _signs_arg(rht_signs)
    return _check("fp4q_quantize_nvfp4_noalloc", lib().fp4q_quantize_nvfp4_noalloc(
        _p(x), dt, rows, cols, layouts, rnd, sr_seed, sp, amax_mode, _p(amax), _p(tensor_scale),
        _p(row_codes), _p(row_scales), _p(col_codes), _p(col_scales), _s(stream)))


def fp4q_quantize_nvfp4_2d(x, dt, rows, cols, amax_mode, amax, tensor_scale, codes, scales, codes_t,
                           ws=None, stream=None) -> int:
    return _check("fp4q_quantize_nvfp4_2d", lib().fp4q_quantize_nvfp4_2d(
        _p(x), dt, rows, cols, amax_mode, _p(amax), _p(tensor_scale), _p(codes), _p(scales), _p(codes_t),
        _p(ws), _s(stream)))


def fp4q_quantize_mxfp4(x, dt, rows, cols, rnd, sr_seed, codes, scales, amax=None, ws=None, stream=None) -> int:
    return _check("fp4q_quantize_mxfp4", lib().fp4q_quantize_mxfp4(
        _p(x), dt, rows, cols, rnd, sr_seed, _p(codes), _p(scales), _p(amax), _p(ws), _s(stream)))


def fp4q_quantize_mxfp6(x, dt, rows, cols, fmt, codes, scales, stream=None) -> int:
    return _check("fp4q_quantize_mxfp6", lib().fp4q_quantize_mxfp6(
        _p(x), dt, rows, cols, fmt, _p(codes), _p(scales), _s(stream)))


def fp4q_quantize_if4(x, dt, rows, cols, amax_mode, amax, tensor_scale, codes, scales, ws=None,
                      stream=None) -> int:
    return _check("fp4q_quantize_if4", lib().fp4q_quantize_if4(
        _p(x), dt, rows, cols, amax_mode, _p(amax), _p(tensor_scale), _p(codes), _p(scales), _p(ws), _s(stream)))


def fp4q_quantize_variant(x, dt, rows, cols, var, amax_mode, amax, tensor_scale, codes, scales, ws=None,
                          stream=None) -> int:
    return _check("fp4q_quantize_variant", lib().fp4q_quantize_variant(
        _p(x), dt, rows, cols, var, amax_mode, _p(amax), _p(tensor_scale), _p(codes), _p(scales), _p(ws),
        _s(stream)))


def fp4q_dequantize_variant(var, codes, scales, tensor_scale, rows, cols, out_dt, y, stream=None) -> int:
    return _check("fp4q_dequantize_variant", lib().fp4q_dequantize_variant(
        var, _p(codes), _p(scales), _p(tensor_scale), rows, cols, out_dt, _p(y), _s(stream)))


def fp4q_rht(x, dt, rows, cols, signs, inverse, y, stream=None) -> int:
    sp, _keep = _signs_arg(signs)
    return _check("fp4q_rht", lib().fp4q_rht(_p(x), dt, rows, cols, sp, int(inverse), _p(y), _s(stream)))


def fp4q_gemm_mxfp4(a_codes, a_scales, b_codes, b_scales, m, n, k, out_dt, c, amax=None, stream=None) -> int:
    return _check("fp4q_gemm_mxfp4", lib().fp4q_gemm_mxfp4(
        _p(a_codes), _p(a_scales), _p(b_codes), _p(b_scales), m, n, k, out_dt, _p(c), _p(amax), _s(stream)))


TILES_A, TILES_B, IF4_A, IF4_B = 1, 2, 4, 8


def fp4q_gemm_nvfp4(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, m, n, k, operand_flags, out_dt, c, amax=None,
                    stream=None) -> int:
    return _check("fp4q_gemm_nvfp4", lib().fp4q_gemm_nvfp4(
        _p(a_codes), _p(a_scales), _p(a_ts), _p(b_codes), _p(b_scales), _p(b_ts), m, n, k, operand_flags, out_dt,
        _p(c), _p(amax), _s(stream)))


def fp4q_dequantize(fmt, codes, scales, tensor_scale, rows, cols, out_dt, y, stream=None) -> int:
    return _check("fp4q_dequantize", lib().fp4q_dequantize(
        fmt, _p(codes), _p(scales), _p(tensor_scale), rows, cols, out_dt, _p(y), _s(stream)))


def fp4q_amax(x, dt, rows, cols, amax, stream=None) -> int:
    return _check("fp4q_amax", lib().fp4q_amax(_p(x), dt, rows, cols, _p(amax), _s(stream)))


def fp4q_rht_signs_from_seed(seed: int) -> list[int]:
    out = (ctypes.c_uint32 * 4)()
    lib().fp4q_rht_signs_from_seed(seed, ctypes.addressof(out))
    return list(out)


def fp4q_status_string(status: int) -> str:
    return lib().fp4q_status_string(status).decode()


def fp4q_abi_version() -> int:
    return lib().fp4q_abi_version()


def fp4q_quantize_mxfp8(x, dt, rows, cols, codes, scales, stream=None) -> int:
    return _check("fp4q_quantize_mxfp8", lib().fp4q_quantize_mxfp8(
        _p(x), dt, rows, cols, _p(codes), _p(scales), _s(stream)))


def fp4q_dequantize_mxfp8(codes, scales, rows, cols, out_dt, y, stream=None) -> int:
    return _check("fp4q_dequantize_mxfp8", lib().fp4q_dequantize_mxfp8(
        _p(codes), _p(scales), rows, cols, out_dt, _p(y), _s(stream)))


def fp4q_rmsnorm_mxfp8(x, residual, dt, rows, cols, gain, eps, codes, scales, sum, rstd, y, stream=None) -> int:
    return _check("fp4q_rmsnorm_mxfp8", lib().fp4q_rmsnorm_mxfp8(
        _p(x), _p(residual), dt, rows, cols, _p(gain), eps, _p(codes), _p(scales), _p(sum), _p(rstd), _p(y),
        _s(stream)))


def fp4q_rmsnorm_backward_scratch(rows: int, cols: int) -> int:
    return lib().fp4q_rmsnorm_backward_scratch(rows, cols)


def fp4q_rmsnorm_backward(dy, s, dsum, dt, rows, cols, gain, rstd, dx, dgain, scratch, scratch_bytes,
                          stream=None) -> int:
    return _check("fp4q_rmsnorm_backward", lib().fp4q_rmsnorm_backward(
        _p(dy), _p(s), _p(dsum), dt, rows, cols, _p(gain), _p(rstd), _p(dx), _p(dgain), _p(scratch), scratch_bytes,
        _s(stream)))


def fp4q_gemm_mxfp8_mxfp4(a_codes, a_scales, b_codes, b_scales, m, n, k, out_dt, c, stream=None) -> int:
    return _check("fp4q_gemm_mxfp8_mxfp4", lib().fp4q_gemm_mxfp8_mxfp4(
        _p(a_codes), _p(a_scales), _p(b_codes), _p(b_scales), m, n, k, out_dt, _p(c), _s(stream)))


ROUTE_COMPUTE, ROUTE_GIVEN = 0, 1


def fp4q_moe_mxfp4(x_codes, x_scales, router_x, router_w, router_dt, w13_codes, w13_scales, w2_codes, w2_scales,
                   tokens, d, hidden, experts, topk, route_mode, ids, weights, out_dt, y, scratch, scratch_bytes,
                   stream=None) -> int:
    return _check("fp4q_moe_mxfp4", lib().fp4q_moe_mxfp4(
        _p(x_codes), _p(x_scales), _p(router_x), _p(router_w), router_dt, _p(w13_codes), _p(w13_scales),
        _p(w2_codes), _p(w2_scales), tokens, d, hidden, experts, topk, route_mode, _p(ids), _p(weights), out_dt,
        _p(y), _p(scratch), scratch_bytes, _s(stream)))


def fp4q_moe_scratch(tokens: int, d: int, hidden: int, experts: int, topk: int) -> int:
    return lib().fp4q_moe_scratch(tokens, d, hidden, experts, topk)


# --- allocation helpers --------------------------------------------------------------

def _dt(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise TypeError(f"libfp4q takes bfloat16 or float32 input, got {x.dtype}")


def _u8(*shape, device):
    return torch.empty(*shape, dtype=torch.uint8, device=device)


def quantize_nvfp4(x: torch.Tensor, layouts: int = ROWWISE | COLWISE, rnd: int = RTN, sr_seed: int = 0,
                   rht_signs=None, amax: torch.Tensor | None = None, ws="auto", stream=None) -> dict:
    """NVFP4 1x16.  If `amax` is given it is used as the tensor amax (AMAX_GIVEN).
    ws: "auto" (the stream's cached workspace), None (no workspace) or a Workspace."""
    rows, cols = x.shape
    dev = x.device
    out = {"tensor_scale": torch.empty(1, dtype=torch.float32, device=dev)}
    mode = AMAX_GIVEN if amax is not None else AMAX_COMPUTE
    out["amax"] = amax if amax is not None else torch.empty(1, dtype=torch.float32, device=dev)
    rc = rs = cc = cs = None
    if layouts & ROWWISE:
        rc, rs = _u8(rows, cols // 2, device=dev), _u8(rows, cols // 16, device=dev)
        out["row_codes"], out["row_scales"] = rc, rs
    if layouts & COLWISE:
        cc, cs = _u8(cols, rows // 2, device=dev), _u8(cols, rows // 16, device=dev)
        out["col_codes"], out["col_scales"] = cc, cs
    fp4q_quantize_nvfp4(x, _dt(x), rows, cols, layouts, rnd, sr_seed, rht_signs, mode, out["amax"],
                        out["tensor_scale"], rc, rs, cc, cs, _ws(ws, stream), stream)
    return out


def quantize_nvfp4_2d(x: torch.Tensor, transposed: bool = False, amax: torch.Tensor | None = None,
                      ws="auto", stream=None) -> dict:
    """NVFP4 16x16.  If `amax` is given it is used as the tensor amax (AMAX_GIVEN)."""
    rows, cols = x.shape
    dev = x.device
    mode = AMAX_GIVEN if amax is not None else AMAX_COMPUTE
    out = {"amax": amax if amax is not None else torch.empty(1, dtype=torch.float32, device=dev),
           "tensor_scale": torch.empty(1, dtype=torch.float32, device=dev),
           "codes": _u8(rows, cols // 2, device=dev), "scales": _u8(rows // 16, cols // 16, device=dev),
           "codes_t": _u8(cols, rows // 2, device=dev) if transposed else None}
    fp4q_quantize_nvfp4_2d(x, _dt(x), rows, cols, mode, out["amax"], out["tensor_scale"], out["codes"],
                           out["scales"], out["codes_t"], _ws(ws, stream), stream)
    return out


def quantize_mxfp4(x: torch.Tensor, rnd: int = RTN, sr_seed: int = 0, with_amax: bool = False,
                   ws="auto", stream=None) -> dict:
    rows, cols = x.shape
    dev = x.device
    out = {"codes": _u8(rows, cols // 2, device=dev), "scales": _u8(rows, cols // 32, device=dev)}
    if with_amax:
        out["amax"] = torch.empty(1, dtype=torch.float32, device=dev)
    fp4q_quantize_mxfp4(x, _dt(x), rows, cols, rnd, sr_seed, out["codes"], out["scales"], out.get("amax"),
                        _ws(ws, stream) if with_amax else None, stream)
    return out


FP6_E2M3, FP6_E3M2 = 0, 1
FMT_MXFP6 = {FP6_E2M3: 4, FP6_E3M2: 5}


def quantize_mxfp6(x: torch.Tensor, fmt: int = FP6_E2M3, stream=None) -> dict:
    """MX FP6: codes [rows][3 cols / 4] (four per three bytes), E8M0 scales [rows][cols/32]."""
    rows, cols = x.shape
    dev = x.device
    out = {"codes": _u8(rows, cols // 4 * 3, device=dev), "scales": _u8(rows, cols // 32, device=dev)}
    fp4q_quantize_mxfp6(x, _dt(x), rows, cols, fmt, out["codes"], out["scales"], stream)
    return out


def quantize_if4(x: torch.Tensor, amax: torch.Tensor | None = None, ws="auto", stream=None) -> dict:
    """IF4.  If `amax` is given it is used as the tensor amax (AMAX_GIVEN)."""
    rows, cols = x.shape
    dev = x.device
    mode = AMAX_GIVEN if amax is not None else AMAX_COMPUTE
    out = {"amax": amax if amax is not None else torch.empty(1, dtype=torch.float32, device=dev),
           "tensor_scale": torch.empty(1, dtype=torch.float32, device=dev),
           "codes": _u8(rows, cols // 2, device=dev), "scales": _u8(rows, cols // 16, device=dev)}
    fp4q_quantize_if4(x, _dt(x), rows, cols, mode, out["amax"], out["tensor_scale"], out["codes"],
                      out["scales"], _ws(ws, stream), stream)
    return out


def rht(x: torch.Tensor, signs, inverse: bool = False, stream=None) -> torch.Tensor:
    rows, cols = x.shape
    y = torch.empty(rows, cols, dtype=torch.float32, device=x.device)
    fp4q_rht(x, _dt(x), rows, cols, signs, inverse, y, stream)
    return y


def gemm_mxfp4(a: dict, b: dict, out_dtype=torch.float32, amax: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """C = A B^T for two row-wise MXFP4 operands as quantize_mxfp4 returns them.

    With ``amax`` (a one-element float32 device tensor) the GEMM also writes max |C| of
    the stored outputs there."""
    m, n, k = a["codes"].shape[0], b["codes"].shape[0], a["codes"].shape[1] * 2
    c = torch.empty(m, n, dtype=out_dtype, device=a["codes"].device)
    fp4q_gemm_mxfp4(a["codes"], a["scales"], b["codes"], b["scales"], m, n, k, _dt(c), c, amax, stream)
    return c


def gemm_nvfp4(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, out_dtype=torch.float32,
               amax: torch.Tensor | None = None, operand_flags: int = 0, stream=None) -> torch.Tensor:
    """C = A B^T / (gs_a gs_b) for two row-wise NVFP4 or IF4 operands (codes, scales, tensor
    scale); ``operand_flags`` marks operands with 16x16 scale tiles (TILES_A, TILES_B) and IF4
    operands (IF4_A, IF4_B); ``amax`` as for gemm_mxfp4."""
    m, n, k = a_codes.shape[0], b_codes.shape[0], a_codes.shape[1] * 2
    c = torch.empty(m, n, dtype=out_dtype, device=a_codes.device)
    fp4q_gemm_nvfp4(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, m, n, k, operand_flags, _dt(c), c, amax, stream)
    return c


def dequantize(fmt: int, codes: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor | None,
               rows: int, cols: int, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    y = torch.empty(rows, cols, dtype=out_dtype, device=codes.device)
    fp4q_dequantize(fmt, codes, scales, tensor_scale, rows, cols, _dt(y), y, stream)
    return y


def amax(x: torch.Tensor, stream=None) -> torch.Tensor:
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    fp4q_amax(x, _dt(x), x.shape[0], x.shape[1], out, stream)
    return out


VAR_46, VAR_NVINT4, VAR_IF3, VAR_IF4, VAR_IF6 = 0, 1, 2, 3, 4
VARIANT_BITS = {VAR_46: 4, VAR_NVINT4: 4, VAR_IF3: 3, VAR_IF4: 4, VAR_IF6: 6}


def quantize_variant(x: torch.Tensor, var: int, amax: torch.Tensor | None = None, ws="auto", stream=None) -> dict:
    """Four Over Six, NVINT4, IF3, IF4 or IF6 (codes [rows][cols * bits / 8], scales [rows][cols/16])."""
    rows, cols = x.shape
    dev = x.device
    mode = AMAX_GIVEN if amax is not None else AMAX_COMPUTE
    out = {"amax": amax if amax is not None else torch.empty(1, dtype=torch.float32, device=dev),
           "tensor_scale": torch.empty(1, dtype=torch.float32, device=dev),
           "codes": _u8(rows, cols * VARIANT_BITS[var] // 8, device=dev), "scales": _u8(rows, cols // 16, device=dev)}
    fp4q_quantize_variant(x, _dt(x), rows, cols, var, mode, out["amax"], out["tensor_scale"], out["codes"],
                          out["scales"], _ws(ws, stream), stream)
    return out


def dequantize_variant(var: int, codes, scales, tensor_scale, rows: int, cols: int, out_dtype=torch.float32,
                       stream=None) -> torch.Tensor:
    y = torch.empty(rows, cols, dtype=out_dtype, device=codes.device)
    fp4q_dequantize_variant(var, codes, scales, tensor_scale, rows, cols, _dt(y), y, stream)
    return y


# --- MXFP8 activations -------------------------------------------------------------------
#
# These helpers check what the C entry points cannot see (the tensors' types, shapes, devices
# and strides) before any address is passed on.  A decode step makes several such calls in a few
# microseconds each, so they call the library directly and each check has a short way through.
# Like the helpers above they take no part in autograd: results carry no gradient, whatever the
# arguments require; rmsnorm_backward is called for one.

_NAMES = {torch.float32: F32, torch.bfloat16: BF16}
_U8, _F32 = torch.uint8, torch.float32


def _need(name: str, t, dtype, shape, device: int) -> int:
    """The address of `t`, a dense tensor of this type, shape and device (index, -1: the CPU)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device \
            and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: {dtype} is needed, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: is on {t.device}, the call's other tensors on device {device}")
    raise ValueError(f"{name}: a dense row-major tensor is needed (call .contiguous())")


def _matrix(name: str, t, dtypes) -> tuple[int, int, int]:
    """(rows, cols, device index) of a dense 2-D tensor of one of `dtypes` on the current device."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name}: a tensor of {' or '.join(str(d) for d in dtypes)} is needed")
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: a dense row-major [rows][cols] tensor on the GPU is needed")
    dev = t.get_device()
    if dev != torch._C._cuda_getDevice():   # kernels are launched on the current device
        raise ValueError(f"{name}: is on {t.device}, but device {torch.cuda.current_device()} is current "
                         "(use torch.cuda.device)")
    rows, cols = t.shape
    return rows, cols, dev


def _tensors(values):
    for v in values:
        if isinstance(v, torch.Tensor):
            if v.is_cuda:
                yield v
        elif isinstance(v, dict):
            yield from _tensors(v.values())


def _elsewhere(stream, helper, *args):
    """helper(*args) on a stream (or its handle) that need not be the current one.  The call's memory comes
    from that stream: what the allocator hands out for the current one may still be in use there.
    It hands out the arguments' memory, and the results', only after both streams have passed their uses."""
    if not isinstance(stream, int):
        s = stream
    else:   # (an ExternalStream of 0 would be a new stream)
        s = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    caller = torch.cuda.current_stream(s.device)
    with torch.cuda.stream(s):
        out = helper(*args)
    for t in _tensors(args):
        t.record_stream(s)
    for t in _tensors((out,) if isinstance(out, (torch.Tensor, dict)) else out):
        t.record_stream(caller)
    return out


def _here(dev: int) -> int:
    """The current stream's handle (see _s)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _done(fn: str, status: int) -> None:
    if status:
        raise Fp4qError(fn, status)


def quantize_mxfp8(x: torch.Tensor, stream=None) -> dict:
    """MXFP8: codes [rows][cols] (E4M3), E8M0 scales [rows][cols/32]."""
    if stream is not None:
        return _elsewhere(stream, quantize_mxfp8, x)
    rows, cols, dev = _matrix("x", x, _NAMES)
    codes = torch.empty_like(x, dtype=_U8)
    scales = codes.new_empty(rows, cols // 32)
    _done("fp4q_quantize_mxfp8", lib().fp4q_quantize_mxfp8(
        x.data_ptr(), _NAMES[x.dtype], rows, cols, codes.data_ptr(), scales.data_ptr(),
        _here(dev)))
    return {"codes": codes, "scales": scales}


def dequantize_mxfp8(q: dict, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """The values of MXFP8 codes and scales as quantize_mxfp8 returns them."""
    if stream is not None:
        return _elsewhere(stream, dequantize_mxfp8, q, out_dtype)
    codes = q["codes"]
    rows, cols, dev = _matrix("codes", codes, (_U8,))
    scales = _need("scales", q["scales"], _U8, (rows, cols // 32), dev)
    y = torch.empty_like(codes, dtype=out_dtype)
    _done("fp4q_dequantize_mxfp8", lib().fp4q_dequantize_mxfp8(
        codes.data_ptr(), scales, rows, cols, _dt(y), y.data_ptr(), _here(dev)))
    return y


def rmsnorm_mxfp8(x: torch.Tensor, gain: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                  with_y: bool = False, in_place: bool = False, stream=None) -> dict:
    """RMS norm of x + residual with `gain` (float32) into MXFP8.

    Returns codes, scales, rstd, sum (x + residual in x's type; x itself without a residual)
    and, with ``with_y``, the unquantized y.  ``in_place`` writes the sum over `residual`."""
    if stream is not None:
        return _elsewhere(stream, rmsnorm_mxfp8, x, gain, residual, eps, with_y, in_place)
    rows, cols, dev = _matrix("x", x, _NAMES)
    gp = _need("gain", gain, _F32, (cols,), dev)
    rp = None if residual is None else _need("residual", residual, x.dtype, x.shape, dev)
    codes = torch.empty_like(x, dtype=_U8)
    scales = codes.new_empty(rows, cols // 32)
    rstd = gain.new_empty(rows)
    total = x if residual is None else residual if in_place else torch.empty_like(x)
    y = torch.empty_like(x) if with_y else None
    _done("fp4q_rmsnorm_mxfp8", lib().fp4q_rmsnorm_mxfp8(
        x.data_ptr(), rp, _NAMES[x.dtype], rows, cols, gp, eps, codes.data_ptr(), scales.data_ptr(),
        None if rp is None else total.data_ptr(), rstd.data_ptr(), None if y is None else y.data_ptr(),
        _here(dev)))
    out = {"codes": codes, "scales": scales, "rstd": rstd, "sum": total}
    if with_y:
        out["y"] = y
    return out


def rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, gain: torch.Tensor, rstd: torch.Tensor,
                     dsum: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dgain) of rmsnorm_mxfp8 from its `sum` and `rstd`; `dsum` is the gradient that reaches
    the sum from elsewhere, added to dx."""
    if stream is not None:
        return _elsewhere(stream, rmsnorm_backward, dy, s, gain, rstd, dsum)
    rows, cols, dev = _matrix("dy", dy, _NAMES)
    sp = _need("s", s, dy.dtype, dy.shape, dev)
    gp = _need("gain", gain, _F32, (cols,), dev)
    rp = _need("rstd", rstd, _F32, (rows,), dev)
    up = None if dsum is None else _need("dsum", dsum, dy.dtype, dy.shape, dev)
    dx, dgain = torch.empty_like(dy), torch.empty_like(gain)
    need = lib().fp4q_rmsnorm_backward_scratch(rows, cols)
    scratch = gain.new_empty(need // 4)
    _done("fp4q_rmsnorm_backward", lib().fp4q_rmsnorm_backward(
        dy.data_ptr(), sp, up, _NAMES[dy.dtype], rows, cols, gp, rp, dx.data_ptr(), dgain.data_ptr(),
        scratch.data_ptr(), need, _here(dev)))
    return dx, dgain


def gemm_mxfp8_mxfp4(a: dict, b: dict, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """C = A B^T for an MXFP8 operand (quantize_mxfp8, rmsnorm_mxfp8) and a row-wise MXFP4 one
    (quantize_mxfp4); k (a multiple of 128) is the columns of both."""
    if stream is not None:
        return _elsewhere(stream, gemm_mxfp8_mxfp4, a, b, out_dtype)
    ac, bc = a["codes"], b["codes"]
    m, k, dev = _matrix("a codes", ac, (_U8,))
    n = bc.shape[0] if isinstance(bc, torch.Tensor) and bc.dim() == 2 else 0
    asp = _need("a scales", a["scales"], _U8, (m, k // 32), dev)
    bcp = _need("b codes", bc, _U8, (n, k // 2), dev)
    bsp = _need("b scales", b["scales"], _U8, (n, k // 32), dev)
    c = torch.empty(m, n, dtype=out_dtype, device=ac.device)
    _done("fp4q_gemm_mxfp8_mxfp4", lib().fp4q_gemm_mxfp8_mxfp4(
        ac.data_ptr(), asp, bcp, bsp, m, n, k, _dt(c), c.data_ptr(), _here(dev)))
    return c


def moe_mxfp4(x: dict, w13: dict, w2: dict, topk: int, router_x: torch.Tensor | None = None,
              router_w: torch.Tensor | None = None, ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None, out_dtype=torch.bfloat16, stream=None) -> dict:
    """A mixture-of-experts layer for up to 64 tokens.

    x: MXFP8 tokens (rmsnorm_mxfp8); w13, w2: MXFP4 experts, codes [experts][2 hidden][d/2] and
    [experts][d][hidden/2] with their scales [..][/32].  Either `router_x` [tokens][d] and
    `router_w` [experts][d] (bfloat16 or float32): the layer routes; or `ids` (int32) and
    `weights` (float32) [tokens][topk], as another router chose them.  Returns y, ids, weights."""
    if stream is not None:
        return _elsewhere(stream, moe_mxfp4, x, w13, w2, topk, router_x, router_w, ids, weights, out_dtype)
    xc, w2c = x["codes"], w2["codes"]
    tokens, d, dev = _matrix("x codes", xc, (_U8,))
    if not isinstance(w2c, torch.Tensor) or w2c.dim() != 3:
        raise ValueError("w2 codes: a tensor [experts][d][hidden/2] is needed")
    experts, hidden = w2c.shape[0], w2c.shape[2] * 2
    xsp = _need("x scales", x["scales"], _U8, (tokens, d // 32), dev)
    w13p = _need("w13 codes", w13["codes"], _U8, (experts, 2 * hidden, d // 2), dev)
    w13sp = _need("w13 scales", w13["scales"], _U8, (experts, 2 * hidden, d // 32), dev)
    w2p = _need("w2 codes", w2c, _U8, (experts, d, hidden // 2), dev)
    w2sp = _need("w2 scales", w2["scales"], _U8, (experts, d, hidden // 32), dev)
    if (router_x is None) != (router_w is None) or (ids is None) != (weights is None) or \
            (router_x is None) == (ids is None):
        raise ValueError("either router_x and router_w or ids and weights are needed")
    where = xc.device
    rxp = rwp = None
    mode, rdt = ROUTE_GIVEN, F32
    if router_x is not None:
        mode, rdt = ROUTE_COMPUTE, _dt(router_x)
        rxp = _need("router_x", router_x, router_x.dtype, (tokens, d), dev)
        rwp = _need("router_w", router_w, router_x.dtype, (experts, d), dev)
        ids = torch.empty(tokens, topk, dtype=torch.int32, device=where)
        weights = torch.empty(tokens, topk, dtype=_F32, device=where)
    ip = _need("ids", ids, torch.int32, (tokens, topk), dev)
    wp = _need("weights", weights, _F32, (tokens, topk), dev)
    y = torch.empty(tokens, d, dtype=out_dtype, device=where)
    need = lib().fp4q_moe_scratch(tokens, d, hidden, experts, topk)
    scratch = xc.new_empty(need)
    _done("fp4q_moe_mxfp4", lib().fp4q_moe_mxfp4(
        xc.data_ptr(), xsp, rxp, rwp, rdt, w13p, w13sp, w2p, w2sp, tokens, d, hidden, experts, topk, mode, ip, wp,
        _dt(y), y.data_ptr(), scratch.data_ptr(), need, _here(dev)))
    return {"y": y, "ids": ids, "weights": weights}
