"""Shapes that the MXFP8 operators refuse, through the helpers (GPU): the status names the shape, also where
an empty output or scratch has no address.  Nothing is enqueued."""
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
E_SHAPE = 2


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device=DEV)


def _fp8(t, d):
    return {"codes": _u8(t, d), "scales": _u8(t, d // 32)}


def _fp4(*shape):
    return {"codes": _u8(*shape[:-1], shape[-1] // 2), "scales": _u8(*shape[:-1], shape[-1] // 32)}


def _f(*shape):
    return torch.zeros(*shape, device=DEV)


def _norm(rows, cols):
    return lambda: B.rmsnorm_mxfp8(_f(rows, cols), _f(cols), residual=_f(rows, cols), with_y=True)


def _gradient(rows, cols):
    return lambda: B.rmsnorm_backward(_f(rows, cols), _f(rows, cols), _f(cols), _f(rows))


def _experts(t, d, h, e, k):
    return lambda: B.moe_mxfp4(_fp8(t, d), _fp4(e, 2 * h, d), _fp4(e, d, h), k, router_x=_f(t, d), router_w=_f(e, d))


@pytest.mark.parametrize("call", [
    lambda: B.quantize_mxfp8(_f(0, 64)), lambda: B.quantize_mxfp8(_f(4, 0)), lambda: B.quantize_mxfp8(_f(4, 48)),
    lambda: B.dequantize_mxfp8(_fp8(0, 64)), lambda: B.dequantize_mxfp8(_fp8(4, 33)),
    _norm(0, 64), _norm(4, 0), _norm(4, 48), _norm(2, 32800),
    _gradient(0, 64), _gradient(4, 0), _gradient(4, 48), _gradient(2, 32800),
    lambda: B.gemm_mxfp8_mxfp4(_fp8(0, 128), _fp4(8, 128)), lambda: B.gemm_mxfp8_mxfp4(_fp8(4, 128), _fp4(0, 128)),
    lambda: B.gemm_mxfp8_mxfp4(_fp8(4, 0), _fp4(8, 0)), lambda: B.gemm_mxfp8_mxfp4(_fp8(4, 192), _fp4(8, 192)),
    _experts(0, 128, 128, 4, 2), _experts(65, 128, 128, 4, 2), _experts(2, 192, 128, 4, 2), _experts(2, 128, 64, 4, 2),
    _experts(2, 128, 128, 4, 0), _experts(2, 128, 128, 4, 5), _experts(2, 128, 128, 32, 17), _experts(2, 128, 128, 0, 0)])
def test_the_status_names_the_shape(call):
    with pytest.raises(B.Fp4qError) as e:
        call()
    assert e.value.status == E_SHAPE
