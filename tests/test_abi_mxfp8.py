"""Refusals of the MXFP8 entry points and their helpers (no GPU needed): bad arguments fail
before anything is enqueued."""
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

A, MIS = 0x10000, 0x10004


def _with(call, base):
    def go(**kw):
        args = dict(base)
        args.update(kw)
        return getattr(B.lib(), call)(*args.values())
    return go


QUANT = dict(x=A, dt=B.BF16, rows=4, cols=64, codes=A, scales=A, stream=0)
DEQUANT = dict(codes=A, scales=A, rows=4, cols=64, dt=B.F32, y=A, stream=0)
NORM = dict(x=A, residual=None, dt=B.BF16, rows=4, cols=64, gain=A, eps=1e-6, codes=A, scales=A, sum=None, rstd=None,
            y=None, stream=0)
BACK = dict(dy=A, s=A, dsum=None, dt=B.BF16, rows=4, cols=64, gain=A, rstd=A, dx=A, dgain=A, scratch=A,
            scratch_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(dt=2), 4), (dict(rows=0), 2),
    (dict(cols=0), 2), (dict(cols=48), 2), (dict(rows=-1), 2), (dict(rows=1 << 31), 2), (dict(cols=1 << 31), 2),
    (dict(rows=1 << 30, cols=1 << 10), 2), (dict(x=MIS), 3), (dict(codes=MIS), 3), (dict(scales=MIS), 3)])
def test_quantize(kw, status):
    assert _with("fp4q_quantize_mxfp8", QUANT)(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), 1), (dict(y=None), 1), (dict(dt=9), 4), (dict(cols=33), 2), (dict(rows=0), 2),
    (dict(y=MIS), 3), (dict(scales=MIS), 3)])
def test_dequantize(kw, status):
    assert _with("fp4q_dequantize_mxfp8", DEQUANT)(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(gain=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(dt=5), 4),
    (dict(eps=-1.0), 4), (dict(eps=float("nan")), 4), (dict(eps=float("inf")), 4), (dict(cols=40), 2),
    (dict(cols=32800), 2), (dict(rows=0), 2), (dict(x=MIS), 3), (dict(residual=MIS), 3), (dict(gain=MIS), 3),
    (dict(sum=MIS), 3), (dict(rstd=A + 2), 3), (dict(y=MIS), 3)])
def test_rmsnorm(kw, status):
    assert _with("fp4q_rmsnorm_mxfp8", NORM)(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(s=None), 1), (dict(rstd=None), 1), (dict(dgain=None), 1), (dict(scratch=None), 1),
    (dict(dt=-1), 4), (dict(cols=33), 2), (dict(cols=1 << 16), 2), (dict(rows=0), 2),
    (dict(scratch_bytes=B.fp4q_rmsnorm_backward_scratch(4, 64) - 1), 4), (dict(dy=MIS), 3), (dict(dsum=MIS), 3),
    (dict(dx=MIS), 3), (dict(dgain=MIS), 3), (dict(scratch=MIS), 3), (dict(rstd=A + 1), 3)])
def test_rmsnorm_backward(kw, status):
    assert _with("fp4q_rmsnorm_backward", BACK)(**kw) == status


def test_scratch_of_a_refused_shape_is_zero():
    assert B.fp4q_rmsnorm_backward_scratch(0, 64) == 0
    assert B.fp4q_rmsnorm_backward_scratch(4, 48) == 0
    assert B.fp4q_rmsnorm_backward_scratch(4, 1 << 16) == 0
    assert B.fp4q_rmsnorm_backward_scratch(1 << 30, 64) <= 1 << 20    # bounded in the rows


def test_helpers_refuse_what_the_library_cannot_see():
    with pytest.raises(TypeError):
        B.quantize_mxfp8(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        B.quantize_mxfp8([[1.0]])
    with pytest.raises(ValueError):                        # not on the GPU
        B.quantize_mxfp8(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        B.rmsnorm_mxfp8(torch.zeros(4, 64), torch.ones(64))
    dev = -1                                               # the CPU's index
    x = torch.zeros(8, 64)
    for bad, err in ((x.double(), TypeError), (torch.zeros(8, 32), ValueError), (torch.zeros(64, 8).t(), ValueError),
                     (None, TypeError)):
        with pytest.raises(err):
            B._need("t", bad, torch.float32, (8, 64), dev)
    with pytest.raises(ValueError):
        B._need("t", x, torch.float32, (8, 64), 0)         # another device
    assert B._need("t", x, torch.float32, (8, 64), dev) == x.data_ptr()


GEMM = dict(ac=A, asc=A, bc=A, bsc=A, m=4, n=8, k=256, dt=B.F32, c=A, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(ac=None), 1), (dict(asc=None), 1), (dict(bc=None), 1), (dict(bsc=None), 1), (dict(c=None), 1),
    (dict(dt=2), 4), (dict(m=0), 2), (dict(n=-1), 2), (dict(k=0), 2), (dict(k=192), 2), (dict(k=(1 << 25) + 128), 2),
    (dict(m=1 << 31), 2), (dict(n=1 << 31), 2), (dict(m=(1 << 31) - 1, n=(1 << 31) - 1), 2), (dict(ac=MIS), 3),
    (dict(asc=MIS), 3), (dict(bc=MIS), 3), (dict(bsc=MIS), 3), (dict(c=MIS), 3)])
def test_gemm(kw, status):
    assert _with("fp4q_gemm_mxfp8_mxfp4", GEMM)(**kw) == status


MOE = dict(xc=A, xs=A, rx=A, rw=A, rdt=B.BF16, w13c=A, w13s=A, w2c=A, w2s=A, tokens=4, d=256, hidden=128, experts=8, topk=2,
           mode=B.ROUTE_COMPUTE, ids=A, weights=A, dt=B.BF16, y=A, scratch=A, scratch_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(xc=None), 1), (dict(xs=None), 1), (dict(rx=None), 1), (dict(rw=None), 1), (dict(w13c=None), 1),
    (dict(w13s=None), 1), (dict(w2c=None), 1), (dict(w2s=None), 1), (dict(ids=None), 1), (dict(weights=None), 1),
    (dict(y=None), 1), (dict(scratch=None), 1), (dict(rdt=3), 4), (dict(dt=2), 4), (dict(mode=2), 4),
    (dict(tokens=0), 2), (dict(tokens=65), 2), (dict(d=192), 2), (dict(d=0), 2), (dict(d=65664), 2),
    (dict(hidden=64), 2), (dict(hidden=65664), 2), (dict(experts=0), 2), (dict(experts=513), 2), (dict(topk=0), 2),
    (dict(topk=9), 2), (dict(experts=64, topk=17), 2),
    (dict(scratch_bytes=B.fp4q_moe_scratch(4, 256, 128, 8, 2) - 1), 4), (dict(xc=MIS), 3), (dict(rx=MIS), 3),
    (dict(w13c=MIS), 3), (dict(w2s=MIS), 3), (dict(ids=A + 2), 3), (dict(weights=A + 1), 3), (dict(y=MIS), 3),
    (dict(scratch=MIS), 3),
    (dict(mode=B.ROUTE_GIVEN, rx=None, rw=None, y=None), 1), (dict(mode=B.ROUTE_GIVEN, rx=None, rw=None, xs=MIS), 3)])
def test_moe(kw, status):
    assert _with("fp4q_moe_mxfp4", MOE)(**kw) == status


def test_moe_scratch():
    assert B.fp4q_moe_scratch(65, 128, 128, 8, 2) == 0 and B.fp4q_moe_scratch(4, 128, 100, 8, 2) == 0
    assert B.fp4q_moe_scratch(64, 128, 65536, 512, 16) >= 64 * 16 * 65536
