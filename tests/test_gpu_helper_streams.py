"""The MXFP8 helpers' `stream` argument (GPU): which stream a call goes to."""
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Recorder:
    """The library with its enqueueing calls recorded; `run` False: not made."""

    def __init__(self, run):
        self.real, self.run, self.calls = B.lib(), run, []

    def __getattr__(self, name):
        fn = getattr(self.real, name)
        if name.endswith("_scratch"):
            return fn

        def call(*args):
            self.calls.append((name, args))
            return fn(*args) if self.run else 0
        return call


def _inputs():
    """Each helper as a call of one argument, the stream."""
    t, d, h, e, k = 4, 128, 128, 8, 2
    g = torch.Generator(device=DEV).manual_seed(0)
    x, res = (torch.randn(t, d, generator=g, device=DEV) for _ in range(2))
    gain, rstd = torch.ones(d, device=DEV), torch.ones(t, device=DEV)
    q = {"codes": torch.zeros(t, d, dtype=torch.uint8, device=DEV),
         "scales": torch.full((t, d // 32), 127, dtype=torch.uint8, device=DEV)}

    def fp4(*shape):
        return {"codes": torch.zeros(*shape[:-1], shape[-1] // 2, dtype=torch.uint8, device=DEV),
                "scales": torch.full((*shape[:-1], shape[-1] // 32), 127, dtype=torch.uint8, device=DEV)}
    w, w13, w2, rw = fp4(24, d), fp4(e, 2 * h, d), fp4(e, d, h), torch.randn(e, d, generator=g, device=DEV)
    ids, wt = torch.zeros(t, k, dtype=torch.int32, device=DEV), torch.ones(t, k, device=DEV)
    torch.cuda.synchronize()
    return {
        "quantize": lambda s: B.quantize_mxfp8(x, stream=s),
        "dequantize": lambda s: B.dequantize_mxfp8(q, torch.bfloat16, stream=s),
        "norm": lambda s: B.rmsnorm_mxfp8(x, gain, residual=res, with_y=True, stream=s),
        "gradient": lambda s: B.rmsnorm_backward(x, res, gain, rstd, dsum=x, stream=s),
        "product": lambda s: B.gemm_mxfp8_mxfp4(q, w, torch.bfloat16, stream=s),
        "experts": lambda s: B.moe_mxfp4(q, w13, w2, k, router_x=x, router_w=rw, stream=s),
        "experts given": lambda s: B.moe_mxfp4(q, w13, w2, k, ids=ids, weights=wt, stream=s),
    }


HELPERS = ["quantize", "dequantize", "norm", "gradient", "product", "experts", "experts given"]


@pytest.mark.parametrize("name", HELPERS)
def test_a_call_goes_to_the_stream_it_names(name, monkeypatch):
    call, side = _inputs()[name], torch.cuda.Stream()
    rec = Recorder(run=False)
    monkeypatch.setattr(B, "lib", lambda: rec)
    with torch.cuda.stream(side):
        for stream, handle in ((0, 0), (torch.cuda.default_stream(), 0), (None, side.cuda_stream)):
            call(stream)
            assert rec.calls[-1][1][-1] == handle
    for stream, handle in ((None, 0), (0, 0), (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
        call(stream)
        assert rec.calls[-1][1][-1] == handle
    assert len(rec.calls) == 7


def _segments():
    return [(s["address"], s["address"] + s["total_size"], s["stream"]) for s in torch.cuda.memory_snapshot()]


def _pool(address, segments):
    return [s for lo, hi, s in segments if lo <= address < hi]


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for v in (out.values() if isinstance(out, dict) else out) if v is not None for t in _tensors(v)]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", HELPERS)
def test_a_call_on_another_stream_takes_memory_of_that_stream(name, as_handle, monkeypatch):
    """What the current stream's allocator hands out may still be in use by work of the current stream that
    the other one does not wait for."""
    call, side = _inputs()[name], torch.cuda.Stream()
    inputs = {t.data_ptr() for c in call.__closure__ if not isinstance(c.cell_contents, int) for t in _tensors(c.cell_contents)}
    rec = Recorder(run=True)
    monkeypatch.setattr(B, "lib", lambda: rec)
    side.wait_stream(torch.cuda.current_stream())
    out = call(side.cuda_stream if as_handle else side)
    side.synchronize()
    segments = _segments()
    made = [t.data_ptr() for t in _tensors(out)] + [a for a in rec.calls[-1][1][:-1] if isinstance(a, int) and _pool(a, segments)]
    made = [a for a in made if a not in inputs]
    assert made
    for a in made:
        assert _pool(a, segments) == [side.cuda_stream]


def test_memory_is_kept_while_either_stream_uses_it():
    side, n = torch.cuda.Stream(), 1 << 22
    torch.cuda.empty_cache()
    x = torch.randn(n // 64, 64, device=DEV)
    B.quantize_mxfp8(x, stream=side)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    out = B.quantize_mxfp8(x, stream=side)                  # waits behind the sleep
    at = x.data_ptr()
    del x                                                   # still to be read
    assert at not in {t.data_ptr() for t in [torch.empty(n // 64, 64, device=DEV) for _ in range(4)]}
    side.synchronize()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    y = out["codes"].clone()                                # waits behind the sleep
    at = out["codes"].data_ptr()
    del out                                                 # still to be read
    with torch.cuda.stream(side):
        assert at not in {t.data_ptr() for t in [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(4)]}
    torch.cuda.synchronize()
    assert y.numel() == n


def test_the_callers_tensors_in_place():
    side = torch.cuda.Stream()
    x, gain = torch.randn(8, 64, device=DEV), torch.ones(64, device=DEV)
    res = torch.randn(8, 64, device=DEV)
    want = B.rmsnorm_mxfp8(x, gain, residual=res.clone())
    side.wait_stream(torch.cuda.current_stream())
    o = B.rmsnorm_mxfp8(x, gain, residual=res, in_place=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert o["sum"] is res and torch.equal(res, want["sum"]) and torch.equal(o["codes"], want["codes"])
    assert set(o) == set(want)


def test_another_stream_inside_a_captured_graph():
    x, gain, side = torch.randn(40, 1024, device=DEV), torch.ones(1024, device=DEV), torch.cuda.Stream()
    w = B.quantize_mxfp4(torch.randn(96, 1024, device=DEV))

    def step(s):
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        y = B.gemm_mxfp8_mxfp4(B.rmsnorm_mxfp8(x, gain, stream=s), w, torch.bfloat16, stream=s)
        if s is not None:
            torch.cuda.current_stream().wait_stream(s)
        return y

    step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(side)
    for _ in range(4):
        x.copy_(torch.randn(40, 1024, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step(None))
        torch.cuda.synchronize()
