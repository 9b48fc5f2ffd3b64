"""The expert layer's router (GPU) where the softmax has nothing, or one finite logit, to stand on; one token
and several take different kernels."""
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B
from test_gpu_moe import _dev, _whole_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("t", [1, 5, 20])
def test_infinite_logits(t):
    d, h, e, k = 256, 128, 9, 3
    x, w13, w2 = (_dev(v) for v in _whole_layer(t, d, h, e, 3))
    rx, rw = torch.zeros(t, d, device=DEV), torch.zeros(e, d, device=DEV)
    rx[:, 0] = 1.0
    call = lambda: B.moe_mxfp4(x, w13, w2, k, router_x=rx, router_w=rw, out_dtype=torch.float32)
    print("moe router", t, flush=True)
    rw[:, 0] = float("-inf")                              # nothing left: 0 / 0
    o = call()
    assert o["ids"].tolist() == [[0, 1, 2]] * t and torch.isnan(o["weights"]).all() and torch.isnan(o["y"]).all()
    rw[7, 0] = -3.4e38                                     # one finite logit takes all, however low
    o = call()
    assert o["ids"].tolist() == [[7, 0, 1]] * t and o["weights"].tolist() == [[1.0, 0.0, 0.0]] * t
    one = torch.full((t, 1), 7, dtype=torch.int32, device=DEV)
    alone = B.moe_mxfp4(x, w13, w2, 1, ids=one, weights=torch.ones(t, 1, device=DEV), out_dtype=torch.float32)
    assert torch.equal(o["y"], alone["y"])                 # the others' outputs are finite: weight 0 adds 0
    rw[4, 0] = float("inf")                                # infinity less itself
    o = call()
    assert o["ids"].tolist() == [[4, 7, 0]] * t and torch.isnan(o["weights"]).any(1).all()
