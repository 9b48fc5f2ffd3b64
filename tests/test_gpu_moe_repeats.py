"""One token of the MXFP4 expert layer whose given choices name an expert more than once, or none.

Whole values that the layer holds exactly: the result must be equal to the plain sum.  The scratch is
filled with NaN codes and NaN scales first, so a hidden row that the call reads but does not write shows.
"""
import numpy as np
import pytest
import torch

import mxfp8_ref as ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_moe import _dev, _whole_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _one_token(x, w13, w2, ids, weights, out):
    """y of the C entry point, on scratch of 0xFF bytes (E4M3's NaN, E8M0's NaN)."""
    d, (e, _, hb) = x["codes"].shape[1], w2["codes"].shape
    need = B.fp4q_moe_scratch(1, d, 2 * hb, e, ids.shape[1])
    scratch = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.empty(1, d, dtype=out, device=DEV)
    B.fp4q_moe_mxfp4(x["codes"], x["scales"], None, None, B.F32, w13["codes"], w13["scales"], w2["codes"], w2["scales"],
                     1, d, 2 * hb, e, ids.shape[1], B.ROUTE_GIVEN, ids, weights, B._dt(y), y, scratch, need)
    return y


@pytest.mark.parametrize("d,h", [(128, 128), (256, 1024), (1152, 640)])
@pytest.mark.parametrize("e,ids", [(4, [3, 3]), (2, [0, 0]), (1, [0]), (8, [1, 1, 1]), (8, [5, 2, 5, -1]), (64, [63, 0, 63, 0]),
                                   (3, [2, 3, 2]), (20, [7] * 16), (5, [-1, 5, -1]), (40, [0, 1, 2, 3, 4, 5, 6, 0])])
def test_repeated_choices_of_one_token(d, h, e, ids):
    x, w13, w2 = _whole_layer(1, d, h, e, d + e)
    weights = np.array([1.0, 0.5, -2.0, 4.0] * 4, np.float32)[:len(ids)]
    gu = np.stack([ref.dequantize(*x) @ ref.fp4(w13[0][i], w13[1][i]).T for i in range(e)])[:, 0]
    hid = gu[:, :h] * gu[:, h:]
    y = np.zeros(d)
    for i, w in zip(ids, weights):
        if 0 <= i < e:
            y += w * (hid[i] @ ref.fp4(w2[0][i], w2[1][i]).T)
    print("moe one token", d, h, e, ids, flush=True)
    chosen, share = torch.tensor([ids], dtype=torch.int32, device=DEV), torch.from_numpy(weights[None]).to(DEV)
    for out in (torch.float32, torch.bfloat16):
        got = _one_token(_dev(x), _dev(w13), _dev(w2), chosen, share, out)
        assert torch.equal(got[0], torch.from_numpy(y).float().to(out).to(DEV))
