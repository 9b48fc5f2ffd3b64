"""dgain of the RMS norm's gradient (GPU) over many rows, against binary64.

Every row is the same, so the terms of a column's sum are equal and the roundings of a running sum do not
cancel.  Roundings of one column's sum, relative to the sum of magnitudes: one for s r, at most 64 for the
rows that a workgroup adds up one after another, one for each such run that it adds to its partial sum, and
32 + 5 for the partial sums of the workgroups (1024 of them up to 4096 columns, 512 up to 8192, then 256)."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
RUN = 64


@pytest.mark.parametrize("rows,cols,dtype", [(1000, 64, "f32"), (1 << 24, 32, "f32"), ((1 << 22) + 4097, 96, "bf16"),
                                             ((1 << 19) + 77, 2080, "bf16"), ((1 << 18) + 1, 4128, "bf16"),
                                             (1 << 17, 8224, "bf16"), (70001, 20000, "bf16"), (40000, 20000, "f32")])
def test_dgain_of_equal_rows(rows, cols, dtype):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(cols)
    s1, d1 = (torch.rand(cols, generator=g).add(0.5).to(dt).to(DEV) for _ in range(2))
    s, dy = s1.expand(rows, cols).contiguous(), d1.expand(rows, cols).contiguous()
    gain, rstd = torch.ones(cols, device=DEV), torch.full((rows,), 0.7, device=DEV)
    print("dgain", rows, cols, dtype, flush=True)
    _, dg = B.rmsnorm_backward(dy, s, gain, rstd)
    del s, dy
    torch.cuda.empty_cache()
    groups = min(rows, 1024 if cols <= 4096 else 512 if cols <= 8192 else 256)
    per = -(-rows // groups)
    bound = (1 + min(per, RUN) + -(-per // RUN) + 32 + 5) * U
    exact = rows * s1.double() * d1.double() * rstd[0].double()
    off = ((dg.double() - exact).abs() / exact).max().item()
    assert off <= bound, (off / U, bound / U)
