"""How far the attention's output is from binary64 (GPU): what include/fp4q.h says of the probabilities' bits."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_attention import _queries, _scale

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rows(case, q, scale, seq, t, h):
    """out, sum p |v| and the bound of the scores' error of one row: products are exact in fp32, their sum is D roundings
    off, the exponent four more (the factor's two, its product's, the exponential's argument's)."""
    n, kv = int(case.q_starts[seq + 1] - case.q_starts[seq]), int(case.kv_lens[seq])
    seen, kvh = kv - n + t + 1, h // (q.shape[1] // case.heads)
    k, v = case.rows(seq, "k")[:seen, kvh], case.rows(seq, "v")[:seen, kvh]
    x = q[int(case.q_starts[seq]) + t, h]
    s = scale * (k @ x)
    p = np.exp(s - s.max())
    e = case.dim * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(x)).max() + 4 * 2.0 ** -24 * np.abs(s).max() + 2.0 ** -22
    return (p @ v) / p.sum(), (p @ np.abs(v)) / p.sum(), e, seen


def _check(case, o, q, scale, bits, rows):
    for seq, t, h in rows:
        out, size, e, seen = _rows(case, q, scale, seq, t, h)
        # p's exponents; p's parts in the products; fp32 sums of as many terms as keys, of p and of p v; the output's own rounding
        tol = (np.expm1(2 * e) + 2.0 ** -bits + 2 * seen * 2.0 ** -24) * size + 2.0 ** -8 * np.abs(out)
        got = o[int(case.q_starts[seq]) + t, h]
        assert np.all(np.abs(got - out) <= tol), (seq, t, h, float((np.abs(got - out) / tol).max()))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,group,bits", [
    ([(1, 50), (1, 700), (1, 17), (1, 333)], 4, 16), ([(1, 3000)], 3, 16), ([(5, 100), (3, 64), (2, 2), (4, 1000)], 5, 16), ([(8, 300)], 4, 16),
    ([(9, 300)], 4, 8), ([(120, 120)], 2, 8)], ids=["tokens", "pieces", "drafts", "32-rows", "36-rows", "prompt"])
def test_probabilities(lens, group, bits, dim):
    """16 bits of each probability count in the products of sequences with up to 32 rows per key/value head, else 8."""
    case = ref.Case(lens, 2, dim, 32)
    cache, batch = case.tensors(DEV)
    q = _queries(case, group)
    o = B.attention_paged(q, cache, batch, scale=_scale(case)).double().cpu().numpy()
    rows = [(s, t, h) for s, (n, _) in enumerate(lens) for t in range(0, n, max(1, n // 5)) for h in range(2 * group)]
    _check(case, o, q.double().cpu().numpy(), _scale(case), bits, rows)


@pytest.mark.parametrize("lens,groups,bits", [([(1, 256)], (), 16), ([(40, 295)], (), 8), ([(1, 256), (1, 256)], [(2, 256)], 8)],
                         ids=["few", "many", "shared"])
def test_a_key_that_dominates_after_another(lens, groups, bits):
    """Of the keys that count one has 1 / 128.5 of the other's weight and comes tiles before it: where the running maximum follows late,
    the larger p is 128.5, halfway between two bf16 numbers."""
    case = ref.Case(lens, 1, 64, 16, groups=groups)
    scale = float(np.float32(np.log(128.5)))
    for s, (n, kv) in enumerate(lens):
        for at in range(kv):
            page, row = int(case.page_table[s, at // 16]), at % 16
            case.k_scales[page, :, row] = case.v_scales[page, :, row] = 127
            case.k_codes[page, :, row] = 0xFE                           # -448: no weight
            if at in (3, 200):
                case.k_codes[page, :, row] = 0x38 if at == 200 else 0   # 1 and 0
                case.v_codes[page, :, row] = 0x38 if at == 200 else 0
    cache, batch = case.tensors(DEV)
    q = torch.zeros(case.tokens, 4, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 5] = 1.0
    o = B.attention_paged(q, cache, batch, scale=scale).double().cpu().numpy()
    rows = [(s, n - 1, h) for s, (n, _) in enumerate(lens) for h in range(4)]
    _check(case, o, q.double().cpu().numpy(), scale, bits, rows)
