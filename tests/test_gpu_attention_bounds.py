"""Attention over the paged cache where a batch goes past its bounds (GPU)."""
import pytest
import torch

import attention_ref as ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_attention import LEFT, _compare, _queries, _scale

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _into(case, q, cache, batch, window):
    """(out, lse) of a call into rows that hold LEFT."""
    c, b = B._kv_cache(cache, 0)[0], B._kv_batch(batch, 0)
    n, h, d = q.shape
    need = B.fp4q_attention_paged_scratch(c, b, n, h, window)
    out, lse = torch.full((case.tokens, h, d), LEFT, dtype=torch.bfloat16, device=DEV), torch.full((case.tokens, h), LEFT, device=DEV)
    B.fp4q_attention_paged(q, n, h, q.stride(0), q.stride(1), c, b, _scale(case), window, B.ATTN_CAUSAL, out, lse,
                           torch.empty(need, dtype=torch.uint8, device=DEV), need)
    return out, lse


@pytest.mark.parametrize("window", [0, 1, 40, 50, 200])
@pytest.mark.parametrize("lens,groups,most", [
    ([(2, 3000), (1, 20)], (), 1), ([(300, 1000), (2, 50)], (), 100), ([(30, 40), (7, 7), (3, 300)], (), 2), ([(500, 500), (9, 90)], (), 9),
    ([(20, 700), (1, 530), (20, 650)], [(3, 512)], 3), ([(20, 700), (60, 650)], [(2, 512)], 12)],
    ids=["token", "prompt", "few", "ends-early", "shared-few", "shared-many"])
def test_sequences_with_more_tokens_than_the_bound(lens, groups, most, window):
    """The first max_q_len tokens see what they see at their places, which the sequence's real length gives; the others' rows are left."""
    case = ref.Case(lens, 2, 64, 16, groups=groups)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    out, lse = _into(case, q, cache, dict(batch, max_q_len=most), window)
    starts = [int(s) for s in case.q_starts]
    done = [t for a, b in zip(starts, starts[1:]) for t in range(a, min(b, a + most))]
    left = [t for t in range(case.tokens) if t not in done]
    assert (out[left] == LEFT).all() and (lse[left] == LEFT).all()
    _compare((out[done], lse[done]), tuple(v[done] for v in want))


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("tokens", [3, 150])
def test_a_sequence_with_more_tokens_than_the_call(tokens, window):
    """The call has the first tokens of a sequence only."""
    case = ref.Case([(300, 1000)], 2, 64, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    out, lse = _into(case, q[:tokens], cache, batch, window)
    assert (out[tokens:] == LEFT).all() and (lse[tokens:] == LEFT).all()
    _compare((out[:tokens], lse[:tokens]), tuple(v[:tokens] for v in want))
