"""Attention over the paged cache at the ends of the shapes that it takes (GPU)."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_attention import LEFT, _compare, _scale

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _some_rows(case, q, tokens, window=0):
    """ref.attention of some tokens, each as the last one of a sequence that ends there."""
    outs = []
    for t in tokens:
        i = int(np.searchsorted(case.q_starts, t, side="right")) - 1
        sub = object.__new__(ref.Case)
        sub.__dict__.update(case.__dict__)
        kv = int(case.kv_lens[i]) - (int(case.q_starts[i + 1]) - t) + 1
        sub.lens, sub.q_starts, sub.kv_lens, sub.page_table = [(1, kv)], np.array([0, 1]), np.array([kv]), case.page_table[i:i + 1]
        outs.append(ref.attention(sub, q[t:t + 1].float().cpu().numpy(), _scale(case), window))
    return tuple(np.concatenate([o[k] for o in outs]) for k in range(4))


def test_most_rows():
    """2^26 - 1 rows, with a shared prefix, whose join has more workgroups than one launch takes: 24573 tokens of 2731 query
    heads, all with the same queries."""
    case = ref.Case([(24573, 24700)], 1, 64, 64, groups=[(1, 64)])
    cache, batch = case.tensors(DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    q = torch.randn(case.tokens, 1, 64, generator=g, device=DEV).to(torch.bfloat16)
    heads, window, tokens = 2731, 9, case.tokens
    assert tokens * heads == (1 << 26) - 1
    c, b = B._kv_cache(cache, 0)[0], B._kv_batch(batch, 0)
    need = B.fp4q_attention_paged_scratch(c, b, tokens, heads, window)
    out = torch.full((tokens, heads, 64), LEFT, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((tokens, heads), LEFT, device=DEV)
    scratch = torch.empty(need, dtype=torch.uint8, device=DEV)
    B.fp4q_attention_paged(q, tokens, heads, 64, 0, c, b, _scale(case), window, B.ATTN_CAUSAL, out, lse, scratch, need)
    torch.cuda.synchronize()
    assert not (lse == LEFT).any() and not any((part[..., 0] == LEFT).any() for part in out.split(1024))
    some = [0, 1, 5000, 24000, 24571, 24572]
    want = _some_rows(case, q, some, window)
    for h in (0, 1, 1365, 2729, 2730):
        _compare((out[some, h:h + 1], lse[some, h:h + 1]), want)
