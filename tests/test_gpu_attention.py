"""Attention over the paged MXFP8 cache (GPU), against binary64 with bounds counted from the roundings."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from block_scaled_fp4_05_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _queries(case, group, seed=0, row_heads=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    heads = case.heads * group
    return torch.randn(case.tokens, row_heads or heads, case.dim, generator=g, device=DEV).to(torch.bfloat16)[:, :heads]


def _compare(got, want):
    (o, lse), (out, want_lse, tol, tol_lse) = got, want
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    nan = np.isnan(out)
    assert np.array_equal(np.isnan(o), nan)
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse)) and np.array_equal(lse == -np.inf, want_lse == -np.inf)
    assert np.all(np.abs(o - out)[~nan] <= tol[~nan]), float((np.abs(o - out) / tol)[~nan].max())
    fin = np.isfinite(want_lse)
    assert np.all(np.abs(lse[fin] - want_lse[fin]) <= tol_lse[fin])


def _scale(case):
    return 0.4 / case.dim ** 0.5     # keys of magnitude about 4, queries of 1: scores of a few units


LENS = {
    "one key": [(1, 1)],
    "decode": [(1, 333)],
    "long": [(1, 9001)],
    "ragged": [(1, 1), (1, 15), (1, 16), (1, 17), (1, 130), (1, 700), (1, 31)],
    "empty": [(0, 0), (1, 50), (0, 40), (2, 1), (3, 0), (5, 5)],      # rows without a key
    "drafts": [(5, 100), (3, 64), (2, 2), (4, 1000)],
    "prompt": [(150, 150)],
    "chunk": [(67, 300), (1, 90), (33, 33)],
}


@pytest.mark.parametrize("window", [0, 1, 40], ids=["all", "self", "window"])
@pytest.mark.parametrize("kv_heads,group,dim,page", [(2, 4, 128, 64), (1, 1, 64, 16), (3, 5, 64, 32), (1, 8, 256, 16), (2, 16, 128, 256),
                                                     (1, 40, 128, 32)])
@pytest.mark.parametrize("lens", LENS, ids=[n.replace(" ", "-") for n in LENS])
def test_attention(lens, kv_heads, group, dim, page, window):
    print("attention", lens, kv_heads, group, dim, page, window, flush=True)
    case = ref.Case(LENS[lens], kv_heads, dim, page, seed=dim + page)
    cache, batch = case.tensors(DEV)
    q = _queries(case, group)
    got = B.attention_paged(q, cache, batch, scale=_scale(case), window=window, with_lse=True)
    _compare(got, ref.attention(case, q.float().cpu().numpy(), _scale(case), window))


@pytest.mark.parametrize("dim,group", [(64, 3), (128, 4), (256, 2)])
def test_every_key(dim, group):
    """Without the causal mask the earlier tokens see the later ones' keys."""
    case = ref.Case([(4, 4), (1, 40), (37, 100), (2, 1)], 2, dim, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, group)
    got = B.attention_paged(q, cache, batch, scale=_scale(case), causal=False, with_lse=True)
    _compare(got, ref.attention(case, q.float().cpu().numpy(), _scale(case), causal=False))


GROUPS = {
    "one": ([(1, 640 + 17 * i) for i in range(9)], [(9, 640)]),
    "three": ([(1, 131), (2, 150), (1, 128), (1, 700), (3, 513), (1, 64), (1, 66)], [(3, 128), (2, 512), (2, 64)]),
    "one of two": ([(1, 260), (1, 300), (2, 77), (1, 5)], [(2, 256)]),        # the last two share nothing
    "nothing": ([(1, 40), (1, 41)], [(2, 0)]),
    "whole": ([(1, 256), (1, 256)], [(2, 256)]),                               # all keys are shared, the new ones too
    "prompts": ([(40, 296), (1, 257), (33, 300)], [(3, 256)]),
    "singles": ([(1, 300 + i) for i in range(5)], [(1, 256)] * 5),
}


@pytest.mark.parametrize("window", [0, 100], ids=["all", "window"])
@pytest.mark.parametrize("kv_heads,group,dim,page", [(2, 4, 128, 64), (1, 3, 64, 16), (1, 8, 256, 32), (2, 1, 64, 64)])
@pytest.mark.parametrize("groups", GROUPS, ids=[n.replace(" ", "-") for n in GROUPS])
def test_shared_prefixes(groups, kv_heads, group, dim, page, window):
    print("shared", groups, kv_heads, group, dim, page, window, flush=True)
    lens, shared = GROUPS[groups]
    case = ref.Case(lens, kv_heads, dim, page, groups=shared)
    cache, batch = case.tensors(DEV)
    q = _queries(case, group)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    _compare(B.attention_paged(q, cache, batch, scale=_scale(case), window=window, with_lse=True), want)
    alone = {n: v for n, v in batch.items() if n not in ("group_starts", "shared_lens", "max_shared_len")}
    _compare(B.attention_paged(q, cache, alone, scale=_scale(case), window=window, with_lse=True), want)


def test_shared_lengths_are_rounded_down_and_bounded():
    """A shared length inside a page counts its whole pages; one past the bound counts the bound's."""
    case = ref.Case([(1, 200), (1, 210), (2, 290)], 1, 64, 32, groups=[(3, 192)])
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case))
    for given in (192, 191, 161, 31, 0, -5, 1 << 30):
        batch["shared_lens"].fill_(given)
        batch["max_shared_len"] = 192
        _compare(B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True), want)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(3, 40)], [(40, 40)], [(2, 300), (1, 7)]], ids=["drafts", "prompt", "split"])
def test_what_is_not_seen_has_no_effect(dim, lens):
    """NaN and overflowing keys and values at the last position: only the last token sees it."""
    case = ref.Case(lens, 2, dim, 16)
    last = [(int(case.page_table[i, (kv - 1) // 16]), (kv - 1) % 16) for i, (_, kv) in enumerate(lens)]
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    clean = B.attention_paged(q, cache, batch, scale=_scale(case))
    ends = [int(e) - 1 for e in case.q_starts[1:]]
    others = [t for t in range(case.tokens) if t not in ends]
    for what in ("nan value", "nan values", "nan key", "large value", "nan scale", "large key"):
        c = {n: t.clone() for n, t in cache.items()}
        for page, row in last:
            if what == "nan value":
                c["v_codes"][page, :, row, 5] = 0x7F
            elif what == "nan values":
                c["v_codes"][page, :, row] = 0xFF
            elif what == "nan key":
                c["k_codes"][page, :, row, 7] = 0x7F
            elif what == "large value":
                c["v_scales"][page, :, row] = 254
            elif what == "nan scale":
                c["v_scales"][page, :, row, 0], c["k_scales"][page, :, row, 1] = 255, 255
            else:
                c["k_scales"][page, :, row] = 254
        o = B.attention_paged(q, c, batch, scale=_scale(case))
        assert torch.equal(o[others], clean[others]), what
        if what == "nan value":       # that element of those that see it
            assert torch.isnan(o[ends][..., 5]).all() and torch.isfinite(o[ends][..., 6:]).all() and torch.isfinite(o[ends][..., :5]).all()
        if what in ("nan values", "nan key", "nan scale"):
            assert torch.isnan(o[ends][..., :32]).all()


def test_pages_outside_the_cache_and_lengths_outside_the_bounds():
    case = ref.Case([(1, 100), (4, 100), (2, 50), (1, 60)], 2, 64, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 2)
    clean = B.attention_paged(q, cache, batch)
    for bad in (-1, case.k_codes.shape[0], 2147483647, -2147483648):
        t = batch["page_table"].clone()
        t[0, 3], t[1, 6] = bad, bad          # seen by sequence 0; positions 96 .. 99, seen by all of sequence 1 but none before
        o = B.attention_paged(q, cache, dict(batch, page_table=t))
        assert torch.isnan(o[:5]).all() and torch.equal(o[5:], clean[5:])
    for bad in (101, -1, 2147483647, -2147483648):
        lens = batch["kv_lens"].clone()
        lens[1] = bad
        o, lse = B.attention_paged(q, cache, dict(batch, kv_lens=lens), with_lse=True)
        assert torch.isnan(o[1:5]).all() and torch.isnan(lse[1:5]).all()
        assert torch.equal(o[0], clean[0]) and torch.equal(o[5:], clean[5:])


def _raw(q, cache, batch, out, lse, scratch=None, **kw):
    c, b = B._kv_cache(cache, 0)[0], B._kv_batch(batch, 0)
    n, h, d = q.shape
    need = B.fp4q_attention_paged_scratch(c, b, n, h, 0)
    scratch = torch.empty(need, dtype=torch.uint8, device=DEV) if scratch is None else scratch
    B.fp4q_attention_paged(q, n, h, q.stride(0), q.stride(1), c, b, d ** -0.5, 0, 0, out, lse, scratch, need)


LEFT = 2.0 ** 100     # no output's value: values are below 2^8


@pytest.mark.parametrize("kv", [40, 3000])
def test_rows_behind_the_last_sequence_and_past_the_bound_are_left(kv):
    case = ref.Case([(2, kv), (1, 20)], 2, 128, 32, extra_tokens=3)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    out = torch.full((case.tokens, 8, 128), LEFT, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((case.tokens, 8), LEFT, device=DEV)
    _raw(q, cache, batch, out, lse)
    assert (out[3:] == LEFT).all() and (lse[3:] == LEFT).all() and not (out[:3] == LEFT).any()
    out2, lse2 = torch.full_like(out, LEFT), torch.full_like(lse, LEFT)
    _raw(q, cache, dict(batch, max_q_len=1), out2, lse2)      # the second token of sequence 0 is past the bound
    assert (out2[1] == LEFT).all() and torch.equal(out2[[0, 2]], out[[0, 2]])


@pytest.mark.parametrize("lens", ["ragged", "long", "chunk"])
def test_the_same_bits_again_and_with_other_scratch_contents(lens):
    case = ref.Case(LENS[lens], 2, 128, 32)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    first = None
    for fill in (0, 0xFF, 0x7F):
        out = torch.empty(case.tokens, 8, 128, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(case.tokens, 8, device=DEV)
        _raw(q, cache, batch, out, lse, scratch=torch.full((1 << 26,), fill, dtype=torch.uint8, device=DEV))
        if first is None:
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_query_strides():
    case = ref.Case([(3, 50), (1, 400)], 2, 128, 32)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4, row_heads=12)                       # inside a projection's rows
    o = B.attention_paged(q, cache, batch)
    assert torch.equal(o, B.attention_paged(q.contiguous(), cache, batch))
    assert torch.equal(o, B.attention_paged(q.transpose(0, 1).contiguous().transpose(0, 1), cache, batch))


def test_large_and_small_queries_and_scores():
    """Queries far apart in size, NaN and infinities in one row, and a scale that saturates the softmax."""
    case = ref.Case([(4, 70)], 1, 128, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 2)
    q[0, 0] *= 2.0 ** 60
    q[0, 1] *= 2.0 ** -100
    q[1, 0, :64] *= 2.0 ** -9
    q[2, 0, 3], q[2, 1, 100] = float("nan"), float("inf")
    for scale in (1e-3, 0.1, 2.0 ** -62):
        o, lse = B.attention_paged(q, cache, batch, scale=scale, with_lse=True)
        want = ref.attention(case, q.float().cpu().numpy(), scale)
        assert torch.isnan(o[2]).all() and torch.isnan(lse[2]).all()
        keep = [0, 1, 3]
        if scale != 2.0 ** -62:
            keep = [1, 3]
        _compare((o[keep], lse[keep]), tuple(v[keep] for v in want))


def test_refusals():
    case = ref.Case([(2, 20)], 2, 64, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 2)
    for bad, err in [(lambda: B.attention_paged(q.float(), cache, batch), TypeError), (lambda: B.attention_paged(q[..., :32], cache, batch), ValueError),
                     (lambda: B.attention_paged(q[0], cache, batch), ValueError), (lambda: B.attention_paged(q.cpu(), cache, batch), ValueError),
                     (lambda: B.attention_paged(q, dict(cache, k_scales=cache["k_scales"][:1]), batch), ValueError),
                     (lambda: B.attention_paged(q, dict(cache, v_codes=cache["v_codes"].int()), batch), TypeError),
                     (lambda: B.attention_paged(q, cache, dict(batch, kv_lens=batch["kv_lens"].long())), TypeError),
                     (lambda: B.attention_paged(q, cache, dict(batch, q_starts=batch["q_starts"][:1])), ValueError),
                     (lambda: B.attention_paged(q, cache, dict(batch, page_table=batch["page_table"].cpu())), ValueError)]:
        with pytest.raises(err):
            bad()
    for bad, status in [(lambda: B.attention_paged(q[:, :3], cache, batch), 2), (lambda: B.attention_paged(q[:0], cache, batch), 2),
                        (lambda: B.attention_paged(q, cache, dict(batch, max_kv_len=1000)), 2), (lambda: B.attention_paged(q, cache, batch, scale=0.0), 4),
                        (lambda: B.attention_paged(q, cache, batch, scale=float("nan")), 4), (lambda: B.attention_paged(q, cache, batch, window=-1), 2),
                        (lambda: B.attention_paged(q, cache, batch, window=3, causal=False), 4)]:
        with pytest.raises(B.Fp4qError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** 127])
def test_smallest_and_largest_scale(scale):
    """Queries that make up for the scale; few rows and many."""
    for lens in ([(2, 40)], [(70, 130)]):
        case = ref.Case(lens, 1, 64, 16)
        cache, batch = case.tensors(DEV)
        q = (_queries(case, 2).float() * (2.0 ** 120 if scale < 1 else 2.0 ** -124)).to(torch.bfloat16)
        want = ref.attention(case, q.double().cpu().numpy(), scale)
        _compare(B.attention_paged(q, cache, batch, scale=scale, with_lse=True), want)


@pytest.mark.parametrize("window", [0, 20], ids=["all", "window"])
@pytest.mark.parametrize("lens", [[(1, 50), (1, 128), (2, 127), (1, 200), (1, 1), (0, 0)], [(50, 50), (40, 127), (1, 300), (33, 140)]],
                         ids=["tokens", "prompts"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_sequences_that_end_within_the_shared_pages(dim, page, lens, window):
    case = ref.Case(lens, 2, dim, page, groups=[(len(lens), 128)])
    cache, batch = case.tensors(DEV)
    q = _queries(case, 3)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    _compare(B.attention_paged(q, cache, batch, scale=_scale(case), window=window, with_lse=True), want)
