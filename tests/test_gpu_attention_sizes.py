"""Attention over the paged cache at the ends of the shapes that it takes (GPU)."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_attention import LEFT, _compare, _queries, _scale

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


def test_more_workgroups_than_a_launch_takes():
    """16500 groups of one token on 1023 heads: a row tile and a joined row for each, all on the same pages.  Every 16th token sees the same."""
    seqs, heads, page = 16500, 1023, 16
    case = ref.Case([(1, 17 + i) for i in range(16)], heads, 64, page, groups=[(16, 16)])
    cache, batch = case.tensors(DEV)
    again = torch.arange(seqs, device=DEV) % 16
    i32 = dict(dtype=torch.int32, device=DEV)
    batch = {"q_starts": torch.arange(seqs + 1, **i32), "kv_lens": batch["kv_lens"][again], "page_table": batch["page_table"][again].contiguous(),
             "max_q_len": 1, "max_kv_len": case.max_kv_len, "group_starts": torch.arange(seqs + 1, **i32),
             "shared_lens": torch.full((seqs,), 16, **i32), "max_shared_len": 16}
    one = torch.randn(1, 1, 64, generator=torch.Generator(device=DEV).manual_seed(0), device=DEV).to(torch.bfloat16)
    o, lse = B.attention_paged(one.expand(seqs, heads, 64), cache, batch, scale=_scale(case), with_lse=True)
    first = o[:16].clone(), lse[:16].clone()
    for at in range(16, seqs, 16):
        n = min(16, seqs - at)
        assert torch.equal(o[at:at + n], first[0][:n]) and torch.equal(lse[at:at + n], first[1][:n]), at
    some = [0, 500, 1022]
    for n in cache:
        setattr(case, n, getattr(case, n)[:, some])
    case.heads = len(some)
    q = one.expand(16, len(some), 64).float().cpu().numpy()
    _compare((first[0][:, some], first[1][:, some]), ref.attention(case, q, _scale(case)))


def _mixed(seqs, long, seed=0):
    """Mostly single tokens, some drafts and some without tokens, and a prompt or a chunk behind every `long`."""
    rng = np.random.default_rng(seed)
    lens = []
    for i in range(seqs):
        n = int(rng.integers(33, 200)) if i % long == long - 1 else int(rng.integers(0, 4))
        lens.append((n, n + int(rng.integers(0, 60))))
    return lens


@pytest.mark.parametrize("seqs,long", [(9, 4), (63, 31), (64, 20), (65, 64), (300, 50)])
@pytest.mark.parametrize("window", [0, 25], ids=["all", "window"])
def test_prompts_among_tokens(seqs, long, window):
    case = ref.Case(_mixed(seqs, long, seqs), 1, 64, 16, seed=seqs, extra_tokens=3)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    got = B.attention_paged(q, cache, batch, scale=_scale(case), window=window, with_lse=True)
    n = int(case.q_starts[-1])
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    _compare(tuple(t[:n] for t in got), tuple(t[:n] for t in want))


@pytest.mark.parametrize("groups", [2, 9, 63, 64, 70, 200])
def test_many_groups(groups):
    """Groups of one to four sequences, some of several tokens, some empty, their prefixes of one to four pages."""
    rng = np.random.default_rng(groups)
    lens, shared = [], []
    for g in range(groups):
        count, prefix = int(rng.integers(1, 5)), 16 * int(rng.integers(1, 5))
        shared.append((count, prefix))
        lens += [(q, prefix + q + int(kv)) for q, kv in zip(rng.choice([0, 1, 1, 1, 2, 9, 40], count).tolist(), rng.integers(0, 40, count))]
    case = ref.Case(lens, 1, 64, 16, groups=shared, seed=groups)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case))
    _compare(B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True), want)


def test_thousands_of_sequences():
    """More than two searches of 64 places in the starts, with prompts between them and groups of two at the end."""
    seqs = 4400
    lens = _mixed(seqs, 500)
    for i in range(4300, seqs, 2):
        lens[i], lens[i + 1] = (1, 40), (2, 50)
    case = ref.Case(lens, 1, 64, 16, groups=[(1, 0)] * 4300 + [(2, 32)] * 50)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    got = B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True)
    some = [0, 1, 700, case.tokens - 1, case.tokens - 2, case.tokens - 3, case.tokens - 75]
    for i in range(499, seqs, 500):
        some += [int(case.q_starts[i]), int(case.q_starts[i]) + 17, int(case.q_starts[i + 1]) - 1]
    _compare(tuple(t[some] for t in got), _some_rows(case, q, some))


@pytest.mark.parametrize("window", [0, 60])
def test_prompts_among_tokens_with_more_tokens_than_the_bound(window):
    lens = [(1, 50)] * 20 + [(300, 1000)] + [(1, 70)] * 20 + [(120, 130), (0, 5)]
    case = ref.Case(lens, 1, 64, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    o, lse = B.attention_paged(q, cache, dict(batch, max_q_len=100), scale=_scale(case), window=window, with_lse=True)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case), window)
    done = [t for a, b in zip(case.q_starts, case.q_starts[1:]) for t in range(int(a), min(int(b), int(a) + 100))]
    _compare((o[done], lse[done]), tuple(v[done] for v in want))


@pytest.mark.parametrize("groups", [(), [(20, 512)]], ids=["own", "shared"])
def test_bounds_far_past_the_lengths(groups):
    """max_kv_len of 2^30: the keys of all pairs that the bounds allow are more than 32 bits can count in units of 128."""
    heads = 64
    lens = [(1, 513 + 71 * i * i) for i in range(10)] + [(i, 600 + 16 * i) for i in range(10)]
    case = ref.Case(lens, heads, 64, 1024 if not groups else 512, groups=groups)
    cache, batch = case.tensors(DEV)
    width = (1 << 30) // case.page
    table = torch.full((len(lens), width), -7, dtype=torch.int32, device=DEV)
    table[:, :case.page_table.shape[1]] = batch["page_table"]
    q, some = _queries(case, 1), [0, 31, 63]
    o, lse = B.attention_paged(q, cache, dict(batch, page_table=table, max_kv_len=1 << 30), scale=_scale(case), with_lse=True)
    for n in cache:
        setattr(case, n, getattr(case, n)[:, some])
    case.heads = len(some)
    _compare((o[:, some], lse[:, some]), ref.attention(case, q[:, some].float().cpu().numpy(), _scale(case)))


def test_a_chunk_among_many_sequences_in_small_pages():
    """1023 single tokens and a chunk of 8192 tokens, where contexts may have 131072 positions in pages of 16."""
    lens = [(1, 40)] * 1023 + [(8192, 20000)]
    case = ref.Case(lens, 1, 64, 16)
    cache, batch = case.tensors(DEV)
    table = torch.full((len(lens), 8192), -7, dtype=torch.int32, device=DEV)
    table[:, :case.page_table.shape[1]] = batch["page_table"]
    q = _queries(case, 4)
    got = B.attention_paged(q, cache, dict(batch, page_table=table, max_kv_len=131072), scale=_scale(case), with_lse=True)
    some = [0, 500, 1022, 1023, 1024, 5000, 9213, 9214]
    _compare(tuple(t[some] for t in got), _some_rows(case, q, some))


def test_captured_and_replayed_while_the_prompts_move():
    """Most tokens are a prompt's, of another sequence in each replay; the bounds and the number of tokens stay."""
    seqs, tokens = 40, 400
    g = np.random.default_rng(0)
    case = ref.Case([(1, 420)] * seqs, 2, 64, 16)
    cache, batch = case.tensors(DEV)
    batch.update(max_q_len=300, group_starts=torch.tensor([0, 3, 40], dtype=torch.int32, device=DEV),
                 shared_lens=torch.zeros(2, dtype=torch.int32, device=DEV), max_shared_len=64)
    q = torch.randn(tokens, 8, 64, device=DEV).to(torch.bfloat16)
    batch["page_table"][1:3, :4] = batch["page_table"][:1, :4]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.attention_paged(q, cache, batch, with_lse=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = B.attention_paged(q, cache, batch, with_lse=True)
    for i in range(12):
        n = g.integers(0, 3, seqs)
        n[(7 * i) % seqs] = 300 if i % 3 else 0
        n[(7 * i + 5) % seqs] = g.integers(9, 40)
        starts = np.minimum(np.concatenate([[0], np.cumsum(n)]), tokens)
        batch["q_starts"].copy_(torch.from_numpy(starts.astype(np.int32)))
        batch["shared_lens"][0] = 64 * (i % 2)
        q.copy_(torch.randn(q.shape, device=DEV))
        out.fill_(LEFT), lse.fill_(LEFT)
        graph.replay()
        torch.cuda.synchronize()
        want = B.attention_paged(q, cache, batch, with_lse=True)
        end = int(starts[-1])
        assert torch.equal(out[:end], want[0][:end]) and torch.equal(lse[:end], want[1][:end]), i
        assert (out[end:] == LEFT).all() and not (lse[:end] == LEFT).any(), i
