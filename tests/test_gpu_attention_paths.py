"""Rotary positions, the cache and its attention as a program uses them (GPU): step after step, captured and
replayed, on another stream, two calls at once, prompts and decoded tokens in one batch."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import mxfp8_ref
from block_scaled_fp4_05_amd import binding as B
from test_gpu_attention import _compare, _queries, _scale

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


class Program:
    """Two sequences in one cache, their tokens given step by step, and the same in binary64 from the inputs."""

    def __init__(self, heads=2, group=3, dim=64, page=16, rot=40):
        self.heads, self.group, self.dim, self.page = heads, group, dim, page
        self.cache = B.kv_cache(40, page, heads, dim)
        self.table = B.rotary_table(512, rot)
        ids = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.pages = torch.stack([ids[:20], ids[20:]]).to(DEV)
        self.lens, self.k, self.v = [0, 0], [[], []], [[], []]
        self.g = torch.Generator(device=DEV).manual_seed(2)

    def step(self, counts):
        """counts[s] more tokens of each sequence: (out, lse) and what they should be, with its bounds."""
        n, h = sum(counts), self.heads
        x = torch.randn(n, h * (self.group + 2), self.dim, generator=self.g, device=DEV).to(torch.bfloat16)
        q, k, v = x[:, :h * self.group], x[:, h * self.group:h * (self.group + 1)], x[:, h * (self.group + 1):]
        starts = np.concatenate([[0], np.cumsum(counts)])
        self.lens = [a + c for a, c in zip(self.lens, counts)]
        batch = {"q_starts": torch.tensor(starts, **I32), "kv_lens": torch.tensor(self.lens, **I32), "page_table": self.pages,
                 "max_q_len": max(max(counts), 1), "max_kv_len": max(self.lens)}
        pos = torch.tensor([p for a, c in zip(self.lens, counts) for p in range(a - c, a)], **I32)
        turned = B.rotary(q, self.table, pos)
        B.kv_append(self.cache, batch, k, v, table=self.table)
        got = B.attention_paged(turned, self.cache, batch, with_lse=True)
        cs = self.table[pos.long()].cpu().numpy()
        kr = ref.rotate(k.float().cpu().numpy(), cs, False)[0]
        for s in range(2):
            self.k[s].append(kr[starts[s]:starts[s + 1]])
            self.v[s].append(v[starts[s]:starts[s + 1]].float().cpu().numpy().astype(np.float64))
        case = ref.Case([(c, a) for c, a in zip(counts, self.lens)], h, self.dim, self.page)
        case.rows = lambda i, name: self._values(getattr(self, name)[i])
        return got, ref.attention(case, turned.float().cpu().numpy(), self.dim ** -0.5)

    def _values(self, parts):
        x = np.concatenate(parts)
        q, c = mxfp8_ref.quantize(x.reshape(-1, self.dim))
        return (q * np.repeat(np.ldexp(1.0, (c - 127).astype(np.int32)), 32, -1)).reshape(x.shape)


def test_prompts_then_tokens_then_drafts():
    p = Program()
    for counts in ([37, 5], [1, 1], [1, 1], [0, 70], [4, 1], [1, 0], [90, 2], [1, 1]):
        _compare(*p.step(counts))


LARGE = {
    "a long prompt": [(1300, 1300)],
    "prompts and tokens": [(1, 5000), (300, 900), (1, 64), (33, 33), (4, 2000)],
    "a chunk far back": [(129, 4100), (1, 1)],
}


@pytest.mark.parametrize("dim,kv_heads,group,page", [(64, 1, 8, 64), (128, 2, 2, 32), (256, 1, 4, 128)])
@pytest.mark.parametrize("lens", LARGE, ids=[n.replace(" ", "-") for n in LARGE])
def test_long_batches(lens, dim, kv_heads, group, page):
    print("long", lens, dim, kv_heads, group, page, flush=True)
    case = ref.Case(LARGE[lens], kv_heads, dim, page)
    cache, batch = case.tensors(DEV)
    q = _queries(case, group)
    got = B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True)
    rows = [0, 1, case.tokens // 2, case.tokens - 2, case.tokens - 1] + list(range(7, case.tokens, 97))
    want = _rows_of(case, q, rows)
    _compare(tuple(t[rows] for t in got), want)


def _rows_of(case, q, rows):
    """ref.attention for some of the query rows."""
    one = [None] * 4
    outs = []
    for t in rows:
        i = int(np.searchsorted(case.q_starts, t, side="right")) - 1
        sub = object.__new__(ref.Case)
        sub.__dict__.update(case.__dict__)
        kv = int(case.kv_lens[i]) - (int(case.q_starts[i + 1]) - t) + 1
        sub.lens, sub.q_starts, sub.kv_lens = [(1, kv)], np.array([0, 1]), np.array([kv])
        sub.page_table = case.page_table[i:i + 1]
        outs.append(ref.attention(sub, q[t:t + 1].float().cpu().numpy(), _scale(case)))
    for k in range(4):
        one[k] = np.concatenate([o[k] for o in outs])
    return tuple(one)


@pytest.mark.parametrize("seqs", [63, 64, 65, 257, 300, 1000])
def test_many_sequences(seqs):
    """More sequences than a wave's or a workgroup's lanes, some without tokens, in the append and the attention."""
    rng = np.random.default_rng(seqs)
    lens = [(int(q), int(q + kv)) for q, kv in zip(rng.integers(0, 3, seqs), rng.integers(0, 90, seqs))]
    case = ref.Case(lens, 1, 64, 32, seed=seqs)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 2)
    want = ref.attention(case, q.float().cpu().numpy(), _scale(case))
    _compare(B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True), want)
    k = torch.randn(case.tokens, 1, 64, device=DEV)
    B.kv_append(cache, batch, k, -k)
    for i, (n, kv) in enumerate(lens):
        for j in range(n):
            at = kv - n + j
            page, row = int(case.page_table[i, at // 32]), at % 32
            t = int(case.q_starts[i]) + j
            assert torch.equal(cache["k_codes"][page, :, row], B.quantize_mxfp8(k[t])["codes"]), (i, j)


def test_captured_and_replayed_while_lengths_change():
    """A decode step in a graph: the batch's lengths, pages and inputs change between the replays."""
    seqs, heads, group, dim, page, width = 5, 2, 4, 128, 16, 40
    g = torch.Generator(device=DEV).manual_seed(0)
    cache = B.kv_cache(seqs * width, page, heads, dim)
    table = B.rotary_table(width * page, dim)
    batch = {"q_starts": torch.arange(seqs + 1, **I32), "kv_lens": torch.ones(seqs, **I32),
             "page_table": torch.randperm(seqs * width, generator=g, device=DEV).to(torch.int32).view(seqs, width),
             "max_q_len": 1, "max_kv_len": width * page, "group_starts": torch.tensor([0, 3, seqs], **I32),
             "shared_lens": torch.zeros(2, **I32), "max_shared_len": 128}
    x = torch.zeros(seqs, heads * (group + 2), dim, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(seqs, **I32)

    def step():
        q = B.rotary(x[:, :heads * group], table, pos)
        B.kv_append(cache, batch, x[:, heads * group:heads * (group + 1)], x[:, heads * (group + 1):], table=table)
        return B.attention_paged(q, cache, batch, with_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(40):
        n = torch.randint(0, 16, (seqs,), generator=g, device=DEV, dtype=torch.int32) * (i % 3 == 0)
        batch["kv_lens"].add_(1 + n).clamp_(max=width * page)
        if i == 20:      # from now on three sequences share their first pages
            batch["page_table"][1:3, :8] = batch["page_table"][:1, :8]
            batch["kv_lens"].clamp_(min=130)
            batch["shared_lens"][0] = 128
        pos.copy_(batch["kv_lens"] - 1)
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        before = {n: t.clone() for n, t in cache.items()}
        graph.replay()
        torch.cuda.synchronize()
        after = {n: t.clone() for n, t in cache.items()}
        got = out.clone(), lse.clone()
        for n, t in cache.items():
            t.copy_(before[n])
        want = step()
        assert all(torch.equal(cache[n], after[n]) for n in cache), i
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def _calls():
    case = ref.Case([(1, 700), (40, 40), (1, 33)], 2, 128, 16, groups=[(1, 512)])
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    k = torch.randn(case.tokens, 2, 128, device=DEV).to(torch.bfloat16)
    table = B.rotary_table(1024, 128)
    pos = torch.arange(case.tokens, **I32)
    return {
        "rotary": lambda s: B.rotary(q, table, pos, stream=s),
        "table": lambda s: B.rotary_table(1024, 128, stream=s),
        "append": lambda s: B.kv_append({n: t.clone() for n, t in cache.items()}, batch, k, k, table=table, stream=s),
        "attention": lambda s: B.attention_paged(q, cache, batch, with_lse=True, stream=s),
    }


def _flat(out):
    return list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("name", ["rotary", "table", "append", "attention"])
def test_another_stream(name):
    call = _calls()[name]
    want = _flat(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handles = {"stream": side, "handle": side.cuda_stream, "null": 0}
    for kind, s in handles.items():
        got = _flat(call(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), kind


def test_two_calls_at_once():
    """Long calls on two streams at the same time, each with scratch of its own."""
    cases = [ref.Case([(1, 4000 + 100 * i), (1, 50)], 4, 128, 64, seed=i) for i in range(2)]
    inputs = [(*c.tensors(DEV), _queries(c, 4)) for c in cases]
    want = [B.attention_paged(q, cache, batch, with_lse=True) for cache, batch, q in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            cache, batch, q = inputs[i]
            with torch.cuda.stream(s):
                got[i].append(B.attention_paged(q, cache, batch, with_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for o in got[i] for a, b in zip(o, want[i]))


def test_before_the_projection():
    """The output goes on as an MXFP8 operand of an MXFP4 weight, as the layer's other activations do."""
    case = ref.Case([(1, 300), (3, 60)], 2, 64, 16)
    cache, batch = case.tensors(DEV)
    q = _queries(case, 4)
    o = B.attention_paged(q, cache, batch, scale=_scale(case))
    w = B.quantize_mxfp4(torch.randn(96, 512, device=DEV).to(torch.bfloat16))
    a = B.quantize_mxfp8(o.view(case.tokens, 512))
    y = B.gemm_mxfp8_mxfp4(a, w)
    x = mxfp8_ref.dequantize(a["codes"].cpu().numpy(), a["scales"].cpu().numpy())
    v = mxfp8_ref.fp4(w["codes"].cpu().numpy(), w["scales"].cpu().numpy())
    # the product's documented cut: 13 bits below the largest of a few neighbours, and fp32 sums of 512 terms
    assert np.all(np.abs(y.cpu().numpy() - x @ v.T) <= (2.0 ** -12 + 2.0 ** -15) * (np.abs(x) @ np.abs(v).T))


@pytest.mark.parametrize("lens,groups", [([(40, 8300)], ()), ([(20, 8250), (20, 8300)], [(2, 8192)]), ([(40, 8300), (33, 8250)], [(2, 8192)])],
                         ids=["own", "shared", "both"])
def test_long_pieces(lens, groups):
    """So many heads and keys that a CU has two workgroups, with long pieces of them; two heads are compared."""
    case = ref.Case(lens, 128, 64, 64, groups=groups)
    cache, batch = case.tensors(DEV)
    q, some = _queries(case, 1), [3, 126]
    o, lse = B.attention_paged(q, cache, batch, scale=_scale(case), with_lse=True)
    for n in cache:
        setattr(case, n, getattr(case, n)[:, some])
    case.heads = len(some)
    _compare((o[:, some], lse[:, some]), ref.attention(case, q[:, some].float().cpu().numpy(), _scale(case)))
