"""Plain binary64 forms of the rotary positions, the paged MXFP8 cache and its attention, for the tests."""
import numpy as np

import mxfp8_ref as ref


def rotary_table(positions, rot, base=10000.0, factor=1.0, original=0.0, low=0.0, high=1.0, amplitude=1.0):
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    if factor != 1.0:
        g = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = f * (g + (1 - g) / factor)
    a = np.arange(positions)[:, None] * f
    return amplitude * np.stack([np.cos(a), np.sin(a)], -1)


def pairs(rot, interleaved):
    """The first and the second elements of the pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cs, interleaved, backward=False):
    """x [tokens][heads][dim], cs [tokens][rot/2][2]: (y, the sums of magnitudes that bound its rounding)."""
    x = np.asarray(x, np.float64)
    cs = np.asarray(cs, np.float64)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1 if backward else 1)
    y, mag = x.copy(), np.zeros(x.shape)
    one, two = pairs(2 * cs.shape[1], interleaved)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    mag[..., one], mag[..., two] = abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)
    return y, mag


def e4m3_codes(rng, *shape):
    """Random finite codes of magnitudes between 1/4 and 15."""
    return ((rng.integers(0, 2, shape) << 7) | (rng.integers(5, 11, shape) << 3) | rng.integers(0, 8, shape)).astype(np.uint8)


class Case:
    """A batch and a cache: `lens` has (query tokens, positions) of each sequence, `groups` a list of (sequences,
    shared positions), whole pages.  Rows of the cache that belong to no sequence hold NaN codes under
    NaN scales; `spare` pages belong to none."""

    def __init__(self, lens, kv_heads, dim, page, groups=(), spare=2, seed=0, extra_tokens=0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.dim, self.page = lens, kv_heads, dim, page
        of = [(g, n) for g, (count, n) in enumerate(groups) for _ in range(count)]
        of += [(None, 0)] * (len(lens) - len(of))
        self.shared_of = of
        width = max(1, max(-(-kv // page) for _, kv in lens)) + 1
        need = sum(-(-kv // page) for _, kv in lens) + sum(n // page for _, n in groups) + spare
        ids = rng.permutation(need)
        self.page_table = np.full((len(lens), width), -7, np.int32)     # entries past the length: nonsense
        self.k_codes = np.full((need, kv_heads, page, dim), 0x7F, np.uint8)
        self.v_codes = np.full((need, kv_heads, page, dim), 0xFF, np.uint8)
        self.k_scales = np.full((need, kv_heads, page, dim // 32), 255, np.uint8)
        self.v_scales = np.full((need, kv_heads, page, dim // 32), 255, np.uint8)
        at, common = 0, []
        for _, n in groups:
            common.append(ids[at:at + n // page])
            at += n // page
        for i, (_, kv) in enumerate(lens):
            g, n = of[i]
            pages = -(-kv // page)
            head = common[g] if g is not None else np.zeros(0, int)
            own = max(0, pages - len(head))
            self.page_table[i, :pages] = np.concatenate([head, ids[at:at + own]])[:pages]
            at += own
            for p in range(pages):
                rows, pid = min(page, kv - p * page), self.page_table[i, p]
                self.k_codes[pid, :, :rows] = e4m3_codes(rng, kv_heads, rows, dim)
                self.v_codes[pid, :, :rows] = e4m3_codes(rng, kv_heads, rows, dim)
                self.k_scales[pid, :, :rows] = rng.integers(123, 127, (kv_heads, rows, dim // 32))
                self.v_scales[pid, :, :rows] = rng.integers(120, 130, (kv_heads, rows, dim // 32))
        self.q_starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.kv_lens = np.array([kv for _, kv in lens], np.int32)
        self.tokens = int(self.q_starts[-1]) + extra_tokens
        self.max_q_len, self.max_kv_len = max(1, max(q for q, _ in lens)), max(1, max(kv for _, kv in lens))
        self.group_starts = np.concatenate([[0], np.cumsum([c for c, _ in groups])]).astype(np.int32) if groups else None
        self.shared_lens = np.array([n for _, n in groups], np.int32) if groups else None

    def rows(self, i, name):
        """Keys or values of sequence i as values [positions][heads][dim]; NaN for pages outside the cache."""
        kv = max(0, int(self.kv_lens[i]))
        out = np.full((kv, self.heads, self.dim), np.nan)
        codes, scales = getattr(self, name + "_codes"), getattr(self, name + "_scales")
        for p in range(-(-kv // self.page)):
            pid, n = int(self.page_table[i, p]), min(self.page, kv - p * self.page)
            if 0 <= pid < codes.shape[0]:
                v = ref.dequantize(codes[pid, :, :n], scales[pid, :, :n])
                v[np.repeat(scales[pid, :, :n], 32, -1) == 255] = np.nan
                out[p * self.page:p * self.page + n] = v.transpose(1, 0, 2)
        return out

    def tensors(self, device):
        import torch

        def put(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(device)
        cache = {n: put(getattr(self, n)) for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
        batch = {n: put(getattr(self, n)) for n in ("q_starts", "kv_lens", "page_table")}
        batch["max_q_len"], batch["max_kv_len"] = self.max_q_len, self.max_kv_len
        if self.group_starts is not None:
            batch["group_starts"], batch["shared_lens"] = put(self.group_starts), put(self.shared_lens)
            batch["max_shared_len"] = int(self.shared_lens.max())
        return cache, batch


def attention(case, q, scale, window=0, causal=True):
    """(out, lse, bound of |out|, bound of |lse|) of q [tokens][q heads][dim]; rows of no sequence are NaN.

    The bounds count: fp32 sums of up to 256 products (exact: eight bits times four), 2^-16 of the sum of their
    magnitudes; the exponential, 2^-21 of its argument's magnitude and 2^-21; p's
    rounding to bf16, 2^-8 of each; fp32 sums of up to 2^14 of them in parts, 2^-16; out's rounding, 2^-8."""
    q = np.asarray(q, np.float64)
    group = q.shape[1] // case.heads
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    tol, tol_lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    with np.errstate(all="ignore"):
        for i in range(len(case.lens)):
            a, b = int(case.q_starts[i]), int(case.q_starts[i + 1])
            kv = int(case.kv_lens[i])
            k, v = case.rows(i, "k"), case.rows(i, "v")
            pos = kv - (b - a) + np.arange(b - a)[:, None]
            key = np.arange(kv)[None]
            see = (key <= pos) if causal else np.broadcast_to(True, (b - a, kv)).copy()
            if window:
                see &= key > pos - window
            for h in range(q.shape[1]):
                x, kk, vv = q[a:b, h], k[:, h // group], v[:, h // group]
                for t in range(b - a):
                    m = see[t]
                    if not m.any():
                        out[a + t, h], lse[a + t, h] = 0.0, -np.inf
                        continue
                    s = scale * (kk[m] @ x[t])
                    mag = scale * (abs(kk[m]) @ abs(x[t]))
                    top = s.max()
                    p = np.exp(s - top)
                    total = p.sum()
                    out[a + t, h] = (p @ vv[m]) / total
                    lse[a + t, h] = top + np.log(total)
                    e = 2.0 ** -16 * mag.max() + 2.0 ** -21 * (abs(s).max() + 1)
                    each = np.exp(2 * e) - 1 + 2.0 ** -8 + 2.0 ** -16
                    tol[a + t, h] = each * ((p @ abs(vv[m])) / total) + 2.0 ** -8 * abs(out[a + t, h]) + 1e-30
                    tol_lse[a + t, h] = e + 2.0 ** -16 + 2.0 ** -22 * abs(lse[a + t, h])
    return out, lse, tol, tol_lse
