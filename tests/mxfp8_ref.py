"""Plain binary64 forms of MXFP8, the RMS norm and MXFP4 decoding, for the tests."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_values() -> np.ndarray:
    """The value of each E4M3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(c >> 7, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Values of magnitude up to 448, rounded to E4M3's nearest, ties to even (as values)."""
    e = np.frexp(v)[1]
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.round(v / step) * step


def scale_code(bmax: np.ndarray) -> np.ndarray:
    """The smallest c >= 0 with bmax <= 448 * 2^(c - 127), by search from the estimate."""
    c = np.zeros(bmax.shape, dtype=np.int64)
    pos = bmax > 0
    c[pos] = np.maximum(np.ceil(np.log2(bmax[pos] / 448.0)).astype(np.int64) + 127 - 1, 0)
    for _ in range(3):
        c = np.where(bmax > np.ldexp(448.0, (c - 127).astype(np.int32)), c + 1, c)
    return c


def quantize(x: np.ndarray):
    """(values of the codes, scale codes) of x [rows][cols] in binary64; NaN where x is not finite."""
    v = x.astype(np.float64).reshape(x.shape[0], -1, 32)
    fin = np.isfinite(v)
    c = scale_code(np.where(fin, np.abs(v), 0).max(-1))
    q = np.where(fin, v, 0) * np.ldexp(1.0, (127 - c).astype(np.int32))[..., None]
    out = np.where(fin, e4m3_round(q), np.nan)
    return out.reshape(x.shape), c


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return e4m3_values()[codes] * np.repeat(np.ldexp(1.0, scales.astype(np.int32) - 127), 32, axis=-1)


def fp4(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """MXFP4 codes [..][k/2] and scales [..][k/32] as values."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(n & 8, -E2M1[n & 7], E2M1[n & 7])
    return v * np.repeat(np.ldexp(1.0, scales.astype(np.int32) - 127), 32, axis=-1)


def rmsnorm(x, gain, residual=None, eps=1e-6):
    """(sum, rstd, y) in binary64."""
    s = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((s * s).mean(-1) + eps)
        return s, r, s * r[:, None] * gain.astype(np.float64)


def rmsnorm_backward(dy, s, gain, r, dsum=None):
    """(dx, dgain) in binary64, and the sums of magnitudes that bound their rounding."""
    dy, s, gain, r = (np.asarray(v, np.float64) for v in (dy, s, gain, r))
    n = s.shape[1]
    a, r1 = dy * gain, r[:, None]
    dx = r1 * a - s * (r1 ** 3) * (a * s).sum(-1, keepdims=True) / n
    mag = np.abs(r1 * a) + np.abs(s) * r1 ** 3 * np.abs(a * s).sum(-1, keepdims=True) / n
    if dsum is not None:
        dx, mag = dx + dsum, mag + np.abs(dsum)
    t = dy * s * r1
    return dx, t.sum(0), mag, np.abs(t).sum(0)
