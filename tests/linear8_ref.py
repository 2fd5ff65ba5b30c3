"""64-bit definitions of the block-scaled 8-bit linear layer (not a test module).

Written from the definitions in include/rankmixer.h with numpy, without the
package.  Values of a quantised array are held as float64 codes and exponents.
"""
import numpy as np

BLOCK = 128
E4M3_HALF = 2.0 ** -4      # half a step of e4m3, relative to the value (3 bits behind the leading one)
BF16_HALF = 2.0 ** -8
F32_HALF = 2.0 ** -24


def decode_e4m3(b: np.ndarray) -> np.ndarray:
    """Values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7, -v, v)


def decode_scale(b: np.ndarray) -> np.ndarray:
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of |x| <= 448, ties to even."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.round(x / step) * step


def block_max(x: np.ndarray, block_rows: int) -> np.ndarray:
    """Largest magnitude of each block of x [.., rows, cols]; NaN for a block that is not finite."""
    rows, cols = x.shape[-2:]
    pr, pc = -rows % block_rows, -cols % BLOCK
    a = np.where(np.isfinite(x), np.abs(x), np.nan)
    a = np.pad(a, [(0, 0)] * (x.ndim - 2) + [(0, pr), (0, pc)])
    a = a.reshape(x.shape[:-2] + ((rows + pr) // block_rows, block_rows, (cols + pc) // BLOCK, BLOCK))
    return a.max(axis=(-3, -1))


def exponents(amax: np.ndarray) -> np.ndarray:
    """Smallest e in [-127, 127] with amax <= 448 * 2^e (0 for a zero block); NaN stays."""
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.ceil(np.log2(amax / 448.0))
        e = np.where(448.0 * 2.0 ** (e - 1) >= amax, e - 1, e)
        e = np.where(448.0 * 2.0 ** e < amax, e + 1, e)
    return np.where(amax == 0, 0.0, np.clip(e, -127, 127))


def spread(s: np.ndarray, rows: int, cols: int, block_rows: int) -> np.ndarray:
    return np.repeat(np.repeat(s, block_rows, -2)[..., :rows, :], BLOCK, -1)[..., :cols]


def quantize(x: np.ndarray, block_rows: int):
    """Code values and scale bytes of x [.., rows, cols]."""
    e = exponents(block_max(x, block_rows))
    with np.errstate(invalid="ignore"):
        codes = round_e4m3(x / spread(2.0 ** e, x.shape[-2], x.shape[-1], block_rows))
    codes = np.where(np.isnan(spread(e, x.shape[-2], x.shape[-1], block_rows)), np.nan, codes)
    return codes, np.where(np.isnan(e), 255, e + 127).astype(np.int64)


def values(codes: np.ndarray, scale_bytes: np.ndarray, block_rows: int) -> np.ndarray:
    return codes * spread(decode_scale(scale_bytes), codes.shape[-2], codes.shape[-1], block_rows)


def activation(v: np.ndarray, act):
    from scipy.special import erf
    if act == "tanh":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    if act == "erf":
        return 0.5 * v * (1 + erf(v / np.sqrt(2)))
    return np.maximum(v, 0) if act == "relu" else v


def rmsnorm(s: np.ndarray, gamma: np.ndarray, eps: float):
    rstd = 1 / np.sqrt((s * s).mean(-1) + eps)
    return s * rstd[:, None] * gamma, rstd


def rmsnorm_grad(dy, s, gamma, rstd, dsum):
    a = dy * gamma
    r = rstd[:, None]
    dx = r * (a - s * r ** 2 * (a * s).mean(-1, keepdims=True)) + dsum
    return dx, (dy * s * r).sum(0)


def assert_quantized(codes, scale_bytes, ref, slack, what=""):
    """codes * 2^(bytes - 127) is ref [.., rows, cols] rounded to e4m3 in blocks of 1 x 128, ref itself known up to
    `slack` (an array of absolute errors): every scale is the right one for some value within the slack, every code
    is within half a step."""
    rows, cols = ref.shape[-2:]
    lo, hi = block_max(np.maximum(np.abs(ref) - slack, 0), 1), block_max(np.abs(ref) + slack, 1)
    e = scale_bytes.astype(np.float64) - 127
    elo, ehi = exponents(lo), exponents(hi)
    assert np.all((e >= elo) & (e <= ehi) | ((lo == 0) & (e == 0))), f"{what}: scale off"
    s = spread(2.0 ** e, rows, cols, 1)
    half = np.maximum(np.abs(ref) * E4M3_HALF, s * 2.0 ** -10)
    bad = np.abs(codes * s - ref) > half * (1 + 1e-12) + slack * (1 + E4M3_HALF)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes more than half a step off"
