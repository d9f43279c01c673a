"""The key/value cache and attention in 64 bits, row by row, from their
definitions (include/qw3.h).  Shares no code with the GPU path.

The only arithmetic in fewer bits is the cache's own definition: the scale
a / L and the quotient x / s are float32 divisions, and a value read back is the
float32 product c s rounded to bf16.
"""
import numpy as np

LIMIT = {"int8": 127.0, "e4m3": 448.0}


def bf16_values(bits):
    """Values of bf16 bit patterns (uint16) as float64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(x):
    """float32 -> bf16 bit patterns, nearest, ties to even; NaN -> 0x7fc0."""
    x = np.asarray(x, np.float32)
    u = x.view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def e4m3_table():
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f and 0xff NaN)."""
    v = np.zeros(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            x = np.nan
        v[c] = -x if s else x
    return v


def code_values(codes, kind):
    """uint8 codes as the numbers they are (the scale not applied)."""
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_table()[codes]


def quantise(rows, kind):
    """float32 rows [..., D] -> (uint8 codes [..., D], float32 scales [...])."""
    rows = np.asarray(rows, np.float32)
    limit = np.float32(LIMIT[kind])
    codes = np.zeros(rows.shape, np.uint8)
    scales = np.zeros(rows.shape[:-1], np.float32)
    positive = e4m3_table()[:127]  # 0 .. 448 in ascending order
    for at in np.ndindex(rows.shape[:-1]):
        x = rows[at]
        if not np.isfinite(x).all():
            scales[at] = np.nan
            continue
        s = np.float32(np.abs(x).max() / limit)
        scales[at] = s
        if not s > 0:
            continue
        y = np.clip((x / s).astype(np.float32), -limit, limit).astype(np.float64)
        if kind == "int8":
            codes[at] = np.rint(y).astype(np.int8).view(np.uint8)
        else:
            hi = np.clip(np.searchsorted(positive, np.abs(y)), 0, 126)
            lo = np.maximum(hi - 1, 0)
            below, above = np.abs(y) - positive[lo], positive[hi] - np.abs(y)
            pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
            codes[at] = pick | (np.signbit(y) << 7)
    return codes, scales


def attend(q, k, v, sees, scale, weight_error=2.0 ** -8):
    """One query row over the keys it sees: (output [D], bound [D]).

    q [D], k and v [n, D] in float64, `sees` the indexes of the visible keys.
    The bound is on what a kernel may be off that multiplies exact operands, holds scores and sums in fp32 and rounds
    each weight and the output to bf16 (8 significant bits, so by at most 2^-8 of their size each): with w_j the normalised weights and A = sum w_j |v_j|,
      2^-8 (A + |o|)          the weights' and the output's rounding (weight_error A + 2^-8 |o| where
                              weights keep more bits: 2^-16 for two bf16 each),
      A (2 d + (n + 64) 2^-23) scores off by d, and the order of n additions in fp32 twice (numerator, denominator),
    d = 2 D 2^-24 scale max_j sum |q k_j|."""
    dim = q.shape[0]
    if len(sees) == 0:
        return np.zeros(dim), np.zeros(dim)
    k, v = k[sees], v[sees]
    s = k @ q * scale
    if not np.isfinite(s).all():
        return np.full(dim, np.nan), np.full(dim, np.inf)
    w = np.exp(s - s.max())
    w /= w.sum()
    o, a = w @ v, w @ np.abs(v)
    d = 2 * dim * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q)).max()
    rounding = weight_error * a + 2.0 ** -8 * np.abs(o)
    return o, 1.02 * rounding + a * (2 * d + (len(sees) + 64) * 2.0 ** -23) + 1e-37


def prompt_sees(i, nq, nk, causal):
    """The keys that row i of a sequence sees."""
    return np.arange(max(0, min(nk, i + nk - nq + 1)) if causal else nk)


def cache_sees(i, n, length, word=None):
    """The cached tokens that new token i of n sees; `word`: its tree mask, None for a chain."""
    ctx = length - n
    seen = list(range(max(0, min(ctx, length))))
    for j in range(n):
        if 0 <= ctx + j < length and (j <= i if word is None else j < 64 and (int(word) >> j) & 1):
            seen.append(ctx + j)
    return np.array(seen, int)


# Counting keys.  With q = 0 every weight is one, and with values that are one in
# one channel and zero elsewhere an output is the share of the row's keys that have
# their one there.  32 neighbouring keys share a channel, so that a lost run of keys
# is not lost from all channels alike, and a channel has at most 96 keys, so that one
# lost or counted twice (1 / 96 of it) is more than bf16 rounds away.

def counting_parts(n, dim):
    """How many sets of values it takes for channels of at most 96 of n keys."""
    return max(1, -(-n // (96 * dim)))


def counting_values(n, dim, part, parts):
    """Values [n, dim]: key j has its one in channel (j // 32) % dim, in set (j // (32 dim)) % parts only."""
    v = np.zeros((n, dim))
    j = np.arange(n)
    j = j[(j // (32 * dim)) % parts == part]
    v[j, (j // 32) % dim] = 1.0
    return v


def miscounted(got, seen, values):
    """Outputs [rows, dim] that are not the shares of the keys `seen` [rows, n]: off by more than the rounding to bf16
    (2^-8) and of one reciprocal and product in fp32."""
    seen = np.asarray(seen, np.float64)
    total = seen.sum(axis=1, keepdims=True)
    want = np.where(total > 0, seen @ values / np.maximum(total, 1), 0.0)
    return ~(np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -20))


# Two weights whose rounding to one bf16 shows: keys of score 0 and of score ln p,
# p = 0.75 + 2^-9 half way between two bf16, whose values cancel.
HALF_WAY = float(np.log(0.75 + 2.0 ** -9))
