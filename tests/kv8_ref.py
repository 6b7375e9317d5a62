"""Plain 64-bit forms of the 8-bit cache's rows, for the tests."""
import numpy as np

from kv4_ref import E4M3, nearest_even

E_MIN, E_MAX = -100, 120
TOP = 240.0 * 2.0 ** 120  # the largest magnitude that is stored


def needed(amax):
    """The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    e = E_MIN
    while amax > 448.0 * 2.0 ** e and e < E_MAX:
        e += 1
    return e


def encode(x, e):
    """Values -> e4m3 codes of x / 2^e, the nearest, ties to the even code."""
    return (nearest_even(np.abs(x) * 2.0 ** -float(e), E4M3) | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def decode(codes, e):
    c = codes.astype(np.int64)
    v = np.where((c & 127) == 127, np.nan, E4M3[np.minimum(c & 127, 126)])
    return np.where(c >= 128, -v, v) * 2.0 ** np.asarray(e, np.float64)


def append(codes, exps, P, x, block):
    """One request's rows of one head in a row of positions: codes [T][hd], exps [T / block] are changed in place by the
    rows x [n][hd] (float64) that are appended at position P."""
    x = np.clip(np.where(np.isnan(x), 0.0, x), -TOP, TOP)
    n = len(x)
    for j in range(P // block, (P + n - 1) // block + 1 if n else P // block):
        lo, hi = max(P, j * block), min(P + n, (j + 1) * block)
        e = needed(np.abs(x[lo - P:hi - P]).max())
        if lo > j * block:
            held = int(exps[j])
            e = max(e, held)
            codes[j * block:lo] = encode(decode(codes[j * block:lo], held), e)
        codes[lo:hi] = encode(x[lo - P:hi - P], e)
        exps[j] = e
