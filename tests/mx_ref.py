"""Plain 64-bit forms of the microscaled operators, from their definitions in
dbf.h (CPU, numpy): the oracle of tests/test_gpu_mx4.py, pinned on hand-worked
values in tests/test_mx_ref_pins.py."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# E4M3: codes 0..126 (sign 0), exponent bias 7, subnormals of 2^-9; 127 is NaN
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def nearest(a, table):
    """Index of the table entry nearest to each |a| (at most the last), ties to the even index."""
    a = np.minimum(np.abs(a), table[-1])
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _blocks(x):
    rows, k = x.shape
    v = np.zeros((rows, -(-k // 32) * 32))
    v[:, :k] = x
    return v.reshape(rows, -1, 32)


def _quantize(x, table, exponent):
    """(values [rows, k], codes, scale bytes) for blocks of 32."""
    x = np.asarray(x, dtype=np.float64)
    v = _blocks(x)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(axis=2)
        good = np.isfinite(amax)
        s = np.array([[exponent(a) if g and a > 0 else -127 for a, g in zip(ra, rg)] for ra, rg in zip(amax, good)])
        byte = np.where(good, s + 127, 255)
        w = np.where(good[:, :, None], v, 0.0) * 2.0 ** -s[:, :, None].astype(np.float64)
        idx = nearest(w, table)
        codes = np.where(good[:, :, None], idx + np.where(np.signbit(w), SIGN[len(table)], 0), 0)
        val = np.where(np.signbit(w), -1.0, 1.0) * table[idx] * 2.0 ** s[:, :, None].astype(np.float64)
        val = np.where(good[:, :, None], val, np.nan)
    return val.reshape(len(x), -1)[:, : x.shape[1]], codes, byte


SIGN = {8: 8, 127: 128}


def _exp4(a):
    return int(np.clip(np.floor(np.log2(a)) - 2, -127, 127))


def _exp8(a):
    s = -127
    while a > 448.0 * 2.0 ** s:
        s += 1
    return s


def mx4(x):
    return _quantize(x, E2M1, _exp4)


def act8(x):
    return _quantize(x, E4M3, _exp8)


def pack4(codes, byte):
    """Packed codes and tiled scales of mx4's answer."""
    rows, nb = byte.shape
    flat = codes.reshape(rows, -1).astype(np.uint8)
    packed = flat[:, 0::2] | (flat[:, 1::2] << 4)
    scales = np.zeros((-(-rows // 128), -(-nb // 4), 32, 4, 4), np.uint8)
    for r in range(rows):
        for b in range(nb):
            scales[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = byte[r, b]
    return packed, scales


def gate(act, g):
    with np.errstate(all="ignore"):
        if act == "silu":
            return g / (1 + np.exp(-g))
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def gate_slope(act, g):
    with np.errstate(all="ignore"):
        if act == "silu":
            s = 1 / (1 + np.exp(-g))
            return s + g * s * (1 - s)
        c = np.sqrt(2 / np.pi)
        th = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * (1 + th) + 0.5 * g * (1 - th ** 2) * c * (1 + 3 * 0.044715 * g ** 2)
