"""Plain binary64 forms of the block-scaled operators for the tests (numpy;
E4M3 encoding by the oracle), and the error bounds of the kernels."""
import numpy as np

import oracle

E4 = oracle.e4m3_table()
# half a step of the output type relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# half the smallest subnormal step
HALF_TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def up(n, b=128):
    return -(-n // b)


def encode(x, block_rows):
    """(codes, scales) of x [rows, cols] f32, one scale per block_rows x 128
    block: s = fl32(amax / 448), 1 when 0; E4M3 of fl32(x / s)."""
    rows, cols = x.shape
    q = np.zeros((rows, cols), np.uint8)
    s = np.zeros((up(rows, block_rows), up(cols)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            a = np.float32(np.abs(x[at]).max())
            s[i, j] = a / np.float32(448.0)
            if s[i, j] == 0:
                s[i, j] = 1
            q[at] = oracle.e4m3_encode_array((x[at] / s[i, j]).astype(np.float32))
    return q, s


def widen(s, rows, cols, block_rows):
    """Block scales [.., ..] spread over [rows, cols], binary64."""
    s = s.astype(np.float64)
    return np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)[:, :cols]


def values(q, s, block_rows):
    return E4[q] * widen(s, *q.shape, block_rows)


def linear(aq, sa, wq, sw):
    """(y, sum of |products|) of the block-scaled layer, binary64."""
    a, w = values(aq, sa, 1), values(wq, sw, 128)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def linear_bound(ref, mag, K, out):
    """What the kernels' roundings can add up to.  Inside a block 128 products
    are exact and added by the tensor core (at most 2^-22 of the magnitudes a
    step: its adder may truncate); each block then takes one rounded scale
    product and one fused multiply-add, and at most 8 partial sums are added;
    one rounding to the output type."""
    return HALF_STEP[out] * np.abs(ref) + HALF_TINY[out] + \
        (1 + HALF_STEP[out]) * (128 * 2.0 ** -22 + (up(K) + 10) * 2.0 ** -24) * mag


def silu(g, u):
    return g / (1 + np.exp(-g)) * u
