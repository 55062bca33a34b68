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


def doubt(h, err, s):
    """Slack of each value of the E4M3 codes of h with scales s (both binary64,
    s spread over h): a step of E4M3 where h, known to +- err, lies next to a
    rounding border, else nothing.  err covers the scale's error too."""
    t, d = np.abs(h) / s, err / s
    e = np.floor(np.log2(np.maximum(t + d, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    to_border = np.abs(t / step - np.floor(t / step) - 0.5) * step
    # below the binade's lower end the steps are half as long: borders lie at its quarters too
    half = step / 2
    to_border = np.minimum(to_border, np.abs(t / half - np.floor(t / half) - 0.5) * half +
                           np.where(t - d < 2.0 ** e, 0.0, np.inf))
    return np.where(to_border <= d, step * s, 0.0)


def route(logits, k, sigmoid=False, renorm=True, factor=1.0):
    """(ids, weights) of logits [T, E], binary64."""
    v = logits.astype(np.float64)
    ids = np.full((v.shape[0], k), -1, np.int32)
    w = np.zeros((v.shape[0], k))
    for t in range(v.shape[0]):
        can = [e for e in range(v.shape[1]) if v[t, e] > -np.inf]
        if not can:
            continue
        order = sorted(can, key=lambda e: (-v[t, e], e))[:k]
        p = 1 / (1 + np.exp(-v[t])) if sigmoid else np.exp(v[t] - v[t][can].max())
        p = p if sigmoid else p / p[can].sum()
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[order]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() else 0.0
    return ids, w * factor


def moe(x, w13, s13, w2, s2, ids, weights, exact_hidden=False):
    """(y, bound of a binary32 evaluation before its last rounding) of the
    mixture-of-experts layer, binary64.  exact_hidden: the hidden values are
    the same in binary32 whatever the order of their sums."""
    T, H = x.shape
    E, F = w2.shape[0], w2.shape[2]
    xq, sx = encode(x, 1)
    y, off = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        ts = [t for t in range(T) if (ids[t] == e).any()]
        if not ts:
            continue
        wt = np.array([weights[t][ids[t] == e].astype(np.float64).sum() for t in ts])
        g, gm = linear(xq[ts], sx[ts], w13[e, :F], s13[e, 0])
        u, um = linear(xq[ts], sx[ts], w13[e, F:], s13[e, 1])
        with np.errstate(over="ignore"):
            h = silu(g, u)
        h32 = h.astype(np.float32)
        hq, sh = encode(h32, 1)
        o, om = linear(hq, sh, w2[e], s2[e])
        slack = 0.0
        if not exact_hidden:
            ge, ue = linear_bound(0, gm, H, "f32"), linear_bound(0, um, H, "f32")
            # |silu'| <= 1.1; the gate itself takes an exponential, a sum, a quotient and a product
            he = (1.1 * ge * (np.abs(u) + ue) + np.abs(silu(g, 1.0)) * ue) + 2.0 ** -20 * np.abs(h)
            s = widen(sh, *h.shape, 1)
            # the scale moves with the largest value of its group: at most by the group's largest relative error
            top = np.maximum.reduceat(he, np.arange(0, F, 128), axis=1)
            rel = np.repeat(top, 128, 1)[:, :F] / (448 * s)
            slack = (doubt(h, he + np.abs(h) * rel, s) + np.abs(E4[hq]) * s * rel) @ np.abs(values(w2[e], s2[e], 128)).T
        y[ts] += wt[:, None] * o
        off[ts] += np.abs(wt)[:, None] * (linear_bound(0, om, F, "f32") + slack + 4 * 2.0 ** -24 * om)
    return y, off + (E + 8) * 2.0 ** -24 * np.abs(y) + (E + 8) * 2.0 ** -24 * off
