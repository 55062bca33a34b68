"""The ends of the block-scaled operators' ranges on the GPU: infinities and
signed zeros in the gate, far logits, scales whose product leaves binary32,
strides and overlapping calls."""
import numpy as np
import pytest
import torch

import oracle

pg = pytest.importorskip("precision_gemm_fp8_b200")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _np(t):
    return t.cpu().numpy()


def _done():
    torch.cuda.synchronize()
    assert pg.device_status() == pg.OK


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_gate_of_infinities_nans_and_zeros(dt):
    """Every pair of special gate and up values in a group of ordinary ones
    (all silu(2) * 3), against the formula in binary32: an infinite value gives
    the infinite scale and zero codes beside it, a NaN its own code only, a zero
    keeps its sign.  No value but the special one and 448 or 0 occurs, so codes
    are equal; scales to 2^-20 (as the gate's other test)."""
    big = float(torch.finfo(DT[dt]).max)
    tiny = float(torch.finfo(DT[dt]).tiny)
    gates = [np.inf, -np.inf, np.nan, 0.0, -0.0, big, -big, tiny, -tiny, 1.0]
    ups = [1.0, -2.0, 0.0, -0.0, np.inf, -np.inf, np.nan, big, -big]
    pairs = [(g, u) for g in gates for u in ups]
    gu = np.empty((len(pairs), 256), np.float32)
    gu[:, :128], gu[:, 128:] = 2.0, 3.0
    for i, (g, u) in enumerate(pairs):
        gu[i, i % 128], gu[i, 128 + i % 128] = g, u
    q, s = (_np(t) for t in pg.fp8_silu_mul_quantize_blocks(_to(gu).to(DT[dt])))
    _done()
    with np.errstate(all="ignore"):
        g, u = gu[:, :128], gu[:, 128:]
        h = g / (np.float32(1) + np.exp(-g)) * u
        assert h.dtype == np.float32
        rs = np.nanmax(np.abs(h), axis=1) / np.float32(448)
        rq = oracle.e4m3_encode_array((h / rs[:, None]).astype(np.float32))
    for i, pair in enumerate(pairs):
        assert np.isinf(s[i, 0]) == np.isinf(rs[i]), pair
        assert np.isinf(rs[i]) or abs(float(s[i, 0]) / float(rs[i]) - 1) <= 2.0 ** -20, pair
        nan = (rq[i] & 0x7F) == 0x7F
        assert np.array_equal((q[i] & 0x7F) == 0x7F, nan), pair
        assert np.array_equal(q[i][~nan], rq[i][~nan]), pair


def _sigmoid_shares(logits, k, renorm):
    """(ids, weights) in binary64 by logarithms: nothing overflows or vanishes."""
    v = logits.astype(np.float64)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = -np.logaddexp(0.0, -np.take_along_axis(v, ids, 1))     # log sigmoid
    if renorm:
        top = w.max(1, keepdims=True)
        w = (w - top) - np.log(np.exp(w - top).sum(1, keepdims=True))   # a top of -3e38 would swallow the logarithm
    return ids, np.exp(w)


@pytest.mark.parametrize("renorm", [True, False])
def test_moe_sigmoid_routing_of_far_logits(renorm):
    """Sigmoids far below binary32's smallest value still have shares: logits
    from -60 to the type's lowest, alone and beside ordinary ones.  Weights
    within the roundings of two exponentials of arguments up to 400 (half a step
    of the argument each: at most 2^-16 of the result), a sum of k terms, two
    quotients and two products, or two steps of the smallest subnormal."""
    T, E, k, H, F = 9, 8, 3, 128, 16
    g = np.random.default_rng(3)
    v = np.full((T, E), -500.0, np.float32)
    v[0, :2] = -95.0, -96.0
    v[1] = -200 - np.arange(E) * 0.75
    v[2, :3] = -87.0, -88.5, -89.25
    v[3] = np.finfo(np.float32).min
    v[4, :3] = 1.5, -70.0, -100.0
    v[5, :3] = -20.0, -95.0, -100.0
    v[6, :3] = -29.0, -31.0, -66.0
    v[7, :3] = -64.0, -64.5, -63.5
    v[8, :3] = -1e30, -1e30, -100.0
    q13 = np.zeros((E, 2 * F, H), np.uint8)
    q13[:, :F] = q13[:, F:] = oracle.e4m3_encode_array(np.array([0.25], np.float32))[0]
    w = (q13, np.ones((E, 2, 1, 1), np.float32), np.full((E, H, F), q13[0, 0, 0], np.uint8),
         np.ones((E, 1, 1), np.float32))
    x = g.integers(1, 3, (T, H)).astype(np.float32)
    x[:, 0] = 448
    y, ids, wt = pg.fp8_moe(_to(x), *(_to(t) for t in w), logits=_to(v), top_k=k, score=pg.MOE_SIGMOID,
                            renormalise=renorm, out_dtype=torch.float32)
    _done()
    rid, rw = _sigmoid_shares(v, k, renorm)
    assert np.array_equal(_np(ids), rid)
    got = _np(wt).astype(np.float64)
    assert np.all(np.abs(got - rw) <= (2.0 ** -15 + (k + 16) * 2.0 ** -24) * rw + 2.0 ** -148), (got, rw)
    if renorm:
        assert np.all(np.abs(got.sum(1) - 1) <= (k + 1) * 2.0 ** -24) and bool((y != 0).all())
