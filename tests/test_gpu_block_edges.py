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
