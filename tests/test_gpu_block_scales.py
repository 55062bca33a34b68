"""GPU parity of the block-scaled E4M3 quantisation, gate and linear layer
against plain binary64 forms."""
import numpy as np
import pytest
import torch

import oracle
from _blocks import E4, HALF_STEP, encode, linear, linear_bound, silu, up, values, widen
from _parity import e4m3_half_step

pg = pytest.importorskip("precision_gemm_fp8_b200")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _done():
    torch.cuda.synchronize()
    assert pg.device_status() == pg.OK


def _x(rows, cols, seed, dt):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    x = torch.where(torch.rand((rows, cols), generator=g) < 0.01, x * 30, x)
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (130, 112), (127, 1040), (257, 384)])
def test_quantize_blocks_is_exact(rows, cols, block_rows, dt):
    x = _x(rows, cols, rows * 3 + cols, dt)
    x[0, :16] = 0                       # an all-zero block where cols == 16
    x[-1, 3] = -0.0
    q, s = pg.fp8_quantize_blocks(x.to(DEV), block_rows=block_rows)
    _done()
    rq, rs = encode(x.float().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_blocks_scales_stay_local(block_rows):
    """A block's codes and scale depend on its own values only: tiny, huge,
    zero and subnormal blocks side by side."""
    x = np.ones((256, 640), np.float32) * np.linspace(-1, 1, 640, dtype=np.float32)
    x[:, 128:256] = 0
    x[:, 256:384] *= np.float32(1e30)
    x[:, 384:512] *= np.float32(1e-42)
    x[:, 512:] *= np.float32(2.0 ** -130)
    q, s = pg.fp8_quantize_blocks(_to(x), block_rows=block_rows)
    _done()
    rq, rs = encode(x, block_rows)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quantize_blocks_nan_and_infinity():
    x = np.ones((2, 256), np.float32)
    x[0, 5] = np.nan
    x[1, 130] = np.inf
    q, s = (t.cpu().numpy() for t in pg.fp8_quantize_blocks(_to(x)))
    _done()
    assert q[0, 5] & 0x7F == 0x7F and np.all(E4[q[0, 6:128]] == 448) and np.all(E4[q[0, 128:]] == 448)
    assert s[0, 0] == s[0, 1] == s[1, 0] == np.float32(1) / np.float32(448) and np.isinf(s[1, 1])
    assert q[1, 130] & 0x7F == 0x7F and np.all(q[1, 131:] == 0) and np.all(q[1, 128:130] == 0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_blocks_strides_batches_and_given_buffers(dt):
    big = _x(300, 1056, 5, dt).to(DEV)
    view = big[7:140, 16:16 + 400]                                   # strided rows
    q = torch.full((133, 400), 0xEE, dtype=torch.uint8, device=DEV)
    s = torch.full((133, 4), -1.0, device=DEV)
    out = pg.fp8_quantize_blocks(view, q=q, scales=s)
    assert out[0] is q and out[1] is s
    _done()
    rq, rs = encode(view.float().cpu().numpy(), 1)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    # a batch of strided matrices, 128 x 128 blocks; every second matrix of a stack
    stack = _x(6 * 150, 144, 6, dt).view(6, 150, 144).to(DEV)
    for t in (stack[::2], stack[:, :140, :128], stack[4:5]):
        q, s = pg.fp8_quantize_blocks(t, block_rows=128)
        _done()
        for i in range(t.shape[0]):
            rq, rs = encode(t[i].float().cpu().numpy(), 128)
            assert np.array_equal(q[i].cpu().numpy(), rq) and np.array_equal(s[i].cpu().numpy(), rs)
    # row groups of a batch
    q, s = pg.fp8_quantize_blocks(stack)
    _done()
    for i in range(6):
        rq, rs = encode(stack[i].float().cpu().numpy(), 1)
        assert np.array_equal(q[i].cpu().numpy(), rq) and np.array_equal(s[i].cpu().numpy(), rs)


def test_quantize_blocks_no_rows():
    q, s = pg.fp8_quantize_blocks(torch.empty((0, 256), device=DEV))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s = pg.fp8_quantize_blocks(torch.empty((0, 32, 256), device=DEV), block_rows=128)
    assert q.shape == (0, 32, 256) and s.shape == (0, 1, 2)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,inter", [(1, 16), (1, 128), (5, 144), (130, 1040)])
def test_silu_mul_quantize_blocks(rows, inter, dt):
    """Scales agree with fl32(amax / 448) of the binary64 values to 2^-20
    (expf, one division and one product: a few units of 2^-24 each); each code
    is a nearest E4M3 value of the value over that scale, within the same error."""
    gu = (_x(rows, 2 * inter, rows + inter, dt).float() * 2).clamp(-200, 200).to(DT[dt])
    gu[0, :8] = -100.0                  # the gate's flat side
    q, s = pg.fp8_silu_mul_quantize_blocks(gu.to(DEV))
    _done()
    g64 = gu.double().numpy()
    with np.errstate(over="ignore"):
        h = silu(g64[:, :inter], g64[:, inter:])
    _, rs = encode(h.astype(np.float32), 1)
    s, q = s.cpu().numpy(), q.cpu().numpy()
    assert np.abs(s / rs - 1).max() <= 2.0 ** -20
    t = h / widen(s, rows, inter, 1)
    err = np.abs(E4[q] - t)
    assert np.all(err <= e4m3_half_step(t) + 2.0 ** -20 * np.abs(t) + 2.0 ** -149)
    assert (oracle.e4m3_encode_array(t.astype(np.float32)) == q).mean() > 0.999


# ------------------------------------------------------------------- linear
def _weights(n, k, seed):
    g = np.random.default_rng(seed)
    return encode(g.standard_normal((n, k)).astype(np.float32) * 0.02, 128)


SHAPES = [(1, 128, 128), (1, 16, 16), (2, 144, 1040), (16, 512, 512), (17, 272, 2064), (33, 256, 4096),
          (64, 1040, 144), (65, 128, 640), (128, 400, 1152), (129, 272, 528), (200, 656, 272), (300, 528, 1040),
          (513, 1296, 400)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_block_linear_within_its_roundings(m, n, k, out):
    aq, sa = encode(_x(m, k, m + n, "f32").numpy(), 1)
    wq, sw = _weights(n, k, n + k)
    y = pg.fp8_block_linear(_to(aq), _to(sa), _to(wq), _to(sw), out_dtype=DT[out])
    _done()
    ref, mag = linear(aq, sa, wq, sw)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= linear_bound(ref, mag, k, out)), (err / linear_bound(ref, mag, k, out)).max()


def _exact_case(m, n, k, seed):
    """Codes of -2..2 and scales that are powers of two: every sum is a whole
    number of 2^-8 below 2^24 of them, exact in binary32 in any order."""
    g = np.random.default_rng(seed)
    codes = oracle.e4m3_encode_array(np.arange(-2, 3).astype(np.float32))
    aq, wq = codes[g.integers(0, 5, (m, k))], codes[g.integers(0, 5, (n, k))]
    sa = 2.0 ** g.integers(-4, 2, (m, up(k)))
    sw = 2.0 ** g.integers(-4, 2, (up(n), up(k)))
    assert k * 4 * 4 * 2 ** 8 <= 2 ** 24
    return aq, sa.astype(np.float32), wq, sw.astype(np.float32)


@pytest.mark.parametrize("m,n,k", SHAPES + [(96, 4096, 256), (8, 22016, 384), (1, 4096, 4000), (700, 1168, 4000)])
def test_block_linear_exact_sums(m, n, k):
    """Whole-number data: any misplaced scale, block, row or column shows as a
    wrong value, with no tolerance at all."""
    aq, sa, wq, sw = _exact_case(m, n, k, m * 7 + n)
    y = pg.fp8_block_linear(_to(aq), _to(sa), _to(wq), _to(sw), out_dtype=torch.float32)
    _done()
    assert np.array_equal(y.cpu().numpy(), linear(aq, sa, wq, sw)[0].astype(np.float32))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [1, 40, 150, 300])
def test_block_linear_dynamic_is_quantise_then_linear(m, dt, out):
    k, n = 784, 400
    x = _x(m, k + 16, m, dt).to(DEV)[:, :k]              # strided rows
    wq, sw = (_to(t) for t in _weights(n, k, 3))
    y = pg.fp8_block_linear_dynamic(x, wq, sw, out_dtype=DT[out])
    aq, sa = pg.fp8_quantize_blocks(x)
    z = pg.fp8_block_linear(aq, sa, wq, sw, out_dtype=DT[out])
    _done()
    assert torch.equal(y, z)
    ref, mag = linear(aq.cpu().numpy(), sa.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy())
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= linear_bound(ref, mag, k, out))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,k", [(16, 16), (144, 128), (272, 4112), (4096, 1040), (12304, 2064), (512, 12304),
                                 (22016, 2832)])
def test_block_linear_dynamic_few_tokens(m, n, k, dt):
    """One launch (up to 4 tokens, where a CTA's share of K fits it) or two:
    bit for bit the quantisation followed by the layer, also with rows that
    hold NaN, infinities, zeros or the smallest values, and the rows around
    the output untouched."""
    x = _x(m, k + 16, m + n, dt)[:, :k]
    if m > 2:
        x[1] = 0
        x[2, k // 2] = float("nan")
    if m > 3:
        x[3, :16] = float("inf")
    if m > 1:
        x[0, -16:] = torch.finfo(DT[dt]).tiny
    x = x.to(DEV)
    g = torch.Generator(device=DEV).manual_seed(k)
    wq = torch.randint(0, 0x7E, (n, k), generator=g, dtype=torch.uint8, device=DEV) | \
        (torch.randint(0, 2, (n, k), generator=g, dtype=torch.uint8, device=DEV) << 7)
    sw = torch.rand((up(n), up(k)), generator=g, device=DEV)
    buf = torch.full((m + 4, n), 3.0, device=DEV)
    y = pg.fp8_block_linear_dynamic(x, wq, sw, y=buf[2:2 + m])
    chained = pg.fp8_block_linear_dynamic(x, wq, sw, out_dtype=torch.float32, flags=pg.FLAG_OVERLAP_PREVIOUS)
    z = pg.fp8_block_linear(*pg.fp8_quantize_blocks(x), wq, sw, out_dtype=torch.float32)
    _done()
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))  # noqa: E731
    ok = [i for i in range(m) if i not in (2, 3) or m <= 2]      # the bits of a NaN are not defined
    assert same(y[ok], z[ok]) and same(chained[ok], z[ok])
    assert torch.equal(torch.isnan(y), torch.isnan(z)) and bool((buf[:2] == 3).all()) and bool((buf[2 + m:] == 3).all())


@pytest.mark.parametrize("m", [3, 64, 100, 260])
def test_block_linear_writes_its_rows_only(m):
    n, k = 272, 400
    aq, sa, wq, sw = _exact_case(m, n, k, m)
    buf = torch.full((m + 40, n), 7.0, device=DEV)
    y = buf[8:8 + m]
    pg.fp8_block_linear(_to(aq), _to(sa), _to(wq), _to(sw), y=y)
    _done()
    assert np.array_equal(y.cpu().numpy(), linear(aq, sa, wq, sw)[0].astype(np.float32))
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + m:] == 7).all())


@pytest.mark.parametrize("m", [5, 90, 300])
def test_block_linear_non_finite_rows_stay_apart(m):
    """A token with a NaN code, an infinite scale or a weight block with a zero
    scale touches its own outputs only."""
    n, k = 272, 656
    aq, sa, wq, sw = _exact_case(m, n, k, 11)
    want = linear(aq, sa, wq, sw)[0]
    aq2, sa2 = aq.copy(), sa.copy()
    aq2[1, 300] = 0x7F
    sa2[3, 2] = np.inf
    y = pg.fp8_block_linear(_to(aq2), _to(sa2), _to(wq), _to(sw), out_dtype=torch.float32).cpu().numpy()
    _done()
    keep = [i for i in range(m) if i not in (1, 3)]
    assert np.array_equal(y[keep], want[keep].astype(np.float32))
    assert np.all(np.isnan(y[1])) and not np.any(np.isfinite(y[3]))


def test_block_linear_no_tokens():
    wq, sw = (_to(t) for t in _weights(128, 256, 1))
    y = pg.fp8_block_linear(torch.empty((0, 256), dtype=torch.uint8, device=DEV), torch.empty((0, 2), device=DEV),
                            wq, sw)
    assert y.shape == (0, 128) and y.dtype == torch.bfloat16
    assert pg.fp8_block_linear_dynamic(torch.empty((0, 256), device=DEV), wq, sw).shape == (0, 128)


@pytest.mark.parametrize("m", [1, 48, 128, 384])
def test_block_linear_runs_the_same_twice_and_on_two_streams(m):
    n, k = 1040, 2064
    x = _x(m, k, 4, "bf16").to(DEV)
    wq, sw = (_to(t) for t in _weights(n, k, 2))
    y0 = pg.fp8_block_linear_dynamic(x, wq, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[pg.fp8_block_linear_dynamic(x, wq, sw, out_dtype=torch.float32, stream=s) for s in streams]
           for _ in range(4)]
    _done()
    assert all(torch.equal(y0, y) for row in got for y in row)


@pytest.mark.parametrize("m", [1, 64, 300])
def test_block_linear_captured_graphs_share_nothing(m):
    """Two captured calls replayed at once on two streams, with new inputs
    copied in: each gives what the eager call gives."""
    n, k = 528, 1168
    wq, sw = (_to(t) for t in _weights(n, k, 8))
    xs = [_x(m, k, s, "bf16").to(DEV) for s in range(4)]
    want = [pg.fp8_block_linear_dynamic(x, wq, sw) for x in xs]
    slots, graphs, outs = [xs[0].clone(), xs[1].clone()], [], []
    torch.cuda.synchronize()
    for x in slots:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pg.fp8_block_linear_dynamic(x, wq, sw))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for pair in ((0, 1), (2, 3)):
        for x, i in zip(slots, pair):
            x.copy_(xs[i])
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        _done()
        for y, i in zip(outs, pair):
            assert torch.equal(y, want[i])


def test_mlp_chain_with_block_scales():
    """quantise -> gate+up -> gate+quantise -> down as a decoder's MLP runs
    them, each launch overlapping the one before, against the binary64 chain
    over the same codes: gate+up within the layer's bound, the down product
    exact to its bound over the codes that the gate kernel wrote."""
    m, h, f = 24, 1040, 656
    x = _x(m, h, 21, "bf16").to(DEV)
    w13 = (torch.randn((2 * f, h), generator=torch.Generator().manual_seed(1)) * 0.05).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn((h, f), generator=torch.Generator().manual_seed(2)) * 0.05).to(torch.bfloat16).to(DEV)
    (q13, s13), (q2, s2) = (pg.fp8_quantize_blocks(w, block_rows=128) for w in (w13, w2))
    aq, sa = pg.fp8_quantize_blocks(x)
    gu = pg.fp8_block_linear(aq, sa, q13, s13, out_dtype=torch.float32, flags=pg.FLAG_OVERLAP_PREVIOUS)
    hq, sh = pg.fp8_silu_mul_quantize_blocks(gu, flags=pg.FLAG_OVERLAP_PREVIOUS)
    y = pg.fp8_block_linear(hq, sh, q2, s2, flags=pg.FLAG_OVERLAP_PREVIOUS)
    _done()
    c = lambda t: t.cpu().numpy()  # noqa: E731
    ref, mag = linear(c(aq), c(sa), c(q13), c(s13))
    assert np.all(np.abs(c(gu) - ref) <= linear_bound(ref, mag, h, "f32"))
    hv = silu(c(gu).astype(np.float64)[:, :f], c(gu).astype(np.float64)[:, f:])
    got = values(c(hq), c(sh), 1)
    step = widen(c(sh), m, f, 1)
    assert np.all(np.abs(got - hv) <= (e4m3_half_step(hv / step) * (1 + 2.0 ** -15) + 2.0 ** -12) * step)
    ref, mag = linear(c(hq), c(sh), c(q2), c(s2))
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= linear_bound(ref, mag, f, "bf16"))
    full = silu(*np.split(x.double().cpu().numpy() @ w13.double().cpu().numpy().T, 2, 1)) @ w2.double().cpu().numpy().T
    # three E4M3 roundings on the way (x, the weights, h), each at most 2^-4 relative a value and independent:
    # sqrt(4) of them in the root mean square (x, w13, h, w2), far below this
    assert np.linalg.norm(y.double().cpu().numpy() - full) < 4 * 2.0 ** -4 * np.linalg.norm(full)
    assert HALF_STEP["bf16"] == torch.finfo(torch.bfloat16).eps / 2
