"""The ends of the block-scaled operators' ranges on the GPU: infinities and
signed zeros in the gate, far logits, scales whose product leaves binary32,
strides and overlapping calls."""
import numpy as np
import pytest
import torch

import oracle
from _blocks import encode, linear, linear_bound, moe, up

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


def _far_scales(m, n, k, seed):
    """Tokens and weight blocks of three kinds: ordinary, large (scales 2^70 and
    2^56 times 1 to 2, small codes, some tokens' all zero) and small (2^-70 and
    2^-56, codes up to 448).  Where two of a kind meet, the scales' products reach the
    ends of binary32's normal range, and results are normal numbers or exact zeros."""
    g = np.random.default_rng(seed)
    codes = lambda top, shape: oracle.e4m3_encode_array(  # noqa: E731
        (g.choice([-1.0, 1.0, 1.0, 1.0], shape) * top * g.choice([0.5, 0.75, 1.0], shape)).astype(np.float32))
    aq, wq = codes(1.0, (m, k)), codes(1.0, (n, k))
    # up to 1.41: 2^127 times two of them stays below 2^128
    sa, sw = (1 + 0.41 * g.random((m, up(k)))).astype(np.float32), (1 + 0.41 * g.random((up(n), up(k)))).astype(np.float32)
    for i in range(m):
        if i % 4 == 0:
            aq[i], sa[i] = codes(448.0, k), np.ldexp(sa[i], -70)
        elif i % 4 in (1, 2):
            aq[i], sa[i] = codes(2.0 ** -7, k) * (i % 4 == 1), np.ldexp(sa[i], 70)
    for j in range(up(n)):
        at = np.s_[j * 128:(j + 1) * 128]
        if j % 3 == 1:
            wq[at], sw[j] = codes(448.0, wq[at].shape), np.ldexp(sw[j], -56)
        elif j % 3 == 2:
            wq[at], sw[j] = codes(2.0 ** -7, wq[at].shape), np.ldexp(sw[j], 57)
    return aq, sa, wq, sw


@pytest.mark.parametrize("m,n,k", [(1, 400, 1040), (3, 272, 400), (7, 528, 2064), (20, 400, 784), (60, 656, 1040),
                                   (90, 4096, 656), (100, 400, 1168), (300, 528, 1040), (520, 1296, 400),
                                   (700, 4096, 656)])
def test_block_linear_scales_at_the_ends_of_the_range(m, n, k):
    """A step of the smallest subnormal for each addition beside the linear bound."""
    c = _far_scales(m, n, k, m + n)
    factors = c[1].astype(np.float64)[:, None] * c[3].astype(np.float64)
    assert (m == 1 or 2.0 ** 127 <= factors.max()) and factors.max() < 2.0 ** 128 and 2.0 ** -126 <= factors.min() < 2.0 ** -124
    y = pg.fp8_block_linear(*(_to(t) for t in c), out_dtype=torch.float32)
    _done()
    ref, mag = linear(*c)
    assert mag.max() < 2.0 ** 127
    err = np.abs(_np(y).astype(np.float64) - ref)
    bound = linear_bound(ref, mag, k, "f32") + (up(k) + 10) * 2.0 ** -149
    assert np.all(err <= bound), (err / bound).max()


def test_block_linear_zero_and_infinite_scales_keep_their_meaning():
    """A zero scale gives zeros beside any finite one, an infinite scale no
    finite value, whatever the size of the other."""
    m, n, k = 6, 256, 384
    g = np.random.default_rng(0)
    aq = oracle.e4m3_encode_array(g.integers(1, 3, (m, k)).astype(np.float32))
    wq = oracle.e4m3_encode_array(g.integers(1, 3, (n, k)).astype(np.float32))
    sa, sw = np.zeros((m, 3), np.float32), np.full((2, 3), 2.0 ** 100, np.float32)
    sa[1] = 2.0 ** -60
    sa[2, 1] = np.inf
    sa[3, 2] = np.nan
    y = _np(pg.fp8_block_linear(_to(aq), _to(sa), _to(wq), _to(sw), out_dtype=torch.float32))
    _done()
    assert not y[[0, 4, 5]].any() and np.isfinite(y[1]).all() and not np.isfinite(y[2]).any() and np.isnan(y[3]).all()


@pytest.mark.parametrize("T", [1, 20, 40])
def test_moe_down_scales_at_the_ends_of_the_range(T):
    """The product of the hidden scale, W2's and the routing weight, with hidden
    codes that do not depend on the order of sums (gates of 28 and more, where
    silu(g) = g), near either end of binary32's range."""
    E, k, H, F = 3, 3, 144, 272
    g = np.random.default_rng(T)
    val = lambda v: int(oracle.e4m3_encode_array(np.array([v], np.float32))[0])  # noqa: E731
    small = oracle.e4m3_encode_array(np.arange(1, 4).astype(np.float32))
    x = g.integers(-2, 3, (T, H)).astype(np.float32)
    x[:, ::128] = 448
    w13 = np.zeros((E, 2 * F, H), np.uint8)
    w13[:, :F, ::128] = val(1 / 16)
    w13[:, F:] = small[g.integers(0, 3, (E, F, H))]
    w2 = small[g.integers(0, 3, (E, H, F))]
    s2 = (1 + g.random((E, up(H), up(F)))).astype(np.float32)
    s2[0], s2[1], s2[2] = np.ldexp(s2[0], -100), np.ldexp(s2[1], 100), np.ldexp(s2[2], -60)
    wt = np.ldexp(1 + g.random((T, k)), [[-20, -120, 8]]).astype(np.float32)
    ids = np.tile(np.arange(3, dtype=np.int32), (T, 1))
    w = (w13, np.ones((E, 2, up(F), up(H)), np.float32), w2, s2)
    for keep in range(3):
        one = np.where(np.arange(3) == keep, ids, -1).astype(np.int32)
        y, _, _ = pg.fp8_moe(_to(x), *(_to(t) for t in w), ids=_to(one), weights=_to(wt), out_dtype=torch.float32)
        _done()
        ref, off = moe(x, *w, one, wt, exact_hidden=True)
        y = _np(y).astype(np.float64)
        bound = off + 2.0 ** -24 * np.abs(ref) + 2.0 ** -149 * (up(F) + 10)
        assert np.all(np.abs(y - ref) <= bound), (keep, (np.abs(y - ref) / bound).max())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 4, 5, 40, 300])
def test_block_linear_dynamic_in_place(m, dt):
    """y may be x, or lie over part of it: x is quantised before a row of y is written."""
    k = n = 1040
    g = torch.Generator(device=DEV).manual_seed(m)
    wq, sw = pg.fp8_quantize_blocks(torch.randn((n, k), generator=g, device=DEV) * 0.02, block_rows=128)
    x = torch.randn((m + 1, k), generator=g, device=DEV).to(DT[dt])
    for at in (0, 1):                      # the same rows; the second overlaps by all but one
        z = x.clone()
        want = pg.fp8_block_linear_dynamic(z[:m], wq, sw, out_dtype=DT[dt])
        y = pg.fp8_block_linear_dynamic(z[:m], wq, sw, y=z[at:at + m])
        _done()
        assert torch.equal(y, want) and (at == 0 or torch.equal(z[0], x[0]))


def _odd_row(width, dt):
    """One row of `width` values whose stride is no multiple of 16 bytes (and of no meaning: there is one row)."""
    big = torch.randn((3, width + 1), generator=torch.Generator().manual_seed(width)).to(DT[dt]).to(DEV)
    view = torch.empty(width + 64, dtype=DT[dt], device=DEV)[:width].view(1, width)
    view.copy_(big[1:2, :width])
    return view.as_strided((1, width), (width + 3, 1))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_row_may_carry_any_stride(dt):
    x = _odd_row(512, dt)
    plain = x.clone(memory_format=torch.contiguous_format).as_strided((1, 512), (512, 1))
    same = lambda a, b: all(torch.equal(s, t) for s, t in zip(a, b))  # noqa: E731
    assert x.stride(0) == 515
    for rows in (1, 128):
        assert same(pg.fp8_quantize_blocks(x, block_rows=rows), pg.fp8_quantize_blocks(plain, block_rows=rows))
        x3 = x.as_strided((1, 1, 512), (1031, 515, 1))
        assert same(pg.fp8_quantize_blocks(x3, block_rows=rows), pg.fp8_quantize_blocks(plain[None], block_rows=rows))
    assert same(pg.fp8_silu_mul_quantize_blocks(x), pg.fp8_silu_mul_quantize_blocks(plain))
    wq, sw = pg.fp8_quantize_blocks(torch.randn((144, 512), device=DEV), block_rows=128)
    assert torch.equal(pg.fp8_block_linear_dynamic(x, wq, sw), pg.fp8_block_linear_dynamic(plain, wq, sw))
    w13, s13 = pg.fp8_quantize_blocks(torch.randn((4, 128, 512), device=DEV), block_rows=128)
    w2, s2 = pg.fp8_quantize_blocks(torch.randn((2, 512, 128), device=DEV), block_rows=128)
    w = (w13.view(2, 256, 512), s13.view(2, 2, 1, 4), w2, s2)
    lg = torch.randn((1, 2), device=DEV)
    assert same(pg.fp8_moe(x, *w, logits=lg, top_k=1), pg.fp8_moe(plain, *w, logits=lg, top_k=1))
    _done()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_quantize_row_groups_of_strided_batches(dt):
    """1 x 128 groups of matrices that do not follow one another: every second
    one, their first rows, the same one again, one row each; in given buffers."""
    stack = torch.randn((6, 150, 144), generator=torch.Generator().manual_seed(1)).to(DT[dt]).to(DEV)
    for x in (stack[::2], stack[:, :140], stack[1:5, 3:4], stack[::3, 5:6, :128], stack[2:3].expand(3, 150, 144),
              stack[:, :, 16:], stack[:0, :140]):
        q, s = pg.fp8_quantize_blocks(x)
        rq, rs = pg.fp8_quantize_blocks(x.contiguous())
        q2 = torch.full((x.shape[0] + 2, *x.shape[1:]), 0xEE, dtype=torch.uint8, device=DEV)
        s2 = torch.full((x.shape[0] + 2, x.shape[1], up(x.shape[2])), -1.0, device=DEV)
        pg.fp8_quantize_blocks(x, q=q2[1:-1], scales=s2[1:-1], flags=pg.FLAG_OVERLAP_PREVIOUS)
        _done()
        assert torch.equal(q, rq) and torch.equal(s, rs) and torch.equal(q2[1:-1], rq) and torch.equal(s2[1:-1], rs)
        for edge in (q2[0], q2[-1]):
            assert bool((edge == 0xEE).all())
        assert bool((s2[0] == -1).all()) and bool((s2[-1] == -1).all())
        for i in range(x.shape[0]):
            eq, es = encode(_np(x[i].float()), 1)
            assert np.array_equal(_np(q[i]), eq) and np.array_equal(_np(s[i]), es)


def test_quantize_row_groups_refuses_a_misaligned_batch_before_any_launch():
    x = torch.zeros(600, device=DEV).as_strided((2, 2, 128), (258, 128, 1))     # the second matrix at 1032 bytes
    q = torch.full((2, 2, 128), 7, dtype=torch.uint8, device=DEV)
    with pytest.raises(pg.Pgf8Error):
        pg.fp8_quantize_blocks(x, q=q)
    _done()
    assert bool((q == 7).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_quantize_tiles_nan_and_infinity(dt):
    """128 x 128 blocks with NaNs, infinities and the ends of the range, whole
    and ragged: NaN is ignored by the scale and keeps its code, an infinity
    gives the infinite scale, zeros with their sign beside it."""
    x = torch.randn((300, 400), generator=torch.Generator().manual_seed(4)).to(DT[dt])
    x[5, 7] = float("nan")
    x[130, 140] = float("inf")
    x[131, 141] = float("nan")
    x[140:150, 130] = -float("inf")
    x[290, 260] = float("nan")
    x[299, 399] = -float("inf")
    x[:128, 384:] = float("nan")                      # nothing but NaN: the scale of zeros
    x[256:, :128] = torch.finfo(DT[dt]).max
    q, s = (_np(t) for t in pg.fp8_quantize_blocks(x.to(DEV), block_rows=128))
    _done()
    v = x.float().numpy()
    for i in range(3):
        for j in range(4):
            at = np.s_[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            b = v[at]
            a = np.float32(np.abs(b[~np.isnan(b)]).max(initial=0.0))
            want = a / np.float32(448) if a else np.float32(1)
            assert s[i, j] == want, (i, j)
            with np.errstate(all="ignore"):
                r = oracle.e4m3_encode_array((b / want).astype(np.float32))
            nan = np.isnan(b / want) if np.isfinite(want) else np.isnan(b) | np.isinf(b)
            assert np.array_equal((q[at] & 0x7F) == 0x7F, nan), (i, j)
            assert np.array_equal(q[at][~nan], r[~nan]), (i, j)


@pytest.mark.parametrize("T", [1, 4, 20, 64])
def test_moe_overlapping_the_kernels_around_it(T):
    """Layers one after another, each launch overlapping the one before: the
    router's input of a layer is the output of the last, the workspace, ids and
    weights the same buffers, equal to the calls one by one."""
    E, k, H, F, layers = 12, 3, 528, 272, 3
    g = torch.Generator(device=DEV).manual_seed(T)
    w = []
    for _ in range(layers):
        w13, s13 = pg.fp8_quantize_blocks(torch.randn((2 * E, F, H), generator=g, device=DEV) * 0.06, block_rows=128)
        w2, s2 = pg.fp8_quantize_blocks(torch.randn((E, H, F), generator=g, device=DEV) * 0.06, block_rows=128)
        wo, so = pg.fp8_quantize_blocks(torch.randn((H, H), generator=g, device=DEV) * 0.06, block_rows=128)
        w.append((w13.view(E, 2 * F, H), s13.view(E, 2, up(F), up(H)), w2, s2, wo, so))
    x0 = torch.randn((T, H), generator=g, device=DEV)
    logits = torch.randn((layers, T, E), generator=g, device=DEV)

    def step(flags, ws, wl, ids, wt, a, b):
        a.copy_(x0)
        for lay, (w13, s13, w2, s2, wo, so) in enumerate(w):
            pg.fp8_block_linear_dynamic(a, wo, so, y=b, workspace=wl, flags=flags)
            pg.fp8_moe(b, w13, s13, w2, s2, logits=logits[lay], top_k=k, y=a, ids=ids, weights=wt, workspace=ws,
                       flags=flags)
        return a.clone()

    def buffers():
        return (torch.empty(pg.fp8_moe_workspace_size(T, H, F, E, k), dtype=torch.uint8, device=DEV),
                torch.empty(pg.fp8_block_linear_dynamic_workspace_size(T, H), dtype=torch.uint8, device=DEV),
                torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV),
                torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV))
    want = step(0, *buffers())
    b = buffers()
    got = [step(pg.FLAG_OVERLAP_PREVIOUS, *b) for _ in range(5)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(pg.FLAG_OVERLAP_PREVIOUS, *b)
    for _ in range(3):
        graph.replay()
    _done()
    assert bool(torch.isfinite(want).all()) and bool((want != 0).any())
    assert all(torch.equal(t, want) for t in got) and torch.equal(out, want)


@pytest.mark.parametrize("T,E,k", [(1, 1, 2), (5, 2, 8), (40, 3, 16), (64, 15, 16)])
def test_moe_ranks_of_fewer_experts_than_choices(T, E, k):
    """Experts dealt over ranks: each call is given the same k choices a token,
    relative to its own E experts, and the ranks' sums are the layer's."""
    H, F, ranks = 272, 144, 3
    g = np.random.default_rng(T)
    q13, s13 = zip(*[encode(g.standard_normal((F, H)).astype(np.float32) * 0.05, 128) for _ in range(2 * E * ranks)])
    q2, s2 = zip(*[encode(g.standard_normal((H, F)).astype(np.float32) * 0.05, 128) for _ in range(E * ranks)])
    w = (np.stack(q13).reshape(E * ranks, 2 * F, H), np.stack(s13).reshape(E * ranks, 2, up(F), up(H)), np.stack(q2),
         np.stack(s2))
    x = g.standard_normal((T, H)).astype(np.float32)
    ids = np.stack([g.integers(0, E * ranks, k) for _ in range(T)]).astype(np.int32)      # some twice
    wt = g.random((T, k)).astype(np.float32)
    for r in range(ranks):
        mine = tuple(t[r * E:(r + 1) * E] for t in w)
        y, _, _ = pg.fp8_moe(_to(x), *(_to(t) for t in mine), ids=_to(ids - r * E), weights=_to(wt),
                             out_dtype=torch.float32)
        _done()
        ref, off = moe(x, *mine, ids - r * E, wt)
        err = np.abs(_np(y).astype(np.float64) - ref)
        assert np.all(err <= off + 2.0 ** -24 * (np.abs(ref) + off) + 2.0 ** -150)


def test_moe_more_choices_than_experts_need_given_ids():
    w13, s13 = torch.zeros((2, 256, 128), dtype=torch.uint8, device=DEV), torch.ones((2, 2, 1, 1), device=DEV)
    w2, s2 = torch.zeros((2, 128, 128), dtype=torch.uint8, device=DEV), torch.ones((2, 1, 1), device=DEV)
    with pytest.raises(pg.Pgf8Error):
        pg.fp8_moe(torch.zeros((4, 128), device=DEV), w13, s13, w2, s2, logits=torch.zeros((4, 2), device=DEV), top_k=3)
