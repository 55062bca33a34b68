"""GPU parity of the mixture-of-experts layer against a plain binary64 form.

Two kinds of data.  Realistic: the hidden values that lie next to a rounding
border of E4M3 may go either way with the order of a binary32 sum, and the
bound counts one step for each of them.  Whole-number: the gate and up sums are
whole numbers and the gate is at least 24, where silu(g) = g in binary32, so the
hidden codes are the same for any order of the sums, and the bound is that of
the down product alone."""
import numpy as np
import pytest
import torch

import oracle
from _blocks import E4, HALF_STEP, HALF_TINY, encode, moe, route, up

pg = pytest.importorskip("precision_gemm_fp8_b200")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _done():
    torch.cuda.synchronize()
    assert pg.device_status() == pg.OK


def _experts(E, H, F, seed):
    g = np.random.default_rng(seed)
    q13, s13 = zip(*[encode(g.standard_normal((F, H)).astype(np.float32) * 0.05, 128) for _ in range(2 * E)])
    q2, s2 = zip(*[encode(g.standard_normal((H, F)).astype(np.float32) * 0.05, 128) for _ in range(E)])
    return (np.stack(q13).reshape(E, 2 * F, H), np.stack(s13).reshape(E, 2, up(F), up(H)), np.stack(q2),
            np.stack(s2))


def _x(T, H, seed, dt="f32"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g)
    return torch.where(torch.rand((T, H), generator=g) < 0.01, x * 20, x).to(DT[dt])


def _ids(T, E, k, seed, away=0.0):
    """k different experts a token; some slots are another rank's (-1 or E)."""
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    gone = g.random((T, k)) < away
    ids[gone] = g.choice(np.array([-1, E, E + 7, -2 ** 31], np.int32), gone.sum())
    return ids, g.random((T, k)).astype(np.float32)


def _check(y, ref, off, out):
    y = y.double().cpu().numpy()
    bound = off + HALF_STEP[out] * (np.abs(ref) + off) + HALF_TINY[out]
    assert np.all(np.isfinite(y)) and np.all(np.abs(y - ref) <= bound), (np.abs(y - ref) / bound).max()


SHAPES = [  # T, E, k, H, F
    (1, 1, 1, 16, 16), (1, 4, 2, 128, 128), (1, 8, 3, 272, 144), (2, 3, 3, 1040, 272), (7, 16, 4, 256, 656),
    (16, 8, 2, 528, 384), (17, 5, 2, 400, 272), (32, 40, 6, 272, 128), (33, 4, 1, 144, 400), (49, 64, 8, 640, 272),
    (64, 8, 2, 1168, 528), (64, 128, 8, 272, 256)]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_moe_given_experts(T, E, k, H, F, out):
    w = _experts(E, H, F, T + E + F)
    ids, wt = _ids(T, E, k, T * 5 + k, away=0.1 if T > 1 else 0.0)
    x = _x(T, H, T + H, "bf16")
    y, _, _ = pg.fp8_moe(x.to(DEV), *(_to(t) for t in w), ids=_to(ids), weights=_to(wt), out_dtype=DT[out])
    _done()
    _check(y, *moe(x.float().numpy(), *w, ids, wt), out)


def _whole(T, E, H, F, seed):
    """x: whole numbers in -2..2 with a 448 in front of each group (its scale is
    then 1), which W1 takes times 1/16 (g = 28 a group), or -1/2 in one row in
    five (a gate far below zero: h = 0), W3 not at all; W3 and W2: -2..2."""
    g = np.random.default_rng(seed)
    x = g.integers(-2, 3, (T, H)).astype(np.float32)
    x[:, ::128] = 448
    small = oracle.e4m3_encode_array(np.arange(-2, 3).astype(np.float32))
    one = lambda v: int(oracle.e4m3_encode_array(np.array([v], np.float32))[0])  # noqa: E731
    w13 = np.zeros((E, 2 * F, H), np.uint8)
    w13[:, :F, ::128] = one(1 / 16)
    w13[:, :F:5, ::128] = one(-0.5)
    w13[:, F:] = small[g.integers(0, 5, (E, F, H))]
    w13[:, F:, ::128] = 0
    s13 = np.ones((E, 2, up(F), up(H)), np.float32)
    w2 = small[g.integers(0, 5, (E, H, F))]
    s2 = (2.0 ** g.integers(-6, -2, (E, up(H), up(F)))).astype(np.float32)
    return x, (w13, s13, w2, s2)


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_moe_whole_numbers(T, E, k, H, F):
    x, w = _whole(T, E, H, F, T * 11 + E)
    ids, wt = _ids(T, E, k, T + k, away=0.2)
    y, _, _ = pg.fp8_moe(_to(x), *(_to(t) for t in w), ids=_to(ids), weights=_to(wt), out_dtype=torch.float32)
    _done()
    _check(y, *moe(x, *w, ids, wt, exact_hidden=True), "f32")


@pytest.mark.parametrize("ldt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 33, 16), (20, 512, 8), (64, 128, 4), (64, 8, 8)])
@pytest.mark.parametrize("sigmoid,renorm,factor", [(False, True, 1.0), (False, False, 2.5), (True, True, 1.0)])
def test_moe_routing(T, E, k, ldt, sigmoid, renorm, factor):
    """ids equal; weights within the roundings of expf (2 units), a sum of E
    terms, two quotients and a product in binary32.  Coarse logits give ties."""
    H, F = 128, 16
    g = torch.Generator().manual_seed(T * 3 + E)
    logits = (torch.randn((T, E + 3), generator=g) * 3).mul(8).round().div(8).to(DT[ldt])[:, :E]   # strided
    x, w = _whole(T, E, H, F, 5)
    y, ids, wt = pg.fp8_moe(_to(x), *(_to(t) for t in w), logits=logits.to(DEV), top_k=k,
                            score=pg.MOE_SIGMOID if sigmoid else pg.MOE_SOFTMAX, renormalise=renorm, factor=factor,
                            out_dtype=torch.float32)
    _done()
    rid, rw = route(logits.float().numpy(), k, sigmoid, renorm, factor)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = wt.cpu().numpy()
    assert np.all(np.abs(got - rw) <= (E + k + 16) * 2.0 ** -24 * np.abs(rw) + 2.0 ** -126)
    _check(y, *moe(x, *w, rid, got, exact_hidden=True), "f32")


def test_moe_routing_masked_logits():
    """-inf and NaN logits are never chosen; a token with too few choices keeps
    -1 and 0 behind them, a token with none gets y = 0."""
    T, E, k, H, F = 5, 8, 3, 128, 32
    x, w = _whole(T, E, H, F, 9)
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(2))
    logits[0] = -np.inf
    logits[1, 2:] = -np.inf
    logits[2, :] = float("nan")
    logits[2, 5] = -3e38
    logits[3, 3] = float("nan")
    logits[3, 4] = torch.finfo(torch.float32).min
    logits[4, :] = torch.finfo(torch.float32).min
    y, ids, wt = pg.fp8_moe(_to(x), *(_to(t) for t in w), logits=logits.to(DEV), top_k=k, out_dtype=torch.float32)
    _done()
    ids, wt = ids.cpu().numpy(), wt.cpu().numpy()
    v = logits.numpy().copy()
    v[np.isnan(v)] = -np.inf
    rid, rw = route(v, k)
    assert np.array_equal(ids, rid) and np.abs(wt - rw).max() <= 32 * 2.0 ** -24
    assert ids[0].tolist() == [-1] * 3 and ids[1, 2] == -1 and ids[2].tolist() == [5, -1, -1] and wt[2, 0] == 1
    assert ids[4].tolist() == [0, 1, 2]
    assert not y[0].any()
    _check(y, *moe(x, *w, rid, wt, exact_hidden=True), "f32")


def test_moe_slots_that_are_left_out():
    """Ids outside the experts leave their slots out whatever weight stands
    there (NaN, infinity); a token with none of them gets y = 0, and so does a
    whole batch; an expert named twice counts with both weights."""
    T, E, k, H, F = 6, 4, 3, 272, 144
    x, w = _whole(T, E, H, F, 3)
    ids = np.array([[0, -1, 4], [-1, -1, -1], [2, 2, 1], [3, 3, 3], [1, 0, 2], [9, -5, 2]], np.int32)
    wt = np.random.default_rng(1).random((T, k)).astype(np.float32)
    wt[0, 1], wt[0, 2], wt[1] = np.nan, np.inf, np.nan
    dw = [_to(t) for t in w]
    y, _, _ = pg.fp8_moe(_to(x), *dw, ids=_to(ids), weights=_to(wt), out_dtype=torch.float32)
    _done()
    _check(y, *moe(x, *w, ids, wt, exact_hidden=True), "f32")
    assert not y[1].any()
    none = np.full((T, k), -1, np.int32)
    y, _, _ = pg.fp8_moe(_to(x), *dw, ids=_to(none), weights=_to(wt), out_dtype=torch.bfloat16)
    _done()
    assert y.shape == (T, H) and not y.any()


def test_moe_tokens_do_not_mix():
    """A token of NaNs or infinities spoils its own row only, and unread
    experts may hold anything."""
    T, E, k, H, F = 20, 6, 2, 272, 272
    x, w = _whole(T, E, H, F, 4)
    ids, wt = _ids(T, E - 1, k, 1)
    w[0][E - 1], w[1][E - 1], w[2][E - 1], w[3][E - 1] = 0x7F, np.nan, 0x7F, np.nan
    want, off = moe(x, *w, ids, wt, exact_hidden=True)
    x2 = x.copy()
    x2[3, 7] = np.nan
    x2[11] = np.inf
    y, _, _ = pg.fp8_moe(_to(x2), *(_to(t) for t in w), ids=_to(ids), weights=_to(wt), out_dtype=torch.float32)
    _done()
    keep = [t for t in range(T) if t not in (3, 11)]
    _check(y[keep], want[keep], off[keep], "f32")
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[11]).all())


@pytest.mark.parametrize("T", [1, 20, 50])
def test_moe_given_buffers_strides_and_streams(T):
    """Outputs in given buffers (rows around them untouched), strided x, the
    same result in every run and on other streams at once."""
    E, k, H, F = 16, 4, 528, 272
    w = [_to(t) for t in _experts(E, H, F, 8)]
    x = _x(T, H + 16, 5, "f16").to(DEV)[:, :H]
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(T)).to(DEV)
    buf = torch.full((T + 4, H), 5.0, device=DEV)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    wt = torch.empty((T, k), device=DEV)
    ws = torch.full((pg.fp8_moe_workspace_size(T, H, F, E, k),), 0xFF, dtype=torch.uint8, device=DEV)
    y, i2, w2 = pg.fp8_moe(x, *w, logits=logits, top_k=k, y=buf[2:2 + T], ids=ids, weights=wt, workspace=ws)
    assert i2 is ids and w2 is wt
    _done()
    assert bool((buf[:2] == 5).all()) and bool((buf[2 + T:] == 5).all())
    _check(y, *moe(x.float().cpu().numpy(), *(t.cpu().numpy() for t in w), ids.cpu().numpy(), wt.cpu().numpy()), "f32")
    again, _, _ = pg.fp8_moe(x, *w, ids=ids, weights=wt, out_dtype=torch.float32, workspace=ws)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [pg.fp8_moe(x, *w, logits=logits, top_k=k, out_dtype=torch.float32, stream=s)[0] for _ in range(3)
           for s in streams]
    _done()
    assert torch.equal(again, y) and all(torch.equal(g, y) for g in got)


@pytest.mark.parametrize("T", [1, 24])
def test_moe_captured_graphs(T):
    """Two captured calls replayed at once with inputs and routing that differ
    from the capture's."""
    E, k, H, F = 12, 3, 400, 272
    w = [_to(t) for t in _experts(E, H, F, 2)]
    xs = [_x(T, H, s, "bf16").to(DEV) for s in range(4)]
    ls = [torch.randn((T, E), generator=torch.Generator().manual_seed(s)).to(DEV) for s in range(4)]
    want = [pg.fp8_moe(x, *w, logits=lg, top_k=k) for x, lg in zip(xs, ls)]
    slots = [(xs[i].clone(), ls[i].clone()) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, lg in slots:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pg.fp8_moe(x, *w, logits=lg, top_k=k))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for pair in ((0, 1), (2, 3)):
        for (x, lg), i in zip(slots, pair):
            x.copy_(xs[i])
            lg.copy_(ls[i])
        torch.cuda.synchronize()
        for _ in range(4):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        _done()
        for got, i in zip(outs, pair):
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


def test_moe_no_tokens():
    w = [_to(t) for t in _experts(2, 128, 128, 1)]
    y, ids, wt = pg.fp8_moe(torch.empty((0, 128), device=DEV), *w, logits=torch.empty((0, 2), device=DEV), top_k=1)
    assert y.shape == (0, 128) and ids.shape == wt.shape == (0, 1)


def test_decoder_layer_tail_of_dense_and_expert_blocks():
    """As a decoder runs them: a dense block-scaled projection, its output
    through the expert layer in one stream, against the binary64 form over the
    dense output."""
    T, H, E, k, F = 12, 528, 8, 2, 272
    x = _x(T, H, 31, "bf16").to(DEV)
    wo = (torch.randn((H, H), generator=torch.Generator().manual_seed(4)) * 0.04).to(DEV)
    wr = (torch.randn((E, H), generator=torch.Generator().manual_seed(5)) * 0.1).to(DEV)
    w = _experts(E, H, F, 6)
    a = pg.fp8_block_linear_dynamic(x, *pg.fp8_quantize_blocks(wo, block_rows=128))
    logits = a.float() @ wr.t()
    y, ids, wt = pg.fp8_moe(a, *(_to(t) for t in w), logits=logits, top_k=k)
    _done()
    rid, rw = route(logits.cpu().numpy(), k)
    assert np.array_equal(ids.cpu().numpy(), rid)
    _check(y, *moe(a.float().cpu().numpy(), *w, rid, wt.cpu().numpy()), "bf16")
    assert E4[0x7E] == 448
