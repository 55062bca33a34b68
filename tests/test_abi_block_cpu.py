"""Host-side argument checks of the block-scaled operators and the
mixture-of-experts layer (CPU only: nothing here is enqueued), and the binding's
checks of shapes, types and devices."""
import ctypes

import pytest
import torch

import precision_gemm_fp8_b200 as pg

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000   # fake 16-byte aligned addresses: checks fail before use
MIS = 0x10008
INV, ALN, UNS = pg.ERR_INVALID_ARG, pg.ERR_ALIGNMENT, pg.ERR_UNSUPPORTED


def test_quantize_blocks_arguments():
    def q(x=A, dt=pg.F32, batch=1, rows=4, cols=64, ldx=64, ldb=256, block=1, q=B, s=C):
        return pg.lib.pgf8_fp8_quantize_blocks(x, dt, batch, rows, cols, ldx, ldb, block, q, s, 0, None)
    assert q(x=None) == q(q=None) == q(s=None) == INV
    assert q(dt=3) == q(dt=-1) == UNS
    assert q(rows=-1) == q(batch=-1) == q(cols=8) == q(ldx=32) == q(block=64) == q(block=0) == INV
    assert q(cols=60, ldx=64) == q(ldx=66) == q(x=MIS) == q(q=B + 8) == q(s=C + 2) == ALN
    assert q(batch=2, ldb=-16) == INV and q(batch=2, ldb=258) == ALN
    assert q(batch=2, ldb=512) == UNS                       # row groups of matrices that do not follow one another
    assert q(dt=pg.BF16, ldx=68) == ALN
    assert q(rows=2 ** 31 - 1, cols=1 << 20, ldx=1 << 20) == UNS   # more CTAs than a grid holds
    assert q(x=None, q=None, s=None, rows=0) == q(x=None, q=None, s=None, batch=0) == pg.OK


def test_silu_mul_quantize_blocks_arguments():
    def s(x=A, dt=pg.BF16, rows=4, inter=64, ldg=128, q=B, sc=C):
        return pg.lib.pgf8_fp8_silu_mul_quantize_blocks(x, dt, rows, inter, ldg, q, sc, 0, None)
    assert s(x=None) == s(q=None) == s(sc=None) == s(inter=0) == s(ldg=120) == s(rows=-1) == INV
    assert s(dt=7) == UNS
    assert s(inter=56) == s(ldg=132) == s(x=MIS) == ALN
    assert s(rows=0, x=None, q=None, sc=None) == pg.OK


def test_block_linear_arguments():
    def f(aq=A, sa=B, M=4, K=256, wq=C, sw=D, N=128, y=A, dt=pg.BF16):
        return pg.lib.pgf8_fp8_block_linear(aq, sa, M, K, wq, sw, N, y, dt, 0, None)
    for k in ("aq", "sa", "wq", "sw", "y"):
        assert f(**{k: None}) == INV, k
    assert f(M=-1) == f(K=0) == f(N=8) == f(M=1 << 24) == INV
    assert f(K=264) == f(N=136) == f(aq=MIS) == f(wq=MIS) == f(y=MIS) == f(sa=B + 2) == f(sw=D + 1) == ALN
    assert f(dt=3) == UNS
    assert f(M=0, aq=None, sa=None, wq=None, sw=None, y=None) == pg.OK

    def d(x=A, xdt=pg.F32, M=4, K=256, ldx=256, wq=C, sw=D, N=128, y=A, dt=pg.BF16, ws=B, nb=1 << 20):
        return pg.lib.pgf8_fp8_block_linear_dynamic(x, xdt, M, K, ldx, wq, sw, N, y, dt, ws, nb, 0, None)
    for k in ("x", "wq", "sw", "y", "ws"):
        assert d(**{k: None}) == INV, k
    need = pg.fp8_block_linear_dynamic_workspace_size(4, 256)
    assert need >= 4 * 256 + 4 * 2 * 4 and d(nb=need - 1) == INV
    assert d(ldx=128) == INV and d(ldx=257) == d(ws=MIS) == d(x=MIS) == ALN and d(xdt=5) == d(dt=5) == UNS
    assert d(M=0, x=None, wq=None, sw=None, y=None, ws=None, nb=0) == pg.OK
    assert pg.fp8_block_linear_dynamic_workspace_size(0, 256) == 0
    assert pg.lib.pgf8_fp8_block_linear_dynamic_scales_offset(3, 272) >= 3 * 272


def _layer(**kw):
    d = dict(x=A, w13=B, s13=C, w2=D, s2=C, logits=A, ids=B, weights=C, y=D, workspace=A, workspace_bytes=1 << 30,
             tokens=4, hidden=256, inter=128, experts=8, top_k=2, ldx=256, ldl=8, xdt=pg.BF16, ldt=pg.F32,
             ydt=pg.BF16, score=pg.MOE_SOFTMAX, renormalise=1, factor=1.0)
    d.update(kw)
    return pg.MoeLayer(**d)


def test_moe_arguments():
    f = lambda **kw: pg.lib.pgf8_fp8_moe(ctypes.byref(_layer(**kw)), 0, None)  # noqa: E731
    assert pg.lib.pgf8_fp8_moe(None, 0, None) == INV
    for k in ("x", "w13", "s13", "w2", "s2", "y", "workspace"):
        assert f(**{k: None}) == INV, k
    assert f(logits=None, ids=None) == f(logits=None, weights=None) == INV
    assert f(tokens=-1) == f(hidden=0) == f(inter=8) == f(experts=0) == f(top_k=0) == f(top_k=9) == INV
    assert f(ldx=128) == f(ldl=7) == f(score=2) == f(factor=float("nan")) == INV
    assert f(tokens=65) == f(experts=513, ldl=513) == f(experts=32, ldl=32, top_k=17) == UNS
    assert f(hidden=(1 << 20) + 16, ldx=1 << 21) == f(xdt=4) == f(ydt=4) == f(ldt=9) == UNS
    assert f(experts=512, ldl=512, hidden=1 << 20, inter=1 << 20, ldx=1 << 20) == UNS      # 2^31 weight rows
    assert f(hidden=264, ldx=264) == f(inter=136) == f(ldx=260) == f(x=MIS) == f(w2=MIS) == f(y=MIS) == ALN
    assert f(workspace=MIS) == f(s13=C + 2) == f(ids=B + 1) == f(logits=A + 2) == ALN
    need = pg.fp8_moe_workspace_size(4, 256, 128, 8, 2)
    assert need > 4 * 256 + 8 * 128 and f(workspace_bytes=need - 1) == INV
    assert f(tokens=0, x=None, w13=None, workspace=None) == pg.OK
    assert pg.fp8_moe_workspace_size(65, 256, 128, 8, 2) == 0 and pg.fp8_moe_workspace_size(4, 256, 128, 8, 9) == 0


def test_moe_constants_match_the_header():
    import re
    values = dict(re.findall(r"\b(PGF8_MOE_[A-Z]+)\s*=\s*(\d+)", open(pg.HEADER_PATH).read()))
    assert values == {"PGF8_MOE_SOFTMAX": str(pg.MOE_SOFTMAX), "PGF8_MOE_SIGMOID": str(pg.MOE_SIGMOID)}


def test_moe_record_matches_the_header():
    """Field order and size of the record as the C struct lays them out."""
    import re
    text = open(pg.HEADER_PATH).read()
    body = re.search(r"typedef struct \{([^}]*)\} pgf8_fp8_moe_layer;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip().lstrip("*") for line in re.findall(r"(?:const )?\w+ ([^;]+);", body) for n in line.split(",")]
    assert names == [n for n, _ in pg.MoeLayer._fields_]
    assert ctypes.sizeof(pg.MoeLayer) == 10 * 8 + 8 + 7 * 8 + 6 * 4


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 256))
    with pytest.raises(ValueError):
        pg.fp8_quantize_blocks(x)                               # host memory
    with pytest.raises(ValueError):
        pg.fp8_quantize_blocks(x, block_rows=64)
    with pytest.raises(ValueError):
        pg.fp8_quantize_blocks(x.t())
    with pytest.raises(TypeError):
        pg.fp8_quantize_blocks(x.double())
    with pytest.raises(ValueError):
        pg.fp8_silu_mul_quantize_blocks(torch.zeros((4, 255)))
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    w, sw = torch.zeros((128, 256), dtype=torch.uint8), torch.zeros((1, 2))
    with pytest.raises(ValueError):
        pg.fp8_block_linear(q, s, w, sw)                        # host memory
    for bad in ((q, s, w, torch.zeros((2, 2))), (q, torch.zeros((4, 3)), w, sw), (q, s, w[:, :128], sw),
                (q.float(), s, w, sw), (q, s, w, sw.double())):
        with pytest.raises(ValueError):
            pg.fp8_block_linear(*bad)
    w13, s13 = torch.zeros((2, 256, 256), dtype=torch.uint8), torch.zeros((2, 2, 1, 2))
    w2, s2 = torch.zeros((2, 256, 128), dtype=torch.uint8), torch.zeros((2, 2, 1))
    good = (x, w13, s13, w2, s2)
    with pytest.raises(ValueError):
        pg.fp8_moe(*good)                                       # neither logits nor ids
    with pytest.raises(ValueError):
        pg.fp8_moe(*good, logits=torch.zeros((4, 2)))           # no top_k
    with pytest.raises(ValueError):
        pg.fp8_moe(*good, logits=torch.zeros((4, 3)), top_k=1)
    with pytest.raises(ValueError):
        pg.fp8_moe(x, w13, s13[:, :1], w2, s2, logits=torch.zeros((4, 2)), top_k=1)
    with pytest.raises(ValueError):
        pg.fp8_moe(*good, ids=torch.zeros((4, 1)), weights=torch.zeros((4, 1)))    # ids not int32
    with pytest.raises(ValueError):
        pg.fp8_moe(*good, logits=torch.zeros((4, 2)), top_k=1)  # host memory
