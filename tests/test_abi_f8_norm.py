"""Host-side checks of the block-scaled FP8 calls and the layer norm (no GPU
needed): every call below is refused, or has nothing to do, before any launch."""
import ctypes

import pytest

P = ctypes.c_void_p
fake = P(0x1000)              # never dereferenced
odd = P(0x1008)               # not 16-byte aligned
INVALID, ALIGNMENT, SHAPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 8


@pytest.fixture(scope="module")
def L():
    from block_floating_point_hif4_b200 import build
    build.build()
    from block_floating_point_hif4_b200 import binding
    return binding.lib()


def test_quantize_f8_refusals(L):
    def q(x=fake, dt=1, rows=130, cols=200, ldx=208, fmt=0, br=1, q=fake, ldq=208, s=fake, lds=132, qt=fake,
          ldqt=144, st=fake, ldst=200):
        return L.hif4_quantize_f8(x, dt, rows, cols, ldx, fmt, br, q, ldq, s, lds, qt, ldqt, st, ldst, None, None)

    assert q(rows=-1) == INVALID and q(cols=-1) == INVALID
    assert q(dt=2) == INVALID and q(dt=-1) == INVALID
    assert q(fmt=2) == INVALID and q(fmt=-1) == INVALID
    assert q(br=0) == INVALID and q(br=64) == INVALID
    assert q(x=None) == INVALID
    assert q(q=None, qt=None) == INVALID
    assert q(s=None) == INVALID and q(st=None) == INVALID
    assert q(ldx=192) == SHAPE
    assert q(ldq=192) == SHAPE and q(lds=129) == SHAPE
    assert q(ldqt=128) == SHAPE and q(ldst=199) == SHAPE
    assert q(br=128, lds=1) == SHAPE and q(br=128, ldst=1) == SHAPE
    assert q(x=odd) == ALIGNMENT and q(ldx=204) == ALIGNMENT
    assert q(q=odd) == ALIGNMENT and q(ldq=204) == ALIGNMENT
    assert q(qt=odd) == ALIGNMENT and q(ldqt=136) == ALIGNMENT
    assert q(s=P(0x1002)) == ALIGNMENT and q(st=P(0x1001)) == ALIGNMENT
    assert q(rows=1 << 31, lds=1 << 31, ldqt=1 << 31) == UNSUPPORTED
    assert q(rows=1 << 30, lds=1 << 30, ldqt=1 << 30) == UNSUPPORTED
    assert q(rows=0, x=None, q=None, qt=None) == 0 and q(cols=0) == 0


def test_gemm_f8_block_refusals(L):
    def g(a=fake, af=0, M=200, K=300, lda=304, sa=fake, lsa=200, b=fake, bf=1, N=250, ldb=304, sb=fake, lsb=3,
          br=128, bias=None, y=fake, ldy=256, flags=0):
        return L.hif4_gemm_f8_block(a, af, M, K, lda, sa, lsa, b, bf, N, ldb, sb, lsb, br, bias, y, ldy, flags, None,
                                    None)

    assert g(M=-1) == INVALID and g(N=-1) == INVALID and g(K=-1) == INVALID
    assert g(af=2) == INVALID and g(bf=5) == INVALID and g(br=64) == INVALID
    assert g(flags=1) == INVALID and g(flags=4) == INVALID
    assert g(K=0, lda=0, ldb=0) == SHAPE                 # no block to sum over
    for name in ("a", "sa", "b", "sb", "y"):
        assert g(**{name: None}) == INVALID, name
    assert g(lda=288) == SHAPE and g(ldb=288) == SHAPE and g(ldy=248) == SHAPE
    assert g(lsa=196) == SHAPE and g(lsb=2) == SHAPE
    assert g(br=1, lsb=248) == SHAPE
    for name in ("a", "b", "y", "sa"):
        assert g(**{name: odd}) == ALIGNMENT, name
    assert g(lda=308) == ALIGNMENT and g(ldb=308) == ALIGNMENT
    assert g(lsa=201) == ALIGNMENT and g(ldy=252) == ALIGNMENT
    assert g(sb=P(0x1002)) == ALIGNMENT
    assert g(br=1, lsb=252, sb=P(0x1004)) == ALIGNMENT and g(br=1, lsb=253) == ALIGNMENT
    assert g(bias=P(0x1001)) == ALIGNMENT
    assert g(M=1 << 31, lsa=1 << 31) == UNSUPPORTED
    assert g(M=0, a=None) == 0 and g(N=0, b=None) == 0


def test_layer_norm_refusals(L):
    def n(x=fake, dt=1, rows=40, cols=300, ldx=304, g=fake, b=fake, pdt=0, eps=1e-6, y=fake, out=1, ldy=304,
          mean=None, rstd=None):
        return L.hif4_layer_norm(x, dt, rows, cols, ldx, g, b, pdt, eps, y, out, ldy, mean, rstd, None)

    def f(x=fake, dt=1, rows=40, cols=300, ldx=304, g=fake, b=fake, pdt=0, eps=1e-6, fmt=0, q=fake, ldq=304, s=fake,
          lds=40):
        return L.hif4_layer_norm_f8(x, dt, rows, cols, ldx, g, b, pdt, eps, fmt, q, ldq, s, lds, None, None, None,
                                    None)

    for c in (n, f):
        assert c(rows=-1) == INVALID and c(cols=-1) == INVALID
        assert c(dt=2) == INVALID and c(pdt=2) == INVALID and c(x=None) == INVALID
        for eps in (-1e-6, float("nan"), float("inf")):
            assert c(eps=eps) == INVALID
        assert c(ldx=296) == SHAPE
        assert c(x=odd) == ALIGNMENT and c(ldx=308) == ALIGNMENT
        assert c(g=P(0x1002)) == ALIGNMENT and c(b=P(0x1001)) == ALIGNMENT
        assert c(pdt=1, g=P(0x1001)) == ALIGNMENT
        assert c(rows=0, x=None) == 0 and c(cols=0) == 0
    assert n(y=None) == INVALID and n(out=2) == INVALID
    assert n(ldy=296) == SHAPE and n(y=odd) == ALIGNMENT and n(ldy=300) == ALIGNMENT
    assert n(mean=P(0x1002)) == ALIGNMENT and n(rstd=P(0x1002)) == ALIGNMENT
    assert n(cols=16385, ldx=16392, ldy=16392) == UNSUPPORTED
    assert n(rows=1 << 31) == UNSUPPORTED
    assert f(q=None) == INVALID and f(s=None) == INVALID and f(fmt=2) == INVALID
    assert f(ldq=288) == SHAPE and f(lds=39) == SHAPE
    assert f(q=odd) == ALIGNMENT and f(ldq=312) == ALIGNMENT and f(s=P(0x1002)) == ALIGNMENT


def test_layer_norm_backward_refusals(L):
    ws = L.hif4_layer_norm_backward_workspace(40, 300)
    assert ws >= 2 * 300 * 4
    assert L.hif4_layer_norm_backward_workspace(0, 300) == 0
    assert L.hif4_layer_norm_backward_workspace(40, 16385) == 0
    assert L.hif4_layer_norm_backward_workspace(1 << 20, 5120) <= 1024 * 2 * 5120 * 4     # does not grow with rows

    def b(dy=fake, lddy=304, x=fake, dt=1, rows=40, cols=300, ldx=304, mean=fake, rstd=fake, g=fake, pdt=0, dx=fake,
          lddx=304, dg=fake, db=fake, work=fake, n=ws):
        return L.hif4_layer_norm_backward(dy, lddy, x, dt, rows, cols, ldx, mean, rstd, g, pdt, dx, lddx, dg, db,
                                          work, n, None)

    assert b(rows=-1) == INVALID and b(dt=3) == INVALID and b(pdt=-1) == INVALID
    for name in ("dy", "x", "mean", "rstd"):
        assert b(**{name: None}) == INVALID, name
    assert b(dx=None, dg=None, db=None) == INVALID
    assert b(lddy=296) == SHAPE and b(ldx=296) == SHAPE and b(lddx=296) == SHAPE
    for name in ("dy", "x", "dx"):
        assert b(**{name: odd}) == ALIGNMENT, name
    assert b(lddy=308) == ALIGNMENT and b(ldx=308) == ALIGNMENT and b(lddx=308) == ALIGNMENT
    assert b(mean=P(0x1002)) == ALIGNMENT and b(dg=P(0x1002)) == ALIGNMENT and b(g=P(0x1002)) == ALIGNMENT
    assert b(work=None) == WORKSPACE and b(n=ws - 1) == WORKSPACE
    assert b(work=P(0x1010)) == ALIGNMENT
    assert b(cols=16385, ldx=16392, lddx=16392, lddy=16392) == UNSUPPORTED
    assert b(cols=0) == 0
    assert b(rows=0, dg=None, db=None) == 0              # no sums wanted, no rows


def test_tiles_of_a_product_refusals(L):
    t = (ctypes.c_int32 * 4)()
    f = L.hif4_debug_gemm_f8_block_tiles
    assert f(0, 10, 10, 1, t) == INVALID and f(10, 0, 10, 1, t) == INVALID and f(10, 10, 0, 1, t) == INVALID
    assert f(10, 10, 10, 2, t) == INVALID and f(10, 10, 10, 128, None) == INVALID
    assert f(1 << 31, 10, 10, 1, t) == UNSUPPORTED
