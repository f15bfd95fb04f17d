"""GPU tests of the block-scaled FP8 quantizer and product against plain 64-bit
forms: the quantizer bit for bit, the product within a bound that counts the
roundings of its definition."""
import numpy as np
import pytest

from tests import _f8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    import block_floating_point_hif4_b200 as h
    from block_floating_point_hif4_b200 import build
    build.build()
    return h


def fmt_of(name):
    import torch
    return {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[name]


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def on_gpu(x, dtype, ld=None):
    """x on the GPU in a buffer with leading dimension ld (default: a multiple of 16), filled with NaN."""
    import torch
    rows, cols = x.shape
    buf = torch.full((rows, ld or R.cdiv(cols, 16) * 16), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)
    return buf[:, :cols]


def host(t):
    """Values in 64 bits."""
    return t.float().cpu().numpy().astype(np.float64)


def matrix(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * rng.lognormal(0, 1.0, (1, cols)) * rng.lognormal(0, 1.0, (rows, 1))
    x[rng.random((rows, cols)) < 0.01] *= 30
    return x


def poisoned(rows, cols, dtype, extra_rows=1, multiple=16):
    """A buffer of bytes 0x5A with room past the rows and columns, and its view."""
    import torch
    ld = R.cdiv(cols, multiple) * multiple + multiple
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full(((rows + extra_rows) * ld * size,), 0x5A, dtype=torch.uint8, device="cuda")
    return raw, raw.view(dtype).view(rows + extra_rows, ld)[:rows, :cols]


def assert_only_view_written(raw, view):
    import torch
    size = view.element_size()
    ld = view.stride(0)
    grid = raw.view(-1, ld * size)
    assert torch.all(grid[view.shape[0]:] == 0x5A), "rows past the last were written"
    assert torch.all(grid[:view.shape[0], view.shape[1] * size:] == 0x5A), "columns past the last were written"


SIZES = [(1, 1), (1, 128), (3, 127), (128, 128), (129, 257), (200, 640), (5, 1000), (300, 72), (257, 16), (64, 2049)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantizer_is_exact(H, rows, cols, block, dt):
    import torch
    rng = np.random.default_rng(rows * 1000 + cols)
    x = matrix(rng, rows, cols)
    if rows > 2:
        x[1] = 0.0                                          # blocks of zeros
        x[2, : cols // 2] = 1e-38 if dt == "f32" else 0.0   # below the smallest block maximum
    for fmt in ("e4m3", "e5m2"):
        xd = on_gpu(x, dtype_of(dt))
        xh = host(xd)
        for layout in ("rows", "cols", "both"):
            outs, raws = [], []
            for direct in {"rows": (1,), "cols": (0,), "both": (1, 0)}[layout]:
                r, c = (rows, cols) if direct else (cols, rows)
                s = (R.cdiv(c, 128), r) if block == 1 else (R.cdiv(r, 128), R.cdiv(c, 128))
                for shape, d in (((r, c), fmt_of(fmt)), (s, torch.float32)):
                    raw, view = poisoned(*shape, d)
                    raws.append(raw)
                    outs.append(view)
            got = H.quantize_f8(xd, fmt_of(fmt), block_rows=block, layout=layout, out=tuple(outs))
            torch.cuda.synchronize()
            for raw, view in zip(raws, outs):
                assert_only_view_written(raw, view)
            got = list(got)
            for direct in {"rows": (1,), "cols": (0,), "both": (1, 0)}[layout]:
                q, s = got.pop(0), got.pop(0)
                want_q, want_s = R.quantize(xh if direct else xh.T, fmt, 1 if block == 1 else 128, 128)
                if block == 1:
                    want_s = want_s.T
                assert np.array_equal(s.cpu().numpy(), want_s), (fmt, layout, direct)
                assert np.array_equal(host(q), want_q), (fmt, layout, direct)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantizer_maps_nonfinite_and_reports_it(H, dt, block):
    import torch
    from block_floating_point_hif4_b200 import binding as B
    xd = on_gpu(np.random.default_rng(3).standard_normal((130, 200)), dtype_of(dt))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for layout in ("rows", "cols", "both"):
        H.quantize_f8(xd, block_rows=block, layout=layout, status=st)
        assert H.get_status(st) == B.OK
    xd[5, 7] = float("nan")
    xd[129, 199] = float("inf")
    xd[6, 0] = float("-inf")
    xd[7, 130] = float("nan")
    x = host(xd)
    for layout in ("rows", "cols", "both"):
        st.zero_()
        got = list(H.quantize_f8(xd, block_rows=block, layout=layout, status=st))
        assert H.get_status(st) == B.ERR_NONFINITE
        for direct in {"rows": (1,), "cols": (0,), "both": (1, 0)}[layout]:
            q, s = host(got.pop(0)), got.pop(0).cpu().numpy()
            want_q, want_s = R.quantize(x if direct else x.T, "e4m3", block, 128)
            assert np.array_equal(q, want_q) and np.array_equal(s, want_s.T if block == 1 else want_s)
            q = q if direct else q.T
            assert q[5, 7] == 0 and q[7, 130] == 0 and q[129, 199] == 448 and q[6, 0] == -448


def operand(H, rng, rows, K, fmt, block):
    import torch
    x = matrix(rng, rows, K)
    q, s = H.quantize_f8(on_gpu(x, torch.float32), fmt_of(fmt), block_rows=block)
    sh = s.cpu().numpy()
    return q, s, host(q), (sh.T if block == 1 else sh)


GEMMS = [(1, 128, 128), (1, 1, 1), (1, 300, 1000), (2, 256, 4096), (7, 100, 129), (16, 512, 640), (17, 130, 640),
         (32, 257, 2048), (33, 384, 100), (64, 1000, 512), (65, 128, 128), (100, 300, 777), (128, 256, 1152),
         (129, 129, 64), (200, 333, 1000), (256, 512, 512), (300, 264, 2048), (513, 640, 384),
         # enough tiles for the CTA pairs, 192 and 256 columns wide; 256 k + 1 rows leave a pair's second
         # CTA without one
         (2305, 2817, 129), (2560, 2500, 300), (2400, 2600, 1024), (513, 3716, 100), (769, 3457, 100),
         (770, 3100, 1100), (900, 3600, 1100)]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("block", [1, 128])
def test_product_matches_the_definition(H, M, N, K, block):
    import torch
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    for af, bf, out, bias in (("e4m3", "e4m3", "bf16", True), ("e5m2", "e4m3", "f32", False),
                              ("e4m3", "e5m2", "f32", True), ("e5m2", "e5m2", "bf16", False)):
        a, sa, av, sav = operand(H, rng, M, K, af, 1)
        b, sb, bv, sbv = operand(H, rng, N, K, bf, block)
        bh = rng.standard_normal(N) if bias else None
        bd = None
        if bias:
            bd = torch.from_numpy(bh).to("cuda", torch.bfloat16)
            bh = host(bd)
        raw, view = poisoned(M, N, dtype_of(out))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = H.gemm_f8_block(a, sa, b, sb, bd, b_block_rows=block, out=view, status=st)
        assert H.get_status(st) == 0
        want, bound = R.gemm(av, sav, bv, sbv, 1 if block == 1 else 128, bh)
        R.assert_within(host(y), want, R.stored(bound, want, out), "%s x %s -> %s" % (af, bf, out))
        assert_only_view_written(raw, view)


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (16, 300, 2000), (200, 300, 4096), (2560, 2500, 300)])
def test_product_is_the_same_every_time(H, M, N, K):
    import torch
    rng = np.random.default_rng(11)
    a, sa, _, _ = operand(H, rng, M, K, "e4m3", 1)
    b, sb, _, _ = operand(H, rng, N, K, "e4m3", 128)
    first = H.gemm_f8_block(a, sa, b, sb, out_f32=True).clone()
    for _ in range(20):
        assert torch.equal(H.gemm_f8_block(a, sa, b, sb, out_f32=True), first)
    assert torch.equal(H.gemm_f8_block(a, sa, b, sb), first.to(torch.bfloat16))


def test_nan_code_reaches_its_row_only(H):
    import torch
    rng = np.random.default_rng(12)
    for M in (3, 150):
        a, sa, _, _ = operand(H, rng, M, 512, "e4m3", 1)
        b, sb, _, _ = operand(H, rng, 200, 512, "e4m3", 128)
        clean = H.gemm_f8_block(a, sa, b, sb, out_f32=True)
        a.view(torch.uint8)[1, 300] = 0x7F
        y = H.gemm_f8_block(a, sa, b, sb, out_f32=True)
        assert torch.all(torch.isnan(y[1]))
        keep = torch.arange(M, device="cuda") != 1
        assert torch.equal(y[keep], clean[keep])


def test_bounded_waits_of_the_product(H):
    """A copy that is never issued: the call ends, reports it, and the next call is right."""
    import torch
    from block_floating_point_hif4_b200 import binding as B
    rng = np.random.default_rng(13)
    for M, N, K in ((1, 512, 4096), (300, 300, 512), (2560, 2500, 300)):
        a, sa, av, sav = operand(H, rng, M, K, "e4m3", 1)
        b, sb, bv, sbv = operand(H, rng, N, K, "e4m3", 128)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        H.lib().hif4_debug_wait_test(1, 20_000_000)
        try:
            H.gemm_f8_block(a, sa, b, sb, status=st)
            code = H.get_status(st)
        finally:
            H.lib().hif4_debug_wait_test(0, 0)
        assert code == B.ERR_TIMEOUT
        st.zero_()
        y = H.gemm_f8_block(a, sa, b, sb, out_f32=True, status=st)
        assert H.get_status(st) == B.OK
        want, bound = R.gemm(av, sav, bv, sbv, 128)
        R.assert_within(host(y), want, R.stored(bound, want, "f32"))


def test_refusals_of_the_binding(H):
    import torch
    x = torch.zeros(4, 256, device="cuda")
    with pytest.raises(ValueError):
        H.quantize_f8(x.t())                                # rows not contiguous
    with pytest.raises(ValueError):
        H.quantize_f8(x.half())
    with pytest.raises(ValueError):
        H.quantize_f8(x, torch.uint8)
    with pytest.raises(ValueError):
        H.quantize_f8(x, block_rows=64)
    with pytest.raises(ValueError):
        H.quantize_f8(x, layout="both", out=H.quantize_f8(x))
    with pytest.raises(H.Hif4Error):
        H.quantize_f8(torch.zeros(4, 130, device="cuda")[:, 1:129])     # misaligned
    with pytest.raises(H.Hif4Error):
        H.quantize_f8(torch.zeros(1, 256, device="cuda").expand(4, 256))    # rows on top of one another
    q, s = H.quantize_f8(x)
    w, sw = H.quantize_f8(x, block_rows=128)
    with pytest.raises(ValueError):
        H.gemm_f8_block(q, s, w[:, :128], sw)
    with pytest.raises(ValueError):
        H.gemm_f8_block(q, s[:1], w, sw)
    with pytest.raises(ValueError):
        H.gemm_f8_block(q, s, w, sw, b_block_rows=1)        # scales of the other kind
    with pytest.raises(ValueError):
        H.gemm_f8_block(q.view(torch.uint8), s, w, sw)
    with pytest.raises(ValueError):
        H.gemm_f8_block(q, s, w, sw, torch.zeros(4, device="cuda"))     # bias not BF16
    with pytest.raises(ValueError):
        H.gemm_f8_block(q, s.cpu(), w, sw)
    assert H.gemm_f8_block(q[:0], s[:, :0], w, sw).shape == (0, 4)
