"""GPU tests of how the block-scaled FP8 product reads its scales: exactly those
of the operands' rows, whatever lies behind them."""
import numpy as np
import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import H, fmt_of, host, on_gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu


def in_exact_storage(s, ld):
    """A block-major scale array whose storage ends with the last row's last scale, NaN between the rows."""
    import torch
    units, rows = s.shape
    buf = torch.full(((units - 1) * ld + rows,), float("nan"), device="cuda")
    view = torch.as_strided(buf, (units, rows), (ld, 1))
    view.copy_(s)
    assert view.untyped_storage().nbytes() == ((units - 1) * ld + rows) * 4
    return view


@pytest.mark.parametrize("M", [1, 2, 3, 5, 31, 33, 129, 130, 131, 2561])
@pytest.mark.parametrize("N,K", [(1, 100), (203, 700), (2917, 129)])
@pytest.mark.parametrize("block", [1, 128])
def test_scales_behind_the_last_row_are_not_read(H, M, N, K, block):  # noqa: F811
    rng = np.random.default_rng(M * 5 + N + K)
    a, sa, av, sav = operand(H, rng, M, K, "e4m3", 1)
    b, sb, bv, sbv = operand(H, rng, N, K, "e4m3", block)
    want, bound = R.gemm(av, sav, bv, sbv, 1 if block == 1 else 128)
    sa = in_exact_storage(sa, R.cdiv(M, 4) * 4 + 8)
    if block == 1:
        sb = in_exact_storage(sb, R.cdiv(N, 4) * 4)
    y = H.gemm_f8_block(a, sa, b, sb, b_block_rows=block, out_f32=True)
    R.assert_within(host(y), want, R.stored(bound, want, "f32"))


# a few tokens, 128 x 128 tiles, K shared by a cluster, pairs of 192 and of 256 columns
TILES = [(3, 300, 700), (30, 200, 2100), (100, 300, 300), (200, 300, 4096), (2560, 2500, 300), (900, 3600, 1100)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("block", [1, 128])
def test_scales_whose_product_overflows_meet_sums_of_zero(H, M, N, K, block):  # noqa: F811
    """Elements of the largest magnitude (what an infinity becomes) at places that the other operand leaves 0."""
    import torch
    top = float(np.finfo(np.float32).max)
    a, b = torch.zeros(M, K, device="cuda"), torch.zeros(N, K, device="cuda")
    a[::2, 0::3], b[1::2, 1::3] = top, -top
    a[1::2], b[0::2] = 1.0, 0.5
    for af in ("e4m3", "e5m2"):
        q, s = H.quantize_f8(on_gpu(a.cpu().numpy(), torch.float32), fmt_of(af))
        w, sw = H.quantize_f8(on_gpu(b.cpu().numpy(), torch.float32), block_rows=block)
        y = H.gemm_f8_block(q, s, w, sw, b_block_rows=block, out_f32=True)
        assert not torch.any(torch.isnan(y))
        # even rows of a and odd rows of b never meet outside 0; the rest as the definition says
        assert not torch.any(y[::2, 1::2])
        want = (dequant(q, s, 1).double() @ dequant(w, sw, block).double().t()).float()
        small = want.abs() < 1e30
        assert torch.allclose(y[small], want[small], rtol=1e-4, atol=0.0)
        assert torch.equal(torch.isinf(y), torch.isinf(want))


def dequant(q, s, block):
    import torch
    rows, cols = q.shape
    f = s.t() if block == 1 else s.repeat_interleave(128, 0)[:rows]
    return q.to(torch.float64) * f.double().repeat_interleave(128, 1)[:, :cols]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("block", [1, 128])
def test_scales_whose_product_overflows_meet_small_sums(H, M, N, K, block):  # noqa: F811
    """Products of scales of 2^128 to 2^134 on codes of 2^-9 to 2^-7: results that FP32 holds, in all their digits; what
    has ordinary scales comes out bit for bit as without the others."""
    import torch
    rng = np.random.default_rng(M + 3 * N + K)

    def codes(rows):
        raw = torch.from_numpy(rng.integers(0, 5, (rows, R.cdiv(K, 16) * 16)).astype(np.uint8)).cuda()
        raw |= torch.from_numpy((rng.integers(0, 2, raw.shape) << 7).astype(np.uint8)).cuda()
        return raw.view(torch.float8_e4m3fn)[:, :K]

    a, b = codes(M), codes(N)
    units = R.cdiv(K, 128)
    sa, sb = np.exp2(rng.uniform(-1, 1, (M, units))), np.exp2(rng.uniform(-1, 1, (N if block == 1 else R.cdiv(N, 128), units)))
    plain = [x.astype(np.float32) for x in (sa, sb)]
    arows, brows = np.arange(M) % 3 == 0, np.arange(sb.shape[0]) % 2 == 0
    sa[arows] *= 2.0 ** 71
    sb[brows] *= 2.0 ** 60                                  # below 2^63 by itself
    far = [x.astype(np.float32) for x in (sa, sb)]

    def on(s, by_row):
        s = torch.from_numpy(s).cuda()
        if by_row:
            buf = torch.zeros(units, R.cdiv(s.shape[0], 4) * 4, device="cuda")
            buf[:, :s.shape[0]] = s.t()
            return buf[:, :s.shape[0]]
        return s.contiguous()

    y = H.gemm_f8_block(a, on(far[0], True), b, on(far[1], block == 1), b_block_rows=block, out_f32=True)
    want, bound = R.gemm(host(a), far[0], host(b), far[1], 1 if block == 1 else 128)
    R.assert_within(host(y), want, R.stored(bound, want, "f32"))
    y0 = H.gemm_f8_block(a, on(plain[0], True), b, on(plain[1], block == 1), b_block_rows=block, out_f32=True)
    cols = np.repeat(brows, 1 if block == 1 else 128)[:N]
    r, c = torch.from_numpy(~arows).cuda(), torch.from_numpy(~cols).cuda()
    assert torch.equal(y[r][:, c], y0[r][:, c])


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("block", [1, 128])
def test_scales_whose_product_is_subnormal(H, M, N, K, block):  # noqa: F811
    """Products of scales near 2^-134: each is off by half a step of a subnormal, 2^-150, and so is its term per unit
    of the block's sum."""
    import torch
    rng = np.random.default_rng(M + 5 * N + K)
    a, _, av, _ = operand(H, rng, M, K, "e4m3", 1)
    b, _, bv, _ = operand(H, rng, N, K, "e4m3", block)
    units = R.cdiv(K, 128)
    sa = np.exp2(rng.uniform(-69, -65, (M, units))).astype(np.float32)
    sb = np.exp2(rng.uniform(-69, -65, (N if block == 1 else R.cdiv(N, 128), units))).astype(np.float32)

    def on(s, by_row):
        s = torch.from_numpy(s).cuda()
        if not by_row:
            return s
        buf = torch.zeros(units, R.cdiv(s.shape[0], 4) * 4, device="cuda")
        buf[:, :s.shape[0]] = s.t()
        return buf[:, :s.shape[0]]

    y = H.gemm_f8_block(a, on(sa, True), b, on(sb, block == 1), b_block_rows=block, out_f32=True)
    want, bound = R.gemm(av, sa, bv, sb, 1 if block == 1 else 128)
    bound = bound + 2.0 ** -150 * (1 + 2 * R.U * units) * (np.abs(av) @ np.abs(bv).T)
    R.assert_within(host(y), want, R.stored(bound, want, "f32"))
