"""GPU tests of how the block-scaled FP8 product reads its scales: exactly those
of the operands' rows, whatever lies behind them."""
import numpy as np
import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import H, host, on_gpu, operand  # noqa: F401

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
