"""GPU tests of the block-scaled FP8 product's give-up path: a copy that is never
issued.  Every wait ends by its own limit; the block leaves only after what its
tensor cores and copies still owe it, in a pair also what the other CTA owes it,
has arrived, so the calls right after it are right, on every kind of tile."""
import numpy as np
import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import H, host, operand  # noqa: F401

pytestmark = pytest.mark.gpu

LIMIT_NS = 20_000_000

# one CTA streaming the weight, K shared by a cluster, 128 x 128 tiles, pairs of 192 and of 256 columns (with one
# tile and with several for a pair)
SHAPES = [(20, 700, 300), (1, 512, 4096), (200, 300, 4096), (300, 300, 512), (2560, 2500, 300), (900, 3600, 1100),
          (2560, 5120, 1400)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
def test_calls_after_a_time_out_are_right(H, M, N, K, block):  # noqa: F811
    import torch
    from block_floating_point_hif4_b200 import binding as B
    rng = np.random.default_rng(M + N + K)
    a, sa, av, sav = operand(H, rng, M, K, "e4m3", 1)
    b, sb, bv, sbv = operand(H, rng, N, K, "e4m3", block)
    want, bound = R.gemm(av, sav, bv, sbv, 1 if block == 1 else 128)
    bound = R.stored(bound, want, "f32")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        st.zero_()
        H.lib().hif4_debug_wait_test(1, LIMIT_NS)
        try:
            H.gemm_f8_block(a, sa, b, sb, b_block_rows=block, status=st)
        finally:
            H.lib().hif4_debug_wait_test(0, 0)
        later = [H.gemm_f8_block(a, sa, b, sb, b_block_rows=block, out_f32=True) for _ in range(2)]
        assert H.get_status(st) == B.ERR_TIMEOUT
        for y in later:                                     # queued right behind the call that gave up
            R.assert_within(host(y), want, bound)
