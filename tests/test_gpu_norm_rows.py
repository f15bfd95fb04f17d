"""GPU tests of the layer norm where a block takes many rows one after the other
(its rows in flight come round in a ring several times): each row's results are
those of a call on few rows, bit for bit, also in place; the column sums are
those of the 64-bit form."""
import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import H, dtype_of  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-6
# one width for each way that a row is spread over threads, forward and backward: 8, 16 and 32 lanes, two to four pieces
# a thread, blocks of up to 160, 320, 512 and 1024 threads
WIDTHS = [60, 128, 250, 512, 517, 1024, 1536, 2890, 5120, 6000, 8192, 9000, 16384]


def lanes_of(cols):
    g = R.cdiv(cols, 8)
    return 8 if g <= 8 else 16 if g <= 16 else 32


def many(cols, wide_v):
    """Rows that give each block of a full GPU at least six, and rows that give a block at most one."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if cols <= 1024:
        per_block, blocks = 256 // lanes_of(cols), 8        # 256 threads
    else:
        per_block, blocks = 1, 2048 // (R.cdiv(R.cdiv(cols, 8), 32 * wide_v) * 32)
    return 6 * sms * blocks * per_block + 5, 100 * per_block


def rows_of(rows, cols, dt, seed):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    buf = torch.randn(rows, R.cdiv(cols, 16) * 16, generator=gen, device="cuda")
    buf *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    buf += torch.randn(rows, 1, generator=gen, device="cuda")
    return buf.to(dtype_of(dt))[:, :cols]


def copy_of(t):
    import torch
    return torch.empty(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")[:, :t.shape[1]].copy_(t)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_of_many_rows(H, cols, dt):  # noqa: F811
    import torch
    rows, few = many(cols, 4)
    x = rows_of(rows, cols, dt, cols)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    g, b = 1 + 0.2 * torch.randn(2, cols, generator=gen, device="cuda")
    y, mean, rstd = H.layer_norm(x, g, b, EPS, save_stats=True)
    q, s = H.layer_norm_f8(x, g, b, EPS)
    for i in range(0, rows, few):
        y1, m1, r1 = H.layer_norm(x[i:i + few], g, b, EPS, save_stats=True)
        q1, s1 = H.layer_norm_f8(x[i:i + few], g, b, EPS)
        assert torch.equal(y[i:i + few], y1) and torch.equal(mean[i:i + few], m1) and torch.equal(rstd[i:i + few], r1)
        assert torch.equal(q[i:i + few].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, i:i + few], s1)
    in_place = copy_of(x)
    assert H.layer_norm(in_place, g, b, EPS, out=in_place) is in_place
    assert torch.equal(in_place, y)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_of_many_rows(H, cols, dt):  # noqa: F811
    import torch
    rows, few = many(cols, 2)
    x, dy = rows_of(rows, cols, dt, cols), rows_of(rows, cols, dt, cols + 1)
    g = 1 + 0.2 * torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    _, mean, rstd = H.layer_norm(x, g, None, EPS, save_stats=True)
    dx, dg, db = H.layer_norm_backward(dy, x, mean, rstd, g)
    for i in range(0, rows, few):
        n = slice(i, min(i + few, rows))
        d1, _, _ = H.layer_norm_backward(dy[n], x[n], mean[n], rstd[n], g)
        assert torch.equal(dx[n], d1)
    # a column's sum takes one term per row of its block (at least 100 blocks run), and at most 64 to join them
    dgw, dbw, dga, dba = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4))
    for i in range(0, rows, 8192):
        d = dy[i:i + 8192].double()
        t = d * (x[i:i + 8192].double() - mean[i:i + 8192].double()[:, None]) * rstd[i:i + 8192].double()[:, None]
        dgw, dbw, dga, dba = dgw + t.sum(0), dbw + d.sum(0), dga + t.abs().sum(0), dba + d.abs().sum(0)
    k = R.cdiv(rows, 100) + 100
    assert torch.all((dg.double() - dgw).abs() <= (k + 3) * R.U * dga + 1e-42)
    assert torch.all((db.double() - dbw).abs() <= k * R.U * dba + 1e-42)
    for which in (0, 1):
        c = [copy_of(x), copy_of(dy)]
        o = H.layer_norm_backward(c[1], c[0], mean, rstd, g, out=(c[which], dg.clone(), db.clone()))
        assert torch.equal(o[0], dx) and torch.equal(o[1], dg) and torch.equal(o[2], db)
