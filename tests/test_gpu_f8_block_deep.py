"""GPU tests of the block-scaled FP8 product in the states that large calls run
in: more units than the block scales in hand at once, several tiles for a pair of
CTAs, K shared by up to eight CTAs, two calls at a time.  Which tiles a shape
takes is asked for and checked, so that a shape keeps testing what it is here for.
The 64-bit products run on the GPU."""
import ctypes

import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import H, fmt_of  # noqa: F401

pytestmark = pytest.mark.gpu


def tiles_of(H, M, N, K, block):  # noqa: F811
    """(rows, columns) of a tile, CTAs that share its K, tiles for a CTA (or pair)."""
    t = (ctypes.c_int32 * 4)()
    assert H.lib().hif4_debug_gemm_f8_block_tiles(M, N, K, block, t) == 0
    rows, cols, split, ctas = t
    if M <= 32:
        tiles = R.cdiv(N, rows) * R.cdiv(M, cols)
    else:
        tiles = R.cdiv(M, rows) * R.cdiv(N, cols)
    return (rows, cols), split, tiles / (ctas / (2 if rows == 256 else split))


def operand64(H, gen, rows, K, fmt, block):  # noqa: F811
    """An operand with its scales, and its dequantized values in 64 bits."""
    import torch
    x = torch.randn(rows, R.cdiv(K, 16) * 16, generator=gen, device="cuda")
    x *= torch.exp(torch.randn(rows, 1, generator=gen, device="cuda"))
    q, s = H.quantize_f8(x[:, :K], fmt_of(fmt), block_rows=block)
    f = s.t() if block == 1 else s.repeat_interleave(128, 0)[:rows]
    return q, s, q.double() * f.double().repeat_interleave(128, 1)[:, :K]


def check(y, a64, b64, bias, K, out):
    """The bound of the reference's gemm(), on the GPU."""
    import torch
    want, mag = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    bound = (4 * 33 * 2 + 3 + R.cdiv(K, 128) + 8 + 1) * R.U * mag
    bound = bound + R.HALF_STEP[out] * (want.abs() + bound) + 1e-42
    over = (y.double() - want).abs() - bound
    assert torch.all(torch.isfinite(y)) and over.max().item() <= 0, over.max().item()


def product(H, seed, M, N, K, block, af="e4m3", bf="e4m3", out="f32", bias=False):  # noqa: F811
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    a, sa, a64 = operand64(H, gen, M, K, af, 1)
    b, sb, b64 = operand64(H, gen, N, K, bf, block)
    bd = torch.randn(N, generator=gen, device="cuda").bfloat16() if bias else None
    y = H.gemm_f8_block(a, sa, b, sb, bd, b_block_rows=block, out_f32=out == "f32")
    check(y, a64, b64, bd, K, out)
    return (a, sa, b, sb, bd), y


# 35 and 69 units (block scales are in hand 32 at a time), odd ones; more tiles than pairs of CTAs
@pytest.mark.parametrize("M,N,K,tile", [(5000, 1500, 4400, (256, 256)), (2500, 2100, 4400, (256, 192)),
                                        (1100, 3300, 8800, (256, 256)), (1000, 2500, 8800, (256, 192)),
                                        (1700, 2600, 4400, (128, 128)), (3000, 3000, 129, (256, 256))])
@pytest.mark.parametrize("block", [1, 128])
def test_deep_products_on_every_tile(H, M, N, K, tile, block):  # noqa: F811
    got, split, per_cta = tiles_of(H, M, N, K, block)
    assert got == tile and split == 1
    assert per_cta > 1 or K > 8000
    product(H, M + N + K, M, N, K, block, "e4m3", "e4m3", "f32", True)
    product(H, M + N + K, M, N, K, block, "e5m2", "e4m3", "bf16", False)


@pytest.mark.parametrize("M", [1, 20, 100, 250])
@pytest.mark.parametrize("block", [1, 128])
def test_k_shared_by_up_to_eight(H, M, block):  # noqa: F811
    seen = set()
    for n in (2, 5, 6, 7, 8, 9, 10, 11, 13, 16, 18, 20, 24):
        N = n * 128 - 27
        split = tiles_of(H, M, N, 8300, block)[1]
        seen.add(split)
        product(H, n, M, N, 8300, block, "e4m3", "e5m2", "f32" if n & 1 else "bf16", n % 3 == 0)
    assert {5, 6, 8} <= seen, seen


@pytest.mark.parametrize("M,N", [(1, 5120), (16, 5120), (32, 1300), (33, 5120), (64, 5120), (130, 5120), (256, 5120)])
def test_few_rows_through_a_deep_linear(H, M, N):  # noqa: F811
    product(H, M, M, N, 13824, 128, out="bf16", bias=True)


@pytest.mark.parametrize("M,N,K,block,tile", [(512, 5120, 13824, 128, (256, 192)), (512, 5120, 13824, 1, (256, 192)),
                                              (1100, 3300, 8800, 128, (256, 256)), (2000, 2500, 14391, 1, None),
                                              (1, 5120, 13824, 128, (128, 16)), (200, 700, 8300, 1, (128, 128))])
def test_the_same_every_time_among_others(H, M, N, K, block, tile):  # noqa: F811
    """The same bits from calls right behind calls on other operands."""
    import torch
    assert tile is None or tiles_of(H, M, N, K, block)[0] == tile
    ours, first = product(H, 1, M, N, K, block)
    other, _ = product(H, 2, M, N, K, block)
    for _ in range(25):
        ys = []
        for _ in range(4):
            ys.append(H.gemm_f8_block(*ours, b_block_rows=block, out_f32=True))
            H.gemm_f8_block(*other, b_block_rows=block, out_f32=True)
        assert all(torch.equal(y, first) for y in ys)


def test_two_calls_at_a_time(H):  # noqa: F811
    """Products on every kind of tile on two streams at once: pairs that take all of a CTA's tensor memory, clusters and
    tiles of one CTA."""
    import torch
    shapes = [(2500, 2100, 4400, 128), (900, 3600, 1100, 1), (1, 1000, 8300, 128), (2500, 2100, 1100, 1),
              (200, 700, 8300, 1), (5000, 1500, 700, 128)]
    assert {tiles_of(H, *s)[0] for s in shapes} == {(256, 256), (256, 192), (128, 128), (128, 16)}
    args = [product(H, i, *s) for i, s in enumerate(shapes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for r in range(6):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                for i in range(len(shapes)):
                    i = (i + 3 * j + r) % len(shapes)
                    got.append((i, H.gemm_f8_block(*args[i][0], b_block_rows=shapes[i][3], out_f32=True)))
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, args[i][1]), shapes[i]


def test_first_call_of_a_process_may_be_captured():
    """No call before the capture: nothing that the calls set up once is refused there."""
    import os
    import subprocess
    import sys
    code = """
import torch, block_floating_point_hif4_b200 as H
x = torch.randn(300, 640, device="cuda")
w = torch.randn(3000, 640, device="cuda")
torch.cuda.synchronize()
def f():
    h, s, mean, rstd = H.layer_norm_f8(x, save_stats=True)
    wq, ws, wt, wts = H.quantize_f8(w, block_rows=128, layout="both")
    y = H.gemm_f8_block(h, s, wq, ws, out_f32=True)
    yt, yts = H.quantize_f8(y, layout="cols")
    xt, xts = H.quantize_f8(x, layout="cols")
    dw = H.gemm_f8_block(yt, yts, xt, xts, b_block_rows=1, out_f32=True)
    z = H.gemm_f8_block(*H.quantize_f8(x[:1]), wq, ws, out_f32=True)
    return (y, dw, z) + H.layer_norm_backward(x, x, mean, rstd)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = f()
x.mul_(0.5).add_(1.0)
g.replay()
torch.cuda.synchronize()
for p, q in zip(outs, f()):
    assert torch.equal(p, q)
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
