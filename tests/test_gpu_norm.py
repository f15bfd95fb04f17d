"""GPU tests of the layer norm's forward and backward pass against plain 64-bit
forms, and of the FP8 layer of norm, quantizer and product as they are used
together."""
import numpy as np
import pytest

from tests import _f8_ref as R
from tests.test_gpu_f8_block import (H, assert_only_view_written, dtype_of, fmt_of, host, on_gpu,  # noqa: F401
                                     poisoned)

pytestmark = pytest.mark.gpu

EPS = 1e-6
SIZES = [(1, 1), (3, 5), (70, 64), (33, 65), (40, 128), (300, 200), (257, 256), (9, 333), (50, 512), (31, 517),
         (17, 1000), (600, 1024), (5, 1025), (700, 1536), (1, 5120), (301, 5120), (4, 8191), (3, 8200), (2, 16384)]


def rows_of(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * rng.lognormal(0, 0.5, (1, cols)) + rng.standard_normal((rows, 1))
    x[:, rng.random(cols) < 0.01] *= 20
    return x


def params(rng, cols, dt):
    import torch
    if dt is None:
        return None, None
    return (torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).to("cuda", dtype_of(dt)),
            torch.from_numpy(0.1 * rng.standard_normal(cols)).to("cuda", dtype_of(dt)))


def num(p):
    return None if p is None else host(p)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward(H, rows, cols, dt):  # noqa: F811
    rng = np.random.default_rng(rows * 31 + cols)
    xd = on_gpu(rows_of(rng, rows, cols), dtype_of(dt))
    for pdt, out in (("f32", "bf16"), ("bf16", "f32"), (None, "bf16")):
        g, b = params(rng, cols, pdt)
        raw, view = poisoned(rows, cols, dtype_of(out))
        y, mean, rstd = H.layer_norm(xd, g, b, EPS, out=view, save_stats=True)
        want, wm, wr, e_y, e_m, e_r = R.norm(host(xd), num(g), num(b), EPS)
        R.assert_within(host(y), want, R.stored(e_y, want, out), "y %s %s" % (pdt, out))
        R.assert_within(host(mean), wm, e_m + 1e-42, "mean")
        R.assert_within(host(rstd), wr, e_r, "rstd")
        assert_only_view_written(raw, view)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_fp8_output_is_the_two_calls(H, rows, cols, dt):  # noqa: F811
    import torch
    rng = np.random.default_rng(rows * 37 + cols)
    xd = on_gpu(rows_of(rng, rows, cols), dtype_of(dt))
    g, b = params(rng, cols, "f32")
    for fmt in ("e4m3", "e5m2"):
        rq, q = poisoned(rows, cols, fmt_of(fmt))
        rs, s = poisoned(R.cdiv(cols, 128), rows, torch.float32)
        _, _, mean, rstd = H.layer_norm_f8(xd, g, b, EPS, fmt_of(fmt), out=(q, s), save_stats=True)
        y, mean2, rstd2 = H.layer_norm(xd, g, b, EPS, out_dtype=torch.float32, save_stats=True)
        q2, s2 = H.quantize_f8(y, fmt_of(fmt))
        assert torch.equal(s, s2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
        assert np.array_equal(host(q), host(q2))
        assert_only_view_written(rq, q)
        assert_only_view_written(rs, s)


@pytest.mark.parametrize("rows,cols", SIZES + [(3001, 96), (2000, 640)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward(H, rows, cols, dt):  # noqa: F811
    import torch
    rng = np.random.default_rng(rows * 41 + cols)
    xd = on_gpu(rows_of(rng, rows, cols), dtype_of(dt))
    dyd = on_gpu(rng.standard_normal((rows, cols)) * rng.lognormal(0, 1, (rows, 1)), dtype_of(dt),
                 ld=R.cdiv(cols, 16) * 16 + 32)
    for pdt in ("f32", "bf16", None):
        g, b = params(rng, cols, pdt)
        _, mean, rstd = H.layer_norm(xd, g, b, EPS, save_stats=True)
        raw, view = poisoned(rows, cols, dtype_of(dt))
        dg, db = torch.full((2, cols), float("nan"), device="cuda")
        H.layer_norm_backward(dyd, xd, mean, rstd, g, out=(view, dg, db))
        want, wg, wb, e_dx, e_dg, e_db = R.norm_backward(host(dyd), host(xd), host(mean), host(rstd), num(g))
        R.assert_within(host(view), want, R.stored(e_dx, want, dt), "dx")
        R.assert_within(host(dg), wg, e_dg, "dgamma")
        R.assert_within(host(db), wb, e_db, "dbeta")
        assert_only_view_written(raw, view)
        # each output alone, and the same again
        dx1, _, _ = H.layer_norm_backward(dyd, xd, mean, rstd, g, out=(poisoned(rows, cols, dtype_of(dt))[1], None, None))
        assert torch.equal(dx1, view)
        _, dg1, none = H.layer_norm_backward(dyd, xd, mean, rstd, g, out=(None, torch.empty_like(dg), None))
        assert none is None and torch.equal(dg1, dg)
        _, _, db1 = H.layer_norm_backward(dyd, xd, mean, rstd, g, out=(None, None, torch.empty_like(db)))
        assert torch.equal(db1, db)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_row_width_class(H, dt):  # noqa: F811
    """Each number of warps that a row is spread over, forward, FP8 forward and backward."""
    import torch
    rng = np.random.default_rng(14)
    for cols in list(range(72, 1025, 136)) + list(range(1032, 16385, 512)) + list(range(1536, 16385, 512)) + [5954]:
        x = on_gpu(rng.standard_normal((3, cols)), dtype_of(dt))
        dy = on_gpu(rng.standard_normal((3, cols)), dtype_of(dt))
        g, b = params(rng, cols, "f32")
        y, mean, rstd = H.layer_norm(x, g, b, EPS, out_dtype=torch.float32, save_stats=True)
        want, wm, wr, e_y, e_m, e_r = R.norm(host(x), num(g), num(b), EPS)
        R.assert_within(host(y), want, R.stored(e_y, want, "f32"), "y %d" % cols)
        q, s = H.layer_norm_f8(x, g, b, EPS)
        q2, s2 = H.quantize_f8(on_gpu(host(y), torch.float32))
        assert torch.equal(s, s2) and np.array_equal(host(q), host(q2)), cols
        dx, dg, db = H.layer_norm_backward(dy, x, mean, rstd, g)
        want, wg, wb, e_dx, e_dg, e_db = R.norm_backward(host(dy), host(x), host(mean), host(rstd), num(g))
        R.assert_within(host(dx), want, R.stored(e_dx, want, dt), "dx %d" % cols)
        R.assert_within(host(dg), wg, e_dg, "dgamma %d" % cols)
        R.assert_within(host(db), wb, e_db, "dbeta %d" % cols)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [3, 8, 60, 264, 517, 1300, 2880, 5112, 5121, 8200])
def test_backward_of_rows_of_one_large_value(H, cols, dt):  # noqa: F811
    """mean * rstd past the largest finite number: nothing of what lies past a row reaches its sums."""
    import torch
    rng = np.random.default_rng(cols)
    x = on_gpu(np.full((5, cols), 2.0 ** 119), dtype_of(dt))
    dy = on_gpu(rng.standard_normal((5, cols)), dtype_of(dt))
    g, _ = params(rng, cols, "f32")
    mean, rstd = torch.full((5,), 2.0 ** 119, device="cuda"), torch.full((5,), 1024.0, device="cuda")
    dx, dg, db = H.layer_norm_backward(dy, x, mean, rstd, g)
    want, wg, wb, e_dx, e_dg, e_db = R.norm_backward(host(dy), host(x), host(mean), host(rstd), num(g))
    R.assert_within(host(dx), want, R.stored(e_dx, want, dt), "dx")
    R.assert_within(host(dg), wg, e_dg, "dgamma")
    R.assert_within(host(db), wb, e_db, "dbeta")


@pytest.mark.parametrize("cols", [24, 200, 1300])
def test_gradients_against_differences(H, cols):  # noqa: F811
    """Directional derivatives of L = sum(c y) by central differences of the 64-bit form."""
    rng = np.random.default_rng(cols)
    rows, eps = 6, 1e-3
    x, c = rows_of(rng, rows, cols), rng.standard_normal((rows, cols))
    xd, cd = on_gpu(x, dtype_of("f32")), on_gpu(c, dtype_of("f32"))
    x, c = host(xd), host(cd)
    g, b = params(rng, cols, "f32")
    gn, bn = num(g), num(b)
    _, mean, rstd = H.layer_norm(xd, g, b, eps, save_stats=True)
    dx, dg, db = (host(t) for t in H.layer_norm_backward(cd, xd, mean, rstd, g))

    def loss(x_, g_, b_):
        return float((c * R.norm(x_, g_, b_, eps)[0]).sum())
    h = 1e-5
    vx, vp = rng.standard_normal((rows, cols)), rng.standard_normal(cols)
    # central differences: truncation h^2 L''' / 6, cancellation 2^-52 |L| / h; FP32 gradients: 1e-5 of their size
    for got, num_d, size in (
            ((dx * vx).sum(), (loss(x + h * vx, gn, bn) - loss(x - h * vx, gn, bn)) / (2 * h), np.abs(dx * vx).sum()),
            ((dg * vp).sum(), (loss(x, gn + h * vp, bn) - loss(x, gn - h * vp, bn)) / (2 * h), np.abs(dg * vp).sum()),
            ((db * vp).sum(), (loss(x, gn, bn + h * vp) - loss(x, gn, bn - h * vp)) / (2 * h), np.abs(db * vp).sum())):
        assert abs(got - num_d) <= 2e-5 * size, (got, num_d, size)


def test_far_from_zero_and_constant_rows(H):  # noqa: F811
    """A large common offset costs the accuracy that the offset's own rounding costs, no more; a constant
    row has variance 0; one enormous element does not spoil the variance of the others' sum."""
    import torch
    rng = np.random.default_rng(5)
    for cols in (60, 700, 5120):
        x = rng.standard_normal((4, cols))
        x[0] += 1000.0
        x[1] = 3.25
        x[2, 0] = 1e4
        xd = on_gpu(x, torch.float32)
        y, mean, rstd = H.layer_norm(xd, None, None, EPS, save_stats=True)
        want, wm, wr, e_y, e_m, e_r = R.norm(host(xd), None, None, EPS)
        R.assert_within(host(y), want, R.stored(e_y, want, "f32"), "y")
        R.assert_within(host(rstd), wr, e_r, "rstd")


def test_nonfinite_rows_stay_their_own(H):  # noqa: F811
    import torch
    from block_floating_point_hif4_b200 import binding as B
    rng = np.random.default_rng(6)
    for cols in (48, 300, 2000):
        xd = on_gpu(rows_of(rng, 40, cols), torch.bfloat16)
        clean = H.layer_norm(xd, None, None, EPS)
        xd[7, 3] = float("nan")
        xd[9, 0] = float("inf")
        y = H.layer_norm(xd, None, None, EPS)
        keep = [i for i in range(40) if i not in (7, 9)]
        assert torch.equal(y[keep], clean[keep])
        assert torch.all(torch.isnan(y[7])) and torch.all(torch.isnan(y[9]))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, s = H.layer_norm_f8(xd, None, None, EPS, status=st)
        assert H.get_status(st) == B.ERR_NONFINITE
        assert torch.all(q[7].float() == 0) and torch.all(q[9].float() == 0)


def test_in_place(H):  # noqa: F811
    import torch
    rng = np.random.default_rng(9)
    for rows, cols in ((700, 96), (700, 640), (900, 2000), (400, 6000)):
        for dt in ("bf16", "f32"):
            x = on_gpu(rows_of(rng, rows, cols), dtype_of(dt))
            dy = on_gpu(rng.standard_normal((rows, cols)), dtype_of(dt))
            g, b = params(rng, cols, "f32")
            y, mean, rstd = H.layer_norm(x, g, b, EPS, save_stats=True)
            dx, dg, db = H.layer_norm_backward(dy, x, mean, rstd, g)
            for t in (x, dy):
                c = [u.clone(memory_format=torch.preserve_format) for u in (x, dy)]
                c = [torch.empty(rows, x.stride(0), dtype=x.dtype, device="cuda")[:, :cols].copy_(u) for u in c]
                o = H.layer_norm_backward(c[1], c[0], mean, rstd, g, out=(c[0] if t is x else c[1], dg, db))
                assert torch.equal(o[0], dx)
            assert H.layer_norm(x, g, b, EPS, out=x) is x
            assert torch.equal(x, y)


def test_no_rows(H):  # noqa: F811
    import torch
    x = torch.empty(0, 320, device="cuda")
    st = torch.empty(0, device="cuda")
    assert H.layer_norm(x).shape == (0, 320)
    assert H.layer_norm_f8(x)[0].shape == (0, 320)
    dx, dg, db = H.layer_norm_backward(x, x, st, st)
    assert dx.shape == (0, 320) and not dg.any() and not db.any()


def test_refusals_of_the_binding(H):  # noqa: F811
    import torch
    x = torch.zeros(4, 256, device="cuda")
    g = torch.ones(256, device="cuda")
    _, mean, rstd = H.layer_norm(x, save_stats=True)
    with pytest.raises(ValueError):
        H.layer_norm(x, g[:255])
    with pytest.raises(ValueError):
        H.layer_norm(x, g, g.bfloat16())
    with pytest.raises(ValueError):
        H.layer_norm(x.double())
    with pytest.raises(ValueError):
        H.layer_norm(x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        H.layer_norm(x, out=torch.empty(4, 255, device="cuda"))
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(H.Hif4Error):
            H.layer_norm(x, eps=eps)
    with pytest.raises(H.Hif4Error):
        H.layer_norm(torch.zeros(2, 16448, device="cuda"))
    with pytest.raises(H.Hif4Error):
        H.layer_norm(torch.zeros(4, 255, device="cuda"))    # rows not 16-byte aligned
    with pytest.raises(ValueError):
        H.layer_norm_backward(x.bfloat16(), x, mean, rstd)
    with pytest.raises(ValueError):
        H.layer_norm_backward(x, x, mean[:3], rstd)
    with pytest.raises(ValueError):
        H.layer_norm_backward(x, x, None, rstd)
    with pytest.raises(H.Hif4Error):
        H.layer_norm_backward(x, x, mean, rstd, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(H.Hif4Error):
        H.layer_norm_backward(x, x, mean, rstd, out=(None, None, None))


# ------------------------------------------------------------- as they are used together

def layer(H, x, dy, g, b, w):  # noqa: F811
    """norm -> FP8 linear and its backward pass: (y, dx, dgamma, dbeta, dw) and the operands between."""
    xq, xs, mean, rstd = H.layer_norm_f8(x, g, b, EPS, save_stats=True)
    wq, ws, wtq, wts = H.quantize_f8(w, block_rows=128, layout="both")
    y = H.gemm_f8_block(xq, xs, wq, ws)
    h = H.layer_norm(x, g, b, EPS)
    htq, hts = H.quantize_f8(h, layout="cols")
    dq, ds, dtq, dts = H.quantize_f8(dy, fmt_of("e5m2"), layout="both")
    dh = H.gemm_f8_block(dq, ds, wtq, wts)
    dw = H.gemm_f8_block(dtq, dts, htq, hts, b_block_rows=1, out_f32=True)
    dx, dg, db = H.layer_norm_backward(dh, x, mean, rstd, g)
    return (y, dx, dg, db, dw), (xq, xs, wq, ws, dq, ds, wtq, wts, dtq, dts, htq, hts, dh, mean, rstd)


def layer_inputs(T=333, D=320, N=456):
    rng = np.random.default_rng(8)
    x = on_gpu(rows_of(rng, T, D), dtype_of("bf16"))
    dy = on_gpu(rng.standard_normal((T, N)) * 1e-3, dtype_of("bf16"))
    g, b = params(rng, D, "f32")
    w = on_gpu(rng.standard_normal((N, D)) / np.sqrt(D), dtype_of("bf16"))
    return x, dy, g, b, w


def test_layer_forward_and_backward(H):  # noqa: F811
    x, dy, g, b, w = layer_inputs()
    (y, dx, dg, db, dw), mid = layer(H, x, dy, g, b, w)
    xq, xs, wq, ws, dq, ds, wtq, wts, dtq, dts, htq, hts, dh, mean, rstd = mid
    # every product against the definition on its own operands
    for got, a, sa, bb, sb, blk, out in ((y, xq, xs, wq, ws, 128, "bf16"), (dh, dq, ds, wtq, wts, 128, "bf16"),
                                         (dw, dtq, dts, htq, hts, 1, "f32")):
        sbv = sb.cpu().numpy()
        want, bound = R.gemm(host(a), sa.cpu().numpy().T, host(bb), sbv.T if blk == 1 else sbv, blk)
        R.assert_within(host(got), want, R.stored(bound, want, out), "product")
    want, wg, wb, e_dx, e_dg, e_db = R.norm_backward(host(dh), host(x), host(mean), host(rstd), host(g))
    R.assert_within(host(dx), want, R.stored(e_dx, want, "bf16"), "dx")
    R.assert_within(host(dg), wg, e_dg, "dgamma")
    R.assert_within(host(db), wb, e_db, "dbeta")
    # and the whole layer against the unquantized one: E4M3 operands are off by at most 2^-4 of each value
    # (independent roundings, so a small part of that in the sum), E5M2 by 2^-3
    h64, _, _, _, _, _ = R.norm(host(x), host(g), host(b), EPS)
    y64 = h64 @ host(w).T
    assert np.linalg.norm(host(y) - y64) <= 2 * 2.0 ** -4 * np.linalg.norm(y64)
    dw64 = host(dy).T @ h64
    assert np.linalg.norm(host(dw) - dw64) <= (2.0 ** -4 + 2.0 ** -3) * np.linalg.norm(dw64)


def test_layer_captured_and_replayed_on_new_inputs(H):  # noqa: F811
    import torch
    x, dy, g, b, w = layer_inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(H, x, dy, g, b, w)                            # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, _ = layer(H, x, dy, g, b, w)
    x.mul_(-1.5)
    dy.add_(dy.flip(0))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    eager, _ = layer(H, x, dy, g, b, w)
    for got, want in zip(outs, eager):
        assert torch.equal(got, want)


def test_pairs_captured_and_replayed(H):  # noqa: F811
    """The products that run on CTA pairs, several in one graph, each replay on new operands."""
    import torch
    rng = np.random.default_rng(10)
    x = on_gpu(rng.standard_normal((900, 1100)), dtype_of("bf16"))
    w = on_gpu(rng.standard_normal((3600, 1100)), dtype_of("bf16"))
    wq, ws = H.quantize_f8(w, block_rows=128)

    def chain():
        q, s = H.quantize_f8(x)
        y = H.gemm_f8_block(q, s, wq, ws)
        return y, H.gemm_f8_block(*H.quantize_f8(y[:700, :1100]), wq, ws, out_f32=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain()
    for _ in range(3):
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, chain()):
            assert torch.equal(got, want)


def test_layer_on_two_streams_at_once(H):  # noqa: F811
    import torch
    x, dy, g, b, w = layer_inputs()
    want, _ = layer(H, x, dy, g, b, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(layer(H, x, dy, g, b, w)[0])
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, want))
    # a stream that is not current: what the call allocates belongs to it
    s = streams[0]
    y = H.layer_norm(x, g, b, EPS, stream=s)
    dx = H.quantize_f8(x, stream=s)
    s.synchronize()
    assert torch.equal(y, H.layer_norm(x, g, b, EPS)) and torch.equal(dx[1], H.quantize_f8(x)[1])
