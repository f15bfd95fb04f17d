"""Plain 64-bit forms of the block-scaled FP8 operators and the layer norm,
written from their definitions, and the error bounds their tests use."""
import numpy as np

F8 = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}   # largest value, mantissa bits, smallest exponent
U = 2.0 ** -24                                             # half a step of FP32, relative
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}         # of a stored result (bf16: 2^-9 of the next power of two)


def cdiv(n, m):
    return -(-n // m)


def round_f8(v, fmt):
    """Round to nearest even onto the format's grid, saturating."""
    top, man, emin = F8[fmt]
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), emin)
    step = np.exp2(e - man)
    return np.copysign(np.minimum(np.rint(a / step) * step, top), v)


def quantize(x, fmt, br, bc):
    """x in br x bc blocks -> (code values, FP32 scales [row blocks, column blocks])."""
    top = F8[fmt][0]
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, -float(np.finfo(np.float32).max), float(np.finfo(np.float32).max)))
    rows, cols = x.shape
    nr, nc = cdiv(rows, br), cdiv(cols, bc)
    pad = np.zeros((nr * br, nc * bc))
    pad[:rows, :cols] = np.abs(x)
    a = np.maximum(pad.reshape(nr, br, nc, bc).max((1, 3)), 2.0 ** -100).astype(np.float32)
    scale = a / np.float32(top)                            # correctly rounded FP32 quotients
    factor = np.float32(top) / a
    f = np.repeat(np.repeat(factor, br, 0), bc, 1)[:rows, :cols].astype(np.float64)
    prod = (x * f).astype(np.float32)                      # exact in 64 bits, then one rounding
    return round_f8(prod, fmt), scale


def dequantize(code, scale, br):
    """Code values times their scales (scale [row blocks, column blocks of 128])."""
    rows, cols = code.shape
    s = np.repeat(np.repeat(scale.astype(np.float64), br, 0), 128, 1)[:rows, :cols]
    return code.astype(np.float64) * s


def gemm(a, sa, b, sb, b_block, bias=None):
    """-> (y, bound on |kernel's FP32 result - y|); a, b code values, sa [M, U] and sb scales per block.

    Bound: the tensor core adds 32 products and the accumulator at a time; aligning
    33 terms to the largest and dropping what lies below FP32 costs at most 33 steps of
    2^-23 of the largest, so 4 x 33 x 2^-23 of a block's sum of magnitudes.  The scale
    product and its application round three times, the sum over blocks (and over at most
    8 parts of K) once per term, the bias once."""
    da, db = dequantize(a, sa, 1), dequantize(b, sb, b_block)
    y = da @ db.T
    mag = np.abs(da) @ np.abs(db).T
    units = sa.shape[1]
    if bias is not None:
        y = y + bias
        mag = mag + np.abs(bias)
    return y, (4 * 33 * 2 + 3 + units + 8 + 1) * U * mag


def stored(bound, y, out):
    """Adds the rounding to the stored type."""
    return bound + HALF_STEP[out] * (np.abs(y) + bound) + 1e-42


def norm(x, gamma, beta, eps):
    """-> (y, mean, rstd, bounds of the three) in 64 bits.

    A row's sums add at most 16 terms in a thread and 10 levels across threads, each
    term once rounded, 2 more for the division: 32 roundings, so the mean is off by at most
    32 u mean|x|, a warp's mean as well.  The sum of squares has a relative error of
    40 u, plus what the means' errors do to (mean_w - mean)."""
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    mean = x.mean(1, keepdims=True)
    d = x - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    e_mean = 32 * U * np.abs(x).mean(1, keepdims=True)
    e_var = 40 * U * var + 4 * np.sqrt(var) * e_mean + 4 * e_mean ** 2
    e_rstd = 0.5 * e_var / (var + eps) + 2 * U             # relative
    xh = d * rstd
    g = 1.0 if gamma is None else np.asarray(gamma, np.float64)
    y = xh * g + (0.0 if beta is None else np.asarray(beta, np.float64))
    e_y = np.abs(g) * (rstd * e_mean + np.abs(xh) * (e_rstd + 3 * U)) * (1 + 1e-3) + 2 * U * np.abs(y)
    return y, mean[:, 0], rstd[:, 0], e_y, e_mean[:, 0] + U * np.abs(mean[:, 0]), (e_rstd * rstd)[:, 0]


def norm_backward(dy, x, mean, rstd, gamma):
    """-> (dx, dgamma, dbeta, bounds of the three), from the given FP32 statistics.

    xh is rounded twice, w once; a row's two sums take 32 roundings as above; a column's
    sum takes one per row of its block (at least 100 blocks run) and at most 64 to join them."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * r
    g = 1.0 if gamma is None else np.asarray(gamma, np.float64)
    w = dy * g
    c1 = w.mean(1, keepdims=True)
    c2 = (w * xh).mean(1, keepdims=True)
    dx = r * (w - c1 - xh * c2)
    a1 = np.abs(w).mean(1, keepdims=True)
    a2 = np.abs(w * xh).mean(1, keepdims=True)
    e_dx = r * (4 * U * np.abs(w) + 38 * U * (a1 + np.abs(xh) * a2) + 4 * U * np.abs(xh * c2)) + U * np.abs(dx)
    k = cdiv(x.shape[0], 100) + 100
    e_dg = (k + 3) * U * np.abs(dy * xh).sum(0)
    e_db = k * U * np.abs(dy).sum(0)
    return dx, (dy * xh).sum(0), dy.sum(0), e_dx, e_dg + 1e-42, e_db + 1e-42


def assert_within(got, want, bound, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.all(np.isfinite(got)), what + ": not finite"
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert i is None or over[i] <= 0, "%s: at %s got %r want %r bound %.3g" % (
        what, tuple(int(k) for k in i), got[i], want[i], bound[i] if np.ndim(bound) else bound)
