"""What is measured of the block-scaled FP8 operators and the layer norm.

Four operators: the FP8 quantizer with one scale per block of 128, the matrix
product that reads its output, the layer norm (plain or with FP8 output) and
the layer norm's backward pass.  Every case is a plain dict; ``prepare`` makes
its inputs on the GPU, ``run`` makes one pass, ``exact`` gives the result in 64
bits.  With ``own`` false ``run`` computes the operators from elementary torch
operations, otherwise it calls the framework.

Layouts (those of the library): matrices are row-major with leading dimensions
of a multiple of 16 bytes; the scales of 1 x 128 blocks are block-major,
[ceil(cols/128), rows] with a leading dimension of a multiple of 4; the scales
of 128 x 128 blocks are [ceil(rows/128), ceil(cols/128)].
"""
import math

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
FMT = {"e4m3": E4M3, "e5m2": E5M2}
TOP = {E4M3: 448.0, E5M2: 57344.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -100                # smallest block maximum the scale is formed from
BLOCK = 128
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # -- quantizer
        # the video tokens that enter one linear of a 14B-class DiT block (57600 = 16 frames of 3600)
        dict(name="quant_acts_57600x5120", op="quantize", rows=57600, cols=5120, dt="bf16", fmt="e4m3", block=1,
             layout="rows"),
        # an output gradient, needed row-wise for the input's gradient and transposed for the weight's;
        # one frame and a partial one, so that the last token block is ragged
        dict(name="quant_grad_both_3651x5120", op="quantize", rows=3651, cols=5120, dt="bf16", fmt="e5m2", block=1,
             layout="both"),
        # an FFN weight, laid out once for the forward and once for the input-gradient product
        dict(name="quant_weight_13824x5120", op="quantize", rows=13824, cols=5120, dt="bf16", fmt="e4m3", block=128,
             layout="both"),
        # -- matrix product
        # the first FFN linear over all video tokens
        dict(name="gemm_57600x13824x5120", op="gemm", M=57600, N=13824, K=5120, a="e4m3", b="e4m3", block=128,
             out="bf16", bias=True),
        # the same linear for a single token: the weight is read once
        dict(name="gemm_1x13824x5120", op="gemm", M=1, N=13824, K=5120, a="e4m3", b="e4m3", block=128, out="bf16",
             bias=True),
        # the second FFN linear for a prompt of 512 text tokens
        dict(name="gemm_512x5120x13824", op="gemm", M=512, N=5120, K=13824, a="e4m3", b="e4m3", block=128,
             out="bf16", bias=False),
        # the gradient of a 5120 x 5120 projection over 14391 tokens (a ragged last block): E5M2
        # gradients, 1 x 128 blocks along the tokens on both sides, FP32 out
        dict(name="gemm_wgrad_5120x5120x14391", op="gemm", M=5120, N=5120, K=14391, a="e5m2", b="e4m3", block=1,
             out="f32", bias=False),
        # -- layer norm
        # the norm before a linear, over all video tokens
        dict(name="norm_57600x5120", op="norm", rows=57600, cols=5120, dt="bf16", param="f32", out="bf16",
             stats=True),
        # one frame's tokens, normalised straight into the FP8 product's operand
        dict(name="norm_f8_3600x5120", op="norm", rows=3600, cols=5120, dt="bf16", param="f32", out="e4m3",
             stats=False),
        # a single token
        dict(name="norm_1x5120", op="norm", rows=1, cols=5120, dt="bf16", param="bf16", out="bf16", stats=False),
        # -- layer norm, backward
        dict(name="norm_bwd_57600x5120", op="norm_bwd", rows=57600, cols=5120, dt="bf16", param="f32"),
        # a head-sized FP32 norm over a ragged batch
        dict(name="norm_bwd_4099x517", op="norm_bwd", rows=4099, cols=517, dt="f32", param="f32"),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; every other one rounded to a multiple of 64 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "norm", "norm_bwd"])
    if op == "quantize":
        return dict(op=op, rows=_size(rng, 1, 16384), cols=_size(rng, 32, 13824), dt=rng.choice(["bf16", "f32"]),
                    fmt=rng.choice(["e4m3", "e5m2"]), block=rng.choice([1, 128]),
                    layout=rng.choice(["rows", "cols", "both"]))
    if op == "gemm":
        block = rng.choice([1, 128])
        return dict(op=op, M=_size(rng, 1, 16384), N=_size(rng, 32, 13824), K=_size(rng, 64, 13824),
                    a=rng.choice(["e4m3", "e5m2"]), b=rng.choice(["e4m3", "e5m2"]), block=block,
                    out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    if op == "norm":
        return dict(op=op, rows=_size(rng, 1, 32768), cols=_size(rng, 32, 8192), dt=rng.choice(["bf16", "f32"]),
                    param=rng.choice(["none", "bf16", "f32"]), out=rng.choice(["bf16", "f32", "e4m3", "e5m2"]),
                    stats=rng.random() < 0.5)
    return dict(op=op, rows=_size(rng, 1, 32768), cols=_size(rng, 32, 8192), dt=rng.choice(["bf16", "f32"]),
                param=rng.choice(["none", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _up(n, m):
    return -(-n // m) * m


def _blocks(n):
    return -(-n // BLOCK)


def _matrix(g, rows, cols, dtype, sigma=1.0, outliers=True):
    """rows x cols of N(0, 1) times a log-normal scale per column, 1 % of the columns 20 times larger, in
    a buffer whose leading dimension is a multiple of 16 bytes."""
    dev = g.device
    ld = _up(cols, 16)
    col = torch.exp(0.5 * torch.randn(ld, generator=g, device=dev)) * sigma
    if outliers:
        col = torch.where(torch.rand(ld, generator=g, device=dev) < 0.01, col * 20.0, col)
    buf = torch.empty(rows, ld, dtype=dtype, device=dev)
    step = max(1, (1 << 27) // ld)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        buf[r:r + n] = (torch.randn(n, ld, generator=g, device=dev) * col).to(dtype)
    return buf[:, :cols]


def _gradient(g, rows, cols, dtype):
    """An output gradient: small, its size differing from token to token."""
    buf = _matrix(g, rows, cols, torch.float32, 1e-4, outliers=False)
    return _pad_copy(buf * torch.exp(torch.randn(rows, 1, generator=g, device=g.device)), dtype)


def _pad_copy(x, dtype):
    out = torch.zeros(x.shape[0], _up(x.shape[1], 16), dtype=dtype, device=x.device)
    out[:, :x.shape[1]] = x.to(dtype)
    return out[:, :x.shape[1]]


def _pad_scale(s):
    out = torch.zeros(s.shape[0], _up(s.shape[1], 4), dtype=torch.float32, device=s.device)
    out[:, :s.shape[1]] = s
    return out[:, :s.shape[1]]


def _operand(g, rows, cols, fmt, block, sigma):
    """An FP8 operand with its scales, as a quantizer leaves them."""
    x = _matrix(g, rows, cols, torch.bfloat16, sigma)
    step = BLOCK * max(1, (1 << 27) // (BLOCK * _up(cols, BLOCK)))
    q = torch.zeros(rows, _up(cols, 16), dtype=torch.uint8, device=g.device).view(fmt)[:, :cols]
    scales = []
    for r in range(0, rows, step):
        qc, sc = _quantize_rows(x[r:r + step], fmt) if block == 1 else _quantize_tiles(x[r:r + step], fmt)
        q[r:r + step] = qc
        scales.append(sc)
    return q, _pad_scale(torch.cat(scales, 1 if block == 1 else 0))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed + 1) + 7)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        dt = DT[case["dt"]]
        st["x"] = (_gradient(g, case["rows"], case["cols"], dt) if case["fmt"] == "e5m2" else
                   _matrix(g, case["rows"], case["cols"], dt))
    elif op == "gemm":
        st["a"], st["sa"] = _operand(g, case["M"], case["K"], FMT[case["a"]], 1, 1.0)
        st["b"], st["sb"] = _operand(g, case["N"], case["K"], FMT[case["b"]], case["block"], 0.015)
        st["bias"] = (torch.randn(case["N"], generator=g, device="cuda") * 0.01).to(torch.bfloat16) \
            if case["bias"] else None
    else:
        rows, cols = case["rows"], case["cols"]
        dt = DT[case["dt"]]
        x = _matrix(g, rows, cols, torch.float32)
        st["x"] = _pad_copy(x + 0.5 * torch.randn(rows, 1, generator=g, device="cuda"), dt)
        st["gamma"] = st["beta"] = None
        if case["param"] != "none":
            pt = DT[case["param"]]
            st["gamma"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(pt)
            st["beta"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(pt)
        if op == "norm_bwd":
            st["dy"] = _gradient(g, rows, cols, dt)
            xd = st["x"].float()
            var, mean = torch.var_mean(xd, 1, correction=0)
            st["mean"], st["rstd"] = mean, torch.rsqrt(var + EPS)
    torch.cuda.synchronize()
    return st


# ------------------------------------------------------------------ plain forms (32 bits)

def _grouped(x):
    """x in FP32 as [rows, blocks, 128], the last block padded with zeros."""
    rows, cols = x.shape
    nb = _blocks(cols)
    xf = x.float()
    if nb * BLOCK != cols:
        xf = torch.cat([xf, xf.new_zeros(rows, nb * BLOCK - cols)], 1)
    return xf.reshape(rows, nb, BLOCK)


def _scale_pair(top, fmt):
    """(scale top/F, factor F/top), each one correctly rounded FP32 quotient (a Python number as an operand
    would turn the quotient into a product with a rounded reciprocal)."""
    f = torch.full_like(top, TOP[fmt])
    return top / f, f / top


def _quantize_rows(x, fmt):
    """1 x 128 blocks -> (codes [rows, cols], scales [blocks, rows])."""
    xg = _grouped(x)
    top = torch.clamp(xg.abs().amax(2), min=TINY)
    scale, factor = _scale_pair(top, fmt)
    q = (xg * factor[:, :, None]).to(fmt)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]], scale.t()


def _quantize_tiles(x, fmt):
    """128 x 128 blocks -> (codes [rows, cols], scales [row blocks, column blocks])."""
    rows, cols = x.shape
    xg = _grouped(x)
    nr = _blocks(rows)
    rmax = xg.abs().amax(2)
    if nr * BLOCK != rows:
        rmax = torch.cat([rmax, rmax.new_zeros(nr * BLOCK - rows, rmax.shape[1])], 0)
    top = torch.clamp(rmax.reshape(nr, BLOCK, -1).amax(1), min=TINY)
    scale, factor = _scale_pair(top, fmt)
    q = (xg * factor.repeat_interleave(BLOCK, 0)[:rows, :, None]).to(fmt)
    return q.reshape(rows, -1)[:, :cols], scale


def _plain_quantize(x, fmt, block, layout):
    out = []
    if layout in ("rows", "both"):
        out += list(_quantize_rows(x, fmt) if block == 1 else _quantize_tiles(x, fmt))
    if layout in ("cols", "both"):
        if block == 1:
            out += list(_quantize_rows(x.t(), fmt))
        else:
            q, s = _quantize_tiles(x, fmt)
            out += [q.t().contiguous(), s.t()]
    return out


def _dequantize(q, s, block):
    rows, cols = q.shape
    per_row = s.t() if block == 1 else s.repeat_interleave(BLOCK, 0)[:rows]
    return q.float() * per_row.repeat_interleave(BLOCK, 1)[:, :cols]


def _plain_gemm(a, sa, b, sb, bias, block, out):
    y = _dequantize(a, sa, 1) @ _dequantize(b, sb, block).t()
    if bias is not None:
        y = y + bias.float()
    return y.to(out)


def _plain_norm(x, gamma, beta):
    xf = x.float()
    mean = xf.mean(1, keepdim=True)
    d = xf - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd
    if gamma is not None:
        y = y * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return y, mean[:, 0], rstd[:, 0]


def _plain_norm_bwd(dy, x, mean, rstd, gamma):
    d = dy.float()
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    w = d if gamma is None else d * gamma.float()
    c1 = w.mean(1, keepdim=True)
    c2 = (w * xh).mean(1, keepdim=True)
    dx = (rstd[:, None] * (w - c1 - xh * c2)).to(x.dtype)
    return dx, (d * xh).sum(0), d.sum(0)


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import block_floating_point_hif4_b200 as H
        if op == "quantize":
            return H.quantize_f8(st["x"], FMT[case["fmt"]], block_rows=case["block"], layout=case["layout"])
        if op == "gemm":
            return H.gemm_f8_block(st["a"], st["sa"], st["b"], st["sb"], st["bias"], b_block_rows=case["block"],
                                   out_f32=case["out"] == "f32")
        if op == "norm":
            if case["out"] in FMT:
                return H.layer_norm_f8(st["x"], st["gamma"], st["beta"], EPS, FMT[case["out"]],
                                       save_stats=case["stats"])
            return H.layer_norm(st["x"], st["gamma"], st["beta"], EPS, out_dtype=DT[case["out"]],
                                save_stats=case["stats"])
        return H.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"])
    if op == "quantize":
        return tuple(_plain_quantize(st["x"], FMT[case["fmt"]], case["block"], case["layout"]))
    if op == "gemm":
        return _plain_gemm(st["a"], st["sa"], st["b"], st["sb"], st["bias"], case["block"], DT[case["out"]])
    if op == "norm":
        y, mean, rstd = _plain_norm(st["x"], st["gamma"], st["beta"])
        out = list(_quantize_rows(y, FMT[case["out"]])) if case["out"] in FMT else [y.to(DT[case["out"]])]
        if case["stats"]:
            out += [mean, rstd]
        return tuple(out) if len(out) > 1 else out[0]
    return _plain_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"])


# ------------------------------------------------------------------ 64 bits

def _codes64(x, inv, fmt):
    """The codes' definition: the value times the block's FP32 factor, rounded to FP32 (the product of two
    FP32 numbers is exact in 64 bits), then to the 8-bit format."""
    return (x * inv).float().to(fmt)


def _block_max64(x, br, bc):
    """Maxima of |x| over br x bc blocks, block by block."""
    rows, cols = x.shape
    out = torch.empty(-(-rows // br), -(-cols // bc), dtype=torch.float64, device=x.device)
    for j in range(out.shape[1]):
        m = x[:, j * bc:(j + 1) * bc].abs().amax(1)
        if br == 1:
            out[:, j] = m
        else:
            for i in range(out.shape[0]):
                out[i, j] = m[i * br:(i + 1) * br].amax()
    return out.clamp(min=TINY)


def _quantize64(x, fmt, br, bc):
    """x [rows, cols] (64 bits) in br x bc blocks -> (codes, scales [row blocks, column blocks])."""
    top = _block_max64(x, br, bc)
    inv = (TOP[fmt] / top).float().double()
    q = torch.empty(x.shape, dtype=fmt, device=x.device)
    for j in range(top.shape[1]):
        f = inv[:, j].repeat_interleave(br)[:x.shape[0], None]
        q[:, j * bc:(j + 1) * bc] = _codes64(x[:, j * bc:(j + 1) * bc], f, fmt)
    return q, top / TOP[fmt]


def _exact_quantize(st, case):
    x, fmt = st["x"].double(), FMT[case["fmt"]]
    out = []
    if case["block"] == 128:
        q, s = _quantize64(x, fmt, 128, 128)
        if case["layout"] != "cols":
            out += [q, s]
        if case["layout"] != "rows":
            out += [q.t().contiguous(), s.t()]
        return tuple(out)
    if case["layout"] != "cols":
        q, s = _quantize64(x, fmt, 1, 128)
        out += [q, s.t()]
    if case["layout"] != "rows":
        q, s = _quantize64(x.t(), fmt, 1, 128)
        out += [q, s.t()]
    return tuple(out)


def _exact_gemm(st, case):
    M, N, K = case["M"], case["N"], case["K"]
    b = st["b"].double()
    for u in range(_blocks(K)):
        k = slice(u * BLOCK, min(K, (u + 1) * BLOCK))
        if case["block"] == 1:
            b[:, k] *= st["sb"][u].double()[:, None]
        else:
            for j in range(_blocks(N)):
                b[j * BLOCK:(j + 1) * BLOCK, k] *= st["sb"][j, u].double()
    y = torch.empty(M, N, dtype=torch.float64, device=b.device)
    for r in range(0, M, 8192):
        a = st["a"][r:r + 8192].double()
        for u in range(_blocks(K)):
            a[:, u * BLOCK:(u + 1) * BLOCK] *= st["sa"][u, r:r + 8192].double()[:, None]
        y[r:r + 8192] = a @ b.t()
    if st["bias"] is not None:
        y += st["bias"].double()
    return y


def _exact_norm(st, case):
    x = st["x"].double()
    n = x.shape[1]
    mean = x.sum(1) / n
    x -= mean[:, None]
    rstd = 1.0 / torch.sqrt((x ** 2).sum(1) / n + EPS)
    x *= rstd[:, None]
    if st["gamma"] is not None:
        x *= st["gamma"].double()
    if st["beta"] is not None:
        x += st["beta"].double()
    if case["out"] in FMT:
        q, s = _quantize64(x, FMT[case["out"]], 1, 128)
        out = [q, s.t()]
    else:
        out = [x]
    if case["stats"]:
        out += [mean, rstd]
    return tuple(out) if len(out) > 1 else out[0]


def _exact_norm_bwd(st, case):
    rows, n = st["x"].shape
    dev = st["x"].device
    dx = torch.empty(rows, n, dtype=torch.float64, device=dev)
    dg = torch.zeros(n, dtype=torch.float64, device=dev)
    db = torch.zeros(n, dtype=torch.float64, device=dev)
    for r in range(0, rows, 8192):
        s = slice(r, min(rows, r + 8192))
        dy = st["dy"][s].double()
        xh = (st["x"][s].double() - st["mean"][s].double()[:, None]) * st["rstd"][s].double()[:, None]
        dg += (dy * xh).sum(0)
        db += dy.sum(0)
        if st["gamma"] is not None:
            dy *= st["gamma"].double()
        dot = (dy * xh).sum(1, keepdim=True) / n
        dx[s] = (dy - dy.sum(1, keepdim=True) / n - xh * dot) * st["rstd"][s].double()[:, None]
    return dx, dg, db


def exact(case, seed):
    st = prepare(case, seed)
    return {"quantize": _exact_quantize, "gemm": _exact_gemm, "norm": _exact_norm,
            "norm_bwd": _exact_norm_bwd}[case["op"]](st, case)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        row_scales = rows * _blocks(cols) if case["block"] == 1 else _blocks(rows) * _blocks(cols)
        col_scales = cols * _blocks(rows) if case["block"] == 1 else row_scales
        b = n * (2 if case["dt"] == "bf16" else 4)
        b += (n + 4 * row_scales) * (case["layout"] != "cols") + (n + 4 * col_scales) * (case["layout"] != "rows")
        return {"bytes": b, "flops": 3 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        sb = N * _blocks(K) if case["block"] == 1 else _blocks(N) * _blocks(K)
        y = M * N * (2 if case["out"] == "bf16" else 4)
        return {"bytes": M * K + N * K + 4 * (M * _blocks(K) + sb) + y + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    n = case["rows"] * case["cols"]
    size = 2 if case["dt"] == "bf16" else 4
    par = {"none": 0, "bf16": 2, "f32": 4}[case["param"]] * case["cols"]
    if op == "norm":
        out = {"bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}[case["out"]] * n
        if case["out"] in FMT:
            out += 4 * case["rows"] * _blocks(case["cols"])
        return {"bytes": n * size + out + 2 * par + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
    return {"bytes": 3 * n * size + par + 8 * case["cols"] + 8 * case["rows"], "flops": 14 * n}
