"""Cases of the MXFP4 linear layer and of the orthogonalised weight update, in their plain form and through the library.

An MXFP4 matrix [rows, K] holds e2m1 codes (two a byte, the lower k in the lower
four bits) and one E8M0 scale per 32 consecutive k of a row.  For a block with
largest magnitude amax > 0 the scale is 2^s, s = max(floor(log2 amax) - 2, -127)
(1 for a block of zeros), and an element is x / 2^s rounded to the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, larger values to 6).  K is
padded with zeros to a multiple of 32.

Operators (`op` of a case):
  quantize   x [rows, K] -> its MXFP4 form, along K and, with both, along the
             rows of x (the form of x^T); returned as the values they stand for
  product    C = A B^T of two MXFP4 matrices
  linear     y = Q(x) W^T, x in bfloat16, W in MXFP4
  backward   the gradients of y = Q(x) W^T: dx = Q(dy) W and dw = Q(dy^T) x,
             from W^T and x^T in MXFP4
  orth       the update direction of a matrix: 5 steps X <- a X + (b A + c A A) X,
             A = X X^T, from X = G / |G| (on G^T where G is tall)
"""
import math

import torch

own = False

STEPS, COEFFS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


def pad32(k):
    return -(-k // 32) * 32


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # the activation of one token, quantised before its products: latency
        dict(name="quantize-token", op="quantize", rows=1, K=4096, dtype="bf16", both=False),
        # an MLP weight requantised after an optimizer step from its fp32 master
        # copy, for the forward product and (transposed) for the input gradient
        dict(name="quantize-weight", op="quantize", rows=14336, K=4096, dtype="fp32", both=True),
        # one 256 x 256 tile: latency
        dict(name="product-256", op="product", M=256, N=256, K=256),
        # odd and ragged sizes, a partial K step
        dict(name="product-ragged", op="product", M=1111, N=2777, K=1184),
        # an MLP projection over a long prompt
        dict(name="product-mlp", op="product", M=16384, N=14336, K=4096),
        # decoding: one token through an MLP projection, bound by reading W
        dict(name="linear-token", op="linear", M=1, N=14336, K=4096),
        # decoding a batch of 16 sequences
        dict(name="linear-batch", op="linear", M=16, N=8192, K=8192),
        # a short prompt or a batch of drafts, on the MLP's way down
        dict(name="linear-prompt", op="linear", M=100, N=4096, K=14336),
        # a training step's gradients, small and odd
        dict(name="backward-small", op="backward", M=500, N=1000, K=768),
        # a training step's gradients of an MLP projection
        dict(name="backward-mlp", op="backward", M=8192, N=14336, K=4096),
        # the update of a small matrix (a router, a low-rank factor): latency
        dict(name="orth-256", op="orth", rows=256, K=256, dtype="fp32"),
        # the update of an MLP weight
        dict(name="orth-mlp", op="orth", rows=14336, K=4096, dtype="bf16"),
    ]


def draw(rng):
    def size(lo, hi):   # spread over the logarithm; every second one a multiple of 64
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v

    op = rng.choice(["quantize", "product", "linear", "backward", "orth"])
    while True:
        if op == "quantize":
            c = dict(op=op, rows=size(1, 16384), K=size(32, 14336), dtype=rng.choice(["bf16", "fp32"]),
                     both=rng.random() < 0.5)
            if c["rows"] * c["K"] <= 14336 * 4096:
                return c
        elif op == "product":
            c = dict(op=op, M=size(1, 16384), N=size(64, 16384), K=pad32(size(32, 16384)))
            if c["M"] * c["N"] * c["K"] <= 16384 * 14336 * 4096:
                return c
        elif op == "linear":
            return dict(op=op, M=size(1, 256), N=size(64, 16384), K=size(64, 16384))
        elif op == "backward":
            c = dict(op=op, M=size(32, 8192), N=size(64, 14336), K=size(64, 14336))
            if c["M"] * c["N"] * c["K"] <= 8192 * 14336 * 4096:
                return c
        else:
            c = dict(op=op, rows=size(16, 14336), K=size(16, 14336), dtype=rng.choice(["bf16", "fp32"]))
            if c["rows"] * c["K"] * min(c["rows"], c["K"]) <= 14336 * 4096 * 4096:
                return c


def work(case):
    """Inputs read once, outputs written once; a product of MXFP4 matrices is 2 M N K
    operations, and each of the two symmetric products of an orthogonalising step
    needs only one triangle of its result."""
    op = case["op"]

    def mx(rows, k):   # codes and scales
        return rows * pad32(k) * 17 / 32

    if op == "quantize":
        r, k, e = case["rows"], case["K"], 4 if case["dtype"] == "fp32" else 2
        b = e * r * k + mx(r, k) + 2 * r * k
        if case["both"]:
            b += mx(k, r) + 2 * r * k
        return {"bytes": b, "flops": 0}
    if op == "orth":
        m, n = sorted((case["rows"], case["K"]))
        e = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": (e + 2) * m * n, "flops": STEPS * (3 * m * m * n + m ** 3)}
    m, n, k = case["M"], case["N"], case["K"]
    if op == "product":
        return {"bytes": mx(m, k) + mx(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "linear":
        return {"bytes": 2 * m * k + mx(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": 2 * m * n + mx(k, n) + mx(k, m) + 2 * m * k + 2 * n * k, "flops": 4 * m * n * k}


# ---- inputs ---------------------------------------------------------------------

def activations(rows, k, g, dtype):
    """Normal values whose columns differ in size, a few of them by much (the
    outlier channels of a transformer's hidden states)."""
    x = torch.randn(rows, k, device="cuda", generator=g)
    col = torch.exp(0.5 * torch.randn(k, device="cuda", generator=g))
    col[torch.rand(k, device="cuda", generator=g) < 0.01] *= 20.0
    return x.mul_(col).to(dtype)


def mx_matrix(rows, k, g, sigma):
    """A random MXFP4 matrix as a quantiser leaves it: codes of normal values
    [rows, pad32(k) / 2] and scales [rows, pad32(k) / 32] (zeros past k)."""
    kp = pad32(k)
    codes = torch.empty(rows, kp // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, kp // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // max(kp, 1))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for r in range(0, rows, step):
        x = sigma * torch.randn(min(step, rows - r), kp, device="cuda", generator=g)
        x[:, k:] = 0
        b = x.view(x.shape[0], -1, 32)
        e = torch.frexp(b.abs().amax(-1))[1].clamp_(min=-60) - 3     # normal values: never near the range's ends
        mag = torch.bucketize(b.abs() * torch.exp2(-e.float())[..., None], mids)
        c = (mag + 8 * (b < 0)).to(torch.uint8).view(x.shape[0], kp // 2, 2)
        codes[r:r + step] = c[..., 0] | (c[..., 1] << 4)
        scales[r:r + step] = (e + 127).to(torch.uint8)
    return codes, scales


def packed(scales, operand):
    """The scales in the order the library's products read them: per 128 rows, per
    128 k, 64 lanes of 8 bytes (weights are laid out once)."""
    rows, nblk = scales.shape
    groups, nk = -(-rows // 128), -(-nblk // 4)
    full = torch.full((groups * 128, nk * 4), 127, dtype=torch.uint8, device=scales.device)
    full[:rows, :nblk] = scales
    x, e = torch.arange(16, device=scales.device)[:, None], torch.arange(8, device=scales.device)[None, :]
    row = 16 * e + x if operand == 0 else 32 * (e >> 1) + 4 * (e & 1) + (x & 3) + 8 * (x >> 2)
    t = full.view(groups, 128, nk, 4)[:, row]                       # [group, x, e, step, block]
    return t.permute(0, 3, 4, 1, 2).contiguous().view(-1)           # [group, step, block, x, e]


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    if op == "quantize":
        s["x"] = activations(case["rows"], case["K"], g, dtype)
    elif op == "orth":
        # a gradient: a few strong directions over a full-rank rest
        m, n = case["rows"], case["K"]
        r = min(16, m, n)
        amp = 0.5 ** torch.arange(r, device="cuda")
        x = torch.randn(m, r, device="cuda", generator=g) * amp @ torch.randn(r, n, device="cuda", generator=g)
        s["x"] = (1e-3 * (x + 0.5 * torch.randn(m, n, device="cuda", generator=g))).to(dtype)
    elif op == "product":
        s["a"], s["sa"] = mx_matrix(case["M"], case["K"], g, 1.0)
        s["b"], s["sb"] = mx_matrix(case["N"], case["K"], g, 0.02)
        s["pa"], s["pb"] = packed(s["sa"], 0), packed(s["sb"], 1)
    elif op == "linear":
        s["x"] = activations(case["M"], case["K"], g, dtype)
        s["w"], s["sw"] = mx_matrix(case["N"], case["K"], g, 0.02)
        s["pw"] = packed(s["sw"], 1)
    else:
        s["dy"] = activations(case["M"], case["N"], g, dtype)
        s["wt"], s["swt"] = mx_matrix(case["K"], case["N"], g, 0.02)
        s["xt"], s["sxt"] = mx_matrix(case["K"], case["M"], g, 1.0)
        s["pwt"], s["pxt"] = packed(s["swt"], 1), packed(s["sxt"], 1)
    return s


# ---- the plain form -------------------------------------------------------------

def pow2(s):
    """2^s in fp32 for whole numbers -127 <= s <= 127, from its bits."""
    return ((s + 127).clamp(min=1) << 23).view(torch.float32) * torch.where(s == -127, 0.5, 1.0)


def decode(codes, scales):
    """The fp32 values of an MXFP4 matrix, [rows, pad32(K)]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=codes.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).int()].view(codes.shape[0], -1, 32)
    return (v * pow2(scales.int() - 127)[..., None]).view(codes.shape[0], -1)


def quantized(x):
    """The fp32 values of x's MXFP4 form along its rows, [rows, pad32(K)]."""
    rows, k = x.shape
    b = torch.nn.functional.pad(x.float(), (0, pad32(k) - k)).view(rows, -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(min=-127), 0)
    a = b.abs() * pow2(-s)                                          # exact
    idx = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)[idx]
    return (torch.copysign(v, b) * pow2(s)).view(rows, -1)


def plain(s):
    op = s["op"]
    if op == "quantize":
        k, rows = s["K"], s["rows"]
        v = quantized(s["x"])[:, :k].to(torch.bfloat16)
        return (v, quantized(s["x"].t())[:, :rows].to(torch.bfloat16)) if s["both"] else v
    if op == "product":
        return (decode(s["a"], s["sa"]) @ decode(s["b"], s["sb"]).t()).to(torch.bfloat16)
    if op == "linear":
        return (quantized(s["x"]) @ decode(s["w"], s["sw"]).t()).to(torch.bfloat16)
    if op == "backward":
        dx = quantized(s["dy"]) @ decode(s["wt"], s["swt"]).t()
        dw = quantized(s["dy"].t()) @ decode(s["xt"], s["sxt"]).t()
        return dx.to(torch.bfloat16), dw.to(torch.bfloat16)
    a, b, c = COEFFS
    x = s["x"].float()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + EPS)
    for _ in range(STEPS):
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.t() if tall else x).to(torch.bfloat16)


def run(state):
    if not own:
        return plain(state)
    import dense_gemm_fp8_amd as hkg
    s, op = state, state["op"]
    A, B = hkg.HKG_MX_OPERAND_A, hkg.HKG_MX_OPERAND_B
    if op == "quantize":
        if s["both"]:
            q, p, qt, pt = hkg.mxfp4_quantize_both(s["x"], B, B)
            return (hkg.mxfp4_dequantize(q, p, B)[:, :s["K"]], hkg.mxfp4_dequantize(qt, pt, B)[:, :s["rows"]])
        q, p = hkg.mxfp4_quantize(s["x"], A)
        return hkg.mxfp4_dequantize(q, p, A)[:, :s["K"]]
    if op == "product":
        return hkg.gemm_mxfp4(s["a"], s["b"], s["pa"], s["pb"])
    if op == "linear":
        return hkg.linear_mxfp4(s["x"], s["w"], s["pw"])
    if op == "backward":
        return hkg.linear_mxfp4_backward(s["dy"], s["wt"], s["pwt"], s["xt"], s["pxt"])
    return hkg.orthogonalize(s["x"], steps=STEPS, coefficients=COEFFS, eps=EPS)


# ---- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    magnitude = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    def power(e):   # 2^e, exact for whole numbers e
        return ((e + 1023).long() << 52).view(torch.float64)

    grid = torch.tensor(magnitude + [-m for m in magnitude], dtype=torch.float64, device="cuda")

    def value(codes, scales):
        rows = codes.shape[0]
        out = torch.empty(rows, 2 * codes.shape[1], dtype=torch.float64, device="cuda")
        out[:, 0::2] = grid[(codes % 16).long()]
        out[:, 1::2] = grid[(codes // 16).long()]
        return out.mul_(torch.repeat_interleave(power(scales.double() - 127), 32, dim=1))

    def nearest(x):
        rows, k = x.shape
        z = torch.zeros(rows, pad32(k), dtype=torch.float64, device="cuda")
        z[:, :k] = x
        z = z.view(-1, 32)
        top = z.abs().max(1).values
        s = torch.floor(torch.log2(torch.where(top > 0, top, 4.0)))
        s = s + (power(s + 1) <= top).double() * (top > 0)        # log2 rounded across a power of two
        s = s - (power(s) > top).double() * (top > 0)
        unit = power((s - 2).clamp(min=-127))[:, None]
        y = z / unit
        gap = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))   # spacing of the grid at y
        return (torch.round(y / gap) * gap).clamp(-6, 6).mul_(unit).view(rows, -1)

    op = case["op"]
    if op == "quantize":
        v = nearest(s["x"].double())[:, :case["K"]]
        return (v, nearest(s["x"].double().t())[:, :case["rows"]]) if case["both"] else v
    if op == "product":
        return value(s["a"], s["sa"]) @ value(s["b"], s["sb"]).T
    if op == "linear":
        return nearest(s["x"].double()) @ value(s["w"], s["sw"]).T
    if op == "backward":
        dy = s["dy"].double()
        return nearest(dy) @ value(s["wt"], s["swt"]).T, nearest(dy.T) @ value(s["xt"], s["sxt"]).T
    g = s["x"].double()
    wide = g.T if case["rows"] > case["K"] else g
    x = wide / (torch.linalg.norm(wide) + EPS)
    for _ in range(STEPS):
        # the same step from the other side where that is smaller: (a + b S + c S^2) x, S = x x^T
        s2 = x @ x.T
        x = COEFFS[0] * x + COEFFS[1] * (s2 @ x) + COEFFS[2] * (s2 @ (s2 @ x))
    return x.T if case["rows"] > case["K"] else x
