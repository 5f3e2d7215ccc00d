"""Cases of the 16-bit linear layer with a fused epilogue, of its gradients and of dropout, in their plain form and
through the library.

Operators (`op` of a case), x and W of one 16-bit type T (bfloat16 or float16):
  linear    z = x W^T + bias,  y = residual + D(act(z))
  backward  its gradients from dy: dz = D(dy) act'(z), dx = dz W, dw = dz^T x, dbias = the sums of dz's columns
  dropout   out = residual + D(x); on dy without a residual it is its own backward pass
D keeps an element or drops it: with q = round(65536 p) / 65536, a kept one is divided by 1 - q, a dropped one is 0.
Which ones is decided by a counter-based generator, Philox-4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011), so that no mask is ever stored: the key is `seed` (low word, high
word), the counter (column / 8, row, offset's low word, offset's high word), and its four words are eight 16-bit
numbers, low halves first, for columns 8 c .. 8 c + 7 of a row; an element is dropped where its number is below 65536 q.
"""
import math

import torch

own = False

C_TANH, A_TANH = math.sqrt(2.0 / math.pi), 0.044715


# ---- the cases ------------------------------------------------------------------

def linear(M, N, K, dtype, bias=None, act=None, residual=None, p=0.0, z=False, **kw):
    """bias, residual: None, "same" (the type of x) or "fp32"; y has residual's type, or x's."""
    return dict(op="linear", M=M, N=N, K=K, dtype=dtype, bias=bias, act=act, residual=residual, p=p, z=z, **kw)


def backward(M, N, K, dtype, act=None, p=0.0, dy="same", **kw):
    return dict(op="backward", M=M, N=N, K=K, dtype=dtype, act=act, p=p, dy=dy, **kw)


def dropout(rows, cols, dtype, p, residual=False, **kw):
    return dict(op="dropout", rows=rows, cols=cols, dtype=dtype, p=p, residual=residual, **kw)


def listed():
    return [
        # decoding: one token through an MLP's up projection, bound by reading W
        linear(1, 14336, 4096, "bf16", bias="fp32", act="silu", name="linear-token"),
        # decoding a batch of 16 sequences through a square projection onto the residual stream
        linear(16, 8192, 8192, "fp16", residual="same", name="linear-batch"),
        # a short prompt on the MLP's way down, the residual stream in fp32
        linear(100, 4096, 14336, "bf16", bias="same", residual="fp32", name="linear-prompt"),
        # odd and ragged sizes, everything at once
        linear(1111, 2777, 1184, "bf16", bias="fp32", act="gelu", residual="same", p=0.1, z=True, name="linear-ragged"),
        # training: an MLP's up projection over a long batch, z kept for the backward pass
        linear(16384, 14336, 4096, "bf16", bias="same", act="gelu_tanh", z=True, name="linear-up"),
        # training: the way down, with dropout before the residual
        linear(8192, 4096, 14336, "bf16", bias="same", residual="same", p=0.1, name="linear-down"),
        # a training step's gradients, small and odd
        backward(500, 1000, 768, "fp16", act="relu", p=0.1, name="backward-small"),
        # a training step's gradients of the up projection
        backward(8192, 14336, 4096, "bf16", act="gelu_tanh", name="backward-up"),
        # of the way down, the gradient of the residual stream in fp32
        backward(8192, 4096, 14336, "bf16", p=0.1, dy="fp32", name="backward-down"),
        # the hidden states of a few tokens: latency
        dropout(16, 4096, "bf16", 0.1, name="dropout-small"),
        # hidden states onto the residual stream
        dropout(16384, 4096, "bf16", 0.1, residual=True, name="dropout-residual"),
        # a wide layer's gradient in fp32
        dropout(8192, 14336, "fp32", 0.25, name="dropout-grad"),
    ]


def draw(rng):
    def size(lo, hi):   # spread over the logarithm; every second one a multiple of 64
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v

    def depth(lo, hi):  # K: rows of whole 16-byte units
        return -(-size(lo, hi) // 8) * 8

    op = rng.choice(["linear", "backward", "dropout"])
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice([None, "relu", "gelu", "gelu_tanh", "silu"])
    p = rng.choice([0.0, 0.05, 0.1, 0.5])
    while True:
        if op == "linear":
            c = linear(size(1, 16384), size(64, 16384), depth(64, 16384), dtype, bias=rng.choice([None, "same", "fp32"]),
                       act=act, residual=rng.choice([None, "same", "fp32"]), p=p, z=rng.random() < 0.5)
            if c["M"] * c["N"] * c["K"] <= 16384 * 14336 * 4096:
                return c
        elif op == "backward":
            c = backward(size(32, 8192), size(64, 14336), depth(64, 14336), dtype, act=act, p=p,
                         dy=rng.choice(["same", "fp32"]))
            if c["M"] * c["N"] * c["K"] <= 8192 * 14336 * 4096:
                return c
        else:
            c = dropout(size(1, 16384), size(32, 16384), rng.choice(["bf16", "fp16", "fp32"]), max(p, 0.05),
                        residual=rng.random() < 0.5)
            if c["rows"] * c["cols"] <= 8192 * 14336:
                return c


def work(case):
    """Inputs read once, outputs written once; a product is 2 M N K operations."""
    def wide(t):
        return 4 if t == "fp32" else 2 if t else 0

    if case["op"] == "dropout":
        n, e = case["rows"] * case["cols"], wide(case["dtype"])
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 0}
    m, n, k = case["M"], case["N"], case["K"]
    operands = 2 * (m * k + n * k)
    if case["op"] == "linear":
        r = wide(case["residual"])
        return {"bytes": operands + n * wide(case["bias"]) + m * n * (r + (r or 2) + (2 if case["z"] else 0)),
                "flops": 2 * m * n * k}
    return {"bytes": 2 * operands + m * n * (wide(case["dy"]) + (2 if case["act"] else 0)) + 4 * n,
            "flops": 4 * m * n * k}


# ---- inputs ---------------------------------------------------------------------

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def activations(rows, k, g, dtype, size=1.0):
    """Normal values whose columns differ in size, a few of them by much (the
    outlier channels of a transformer's hidden states)."""
    x = torch.randn(rows, k, device="cuda", generator=g)
    col = size * torch.exp(0.5 * torch.randn(k, device="cuda", generator=g))
    col[torch.rand(k, device="cuda", generator=g) < 0.01] *= 10.0
    return x.mul_(col).to(dtype)


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    s = dict(case)
    t = TYPES[case["dtype"]]
    s["rng"] = ((seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), (seed * 7919 + (seed << 33)) % (1 << 48))

    def of(kind, *shape, size=1.0):
        if kind is None:
            return None
        return (size * torch.randn(*shape, device="cuda", generator=g)).to(t if kind == "same" else torch.float32)

    if case["op"] == "dropout":
        s["x"] = activations(case["rows"], case["cols"], g, t)
        s["residual"] = of("same" if case["residual"] else None, case["rows"], case["cols"])
        return s
    m, n, k = case["M"], case["N"], case["K"]
    s["x"] = activations(m, k, g, t)
    s["W"] = (torch.randn(n, k, device="cuda", generator=g) / k ** 0.5).to(t)
    if case["op"] == "linear":
        s["bias"] = of(case["bias"], n, size=0.2)
        s["residual"] = of(case["residual"], m, n)
    else:
        s["z"] = activations(m, n, g, t) if case["act"] else None
        s["dy"] = activations(m, n, g, t if case["dy"] == "same" else torch.float32, 0.05)
    return s


# ---- the plain form -------------------------------------------------------------

def numbers(rows, cols, rng):
    """The 16-bit numbers of a [rows, cols] matrix, Philox-4x32-10 in 64-bit words."""
    seed, offset = rng
    low = 0xFFFFFFFF
    c0 = torch.arange(-(-cols // 8), device="cuda")[None, :]
    c1 = torch.arange(rows, device="cuda")[:, None]
    c = [c0.expand(rows, -1), c1.expand(-1, c0.shape[1]),
         torch.full((1, 1), offset & low, device="cuda"), torch.full((1, 1), offset >> 32, device="cuda")]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # 64-bit products: their bits are right though the sign is not
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = [(w >> s) & 0xFFFF for w in c for s in (0, 16)]
    return torch.stack(halves, -1).view(rows, -1)[:, :cols]


def keep_and_scale(rows, cols, p, rng):
    t = round(65536 * p)
    return numbers(rows, cols, rng) >= t, 65536.0 / (65536 - t)


def dropped(v, p, rng):
    if p == 0.0:
        return v
    keep, scale = keep_and_scale(v.shape[0], v.shape[1], p, rng)
    return torch.where(keep, v * scale, 0.0)


def sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def activation(z, act):
    if act is None:
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":      # 1/2 (1 + tanh u) = 1 / (1 + exp(-2 u))
        return z * sigmoid(2.0 * C_TANH * (z + A_TANH * z * z * z))
    return z * sigmoid(z)


def slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        s = sigmoid(2.0 * C_TANH * (z + A_TANH * z * z * z))
        return s + z * s * (1.0 - s) * 2.0 * C_TANH * (1.0 + 3.0 * A_TANH * z * z)
    s = sigmoid(z)
    return s + z * s * (1.0 - s)


def plain(s):
    t = TYPES[s["dtype"]]
    if s["op"] == "dropout":
        v = dropped(s["x"].float(), s["p"], s["rng"])
        return (v if s["residual"] is None else s["residual"].float() + v).to(t)
    if s["op"] == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = dropped(activation(z, s["act"]), s["p"], s["rng"])
        if s["residual"] is not None:
            y = s["residual"].float() + y
            y = y.to(s["residual"].dtype)
        y = y.to(t) if s["residual"] is None else y
        zt = s.get("z")
        return (y, z.to(t)) if zt else y
    dz = dropped(s["dy"].float(), s["p"], s["rng"])
    if s["act"] is not None:
        dz = dz * slope(s["z"].float(), s["act"])
    return (dz @ s["W"].float()).to(t), (dz.t() @ s["x"].float()).to(t), dz.sum(0)


def run(state):
    if not own:
        return plain(state)
    import dense_gemm_fp8_amd as hkg
    s = state
    if s["op"] == "dropout":
        return hkg.dropout(s["x"], s["p"], s["rng"], residual=s["residual"])
    if s["op"] == "linear":
        if not s["z"]:
            return hkg.linear(s["x"], s["W"], bias=s["bias"], activation=s["act"], residual=s["residual"], p=s["p"],
                              rng=s["rng"])
        z = torch.empty(s["M"], s["N"], dtype=s["x"].dtype, device="cuda")
        y = hkg.linear(s["x"], s["W"], bias=s["bias"], activation=s["act"], residual=s["residual"], p=s["p"],
                       rng=s["rng"], z=z)
        return y, z
    return hkg.linear_backward(s["dy"], s["x"], s["W"], z=s["z"], activation=s["act"], p=s["p"], rng=s["rng"])


# ---- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)

    def mulhilo(m, v):
        """High and low 32 bits of m v for 32-bit whole numbers, by 16-bit limbs."""
        m1, m0, v1, v0 = m >> 16, m & 65535, v // 65536, v % 65536
        mid = m0 * v0 // 65536 + m1 * v0 % 65536 + m0 * v1 % 65536
        hi = m1 * v1 + m1 * v0 // 65536 + m0 * v1 // 65536 + mid // 65536
        return hi, mid % 65536 * 65536 + m0 * v0 % 65536

    def masked(v):
        below = round(65536 * case["p"])
        if below == 0:
            return v
        rows, cols = v.shape
        groups = (cols + 7) // 8
        at = torch.arange(rows * groups, device="cuda")
        w, x = at % groups, at // groups
        y, z = torch.full_like(at, s["rng"][1] % 2 ** 32), torch.full_like(at, s["rng"][1] // 2 ** 32)
        for r in range(10):
            k0, k1 = (s["rng"][0] + r * 0x9E3779B9) % 2 ** 32, (s["rng"][0] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
            (h0, l0), (h1, l1) = mulhilo(0xD2511F53, w), mulhilo(0xCD9E8D57, y)
            w, x, y, z = h1 ^ x ^ k0, l1, h0 ^ z ^ k1, l0
        out = v.clone()
        for col, word in enumerate((w, x, y, z)):
            for half in range(2):
                n = (word // 65536 if half else word % 65536).view(rows, groups)
                part = out[:, 2 * col + half::8]
                n = n[:, :part.shape[1]]
                part[n < below] = 0.0
        return out.mul_(65536 / (65536 - below))

    def cdf(v):
        return torch.special.ndtr(v)

    def f(v, act):
        if act == "relu":
            return v.clamp(min=0)
        if act == "gelu":
            return v * cdf(v)
        if act == "gelu_tanh":
            return v / 2 * (1 + torch.tanh(C_TANH * (v + A_TANH * v ** 3)))
        return v * torch.special.expit(v) if act == "silu" else v

    def derivative(v, act):
        if act == "relu":
            return (v > 0).double()
        if act == "gelu":
            return cdf(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        if act == "gelu_tanh":
            u = C_TANH * (v + A_TANH * v ** 3)
            return (1 + torch.tanh(u)) / 2 + v / 2 / torch.cosh(u).square() * C_TANH * (1 + 3 * A_TANH * v * v)
        e = torch.special.expit(v)
        return e * (1 + v * torch.special.expit(-v))

    if case["op"] == "dropout":
        v = masked(s["x"].double())
        return v if s["residual"] is None else v.add_(s["residual"])
    if case["op"] == "linear":
        v = s["x"].double() @ s["W"].double().T
        if s["bias"] is not None:
            v += s["bias"]
        y = masked(f(v, case["act"]))
        if s["residual"] is not None:
            y = y + s["residual"]
        return (y, v) if case["z"] else y
    v = masked(s["dy"].double())
    if case["act"] is not None:
        v *= derivative(s["z"].double(), case["act"])
    return v @ s["W"].double(), v.T @ s["x"].double(), v.sum(0)
