"""The linear layer's calls that move where results are written -- pitches, odd addresses, y
on the residual itself, rows beyond 2^32 bytes, a workspace of the caller's -- in every kernel
that writes.  Results are compared with the same call's on dense matrices (whose values
test_gpu_linear.py and test_gpu_linear_kernels.py hold against the definition)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402
from dense_gemm_fp8_amd import linear16 as lin  # noqa: E402

RNG = (0x1234567, 0x89abcdef)
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# M, N, K of products that take: few rows in blocks of 32 and 64; 128-tiles of one and of two
# groups of waves; K in parts that are joined; 192-tiles; 256-tiles; 256- and 128-tiles cut by
# rows and by columns
FORWARD = {"rows": (300, 333, 264), "rows64": (70, 4100, 72), "tile128": (1000, 4090, 64), "tile2": (1000, 1030, 744),
           "join": (130, 4100, 4104), "tile192": (2100, 2304, 72), "tile256": (4000, 4090, 64), "cut_rows": (4200, 4200, 72),
           "cut_columns": (400, 38400, 72)}
# of gradients: dx joined and dw 256-tiles; dx 256-tiles, dw cut by columns; dx joined, dw cut by
# rows; 128-tiles for both; dx joined, dw 128-tiles of two groups; dx 256-tiles, dw parts of two
# groups; one launch for both
BACKWARD = [(600, 4160, 2048), (72, 400, 38400), (77, 4200, 4200), (2049, 2051, 2056), (1000, 4100, 264), (13000, 1100, 1032),
            (500, 1000, 768)]


def rand(seed, *shape, kind="bf16", size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (size * torch.randn(*shape, device="cuda", generator=g)).to(TYPE[kind])


def inside(seed, rows, cols, at, kind="bf16"):
    """A matrix in the middle of a wider one, which comes with it."""
    t = rand(seed, rows + 3, cols + at + 9, kind=kind)
    return t, t[1:1 + rows, at:at + cols]


def beside(whole, before, rows, cols, at):
    """Whether `whole` is what it was outside of the matrix."""
    a, b = whole.clone(), before.clone()
    a[1:1 + rows, at:at + cols] = 0
    b[1:1 + rows, at:at + cols] = 0
    return torch.equal(a, b)


def operands(M, N, K, kind="bf16"):
    return rand(1, M, K, kind=kind), rand(2, N, K, kind=kind, size=K ** -0.5), rand(3, N, kind=kind)


def test_the_joined_size_is_split():
    assert lin._lib().hkg_linear_workspace_bytes(*FORWARD["join"]) > 0
    assert all(lin._lib().hkg_linear_workspace_bytes(*v) == 0 for k, v in FORWARD.items() if k != "join")


@pytest.mark.parametrize("path", FORWARD)
@pytest.mark.parametrize("kind,yk", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
def test_pitches_and_odd_addresses(kind, yk, path):
    M, N, K = FORWARD[path]
    x, W, b = operands(M, N, K, kind)
    _, r = inside(4, M, N, 3, yk)
    yw, y = inside(5, M, N, 1, yk)
    zw, z = inside(6, M, N, 5, kind)
    y_before, z_before = yw.clone(), zw.clone()
    hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.2, rng=RNG, y=y, z=z)
    dense = torch.empty(M, N, dtype=TYPE[kind], device="cuda")
    want = hkg.linear(x, W, bias=b, activation="silu", residual=r.contiguous(), p=0.2, rng=RNG, z=dense)
    assert torch.equal(y, want) and torch.equal(z, dense)
    assert beside(yw, y_before, M, N, 1) and beside(zw, z_before, M, N, 5)


@pytest.mark.parametrize("path", FORWARD)
@pytest.mark.parametrize("yk", ["bf16", "fp32"])
def test_onto_the_residual_itself(yk, path):
    M, N, K = FORWARD[path]
    x, W, b = operands(M, N, K)
    whole, r = inside(4, M, N, 3, yk)
    before = whole.clone()
    want = hkg.linear(x, W, bias=b, activation="gelu", residual=r, p=0.1, rng=RNG)
    assert hkg.linear(x, W, bias=b, activation="gelu", residual=r, p=0.1, rng=RNG, y=r) is r
    assert torch.equal(r, want) and beside(whole, before, M, N, 3)
    dense = before[1:1 + M, 3:3 + N].contiguous()
    assert torch.equal(hkg.linear(x, W, bias=b, activation="gelu", residual=dense, p=0.1, rng=RNG, y=dense), want)


@pytest.mark.parametrize("path", FORWARD)
def test_rows_beyond_32_bits(path):
    """y on the residual (fp32), and z, in rows whose offsets pass 2^32 bytes."""
    M, N, K = FORWARD[path]
    x, W, b = operands(M, N, K)
    pitch = (1 << 31) // (M - 40) + N | 1                   # in bytes beyond 2^32 from 40 rows before the end at the latest
    y_all = torch.empty(M * pitch, dtype=torch.float32, device="cuda")
    z_all = torch.empty(M * pitch, dtype=torch.bfloat16, device="cuda")
    y, z = (t.view(M, pitch)[:, 1:1 + N] for t in (y_all, z_all))
    assert (M - 40) * pitch * 2 >= 1 << 32
    r = rand(4, M, N, kind="fp32")
    y.copy_(r)
    hkg.linear(x, W, bias=b, activation="silu", residual=y, p=0.2, rng=RNG, y=y, z=z)
    dense = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    want = hkg.linear(x, W, bias=b, activation="silu", residual=r, p=0.2, rng=RNG, z=dense)
    assert torch.equal(y, want) and torch.equal(z, dense)


@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_gradients_with_pitches_and_odd_addresses(kind, M, N, K):
    x, W, _ = operands(M, N, K, kind)
    _, dy = inside(3, M, N, 3, "fp32")
    _, z = inside(4, M, N, 5, kind)
    xw, dx = inside(5, M, K, 3, kind)
    ww, dw = inside(6, N, K, 1, kind)
    bw = rand(7, N + 9, kind="fp32")
    before = [t.clone() for t in (xw, ww, bw)]
    want = hkg.linear_backward(dy.contiguous(), x, W, z=z.contiguous(), activation="gelu", p=0.1, rng=RNG)
    got = hkg.linear_backward(dy, x, W, z=z, activation="gelu", p=0.1, rng=RNG, dx=dx, dw=dw, dbias=bw[1:1 + N])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert beside(xw, before[0], M, K, 3) and beside(ww, before[1], N, K, 1)
    assert torch.equal(bw[:1], before[2][:1]) and torch.equal(bw[1 + N:], before[2][1 + N:])


@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_gradients_rows_beyond_32_bits(M, N, K):
    x, W, _ = operands(M, N, K)
    dy = rand(3, M, N)
    far = []
    for rows in (M, N):
        pitch = (1 << 31) // (rows - 40) + K | 1
        far.append(torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda").view(rows, pitch)[:, 1:1 + K])
    want = hkg.linear_backward(dy, x, W, p=0.1, rng=RNG)
    hkg.linear_backward(dy, x, W, p=0.1, rng=RNG, dx=far[0], dw=far[1])
    assert torch.equal(far[0], want[0]) and torch.equal(far[1], want[1])


# ---- a workspace of the caller's -----------------------------------------------------------

class Workspace:
    """`need` bytes between two runs of a pattern, filled with what no sum should be read from."""

    def __init__(self, need):
        self.need = need
        self.all = torch.empty(4096 + need + 4096, dtype=torch.uint8, device="cuda")
        self.all.fill_(0xff)                                # bf16, fp16 and fp32 NaNs
        self.edges = torch.randint(0, 256, (2, 4096), dtype=torch.uint8, device="cuda")
        self.all[:4096], self.all[4096 + need:] = self.edges[0], self.edges[1]

    def of(self, need):
        """The last `need` bytes, so that what follows is the pattern."""
        at = 4096 + (self.need - need) // 16 * 16
        return self.all[at:at + need]

    def whole(self):
        return torch.equal(self.all[:4096], self.edges[0]) and torch.equal(self.all[4096 + self.need:], self.edges[1])


def test_linear_in_a_workspace_of_exactly_the_stated_size():
    sizes = [(130, 4100, 4104), (100, 4096, 14336), (260, 2100, 8200), (128, 8192, 8192)]
    needs = [lin._lib().hkg_linear_workspace_bytes(*s) for s in sizes]
    assert min(needs) > 0
    for i, (s, n) in enumerate(zip(sizes, needs)):
        ws = Workspace(n)
        x, W, b = operands(*s)
        want = hkg.linear(x, W, bias=b, activation="silu")
        # first on NaNs, then on another size's sums, in the same bytes
        assert torch.equal(hkg.linear(x, W, bias=b, activation="silu", workspace=ws.of(n)), want) and ws.whole()
        j = min(range(len(sizes)), key=lambda k: needs[k])
        other = operands(*sizes[j])
        hkg.linear(other[0], other[1], workspace=ws.of(needs[j]))
        assert torch.equal(hkg.linear(x, W, bias=b, activation="silu", workspace=ws.of(n)), want) and ws.whole(), i


@pytest.mark.parametrize("M,N,K", BACKWARD + [(5000, 77, 520), (1, 1, 8), (65, 130, 72)])
def test_gradients_in_a_workspace_of_exactly_the_stated_size(M, N, K):
    n = lin._lib().hkg_linear_backward_workspace_bytes(M, N, K)
    ws = Workspace(n)
    x, W, _ = operands(M, N, K)
    dy, z = rand(3, M, N), rand(4, M, N)
    want = hkg.linear_backward(dy, x, W, z=z, activation="gelu", p=0.1, rng=RNG)
    for _ in range(2):
        got = hkg.linear_backward(dy, x, W, z=z, activation="gelu", p=0.1, rng=RNG, workspace=ws.of(n))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert ws.whole()
        small = (rand(5, 3, 5), rand(6, 3, 16), rand(7, 5, 16))
        need = lin._lib().hkg_linear_backward_workspace_bytes(3, 5, 16)
        if need <= n:                                       # another shape's leftovers
            hkg.linear_backward(*small, workspace=ws.of(need))


def test_a_workspace_too_small_leaves_the_outputs():
    M, N, K = FORWARD["join"]
    x, W, _ = operands(M, N, K)
    n = lin._lib().hkg_linear_workspace_bytes(M, N, K)
    y = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad in (ws[:n - 1], ws[:16]):
        with pytest.raises(hkg.HkgError) as e:
            hkg.linear(x, W, y=y, workspace=bad)
        assert e.value.status == hkg.HKG_ERR_WORKSPACE
    m = lin._lib().hkg_linear_backward_workspace_bytes(M, N, K)
    dx = torch.full((M, K), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hkg.HkgError):
        hkg.linear_backward(y, x, W, dx=dx, workspace=torch.empty(m - 16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert (y == 3.0).all() and (dx == 3.0).all()


def test_split_products_on_two_streams_at_once():
    sizes = (FORWARD["join"], (260, 2100, 8200))
    data = [operands(*s) + (rand(9, s[0], s[1]),) for s in sizes]

    def calls(x, W, b, dy, stream=None):
        return (hkg.linear(x, W, bias=b, activation="silu", stream=stream), *hkg.linear_backward(dy, x, W, stream=stream))
    want = [calls(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(6):
        for i in range(2):
            got[i].append(calls(*data[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            for u, v in zip(one, want[i]):
                assert torch.equal(u, v)
