"""How exactly the linear layer evaluates its activations: the bounds that
include/hkg_linear.h states, over all of their range and in every kernel that applies them."""
import numpy as np
import pytest

from oracle import linear as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("no GPU", allow_module_level=True)

import dense_gemm_fp8_amd as hkg  # noqa: E402

TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# what takes 4096 columns: few rows, 128-tiles of one and of two groups of waves, K in parts,
# 192-tiles, 256-tiles
PATHS = [(1, 8), (300, 64), (1000, 64), (1000, 1024), (130, 4104), (2048, 64), (4096, 64)]


def values(seed):
    """4096 z: magnitudes from 2^-14 to 2^7 on either side, evenly over the logarithm."""
    g = np.random.Generator(np.random.PCG64(seed))
    return (np.exp2(g.uniform(-14, 7, 4096)) * np.where(g.random(4096) < 0.7, -1, 1)).astype(np.float32)


def evaluated(z, act, y_type, M, K, seed):
    """act(z) out of a product that is 0: z is the bias."""
    kind = "fp16" if y_type == "fp16" else "bf16"
    x, W = (torch.zeros(n, K, dtype=TYPE[kind], device="cuda") for n in (M, len(z)))
    y = torch.empty(M, len(z), dtype=TYPE[y_type], device="cuda")
    hkg.linear(x, W, bias=torch.from_numpy(z).cuda(), activation=act, y=y)
    assert (y == y[0]).all()            # one value a column, whichever lane of which tile formed it
    return y[0].double().cpu().numpy()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,K", PATHS)
def test_fp32_results(act, M, K):
    for seed in range(1, 5 if M < 2000 else 2):
        z = values(seed)
        got, want = evaluated(z, act, "fp32", M, K, seed), ref.act(z, act)
        off = np.abs(got - want) / (2.0 ** -20 * np.abs(want) + 2.0 ** -116)
        i = off.argmax()
        assert off[i] <= 1, "%.2f times the bound, %d of %d out; z %r got %r want %r" % (
            off[i], (off > 1).sum(), off.size, z[i], got[i], want[i])


@pytest.mark.parametrize("y_type", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_16_bit_results(act, y_type):
    for M, K in PATHS[:3]:
        z = values(9)
        got, want = evaluated(z, act, y_type, M, K, 9), ref.act(z, act)
        e = 2.0 ** -15 * np.abs(want) + 2.0 ** -116
        off = np.abs(got - want) - e - ref.HALF[y_type] * (np.abs(want) + e) - ref.TINY[y_type]
        assert off.max() <= 0, (z[off.argmax()], got[off.argmax()], want[off.argmax()])


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_the_ends(act):
    z = np.array([-np.inf, np.inf, np.nan, -3.4e38, 3.4e38, -1e20, 1e20, -101, 101, 0.0, -0.0, 1e-38, -1e-38] + [0.0] * 3, dtype=np.float32)
    with np.errstate(invalid="ignore"):
        want = ref.act(z, act)
    for M, K in ((1, 8), (300, 64)):
        x, W = (torch.zeros(n, K, dtype=torch.bfloat16, device="cuda") for n in (M, len(z)))
        for kind in ("fp32", "bf16"):
            y = torch.empty(M, len(z), dtype=TYPE[kind], device="cuda")
            hkg.linear(x, W, bias=torch.from_numpy(z).cuda(), activation=act, y=y)
            got = y.double().cpu().numpy()
            np.testing.assert_array_equal(np.isnan(got), np.broadcast_to(np.isnan(want), got.shape))
            fine = ~np.isnan(want)
            with np.errstate(invalid="ignore"):
                same = (got == want) | (np.abs(got - want) <= ref.HALF[kind] * 1.01 * np.abs(want) + 2.0 ** -20 * np.abs(want) + 2.0 ** -116)
            # 3.4e38 is beyond bf16's largest number less half a step
            assert same[:, fine & ((kind == "fp32") | (np.abs(z) < 3e38) | np.isinf(z))].all()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slopes(act):
    """dbias of one row is D(dy) act'(z), in fp32."""
    z = torch.from_numpy(values(3)).to(torch.bfloat16)[None].cuda()
    W = torch.zeros(4096, 8, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(1, 4096, device="cuda")
    _, _, db = hkg.linear_backward(dy, None, W, z=z, activation=act, need_dx=False, need_dw=False)
    want = ref.slope(z.double().cpu().numpy()[0], act)
    assert np.abs(db.double().cpu().numpy() - want).max() <= 2.0 ** -19
