"""The linear layer's ReLU at the values where fmaxf(z, 0) and a product with its derivative differ from the definition:
NaN stays NaN, and a gradient is passed on where z > 0 and nowhere else."""
import pytest
import torch

from ops_helpers import device_ok, randn
from test_gpu_ops_linear import check_bwd, check_fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from comm_overlap_gb300 import build
    build.build()
    from comm_overlap_gb300 import torch_ops
    yield torch_ops
    device_ok()


# the kernel of few rows (whole and cut reductions), that of many (whole and cut, several rounds of tiles)
SIZES = [(5, 264, 520), (64, 4608, 2048), (40, 256, 4096), (300, 520, 1040), (257, 264, 8192), (5000, 2056, 264)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("where", ["x", "bias", "weight"])
def test_nan_passes_the_activation(ops, m, n, k, where):
    x, w, b = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5), randn(n, seed=3)
    clean, _ = ops.linear_fwd(x, w, b, "relu")
    assert (clean == 0).any()
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    if where == "x":  # whole rows: NaN, and inf - inf in the sum
        x[1, 3], x[3, 0], x[3, 1] = float("nan"), float("inf"), float("inf")
        w[:, 0], w[:, 1] = w[:, 0].abs() + 0.01, -w[:, 1].abs() - 0.01
        clean, _ = ops.linear_fwd(torch.where(x.isfinite(), x, torch.zeros_like(x)), w, b, "relu")
        bad[[1, 3]] = True
    elif where == "bias":
        b[[0, n - 1]] = float("nan")
        bad[:, [0, n - 1]] = True
    else:
        w[7, k - 1] = float("nan")
        bad[:, 7] = True
    y, z = ops.linear_fwd(x, w, b, "relu", save=True)
    assert torch.equal(torch.isnan(z), bad)
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("m,n,k", SIZES)
def test_infinities_and_zeros(ops, m, n, k):
    x, w, b = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5), randn(n, seed=3)
    b[0], b[1] = float("inf"), -float("inf")
    y, _ = ops.linear_fwd(x, w, b, "relu")
    assert (y[:, 0] == float("inf")).all() and (y[:, 1] == 0).all()
    check_fwd(x, w[2:], b[2:], "relu", None, y[:, 2:], None)
    y, _ = ops.linear_fwd(torch.zeros_like(x), w, None, "relu")
    assert not y.any()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gradients_pass_where_the_value_is_above_zero_alone(ops, m, n, k):
    """Infinite and NaN output gradients at values that ReLU has cut have no effect: a choice, not a product with zero."""
    x, w, gy, z = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5), randn(m, n, seed=3), randn(m, n, seed=4)
    z[0, 0], z[1, 1], z[1, 2], z[2, 3] = 0.0, -0.0, -float("inf"), float("nan")
    cut = ~(z > 0)
    assert cut[0, 0] and cut[1, 1] and cut[1, 2] and cut[2, 3]
    want = ops.linear_bwd(torch.where(cut, torch.zeros_like(gy), gy), x, w, z, "relu")
    check_bwd(gy, x, w, torch.where(z.isnan(), -torch.ones_like(z), z), "relu", *want)
    for bad in (float("inf"), -float("inf"), float("nan")):
        got = ops.linear_bwd(torch.where(cut, torch.full_like(gy, bad), gy), x, w, z, "relu")
        assert all(torch.equal(a, b) for a, b in zip(got, want)), bad
