"""LayerNorm's forward of many wide rows, which streams them through shared memory: every width of a team (one, two, four
and eight warps a row), rings of two and of three buffers, widths that end inside a team's pieces, and rows that hold
what their neighbours may not notice."""
import pytest
import torch

from ops_helpers import device_ok, randn
from test_gpu_ops_norm import check_fwd

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


# just above the 2.2 M values from which rows are streamed, one to several rows a team
SIZES = [(2200, 1032), (450, 5000), (300, 8192), (280, 8200), (190, 12288), (150, 16376), (140, 16384), (1000, 8184), (5001, 1160)]


@pytest.mark.parametrize("rows,h", SIZES)
@pytest.mark.parametrize("bias", [True, False])
def test_forward(ops, rows, h, bias):
    x, w = randn(rows, h, seed=1, mean=0.5), randn(h, seed=2, std=0.2, mean=1.0)
    b = randn(h, seed=3) if bias else None
    got = ops.layer_norm_fwd(x, w, b, 1e-5)
    check_fwd(x, w, b, 1e-5, got)
    assert all(torch.equal(a, c) for a, c in zip(got, ops.layer_norm_fwd(x, w, b, 1e-5)))


@pytest.mark.parametrize("rows,h", SIZES)
def test_rows_stay_apart(ops, rows, h):
    """Rows whose squares or sums leave fp32's range, with infinities and NaN: right themselves, unnoticed by the others."""
    x, w, b = randn(rows, h, seed=1), randn(h, seed=2, mean=1.0), randn(h, seed=3)
    clean, *_ = ops.layer_norm_fwd(x, w, b)
    dirty = x.clone()
    huge = {3: 1e18, 11: 1e19, 12: 1e20, 13: 1e25, 14: 1e30, 15: 3e37, 16: 1e-20, 17: 1e-38}
    for r, scale in huge.items():
        dirty[r] = (x[r].float() * scale).to(torch.bfloat16)
    dirty[20], dirty[20, h // 2:] = 0.0, 1e20  # zeros where every thread looks first
    dirty[21], dirty[21, -1] = 1.0, 2e19
    inf = float("inf")
    bad = {30: (0, inf), 31: (h - 1, inf), 32: (h // 2, -inf), 33: (0, float("nan")), 34: (h - 1, float("nan")), 35: (slice(None), inf),
           36: (slice(8, None), -inf)}
    for r, (at, value) in bad.items():
        dirty[r, at] = value
    y, mean, rstd = ops.layer_norm_fwd(dirty, w, b)
    touched = torch.zeros(rows, dtype=torch.bool, device="cuda")
    touched[[*huge, 20, 21, *bad]] = True
    assert torch.equal(y[~touched], clean[~touched])
    some = torch.tensor([*huge, 20, 21], device="cuda")
    check_fwd(dirty[some], w, b, 1e-5, (y[some], mean[some], rstd[some]))
    for r in bad:  # the mean or the variance is undefined, and so is every value
        assert torch.isnan(y[r]).all(), r


@pytest.mark.parametrize("rows,h", SIZES)
def test_output_in_the_inputs_place(ops, rows, h):
    from comm_overlap_gb300 import domino as dm
    x, w = randn(rows, h, seed=1), randn(h, seed=2)
    y, _, _ = ops.layer_norm_fwd(x, w)
    wide = torch.full((rows, h + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    z = wide[:, 8:h + 8]
    z.copy_(x)
    ops._call(dm.domino_layernorm_fwd, x, z, h + 16, w, None, 1e-5, z, h + 16, None, None, rows, h)
    assert torch.equal(z, y)
    z.fill_(7.0)
    assert (wide == 7.0).all()
