"""LayerNorm of rows whose values are all alike, or nearly: their mean is that value, their variance zero, and the bias
remains, whatever the value's size and the number of columns."""
import pytest
import torch

from ops_helpers import U32, close, device_ok, randn
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


VALUES = [0.0, 2.5, -1.0, 0.1, 1000.0, -3.1e4, 999424.0, 1e9, -1e15, 1e20, 1e30, 1e35, -3.3e38, 1e-20, 1e-38]
# one warp a row to sixteen, one piece a thread to four, widths that are no powers of two; rows in registers, then streamed
SIZES = [(40, 8), (40, 24), (40, 584), (600, 904), (600, 1032), (100, 2056), (100, 5000), (40, 8200), (40, 16376), (2200, 1032), (450, 5000),
         (300, 8200), (150, 16376)]


@pytest.mark.parametrize("rows,h", SIZES)
@pytest.mark.parametrize("bias", [True, False])
def test_constant_rows(ops, rows, h, bias):
    x, w, b = randn(rows, h, seed=1), randn(h, seed=2, mean=1.0), randn(h, seed=3) if bias else None
    want = torch.zeros(h, dtype=torch.bfloat16, device="cuda") if b is None else b
    clean, *_ = ops.layer_norm_fwd(x, w, b)
    for i, v in enumerate(VALUES):
        x[2 * i] = v
    y, mean, rstd = ops.layer_norm_fwd(x, w, b)
    for i, v in enumerate(VALUES):
        r = 2 * i
        assert torch.equal(y[r], want), (v, (y[r].float() - want.float()).abs().max())
        assert mean[r] == x[r, 0].float(), v
    # 1 / sqrt(eps): half of the rounding of eps to fp32, the root's and the division's, 2.5 x 2^-24 to first order
    want = torch.full((len(VALUES),), 1e-5 ** -0.5, device="cuda", dtype=torch.float64)
    close(rstd[0:2 * len(VALUES):2], want, 2.6 * U32 * want, rounding=0, what="rstd")
    assert torch.equal(y[1:2 * len(VALUES):2], clean[1:2 * len(VALUES):2])


@pytest.mark.parametrize("rows,h", SIZES)
def test_one_value_apart(ops, rows, h):
    """Constant but for one value a bf16 step above: all of the variance is that value's."""
    x, w, b = randn(rows, h, seed=1), randn(h, seed=2, mean=1.0), randn(h, seed=3)
    for i, v in enumerate((1.0, 1000.0, 999424.0, -1e15)):
        x[3 * i] = v
        x[3 * i, (h - 1) * (i % 2)] = x[3 * i, h // 2] * (1 + 2.0 ** -6)
    check_fwd(x, w, b, 1e-5, ops.layer_norm_fwd(x, w, b))
