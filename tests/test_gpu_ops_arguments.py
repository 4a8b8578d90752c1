"""What the PyTorch functions refuse of tensors on the GPU."""
import pytest
import torch

from ops_helpers import device_ok, randn

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from comm_overlap_gb300 import build
    build.build()
    from comm_overlap_gb300 import torch_ops
    yield torch_ops
    device_ok()


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("shape", [(3, 2, 128), (2, 1, 128), (1, 128), (128,), (3, 128), (6, 64), (12, 64), (2, 3, 64), (2, 3, 2, 64)])
def test_residual_of_another_shape(ops, shape, grad):
    """As many values in another shape are not the output's values."""
    x, w = randn(2, 3, 64, seed=1).requires_grad_(grad), randn(128, 64, seed=2)
    with pytest.raises(ValueError, match="residual"):
        ops.linear(x, w, residual=randn(*shape, seed=3))
    layer = ops.DominoLinear(64, 128)
    with pytest.raises(ValueError, match="residual"):
        layer(x, randn(*shape, seed=3))


@pytest.mark.parametrize("grad", [True, False])
def test_residual_of_the_outputs_shape_or_its_rows(ops, grad):
    x, w, r = randn(2, 3, 64, seed=1).requires_grad_(grad), randn(128, 64, seed=2), randn(2, 3, 128, seed=3)
    y = ops.linear(x, w, residual=r)
    assert y.shape == (2, 3, 128)
    assert torch.equal(y, ops.linear(x, w, residual=r.view(6, 128)))
    assert torch.equal(y, ops.linear(x, w, residual=r.transpose(0, 1).contiguous().transpose(0, 1)))
    assert torch.equal(y[1, 2], ops.linear(x[1, 2], w, residual=r[1, 2]))


def test_scalars_and_what_is_no_tensor(ops):
    x, w, scalar = randn(4, 64, seed=1), randn(128, 64, seed=2), randn(seed=3)
    g = randn(64, seed=4)
    with pytest.raises(ValueError, match="x"):
        ops.layer_norm(scalar, g)
    with pytest.raises(ValueError, match="x"):
        ops.linear(scalar, w)
    with pytest.raises(ValueError, match="x"):
        ops.DominoLayerNorm(64)(scalar)
    with pytest.raises(ValueError, match="weight"):
        ops.linear(x, None)
    with pytest.raises(ValueError, match="weight"):
        ops.linear(x, scalar)
    with pytest.raises(ValueError, match="weight"):
        ops.layer_norm(x, None)
    with pytest.raises(ValueError, match="residual"):
        ops.linear(x, w, residual=1.0)
    q = randn(4, 2, D, seed=5)
    for cu in ([0, 4], None, torch.tensor([0, 4], dtype=torch.int32)):
        with pytest.raises(ValueError, match="cu_q"):
            ops.packed_attention(q, q, q, cu)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="cu_q"):
        ops.packed_attention(q, q, q, cu.long())
    with pytest.raises(ValueError, match="cu_q"):
        ops.packed_attention(q, q, q, cu.view(1, 2))
    with pytest.raises(ValueError, match="k_len"):
        ops.packed_attention(q, q, q, cu, cu[:1], [4])
