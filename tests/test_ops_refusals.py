"""What the sublayer operators refuse, at the C ABI (no device is touched: arguments are checked before the
handle) and in the PyTorch functions."""
import pytest
import torch

from comm_overlap_gb300 import domino as dm
from comm_overlap_gb300 import torch_ops as ops

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_overlap_gb300 import build
    build.build()


def status(fn, **kw):
    with pytest.raises(dm.DominoError) as e:
        fn(**kw)
    assert dm.domino_last_error()
    return e.value.status


def ln_fwd(**kw):
    a = dict(handle=None, X=P, ld_x=64, gamma=P, beta=P, eps=1e-5, Y=P, ld_y=64, mean=P, rstd=P, rows=4, h=64, stream=0)
    dm.domino_layernorm_fwd(**{**a, **kw})


def ln_bwd(**kw):
    a = dict(handle=None, gY=P, ld_gy=64, X=P, ld_x=64, gamma=P, mean=P, rstd=P, gres=None, ld_gres=0, gX=P, ld_gx=64,
             ggamma=P, gbeta=P, accumulate=0, rows=4, h=64, workspace=P, workspace_bytes=1 << 20, stream=0)
    dm.domino_layernorm_bwd(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(h=0), INVALID), (dict(rows=-1), INVALID), (dict(h=60), ALIGNMENT), (dict(h=16392, ld_x=16392, ld_y=16392), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(ld_x=56), INVALID), (dict(ld_y=68), ALIGNMENT),
    (dict(ld_x=(1 << 32) + 8), UNSUPPORTED), (dict(X=None), INVALID), (dict(gamma=None), INVALID), (dict(Y=None), INVALID),
    (dict(X=P + 2), ALIGNMENT), (dict(beta=P + 8), ALIGNMENT), (dict(mean=P + 4), ALIGNMENT),
    (dict(), INVALID),                # everything fine but the handle
    (dict(beta=None, mean=None, rstd=None, X=P, rows=0), INVALID)])
def test_layernorm_forward(kw, code):
    assert status(ln_fwd, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(h=60), ALIGNMENT), (dict(rows=-1), INVALID), (dict(accumulate=2), INVALID), (dict(ld_gy=56), INVALID),
    (dict(ld_x=56), INVALID), (dict(ld_gx=66), ALIGNMENT), (dict(gres=P, ld_gres=8), INVALID), (dict(gres=P + 2, ld_gres=64), ALIGNMENT),
    (dict(gY=None), INVALID), (dict(mean=None), INVALID), (dict(ggamma=None), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 16), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE), (dict(), INVALID), (dict(gbeta=None), INVALID)])
def test_layernorm_backward(kw, code):
    assert status(ln_bwd, **kw) == code


def test_layernorm_workspace_size():
    assert dm.domino_layernorm_bwd_workspace_size(0, 64) == 0
    # no more partial rows than two per SM, and never more rows than inputs
    assert dm.domino_layernorm_bwd_workspace_size(1 << 20, 4096) == 304 * 2 * 4096 * 4
    assert dm.domino_layernorm_bwd_workspace_size(1, 4096) == 2 * 4096 * 4
    assert status(dm.domino_layernorm_bwd_workspace_size, rows=1, h=12) == ALIGNMENT


def test_functions_refuse_what_they_cannot_take():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm_bwd(x, x, w, w, w)
    with pytest.raises(ValueError, match="columns"):
        ops.DominoLayerNorm(128, device="cpu")(x)
