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
    # a partial row per SM for many rows, no more than two per SM otherwise, and never more rows than inputs
    assert dm.domino_layernorm_bwd_workspace_size(1 << 20, 4096) == 152 * 2 * 4096 * 4
    assert all(0 < dm.domino_layernorm_bwd_workspace_size(rows, h) <= min(rows, 304) * 2 * h * 4
               for rows in (1, 7, 300, 5000) for h in (8, 512, 2056, 16384))
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


def lin_fwd(**kw):
    a = dict(handle=None, X=P, ld_x=64, W=P, bias=P, act=dm.ACT_GELU, R=P, ld_r=128, Y=P, ld_y=128, Z=P, ld_z=128, M=4, N=128,
             K=64, stream=0)
    dm.domino_linear_fwd(**{**a, **kw})


def lin_bwd(**kw):
    a = dict(handle=None, gY=P, ld_gy=128, X=P, ld_x=64, W=P, Z=P, ld_z=128, act=dm.ACT_GELU, gX=P, ld_gx=64, gW=P, gW_main=None,
             gbias=P, accumulate=0, M=4, N=128, K=64, workspace=P, workspace_bytes=1 << 30, stream=0)
    dm.domino_linear_bwd(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(act=dm.ACT_SWIGLU), UNSUPPORTED), (dict(act=dm.ACT_BILINEAR), UNSUPPORTED), (dict(N=132), ALIGNMENT),
    (dict(K=60), ALIGNMENT), (dict(N=(1 << 20) + 8), UNSUPPORTED), (dict(M=(1 << 31) - 256), UNSUPPORTED),
    (dict(M=(1 << 31) - 257, N=1 << 16, ld_y=1 << 16, ld_r=1 << 16, ld_z=1 << 16), UNSUPPORTED), (dict(ld_x=56), INVALID),
    (dict(ld_x=68), ALIGNMENT), (dict(ld_y=120), INVALID), (dict(ld_r=64), INVALID), (dict(ld_z=130), ALIGNMENT),
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID), (dict(W=P + 8), ALIGNMENT), (dict(bias=P + 2), ALIGNMENT),
    (dict(R=P + 2), ALIGNMENT), (dict(Z=P + 4), ALIGNMENT), (dict(), INVALID), (dict(bias=None, R=None, Z=None), INVALID)])
def test_linear_forward(kw, code):
    assert status(lin_fwd, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(act=dm.ACT_SWIGLU), UNSUPPORTED), (dict(N=100), ALIGNMENT), (dict(accumulate=3), INVALID),
    (dict(gW_main=P), INVALID), (dict(gW=None, gW_main=P + 4), ALIGNMENT), (dict(gY=None), INVALID), (dict(X=None), INVALID),
    (dict(W=None), INVALID), (dict(Z=None), INVALID), (dict(ld_z=64), INVALID), (dict(ld_gy=120), INVALID), (dict(ld_gx=8), INVALID),
    (dict(gX=P + 2), ALIGNMENT), (dict(gbias=P + 4), ALIGNMENT), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE),
    (dict(), INVALID), (dict(gX=None, W=None, gbias=None), INVALID), (dict(gW=None, X=None, ld_x=0), INVALID)])
def test_linear_backward(kw, code):
    assert status(lin_bwd, **kw) == code


def test_linear_workspace_size():
    size = dm.domino_linear_bwd_workspace_size
    assert size(0, 128, 4096, dm.ACT_GELU) == 0
    assert size(4, 128, 64, dm.ACT_GELU) == 1024 + 1024  # gZ, one row of partial sums
    assert size(4, 128, 64, dm.ACT_NONE) == 1024
    assert status(size, M=4, N=128, K=64, act=dm.ACT_SWIGLU) == UNSUPPORTED


def test_linear_functions_refuse_what_they_cannot_take():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear_bwd(x, x, w)
    with pytest.raises(ValueError, match="act"):
        ops.DominoLinear(64, 128, act="tanh", device="cpu")
    with pytest.raises(ValueError, match="act"):
        ops.DominoLinear(64, 128, act=dm.ACT_SWIGLU, device="cpu")


def attn(**kw):
    a = dict(handle=None, Q=P, ld_q=1024, K=P, ld_k=256, V=P, ld_v=256, cu_q=P, k_start=P, k_len=P, scale=0.1, O=P, ld_o=1024, lse=P,
             tq=4, n=2, heads=8, kv_heads=2, tk=100, workspace=P, workspace_bytes=1 << 30, stream=0)
    dm.domino_attn_packed_fwd(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(tq=-1), INVALID), (dict(n=-1), INVALID), (dict(tk=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=3), INVALID), (dict(heads=129, kv_heads=1), UNSUPPORTED), (dict(heads=8192, kv_heads=8192), UNSUPPORTED),
    (dict(tq=1 << 31), UNSUPPORTED), (dict(tk=(1 << 31) - 1023), UNSUPPORTED), (dict(n=1 << 25), UNSUPPORTED),
    (dict(tq=1 << 30, heads=8, kv_heads=8), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(ld_q=1016), INVALID), (dict(ld_k=260), ALIGNMENT),
    (dict(ld_v=128), INVALID), (dict(ld_o=1025), ALIGNMENT), (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=P + 2), ALIGNMENT),
    (dict(O=P + 8), ALIGNMENT), (dict(lse=P + 4), ALIGNMENT), (dict(cu_q=None), INVALID), (dict(k_start=None), INVALID),
    (dict(k_len=P + 2), ALIGNMENT), (dict(workspace=None), WORKSPACE), (dict(workspace=P + 64), WORKSPACE),
    (dict(workspace_bytes=1000), WORKSPACE), (dict(), INVALID), (dict(cu_q=P + 4, lse=None, K=None, V=None, tk=0), INVALID)])
def test_packed_attention(kw, code):
    assert status(attn, **kw) == code


def test_packed_attention_workspace_size():
    size = dm.domino_attn_packed_workspace_size
    assert size(0, 4, 8, 2, 100) == 0 and size(4, 0, 8, 2, 100) == 0
    # keys too few to be cut: the list of work alone
    assert size(64, 64, 8, 2, 512) < 1 << 16
    # four partial tiles a CTA
    assert 0 < size(64, 64, 8, 2, 1 << 20) - 4 * 152 * 128 * (128 + 2) * 4 < 1 << 16
    assert status(size, tq=1, n=1, heads=3, kv_heads=2, tk=1) == INVALID


def test_packed_attention_function_refuses_what_it_cannot_take():
    q, cu = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.packed_attention(q, q, q, cu)
