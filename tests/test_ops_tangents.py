"""Forward-mode differentiation: the operators have no such derivative, and a tangent may not be lost without a word."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from comm_overlap_gb300 import torch_ops as ops

D = 128


def randn(*shape, device):
    return torch.randn(shape).to(torch.bfloat16).to(device)


def calls(device):
    """(name, arguments that may carry a tangent, call)"""
    x, w, b, r = randn(4, 64, device=device), randn(128, 64, device=device), randn(128, device=device), randn(4, 128, device=device)
    g, h = randn(64, device=device), randn(64, device=device)
    q = randn(4, 2, D, device=device)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=device)
    return [("layer_norm", (x, g, h), lambda x, g, h: ops.layer_norm(x, g, h)),
            ("linear", (x, w, b, r), lambda x, w, b, r: ops.linear(x, w, b, "gelu", r)),
            ("packed_attention", (q, q.clone(), q.clone()), lambda q, k, v: ops.packed_attention(q, k, v, cu))]


def check(device, grad):
    for name, args, call in calls(device):
        for i in range(len(args)):
            with torch.set_grad_enabled(grad), forward_ad.dual_level():
                dual = list(args)
                dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                assert not dual[i].requires_grad
                with pytest.raises(NotImplementedError, match=name):
                    call(*dual)


@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(grad):
    check("cpu", grad)


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused_on_the_gpu(grad):
    from comm_overlap_gb300 import build
    build.build()
    check("cuda", grad)
    # within a level, tensors without a tangent are served as ever
    for name, args, call in calls("cuda"):
        with torch.no_grad():
            want = call(*args)
            with forward_ad.dual_level():
                assert torch.equal(call(*args), want), name
