"""Shared by the sublayer operators' GPU tests: inputs, 64-bit references' comparisons.

A value rounded once to bf16 is off by at most half a step, 2^-8 of it; everything before that rounding
is fp32 arithmetic, whose bound each test derives (`slop`, in units of 2^-24 of the magnitudes summed).
"""
import torch

BF16 = 2.0 ** -8
U32 = 2.0 ** -24


def randn(*shape, seed=0, std=1.0, mean=0.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cpu").manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def close(got, ref, slop, rounding=BF16, what=""):
    """|got - ref| <= rounding |ref| + slop (+ slop's own rounding), element by element."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.numel() == 0:
        return
    slop = torch.as_tensor(slop, dtype=torch.float64, device=ref.device)
    bad = ~((got - ref).abs() <= rounding * ref.abs() + (1 + rounding) * slop)
    if bad.any():
        i = int((((got - ref).abs() - rounding * ref.abs()) / (slop + 1e-300)).nan_to_num(1e300).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst at {i}: "
                             f"{got.reshape(-1)[i].item()!r} for {ref.reshape(-1)[i].item()!r}, "
                             f"slop {slop.expand_as(ref).reshape(-1)[i].item():.3g}")


def device_ok():
    """No kernel's wait ran out since the last look."""
    from comm_overlap_gb300 import domino as dm
    from comm_overlap_gb300 import torch_ops as ops
    for h in ops._handles.values():
        st, site = dm.domino_device_status(h)
        assert st == 0, f"device error word {site:#x}"
