"""Angles of the rotation, each to fp32's precision for itself: slow pairs at small positions, angles next to quarter turns."""
import math

import pytest
import torch

from cache_helpers import D
from ops_helpers import BF16, device_ok

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def ops():
    from comm_overlap_gb300 import torch_ops
    return torch_ops


def parts(ops, positions, f, layout, way):
    """Cosines and sines [tokens, 64] as the rotation of (1, 0) gives them, forward or back."""
    x = torch.zeros(len(positions), 1, D, dtype=BF, device="cuda")
    a, b = (slice(0, 64), slice(64, 128)) if layout == "half" else (slice(0, D, 2), slice(1, D, 2))
    x[..., a] = 1
    if way == "forward":
        y = ops.qk_rotary_fwd(x, None, positions, f, layout=layout)[0]
    else:
        y = ops.qk_rotary_bwd(x, None, None, None, positions, f, layout=layout)[0]
    return y[:, 0, a].double(), y[:, 0, b].double() * (1 if way == "forward" else -1)


def check(ops, positions, f, angle, layout, way):
    """Against the angles [tokens, 64] in 64 bits.  Each value is rounded once to bf16; before it the fraction of a turn, the product with
    pi and sincospif's two results are off by a few 2^-24 of themselves (2^-20 here), and the angle by the position times the rounding of
    its frequency's turns to 53 bits, 2^-52 of them."""
    far = 2.0 ** -52 * positions.double().abs()[:, None] * f.abs()
    for got, ref, size in zip(parts(ops, positions, f, layout, way), (angle.cos(), angle.sin()), (angle.sin(), angle.cos())):
        slop = 2.0 ** -20 * ref.abs() + far * size.abs()
        assert ((got - ref).abs() <= BF16 * ref.abs() + (1 + BF16) * slop).all(), float(((got - ref).abs() / ref.abs()).max())
    device_ok()


@pytest.mark.parametrize("way", ["forward", "back"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("factor", [1.0, 8.0, 4096.0])
def test_slow_pairs_at_small_positions(ops, factor, layout, way):
    positions = torch.cat([torch.arange(1, 21), -torch.arange(1, 21)]).int().cuda()
    f = ops.rotary_frequencies(D, 500000.0, factor=factor)
    check(ops, positions, f, positions.double()[:, None] * f, layout, way)


@pytest.mark.parametrize("quarter", [1, 2, 3, -1, -2])
def test_next_to_quarter_turns(ops, quarter):
    """quarter turns and 2^-16 to 2^-36 of a radian: the smaller of cosine and sine is that."""
    little = torch.exp2(-16 - 20 * torch.arange(64, dtype=torch.float64) / 63) * torch.where(torch.arange(64) % 2 == 0, 1.0, -1.0)
    f = (quarter * (math.pi / 2) + little).cuda()
    # what is left of f beside the quarter turns, pi / 2 taken to 2^-107
    rest = (f - quarter * (math.pi / 2)) - quarter * 6.123233995736766e-17
    positions = torch.ones(3, dtype=torch.int32, device="cuda")
    got = parts(ops, positions, f, "half", "forward")
    near = [(rest.cos(), rest.sin()), (-rest.sin(), rest.cos()), (-rest.cos(), -rest.sin()), (rest.sin(), -rest.cos())][quarter % 4]
    for x, ref in zip(got, near):
        # the turns are rounded to 53 bits, which is 2^-53 of `quarter` quarter turns
        assert ((x - ref).abs() <= BF16 * ref.abs() + (1 + BF16) * (2.0 ** -20 * ref.abs() + 2.0 ** -51 * abs(quarter) * math.pi / 2)).all()
    device_ok()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_frequencies_that_are_not_finite(ops, layout):
    """Their pairs are NaN at every position, forward and back, and no others."""
    f = ops.rotary_frequencies(D)
    broken = f.clone()
    broken[3], broken[17], broken[63] = float("nan"), float("inf"), -float("inf")
    hit = torch.zeros(64, dtype=torch.bool, device="cuda")
    hit[[3, 17, 63]] = True
    positions = torch.tensor([0, 1, -5, 100000], dtype=torch.int32, device="cuda")
    for way in ("forward", "back"):
        for got, want in zip(parts(ops, positions, broken, layout, way), parts(ops, positions, f, layout, way)):
            assert got[:, hit].isnan().all() and torch.equal(got[:, ~hit], want[:, ~hit])
    x, w = torch.ones(4, 2, D, dtype=BF, device="cuda"), torch.ones(D, dtype=BF, device="cuda")
    g, _, gw, _ = ops.qk_rotary_bwd(x, None, x, None, positions, broken, w, layout=layout)
    gw = gw.view(2, 64).t() if layout == "half" else gw.view(64, 2)
    assert g.isnan().all() and gw[hit].isnan().all() and gw[~hit].isfinite().all()
    cache = ops.QuantizedCache.empty(4, 2)
    ops.cache_write(cache, torch.arange(4, dtype=torch.int32, device="cuda"), x, x, None, positions, broken, layout=layout)
    k, v = ops.cache_read(cache, torch.arange(4, dtype=torch.int32, device="cuda"))
    k = k.unflatten(-1, (2, 64)).movedim(-2, -1) if layout == "half" else k.unflatten(-1, (64, 2))
    assert k[:, :, hit].isnan().all() and k[:, :, ~hit].isfinite().all() and torch.equal(v, x)
    device_ok()
