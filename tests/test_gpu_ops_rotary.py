"""Norm and rotation of query and key heads, forward and backward, and the 8-bit cache written and read, against the
definitions in 64 bits.

fp32 slop (in units U32 of the magnitudes): a norm's factor is a sum of 128 squares (each lane 8 + 8 in two chains, 3
shuffles: at most 13 roundings), rsqrt (2 ulp = 4 halves) and two products: under 24; an angle's distance from a quarter turn is
rounded to 24 bits, pi / 4 units of the pair's size at most, and sincospif is good to 2 ulp: under pi + 4, the rotation itself 3.  40 covers them.  The backward
adds a dot product of 128 terms (19 roundings) and three products to each side: 80."""
import pytest
import torch

from cache_helpers import D, cos_sin, e4m3, exponents, held, power, random_cache, rotary, rotary_grad, turn, values
from ops_helpers import BF16, U32, close, device_ok, randn

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


def inputs(ops, tokens, hq, hkv, rot, norm, seed=0, far=5000):
    qkv = randn(tokens, hq + 2 * hkv, D, seed=seed)
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, far, (tokens,), generator=g, dtype=torch.int32).cuda() if rot else None
    freq = ops.rotary_frequencies(rot, 10000.0) if rot else None
    wq, wk = (randn(D, seed=seed + 1, std=0.3, mean=1.0), randn(D, seed=seed + 2, std=0.3, mean=1.0)) if norm else (None, None)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, freq, wq, wk


SHAPES = [(1, 32, 8), (1, 1, 1), (3, 5, 5), (7, 16, 1), (65, 7, 2), (1000, 28, 4)]
ROTS = [(128, "half"), (128, "interleaved"), (64, "half"), (16, "half"), (96, "interleaved"), (112, "half"), (0, "half")]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot,layout", ROTS)
@pytest.mark.parametrize("tokens,hq,hkv", SHAPES)
def test_forward(ops, tokens, hq, hkv, rot, layout, norm):
    q, k, _, pos, freq, wq, wk = inputs(ops, tokens, hq, hkv, rot, norm)
    amplitude = 1.0 if rot < 100 else 1.25
    yq, yk = ops.qk_rotary_fwd(q, k, pos, freq, wq, wk, layout, amplitude=amplitude)
    for y, x, w in ((yq, q, wq), (yk, k, wk)):
        ref, size = rotary(x, w, pos, freq, layout, amplitude=amplitude)
        if rot == 0 and not norm:
            assert torch.equal(y, x)
        close(y, ref, 40 * U32 * size, what=f"{tokens} {hq} {hkv}")
    device_ok()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot,layout", ROTS)
@pytest.mark.parametrize("tokens,hq,hkv", SHAPES)
def test_backward(ops, tokens, hq, hkv, rot, layout, norm):
    q, k, _, pos, freq, wq, wk = inputs(ops, tokens, hq, hkv, rot, norm)
    gq, gk = randn(tokens, hq, D, seed=5), randn(tokens, hkv, D, seed=6)
    got = ops.qk_rotary_bwd(gq, gk, q, k, pos, freq, wq, wk, layout, amplitude=0.75 if rot else 1.0)
    for i, (gy, x, w) in enumerate(((gq, q, wq), (gk, k, wk))):
        gx, gw, size, wsize = rotary_grad(gy, x, w, pos, freq, layout, amplitude=0.75 if rot else 1.0)
        close(got[i], gx, 80 * U32 * size, what=f"g{i}")
        if norm:  # a lane adds up its heads (at most all of the tokens' groups of four), then lanes, warps, blocks
            chain = tokens * -(-(hq if i == 0 else hkv) // 4)
            close(got[2 + i], gw, (60 + min(chain, 400) + 100) * U32 * wsize, rounding=U32, what=f"w{i}")
        else:
            assert got[2 + i] is None
    device_ok()


def test_gradients_match_differences(ops):
    """<gy, y(x + e d) - y(x - e d)> / 2 e in 64 bits against <gx, d>: the definition used above is the forward's gradient."""
    q, k, _, pos, freq, wq, wk = inputs(ops, 3, 4, 2, 64, True, seed=3)
    gy, d, dw = (randn(3, 4, D, seed=i).double() for i in (7, 8, 9))
    dw = dw[0, 0]
    gx, gw, _, _ = rotary_grad(gy, q, wq, pos, freq, "interleaved", amplitude=1.5)
    e = 1e-6
    up, _ = rotary(q.double() + e * d, wq.double() + e * dw, pos, freq, "interleaved", amplitude=1.5)
    down, _ = rotary(q.double() - e * d, wq.double() - e * dw, pos, freq, "interleaved", amplitude=1.5)
    want = ((up - down) * gy).sum() / (2 * e)
    have = (gx * d).sum() + (gw * dw).sum()
    assert abs(want - have) <= 1e-6 * (gx * d).abs().sum()


def test_far_positions(ops):
    """Angles keep their digits at any int32 position, and turn the other way for negative ones.  The reference takes the
    fraction of a turn by whole numbers of any size."""
    from fractions import Fraction
    pos = torch.tensor([0, 1, -1, 999_983, 123_456_789, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    freq = ops.rotary_frequencies(128, 500000.0)
    x = randn(len(pos), 4, D, seed=1)
    y, _ = ops.qk_rotary_fwd(x, None, pos, freq)
    # 1 / (2 pi) to 60 digits
    inverse = Fraction(159154943091895335768883763372514362034459645740456448747667, 10**60)
    turns = [[float((int(p) * Fraction(float(f)) * inverse) % 1) for f in freq.cpu()] for p in pos.cpu()]
    angle = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64, device="cuda")
    ref = turn(x.double(), angle.cos(), angle.sin(), "half")
    size = x.double().abs()
    size[..., :64] += x.double().abs()[..., 64:]
    size[..., 64:] += x.double().abs()[..., :64]
    # the frequency itself, as a fraction of a turn, is good to 2^-53: 2^31 positions x 0.16 turns x 2 pi x 2^-53 < 2^-21
    close(y, ref, (40 * U32 + 2.0 ** -21) * size)


def test_strides_in_place_and_given_outputs(ops):
    q, k, v, pos, freq, wq, wk = inputs(ops, 33, 6, 3, 128, True, seed=4)
    yq, yk = ops.qk_rotary_fwd(q, k, pos, freq, wq, wk)
    wide = torch.full((33, 9, D), 7.0, dtype=BF, device="cuda")
    a, b = ops.qk_rotary_fwd(q.contiguous(), k.contiguous(), pos, freq, wq, wk, out=(wide[:, :6], wide[:, 6:]))
    assert torch.equal(a, yq) and torch.equal(b, yk) and torch.equal(wide[:, :6], yq) and torch.equal(wide[:, 6:], yk)
    odd = torch.empty(33 * 6 * D + 1, dtype=BF, device="cuda")[1:].view(33, 6, D)  # not 16-byte aligned: copied
    odd.copy_(q)
    assert torch.equal(ops.qk_rotary_fwd(odd, None, pos, freq, wq)[0], yq)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)  # heads first: copied
    assert torch.equal(ops.qk_rotary_fwd(turned, None, pos, freq, wq)[0], yq)
    v_was = v.clone()
    ops.qk_rotary_fwd(q, k, pos, freq, wq, wk, out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(v, v_was)
    with pytest.raises(ValueError, match="overlap"):
        ops.qk_rotary_fwd(q, None, pos, freq, wq, out=(turned, None))


def test_extreme_heads(ops):
    """Heads whose squares leave fp32's range, zeros, infinities and NaN: each concerns its own head alone."""
    x = randn(6, 8, D, seed=2)
    x[0, 0] *= 2.0 ** 100
    x[1, 1] = 0
    x[2, 2] *= 2.0 ** -100
    x[3, 3, 5] = float("inf")
    x[4, 4, 7] = float("nan")
    x[5, 5] = 3.0e38
    w = randn(D, seed=3, std=0.2, mean=1.0)
    pos, freq = torch.arange(6, dtype=torch.int32, device="cuda"), ops.rotary_frequencies(64)
    y, _ = ops.qk_rotary_fwd(x, None, pos, freq, w)
    ref, size = rotary(x, w, pos, freq)
    fine = torch.ones(6, 8, dtype=torch.bool, device="cuda")
    fine[3, 3] = fine[4, 4] = False
    assert y[4, 4].isnan().all() and y[3, 3].isnan().any()
    close(y[fine], ref[fine], 40 * U32 * size[fine])
    gy = randn(6, 8, D, seed=4)
    gx, _, gw, _ = ops.qk_rotary_bwd(gy, None, x, None, pos, freq, w)
    ref, _, size, _ = rotary_grad(gy, x, w, pos, freq)
    # (2^-133 is bf16's smallest value: what lies below rounds to it or to zero)
    close(gx[fine], ref[fine], 80 * U32 * size[fine] + 2.0 ** -133)
    plain, _ = ops.qk_rotary_fwd(x, None, pos, freq)  # without norm, what is not rotated stays whatever it is
    assert torch.equal(plain[..., 64:].view(torch.int16), x[..., 64:].view(torch.int16))


def test_autograd_module_and_accumulation(ops):
    tokens, hq, hkv = 50, 8, 2
    m = ops.DominoQKRotary(64, 500000.0, "interleaved", amplitude=1.1, factor=8.0, original=8192)
    assert m.frequencies.dtype == torch.float64
    m = m.to(BF)
    assert m.frequencies.dtype == torch.float64
    qkv = randn(tokens, hq + 2 * hkv, D, seed=6).requires_grad_()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") + 30000
    yq, yk = m(qkv[:, :hq], qkv[:, hq:hq + hkv], pos)
    gq, gk = randn(tokens, hq, D, seed=7), randn(tokens, hkv, D, seed=8)
    torch.autograd.backward([yq, yk], [gq, gk])
    plain = ops.qk_rotary_bwd(gq, gk, qkv[:, :hq].detach(), qkv[:, hq:hq + hkv].detach(), pos, m.frequencies, m.q_weight.detach(),
                              m.k_weight.detach(), "interleaved", 1e-6, 1.1)
    assert torch.equal(qkv.grad[:, :hq], plain[0]) and torch.equal(qkv.grad[:, hq:hq + hkv], plain[1])
    assert not qkv.grad[:, hq + hkv:].any()
    assert torch.equal(m.q_weight.grad, plain[2].to(BF)) and torch.equal(m.k_weight.grad, plain[3].to(BF))
    buffers = torch.ones(D, device="cuda"), torch.full((D,), 2.0, device="cuda")
    again = ops.qk_rotary_bwd(gq, gk, qkv[:, :hq].detach(), qkv[:, hq:hq + hkv].detach(), pos, m.frequencies, m.q_weight.detach(),
                              m.k_weight.detach(), "interleaved", 1e-6, 1.1, grads=buffers)
    assert again[2] is buffers[0] and torch.equal(buffers[0], plain[2] + 1) and torch.equal(buffers[1], plain[3] + 2)
    bare = ops.DominoQKRotary(128, norm=False)
    assert not list(bare.parameters())
    x = randn(3, 2, D, seed=9).requires_grad_()
    y, none = ops.qk_rotary(x, None, pos[:3], bare.frequencies)
    y.backward(torch.ones_like(y))
    assert none is None and x.grad is not None


def test_offsets_beyond_32_bits(ops):
    """Three tokens 1.2e9 elements apart in inputs and outputs."""
    step, far = 1_200_000_000, 2_400_000_000 + 4096
    big, out = (torch.empty(far, dtype=BF, device="cuda") for _ in range(2))
    view = lambda t, at, h: t.as_strided((3, h, D), (step, D, 1), at)
    q, k, pos, freq = randn(3, 16, D, seed=1), randn(3, 4, D, seed=2), torch.tensor([5, 70000, 3], dtype=torch.int32, device="cuda"), ops.rotary_frequencies(128)
    wq, wk = randn(D, seed=3, mean=1.0), randn(D, seed=4, mean=1.0)
    view(big, 0, 16).copy_(q), view(big, 2048, 4).copy_(k)
    want = ops.qk_rotary_fwd(q, k, pos, freq, wq, wk)
    got = ops.qk_rotary_fwd(view(big, 0, 16), view(big, 2048, 4), pos, freq, wq, wk, out=(view(out, 0, 16), view(out, 2048, 4)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = ops.qk_rotary_bwd(*got, view(big, 0, 16), view(big, 2048, 4), pos, freq, wq, wk)
    again = ops.qk_rotary_bwd(*ops.qk_rotary_fwd(q, k, pos, freq, wq, wk), q, k, pos, freq, wq, wk)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    cache, other = ops.QuantizedCache.empty(3, 4), ops.QuantizedCache.empty(3, 4)
    rows = torch.arange(3, dtype=torch.int32, device="cuda")
    y = ops.cache_write(cache, rows, view(big, 2048, 4), view(big, 2048, 4), view(big, 0, 16), pos, freq, wq, wk)
    assert torch.equal(y, ops.cache_write(other, rows, k, k, q, pos, freq, wq, wk))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, other))
    kk, vv = ops.cache_read(cache, rows, out=(view(out, 0, 4), view(out, 2048, 4)))
    assert all(torch.equal(a, b) for a, b in zip((kk, vv), ops.cache_read(other, rows)))
    device_ok()


def test_gradients_of_one_value(ops):
    """Gradients that are one value everywhere, without strides, and outputs of which one alone is used."""
    q, k = randn(9, 4, D, seed=1).requires_grad_(), randn(9, 2, D, seed=2).requires_grad_()
    m, pos = ops.DominoQKRotary(64), torch.arange(9, dtype=torch.int32, device="cuda")
    yq, yk = m(q, k, pos)
    yq.sum().backward()
    want = ops.qk_rotary_bwd(torch.ones(9, 4, D, dtype=BF, device="cuda"), torch.zeros(9, 2, D, dtype=BF, device="cuda"), q.detach(), k.detach(),
                             pos, m.frequencies, m.q_weight.detach(), m.k_weight.detach())
    assert torch.equal(q.grad, want[0]) and not k.grad.any() and torch.equal(m.q_weight.grad, want[2].to(BF)) and not m.k_weight.grad.any()
    with torch.no_grad():
        assert not m(q, k, pos)[0].requires_grad
    q.grad = None
    x, _ = ops.qk_rotary(q, None, pos, m.frequencies, m.q_weight)
    x.backward(torch.ones_like(x))
    assert torch.equal(q.grad, want[0])


def test_no_tokens(ops):
    q, freq, w = torch.empty(0, 4, D, dtype=BF, device="cuda"), ops.rotary_frequencies(128), randn(D)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    yq, yk = ops.qk_rotary_fwd(q, q, pos, freq, w, w)
    assert yq.shape == q.shape and yk.shape == q.shape
    _, _, gwq, gwk = ops.qk_rotary_bwd(q, q, q, q, pos, freq, w, w)
    assert not gwq.any() and not gwk.any()
    cache = ops.QuantizedCache.empty(10, 4)
    assert ops.cache_write(cache, pos, q, q, q, pos, freq, w, w).shape == q.shape
    assert ops.cache_read(cache, pos)[0].shape == (0, 4, D)
    none = ops.QuantizedCache.empty(0, 4)
    k, v = ops.cache_read(none, torch.tensor([-1], dtype=torch.int32, device="cuda"))
    assert not k.any() and not v.any()


# ---- the cache

@pytest.mark.parametrize("tokens,hkv", [(1, 1), (1, 8), (9, 3), (130, 4), (1000, 5)])
def test_written_as_is_and_read_back(ops, tokens, hkv):
    """Without norm and rotation the codes are a function of bf16 values: exact."""
    k = randn(tokens, hkv, D, seed=1) * torch.exp2(torch.arange(tokens) % 90 - 45.0).cuda().to(BF)[:, None, None]
    v = randn(tokens, hkv, D, seed=2)
    cache = random_cache(tokens + 37, hkv, seed=3)
    was = [t.clone() for t in cache]
    g = torch.Generator().manual_seed(4)
    rows = torch.randperm(tokens + 37, generator=g)[:tokens].int().cuda()
    assert ops.cache_write(cache, rows, k, v) is None
    gk, gv = ops.cache_read(cache, rows)
    for got, x, e in ((gk, k, cache.k_exp), (gv, v, cache.v_exp)):
        assert torch.equal(got.double(), held(x.double()))
        assert torch.equal(e[:, rows.long()].t().int() - 127, exponents(x.double()).int())
    others = torch.ones(tokens + 37, dtype=torch.bool, device="cuda")
    others[rows.long()] = False
    for now, before in zip(cache, was):
        a, b = (t.view(torch.uint8) for t in (now, before))
        a, b = (a[others], b[others]) if a.dim() == 3 else (a[:, others], b[:, others])
        assert torch.equal(a, b)
    device_ok()


@pytest.mark.parametrize("tokens,hq,hkv,rot,layout,norm", [
    (1, 32, 8, 128, "half", True), (64, 32, 8, 128, "half", True), (777, 28, 4, 64, "interleaved", False), (5, 3, 1, 16, "half", False),
    (33, 5, 5, 96, "interleaved", True), (40, 4, 2, 0, "half", True)])
def test_written_with_norm_and_rotation(ops, tokens, hq, hkv, rot, layout, norm):
    q, k, v, pos, freq, wq, wk = inputs(ops, tokens, hq, hkv, rot, norm, seed=11)
    cache = ops.QuantizedCache.empty(tokens + 5, hkv)
    rows = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device="cuda") + 2
    y = ops.cache_write(cache, rows, k, v, q, pos, freq, wq, wk, layout)
    want, _ = ops.qk_rotary_fwd(q, k, pos, freq, wq, wk, layout)
    assert torch.equal(y, want)
    gk, gv = ops.cache_read(cache, rows)
    assert torch.equal(gv.double(), held(v.double()))
    ref, size = rotary(k, wk, pos, freq, layout)
    p = power(exponents(ref))[..., None]
    # half a step of E4M3 at the value itself; at a border of the power of two the other scale has the same steps, but for
    # the smallest values, whose step may double
    half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -9 * p)
    assert ((gk.double() - ref).abs() <= half + 40 * U32 * size).all()
    same = (gk.double() == held(ref)).double().mean()
    assert same > 0.999
    device_ok()


def test_written_special_values(ops):
    k = randn(8, 1, D, seed=1)
    k[0] = 0
    k[1, 0, 3] = float("inf")
    k[2, 0, 4] = float("nan")
    k[3] = 3.0e38
    k[4] = 2.0 ** -120
    k[5, 0, :] = 448.0
    k[6, 0, :] = 449.0 * 2  # rounds to 896 or 900 in bf16: above 1.75 x 2^9
    k[6, 0, 0] = 904.0
    k[7] = -0.0
    cache = ops.QuantizedCache.empty(8, 1)
    rows = torch.arange(8, dtype=torch.int32, device="cuda")
    ops.cache_write(cache, rows, k, k)
    got, _ = ops.cache_read(cache, rows)
    e = cache.k_exp[0].int().cpu() - 127
    assert e[0] == 0 and e[3] == 51 and e[4] == -51 and e[5] == 0 and e[6] == 2 and e[7] == 0
    assert not got[0].any() and not got[4].any() and not got[7].any()
    assert got[1, 0, 3].isnan() and got[1].isnan().sum() == 1 and got[2, 0, 4].isnan() and got[2].isnan().sum() == 1
    for i in (1, 2):
        x = k[i].double().clone()
        x[~x.isfinite()] = 0
        keep = k[i].isfinite()
        assert torch.equal(got[i].double()[keep], held(x)[keep])
    assert (got[3].double() == 448 * 2.0 ** 51).all()
    assert torch.equal(got[5], k[5])
    assert torch.equal(e4m3(got[5].double()), k[5].double())


def test_rows_beyond_and_negative(ops):
    from comm_overlap_gb300 import domino as dm
    k, v = randn(4, 2, D, seed=1), randn(4, 2, D, seed=2)
    cache = random_cache(10, 2, seed=5)
    was = [t.clone() for t in cache]
    rows = torch.tensor([3, -1, -5, 7], dtype=torch.int32, device="cuda")
    ops.cache_write(cache, rows, k, v)
    device_ok()
    touched = torch.zeros(10, dtype=torch.bool, device="cuda")
    touched[[3, 7]] = True
    assert torch.equal(cache.k.view(torch.uint8)[~touched], was[0].view(torch.uint8)[~touched])
    gk, gv = ops.cache_read(cache, rows)
    assert not gk[1:3].any() and not gv[1:3].any() and torch.equal(gk[0].double(), held(k[0].double()))
    was = [t.clone() for t in cache]
    ops.cache_write(cache, torch.tensor([10, 2**31 - 1, -1, -1], dtype=torch.int32, device="cuda"), k, v)
    with pytest.raises(dm.DominoError, match="INVALID_ARG"):
        ops.device_status()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, was))
    gk, _ = ops.cache_read(cache, torch.tensor([10, 0], dtype=torch.int32, device="cuda"))
    assert not gk[0].any() and torch.equal(gk[1].double(), values(cache, "k", [0])[0])
    with pytest.raises(dm.DominoError, match="INVALID_ARG"):
        ops.device_status()
    ops.device_status()


def test_layers_of_one_cache_and_given_outputs(ops):
    """A layer of a larger cache, its exponents with a stride; outputs and sources that are slices."""
    layers, rows, hkv = 3, 20, 4
    codes = torch.zeros(2, layers, rows, hkv, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    exps = torch.full((2, layers, hkv, rows + 12), 127, dtype=torch.uint8, device="cuda")
    layer = ops.QuantizedCache(codes[0, 1], codes[1, 1], exps[0, 1, :, 5:25], exps[1, 1, :, 5:25])
    qkv = randn(6, 12, D, seed=3)
    at = torch.tensor([0, 19, 4, 3, 2, 1], dtype=torch.int32, device="cuda")
    ops.cache_write(layer, at, qkv[:, 4:8], qkv[:, 8:])
    both = torch.full((6, 9, D), 5.0, dtype=BF, device="cuda")
    k, v = ops.cache_read(layer, at, out=(both[:, :4], both[:, 4:8]))
    assert torch.equal(k.double(), held(qkv[:, 4:8].double())) and torch.equal(v.double(), held(qkv[:, 8:].double()))
    assert (both[:, 8] == 5).all()
    assert not codes.view(torch.uint8)[:, [0, 2]].any() and (exps[:, [0, 2]] == 127).all()
    assert (exps[:, 1, :, :5] == 127).all() and (exps[:, 1, :, 25:] == 127).all()


def test_same_bits_again(ops):
    q, k, v, pos, freq, wq, wk = inputs(ops, 3000, 16, 4, 128, True, seed=8)
    gq, gk = randn(3000, 16, D, seed=5), randn(3000, 4, D, seed=6)
    first = ops.qk_rotary_bwd(gq, gk, q, k, pos, freq, wq, wk)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, ops.qk_rotary_bwd(gq, gk, q, k, pos, freq, wq, wk)))
    assert BF16 == 2.0 ** -8 and cos_sin(None, None) == (None, None)
