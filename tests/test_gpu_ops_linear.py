"""The linear layer, forward and backward, against its definition in 64 bits.

The tensor core adds K / 16 groups of sixteen exact products to an fp32 accumulator that may truncate: each
addition is off by at most 2^-23 of the running magnitude, each group of sixteen by as much again.  `mma`
below is that bound.  Phi by Abramowitz & Stegun 7.1.26 with CUDA's fast exponential and division is off
by less than 1e-6, act' by less than 2e-6."""
import pytest
import torch

from ops_helpers import BF16, U32, close, device_ok, randn

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


def mma(k, a, b):
    """Bound of the accumulation's error of a @ b.t() (64-bit magnitudes) over k terms."""
    return (k / 8 + 96) * 2.0 ** -23 * (a.double().abs() @ b.double().abs().t())


def act64(act, z):
    return {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "gelu": lambda t: t * torch.special.ndtr(t)}[act](z)


def grad64(act, z):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    return torch.ones_like(z)


def check_fwd(x, w, b, act, r, y, z):
    zd = x.double() @ w.double().t() + (b.double() if b is not None else 0)
    s = mma(x.shape[1], x, w) + 2 * U32 * zd.abs()
    if z is not None:
        close(z, zd, s, what="z")
    yd = act64(act, zd)
    sy = 1.13 * s + (1e-6 * zd.abs() if act == "gelu" else 0)
    if r is not None:
        sy = sy + 2 * U32 * (yd.abs() + r.double().abs())
        yd = yd + r.double()
    close(y, yd, sy, what="y")


# one step of the reduction and fewer; tiles' edges in every direction and width; one row to several rounds of tiles; few
# tiles, whose reduction is cut over clusters of two and four pairs
SIZES = [(1, 8, 8), (2, 40, 56), (31, 248, 72), (33, 264, 512), (127, 256, 520), (129, 512, 576), (255, 8, 1096),
         (257, 2560, 264), (1, 4096, 4096), (5, 16384, 1024), (300, 768, 8192), (777, 2560, 2560), (5000, 2056, 264),
         (5000, 2056, 1096), (4864, 4096, 128)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act,bias,res,save", [("gelu", True, False, True), ("none", False, True, False),
                                               ("relu", True, True, True), ("none", False, False, False)])
def test_forward(ops, m, n, k, act, bias, res, save):
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5)
    b, r = randn(n, seed=3) if bias else None, randn(m, n, seed=4) if res else None
    y, z = ops.linear_fwd(x, w, b, act, r, save=save)
    assert (z is not None) == save
    check_fwd(x, w, b, act, r, y, z)
    y2, z2 = ops.linear_fwd(x, w, b, act, r, save=save)
    assert torch.equal(y, y2) and (z is None or torch.equal(z, z2))


def ints(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (300, 520, 256), (129, 264, 200), (2500, 1040, 136)])
def test_small_integers_are_exact(ops, m, n, k):
    """Sums of at most 256 terms of -1, 0, 1 are exact in bf16: any misplaced element shows."""
    x, w, gy = ints(m, k, seed=1), ints(n, k, seed=2), ints(m, n, seed=3)
    y, _ = ops.linear_fwd(x, w)
    assert torch.equal(y.double(), x.double() @ w.double().t())
    few = gy * (torch.rand(m, n, generator=torch.Generator().manual_seed(5)).cuda() < 0.05)  # sums below 256
    gx, gw, gb = ops.linear_bwd(few, x, w)
    want = (few.double() @ w.double(), few.double().t() @ x.double(), few.double().sum(0))
    assert max(float(t.abs().max()) for t in want[:2]) <= 256
    for got, t in zip((gx, gw, gb), want):
        assert torch.equal(got.double(), t)


def bf16_pair(lo, hi):
    return lo.to(torch.bfloat16).double(), hi.to(torch.bfloat16).double()


def check_bwd(gy, x, w, z, act, gx, gw, gb, gw_start=None, gb_start=None):
    m, n = gy.shape
    k = x.shape[1]
    g = gy.double()
    gz = g * grad64(act, z.double()) if act != "none" else g
    delta = (2e-6 if act == "gelu" else 0) * g.abs() + 2 * U32 * gz.abs() if act != "none" else torch.zeros_like(g)
    # the rounding of gZ: where the kernel's fp32 value may round the other way, the difference counts
    lo, hi = bf16_pair((gz - delta).float(), (gz + delta).float())
    mid, flip = gz.float().to(torch.bfloat16).double(), (hi - lo).abs()
    if gx is not None:
        close(gx, mid @ w.double(), mma(n, mid, w.t()) + flip @ w.double().abs(), what="gx")
    if gw is not None:
        want, slop = mid.t() @ x.double(), mma(m, mid.t(), x.t()) + flip.t() @ x.double().abs()
        if gw_start is None:
            close(gw, want, slop, what="gweight")
        else:
            close(gw, want + gw_start.double(), slop + U32 * (want.abs() + gw_start.double().abs()), rounding=0, what="gweight")
    if gb is not None:
        start = gb_start.double() if gb_start is not None else 0
        depth = m / 8 + 300  # additions a column's sum passes through: rows of a warp, warps, row ranges
        close(gb, gz.sum(0) + start, delta.sum(0) + depth * U32 * (gz.abs().sum(0) + abs(start)), rounding=0, what="gbias")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act", ["gelu", "none", "relu"])
def test_backward(ops, m, n, k, act):
    x, w, gy = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5), randn(m, n, seed=3)
    z = randn(m, n, seed=4) if act != "none" else None
    if z is not None:
        z[0, 0] = 0.0
    got = ops.linear_bwd(gy, x, w, z, act)
    check_bwd(gy, x, w, z, act, *got)
    assert all(torch.equal(a, b) for a, b in zip(got, ops.linear_bwd(gy, x, w, z, act)))


# few rows: whole and cut reductions (two and four parts), tiles of every height, several rounds of tiles, all of the 16-row
# chunks, and the first count that the kernel for many rows takes
FEW = [(1, 8, 4096), (2, 2560, 10240), (3, 6144, 4096), (7, 20000, 264), (16, 1024, 1096), (17, 4096, 2056), (47, 9728, 520),
       (64, 4608, 2048), (64, 6144, 1032), (50, 39000, 72), (65, 4096, 1096)]


@pytest.mark.parametrize("m,n,k", FEW)
@pytest.mark.parametrize("act,bias,res,save", [("gelu", True, False, True), ("none", False, True, False), ("relu", True, True, True)])
def test_few_rows(ops, m, n, k, act, bias, res, save):
    """Strided inputs and outputs whose other columns and rows stay as they were; junk behind X's rows."""
    x = torch.full((m + 3, k + 8), float("nan"), dtype=torch.bfloat16, device="cuda")[:m, :k]
    x.copy_(randn(m, k, seed=1))
    w = randn(n, k, seed=2, std=k ** -0.5)
    b = randn(n, seed=3) if bias else None
    r = randn(m, n + 8, seed=4)[:, :n] if res else None
    y, z = ops.linear_fwd(x, w, b, act, r, save=save)
    check_fwd(x, w, b, act, r, y, z)
    again, _ = ops.linear_fwd(x, w, b, act, r, save=save)
    assert torch.equal(y, again)


# rows of both operands that begin between 128-byte lines: pairs of tiles side by side, an odd count of tiles in either
# direction, one to several rounds, fewer steps than the ring has stages, rows in the second half of the last tile alone
@pytest.mark.parametrize("m,n,k", [(129, 520, 72), (400, 264, 1032), (385, 2568, 2568), (777, 2568, 520), (1300, 4104, 1032),
                                   (5000, 1544, 328), (2049, 8200, 200)])
@pytest.mark.parametrize("act", ["gelu", "none"])
def test_rows_between_lines(ops, m, n, k, act):
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5)
    b, r, gy = randn(n, seed=3), randn(m, n, seed=4), randn(m, n, seed=5)
    y, z = ops.linear_fwd(x, w, b, act, None if act == "gelu" else r, save=act == "gelu")
    check_fwd(x, w, b, act, None if act == "gelu" else r, y, z)
    got = ops.linear_bwd(gy, x, w, z, act)
    check_bwd(gy, x, w, z, act, *got)
    assert torch.equal(y, ops.linear_fwd(x, w, b, act, None if act == "gelu" else r)[0])
    assert all(torch.equal(p, q) for p, q in zip(got, ops.linear_bwd(gy, x, w, z, act)))


def test_offsets_beyond_32_bits(ops):
    """Outputs, residual, Z and gZ of more than 2^31 values."""
    m, n, k = 270000, 8192, 72
    big = dict(device="cuda", dtype=torch.bfloat16)
    x, w, b, r = torch.randn(m, k, **big), randn(n, k, seed=2, std=0.1), randn(n, seed=3), torch.randn(m, n, **big)
    y, z = ops.linear_fwd(x, w, b, "gelu", r, save=True)
    rows = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 262145, 267001, m - 1], device="cuda")
    check_fwd(x[rows], w, b, "gelu", r[rows], y[rows], z[rows])
    gx, _, _ = ops.linear_bwd(r, x, w, z, "gelu", weight_grad=False, bias_grad=False)
    check_bwd(r[rows], x[rows], w, z[rows], "gelu", gx[rows], None, None)


@pytest.mark.parametrize("m,n,k", [(1, 1 << 20, 8), (1, 8, 1 << 20), (64, 8, 1 << 18), (100, 8, 1 << 18), (65, 1 << 17, 8), (300000, 8, 8)])
def test_extreme_shapes(ops, m, n, k):
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, std=k ** -0.5)
    y, _ = ops.linear_fwd(x, w)
    check_fwd(x, w, None, "none", None, y, None)
    gx, gw, _ = ops.linear_bwd(y, x, w, bias_grad=False)
    check_bwd(y, x, w, None, "none", gx, gw, None)


def test_few_rows_and_outputs_of_ones_own(ops):
    from comm_overlap_gb300 import domino as dm
    m, n, k = 5, 264, 520
    x, w, r = randn(m, k, seed=1), randn(n, k, seed=2, std=0.05), randn(m, n, seed=3)
    want, _ = ops.linear_fwd(x, w, None, "gelu", r)
    wide = torch.full((m + 2, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y = wide[1:m + 1, 8:n + 8]
    y.copy_(r)  # the residual's own place
    h = dm.domino_create()
    dm.domino_linear_fwd(h, x, k, w, None, dm.ACT_GELU, y, wide.stride(0), y, wide.stride(0), None, 0, m, n, k, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    dm.domino_destroy(h)
    assert torch.equal(y, want)
    rest = wide.clone()
    rest[1:m + 1, 8:n + 8] = 7.0
    assert (rest == 7.0).all()
    # a row of NaN stays a row of NaN
    x[2] = float("nan")
    got, _ = ops.linear_fwd(x, w, None, "gelu", r)
    keep = [0, 1, 3, 4]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[2]).all()


def test_parts_of_the_backward(ops):
    """Each gradient alone, and accumulation into fp32 buffers."""
    m, n, k = 333, 264, 1160
    x, w, gy, z = randn(m, k, seed=1), randn(n, k, seed=2), randn(m, n, seed=3), randn(m, n, seed=4)
    full = ops.linear_bwd(gy, x, w, z, "gelu")
    for i in range(3):
        one = ops.linear_bwd(gy, x, w, z, "gelu", *(i == j for j in range(3)))
        assert [o is not None for o in one] == [i == j for j in range(3)] and torch.equal(one[i], full[i])
    gw0, gb0 = randn(n, k, seed=5, dtype=torch.float32), randn(n, seed=6, dtype=torch.float32)
    gw, gb = gw0.clone(), gb0.clone()
    gx, none, same = ops.linear_bwd(gy, x, w, z, "gelu", main_grad=gw, bias_main_grad=gb)
    assert none is None and same is gb and torch.equal(gx, full[0])
    check_bwd(gy, x, w, z, "gelu", None, gw, gb, gw0, gb0)


def test_strides_and_outputs_left_alone(ops):
    """Column slices as inputs; outputs inside larger buffers, whose other elements stay as they were."""
    from comm_overlap_gb300 import domino as dm
    m, n, k = 77, 136, 200
    xw, rw = randn(m, 3 * k, seed=1), randn(m, n + 24, seed=2)
    x, r, w = xw[:, k:2 * k], rw[:, 8:8 + n], randn(n, k, seed=3)
    y, z = ops.linear_fwd(x, w, None, "gelu", r, save=True)
    check_fwd(x, w, None, "gelu", r, y, z)
    big = torch.full((m + 2, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[1:-1, 8:8 + n]
    ops._call(dm.domino_linear_fwd, x, x, xw.shape[1], w, None, dm.ACT_GELU, r, rw.shape[1], out, big.shape[1], None, 0, m, n, k)
    assert torch.equal(out, y)
    big[1:-1, 8:8 + n] = 7.0
    assert (big == 7.0).all()
    # the residual's buffer as the output
    r2 = r.clone()
    ops._call(dm.domino_linear_fwd, x, x, xw.shape[1], w, None, dm.ACT_GELU, r2, n, r2, n, None, 0, m, n, k)
    assert torch.equal(r2, y)
    # an output gradient broadcast over its rows
    e = r[:1].expand(m, n)
    check_bwd(e, x, w, None, "none", *ops.linear_bwd(e, x, w))


def test_no_rows(ops):
    w, x = randn(64, 128, seed=1), torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    y, z = ops.linear_fwd(x, w, None, "gelu", save=True)
    assert y.shape == z.shape == (0, 64)
    gx, gw, gb = ops.linear_bwd(y, x, w, z, "gelu")
    assert gx.shape == (0, 128) and not gw.any() and not gb.any()


def test_nonfinite_rows_stay_apart(ops):
    m, n, k = 300, 520, 1040
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, std=0.03)
    clean, _ = ops.linear_fwd(x, w, None, "gelu")
    x[7, 3], x[260, 0] = float("nan"), float("inf")
    y, _ = ops.linear_fwd(x, w, None, "gelu")
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[[7, 260]] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[7]).all()


def test_autograd_and_differences(ops):
    m, n, k = 40, 72, 136
    layer = ops.DominoLinear(k, n, act="gelu")
    with torch.no_grad():
        layer.weight.copy_(randn(n, k, seed=1, std=0.1))
        layer.bias.copy_(randn(n, seed=2))
    x, r, gy = randn(2, m // 2, k, seed=3).requires_grad_(), randn(2, m // 2, n, seed=4).requires_grad_(), randn(2, m // 2, n, seed=5)
    layer(x, r).backward(gy)
    x64, w64, b64 = (t.detach().double().requires_grad_() for t in (x.view(m, k), layer.weight, layer.bias))
    (act64("gelu", x64 @ w64.t() + b64) * gy.view(m, n).double()).sum().backward()
    assert torch.equal(r.grad, gy)
    # Z and gZ are each rounded to bf16 on the way (half a step, |act''| < 0.8 and |z| < 8)
    for got, want in ((x.grad.view(m, k), x64.grad), (layer.weight.grad, w64.grad), (layer.bias.grad, b64.grad)):
        assert (got.double() - want).norm() <= 2 * BF16 * want.norm()
    d, step = randn(m, k, seed=6).double(), 1e-5
    f = lambda t: (act64("gelu", t @ w64.detach().t() + b64.detach()) * gy.view(m, n).double()).sum()  # noqa: E731
    numeric = (f(x64.detach() + step * d) - f(x64.detach() - step * d)) / (2 * step)
    assert abs(numeric - (x64.grad * d).sum()) <= 1e-6 * (x64.grad * d).abs().sum()
    # fp32 main_grad buffers instead of .grad, over two backward passes
    fused = ops.DominoLinear(k, n, act="gelu", fuse_wgrad=True)
    fused.load_state_dict(layer.state_dict())
    for _ in range(2):
        fused(x).backward(gy)
    assert fused.weight.grad is None and fused.bias.grad is None
    assert (fused.weight.main_grad.double() - 2 * w64.grad).norm() <= 4 * BF16 * w64.grad.norm()
    assert (fused.bias.main_grad.double() - 2 * b64.grad).norm() <= 4 * BF16 * b64.grad.norm()
    fused.zero_main_grad()
    assert not fused.weight.main_grad.any()


def test_capture_and_streams(ops):
    """Captured passes replay on new inputs with the eager bits; two streams at once share nothing."""
    m, n, k = 300, 768, 2056
    x, w, b, gy = randn(m, k, seed=1), randn(n, k, seed=2, std=0.02), randn(n, seed=3), randn(m, n, seed=4)

    def step():
        y, z = ops.linear_fwd(x, w, b, "gelu", gy, save=True)
        return (y, z, *ops.linear_bwd(gy, x, w, z, "gelu"))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        here = step()
        with torch.cuda.stream(side):
            there = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(here, want)) and all(torch.equal(a, c) for a, c in zip(there, want))
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        out1 = step()
    with torch.cuda.graph(two):
        out2 = step()
    x.copy_(randn(m, k, seed=9))
    want = step()
    torch.cuda.synchronize()
    one.replay()
    with torch.cuda.stream(side):
        two.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out1, want)) and all(torch.equal(a, c) for a, c in zip(out2, want))
