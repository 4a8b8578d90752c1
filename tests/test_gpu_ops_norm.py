"""LayerNorm with weight and bias, forward and backward, against its definition in 64 bits."""
import pytest
import torch

from ops_helpers import U32, close, device_ok, randn

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


# one piece a thread to four, one warp to sixteen, several teams in a block, widths that end inside a
# warp's pieces, fewer rows than teams, rows that the grid walks more than once
SIZES = [(0, 64), (1, 8), (1, 4096), (3, 256), (7, 264), (5, 2048), (9, 2056), (17, 4096), (33, 8192), (13, 8200),
         (6, 16384), (3, 16376), (1237, 2560), (5000, 512), (9001, 64)]


def fwd64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = ((x - mean[:, None]).square().mean(1) + eps).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None] * w.double() + (b.double() if b is not None else 0)
    return y, mean, rstd


def sum_depth(h):
    """Additions that one value of a row's sum passes through: 32 in a thread, 5 in a warp, 16 warps."""
    return 53


def check_fwd(x, w, b, eps, got):
    y, mean, rstd = fwd64(x, w, b, eps)
    h = x.shape[1]
    ax = x.double().abs().mean(1) if h else 0
    # the mean is off by (depth + 1) units of the mean magnitude; the centred values by that and their own
    # rounding, the variance by depth units and twice the mean's (second order), its root by half of it
    dm_ = (sum_depth(h) + 1) * U32 * ax
    close(got[1], mean, dm_, rounding=0, what="mean")
    rel = (0.5 * (sum_depth(h) + 4) + 3) * U32 + (dm_ * rstd) ** 2
    close(got[2], rstd, rel * rstd, rounding=0, what="rstd")
    xh = (x.double() - mean[:, None]).abs() * rstd[:, None]
    slop = w.double().abs() * (xh * (rel[:, None] + 4 * U32) + (dm_ * rstd)[:, None])
    if b is not None:
        slop = slop + b.double().abs() * 2 * U32
    close(got[0], y, slop, what="y")


@pytest.mark.parametrize("rows,h", SIZES)
@pytest.mark.parametrize("bias", [True, False])
def test_forward(ops, rows, h, bias):
    x, w = randn(rows, h, seed=1, mean=0.5), randn(h, seed=2, std=0.2, mean=1.0)
    b = randn(h, seed=3) if bias else None
    check_fwd(x, w, b, 1e-5, ops.layer_norm_fwd(x, w, b, 1e-5))


def bwd64(gy, x, w, mean, rstd, gres):
    gy, x, w, mean, rstd = (t.double() for t in (gy, x, w, mean, rstd))
    n = (x - mean[:, None]) * rstd[:, None]
    u = gy * w
    gx = rstd[:, None] * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True))
    return gx + (gres.double() if gres is not None else 0), (gy * n).sum(0), gy.sum(0)


def check_bwd(gy, x, w, mean, rstd, gres, got, start=None):
    gx, gw, gb = bwd64(gy, x, w, mean, rstd, gres)
    rows, h = x.shape
    g, an = gy.double().abs(), (x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    u = g * w.double().abs()
    d = sum_depth(h) + 6
    slop = rstd.double()[:, None] * U32 * (8 * u * (1 + an) + d * (u.mean(1, keepdim=True) + 2 * an * (u * an).mean(1, keepdim=True)))
    close(got[0], gx, slop + (2 * U32 * gres.double().abs() if gres is not None else 0), what="gx")
    # a column's sum passes through at most every row of a team, 8 teams, 32 groups of partial sums of up to ten
    # additions, and the buffer
    depth = rows + 60
    s_w, s_b = (g * an).sum(0), g.sum(0)
    if start is not None:
        gw, gb = gw + start[0].double(), gb + start[1].double()
        s_w, s_b = s_w + start[0].double().abs(), s_b + start[1].double().abs()
    depth = min(depth, 1200)
    close(got[1], gw, depth * U32 * s_w, rounding=0, what="gweight")
    if got[2] is not None:
        close(got[2], gb, depth * U32 * s_b, rounding=0, what="gbias")


@pytest.mark.parametrize("rows,h", SIZES)
@pytest.mark.parametrize("res", [True, False])
def test_backward(ops, rows, h, res):
    x, w, gy = randn(rows, h, seed=1, mean=0.5), randn(h, seed=2, std=0.2, mean=1.0), randn(rows, h, seed=4)
    gres = randn(rows, h, seed=5) if res else None
    _, mean, rstd = fwd64(x, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    got = ops.layer_norm_bwd(gy, x, w, mean, rstd, gres)
    check_bwd(gy, x, w, mean, rstd, gres, got)
    again = ops.layer_norm_bwd(gy, x, w, mean, rstd, gres)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# many rows: one warp a row with one to four pieces a thread, two to sixteen warps a row, uneven last pieces, blocks with
# spare warps, rows that do not divide among the teams
MANY = [(8003, 136), (2100, 512), (3000, 760), (1200, 904), (701, 1576), (640, 2048), (501, 2056), (2500, 2560), (300, 4096),
        (211, 5000), (130, 8200), (70, 16384)]


@pytest.mark.parametrize("rows,h", MANY)
@pytest.mark.parametrize("res", [True, False])
def test_many_rows(ops, rows, h, res):
    """Forward and backward of strided rows; sums added to buffers; junk between the rows."""
    def strided(seed, **kw):
        wide = torch.full((rows, h + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :h] = randn(rows, h, seed=seed, **kw)
        return wide[:, :h]

    x, gy, w, b = strided(1, mean=0.5), strided(4), randn(h, seed=2, std=0.2, mean=1.0), randn(h, seed=3)
    gres = strided(5) if res else None
    fwd = ops.layer_norm_fwd(x, w, b)
    check_fwd(x, w, b, 1e-5, fwd)
    start = (randn(h, seed=6, dtype=torch.float32), randn(h, seed=7, dtype=torch.float32))
    grads = tuple(t.clone() for t in start)
    got = ops.layer_norm_bwd(gy, x, w, *fwd[1:], gres, grads=grads)
    check_bwd(gy, x, w, *fwd[1:], gres, got, start)
    plain = ops.layer_norm_bwd(gy, x, w, *fwd[1:], gres)
    check_bwd(gy, x, w, *fwd[1:], gres, plain)
    again = ops.layer_norm_bwd(gy, x, w, *fwd[1:], gres)
    assert all(torch.equal(p, q) for p, q in zip(plain, again))


def test_many_rows_in_place_and_apart(ops):
    """gX in the place of gY or of the residual's gradient; a row of NaN leaves the other rows' gX alone."""
    from comm_overlap_gb300 import domino as dm
    rows, h = 900, 1576
    x, gy, gres, w = (randn(rows, h, seed=i, mean=0.1) for i in (1, 2, 3, 4))
    w = w[0].contiguous()
    _, mean, rstd = ops.layer_norm_fwd(x, w)
    want = ops.layer_norm_bwd(gy, x, w, mean, rstd, gres)
    handle, stream = dm.domino_create(), torch.cuda.current_stream().cuda_stream
    n = dm.domino_layernorm_bwd_workspace_size(rows, h)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for own in range(2):
        g, r, gw, gb = gy.clone(), gres.clone(), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
        gx = (g, r)[own]
        dm.domino_layernorm_bwd(handle, g, h, x, h, w, mean, rstd, r, h, gx, h, gw, gb, 0, rows, h, ws, n, stream)
        torch.cuda.synchronize()
        assert torch.equal(gx, want[0]) and torch.equal(gw, want[1]) and torch.equal(gb, want[2])
    dm.domino_destroy(handle)
    gy[17] = float("nan")
    got = ops.layer_norm_bwd(gy, x, w, mean, rstd, gres)
    keep = torch.arange(rows, device="cuda") != 17
    assert torch.equal(got[0][keep], want[0][keep]) and torch.isnan(got[0][17]).all() and torch.isnan(got[1]).all()


def test_offsets_beyond_32_bits(ops):
    rows, h = 560000, 4096
    x, w, b = torch.randn(rows, h, device="cuda", dtype=torch.bfloat16), randn(h, seed=2), randn(h, seed=3)
    y, mean, rstd = ops.layer_norm_fwd(x, w, b)
    some = torch.tensor([0, 262143, 262144, 524287, 524288, 524289, 550001, rows - 1], device="cuda")
    check_fwd(x[some], w, b, 1e-5, (y[some], mean[some], rstd[some]))
    gx, _, _ = ops.layer_norm_bwd(y, x, w, mean, rstd, x)
    alone = ops.layer_norm_bwd(y[some], x[some], w, mean[some], rstd[some], x[some])
    check_bwd(y[some], x[some], w, mean[some], rstd[some], x[some], (gx[some], *alone[1:]))


def test_strided_rows_and_accumulation(ops):
    rows, h = 37, 520
    wide, gwide = randn(rows, 3 * h, seed=1), randn(rows, 2 * h, seed=2)
    x, gy, w = wide[:, h:2 * h], gwide[:, h:], randn(h, seed=3)
    y, mean, rstd = ops.layer_norm_fwd(x, w, None)
    check_fwd(x, w, None, 1e-5, (y, mean, rstd))
    start = (randn(h, seed=6, dtype=torch.float32), randn(h, seed=7, dtype=torch.float32))
    bufs = tuple(s.clone() for s in start)
    got = ops.layer_norm_bwd(gy, x, w, mean, rstd, None, grads=bufs)
    assert got[1] is bufs[0] and got[2] is bufs[1]
    check_bwd(gy, x, w, mean, rstd, None, got, start)
    # no bias gradient; a gradient broadcast over the rows; rows that cannot be strided over are copied
    e = gy[:1].expand(rows, h)
    got = ops.layer_norm_bwd(e, x.t().contiguous().t(), w, mean, rstd, bias_grad=False)
    assert got[2] is None
    check_bwd(e, x, w, mean, rstd, None, got)
    odd = torch.empty(rows * h + 1, dtype=torch.bfloat16, device="cuda")[1:].view(rows, h).copy_(x)
    assert odd.data_ptr() % 16 and torch.equal(ops.layer_norm_fwd(odd, w)[0], y)


def test_rows_stay_apart(ops):
    """Constant rows, huge rows, and rows with infinities and NaN: the others do not notice."""
    rows, h = 64, 1032
    x, w, b = randn(rows, h, seed=1), randn(h, seed=2, mean=1.0), randn(h, seed=3)
    clean, *_ = ops.layer_norm_fwd(x, w, b)
    dirty = x.clone()
    dirty[3], dirty[5, 7], dirty[9, 0], dirty[11] = 2.5, float("inf"), float("nan"), x[11] * 1e18
    y, mean, rstd = ops.layer_norm_fwd(dirty, w, b)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[3, 5, 9, 11]] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(y[3], b) and mean[3] == 2.5  # variance zero: the bias remains
    assert not torch.isfinite(y[5]).any() and not torch.isfinite(y[9]).any()
    check_fwd(dirty[11:12], w, b, 1e-5, (y[11:12], mean[11:12], rstd[11:12]))


def test_in_place_outputs(ops):
    """Y may be X, and gX may be gY or gres."""
    from comm_overlap_gb300 import domino as dm
    rows, h = 300, 768
    x, w, gy, gres = randn(rows, h, seed=1), randn(h, seed=2), randn(rows, h, seed=3), randn(rows, h, seed=4)
    y, mean, rstd = ops.layer_norm_fwd(x, w)
    z = x.clone()
    ops._call(dm.domino_layernorm_fwd, x, z, h, w, None, 1e-5, z, h, None, None, rows, h)
    assert torch.equal(z, y)
    want, gw, gb = ops.layer_norm_bwd(gy, x, w, mean, rstd, gres)
    ws = torch.empty(dm.domino_layernorm_bwd_workspace_size(rows, h), dtype=torch.uint8, device="cuda")
    for which in (0, 1):
        g, r = gy.clone(), gres.clone()
        ops._call(dm.domino_layernorm_bwd, x, g, h, x, h, w, mean, rstd, r, h, (g, r)[which], h, gw, gb, 0, rows, h, ws, ws.numel())
        assert torch.equal((g, r)[which], want)


def test_autograd_and_differences(ops):
    """The module's gradients are the formula's, and the formula's are the forward's differences (64 bits)."""
    rows, h = 24, 136
    m = ops.DominoLayerNorm(h)
    with torch.no_grad():
        m.weight.copy_(randn(h, seed=2, mean=1.0))
        m.bias.copy_(randn(h, seed=3))
    x, gy = randn(2, rows // 2, h, seed=1).requires_grad_(), randn(2, rows // 2, h, seed=4)
    y = m(x)
    y.backward(gy)
    x2, gy2 = x.detach().view(rows, h), gy.view(rows, h)
    _, mean, rstd = fwd64(x2, m.weight, m.bias, 1e-5)
    gx, gw, gb = bwd64(gy2, x2, m.weight.detach(), mean, rstd, None)
    close(x.grad.view(rows, h), gx, 1e-4 * gx.abs().max(), what="gx")
    close(m.weight.grad, gw, 1e-5 * gw.abs().max(), what="gweight")
    close(m.bias.grad, gb, 1e-5 * gb.abs().max(), what="gbias")
    step, d = 1e-5, randn(rows, h, seed=8).double()
    up, down = (fwd64(x2.double() + s * step * d, m.weight, m.bias, 1e-5)[0] for s in (1, -1))
    numeric = ((up - down) * gy2.double()).sum() / (2 * step)
    assert abs(numeric - (gx * d).sum()) <= 1e-6 * (gx * d).abs().sum()


def test_capture_and_streams(ops):
    """A captured forward and backward replays on new inputs with the eager bits; another stream too."""
    rows, h = 515, 2056
    x, w, gy = randn(rows, h, seed=1), randn(h, seed=2), randn(rows, h, seed=3)

    def step():
        y, mean, rstd = ops.layer_norm_fwd(x, w)
        return (y, *ops.layer_norm_bwd(gy, x, w, mean, rstd, y))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(on_side, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(randn(rows, h, seed=9))
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
