"""Calls that take seconds: no wait of a kernel runs out because the work before it is long."""
import pytest
import torch

from ops_helpers import close, device_ok, randn
from test_gpu_ops_attention import attend64

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


def test_second_tile_waits_for_many_single_tokens(ops):
    """1.8 million single tokens over one cache, which use a CTA's first tile alone, and a prompt of two tiles after them."""
    n, tk, prompt = 1800000, 32768, 200
    q, k, v = randn(n + prompt, 1, D, seed=1), randn(tk, 1, D, seed=2), randn(tk, 1, D, seed=3)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.arange(n + 2, **i32)
    cu[-1] = n + prompt
    start, length = torch.zeros(n + 1, **i32), torch.full((n + 1,), tk, **i32)
    length[-1] = prompt
    torch.cuda.synchronize()
    o, lse = ops.packed_attention(q, k, v, cu, start, length, return_lse=True)
    ops.device_status()
    for a, b, keys in ((0, 1, tk), (n // 2, n // 2 + 1, tk), (n - 1, n, tk), (n, n + prompt, prompt)):
        ro, rl, so, sl = attend64(q[a:b], k[:keys], v[:keys], D ** -0.5)
        close(o[a:b], ro, so, what=f"O from {a}")
        close(lse[a:b], rl, sl, rounding=0, what=f"lse from {a}")


@pytest.mark.parametrize("main", [True, False])
def test_weight_gradient_of_many_rows(ops, main):
    """A reduction over 2^30 rows, nearly all of them zero: small integers, whose sums are exact."""
    m, n, k = (1 << 30) + 77, 16, 8
    g = torch.Generator().manual_seed(5)
    rows = torch.cat([torch.randint(0, m, (3000,), generator=g), torch.tensor([0, 63, 64, m - 78, m - 77, m - 1])]
                     + [torch.tensor([i << 26, (i << 26) - 1]) for i in range(1, 17)]).unique().cuda()
    some_x = torch.randint(-2, 3, (len(rows), k), generator=g).to(torch.bfloat16).cuda()
    some_g = torch.randint(-1, 2, (len(rows), n), generator=g).to(torch.bfloat16).cuda()
    w = randn(n, k, seed=1)
    x, gy = (torch.zeros(m, c, dtype=torch.bfloat16, device="cuda") for c in (k, n))
    x[rows], gy[rows] = some_x, some_g
    start = torch.arange(n * k, dtype=torch.float32, device="cuda").view(n, k)
    buf = start.clone() if main else None
    _, gw, gb = ops.linear_bwd(gy, x, w, x_grad=False, main_grad=buf)
    ops.device_status()
    want = some_g.double().t() @ some_x.double()
    assert torch.equal(buf.double(), want + start.double()) if main else torch.equal(gw, want.to(torch.bfloat16))
    assert torch.equal(gb.double(), some_g.double().sum(0))
