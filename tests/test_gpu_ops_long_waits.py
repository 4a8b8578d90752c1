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
