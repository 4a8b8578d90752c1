"""The packed attention's plan, read from the workspace: pairs of tiles that stay whole are dealt heaviest first, the first
of equals first.  The order decides how even the shares look and with that whether pairs are cut, so it may not depend on
which thread came first."""
import pytest
import torch

from ops_helpers import close, device_ok, randn
from test_gpu_ops_attention import attend64

pytestmark = pytest.mark.gpu
D = 128
PAIRS_AT, PAIR_BYTES = 1024, 32  # the list of pairs in the workspace, behind its header and the ranges' starts


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from comm_overlap_gb300 import build
    build.build()
    from comm_overlap_gb300 import torch_ops
    yield torch_ops
    device_ok()


# key counts of single queries over one cache: heaviest below, at and far above the bins of the counting sort (512 half
# blocks of 64 keys), rising by one and a half half blocks, falling, and mixed
LENGTHS = {"below": [12000 + 64 * i for i in range(304)], "rising": [40000 + 98 * i for i in range(304)],
           "falling": [69700 - 98 * i for i in range(304)], "mixed": [60000 + (i * 7919) % 1800 for i in range(456)],
           "long": [250000 + (i * 7919) % 900 for i in range(152)], "doubled": [45000 + (i // 2 * 331) % 4000 for i in range(304)]}


@pytest.mark.parametrize("name", LENGTHS)
def test_order_of_whole_pairs(ops, name):
    from comm_overlap_gb300 import domino as dm
    lens = LENGTHS[name]
    n, tk = len(lens), max(lens)
    q, k, v = randn(n, 1, D, seed=1), randn(tk, 1, D, seed=2), randn(tk, 1, D, seed=3)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, start, length = torch.arange(n + 1, **i32), torch.zeros(n, **i32), torch.tensor(lens, **i32)
    size = dm.domino_attn_packed_workspace_size(n, n, 1, 1, tk)
    ws, o, lse = torch.zeros(size, dtype=torch.uint8, device="cuda"), torch.empty_like(q), torch.empty(n, 1, device="cuda")
    ops._call(dm.domino_attn_packed_fwd, q, q, D, k, D, v, D, cu, start, length, D ** -0.5, o, D, lse, n, n, 1, 1, tk, ws, size)
    host = ws.cpu()
    pairs, whole = host[16:24].view(torch.int32).tolist()
    assert pairs == n and whole == 1, "the lengths are meant to stay whole"
    halves = host[PAIRS_AT:PAIRS_AT + n * PAIR_BYTES].view(torch.int32).view(n, 8)[:, 5].tolist()
    assert halves == [(x + 63) // 64 for x in lens]
    room = n // 256 + n  # pairs that the list has room for
    at = (PAIRS_AT + room * PAIR_BYTES + 255) // 256 * 256
    order = host[at:at + 4 * n].view(torch.int32).tolist()
    assert sorted(order) == list(range(n))
    if name == "below":  # equals may come in any order: it changes neither a share nor a sum
        assert [halves[i] for i in order] == sorted(halves, reverse=True)
    else:
        assert order == sorted(range(n), key=lambda i: (-halves[i], i))
    for s in (0, n // 2, n - 1):
        ro, rl, so, sl = attend64(q[s:s + 1], k[:lens[s]], v[:lens[s]], D ** -0.5)
        close(o[s:s + 1], ro, so, what=f"O of sequence {s}")
        close(lse[s:s + 1], rl, sl, rounding=0, what=f"lse of sequence {s}")
