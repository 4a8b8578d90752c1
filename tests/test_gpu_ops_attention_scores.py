"""Packed attention with scores far beyond what an exponential can tell apart: the keys of the largest score share the
weight, whatever its size.  Queries and keys have one column other than zero, so that scores are exact: a power of two
times a small integer of the key's."""
import pytest
import torch

from ops_helpers import BF16, U32, close, device_ok, randn

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


# prompts, single tokens, a cut cache, a chunk of two tiles and more over a cut cache
BATCHES = {"prompts": [(300, 300), (5, 5), (129, 129)], "tokens": [(1, 77), (1, 1), (1, 900)], "cut": [(1, 20000)], "chunk": [(200, 9000), (1, 40)]}


@pytest.mark.parametrize("power", [7, 10, 13, 14, 15, 16, 18, 24, 40, 60])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("sign", [1, -1])
def test_largest_scores_share_the_weight(ops, power, batch, sign):
    seqs, hq, hkv = BATCHES[batch], 8, 2
    tq, tk = sum(a for a, _ in seqs), sum(b for _, b in seqs)
    g = torch.Generator().manual_seed(power)
    c = sign * torch.randint(1, 120, (tk, hkv), generator=g).double()
    q, k, v = torch.zeros(tq, hq, D, dtype=torch.bfloat16), torch.zeros(tk, hkv, D, dtype=torch.bfloat16), randn(tk, hkv, D, seed=3)
    q[:, :, 5] = 2.0 ** power
    k[:, :, 5] = (c * 2.0 ** power).to(torch.bfloat16)
    q, k = q.cuda(), k.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, start = [0], [0]
    for a, b in seqs:
        cu.append(cu[-1] + a)
        start.append(start[-1] + b)
    o, lse = ops.packed_attention(q, k, v, torch.tensor(cu, **i32), torch.tensor(start[:-1], **i32), torch.tensor([b for _, b in seqs], **i32),
                                  return_lse=True)
    for s, (a, b) in enumerate(seqs):
        score = c[start[s]:start[s] + b].t().cuda().repeat_interleave(hq // hkv, 0)[:, None, :].expand(hq, a, b)  # [head, query, key]
        hidden = torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1)
        score = score.masked_fill(hidden, -1e9)
        top = score.amax(2, keepdim=True)
        p = (score == top).double()
        ties, vs = p.sum(2, keepdim=True), v[start[s]:start[s] + b].double().transpose(0, 1).repeat_interleave(hq // hkv, 0)
        # The ties have one weight, 2^r, r the rounding of the largest score's product with the scale (and up to 8 that the
        # running maximum may lag behind): it is rounded to bf16 for its product with V, by at most half a step, 2^-8 of
        # it, and not in the denominator.  Beside that only the sums over the ties, their division and one rounding are left.
        slop = (p @ vs.abs()) / ties * (BF16 + (4 + ties / 16) * U32)
        close(o[cu[s]:cu[s + 1]], (p @ vs / ties).transpose(0, 1), slop.transpose(0, 1), what=f"O of sequence {s}")
        # scale, its product with log2(e), that with the score, ln 2 and the sum: less than eight roundings of the size of lse
        want = (top * 2.0 ** (2 * power) * D ** -0.5 + ties.log()).squeeze(2).t()
        close(lse[cu[s]:cu[s + 1]], want, 8 * U32 * want.abs() + 2.0 ** -20, rounding=0, what=f"lse of sequence {s}")


@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 8)])
def test_rows_of_every_size_side_by_side(ops, hq, hkv):
    """Rows of ordinary scores keep their bits beside rows of huge ones, in the same warp and in the same tile."""
    n = 700
    q, k, v = randn(n, hq, D, seed=1), randn(n, hkv, D, seed=2), randn(n, hkv, D, seed=3)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    # a row's rescaling depends on its warp's, so the ordinary rows are held against a scale that changes no value: a
    # query of zeros, whose scores are zero, has the mean of the keys it sees, exactly as many of them
    q[::3] = 0.0
    q[1::3] *= 2.0 ** 40
    o, lse = ops.packed_attention(q, k, v, cu, return_lse=True)
    seen = torch.arange(1, n + 1, device="cuda").double()[::3]
    vs = v.double().repeat_interleave(hq // hkv, 1)
    mean = vs.cumsum(0)[::3] / seen[:, None, None]
    close(o[::3], mean, (n / 16 + 8) * 2.0 ** -23 * (vs.abs().cumsum(0)[::3] / seen[:, None, None]), what="O of zero queries")
    close(lse[::3], seen.log()[:, None].expand(-1, hq), 2.0 ** -20, rounding=0, what="lse of zero queries")
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    assert not (o == 0).all(-1).any()
