"""Causal attention over packed sequences against its definition in 64 bits, sequence by sequence.

Bound of a value of O: with p the softmax's numerators, each p is off by half a bf16 step (2^-8, its
rounding for the product) and by `d`, the error of its exponent: the score's accumulation (see mma in
test_gpu_ops_linear.py), its product with the scale and the exponential, a few units of 2^-24 of the score;
the numerator's and denominator's sums over the keys are fp32 (2^-23 a step of sixteen terms)."""
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


def attend64(q, k, v, scale):
    """One sequence, q [tq, heads, D]: O, lse, and their bounds."""
    tq, hq, _ = q.shape
    tk, hkv, _ = k.shape
    g = hq // hkv
    q, k, v = (t.double().transpose(0, 1) for t in (q, k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)))
    s = q @ k.transpose(1, 2) * scale
    mag = q.abs() @ k.abs().transpose(1, 2) * scale
    hidden = torch.ones(tq, tk, dtype=torch.bool, device=q.device).triu(tk - tq + 1)
    s = s.masked_fill(hidden, -float("inf"))
    if tk == 0:
        z = torch.zeros(tq, hq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((tq, hq), -float("inf"), dtype=torch.float64, device=q.device), z, z[..., 0]
    top = s.amax(2, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(2, keepdim=True)
    d = ((D / 8 + 96) * 2.0 ** -23 * mag + 4 * U32 * s.masked_fill(hidden, 0).abs() + 2.0 ** -20).masked_fill(hidden, 0)
    safe = total.clamp(min=1e-300)
    o = (p @ v) / safe
    keys = (tk / 8 + 300) * 2.0 ** -23
    slop = ((p * (BF16 + 1.01 * d + keys)) @ v.abs()) / safe + o.abs() * ((p * d).sum(2, keepdim=True) / safe + keys)
    lse = (top + total.log()).squeeze(2)
    ls = (p * d).sum(2) / safe.squeeze(2) + keys + 4 * U32 * (lse.abs() + top.squeeze(2).abs())
    return o.transpose(0, 1), lse.t(), slop.transpose(0, 1), ls.t()


class Batch:
    """Sequences (queries, keys) laid into one buffer: rows that belong to none hold NaN and infinities, keys in
    another order than the sequences, heads as slices of one buffer."""

    def __init__(self, seqs, hq, hkv, seed=0, gap=3, junk=True):
        self.seqs, self.hq, self.hkv = seqs, hq, hkv
        tq = gap + sum(a for a, _ in seqs) + gap
        order = sorted(range(len(seqs)), key=lambda i: (i * 7919 + 3) % max(len(seqs), 1))
        at, self.start = gap, [0] * len(seqs)
        for i in order:
            self.start[i] = at
            at += seqs[i][1] + gap
        q = randn(tq, hq, D, seed=seed)
        kv = randn(at, 2 * hkv + 1, D, seed=seed + 1)
        self.k, self.v = kv[:, :hkv], kv[:, hkv:2 * hkv]
        own_q, own_k = torch.zeros(tq, dtype=torch.bool), torch.zeros(at, dtype=torch.bool)
        cu = [gap]
        for (a, b), s in zip(seqs, self.start):
            own_q[cu[-1]:cu[-1] + a] = True
            own_k[s:s + b] = True
            cu.append(cu[-1] + a)
        self.q, self.cu, self.own_q = q, cu, own_q.cuda()
        if junk:
            bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(torch.bfloat16)
            self.q[~self.own_q] = bad[0]
            rows = (~own_k).nonzero().squeeze(1).cuda()
            kv[rows] = bad[torch.arange(rows.numel(), device="cuda") % 3].view(-1, 1, 1)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.args = (torch.tensor(cu, **i32), torch.tensor(self.start, **i32), torch.tensor([b for _, b in seqs], **i32))

    def run(self, ops, scale=None):
        out = torch.full((self.q.shape[0], self.hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        return ops.packed_attention(self.q, self.k, self.v, *self.args, scale=scale, return_lse=True, out=out)

    def check(self, o, lse, scale=None):
        assert (o[~self.own_q] == 7.0).all(), "rows that belong to no sequence were written"
        for i, (a, b) in enumerate(self.seqs):
            c, s = self.cu[i], self.start[i]
            ro, rl, so, sl = attend64(self.q[c:c + a], self.k[s:s + b], self.v[s:s + b], D ** -0.5 if scale is None else scale)
            close(o[c:c + a], ro, so, what=f"O of sequence {i}: {a} queries, {b} keys")
            got = lse[c:c + a].double()
            empty = rl.isinf()
            assert torch.equal(got.isinf(), empty) and (got[empty] < 0).all()
            close(got.masked_fill(empty, 0), rl.masked_fill(empty, 0), sl.masked_fill(empty, 0), rounding=0, what=f"lse of sequence {i}")


PROMPTS = [(n, n) for n in (1, 2, 127, 128, 129, 0, 255, 256, 257, 300, 513)]
DECODE = [(1, n) for n in (1, 2, 127, 128, 129, 0, 255, 256, 257, 1000, 1500)]
CHUNKS = [(5, 700), (130, 900), (64, 64), (20, 7), (300, 130), (1, 77), (3, 0), (257, 1029), (128, 256), (40, 39)]
HEADS = [(1, 1), (4, 1), (8, 2), (10, 2), (21, 3), (16, 1), (128, 1), (100, 2)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("seqs", [PROMPTS, DECODE, CHUNKS, [(1, 1)], [(0, 5)], [(700, 0)]], ids=["prompts", "decode", "chunks", "one", "none", "nokeys"])
def test_sequences(ops, hq, hkv, seqs):
    b = Batch(seqs, hq, hkv, seed=hq)
    o, lse = b.run(ops)
    b.check(o, lse)
    o2, lse2 = b.run(ops)
    assert torch.equal(o, o2) and torch.equal(lse[b.own_q], lse2[b.own_q])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (8, 2), (5, 1)])
@pytest.mark.parametrize("seqs", [[(1, 20000)], [(200, 9000)], [(1, 6000), (1, 3), (150, 5000), (0, 9), (1, 0)],
                                  [(600, 4500), (2, 1)]], ids=["token", "chunk", "mixed", "pairs"])
def test_long_keys_are_cut_into_parts(ops, hq, hkv, seqs):
    b = Batch(seqs, hq, hkv, seed=3)
    o, lse = b.run(ops)
    b.check(o, lse)
    o2, lse2 = b.run(ops)
    assert torch.equal(o, o2) and torch.equal(lse[b.own_q], lse2[b.own_q])


@pytest.mark.parametrize("scale", [1.0, 0.02, 1e-6])
def test_scales(ops, scale):
    b = Batch([(70, 70), (1, 400), (33, 200)], 8, 4, seed=5)
    b.check(*b.run(ops, scale), scale)


def test_scores_that_grow_along_the_keys(ops):
    """The running maximum rises in every block, by more and by less than the lazy rescale's threshold."""
    b = Batch([(200, 1000)], 4, 2, seed=6)
    s, n = b.start[0], 1000
    b.q[3:203] = 1.0
    b.k[s:s + n] = (torch.arange(n, device="cuda") / 40).view(-1, 1, 1).to(torch.bfloat16) * torch.tensor([1.0, 0.1], device="cuda").view(1, 2, 1).to(torch.bfloat16)
    b.check(*b.run(ops))


def test_own_rows_and_slices_of_a_projection(ops):
    """Without k_start and k_len the keys are the queries' rows; q, k, v as slices of one projection."""
    cu = [0, 100, 100, 357, 358]
    qkv = randn(358, 12, D, seed=8)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = ops.packed_attention(q, k, v, cu_t)
    same = ops.packed_attention(q.contiguous(), k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1), cu_t)
    assert torch.equal(o, same)
    for a, b in zip(cu, cu[1:]):
        ro, _, so, _ = attend64(q[a:b], k[a:b], v[a:b], D ** -0.5)
        close(o[a:b], ro, so, what=f"rows {a} to {b}")


def test_many_sequences(ops):
    """More sequences than the planning block has threads."""
    n = 2500
    seqs = [(i % 3, (i * 37) % 50 + i % 3) for i in range(n)]
    b = Batch(seqs, 2, 1, seed=9, gap=1)
    o, lse = b.run(ops)
    keep = [i for i in range(n) if i % 97 < 3]
    assert (o[~b.own_q] == 7.0).all()
    for i in keep:
        (x, y), c, s = seqs[i], b.cu[i], b.start[i]
        ro, _, so, _ = attend64(b.q[c:c + x], b.k[s:s + y], b.v[s:s + y], D ** -0.5)
        close(o[c:c + x], ro, so, what=f"sequence {i}")


@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 16), (22, 11), (24, 12)])
@pytest.mark.parametrize("few", [False, True])
def test_long_and_short_sequences_together(ops, hq, hkv, few):
    """One sequence far longer than the mean share, cut over many ranges that lie across the heads' groups, among short ones,
    fewer and more than the planning block has threads."""
    seqs = [(1, 1 + i * 7 % 60) for i in range(20 if few else 700)]
    seqs[11:11] = [(3, 9000), (0, 4000), (1, 0)]
    b = Batch(seqs, hq, hkv, seed=hkv, gap=1)
    o, lse = b.run(ops)
    assert (o[~b.own_q] == 7.0).all()
    for i in [*range(0, 16), len(seqs) - 1]:
        (x, y), c, s = seqs[i], b.cu[i], b.start[i]
        ro, rl, so, sl = attend64(b.q[c:c + x], b.k[s:s + y], b.v[s:s + y], D ** -0.5)
        close(o[c:c + x], ro, so, what=f"sequence {i}")
        if y >= x:
            close(lse[c:c + x], rl, sl, rounding=0, what=f"lse of sequence {i}")
    again = b.run(ops)
    assert torch.equal(o, again[0]) and torch.equal(lse[b.own_q], again[1][b.own_q])


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("cached", [0, 1500])
def test_nonfinite_keys_that_a_query_does_not_see(ops, hq, hkv, cached):
    """Junk in K from a position on leaves the queries before it alone; junk in V those 192 and more before it."""
    n, at = 700, 600
    b = Batch([(n, cached + n)], hq, hkv, seed=21, junk=False)
    clean, _ = b.run(ops)
    c, s = b.cu[0], b.start[0] + cached
    for t, reach in ((b.k, 0), (b.v, 191)):
        keep = t[s + at:s + at + 40].clone()
        for bad in (float("nan"), float("inf"), -float("inf")):
            t[s + at:s + at + 40:3] = bad
            o, _ = b.run(ops)
            assert torch.equal(o[c:c + at - reach], clean[c:c + at - reach])
            if bad != bad:
                assert torch.isnan(o[c + at:c + n].float()).any(-1).all()
        t[s + at:s + at + 40] = keep


def test_offsets_beyond_32_bits(ops):
    """A cache whose rows pass 2^31 values and 2^32 bytes."""
    tk, hkv, hq = 2300000, 8, 32
    k, v = (torch.randn(tk, hkv, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    starts, lens = [0, 1048570, 2097140, 2099000, tk - 1000], [700, 40, 900, 3000, 1000]
    q = randn(len(starts), hq, D, seed=1)
    i32 = dict(dtype=torch.int32, device="cuda")
    o, lse = ops.packed_attention(q, k, v, torch.arange(len(starts) + 1, **i32), torch.tensor(starts, **i32),
                                  torch.tensor(lens, **i32), return_lse=True)
    for s, (a, n) in enumerate(zip(starts, lens)):
        ro, rl, so, sl = attend64(q[s:s + 1], k[a:a + n], v[a:a + n], D ** -0.5)
        close(o[s:s + 1], ro, so, what=f"O of sequence {s}")
        close(lse[s:s + 1], rl, sl, rounding=0, what=f"lse of sequence {s}")


def test_same_keys_for_several_sequences(ops):
    """A shared prefix: sequences may read the same cache rows."""
    q, kv = randn(6, 4, D, seed=1), randn(500, 2, 2, D, seed=2)
    k, v = kv[:, 0], kv[:, 1]
    i32 = dict(dtype=torch.int32, device="cuda")
    o = ops.packed_attention(q, k, v, torch.tensor([0, 1, 3, 6], **i32), torch.tensor([0, 0, 10], **i32), torch.tensor([400, 500, 300], **i32))
    for a, b, s, n in ((0, 1, 0, 400), (1, 3, 0, 500), (3, 6, 10, 300)):
        ro, _, so, _ = attend64(q[a:b], k[s:s + n], v[s:s + n], D ** -0.5)
        close(o[a:b], ro, so)


def test_lengths_outside_the_tensors_are_recorded(ops):
    """A sequence whose rows leave its tensors is skipped; the others are computed; the status tells."""
    from comm_overlap_gb300 import domino as dm
    ops.device_status()
    good = Batch([(5, 40), (6, 50), (7, 60)], 4, 2, seed=1, junk=False)
    tq, tk = good.q.shape[0], good.k.shape[0]
    want, _ = good.run(ops)
    for which, value in ((1, -1), (1, tk - 20), (2, -3), (2, tk + 1), (1, 2 ** 31 - 1), (2, 2 ** 31 - 1)):
        args = [t.clone() for t in good.args]
        args[which][1] = value
        out = torch.full((tq, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.packed_attention(good.q, good.k, good.v, *args, out=out)
        c = good.cu
        assert torch.equal(out[c[0]:c[1]], want[c[0]:c[1]]) and torch.equal(out[c[2]:c[3]], want[c[2]:c[3]])
        assert (out[c[1]:c[2]] == 7.0).all()
        with pytest.raises(dm.DominoError, match="lengths"):
            ops.device_status()
    for cu in ([3, 2, 14, 21], [-1, 8, 14, 21], [3, 8, 14, tq + 1], [0, 2 ** 31 - 1, -2 ** 31, 5]):
        ops.packed_attention(good.q, good.k, good.v, torch.tensor(cu, dtype=torch.int32, device="cuda"), *good.args[1:])
        with pytest.raises(dm.DominoError, match="lengths"):
            ops.device_status()
    ops.device_status()


def test_capture_and_streams(ops):
    """One captured call serves new lengths and keys; calls on two streams at once do not meet."""
    b = Batch([(1, 700), (130, 500), (1, 3000)], 8, 2, seed=4, junk=False)
    want, _ = b.run(ops)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        here, _ = b.run(ops)
        with torch.cuda.stream(side):
            there, _ = b.run(ops)
    torch.cuda.synchronize()
    assert torch.equal(here, want) and torch.equal(there, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = b.run(ops)
    b.args[2].copy_(torch.tensor([650, 130, 2222], dtype=torch.int32))
    b.k.copy_(randn(*b.k.shape, seed=11))
    b.seqs = [(1, 650), (130, 130), (1, 2222)]
    graph.replay()
    torch.cuda.synchronize()
    b.check(o, lse)
