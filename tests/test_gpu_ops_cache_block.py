"""The rotation, the 8-bit cache and its attention together, as an attention sublayer uses them: prompts and chunks, single tokens,
drafts and shared rows over one cache, captured and replayed, on several streams, and a training step.

Every stage is compared with its definition in 64 bits on the values that it was given, with the bounds of the operators' own
tests, so no bound has to be carried through the block."""
import threading

import pytest
import torch

import test_gpu_ops_cached as cached
import test_gpu_ops_linear as lin
from cache_helpers import D, cos_sin, exponents, held, power, rotary, rotary_grad, turn
from ops_helpers import BF16, U32, close, device_ok, randn
from test_gpu_ops_attention import attend64

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from comm_overlap_gb300 import build
    build.build()
    from comm_overlap_gb300 import torch_ops
    yield torch_ops
    device_ok()


class Block:
    """y = x + out(attention(rotary(qkv(x)))) over an 8-bit cache of `room` rows a sequence behind `front` shared rows."""

    def __init__(self, ops, hq, hkv, n, room, front=0, seed=0, **rotation):
        h = hq * D
        self.ops, self.hq, self.hkv, self.h, self.n, self.room, self.front = ops, hq, hkv, h, n, room, front
        self.qkv, self.out = ops.DominoLinear(h, h + 2 * hkv * D), ops.DominoLinear(h, h)
        self.rot = ops.DominoQKRotary(**rotation)
        with torch.no_grad():
            for i, m in enumerate((self.qkv, self.out)):
                m.weight.copy_(randn(*m.weight.shape, seed=seed + i, std=h ** -0.5))
                m.bias.copy_(randn(m.bias.numel(), seed=seed + 2 + i, std=0.3))
            if self.rot.q_weight is not None:
                self.rot.q_weight.copy_(randn(D, seed=seed + 4, std=0.2, mean=1.2))
                self.rot.k_weight.copy_(randn(D, seed=seed + 5, std=0.2, mean=1.2))
        self.cache = ops.QuantizedCache.empty(front + n * room, hkv)
        self.cache.k.view(torch.uint8).fill_(127)  # rows that nothing has filled hold NaN
        self.cache.v.view(torch.uint8).fill_(127)

    def lists(self, new, old, shared=0):
        """rows, positions, start and length of sequences with `old` keys of their own behind the shared ones and `new` tokens."""
        rows, at = [], []
        for s, (a, c) in enumerate(zip(new, old)):
            rows += range(self.front + s * self.room + c, self.front + s * self.room + c + a)
            at += range(shared + c, shared + c + a)
        return (torch.tensor(rows, **I32), torch.tensor(at, **I32), self.front + torch.arange(len(new), **I32) * self.room,
                torch.tensor([a + c for a, c in zip(new, old)], **I32))

    def heads(self, x):
        return self.qkv(x).view(-1, self.hq + 2 * self.hkv, D).split([self.hq, self.hkv, self.hkv], 1)

    def decode(self, x, rows, at, start, length, prefix=None):
        """x [n x t, h]: the last t tokens of each sequence."""
        with torch.no_grad():
            q, k, v = self.heads(x)
            r = self.rot.write(self.cache, rows, q, k, v, at)
            r = r.view(start.numel(), -1, self.hq, D)
            o = self.ops.cached_attention(r, self.cache, start, length, prefix)
            return dict(x=x, q=q, k=k, v=v, r=r, o=o, y=self.out(o.view(-1, self.h), residual=x))

    def chunk(self, x, rows, at, cu, everything, first, length):
        """Packed tokens: their keys into the cache, the cache's `everything` read back in order, causal attention."""
        with torch.no_grad():
            q, k, v = self.heads(x)
            r = self.rot.write(self.cache, rows, q, k, v, at)
            o = self.ops.packed_attention(r, *self.ops.cache_read(self.cache, everything), cu, first, length)
            return dict(x=x, q=q, k=k, v=v, r=r, o=o, y=self.out(o.view(-1, self.h), residual=x))

    def check_written(self, st, rows, at):
        how = (at, self.rot.frequencies, self.rot.layout, self.rot.eps, self.rot.amplitude)
        ref, size = rotary(st["q"], self.rot.q_weight, *how)
        close(st["r"].reshape(ref.shape), ref, 40 * U32 * size, what="q")
        k, v = self.ops.cache_read(self.cache, rows)
        assert torch.equal(v.double(), held(st["v"].double()))
        ref, size = rotary(st["k"], self.rot.k_weight, *how)
        half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -9 * power(exponents(ref))[..., None])
        assert ((k.double() - ref).abs() <= half + 40 * U32 * size).all()

    def check_decode(self, st, rows, at, start, length, prefix=None):
        self.check_written(st, rows, at)
        ro, so, _, _ = cached.reference(st["r"], self.cache, start.tolist(), length.tolist(), prefix.tolist() if prefix is not None else None)
        close(st["o"], ro, so, what="o")
        lin.check_fwd(st["o"].view(-1, self.h), self.out.weight, self.out.bias, "none", st["x"], st["y"], None)


ROTATIONS = [dict(), dict(rot=64, layout="interleaved", norm=False, base=5e5), dict(rot=96, factor=4.0, original=1024, amplitude=1.1)]


@pytest.mark.parametrize("rotation", ROTATIONS, ids=str)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (6, 1), (5, 5)])
def test_prompts_chunks_tokens_and_drafts(ops, hq, hkv, rotation):
    n, room = 4, 700
    block = Block(ops, hq, hkv, n, room, **rotation)
    old = [0] * n
    for new in ([1, 130, 257, 64], [1, 70, 1, 300]):  # prompts; a chunk for some and a token for others
        rows, at, start, length = block.lists(new, old)
        old = length.tolist()
        everything = torch.cat([torch.arange(s * room, s * room + c, **I32) for s, c in enumerate(old)])
        edge = torch.tensor([0, *old], **I32).cumsum(0, dtype=torch.int32)
        cu = torch.tensor([0, *new], **I32).cumsum(0, dtype=torch.int32)
        st = block.chunk(randn(sum(new), block.h, seed=sum(new)), rows, at, cu, everything, edge[:-1].contiguous(), length)
        block.check_written(st, rows, at)
        kk, vv = block.ops.cache_read(block.cache, everything)
        c, e = cu.tolist(), edge.tolist()
        for s in range(n):
            ro, _, so, _ = attend64(st["r"][c[s]:c[s + 1]], kk[e[s]:e[s + 1]], vv[e[s]:e[s + 1]], D ** -0.5)
            close(st["o"][c[s]:c[s + 1]], ro, so, what=f"o of sequence {s}")
    for t in (1, 3, 1, 5):  # single tokens, and drafts of which the next step keeps two at most
        rows, at, start, length = block.lists([t] * n, old)
        st = block.decode(randn(n * t, block.h, seed=t), rows, at, start, length)
        block.check_decode(st, rows, at, start, length)
        old = [c + min(t, 2) for c in old]


def test_shared_rows_and_sequences_without_any(ops):
    """A prompt that all sequences share, written once; a sequence that leaves its batch as row -1 and length 0."""
    block = Block(ops, 8, 2, 5, 40, front=300)
    at = torch.arange(300, **I32)
    with torch.no_grad():
        q, k, v = block.heads(randn(300, block.h, seed=1))
        block.rot.write(block.cache, at, q, k, v, at)
    prefix = torch.tensor([0, 300], **I32)
    old = [0] * 5
    for step in range(3):
        rows, at, start, length = block.lists([1] * 5, old, shared=300)
        st = block.decode(randn(5, block.h, seed=step), rows, at, start, length, prefix)
        block.check_decode(st, rows, at, start, length, prefix)
        old = length.tolist()
    rows, at, start, length = block.lists([1] * 5, old, shared=300)
    rows[2], length[2] = -1, 0
    was = [x.clone() for x in block.cache]
    st = block.decode(randn(5, block.h, seed=9), rows, at, start, length)
    assert not st["o"][2].any() and st["o"][3].any()
    mine = slice(300 + 2 * 40, 300 + 3 * 40)
    assert all(torch.equal(a.view(torch.uint8)[mine], b.view(torch.uint8)[mine]) for a, b in zip(block.cache[:2], was))


def test_captured_steps(ops):
    """A step of single tokens captured once and replayed with other inputs, rows, positions, lengths and shared rows."""
    n = 6
    block = Block(ops, 8, 2, n, 200, front=100)
    at = torch.arange(100, **I32)
    with torch.no_grad():
        q, k, v = block.heads(randn(100, block.h, seed=1))
        block.rot.write(block.cache, at, q, k, v, at)
    prefix = torch.tensor([0, 100], **I32)
    x, old = randn(n, block.h, seed=2), [0] * n
    arg = block.lists([1] * n, old, shared=100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.decode(x, *arg, prefix)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = block.decode(x, *arg, prefix)
    for i in range(40):
        now = block.lists([1] * n, old, shared=100 - i)
        x.copy_(randn(n, block.h, seed=10 + i))
        for a, b in zip(arg, now):
            a.copy_(b)
        prefix[1] = 100 - i
        graph.replay()
        if i % 13 == 0:
            block.check_decode(st, *arg, prefix)
            got = {name: t.clone() for name, t in st.items()}
            again = block.decode(x, *arg, prefix)
            assert all(torch.equal(got[name], again[name]) for name in got)
        old = [c + 1 + (s == i % n) for s, c in enumerate(old)]
        # (a row that was passed over holds NaN: fill it as the step before would have)
        for c in block.cache[:2]:
            u = c.view(torch.uint8)
            u[u == 127] = 0


def test_two_captured_steps_at_once(ops):
    """Two captured steps of two blocks replayed on two streams at the same time, an eager one beside them: bits as alone."""
    runs = []
    for i in range(2):
        block = Block(ops, 8, 2, 3, 3000, seed=10 * i)
        for c in block.cache[:2]:
            c.view(torch.uint8).copy_(torch.randint(0, 100, c.shape, dtype=torch.uint8, device="cuda"))
        arg = block.lists([4] * 3, [2500 - i, 7, 1900])
        x = randn(12, block.h, seed=60 + i)
        block.decode(x, *arg)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st = block.decode(x, *arg)
        want = {name: t.clone() for name, t in block.decode(x, *arg).items()}
        runs.append((block, graph, st, want, (x, *arg), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for _, graph, _, _, _, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        block, _, _, want, arg, _ = runs[0]
        eager = ops.cached_attention(want["r"], block.cache, arg[3], arg[4])
    torch.cuda.synchronize()
    assert torch.equal(eager, runs[0][3]["o"])
    for _, _, st, want, _, _ in runs:
        assert all(torch.equal(st[name], want[name]) for name in want)


def test_threads_on_streams_of_their_own(ops):
    """Four threads call the operators at once, each on its stream: the bits of one thread alone, and no memory kept."""
    def work(i, times, stream):
        n, t, hq, hkv = 5 + i, 1 + i % 2, 8, 2
        tokens = n * t
        qkv = randn(tokens, hq + 2 * hkv, D, seed=i)
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        w, at = randn(D, seed=i + 20, mean=1.0), torch.arange(tokens, **I32) * 37
        f, cache = ops.rotary_frequencies(128), cached.random_cache(3000, hkv, seed=i)
        rows = torch.arange(tokens, **I32) + 7
        start, length, prefix = torch.arange(n, **I32) * 100, torch.arange(n, **I32) * 150, torch.tensor([0, 200 * i], **I32)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(times):
                r = ops.cache_write(cache, rows, k, v, q, at, f, w, w)
                o = ops.cached_attention(r.view(n, t, hq, D), cache, start, length, prefix)
                y = ops.qk_rotary_fwd(q, k, at, f, w, w)
                out = (r, o, *y, *ops.qk_rotary_bwd(*y, q, k, at, f, w, w), *ops.cache_read(cache, rows))
            stream.synchronize()
        return [t.clone() for t in out]

    streams = [torch.cuda.Stream() for _ in range(4)]
    want = [work(i, 1, streams[i]) for i in range(4)]
    got, failures = [None] * 4, []

    def run(i):
        try:
            got[i] = work(i, 50, streams[i])
        except Exception as e:  # shown below: a thread's exception ends that thread alone
            failures.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    del got, a, b
    before = torch.cuda.memory_allocated()
    work(0, 20, streams[0])
    assert torch.cuda.memory_allocated() == before


@pytest.mark.parametrize("rotation", ROTATIONS, ids=str)
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 4, 1), (130, 6, 2)])
def test_training_step(ops, tokens, hq, hkv, rotation):
    """Projection and rotation of a training step: every gradient against its formula on the stages' own values, and the same
    from a captured step."""
    block = Block(ops, hq, hkv, 1, 1, **rotation)
    rot, h = block.rot, block.h
    x, at = randn(tokens, h, seed=1).requires_grad_(), torch.arange(tokens, **I32) * 5
    gq, gk, gv = randn(tokens, hq, D, seed=2), randn(tokens, hkv, D, seed=3), randn(tokens, hkv, D, seed=4)
    parameters = [x, *block.qkv.parameters(), *rot.parameters()]

    def step():
        qkv = block.qkv(x)
        q, k, v = qkv.view(tokens, -1, D).split([hq, hkv, hkv], 1)
        rq, rk = rot(q, k, at)
        return qkv, rq, rk, torch.autograd.grad((rq, rk, v), [qkv, *parameters], (gq, gk, gv))

    qkv, rq, rk, (gqkv, gx, gw, gb, *gn) = step()
    how = (at, rot.frequencies, rot.layout, rot.eps, rot.amplitude)
    with torch.no_grad():
        heads, inner = qkv.view(tokens, -1, D), gqkv.view(tokens, -1, D)
        for i, (lo, n, y, gy, w) in enumerate(((0, hq, rq, gq, rot.q_weight), (hq, hkv, rk, gk, rot.k_weight))):
            ref, size = rotary(heads[:, lo:lo + n], w, *how)
            close(y, ref, 40 * U32 * size, what="y")
            ref, gref, size, gsize = rotary_grad(gy, heads[:, lo:lo + n], w, *how)
            close(inner[:, lo:lo + n], ref, 80 * U32 * size, what="gradient of the projection's output")
            if w is not None:
                close(gn[i], gref, (60 + tokens * 2 + 100) * U32 * gsize, what="gradient of the norm's weight")
        assert torch.equal(inner[:, hq + hkv:], gv)
        # the linear layer's, from the gradient that it got
        lin.check_bwd(gqkv, x, block.qkv.weight, None, "none", gx, gw, None)
        close(gb, gqkv.double().sum(0), (tokens / 8 + 300) * U32 * gqkv.double().abs().sum(0), what="gradient of the bias")
    # The same captured, without an eager step's graph alive: PyTorch's engine would wait for the streams of the leaves' nodes in
    # it, which a capture may not (with any function).
    del heads, inner, y
    first = [t.detach() for t in (qkv, rq, rk, gqkv, gx, gw, gb, *gn)]
    del qkv, rq, rk
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        again = step()
    again = [t.detach() for t in (*again[:3], *again[3])]
    with torch.no_grad():
        x.copy_(randn(tokens, h, seed=8))
    graph.replay()
    fresh = step()
    for a, b in zip(again, (*fresh[:3], *fresh[3])):
        assert torch.equal(a, b)
    with torch.no_grad():
        x.copy_(randn(tokens, h, seed=1))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(again, first):
        assert torch.equal(a, b)


def test_gradients_through_attention_match_differences(ops):
    """Dense causal attention in PyTorch's fp64 around the rotation: its gradients through the module against differences of the
    64-bit whole along random directions."""
    tokens, hq = 24, 2
    rot = ops.DominoQKRotary(rot=64, layout="interleaved")
    at = torch.arange(tokens, **I32) + 100
    q, k, v = (randn(tokens, hq, D, seed=i).requires_grad_() for i in range(3))
    go = randn(tokens, hq, D, seed=5)

    def whole(rq, rk, v):
        s = torch.einsum("qhd,khd->hqk", rq, rk) * D ** -0.5
        s = s.masked_fill(torch.ones(tokens, tokens, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        return (torch.einsum("hqk,khd->qhd", s.softmax(-1), v) * go.double()).sum()

    rq, rk = rot(q, k, at)
    a, b = rq.detach().double().requires_grad_(), rk.detach().double().requires_grad_()
    v64 = v.detach().double().requires_grad_()
    whole(a, b, v64).backward()
    # the gradients that reach the rotation are rounded to bf16 there, as every activation's
    torch.autograd.backward((rq, rk), (a.grad.bfloat16(), b.grad.bfloat16()))

    def f(q, k, wq, wk):
        def r(x, w):
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
            return turn(x, *cos_sin(at, rot.frequencies), "interleaved")
        return whole(r(q, wq), r(k, wk), v.detach().double())

    point = [p.detach().double() for p in (q, k, rot.q_weight, rot.k_weight)]
    grads = [p.grad.double() for p in (q, k, rot.q_weight, rot.k_weight)]
    for i, (p, g) in enumerate(zip(point, grads)):
        # along the gradient itself the slope is its norm; 1e-5 of the point's norm leaves differences of 1e-9 relative
        d = g / g.norm()
        e = 1e-5 * p.norm()
        moved = [[x + s * e * d if j == i else x for j, x in enumerate(point)] for s in (1, -1)]
        slope = (f(*moved[0]) - f(*moved[1])) / (2 * e)
        # rotated heads, their gradients and the results are each rounded to bf16 once, of which the heads' reach the
        # gradient through scores whose size is at most 4 here
        assert abs(slope - g.norm()) <= 12 * BF16 * g.norm(), (i, float(slope), float(g.norm()))
