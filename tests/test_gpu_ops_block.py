"""The sublayer operators together: a pre-LN block that serves prompts, chunks and single tokens over a cache, and a
training step of its LayerNorm and linear layers.

Every stage is compared with its definition in 64 bits on the bf16 values that it was given, with the bounds of the
operators' own tests, so no bound has to be carried through the block."""
import pytest
import torch

import test_gpu_ops_linear as lin
import test_gpu_ops_norm as norm
from ops_helpers import BF16, close, device_ok, randn
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


class Block:
    """y = t + MLP(LN(t)), t = x + out(attention(qkv(LN(x)))), over caches of `room` rows a sequence."""

    def __init__(self, ops, hq, hkv, f, n, room):
        h = hq * D
        self.ops, self.hq, self.hkv, self.h, self.room = ops, hq, hkv, h, room
        self.n1, self.n2 = (ops.DominoLayerNorm(h) for _ in range(2))
        self.qkv, self.out = ops.DominoLinear(h, h + 2 * hkv * D, init_std=h ** -0.5), ops.DominoLinear(h, h, init_std=h ** -0.5)
        self.up, self.down = ops.DominoLinear(h, f, act="gelu", init_std=h ** -0.5), ops.DominoLinear(f, h, init_std=f ** -0.5)
        with torch.no_grad():
            for i, m in enumerate((self.n1, self.n2, self.qkv, self.out, self.up, self.down)):
                m.bias.copy_(randn(m.bias.numel(), seed=i, std=0.3))
                if i < 2:
                    m.weight.copy_(randn(h, seed=10 + i, std=0.2, mean=1.0))
                else:
                    std = m.weight.shape[1] ** -0.5
                    m.weight.copy_(randn(*m.weight.shape, seed=20 + i, std=std))
        # rows that no sequence has filled hold NaN
        self.k, self.v = (torch.full((n * room, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(self, x, rows, cu, start, length):
        """One pass over packed tokens; `rows`: where their keys and values go.  Returns all stages."""
        with torch.no_grad():
            a = self.n1(x)
            qkv = self.qkv(a)
            heads = qkv.view(-1, self.hq + 2 * self.hkv, D)
            q, k, v = heads.split([self.hq, self.hkv, self.hkv], 1)
            self.k.index_copy_(0, rows, k)
            self.v.index_copy_(0, rows, v)
            o = self.ops.packed_attention(q, self.k, self.v, cu, start, length)
            t = self.out(o.view(-1, self.h), residual=x)
            b = self.n2(t)
            u = self.up(b)
            return dict(x=x, a=a, qkv=qkv, o=o, t=t, b=b, u=u, y=self.down(u, residual=t))

    def lengths(self, queries, cached):
        """rows, cu, start, length of sequences with `cached` keys and as many new tokens as `queries` says."""
        i64, i32 = dict(dtype=torch.int64, device="cuda"), dict(dtype=torch.int32, device="cuda")
        cu = [0]
        rows = []
        for s, (a, c) in enumerate(zip(queries, cached)):
            cu.append(cu[-1] + a)
            rows += range(s * self.room + c, s * self.room + c + a)
        return (torch.tensor(rows, **i64), torch.tensor(cu, **i32), torch.arange(len(queries), **i32) * self.room,
                torch.tensor([a + c for a, c in zip(queries, cached)], **i32))

    def check(self, st, cu, start, length):
        def stats(w, b, x, y):
            norm.check_fwd(x, w, b, 1e-5, (y, *self.ops.layer_norm_fwd(x, w, b)[1:]))

        with torch.no_grad():
            stats(self.n1.weight, self.n1.bias, st["x"], st["a"])
            lin.check_fwd(st["a"], self.qkv.weight, self.qkv.bias, "none", None, st["qkv"], None)
            q = st["qkv"].view(-1, self.hq + 2 * self.hkv, D)[:, :self.hq]
            c, s0, n = cu.tolist(), start.tolist(), length.tolist()
            for s in range(len(n)):
                ro, _, so, _ = attend64(q[c[s]:c[s + 1]], self.k[s0[s]:s0[s] + n[s]], self.v[s0[s]:s0[s] + n[s]], D ** -0.5)
                close(st["o"][c[s]:c[s + 1]], ro, so, what=f"O of sequence {s}")
            lin.check_fwd(st["o"].view(-1, self.h), self.out.weight, self.out.bias, "none", st["x"], st["t"], None)
            stats(self.n2.weight, self.n2.bias, st["t"], st["b"])
            lin.check_fwd(st["b"], self.up.weight, self.up.bias, "gelu", None, st["u"], None)
            lin.check_fwd(st["u"], self.down.weight, self.down.bias, "none", st["t"], st["y"], None)


@pytest.mark.parametrize("hq,hkv", [(4, 2), (6, 1), (5, 5)])
def test_serving_block(ops, hq, hkv):
    """Prompts, then a chunk for some and a token for others, then single tokens, the last captured and replayed."""
    block = Block(ops, hq, hkv, 1032, 4, 700)
    cached = [0] * 4
    for queries in ([1, 130, 257, 64], [1, 70, 1, 300], [1, 0, 1, 1]):
        rows, cu, start, length = block.lengths(queries, cached)
        st = block.step(randn(sum(queries), block.h, seed=sum(queries)), rows, cu, start, length)
        block.check(st, cu, start, length)
        cached = [a + b for a, b in zip(queries, cached)]
    # single tokens through a captured graph: new inputs, rows and lengths in its buffers
    queries = [1, 1, 1, 1]
    x = randn(4, block.h, seed=9)
    rows, cu, start, length = block.lengths(queries, cached)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, rows, cu, start, length)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block.step(x, rows, cu, start, length)
    for i in range(3):
        now = block.lengths(queries, cached)
        x.copy_(randn(4, block.h, seed=30 + i))
        rows.copy_(now[0])
        length.copy_(now[3])
        graph.replay()
        block.check(held, cu, start, length)
        again = block.step(x, rows, cu, start, length)
        assert all(torch.equal(held[name], again[name]) for name in held)
        cached = [c + 1 for c in cached]


def test_modules_without_gradients(ops):
    """The same bits with and without a backward pass to follow, and nothing kept for one without."""
    ln, up = ops.DominoLayerNorm(520), ops.DominoLinear(520, 1032, act="gelu")
    x, r = randn(3, 70, 520, seed=1), randn(3, 70, 1032, seed=2)
    want = up(ln(x), r)
    assert want.requires_grad and want.shape == (3, 70, 1032)
    with torch.no_grad():
        got = up(ln(x), r)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        held = up(ln(x), r)
        # the two outputs alone, in the allocator's steps of 512 bytes, and the scratch that it has given back
        assert torch.cuda.memory_allocated() - before <= held.numel() * 2 + 512
    for p in (*ln.parameters(), *up.parameters()):
        p.requires_grad_(False)
    frozen = up(ln(x), r)
    assert torch.equal(got, want) and torch.equal(frozen, want) and torch.equal(held, want)
    assert not got.requires_grad and not frozen.requires_grad
    x.requires_grad_()
    up(ln(x), r).sum().backward()  # a frozen layer still passes the gradient on
    assert x.grad is not None and torch.isfinite(x.grad).all()


def test_threads_on_streams_of_their_own(ops):
    """Four threads call the operators at once, each on its stream: the bits of one thread alone, and no memory kept."""
    import threading

    def work(i, times, stream):
        m, h, f = 40 + 300 * (i % 2), 520, 1032
        x, w, b = randn(m, h, seed=i), randn(f, h, seed=i + 10, std=0.05), randn(f, seed=i + 20)
        g, q = randn(h, seed=i + 30, mean=1.0), randn(m, 3, D, seed=i + 40)
        cu = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(times):
                n, mean, rstd = ops.layer_norm_fwd(x, g)
                y, z = ops.linear_fwd(n, w, b, "gelu", save=True)
                gx, gw, gb = ops.linear_bwd(y, n, w, z, "gelu")
                out = (y, gx, gw, gb, *ops.layer_norm_bwd(gx, x, g, mean, rstd), ops.packed_attention(q, q[:, :1], q[:, 1:2], cu))
            stream.synchronize()
        return [t.clone() for t in out if t is not None]

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


def test_two_captured_steps_at_once(ops):
    """Two captured steps of two blocks, replayed on two streams at the same time, and an eager one beside them."""
    runs = []
    for i in range(2):
        block = Block(ops, 4, 2, 1032, 3, 2000)
        queries, cached = [1, 1, 1], [1500 - i, 7, 1900]
        block.k[:], block.v[:] = randn(*block.k.shape, seed=40 + i), randn(*block.v.shape, seed=50 + i)
        rows, cu, start, length = block.lengths(queries, cached)
        x = randn(3, block.h, seed=60 + i)
        block.step(x, rows, cu, start, length)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = block.step(x, rows, cu, start, length)
        want = {name: t.clone() for name, t in block.step(x, rows, cu, start, length).items()}
        runs.append((block, graph, held, want, (x, rows, cu, start, length), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, graph, _, _, _, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = runs[0][0].ops.linear_fwd(runs[0][4][0], runs[0][0].qkv.weight)[0]
    torch.cuda.synchronize()
    for _, _, held, want, _, _ in runs:
        assert all(torch.equal(held[name], want[name]) for name in want)
    lin.check_fwd(runs[0][4][0], runs[0][0].qkv.weight, None, "none", None, eager, None)


@pytest.mark.parametrize("rows,h,f", [(1, 512, 1024), (300, 520, 1032), (777, 1024, 256)])
def test_training_step(ops, rows, h, f):
    """y = x + down(gelu(up(LN(x)))): every gradient against its formula on the stages' own values, and the whole
    against 64-bit differentiation."""
    ln, up = ops.DominoLayerNorm(h), ops.DominoLinear(h, f, act="gelu")
    down = ops.DominoLinear(f, h, fuse_wgrad=True)
    with torch.no_grad():
        ln.weight.copy_(randn(h, seed=1, std=0.2, mean=1.0))
        for i, p in enumerate((ln.bias, up.bias, down.bias)):
            p.copy_(randn(p.numel(), seed=2 + i, std=0.3))
        up.weight.copy_(randn(f, h, seed=5, std=h ** -0.5))
        down.weight.copy_(randn(h, f, seed=6, std=f ** -0.5))
    x, gy = randn(rows, h, seed=7, mean=0.5).requires_grad_(), randn(rows, h, seed=8)
    a = ln(x)
    a.retain_grad()
    u = up(a)
    u.retain_grad()
    y = down(u, residual=x)
    y.backward(gy)
    with torch.no_grad():
        _, mean, rstd = ops.layer_norm_fwd(x, ln.weight, ln.bias)
        norm.check_fwd(x, ln.weight, ln.bias, 1e-5, (a, mean, rstd))
        _, z = ops.linear_fwd(a, up.weight, up.bias, "gelu", save=True)
        lin.check_fwd(a, up.weight, up.bias, "gelu", None, u, z)
        lin.check_fwd(u, down.weight, down.bias, "none", x, y, None)
        zero_w, zero_b = torch.zeros_like(down.weight.main_grad), torch.zeros_like(down.bias.main_grad)
        lin.check_bwd(gy, u, down.weight, None, "none", u.grad, down.weight.main_grad, down.bias.main_grad, zero_w, zero_b)
        lin.check_bwd(u.grad, a, up.weight, z, "gelu", a.grad, up.weight.grad, None)
        # the bias gradient of bf16 parameters is rounded once more than the operator's
        gz = u.grad.double() * lin.grad64("gelu", z.double())
        close(up.bias.grad, gz.sum(0), 2e-6 * u.grad.double().abs().sum(0) + (rows / 8 + 300) * 2.0 ** -24 * gz.abs().sum(0), what="gbias")
        # the residual's gradient is added to LayerNorm's, which was rounded before
        gx, gw, gb = norm.bwd64(a.grad, x, ln.weight, mean, rstd, None)
        inner = ops.layer_norm_bwd(a.grad, x, ln.weight, mean, rstd)
        norm.check_bwd(a.grad, x, ln.weight, mean, rstd, None, inner)
        close(x.grad, inner[0].double() + gy.double(), 0, what="gx")
        close(ln.weight.grad, inner[1], 0, what="gweight")
        close(ln.bias.grad, inner[2], 0, what="gbias of LayerNorm")
    # The whole in 64 bits.  Eight roundings to bf16 lie between x and a gradient, each at most half a step of its
    # tensor's norm; a product passes an error on with at most 2.5 times the gain that it has for what it is given
    # (the largest singular value of a matrix of independent values over their root mean square: 1 + sqrt of its
    # sides' ratio, at most 3 here for one of the two products and 1.6 for the other, between which the norm's
    # projection and gelu' <= 1.13 do not add).
    x64 = x.detach().double().requires_grad_()
    p = [t.detach().double().requires_grad_() for t in (ln.weight, ln.bias, up.weight, up.bias, down.weight, down.bias)]
    n64 = torch.nn.functional.layer_norm(x64, (h,), p[0], p[1], 1e-5)
    y64 = lin.act64("gelu", n64 @ p[2].t() + p[3]) @ p[4].t() + p[5] + x64
    y64.backward(gy.double())
    got = (x.grad, ln.weight.grad, ln.bias.grad, up.weight.grad, up.bias.grad, down.weight.main_grad, down.bias.main_grad)
    for g, w in zip(got, (x64, *p)):
        assert (g.double() - w.grad).norm() <= 20 * BF16 * w.grad.norm()
