"""The short way of the rotation, the 8-bit cache and its attention (torch_calls): the bits of the long way, taken for everything of the
plain form and for nothing else."""
import threading

import pytest
import torch

from cache_helpers import D, random_cache
from ops_helpers import device_ok, randn

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from comm_overlap_gb300 import build
    build.build()
    from comm_overlap_gb300 import torch_ops
    torch_ops.cache_read(torch_ops.QuantizedCache.empty(1, 1), torch.zeros(1, **I32))  # the device's first call
    assert torch_ops._short is not None, "torch_calls was not built"
    yield torch_ops
    device_ok()


def state(ops, tokens=6, hq=8, hkv=2, rot=64):
    q, k, v = randn(tokens, hq + 2 * hkv, D, seed=1).split([hq, hkv, hkv], 1)
    return dict(q=q, k=k, v=v, at=torch.arange(tokens, **I32) * 100, f=ops.rotary_frequencies(rot), wq=randn(D, seed=2), wk=randn(D, seed=3),
                cache=random_cache(300 + 30 * tokens, hkv), rows=torch.arange(tokens, **I32) + 5, start=torch.arange(tokens, **I32) * 7,
                length=torch.arange(tokens, **I32) * 20, prefix=torch.tensor([200, 40], **I32))


def first(x):
    return None if x is None else x[0]


def calls(ops, s):
    """(name, call, the short way's call with the same arguments)"""
    t, code = ops._short, ops.LAYOUTS
    rot, far = (s["at"], s["f"], s["wq"], s["wk"]), ("half", 1e-5, 1.5)
    how = dict(zip(("layout", "eps", "amplitude"), far))
    short = (code["half"], 1e-5, 1.5)
    bare = (None, None, None, None)
    return [
        ("fwd", lambda: ops.qk_rotary_fwd(s["q"], s["k"], *rot, **how), lambda: t.qk_rotary_fwd(s["q"], s["k"], *rot, *short)),
        ("fwd, queries alone", lambda: ops.qk_rotary_fwd(s["q"], None, *rot[:3], **how), lambda: t.qk_rotary_fwd(s["q"], None, *rot[:3], None, *short)),
        ("bwd", lambda: ops.qk_rotary_bwd(s["q"], s["k"], s["q"], s["k"], *rot, **how),
         lambda: t.qk_rotary_bwd(s["q"], s["k"], s["q"], s["k"], *rot, *short)),
        ("bwd, no norm", lambda: ops.qk_rotary_bwd(s["q"], s["k"], None, None, *rot[:2]),
         lambda: t.qk_rotary_bwd(s["q"], s["k"], None, None, *rot[:2], None, None, 0, 1e-6, 1.0)),
        ("write", lambda: ops.cache_write(s["cache"], s["rows"], s["k"], s["v"], s["q"], *rot, **how),
         lambda: first(t.cache_write(s["cache"], s["rows"], s["k"], s["v"], s["q"], *rot, *short))),
        ("write, bare", lambda: ops.cache_write(s["cache"], s["rows"], s["k"], s["v"]),
         lambda: first(t.cache_write(s["cache"], s["rows"], s["k"], s["v"], None, *bare, 0, 1e-6, 1.0))),
        ("read", lambda: ops.cache_read(s["cache"], s["rows"]), lambda: t.cache_read(s["cache"], s["rows"])),
        ("attention", lambda: ops.cached_attention(s["q"], s["cache"], s["start"], s["length"], s["prefix"], return_lse=True),
         lambda: t.cached_attention(s["q"], s["cache"], s["start"], s["length"], s["prefix"], D ** -0.5, True)),
        ("attention, two tokens", lambda: ops.cached_attention(s["q"].view(-1, 2, *s["q"].shape[1:]), s["cache"], s["start"][:3], s["length"][:3]),
         lambda: first(t.cached_attention(s["q"].view(-1, 2, *s["q"].shape[1:]), s["cache"], s["start"][:3], s["length"][:3], None, D ** -0.5,
                                          False))),
    ]


def flat(x, s):
    x = x if isinstance(x, tuple) else (x,)
    return [t.clone() for t in x if t is not None] + [c.view(torch.uint8).clone() for c in s["cache"]]


@pytest.mark.parametrize("i", range(9))
def test_same_bits_both_ways(ops, monkeypatch, i):
    s = state(ops)
    name, call, short = calls(ops, s)[i]
    with torch.no_grad():
        was = [c.clone() for c in s["cache"]]
        got = flat(short(), s)
        for c, b in zip(s["cache"], was):
            c.copy_(b)
        way = flat(call(), s)
        for c, b in zip(s["cache"], was):
            c.copy_(b)
        monkeypatch.setattr(ops, "_short", None)
        want = flat(call(), s)
    assert len(got) == len(want) == len(way)
    for a, b, c in zip(got, want, way):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b) and torch.equal(c, b), name


def other(x, kind):
    """A tensor of another form, or none."""
    if not isinstance(x, torch.Tensor):
        return None
    if kind == "cpu":
        return x.cpu()
    if kind == "type":
        return x.view(torch.uint8)[..., ::2] if x.element_size() == 2 else x.double() if x.dtype != torch.float64 else x.float()
    if kind == "dimension":
        return x[None]
    if kind == "strides":
        y = torch.empty((*x.shape, 2), dtype=x.dtype, device=x.device)[..., 0]
        return y.copy_(x)
    if kind == "alignment":
        y = torch.empty(x.numel() + 16, dtype=x.dtype, device=x.device)
        return y[1:x.numel() + 1].view(x.shape).copy_(x) if x.dtype == torch.bfloat16 else None
    if kind == "longer":
        return torch.cat([x, x], 0)


@pytest.mark.parametrize("kind", ["none", "cpu", "type", "dimension", "strides", "alignment", "longer"])
def test_what_is_not_plain_is_left(ops, kind):
    """Every tensor of every call in another form: the short way does not take it."""
    for i in (0, 2, 4, 6, 7):
        s = state(ops)
        names = {0: "q k at f wq wk", 2: "q k at f wq wk", 4: "q k v at f wq wk rows", 6: "rows", 7: "q start length prefix"}[i].split()
        for name in names:
            if kind == "longer" and (i, name) == (6, "rows") or kind == "none" and (i, name) == (7, "prefix"):
                continue  # (as good as the other)
            # (frequencies of another number are another rotation; without queries there is one weight too many)
            if kind == "longer" and name == "f":
                new = torch.cat([s["f"], s["f"], s["f"]])
            else:
                new = None if kind == "none" else other(s[name], kind)
                if new is None and kind != "none":
                    continue
            with torch.no_grad():
                assert calls(ops, dict(s, **{name: new}))[i][2]() is None, (kind, i, name)
    s = state(ops)
    if kind not in ("none", "alignment"):
        for part in range(4):
            cache = list(s["cache"])
            cache[part] = other(cache[part], kind)
            for i in (4, 6, 7):
                assert calls(ops, dict(s, cache=tuple(cache)))[i][2]() is None, (kind, i, part)


def test_other_arguments_are_left(ops):
    s, t = state(ops), ops._short
    rot = (s["at"], s["f"], s["wq"], s["wk"])
    for bad in ((2, 1e-6, 1.0), (None, 1e-6, 1.0), ("half", 1e-6, 1.0), (True, 1e-6, 1.0), (0, None, 1.0), (0, 1e-6, "1"), (0, 0.0, 1.0),
                (0, 1e-6, float("nan")), (1 << 80, 1e-6, 1.0), (0, 1 << 2000, 1.0)):
        assert t.qk_rotary_fwd(s["q"], s["k"], *rot, *bad) is None, bad
    assert t.qk_rotary_fwd(s["q"], s["k"]) is None and t.cache_read(s["cache"]) is None
    for scale in (None, 1, 0.0, -1.0, float("inf"), float("nan"), 1e5):
        assert t.cached_attention(s["q"], s["cache"], s["start"], s["length"], None, scale, False) is None, scale
    assert t.cached_attention(s["q"][:, :7], s["cache"], s["start"], s["length"], None, 0.1, False) is None
    assert t.cache_read(list(s["cache"]), s["rows"]) is None and t.cache_read(s["cache"][:3], s["rows"]) is None
    # gradients and subclasses
    q = s["q"].detach().requires_grad_()
    assert t.cached_attention(q, s["cache"], s["start"], s["length"], None, 0.1, False) is None
    assert t.cache_write(s["cache"], s["rows"], s["k"], s["v"], q, *rot, 0, 1e-6, 1.0) is None
    assert t.cache_write(s["cache"], s["rows"], s["k"], s["v"], s["q"], *rot[:2], torch.nn.Parameter(s["wq"]), s["wk"], 0, 1e-6, 1.0) is None
    with torch.no_grad():
        assert t.cached_attention(q, s["cache"], s["start"], s["length"], None, 0.1, False) is not None
        assert t.cached_attention(s["q"].as_subclass(type("T", (torch.Tensor,), {})), s["cache"], s["start"], s["length"], None, 0.1, False) is None
    with pytest.raises(ValueError, match="no backward"):
        ops.cached_attention(q, s["cache"], s["start"], s["length"])


def test_refusals_are_the_long_ways(ops):
    """Through the functions, which say what is wrong."""
    s = state(ops)
    f24 = ops.rotary_frequencies(24)
    for call, match in ((lambda: ops.qk_rotary_fwd(s["q"], s["k"], s["at"], f24, s["wq"], s["wk"]), "multiple of 8 frequencies"),
                        (lambda: ops.qk_rotary_fwd(s["q"], s["k"], s["at"].long(), s["f"], s["wq"], s["wk"]), "positions must be"),
                        (lambda: ops.qk_rotary_fwd(s["q"], s["k"], s["at"], s["f"], s["wq"]), "go together"),
                        (lambda: ops.qk_rotary_fwd(s["q"], s["k"], s["at"], s["f"], layout="third"), "layout must be"),
                        (lambda: ops.cache_write(s["cache"], s["rows"][:3], s["k"], s["v"]), "rows must have shape"),
                        (lambda: ops.cache_write(s["cache"], s["rows"], s["q"], s["v"]), "v has 2 heads, k 8"),
                        (lambda: ops.cache_read(s["cache"], s["rows"].long()), "rows must be"),
                        (lambda: ops.cached_attention(s["q"], s["cache"], s["start"], s["length"][:2]), "k_len must have shape"),
                        (lambda: ops.cached_attention(s["q"][:, :7], s["cache"], s["start"], s["length"]), "multiple of the cache's heads")):
        with torch.no_grad(), pytest.raises(ValueError, match=match):
            call()
    from comm_overlap_gb300 import domino as dm
    with torch.no_grad(), pytest.raises(dm.DominoError):
        ops.cached_attention(s["q"], s["cache"], s["start"], s["length"], scale=-1.0)
    # and nothing is left behind: the lock is free
    assert ops._lock.acquire(blocking=False)
    ops._lock.release()


def test_where_another_thread_has_the_lock(ops):
    """The short way does not wait: the long one does."""
    s = state(ops)
    want = ops.cache_read(s["cache"], s["rows"])
    got = []
    with ops._lock:
        assert ops._short.cache_read(s["cache"], s["rows"]) is None
        thread = threading.Thread(target=lambda: got.append(ops.cache_read(s["cache"], s["rows"])))
        thread.start()
        thread.join(0.2)
        assert thread.is_alive() and not got
    thread.join()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want))


def test_memory_is_given_back(ops):
    s = state(ops, tokens=64)
    run = [c for _, _, c in calls(ops, s)[:8]]
    with torch.no_grad():
        for c in run:
            c()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        for _ in range(20):
            for c in run:
                assert c() is not None or c is run[5]
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before
