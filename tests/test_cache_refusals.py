"""What the rotation, the 8-bit cache and its attention refuse, at the C ABI (no device is touched: arguments are checked before the
handle) and in the PyTorch functions."""
import pytest
import torch

from comm_overlap_gb300 import domino as dm
from comm_overlap_gb300 import torch_ops as ops

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # an aligned address that is never read
O = 0x20000


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_overlap_gb300 import build
    build.build()


def status(fn, **kw):
    with pytest.raises(dm.DominoError) as e:
        fn(**kw)
    assert dm.domino_last_error()
    return e.value.status


def rotary_fwd(**kw):
    a = dict(handle=None, Q=P, ld_q=1024, K=P, ld_k=256, positions=P, frequencies=P, rot=128, layout=0, amplitude=1.0, wq=P, wk=P,
             eps=1e-6, Yq=O, ld_yq=1024, Yk=O, ld_yk=256, tokens=4, heads=8, kv_heads=2, stream=0)
    dm.domino_qk_rotary_fwd(**{**a, **kw})


ROTATION = [
    (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(heads=0, kv_heads=0), INVALID), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(heads=5000, ld_q=640000, ld_yq=640000), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=144), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(layout=2), INVALID), (dict(amplitude=float("nan")), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(positions=None), INVALID), (dict(positions=P + 2), ALIGNMENT),
    (dict(frequencies=None), INVALID), (dict(frequencies=P + 4), ALIGNMENT), (dict(wq=None), INVALID), (dict(wk=None), INVALID),
    (dict(wq=P + 2), ALIGNMENT), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(Q=None), INVALID),
    (dict(Q=P + 8), ALIGNMENT), (dict(K=None), INVALID), (dict(ld_q=1016), INVALID), (dict(ld_q=1028), ALIGNMENT), (dict(ld_k=128), INVALID),
    (dict(), INVALID),  # everything fine but the handle
    (dict(rot=0, positions=None, frequencies=None), INVALID), (dict(wq=None, wk=None, eps=0.0), INVALID),
    (dict(kv_heads=0, K=None, wk=None, ld_k=0, Yk=None), INVALID), (dict(tokens=0, Q=None, K=None, positions=None), INVALID)]


@pytest.mark.parametrize("kw,code", ROTATION + [
    (dict(Yq=None), INVALID), (dict(Yk=O + 4), ALIGNMENT), (dict(ld_yq=8), INVALID), (dict(Yq=P, ld_q=1032), INVALID),
    (dict(Yk=P, ld_yk=264), INVALID), (dict(Yq=P, Yk=P), INVALID)])
def test_rotation_forward(kw, code):
    assert status(rotary_fwd, **kw) == code


def rotary_bwd(**kw):
    a = dict(handle=None, gYq=P, ld_gyq=1024, gYk=P, ld_gyk=256, Q=P, ld_q=1024, K=P, ld_k=256, positions=P, frequencies=P, rot=128, layout=0,
             amplitude=1.0, wq=P, wk=P, eps=1e-6, gQ=O, ld_gq=1024, gK=O, ld_gk=256, gwq=P, gwk=P, accumulate=0, tokens=4, heads=8, kv_heads=2,
             workspace=P, workspace_bytes=1 << 20, stream=0)
    dm.domino_qk_rotary_bwd(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [x for x in ROTATION if "kv_heads" not in x[0] or x[0].get("heads") == 0] + [
    (dict(gYq=None), INVALID), (dict(gYk=P + 2), ALIGNMENT), (dict(ld_gyq=8), INVALID), (dict(gQ=None), INVALID), (dict(ld_gk=132), INVALID),
    (dict(gwq=None), INVALID), (dict(gwk=P + 4), ALIGNMENT), (dict(accumulate=2), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 16), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE), (dict(gQ=P, ld_gq=1032), INVALID),
    (dict(wq=None, wk=None, Q=None, K=None, gwq=None, gwk=None, workspace=None, workspace_bytes=0), INVALID)])
def test_rotation_backward(kw, code):
    if "ld_q" in kw and "ld_yq" in kw:
        kw = dict(kw, ld_gyq=640000, ld_gq=640000)
        kw.pop("ld_yq")
    assert status(rotary_bwd, **kw) == code


def test_rotation_workspace_size():
    size = dm.domino_qk_rotary_bwd_workspace_size
    assert size(0, 8, 2) == 0
    # 128 partial sums a block; a token's steps of eight heads by a warp each, four warps a block, each kind its own
    assert size(1, 8, 2) == 2 * 512 and size(1, 32, 8) == 2 * 512 and size(1, 64, 1) == 3 * 512
    assert size(1 << 20, 32, 8) <= 152 * 3 * 512
    assert status(size, tokens=-1, heads=8, kv_heads=2) == INVALID


def write(**kw):
    a = dict(handle=None, Q=P, ld_q=1024, K=P, ld_k=256, V=P, ld_v=256, positions=P, frequencies=P, rot=64, layout=1, amplitude=1.0, wq=P, wk=P,
             eps=1e-6, Yq=O, ld_yq=1024, rows=P, k8=O, v8=O, k_exp=O, v_exp=O, ld_exp=100, cache_rows=100, tokens=4, heads=8, kv_heads=2,
             stream=0)
    dm.domino_cache_write(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(kv_heads=0), INVALID), (dict(tokens=-1), INVALID), (dict(cache_rows=-1), INVALID), (dict(cache_rows=1 << 31, ld_exp=1 << 31), UNSUPPORTED),
    (dict(ld_exp=99), INVALID), (dict(ld_exp=(1 << 32) + 1), UNSUPPORTED), (dict(k8=None), INVALID), (dict(v8=O + 8), ALIGNMENT),
    (dict(k_exp=None), INVALID), (dict(v_exp=None), INVALID), (dict(rows=None), INVALID), (dict(rows=P + 2), ALIGNMENT), (dict(V=None), INVALID),
    (dict(ld_v=128), INVALID), (dict(K=P + 2), ALIGNMENT), (dict(rot=40), UNSUPPORTED), (dict(layout=7), INVALID), (dict(positions=None), INVALID),
    (dict(wk=None), INVALID), (dict(eps=-1.0), INVALID), (dict(Yq=None), INVALID), (dict(Yq=P, ld_yq=1032), INVALID), (dict(), INVALID),
    (dict(heads=0, Q=None, Yq=None, wq=None), INVALID), (dict(k_exp=O + 1, v_exp=O + 3), INVALID)])
def test_cache_write(kw, code):
    assert status(write, **kw) == code


def read(**kw):
    a = dict(handle=None, k8=P, v8=P, k_exp=P, v_exp=P, ld_exp=100, cache_rows=100, rows=P, K=O, ld_k=256, V=O, ld_v=256, tokens=4, kv_heads=2,
             stream=0)
    dm.domino_cache_read(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(kv_heads=0), INVALID), (dict(tokens=-1), INVALID), (dict(ld_exp=10), INVALID), (dict(k8=P + 4), ALIGNMENT), (dict(v_exp=None), INVALID),
    (dict(rows=None), INVALID), (dict(K=None), INVALID), (dict(ld_v=250), INVALID), (dict(V=O + 2), ALIGNMENT), (dict(), INVALID),
    (dict(cache_rows=0, ld_exp=0, k8=None, v8=None, k_exp=None, v_exp=None), INVALID)])
def test_cache_read(kw, code):
    assert status(read, **kw) == code


def attn(**kw):
    a = dict(handle=None, Q=P, ld_q=1024, k8=P, v8=P, k_exp=P, v_exp=P, ld_exp=100, cache_rows=100, k_start=P, k_len=P, prefix=P, scale=0.1, O=O,
             ld_o=1024, lse=P, n=2, t=3, heads=8, kv_heads=2, workspace=P, workspace_bytes=1 << 30, stream=0)
    dm.domino_attn_cached_fwd(**{**a, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(t=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID),
    (dict(heads=8192, kv_heads=8192), UNSUPPORTED), (dict(n=1 << 25), UNSUPPORTED), (dict(t=1 << 25), UNSUPPORTED),
    (dict(n=1 << 20, t=1 << 10), UNSUPPORTED), (dict(cache_rows=-1), INVALID), (dict(ld_exp=8), INVALID), (dict(k8=None), INVALID),
    (dict(v8=P + 8), ALIGNMENT), (dict(k_exp=None), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=8200.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(ld_q=1000), INVALID),
    (dict(ld_o=1028), ALIGNMENT), (dict(Q=None), INVALID), (dict(O=O + 2), ALIGNMENT), (dict(O=P), INVALID), (dict(lse=P + 4), ALIGNMENT),
    (dict(k_start=None), INVALID), (dict(k_len=P + 2), ALIGNMENT), (dict(prefix=P + 1), ALIGNMENT), (dict(workspace=None), WORKSPACE),
    (dict(workspace=P + 64), WORKSPACE), (dict(workspace_bytes=1000), WORKSPACE), (dict(), INVALID), (dict(prefix=None, lse=None), INVALID)])
def test_cached_attention(kw, code):
    assert status(attn, **kw) == code


def test_cached_attention_workspace_size():
    size = dm.domino_attn_cached_workspace_size
    assert size(0, 1, 8, 2, 0) == 0 and size(4, 0, 8, 2, 1) == 0
    # two partial results of a block's rows (8, 16 or 32, of 132 floats) for each of 304 blocks
    for t, rows in ((1, 8), (2, 8), (3, 16), (5, 32), (100, 32)):
        assert 0 < size(4, t, 8, 2, 0) - 2 * 304 * rows * 132 * 4 < 1024
    # with shared rows blocks hold rows of all sequences, and what was not cut is kept as well
    assert 0 < size(4, 1, 8, 2, 1) - 2 * 304 * 16 * 132 * 4 - 2 * 4 * 8 * 132 * 4 < 1024
    assert status(size, n=1, t=1, heads=3, kv_heads=2, prefix=0) == INVALID


def test_frequencies():
    f = ops.rotary_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(ops.rotary_frequencies(8, factor=4.0, device="cpu"), f / 4)
    # over 1000 positions the pairs turn 159, 15.9, 1.59 and 0.159 times: the first two stay, the last is divided, the third on the ramp
    g = ops.rotary_frequencies(8, factor=4.0, original=1000, device="cpu")
    keep = (10 / (2 * torch.pi) - 1) / 3
    assert torch.equal(g[:2], f[:2]) and g[3] == f[3] / 4 and abs(float(g[2] / f[2]) - (keep + (1 - keep) / 4)) < 1e-12
    for kw in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=-1.0), dict(rot=8, original=10, slow=4.0, fast=4.0)):
        with pytest.raises(ValueError):
            ops.rotary_frequencies(device="cpu", **kw)


def test_functions_refuse_what_they_cannot_take():
    q, v = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    w = torch.zeros(128, dtype=torch.bfloat16)
    cache = ops.QuantizedCache.empty(10, 8, device="cpu")
    f = ops.rotary_frequencies(128, device="cpu")
    for call in (lambda: ops.qk_rotary_fwd(q, q, v, f, w, w), lambda: ops.qk_rotary(q, q, v, f), lambda: ops.qk_rotary_bwd(q, q, q, q, v, f, w, w),
                 lambda: ops.cache_write(cache, v, q, q), lambda: ops.cache_read(cache, v), lambda: ops.cached_attention(q, cache, v, v),
                 lambda: ops.qk_rotary_fwd(None, None, None, None), lambda: ops.cache_read(cache, [1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="layout"):
        ops.DominoQKRotary(128, layout="diagonal", device="cpu")
    assert cache.k.dtype == torch.float8_e4m3fn and cache.k.shape == (10, 8, 128) and cache.k_exp.shape == (8, 10)


@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(grad):
    import torch.autograd.forward_ad as forward_ad
    x, w = torch.randn(4, 2, 128).bfloat16(), torch.ones(128).bfloat16()
    at, cache = torch.zeros(4, dtype=torch.int32), ops.QuantizedCache.empty(10, 2, device="cpu")
    f = ops.rotary_frequencies(128, device="cpu")
    for name, args, call in (("qk_rotary", (x, x, w, w), lambda q, k, a, b: ops.qk_rotary(q, k, at, f, a, b)),
                             ("cache_write", (x, x, x, w, w), lambda k, v, q, a, b: ops.cache_write(cache, at, k, v, q, at, f, a, b)),
                             ("cached_attention", (x,), lambda q: ops.cached_attention(q, cache, at, at))):
        for i in range(len(args)):
            with torch.set_grad_enabled(grad), forward_ad.dual_level():
                dual = list(args)
                dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(NotImplementedError, match=name):
                    call(*dual)


def test_no_backward_is_refused():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, requires_grad=True)
    y, at, cache = x.detach(), torch.zeros(4, dtype=torch.int32), ops.QuantizedCache.empty(10, 2, device="cpu")
    for call in (lambda: ops.cache_write(cache, at, x, y), lambda: ops.cache_write(cache, at, y, x), lambda: ops.cache_write(cache, at, y, y, x)):
        with pytest.raises(ValueError, match="no backward"):
            call()


def test_the_short_way_leaves_what_is_not_on_a_gpu():
    """torch_calls is built beside the library; without a handle, and for tensors of the CPU, it takes nothing."""
    from comm_overlap_gb300 import torch_calls as t
    x, at, f = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), ops.rotary_frequencies(128, device="cpu")
    cache = ops.QuantizedCache.empty(10, 2, device="cpu")
    assert t.qk_rotary_fwd(x, x, at, f, None, None, 0, 1e-6, 1.0) is None
    assert t.qk_rotary_bwd(x, x, None, None, at, f, None, None, 0, 1e-6, 1.0) is None
    assert t.cache_write(cache, at, x, x, None, None, None, None, None, 0, 1e-6, 1.0) is None
    assert t.cache_read(cache, at) is None and t.cached_attention(x, cache, at, at, None, 0.1, False) is None
    for args in ((), (1, 2, 3), (None,) * 12):
        assert t.qk_rotary_fwd(*args) is None and t.cache_read(*args) is None and t.cached_attention(*args) is None
    with pytest.raises(TypeError):
        t.use(1)
    with pytest.raises(TypeError):
        t.use_handle("device", 0)
