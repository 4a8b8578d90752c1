"""Outputs of the rotation, the 8-bit cache and its attention that overlap an input, at the C ABI: refused where one row tells (no device is
touched: the addresses are never read)."""
import pytest

from comm_overlap_gb300 import domino as dm

P, FAR, LD, D = 0x1000000, 0x9000000, 4096, 128  # bytes, bytes, elements, elements
ROW, HEAD = 2 * LD, 2 * D


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_overlap_gb300 import build
    build.build()


def said(fn, **kw):
    with pytest.raises(dm.DominoError) as e:
        fn(handle=None, stream=0, **kw)
    assert e.value.status == 1
    return dm.domino_last_error()


def forward(**kw):
    a = dict(Q=P, ld_q=LD, K=P + 8 * HEAD, ld_k=LD, positions=P, frequencies=P, rot=128, layout=0, amplitude=1.0, wq=None, wk=None, eps=1e-6,
             Yq=FAR, ld_yq=LD, Yk=FAR + 8 * HEAD, ld_yk=LD, tokens=10, heads=8, kv_heads=2)
    return said(dm.domino_qk_rotary_fwd, **{**a, **kw})


def backward(**kw):
    a = dict(gYq=P, ld_gyq=LD, gYk=P + 8 * HEAD, ld_gyk=LD, Q=2 * FAR, ld_q=LD, K=2 * FAR + 8 * HEAD, ld_k=LD, positions=P, frequencies=P, rot=128,
             layout=0, amplitude=1.0, wq=P, wk=P, eps=1e-6, gQ=FAR, ld_gq=LD, gK=FAR + 8 * HEAD, ld_gk=LD, gwq=P, gwk=P, accumulate=0, tokens=10,
             heads=8, kv_heads=2, workspace=P, workspace_bytes=1 << 20)
    return said(dm.domino_qk_rotary_bwd, **{**a, **kw})


def write(**kw):
    a = dict(Q=P, ld_q=LD, K=P + 8 * HEAD, ld_k=LD, V=P + 10 * HEAD, ld_v=LD, positions=P, frequencies=P, rot=64, layout=1, amplitude=1.0, wq=None,
             wk=None, eps=1e-6, Yq=FAR, ld_yq=LD, rows=P, k8=P, v8=P, k_exp=P, v_exp=P, ld_exp=100, cache_rows=100, tokens=10, heads=8, kv_heads=2)
    return said(dm.domino_cache_write, **{**a, **kw})


def attention(**kw):
    a = dict(Q=P, ld_q=LD, k8=P, v8=P, k_exp=P, v_exp=P, ld_exp=100, cache_rows=100, k_start=P, k_len=P, prefix=None, scale=0.1, O=FAR, ld_o=LD,
             lse=None, n=5, t=2, heads=8, kv_heads=2, workspace=P, workspace_bytes=1 << 30)
    return said(dm.domino_attn_cached_fwd, **{**a, **kw})


@pytest.mark.parametrize("call,out", [(forward, "Yq"), (backward, "gQ"), (write, "Yq"), (attention, "O")])
def test_overlaps(call, out):
    at = "gYq" if call is backward else "Q"
    # a head, a row and more on or back, up to the last value in common
    for by in (HEAD, -HEAD, 7 * HEAD, -7 * HEAD, ROW, -ROW, 9 * ROW, -9 * ROW, 9 * ROW + 7 * HEAD, -9 * ROW - 7 * HEAD, 8 * HEAD - 16, 3 * ROW - 8 * HEAD + 16):
        assert f"{out} and {at} overlap" in call(**{out: P + by}), by
    # beside the others of a row, and past the ends
    free = 8 + 2 + 2  # heads of the inputs
    for by in (free * HEAD, -8 * HEAD, ROW - 8 * HEAD, 10 * ROW, -10 * ROW, 10 * ROW + HEAD, -10 * ROW - HEAD, 9 * ROW + free * HEAD):
        assert "overlap" not in call(**{out: P + by}), by
    name = {"Yq": "ld_yq", "gQ": "ld_gq", "O": "ld_o"}[out]
    assert "overlap" not in call(**{out: P + ROW // 2, name: 2 * LD})  # another stride: not told


def test_one_token():
    for call, out, n in ((forward, "Yq", "tokens"), (write, "Yq", "tokens")):
        for by, bad in ((HEAD, True), (-HEAD, True), (12 * HEAD, False), (-8 * HEAD, False), (8 * HEAD, True), (10 * HEAD, call is write)):
            assert ("overlap" in call(**{out: P + by, n: 1, "ld_yq": 1024})) == bad, (call, by)
    assert "overlap" in attention(O=P + 7 * HEAD, n=1, t=1) and "overlap" not in attention(O=P + 8 * HEAD, n=1, t=1)


def test_in_place_and_crosswise():
    assert "handle" in forward(Yq=P, Yk=P + 8 * HEAD) and "handle" in write(Yq=P)
    assert "handle" in backward(gQ=P, gK=P + 8 * HEAD) and "handle" in backward(gQ=2 * FAR, gK=2 * FAR + 8 * HEAD)
    assert "Yq and K overlap" in forward(Yq=P + 8 * HEAD, Q=2 * FAR, ld_q=LD) and "Yk and Q overlap" in forward(Yk=P + 2 * HEAD)
    assert "gQ and K overlap" in backward(gQ=2 * FAR + 9 * HEAD) and "gK and Q overlap" in backward(gK=2 * FAR)
    assert "gQ and gYk overlap" in backward(gQ=P + 9 * HEAD) and "gK and gYq overlap" in backward(gK=P + 6 * HEAD)
    assert "gK and K overlap" in backward(gK=2 * FAR + 9 * HEAD)
    assert "Yq and K overlap" in write(Yq=P + 9 * HEAD) and "Yq and V overlap" in write(Yq=P + 11 * HEAD)
    assert "different row strides" in backward(gQ=2 * FAR, ld_gq=2 * LD) and "different row strides" in backward(gK=2 * FAR + 8 * HEAD, ld_gk=2 * LD)
