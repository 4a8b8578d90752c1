"""Outputs in their inputs' place: allowed where both have the same row stride, refused where a row written would lie on
rows still to be read.  The C ABI alone, no device is touched; a call that passes every check stops at the NULL handle."""
import pytest

from comm_overlap_gb300 import domino as dm

P, Q = 0x10000, 0x200000  # aligned addresses that are never read
INVALID = 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_overlap_gb300 import build
    build.build()


def refusal(fn, *args):
    with pytest.raises(dm.DominoError) as e:
        fn(*args, stream=0)
    assert e.value.status == INVALID
    return dm.domino_last_error()


def ln_fwd(X, ld_x, Y, ld_y, rows=4):
    return refusal(dm.domino_layernorm_fwd, None, X, ld_x, P, P, 1e-5, Y, ld_y, None, None, rows, 64)


def ln_bwd(gY, ld_gy, gres, ld_gres, gX, ld_gx, rows=4):
    return refusal(dm.domino_layernorm_bwd, None, gY, ld_gy, Q + 4096, 64, P, P, P, gres, ld_gres, gX, ld_gx, P, P, 0, rows, 64, P, 1 << 20)


def lin_fwd(R, ld_r, Y, ld_y, M=4):
    return refusal(dm.domino_linear_fwd, None, P, 64, P, None, 0, R, ld_r, Y, ld_y, None, 0, M, 128, 64)


@pytest.mark.parametrize("fn,wrong,right", [
    (ln_fwd, [(P, 64, P, 72), (P, 128, P, 64)], [(P, 64, P, 64), (P, 128, P, 128), (P, 64, Q, 72), (P, 64, P, 72, 1), (P, 64, P, 72, 0)]),
    (ln_bwd, [(P, 64, None, 0, P, 72), (P, 128, None, 0, P, 64), (P, 64, Q, 64, Q, 72), (P, 64, Q, 72, Q, 64)],
     [(P, 64, None, 0, P, 64), (P, 128, Q, 64, P, 128), (P, 64, Q, 72, Q, 72), (P, 64, Q, 72, P + 16, 80), (P, 64, Q, 72, P, 80, 1),
      (P, 64, None, 0, P, 80, 0)]),
    (lin_fwd, [(P, 128, P, 136), (P, 256, P, 128), (P, 136, P, 128, 200)],
     [(P, 128, P, 128), (P, 256, P, 256), (P, 128, Q, 136), (None, 0, P, 136), (P, 128, P, 136, 1), (P, 128, P, 136, 0)])],
    ids=["layernorm_fwd", "layernorm_bwd", "linear_fwd"])
def test_strides_in_place(fn, wrong, right):
    for args in wrong:
        assert "stride" in fn(*args), args
    for args in right:
        assert "stride" not in fn(*args), args
