"""The packed attention's scale works in base 2, where it has to be finite too.  The C ABI alone, no device is touched."""
import pytest

from comm_overlap_gb300 import domino as dm

P = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_overlap_gb300 import build
    build.build()


@pytest.mark.parametrize("scale,refused", [(3e38, True), (2.4e38, True), (float("inf"), True), (float("nan"), True), (0.0, True), (1e-60, True),
                                           (2.3e38, False), (1.0, False), (1e-38, False), (1e-45, False)])
def test_scale(scale, refused):
    with pytest.raises(dm.DominoError) as e:
        dm.domino_attn_packed_fwd(None, P, 1024, P, 256, P, 256, P, P, P, scale, P, 1024, None, 4, 2, 8, 2, 100, P, 1 << 30, stream=0)
    assert e.value.status == 1 and ("scale" in dm.domino_last_error()) == refused  # the other calls stop at the handle
