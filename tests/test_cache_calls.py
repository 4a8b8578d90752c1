"""The PyTorch functions of the 8-bit cache's attention and the rotation around their short way, without a GPU."""
import sys
import types

import pytest
import torch

from comm_overlap_gb300 import build
from comm_overlap_gb300 import torch_ops as ops


class Noted:
    """In the short way's place: notes its arguments and returns a pair."""

    def cached_attention(self, *args):
        self.args = args
        return "o", "lse" if args[-1] is True else None


def test_any_true_value_asks_for_the_logarithms(monkeypatch):
    """The short way looks for True itself."""
    monkeypatch.setattr(ops, "_short", Noted())
    for asked, want in ((True, ("o", "lse")), (1, ("o", "lse")), (torch.tensor(True), ("o", "lse")), (False, "o"), (0, "o"), (None, "o")):
        assert ops.cached_attention(torch.zeros(1), None, None, None, return_lse=asked) == want


def test_the_short_way_is_built_again_for_another_pytorch(monkeypatch, tmp_path):
    build.build()
    assert not build._calls_need_build()
    monkeypatch.setattr(build, "_torch_version", lambda: "1.0")
    assert build._calls_need_build()
    monkeypatch.undo()
    monkeypatch.setattr(build, "CALLS_FOR", str(tmp_path / "none"))
    assert build._calls_need_build()
    monkeypatch.undo()

    def unknown(name):
        raise build.importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(build.importlib.metadata, "version", unknown)
    assert build._torch_version() == torch.__version__


def test_the_short_way_is_taken_in_any_build_of_its_version(monkeypatch):
    build.build()
    from comm_overlap_gb300 import torch_calls
    monkeypatch.setattr(ops, "_short", None)
    monkeypatch.setattr(torch, "__version__", torch_calls.built_for + "a0+145a3a7.other")
    used = []
    monkeypatch.setattr(torch_calls, "use", lambda *a: used.append(a))
    monkeypatch.setattr(torch_calls, "use_handle", lambda *a: None)
    ops._shorten(0, 0)
    assert ops._short is torch_calls and used


@pytest.mark.parametrize("built", ["1.0", None])
def test_the_short_way_of_another_pytorch_is_not_taken(monkeypatch, built):
    """It reads fields of tensors, which lie elsewhere in another version."""
    import comm_overlap_gb300
    build.build()
    from comm_overlap_gb300 import torch_calls
    assert torch.__version__.startswith(torch_calls.built_for)
    other = types.ModuleType("comm_overlap_gb300.torch_calls")
    if built:
        other.built_for = built
    other.use = other.use_handle = lambda *a: pytest.fail("it is used")
    monkeypatch.setitem(sys.modules, "comm_overlap_gb300.torch_calls", other)
    monkeypatch.setattr(comm_overlap_gb300, "torch_calls", other)
    monkeypatch.setattr(ops, "_short", None)
    with pytest.warns(UserWarning, match="torch_calls"):
        ops._shorten(0, 1)
    assert ops._short is None


def test_a_module_built_without_memory_gets_its_frequencies():
    want = ops.DominoQKRotary(64, 5e5, device="cpu", factor=4.0, original=1000)
    module = ops.DominoQKRotary(64, 5e5, device="meta", factor=4.0, original=1000)
    assert module.frequencies.is_meta and module.half().frequencies.is_meta
    module = module.bfloat16().to_empty(device="cpu")
    assert torch.equal(module.frequencies, want.frequencies) and module.frequencies.dtype == torch.float64
    module.load_state_dict(want.state_dict())
    assert torch.equal(module.q_weight, want.q_weight) and module.q_weight.dtype == torch.bfloat16
    assert torch.equal(module.float().frequencies, want.frequencies)
    # what a user has put there stays through a cast
    module.frequencies = want.frequencies * 2
    assert torch.equal(module.bfloat16().frequencies, want.frequencies * 2)
    assert module.to("meta").frequencies.is_meta
