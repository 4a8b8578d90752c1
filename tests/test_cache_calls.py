"""The PyTorch functions of the 8-bit cache's attention and the rotation around their short way, without a GPU."""
import torch

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
