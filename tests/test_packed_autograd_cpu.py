"""varlen_attention's dispatch to its autograd function, on the CPU: the launch is replaced."""
import pytest
import torch
from torch.autograd import forward_ad as fw

from block_sparse_attention_stats_b200 import packed as K


@pytest.fixture()
def args(monkeypatch):
    monkeypatch.setattr(K, "pisa_varlen_attention", lambda q, *a, **k: torch.zeros_like(q))
    q, k = torch.randn(4, 5, 64).bfloat16(), torch.randn(2, 5, 64).bfloat16()
    return [q, k, k.clone(), torch.tensor([0, 5], dtype=torch.int32)]


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("leaf", [False, True])
def test_forward_mode_is_refused(args, which, leaf):
    """A tangent is refused, never dropped."""
    with fw.dual_level():
        x = list(args)
        if leaf:
            x[1 if which == 0 else 0].requires_grad_()
        x[which] = fw.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises((ValueError, NotImplementedError, RuntimeError)):
            K.varlen_attention(*x)
        # under no_grad tangents flow too
        with torch.no_grad(), pytest.raises((ValueError, NotImplementedError, RuntimeError)):
            K.varlen_attention(*x)


def test_a_level_without_tangents_is_no_reason(args):
    with fw.dual_level():
        assert K.varlen_attention(*args).shape == args[0].shape
    assert K.varlen_attention(*args).grad_fn is None
