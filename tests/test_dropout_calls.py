"""BLDropout's states on the host: which call takes which, in forwards that the backward runs
again.  The two library calls are stood in for by the oracle (CPU only)."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from block_sparse_attention_fwd_gb300 import api, linear
from oracle import linear as OL


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    def dropout(x, p, state, residual=None):
        seed, offset = state.tolist()
        keep = torch.from_numpy(OL.kept(x.numel(), p, seed, offset)).view(x.shape)
        y = torch.where(keep, x / (1 - p), 0.0)
        return y if residual is None else y + residual

    def dropout_next(state):
        used = state.clone()
        state[1] += 1
        return used

    monkeypatch.setattr(linear, "dropout", dropout)
    monkeypatch.setattr(linear, "dropout_next", dropout_next)


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_call_run_again_takes_the_state_that_it_is_given(reentrant):
    drop = api.BLDropout(0.5, seed=3, device="cpu")
    x = torch.ones(40, requires_grad=True)
    for call in range(2):
        # what comes behind is saved from the second run: its mask has to be the first's too
        y = checkpoint(lambda x, used: drop(x, used=used).exp(), x, linear.dropout_next(drop.state),
                       use_reentrant=reentrant)
        g, = torch.autograd.grad(y.sum(), x) if not reentrant else (None,)
        if reentrant:
            x.grad = None
            y.sum().backward()
            g = x.grad
        keep = torch.from_numpy(OL.kept(40, 0.5, 3, call))
        assert torch.equal(y.detach(), torch.where(keep, 2.0, 0.0).exp())
        assert torch.equal(g, torch.where(keep, 2 * torch.tensor(2.0).exp(), 0.0))
        assert drop.state.tolist() == [3, call + 1]


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_call_run_again_without_its_state_is_refused(reentrant):
    drop = api.BLDropout(0.5, seed=3, device="cpu")
    x = torch.ones(40, requires_grad=True)
    y = checkpoint(lambda x: drop(x).exp(), x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="dropout_next"):
        y.sum().backward()
    assert drop.state.tolist() == [3, 1]
    drop.eval()                                          # nothing is drawn
    checkpoint(lambda x: drop(x).exp(), x, use_reentrant=reentrant).sum().backward()


def test_a_call_may_not_take_the_state_that_goes_on():
    drop = api.BLDropout(0.5, seed=3, device="cpu")
    with pytest.raises(ValueError):
        drop(torch.ones(4), used=drop.state)
    y = drop(torch.ones(40), used=torch.tensor([3, 7]))
    assert torch.equal(y != 0, torch.from_numpy(OL.kept(40, 0.5, 3, 7))) and drop.state.tolist() == [3, 0]
