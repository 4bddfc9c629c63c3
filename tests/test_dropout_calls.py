"""BLDropout's states on the host: which call takes which, in forwards that the backward runs
again and on the ranks of a data-parallel wrapper, and how they are kept.  The two library
calls are stood in for by the oracle (CPU only)."""
import copy

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp
from torch.utils.checkpoint import checkpoint

from block_sparse_attention_fwd_gb300 import api, linear
from oracle import linear as OL
from tests.test_multi_rank import _free_port


def _dropout(x, p, state, residual=None):
    seed, offset = state.tolist()
    keep = torch.from_numpy(OL.kept(x.numel(), p, seed, offset)).view(x.shape)
    y = torch.where(keep, x / (1 - p), 0.0)
    return y if residual is None else y + residual


def _dropout_next(state):
    used = state.clone()
    state[1] += 1
    return used


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(linear, "dropout", _dropout)
    monkeypatch.setattr(linear, "dropout_next", _dropout_next)


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
    with pytest.raises(TypeError):
        drop(torch.ones(4), used=7)
    y = drop(torch.ones(40), used=torch.tensor([3, 7]))
    assert torch.equal(y != 0, torch.from_numpy(OL.kept(40, 0.5, 3, 7))) and drop.state.tolist() == [3, 0]


def _rank(rank, world, port, out):
    linear.dropout, linear.dropout_next = _dropout, _dropout_next
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=world)
    try:
        # a buffer, so that the wrapper has something to send
        model = torch.nn.Sequential(torch.nn.BatchNorm1d(40), api.BLDropout(0.5, seed=100 + rank, device="cpu"))
        ddp = torch.nn.parallel.DistributedDataParallel(model)
        for _ in range(3):
            y = ddp(torch.randn(4, 40))
            y.sum().backward()
        out[rank] = (model[1].state.tolist(), (y != 0).tolist())
    finally:
        dist.destroy_process_group()


def test_ranks_of_a_data_parallel_wrapper_keep_their_states():
    out = mp.get_context("spawn").Manager().dict()
    mp.start_processes(_rank, args=(2, _free_port(), out), nprocs=2, join=True, start_method="spawn")
    for rank in range(2):
        state, kept = out[rank]
        assert state == [100 + rank, 3]
        assert kept == torch.from_numpy(OL.kept(160, 0.5, 100 + rank, 2)).view(4, 40).tolist()


def test_states_are_saved_loaded_copied_and_moved():
    stack = torch.nn.Sequential(torch.nn.Linear(4, 4), api.BLDropout(0.5, seed=7, device="cpu"))
    drop = stack[1]
    drop(torch.ones(8))
    saved = stack.state_dict()
    assert saved["1.state"].tolist() == [7, 1] and not dict(drop.named_buffers())
    other = torch.nn.Sequential(torch.nn.Linear(4, 4), api.BLDropout(0.5, seed=8, device="cpu"))
    held = other[1].state
    other.load_state_dict({k: v.clone() for k, v in saved.items()})
    assert other[1].state is held and held.tolist() == [7, 1]
    other.load_state_dict({k: v.clone() for k, v in saved.items()}, assign=True)
    assert other[1].state.tolist() == [7, 1]
    twin = copy.deepcopy(stack)[1]
    assert twin.state.tolist() == [7, 1] and twin.state.data_ptr() != drop.state.data_ptr()
    twin.state[0] = 9
    assert not torch.equal(twin(torch.ones(99)), drop(torch.ones(99)))
    assert drop.half().state.dtype == torch.int64 and drop.to("meta").state.is_meta
    with pytest.raises(RuntimeError, match="Missing.*1.state"):
        other.load_state_dict({k: v for k, v in saved.items() if k != "1.state"})
    other.load_state_dict({k: v for k, v in saved.items() if k != "1.state"}, strict=False)
    with pytest.raises(RuntimeError, match="Unexpected.*1.scale"):
        other.load_state_dict({**saved, "1.scale": torch.ones(1)})
    with pytest.raises(RuntimeError, match="two int64"):
        other.load_state_dict({**saved, "1.state": torch.ones(2)})
    # a state_dict holds the tensors themselves, as a buffer's: drop has gone on
    assert other[1].state.tolist() == saved["1.state"].tolist() == [7, 2]
