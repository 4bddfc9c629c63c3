"""The linear layers around the attention where they may go wrong: waits that run out in
products of few blocks, dropout in forwards that the backward runs again.  Inputs,
tolerances and the oracle are those of test_gpu_linear_ops.py."""
import pytest
import torch

from oracle import linear as OL
from tests.test_gpu_linear_ops import _product, _randn, _run, bl, built  # noqa: F401

pytestmark = pytest.mark.gpu


# --- products --------------------------------------------------------------------

@pytest.mark.parametrize("form,M,N,K", [
    ("y", 1000, 1024, 128), ("y", 300, 4096, 256), ("y", 3000, 2560, 128), ("y", 8, 4000, 128),
    ("y", 40, 9000, 512), ("g_x", 500, 128, 2000), ("g_x", 30, 300, 5000), ("g_w", 100, 1500, 1500),
    ("g_w", 500, 512, 512)])
def test_product_of_few_blocks_whose_waits_run_out(bl, form, M, N, K):  # noqa: F811
    """One to four blocks of the summed dim a CTA: its issuers are done before the accumulating
    warps give up, and its last products still under way.  What is left is NaN, the rest right,
    and so are calls behind it."""
    from block_sparse_attention_fwd_gb300 import _lib
    a, b, _ = _product(bl, form, M, N, K, "fp32", seed=9)
    want = _run(bl, form, a, b)
    for _ in range(5):
        was = _lib.set_wait_limit(0.0)
        try:
            left = [_run(bl, form, a, b) for _ in range(3)]
            torch.cuda.synchronize()
        finally:
            _lib.set_wait_limit(was)
        for got in left:
            assert (torch.isnan(got) | (got == want)).all()
        assert torch.equal(_run(bl, form, a, b), want)


# --- dropout ---------------------------------------------------------------------

@pytest.mark.parametrize("reentrant", [False, True])
def test_dropout_in_a_forward_that_is_run_again(bl, reentrant):  # noqa: F811
    """Under either kind of recomputation, with the call's state passed in, gradients are those of
    the same layers without it; without the state the backward is refused."""
    from torch.utils.checkpoint import checkpoint
    lin = bl.BLLinear8(256, 192, device="cuda", dtype=torch.bfloat16)
    drop = bl.BLDropout(0.4, seed=11, device="cuda")
    out = bl.BLLinear8(192, 256, device="cuda", dtype=torch.bfloat16)
    x = _randn(50, 256, dtype=torch.bfloat16, seed=1).requires_grad_()
    g = _randn(50, 256, dtype=torch.bfloat16, seed=2)
    leaves = [x, lin.weight, out.weight]

    def layers(x, used=None):
        return out(drop(lin(x), used=used))

    def gradients(y):
        for t in leaves:
            t.grad = None
        y.backward(g)
        return [t.grad for t in leaves]

    for call in range(2):
        used = bl.dropout_next(drop.state)
        y = checkpoint(layers, x, used, use_reentrant=reentrant)
        got = gradients(y)
        drop.state[1] -= 1
        plain = layers(x)
        want = gradients(plain)
        assert drop.state.tolist() == [11, call + 1]
        assert torch.equal(y, plain)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    y = checkpoint(layers, x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="dropout_next"):
        y.backward(g)


def test_dropout_run_again_replays_from_a_graph(bl):  # noqa: F811
    """A captured step with a recomputed forward: every replay draws anew, once, and its gradient
    has the mask of its output."""
    from torch.utils.checkpoint import checkpoint
    drop = bl.BLDropout(0.5, seed=4, device="cuda")
    x, g = _randn(33, 40, seed=1).requires_grad_(), _randn(33, 40, seed=2)

    def step():
        used = bl.dropout_next(drop.state)
        y = checkpoint(lambda x, used: drop(x, used=used) * 3, x, used, use_reentrant=False,
                       preserve_rng_state=False)
        return y.detach(), torch.autograd.grad(y, x, g)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, gx = step()
    for call in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        keep = torch.from_numpy(OL.kept(x.numel(), 0.5, 4, call)).view(x.shape).cuda()
        assert torch.equal(y != 0, keep) and torch.equal(gx != 0, keep)
        assert drop.state.tolist() == [4, call + 1]


def test_a_state_that_went_on_is_not_read_by_a_backward(bl):  # noqa: F811
    """A call given a tensor that dropout_next then moves on: its backward would form another mask,
    and is refused as after any change in place."""
    drop = bl.BLDropout(0.5, seed=4, device="cuda")
    x = _randn(8, 40, seed=1).requires_grad_()
    mine = torch.tensor([4, 7], device="cuda")
    y = drop(x, used=mine)
    bl.dropout_next(mine)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    drop(x, used=mine).sum().backward()
    with torch.inference_mode():
        state = torch.tensor([4, 7], device="cuda")
        assert bl.dropout_next(state).tolist() == [4, 7] and state.tolist() == [4, 8]
