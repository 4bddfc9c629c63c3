"""The linear layers around the attention where they may go wrong: waits that run out in
products of few blocks.  Inputs, tolerances and the oracle are those of
test_gpu_linear_ops.py."""
import pytest
import torch

from tests.test_gpu_linear_ops import _product, _run, bl, built  # noqa: F401

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
