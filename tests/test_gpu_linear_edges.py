"""The linear layers around the attention where they may go wrong: waits that run out in
products of few blocks, norms of rows far from zero, dropout in forwards that the backward
runs again.  Inputs, tolerances and the oracle are those of test_gpu_linear_ops.py where
nothing else is said."""
import numpy as np
import pytest
import torch

from oracle import linear as OL
from tests.test_gpu_linear_ops import (TYPES, F, _close, _f64, _norm_inputs, _product, _randn, _run,  # noqa: F401
                                       _state, bl, built)

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


@pytest.mark.parametrize("M", [5, 300])
def test_products_of_scales_beyond_fp32(bl, M):  # noqa: F811
    """Scales whose product is beyond 2^128: infinite where the block's codes have a sum, NaN where
    they have none; other blocks, and products of as large a scale with a small one, are right."""
    N, K = 256, 256
    codes = torch.ones(M, K, device="cuda")
    codes[1] = 0
    codes = codes.to(torch.float8_e4m3fn)
    ones = torch.ones(N, K, device="cuda").to(torch.float8_e4m3fn)
    sa = torch.full((M, 2), 2.0 ** 70, device="cuda")
    sa[3] = 1.0
    sb = torch.full((2, 2), 2.0 ** -70, device="cuda")
    sb[1] = 2.0 ** 70
    y = bl.matmul8(bl.Act8(codes, sa, 128, torch.float32), bl.Weight8(ones, sb, torch.float32))
    assert torch.isnan(y[1, 128:]).all() and (y[1, :128] == 0).all()
    assert (y[3, :128] == 256 * 2.0 ** -70).all() and (y[3, 128:] == 256 * 2.0 ** 70).all()
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[1] = rest[3] = False
    assert (y[rest, :128] == 256).all() and (y[rest, 128:] == float("inf")).all()


# --- layer norm ------------------------------------------------------------------

FAR = [1, 24, 128, 200, 520, 1000, 1001, 1024, 2561, 4096, 5120, 8192, 8200, 12288, 16383]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", FAR)
def test_layer_norm_of_one_number(bl, cols, dtype):  # noqa: F811
    """Rows of one number c whose sum is exact in fp32 (at most 11 bits times 2^14): the mean is c,
    y the bias, and g_w 0; whatever the width, the alignment and the output."""
    t = TYPES[dtype]
    c = torch.tensor([1000.0, -0.75, 3.0, 0.0, 40.0], dtype=t, device="cuda")
    wide = torch.zeros(5, cols + 16, dtype=t, device="cuda")
    w, b = 1 + 0.3 * _randn(cols, seed=1), 0.3 * _randn(cols, seed=2)
    for off in (0, 1, 8):
        x = wide[:, off:off + cols]
        x.copy_(c[:, None].expand(5, cols))
        for weight, bias in ((w, b), (None, None), (w.to(t), b.to(t))):
            y, _, mean, rstd = bl.layer_norm_fwd(x, weight, bias)
            want = torch.zeros_like(y) if bias is None else bias.to(t).expand(5, cols)
            assert torch.equal(y, want) and torch.equal(mean, c.float())
            assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-3)
            for group in (128, 0):
                y8 = bl.layer_norm_fwd_8bit(x, weight, bias, group=group)[0]
                # the codes of the bias, the same in every row
                assert (y8.codes.view(torch.uint8) == y8.codes.view(torch.uint8)[:1]).all()
                assert bias is not None or (y8.codes.float() == 0).all()
    g = _randn(5, cols, dtype=t, seed=3)
    for weight in (None, w):
        _, gw, _ = bl.layer_norm_bwd(g, x.contiguous(), mean, rstd, weight)
        assert (gw == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", FAR)
def test_layer_norm_takes_the_mean_away_first(bl, cols, dtype):  # noqa: F811
    """y from the mean and rstd that are returned: one rounding each of h - mean, of its product
    with rstd and of the last multiply-add, whatever the mean is."""
    t = TYPES[dtype]
    wide = torch.zeros(6, cols + 16, dtype=t, device="cuda")
    w, b = 1 + 0.3 * _randn(cols, seed=1), 0.3 * _randn(cols, seed=2)
    for off in (0, 3):
        x = wide[:, off:off + cols]
        x.copy_(1000 + 4 * _randn(6, cols, seed=cols))
        for weight, bias in ((w, b), (None, None)):
            y, _, mean, rstd = bl.layer_norm_fwd(x, weight, bias)
            u = (_f64(x) - _f64(mean)[:, None]) * _f64(rstd)[:, None]
            wv, bv = (1.0, 0.0) if weight is None else (_f64(weight), _f64(bias))
            _close(y, u * wv + bv, 4 * F * (np.abs(u * wv) + np.abs(bv)), t)


@pytest.mark.parametrize("saved", [None, "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", FAR)
def test_layer_norm_backward_of_rows_far_from_zero(bl, cols, dtype, saved):  # noqa: F811
    """Of the mean and rstd that it is given: u carries 3 F of itself (h - mean and the product,
    or the multiply-add of a code), whatever the mean is."""
    t = TYPES[dtype]
    rows = 40
    x = (1000 + 4 * _randn(rows, cols, seed=cols)).to(t)
    _, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
    h = x if saved is None else bl.act_save(x, saved, 128)
    hv = _f64(x)
    if saved is not None:                                # code times scale, unrounded
        hv = _f64(h.codes.float()) * np.repeat(_f64(h.scales), 128, 1)[:, :cols]
    g, w = _randn(rows, cols, dtype=t, seed=8), 1 + 0.3 * _randn(cols, seed=9)
    gx, gw, gb = bl.layer_norm_bwd(g, h, mean, rstd, w)
    rx, rw, rb = OL.layer_norm_backward(g, hv, mean, rstd, w)
    s = _f64(rstd)[:, None]
    u = np.abs((hv - _f64(mean)[:, None]) * s)
    du = 3 * F * u
    gv = np.abs(_f64(g))
    wg = gv * _f64(w)
    c, dc = (wg * u).mean(1, keepdims=True), (wg * du).mean(1, keepdims=True)
    terms = s * (wg + wg.mean(1, keepdims=True) + u * c)
    _close(gx, rx, 64 * F * terms + s * (du * c + u * dc + du * dc), t)
    _close(gw, rw, (rows + 64) * F * (gv * u).sum(0) + (gv * du).sum(0), torch.float32)
    _close(gb, rb, (rows + 64) * F * gv.sum(0), torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [768, 1024, 2048, 4096, 5120, 8192])
def test_layer_norm_of_rows_that_begin_with_outliers(bl, cols, dtype):  # noqa: F811
    """Rows whose first 8 elements, whose first lane's 16 and whose first warp's elements stand
    apart from the rest: the pivots of the sums of squares are as far off as they can be.  Of a
    sum within 64 F of itself, 31 parts in 32 go where a warp's elements are put right and 15 in
    16 over the warps: the variance within 64 (32 + 16) F, rstd within half of that; 1600 F with
    what the mean adds."""
    t = TYPES[dtype]
    threads = (cols // 8 + (0 if cols <= 1024 else 1)) // (1 if cols <= 1024 else 2)
    threads = -(-threads // 32) * 32
    where = torch.zeros(5, cols, dtype=torch.bool, device="cuda")
    where[0, :8] = where[1, :8] = where[2, :256] = where[3, -8:] = True
    if cols > 1024:                                      # a lane's second chunk
        where[1, threads * 8:threads * 8 + 8] = where[2, threads * 8:threads * 8 + 256] = True
    for apart, spread in ((1.0, 1e-3), (-300.0, 1.0), (1.0, 0.0)):
        x = (spread * _randn(5, cols, seed=cols) + apart * where).to(t)
        y, _, mean, rstd = bl.layer_norm_fwd(x, None, None, 0.0 if spread else 1e-5)
        ry, _, rm, rs = OL.layer_norm(x, None, None, 0.0 if spread else 1e-5)
        xv = _f64(x)
        _close(mean, rm, 64 * F * np.abs(xv).mean(1), torch.float32)
        rows = slice(0, 5) if spread else slice(0, 4)    # the last row without a spread is zeros
        _close(rstd[rows], rs[rows], 1600 * F * rs[rows], torch.float32)
        off = (64 * F * np.abs(xv).mean(1, keepdims=True) + 2 * F * np.abs(xv)) * rs[:, None]
        _close(y, ry, off + 1600 * F * np.abs(ry), t)


FORMS = [("fp16", "fp16", None, 0), ("fp16", "fp32", None, 0), ("bf16", "bf16", None, 0),
         ("bf16", "bf16", "int8", 32), ("bf16", "fp32", "e4m3", 64), ("bf16", "bf16", "int8", 0),
         ("fp16", "fp16", "e4m3", 32), ("fp16", "fp32", "int8", 64), ("fp16", "fp16", "e4m3", 0),
         ("fp32", "fp32", "int8", 32), ("fp32", "fp32", "e4m3", 0), ("fp16", "fp32", "int8", 128)]


@pytest.mark.parametrize("dtype,wtype,saved,group", FORMS)
@pytest.mark.parametrize("rows,cols", [(3, 7), (33, 128), (40, 264), (9, 520), (5, 1001), (300, 1024), (5, 2561),
                                       (1200, 4096), (4, 5120), (3, 8200), (2, 16384)])
def test_layer_norm_backward_of_other_forms(bl, rows, cols, dtype, wtype, saved, group):  # noqa: F811
    """fp16, weights of 16 bits, and 8 bits with groups of 32 and 64 and with a scale a row."""
    t, wt = TYPES[dtype], TYPES[wtype]
    x, _, w, _ = _norm_inputs(rows, cols, t, wt, seed=cols + 3)
    _, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
    h, hv = x, _f64(x)
    if saved is not None:
        h = bl.act_save(x, saved, group)
        hv = _f64(h.codes.float()) * np.repeat(_f64(h.scales).reshape(rows, -1), group or cols, 1)[:, :cols]
    g, gh = _randn(rows, cols, dtype=t, seed=8), _randn(rows, cols, dtype=t, seed=9)
    for g_h in (gh, None):
        gx, gw, gb = bl.layer_norm_bwd(g, h, mean, rstd, w, g_h=g_h)
        rx, rw, rb = OL.layer_norm_backward(g, hv, mean, rstd, w, g_h)
        s = _f64(rstd)[:, None]
        u = np.abs((hv - _f64(mean)[:, None]) * s)
        du = 3 * F * u
        gv = np.abs(_f64(g))
        wg = gv * np.abs(_f64(w))
        c, dc = (wg * u).mean(1, keepdims=True), (wg * du).mean(1, keepdims=True)
        terms = s * (wg + wg.mean(1, keepdims=True) + u * c)
        slack = 64 * F * terms + s * (du * c + u * dc + du * dc)
        _close(gx, rx, slack if g_h is None else slack + F * np.abs(_f64(g_h)), t)
        assert gw.dtype == wt and gb.dtype == wt
        _close(gw, rw, (rows + 64) * F * (gv * u).sum(0) + (gv * du).sum(0), wt)
        _close(gb, rb, (rows + 64) * F * gv.sum(0), wt)


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


def test_dropout_past_the_counter_s_upper_word(bl):  # noqa: F811
    """Elements on either side of 2^34, where the counter of four elements passes 32 bits: in place
    on a dense tensor, and element by element on one that starts at an odd place."""
    from block_sparse_attention_fwd_gb300 import linear
    n, st = 2 ** 34 + 43, _state(3, 4)
    buf = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")
    places = (0, 2 ** 32 - 20, 2 ** 33 - 20, 2 ** 34 - 60, 2 ** 34 - 20, n - 48)
    for off in (0, 1):
        buf.fill_(1.0)
        x = buf[off:off + n]
        linear._launch("bl_dropout", x.device, 1, n, 0, x.data_ptr(), n, None, n, 0.5, st.data_ptr(),
                       x.data_ptr())
        for at in places:
            keep = OL.kept(48, 0.5, 3, 4, first=at)
            assert (_f64(x[at:at + 48])[:n - at] == np.where(keep, 2.0, 0.0)[:n - at]).all(), (off, at)
        assert float(buf[n - off * n]) == 1.0            # the neighbour stays
