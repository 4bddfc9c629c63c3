"""Products in 8 bits, the layer norm and dropout on the GPU against the fp64 oracle,
element by element.

Tolerances count roundings.  half(t) = finfo(t).eps / 2 is one rounding to the type t,
relative; F = 2^-24 is one in fp32.
 * product: within a block of 128 the tensor core adds exact products in fp32 and may
   truncate (2 F of the running sum a term); over the blocks a sum in order and the
   product of two scales: (2 * 128 + blocks + 4) F of the sum of the terms' magnitudes.
 * layer norm: the mean is off by at most 64 F of the mean magnitude (32 elements a
   thread and 15 levels of adding, and its base), an element's distance from it by that
   and 2 F |h|, the residual's addition by F.  The squares: 64 F of their sum, the
   distance's own error, and what putting parts with other means together takes away, at
   most 10 times the rest: rstd within 256 F (1 + rms(h) / sigma).
 * layer norm backward: u carries 4 F (|h| + |m|) rstd; a term of g_x 64 F of all terms'
   magnitudes and what u's error makes of them.  g_w, g_b: (rows + 64) F of the sum of
   magnitudes.
 * dropout: the scale's rounding and the product's, 2 F |x scale|, and one of the sum.
An fp16 result below the smallest normal is off by half a subnormal step more.
"""
import numpy as np
import pytest
import torch

from oracle import linear as OL
from oracle.attention import _f64 as _np64

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(scope="module")
def bl():
    import block_sparse_attention_fwd_gb300 as bl
    return bl


def _f64(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, slack, dtype):
    """|got - ref| <= half a step of the type, plus `slack` from the fp32 arithmetic."""
    info = torch.finfo(dtype)
    got = _f64(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    bound = info.eps / 2 * (np.abs(ref) + slack) + slack + info.smallest_normal * info.eps / 2
    over = np.abs(got - ref) > bound
    assert not over.any(), (int(over.sum()), np.argwhere(over)[:3].tolist(),
                            float((np.abs(got - ref) - bound).max()))


def _randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


# --- saving ----------------------------------------------------------------------

TILES = [(1, 1), (1, 128), (128, 128), (129, 127), (5, 300), (200, 16), (384, 640), (77, 1001), (256, 40),
         (130, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", TILES)
def test_saved_rows_columns_and_blocks(bl, rows, cols, dtype):
    """Bit for bit: rows as act_save, columns as act_save of the transposed tensor, blocks as
    the definition; and the values that they load as."""
    t = TYPES[dtype]
    x = _randn(rows, cols, dtype=t, seed=rows + cols) * torch.exp2(_randn(cols, seed=1)).to(t)
    a, c = bl.act_save_both(x)
    want = bl.act_save(x, "e4m3", 128)
    assert torch.equal(a.codes.view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(a.scales, want.scales)
    down = bl.act_save(x.t().contiguous(), "e4m3", 128)
    assert torch.equal(c.codes.view(torch.uint8), down.codes.view(torch.uint8).t())
    assert torch.equal(c.scales, down.scales.t())
    only_a, none = bl.act_save_both(x, cols=False)
    none_a, only_c = bl.act_save_both(x, rows=False)
    assert none is None and none_a is None
    assert torch.equal(only_a.codes.view(torch.uint8), a.codes.view(torch.uint8))
    assert torch.equal(only_c.codes.view(torch.uint8), c.codes.view(torch.uint8))
    w = bl.weight_save(x)
    scales = OL.block_scales(x.float().cpu().numpy(), 128, 128)
    assert (w.scales.cpu().numpy() == scales).all()
    each = OL.spread(scales, 128, 128, rows, cols)
    values = OL.encode(x.float().cpu().numpy(), each)
    assert (OL.e4m3_values(w.codes.contiguous().view(torch.uint8).cpu().numpy()) == values).all()
    loaded = torch.from_numpy((values.astype(np.float32) * each)).cuda().to(t)
    assert torch.equal(bl.act_load(w), loaded)
    assert torch.equal(bl.act_load(c), bl.act_load(down).t())


def test_saved_views_and_edges(bl):
    x = _randn(300, 400, dtype=torch.bfloat16, seed=3)
    for v in (x[:, 8:264], x[10:, 3:300], x[::2], x.view(3, 100, 400)[1]):
        a, c = bl.act_save_both(v)
        b, d = bl.act_save_both(v.contiguous())
        assert torch.equal(a.scales, b.scales) and torch.equal(c.scales, d.scales)
        assert torch.equal(bl.act_load(a), bl.act_load(b)) and torch.equal(bl.act_load(c), bl.act_load(d))
    # several dims: rows as they are, columns over all tokens
    a, c = bl.act_save_both(x.view(3, 100, 400))
    assert a.shape == (3, 100, 400) and c.shape == (300, 400) and c.scales.shape == (3, 400)
    # zeros, the largest values, and what is not finite: its group alone loads as NaN
    y = torch.zeros(256, 256, device="cuda")
    y[0, 0], y[130, 5], y[200, 200] = 3.4e38, float("nan"), float("-inf")
    a, c = bl.act_save_both(y)
    w = bl.act_load(bl.weight_save(y))
    a, c = bl.act_load(a), bl.act_load(c)
    assert a[0, 0] > 3e38 and c[0, 0] > 3e38 and w[0, 0] > 3e38
    assert torch.isnan(a[130, :128]).all() and torch.isnan(a[200, 128:]).all()
    assert torch.isnan(c[128:, 5]).all() and torch.isnan(c[128:, 200]).all()
    assert torch.isnan(w[128:, :]).all() and torch.isfinite(w[:128]).all()
    assert int(torch.isnan(a).sum()) == 256 and int(torch.isnan(c).sum()) == 256
    empty, none = bl.act_save_both(torch.zeros(0, 64, device="cuda"))
    assert empty.shape == (0, 64) and none.shape == (0, 64) and none.scales.shape == (0, 64)


def test_saved_codes_leave_their_neighbours(bl):
    """Code tensors that are views: the bytes behind their columns stay."""
    from block_sparse_attention_fwd_gb300 import linear
    x = _randn(140, 100, dtype=torch.bfloat16, seed=4)
    wide = torch.full((140, 128), 77, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, 100, device="cuda")
    linear._launch("bl_tile8_save", x.device, linear._TILE8_ARGS.pack(
        140, 100, 100, 0, 128, 0, x.data_ptr(), 0, 0, wide.data_ptr() + 9, scales.data_ptr(), 0, 0, 0))
    _, c = bl.act_save_both(x)
    assert torch.equal(wide[:, 9:109], c.codes.view(torch.uint8))
    assert (wide[:, :9] == 77).all() and (wide[:, 109:] == 77).all()


# --- products --------------------------------------------------------------------

def _codes(rows, cols, seed, pitch=None):
    """e4m3 codes of all finite kinds, subnormal ones among them."""
    g = torch.Generator("cuda").manual_seed(seed)
    c = torch.randn(rows, pitch or cols, generator=g, device="cuda") * 40
    c[::3] *= 0.01
    return c.to(torch.float8_e4m3fn)[:, :cols]


def _scales(*shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.exp2(4 * torch.rand(shape, generator=g, device="cuda") - 10)


def _product(bl, form, M, N, K, dtype, seed=0, pitched=True):
    """(operands, fp64 values of both factors laid out [i, k] and [j, k])."""
    cd = lambda n: -(-n // 128)      # noqa: E731
    p = (lambda n: -(-n // 16) * 16) if pitched else (lambda n: n)
    t = TYPES[dtype]
    if form == "g_w":
        a = bl.Cols8(_codes(M, N, seed, p(N)), _scales(cd(M), N, seed=seed + 1), t)
        b = bl.Cols8(_codes(M, K, seed + 2, p(K)), _scales(cd(M), K, seed=seed + 3), t)
        values = [(_np64(x.codes.double()) * np.repeat(_f64(x.scales), 128, 0)[:M]).T for x in (a, b)]
        return a, b, values
    inner = K if form == "y" else N
    a = bl.Act8(_codes(M, inner, seed).contiguous(), _scales(M, cd(inner), seed=seed + 1), 128, t)
    b = bl.Weight8(_codes(N, K, seed + 2, p(K)), _scales(cd(N), cd(K), seed=seed + 3), t)
    av = _np64(a.codes.double()) * np.repeat(_f64(a.scales), 128, 1)[:, :inner]
    bv = _np64(b.codes.double()) * OL.spread(_f64(b.scales), 128, 128, N, K)
    return a, b, [av, bv if form == "y" else bv.T]


def _run(bl, form, a, b, t=None):
    return {"y": bl.matmul8, "g_x": bl.matmul8_gx, "g_w": bl.matmul8_gw}[form](a, b, t)


def _check_product(got, values, dtype):
    a, b = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in values)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    blocks = -(-a.shape[1] // 128)
    _close(got, ref.cpu().numpy(), (2 * 128 + blocks + 4) * F * mag.cpu().numpy(), TYPES[dtype])


PRODUCTS = [
    (1, 1, 1), (1, 16, 16), (2, 7, 5), (8, 128, 256), (16, 300, 130), (17, 128, 2048), (33, 5000, 520),
    (51, 700, 3100), (64, 257, 1000), (65, 130, 1030), (100, 1500, 4000), (128, 128, 128), (200, 384, 640),
    (257, 2050, 129), (1000, 512, 512), (3000, 512, 512), (3000, 1000, 130), (2500, 2500, 300),
    (5000, 4100, 256), (7, 130, 9000),
]


@pytest.mark.parametrize("form", ["y", "g_x", "g_w"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products(bl, M, N, K, form):
    for dtype in ("fp32", "bf16"):
        a, b, values = _product(bl, form, M, N, K, dtype, seed=M + N + K)
        got = _run(bl, form, a, b)
        assert got.dtype == TYPES[dtype] and got.is_contiguous()
        _check_product(got, values, dtype)


@pytest.mark.parametrize("form", ["y", "g_x", "g_w"])
@pytest.mark.parametrize("M,N,K", [(40, 1001, 333), (300, 77, 1030)])
def test_products_of_rows_that_start_anywhere(bl, M, N, K, form):
    """Codes whose rows are not 16-byte aligned go through the workspace."""
    a, b, values = _product(bl, form, M, N, K, "fp16", seed=5, pitched=False)
    _check_product(_run(bl, form, a, b), values, "fp16")
    _check_product(_run(bl, form, a, b, torch.float32), values, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(130, 4100, 4112), (100, 1000, 1008), (3, 200, 272), (260, 4200, 4104)])
def test_weight_gradients_of_few_tokens(bl, M, N, K, dtype):
    """More tiles than SMs, a block or two of tokens each; rows of whole 32 bytes that end inside a
    tile, and (4104 elements of 16 bits) rows that are not; what lies behind the result stays."""
    a, b, values = _product(bl, "g_w", M, N, K, dtype, seed=11)
    _check_product(_run(bl, "g_w", a, b), values, dtype)
    from block_sparse_attention_fwd_gb300 import linear
    t = TYPES[dtype]
    flat = torch.full((N * K + 512,), 9.0, dtype=t, device="cuda")
    linear._launch("bl_matmul8", flat.device, linear._MATMUL8_ARGS.pack(
        M, N, K, a.codes.data_ptr(), a.scales.data_ptr(), a.stride, b.codes.data_ptr(), b.scales.data_ptr(),
        b.stride, flat.data_ptr(), 0, 0, 2, ["bf16", "fp16", "fp32"].index(dtype)))
    assert torch.equal(flat[:N * K].view(N, K), _run(bl, "g_w", a, b)) and (flat[N * K:] == 9).all()


def test_products_keep_the_batch_dims_and_repeat(bl):
    a, b, values = _product(bl, "y", 60, 200, 256, "bf16")
    x8 = bl.Act8(a.codes.view(3, 4, 5, 256), a.scales.view(3, 4, 5, 2), 128, torch.bfloat16)
    y = bl.matmul8(x8, b)
    assert y.shape == (3, 4, 5, 200) and torch.equal(y.view(60, 200), bl.matmul8(a, b))
    for form, M, N, K in (("y", 100, 1500, 4000), ("g_w", 3000, 512, 512), ("g_x", 8, 4000, 300)):
        a, b, _ = _product(bl, form, M, N, K, "fp32", seed=9)
        first = _run(bl, form, a, b)
        for _ in range(5):
            assert torch.equal(_run(bl, form, a, b), first)


def test_products_of_no_tokens(bl):
    w = bl.weight_save(_randn(40, 70))
    for cols, fn, out in ((70, bl.matmul8, 40), (40, bl.matmul8_gx, 70)):
        a, _ = bl.act_save_both(torch.zeros(2, 0, cols, device="cuda"))
        assert fn(a, w).shape == (2, 0, out)
    _, g = bl.act_save_both(torch.zeros(0, 40, device="cuda"))
    _, x = bl.act_save_both(torch.zeros(0, 70, device="cuda"))
    assert torch.equal(bl.matmul8_gw(g, x), torch.zeros(40, 70, device="cuda"))


def test_products_with_scales_that_are_nan(bl):
    """A block that loads as NaN reaches its row (or its 128 columns), and nothing else."""
    x, w = _randn(70, 300, seed=1), _randn(200, 300, seed=2)
    x[3, 200] = float("inf")
    w[150, 10] = float("nan")
    (x8, xc), w8 = bl.act_save_both(x), bl.weight_save(w)
    y = bl.matmul8(x8, w8)
    want = torch.zeros(70, 200, dtype=torch.bool, device="cuda")
    want[3], want[:, 128:] = True, True
    assert torch.equal(torch.isnan(y), want)
    g8, gc = bl.act_save_both(_randn(70, 200, seed=3))
    assert torch.equal(torch.isnan(bl.matmul8_gx(g8, w8)).all(0).cpu(), torch.arange(300) < 128)
    bad = torch.isnan(bl.matmul8_gw(gc, xc))
    assert bad[:, 200].all() and int(bad.sum()) == 200


def test_products_of_any_size_of_scales(bl):
    """Results from 1e-30 to 1e30; the product of two scales stays a normal number."""
    a, b, _ = _product(bl, "y", 20, 256, 512, "fp32", seed=3)
    for e in (-90, -40, 0, 40, 80):
        s = bl.Act8(a.codes, torch.ldexp(a.scales, torch.tensor(e, device="cuda")), 128, torch.float32)
        assert torch.equal(bl.matmul8(s, b), torch.ldexp(bl.matmul8(a, b), torch.tensor(e, device="cuda")))


def test_product_refusals(bl):
    x8, xc = bl.act_save_both(_randn(4, 256))
    w8 = bl.weight_save(_randn(100, 256))
    for x in (bl.act_save(_randn(4, 256), "int8", 128), bl.act_save(_randn(4, 256), "e4m3", 64),
              bl.act_save(_randn(4, 256), "e4m3"), bl.act_save(_randn(4, 128), "e4m3", 128)):
        with pytest.raises(ValueError):
            bl.matmul8(x, w8)
    with pytest.raises(ValueError):
        bl.matmul8_gx(x8, w8)
    with pytest.raises(ValueError):
        bl.matmul8_gw(xc, bl.act_save_both(_randn(5, 256))[1])
    for call in (lambda: bl.matmul8(xc, w8), lambda: bl.matmul8(x8, x8), lambda: bl.matmul8_gw(x8, xc),
                 lambda: bl.matmul8(x8, w8, torch.float64), lambda: bl.matmul8_gx(x8, xc)):
        with pytest.raises(TypeError):
            call()
    codes = torch.zeros(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")      # noqa: E731
    for call in (lambda: bl.Weight8(codes, f(1, 3), torch.float32), lambda: bl.Cols8(codes, f(1, 2), torch.float32),
                 lambda: bl.Weight8(codes.view(1, 4, 256), f(1, 2), torch.float32),
                 lambda: bl.Weight8(codes.t(), f(2, 1), torch.float32),
                 lambda: bl.Weight8(codes[:1].expand(4, 256), f(1, 2), torch.float32),
                 lambda: bl.weight_save(_randn(2, 3, 4)), lambda: bl.act_save_both(_randn(4, 4), False, False)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bl.Weight8(codes.view(torch.int8), f(1, 2), torch.float32),
                 lambda: bl.Weight8(codes, f(1, 2).half(), torch.float32),
                 lambda: bl.Weight8(codes, f(1, 2), torch.float64)):
        with pytest.raises(TypeError):
            call()


def test_product_whose_waits_run_out(bl):
    """With a wait limit of zero a call may leave tiles, which are NaN, and the next call under
    the ordinary limit is right."""
    from block_sparse_attention_fwd_gb300 import _lib
    cases = [_product(bl, f, *s, "fp32", seed=7) for f, s in
             (("y", (3000, 2560, 1024)), ("y", (100, 1500, 4000)), ("g_x", (8, 4000, 300)),
              ("g_w", (3000, 512, 512)))]
    right = [_run(bl, f, a, b) for f, (a, b, _) in zip(("y", "y", "g_x", "g_w"), cases)]
    was = _lib.set_wait_limit(0.0)
    try:
        left = [_run(bl, f, a, b) for f, (a, b, _) in zip(("y", "y", "g_x", "g_w"), cases)]
        torch.cuda.synchronize()
    finally:
        _lib.set_wait_limit(was)
    for got, want, f, (a, b, _) in zip(left, right, ("y", "y", "g_x", "g_w"), cases):
        assert (torch.isnan(got) | (got == want)).all()
        assert torch.equal(_run(bl, f, a, b), want)


# --- layer norm --------------------------------------------------------------------

NORMS = [(1, 1), (3, 7), (5, 64), (2, 100), (33, 128), (7, 256), (9, 520), (5, 1001), (4, 1024), (6, 2048),
         (5, 2561), (3, 4096), (1001, 4096), (4, 5120), (3, 5128), (2, 8192), (3, 12288), (2, 16384), (2, 16383)]


def _norm_inputs(rows, cols, t, wt, shift=0.5, seed=0):
    size = torch.exp(0.7 * _randn(cols, seed=seed + 1))
    x = ((shift + _randn(rows, cols, seed=seed + 2)) * size).to(t)
    r = (2 * _randn(rows, cols, seed=seed + 3) * size).to(t)
    w = (1 + 0.3 * _randn(cols, seed=seed + 4)).to(wt)
    b = (0.3 * _randn(cols, seed=seed + 5)).to(wt)
    return x, r, w, b


def _norm_slack(h, mean, rstd, w, b, eps):
    """(slack of y, of mean, of rstd): see the head of this file."""
    size = np.abs(h).mean(1)
    sigma = np.sqrt(np.maximum(((h - mean[:, None]) ** 2).mean(1) + eps, 1e-300))
    ratio = np.sqrt((h * h).mean(1)) / sigma
    off = 64 * F * size[:, None] + 2 * F * np.abs(h) + 2 * F * np.abs(mean)[:, None]
    rel = 256 * F * (1 + ratio)
    u = np.abs(h - mean[:, None]) * rstd[:, None]
    w = 1.0 if w is None else np.abs(_np64(w))
    b = 0.0 if b is None else np.abs(_np64(b))
    return w * (off * rstd[:, None] + u * (rel[:, None] + 4 * F)) + F * b, 64 * F * size, rel * rstd


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", NORMS)
def test_layer_norm_forward(bl, rows, cols, dtype):
    t = TYPES[dtype]
    for wt in {t, torch.float32}:
        x, r, w, b = _norm_inputs(rows, cols, t, wt, seed=cols)
        for residual, weight, bias in ((None, w, b), (r, w, b), (r, None, None), (None, w, None), (None, None, b)):
            y, h, mean, rstd = bl.layer_norm_fwd(x, weight, bias, 1e-5, residual)
            ry, rh, rm, rs = OL.layer_norm(x, weight, bias, 1e-5, residual)
            sy, sm, ss = _norm_slack(rh, rm, rs, weight, bias, 1e-5)
            _close(y, ry, sy, t)
            _close(mean, rm, sm, torch.float32)
            _close(rstd, rs, ss, torch.float32)
            if residual is None:
                assert h is x
            else:
                _close(h, rh, F * np.abs(rh), t)


@pytest.mark.parametrize("fmt,group", [("e4m3", 128), ("int8", 32), ("e4m3", 0), ("int8", 64)])
@pytest.mark.parametrize("rows,cols", [(5, 40), (33, 128), (5, 1001), (6, 2048), (7, 4096), (5, 5120), (3, 12288)])
def test_layer_norm_forward_in_8_bits(bl, rows, cols, fmt, group):
    """The codes are those of y before its rounding: off by half a step of the code from the
    oracle's y, whose scale is within F of the group's largest; y beside them as without."""
    for t, residual in ((torch.bfloat16, True), (torch.float32, False)):
        x, r, w, b = _norm_inputs(rows, cols, t, torch.float32, seed=cols + 1)
        r = r if residual else None
        y, h, mean, rstd = bl.layer_norm_fwd(x, w, b, residual=r)
        y2, y8, h2, mean2, rstd2 = bl.layer_norm_fwd_8bit(x, w, b, residual=r, fmt=fmt, group=group, with_y=True)
        alone = bl.layer_norm_fwd_8bit(x, w, b, residual=r, fmt=fmt, group=group)[0]
        assert torch.equal(alone.codes.view(torch.uint8), y8.codes.view(torch.uint8))
        assert torch.equal(alone.scales, y8.scales) and torch.equal(h, h2)
        for p, q in ((mean, mean2), (rstd, rstd2)):
            assert torch.allclose(p, q, rtol=512 * F, atol=1e-30)   # two ways to add
        _, rh, rm, rs = OL.layer_norm(x, w, b, 1e-5, r)
        ry = OL.layer_norm(x, w, b, 1e-5, r)[0]
        slack = _norm_slack(rh, rm, rs, w, b, 1e-5)[0]
        _close(y2, ry, slack, t)
        size = group or cols
        scales = _f64(y8.scales).reshape(rows, -1)
        each = np.repeat(scales, size, 1)[:, :cols]
        codes = _f64(y8.codes.float())
        step = np.ones_like(codes) if fmt == "int8" else np.maximum(2.0 ** (np.frexp(np.abs(codes))[1] - 4), 2.0 ** -9)
        assert (np.abs(codes * each - ry) <= each * step / 2 * (1 + 1e-3) + slack + 8 * F * np.abs(ry)).all()
        top = np.abs(np.pad(ry, ((0, 0), (0, scales.shape[1] * size - cols)))).reshape(rows, -1, size).max(2)
        most = np.pad(slack, ((0, 0), (0, scales.shape[1] * size - cols))).reshape(rows, -1, size).max(2)
        qmax = 127.0 if fmt == "int8" else 448.0
        assert (np.abs(scales * qmax - top) <= most + 8 * F * top).all()


@pytest.mark.parametrize("saved", [None, "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (33, 128), (700, 136), (9, 520), (5, 1001), (300, 1024),
                                       (5, 2561), (1200, 4096), (4, 5120), (3, 8200), (2, 16384)])
def test_layer_norm_backward(bl, rows, cols, dtype, saved):
    t = TYPES[dtype]
    x, _, w, _ = _norm_inputs(rows, cols, t, torch.float32 if dtype == "bf16" else t, seed=cols + 2)
    _, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
    h = x if saved is None else bl.act_save(x, saved, 128)
    hv = _f64(x) if saved is None else _f64(bl.act_load(bl.Act8(h.codes, h.scales, 128, torch.float32)))
    g, gh = _randn(rows, cols, dtype=t, seed=8), _randn(rows, cols, dtype=t, seed=9)
    for g_h, weight in ((gh, w), (None, w), (None, None)):
        gx, gw, gb = bl.layer_norm_bwd(g, h, mean, rstd, weight, g_h=g_h)
        rx, rw, rb = OL.layer_norm_backward(g, hv, mean, rstd, weight, g_h)
        m, s = np.abs(_f64(mean))[:, None], _f64(rstd)[:, None]
        u = (hv - _f64(mean)[:, None]) * s
        du = 4 * F * (np.abs(hv) + m) * s
        wg = np.abs(_f64(g)) * (1.0 if weight is None else np.abs(_f64(weight)))
        c = (wg * np.abs(u)).mean(1, keepdims=True)
        all_terms = s * (wg + wg.mean(1, keepdims=True) + np.abs(u) * c)
        slack = 64 * F * all_terms + s * (du * c + np.abs(u) * (wg * du).mean(1, keepdims=True))
        if g_h is not None:
            slack = slack + F * np.abs(_f64(g_h))
        _close(gx, rx, slack, t)
        terms = np.abs(_f64(g))
        wt = torch.float32 if weight is None else weight.dtype
        assert gw.dtype == wt and gb.dtype == wt
        _close(gw, rw, (rows + 64) * F * (terms * np.abs(u)).sum(0) + (terms * du).sum(0), wt)
        _close(gb, rb, (rows + 64) * F * terms.sum(0), wt)
    same = bl.layer_norm_bwd(g, h, mean, rstd, w, need_g_w=False, need_g_b=False)
    assert same[1] is None and same[2] is None
    again = bl.layer_norm_bwd(g, h, mean, rstd, w)
    assert torch.equal(again[0], same[0])
    one = bl.layer_norm_bwd(g, h, mean, rstd, w, need_g_w=False)
    assert one[1] is None and torch.equal(one[2], again[2])


def test_layer_norm_of_rows_far_from_zero(bl):
    """Rows whose mean is 1000 times their spread, rows that are one number, rows of one
    element, an outlier where the sums begin."""
    for cols in (128, 1024, 4096, 5120, 1001):
        x = 1000 + _randn(9, cols, seed=cols)
        y, _, mean, rstd = bl.layer_norm_fwd(x, None, None, 0.0)
        ry, rh, rm, rs = OL.layer_norm(x, None, None, 0.0)
        sy, sm, ss = _norm_slack(rh, rm, rs, None, None, 0.0)
        _close(y, ry, sy, torch.float32)
        _close(rstd, rs, ss, torch.float32)
        x = torch.full((3, cols), 0.1, device="cuda")
        y, _, mean, rstd = bl.layer_norm_fwd(x, None, None, 1e-5)
        assert (y.abs() <= 0.1 * 128 * F * 1e-5 ** -0.5).all() and torch.allclose(mean, x[:, 0], rtol=64 * F)
        x = _randn(4, cols, seed=1)
        x[:, 0] = 3e4
        y, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
        _close(rstd, OL.layer_norm(x, None, None, 1e-5)[3], 2 * 256 * F * _f64(rstd), torch.float32)
    y, _, mean, rstd = bl.layer_norm_fwd(torch.full((5, 1), 7.0, device="cuda"), None, None, 1e-4)
    assert (y == 0).all() and (mean == 7).all() and torch.allclose(rstd, torch.full_like(rstd, 100.0))


def test_layer_norm_rows_that_are_not_finite(bl):
    x = _randn(6, 1024, dtype=torch.bfloat16)
    x[1, 3], x[4, 1000] = float("nan"), float("inf")
    y, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
    bad = torch.zeros(6, dtype=torch.bool, device="cuda")
    bad[1] = bad[4] = True
    assert torch.equal(torch.isnan(y).all(1), bad) and torch.equal(torch.isnan(y).any(1), bad)
    assert torch.equal(torch.isnan(rstd), bad) and torch.isfinite(mean[~bad]).all()
    clean = x.clone()
    clean[1] = clean[4] = 0
    assert torch.equal(y[~bad], bl.layer_norm_fwd(clean, None, None)[0][~bad])
    y8 = bl.layer_norm_fwd_8bit(x, None, None)[0]
    assert torch.equal(torch.isnan(bl.act_load(y8)).all(1), bad)


def test_layer_norm_takes_views(bl):
    for cols in (128, 1024, 1001, 4096):
        big = _randn(2, 9, 3 * cols + 8, dtype=torch.bfloat16, seed=cols)
        with pytest.raises(ValueError):                # rows that are not equally spaced
            bl.layer_norm_fwd(big[:, ::2, cols:2 * cols], None, None)
        for x in (big[..., 8:8 + cols], big[:, 1:9:3, cols:2 * cols], big[0, :, 3:3 + cols]):
            r = _randn(*x.shape, dtype=torch.bfloat16, seed=1)
            got, want = (bl.layer_norm_fwd(v, None, None, residual=s) for v, s in ((x, r), (x.contiguous(), r)))
            for p, q in zip(got, want):
                # rows that start anywhere are summed in another order
                assert torch.allclose(p.float(), q.float(), rtol=2.0 ** -7, atol=1e-4) and p.is_contiguous()


@pytest.mark.parametrize("cols", [1001, 24, 1000])
@pytest.mark.parametrize("off", [1, 2, 5])
def test_layer_norm_outputs_keep_their_neighbours(bl, cols, off):
    from block_sparse_attention_fwd_gb300 import linear
    rows, t = 5, torch.bfloat16
    x = _randn(rows, cols, dtype=t, seed=2)
    flat = torch.full((rows * cols + 64,), 9.0, dtype=t, device="cuda")
    stats = torch.full((2, rows + 2), 9.0, device="cuda")
    y = flat[off:off + rows * cols]
    linear._launch("bl_layer_norm_fwd", x.device, linear._LAYER_NORM_ARGS.pack(
        rows, cols, cols, cols, x.data_ptr(), 0, 0, 0, y.data_ptr(), 0, stats[0, 1:].data_ptr(),
        stats[1, 1:].data_ptr(), 0, 1e-5, 0, 0))
    ry, rh, rm, rs = OL.layer_norm(x, None, None, 1e-5)
    _close(y.view(rows, cols), ry, _norm_slack(rh, rm, rs, None, None, 1e-5)[0], t)
    assert (flat[:off] == 9).all() and (flat[off + rows * cols:] == 9).all()
    assert (stats[:, 0] == 9).all() and (stats[:, -1] == 9).all()


def test_layer_norm_empty_and_refusals(bl):
    x = _randn(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    y, h, mean, rstd = bl.layer_norm_fwd(x[:0], w, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    gx, gw, gb = bl.layer_norm_bwd(x[:0], x[:0], mean, rstd, w)
    assert gx.shape == (0, 64) and (gw == 0).all() and (gb == 0).all()
    _, _, mean, rstd = bl.layer_norm_fwd(x, w, w)
    for call in (lambda: bl.layer_norm_fwd(x, w[:5], w), lambda: bl.layer_norm_fwd(x, w, w[:5]),
                 lambda: bl.layer_norm_fwd(x, w, w, residual=x[:2]), lambda: bl.layer_norm_fwd(x.t(), None, None),
                 lambda: bl.layer_norm_bwd(x, x, mean[:2], rstd, w), lambda: bl.layer_norm_bwd(x, x[:2], mean, rstd, w),
                 lambda: bl.layer_norm_bwd(x.t(), x, mean, rstd, w),
                 lambda: bl.layer_norm_fwd_8bit(x, w, w, fmt="fp8"), lambda: bl.layer_norm_fwd_8bit(x, w, w, group=7),
                 lambda: bl.layer_norm_fwd(_randn(1, 16385), None, None)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bl.layer_norm_fwd(x, w.half(), None), lambda: bl.layer_norm_fwd(x, None, w.half()),
                 lambda: bl.layer_norm_fwd(x, w, w.bfloat16()), lambda: bl.layer_norm_fwd(x.double(), None, None),
                 lambda: bl.layer_norm_bwd(x, x.half(), mean, rstd, w),
                 lambda: bl.layer_norm_bwd(x, bl.act_save(x.half()), mean, rstd, w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(bl.BLError):
        bl.layer_norm_fwd(x, w, w, -1.0)


# --- dropout -----------------------------------------------------------------------

def _state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (3, 5), (13, 101), (2, 3, 128), (700,)])
def test_dropout(bl, shape, dtype):
    t = TYPES[dtype]
    x, r = _randn(*shape, dtype=t, seed=1), _randn(*shape, dtype=t, seed=2)
    n = x.numel()
    for p, seed, offset in ((0.1, 5, 0), (0.5, -3, 2 ** 40 + 1), (0.25, 2 ** 62 + 11, -1)):
        keep = OL.kept(n, p, seed, offset).reshape(shape)
        scale = 1 / (1 - p)
        for residual in (None, r):
            y = bl.dropout(x, p, _state(seed, offset), residual)
            ref = np.where(keep, _f64(x) * scale, 0.0)
            slack = 2 * F * np.abs(ref)
            if residual is not None:
                ref = ref + _f64(r)
                slack = slack + F * np.abs(ref)
            _close(y, ref, slack, t)
            if residual is None:
                assert (_f64(y)[~keep] == 0).all()


def test_dropout_at_the_ends_and_of_what_is_not_finite(bl):
    x, r, st = _randn(5, 33, seed=1), _randn(5, 33, seed=2), _state(1, 2)
    assert torch.equal(bl.dropout(x, 0.0, st), x) and torch.equal(bl.dropout(x, 0.0, st, r), x + r)
    assert (bl.dropout(x, 1.0, st) == 0).all() and torch.equal(bl.dropout(x, 1.0, st, r), r)
    # round(p 2^32) = 2^32, which no word reaches
    big = torch.ones(2 ** 24, device="cuda")
    assert (bl.dropout(big, 1 - 2.0 ** -34, st) == 0).all()
    keep = torch.from_numpy(OL.kept(165, 0.5, 1, 2)).view(5, 33).cuda()
    for v in (float("inf"), float("-inf"), float("nan")):
        y = bl.dropout(torch.full_like(x, v), 0.5, st)
        assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()
        assert torch.equal(bl.dropout(torch.full_like(x, v), 0.5, st, r)[~keep], r[~keep])
        assert (bl.dropout(torch.full_like(x, v), 1.0, st) == 0).all()


def test_dropout_masks_do_not_depend_on_layout(bl):
    """Views, rows that start anywhere, in place."""
    big, st = _randn(40, 400, dtype=torch.bfloat16, seed=3), _state(7, 8)
    for v in (big[:, 8:264], big[:, 3:104], big[::3], big[1:, :5]):
        assert torch.equal(bl.dropout(v, 0.3, st), bl.dropout(v.contiguous(), 0.3, st))
        assert torch.equal(bl.dropout(v, 0.3, st, v), bl.dropout(v.contiguous(), 0.3, st, v.contiguous()))
    flat = _randn(1003, dtype=torch.bfloat16, seed=4)
    assert torch.equal(bl.dropout(flat[3:], 0.3, st), bl.dropout(flat[3:].clone(), 0.3, st))
    from block_sparse_attention_fwd_gb300 import linear
    want = bl.dropout(flat, 0.3, st, flat)
    buf = flat.clone()
    linear._launch("bl_dropout", buf.device, 1, 1003, 0, buf.data_ptr(), 1003, buf.data_ptr(), 1003, 0.3,
                   st.data_ptr(), buf.data_ptr())
    assert torch.equal(buf, want)


def test_dropout_past_32_bits(bl):
    """2^32 + 40 elements: the counter's index passes 2^30; and by the oracle around 2^34 (its
    upper word) through the rows' own places."""
    n = 2 ** 32 + 40
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = bl.dropout(x, 0.5, _state(3, 4))
    for at in (0, 2 ** 31 - 16, 2 ** 32 - 20, n - 48):
        keep = OL.kept(40, 0.5, 3, 4, first=at)
        assert (_f64(y[at:at + 40]) == np.where(keep, 2.0, 0.0)).all()
    assert abs(float((y[:2 ** 26] != 0).float().mean()) - 0.5) < 5 * 0.5 / 2 ** 13


def test_dropout_next(bl):
    st = _state(9, 2 ** 63 - 1)
    used = [bl.dropout_next(st) for _ in range(3)]
    assert [u.tolist() for u in used] == [[9, 2 ** 63 - 1], [9, -2 ** 63], [9, 1 - 2 ** 63]]
    assert st.tolist() == [9, 2 - 2 ** 63]


def test_dropout_refusals_and_empty(bl):
    x, st = _randn(4, 8), _state(0, 0)
    assert bl.dropout(x[:0], 0.5, st).shape == (0, 8)
    for call in (lambda: bl.dropout(x, -0.1, st), lambda: bl.dropout(x, 1.1, st), lambda: bl.dropout(x, 0.1, st[:1]),
                 lambda: bl.dropout(x, float("nan"), st), lambda: bl.dropout(x, 0.1, st, x[:2]),
                 lambda: bl.dropout(x, 0.1, st, x.half()), lambda: bl.dropout(x.t(), 0.1, st)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bl.dropout(x.double(), 0.1, st), lambda: bl.dropout(x, 0.1, st.int()),
                 lambda: bl.dropout(x, 0.1, st.cpu()), lambda: bl.dropout_next(st.cpu())):
        with pytest.raises(TypeError):
            call()


# --- long ones -----------------------------------------------------------------------

def test_offsets_past_32_bits(bl):
    """Tensors of more than 2^32 elements: their last rows as those of small ones."""
    rows, cols = 2 ** 19 + 3, 8192
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = _randn(130, cols, dtype=torch.bfloat16, seed=5)
    x[-130:] = tail
    y, _, mean, rstd = bl.layer_norm_fwd(x, None, None)
    ty, _, tm, ts = bl.layer_norm_fwd(tail, None, None)
    assert torch.equal(y[-130:], ty) and torch.equal(mean[-130:], tm) and torch.equal(rstd[-130:], ts)
    gx, _, _ = bl.layer_norm_bwd(x, x, mean, rstd, None)
    tx, _, _ = bl.layer_norm_bwd(tail, tail, tm, ts, None)
    assert torch.equal(gx[-130:], tx)
    del y, gx
    a, c = bl.act_save_both(x)
    at = 2 ** 19 - 128                       # the last groups of 128 rows begin there
    ta, tc = bl.act_save_both(x[at:].contiguous())
    assert torch.equal(a.codes[at:].view(torch.uint8), ta.codes.view(torch.uint8))
    assert torch.equal(c.codes[at:].view(torch.uint8), tc.codes.view(torch.uint8))
    assert torch.equal(c.scales[at // 128:], tc.scales)
    w8 = bl.weight_save(_randn(40, cols, dtype=torch.bfloat16, seed=6))
    got, want = bl.matmul8(a, w8), bl.matmul8(ta, w8)
    assert torch.allclose(got[at:].float(), want.float(), rtol=2.0 ** -7, atol=1e-3)
