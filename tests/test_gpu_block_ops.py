"""Rotary positions, the residual norm and 8-bit activations on the GPU against
the fp64 oracle, element by element.

Tolerances count roundings.  half(t) = finfo(t).eps / 2 is one rounding to the
type t, relative; F = 2^-24 is one in fp32.
 * rope: two products and a sum (4 F of |u| + |v|, fused or not), the angle's 32
   bits rounded to 24 (pi F / 2), sincospi's two ulps (2 F each): 16 F (|u| + |v|).
 * norm: a sum of squares over a thread's up to 32 elements and 15 levels of
   adding partial sums, each F of a sum of positive terms (47 F of the sum, half of
   it in rstd), the mean, root and quotient (4 F), two products (2 F), the residual's
   addition (2 F): 64 F.
 * norm backward: each term of g_x carries the errors of u (2 F), of the products
   (4 F) and of the dot product, (47 + 4) F of the sum of its terms' magnitudes: 64 F
   of all terms' magnitudes.  g_w: as many roundings as a thread has rows, plus
   32 + log2 of the partial sums: (rows + 64) F of the sum of magnitudes.
An fp16 result below the smallest normal is off by half a subnormal step more.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import block as OB
from tests import parity_util as U

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


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _tiny(dtype):
    info = torch.finfo(dtype)
    return info.smallest_normal * info.eps / 2


def _close(got, ref, slack, dtype):
    """|got - ref| <= half a step of the type, plus `slack` from the fp32 arithmetic."""
    got = _f64(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    bound = _half(dtype) * (np.abs(ref) + slack) + slack + _tiny(dtype)
    over = np.abs(got - ref) > bound
    assert not over.any(), (int(over.sum()), np.argwhere(over)[:3].tolist(),
                            float((np.abs(got - ref) - bound).max()))


def _randn(*shape, dtype, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


# --- rotary ---------------------------------------------------------------------

ROPE = [
    # B, n, H, Hk, d, sections, layout
    (1, 1, 1, 1, 64, (32,), "half"),
    (3, 1, 32, 8, 128, (64,), "half"),
    (2, 7, 5, 1, 128, (22, 21, 21), "interleaved"),
    (1, 33, 3, 2, 128, (16, 24, 24), "half"),
    (2, 19, 4, 4, 80, (5, 6, 7, 8), "interleaved"),     # part of a vector turns
    (1, 300, 40, 40, 128, (22, 21, 21), "interleaved"),  # several heads a thread
    (1, 700, 9, 3, 64, (8,), "half"),                    # a part of the head passes through
    (2, 11, 3, 1, 36, (3, 5), "half"),                   # element by element
    (1, 9, 2, 2, 7, (3,), "interleaved"),                # odd head
    (1, 5, 6, 0, 64, (32,), "half"),                     # q alone
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}+{c[3]}x{c[4]}")
def test_rope_and_its_inverse(bl, case, dtype):
    B, n, H, Hk, d, sections, layout = case
    t = TYPES[dtype]
    q = _randn(B, n, H, d, dtype=t, seed=1)
    k = _randn(B, n, Hk, d, dtype=t, seed=2) if Hk else None
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-1000, 1000000, (B, n, len(sections)), generator=g, dtype=torch.int32)
    plan = bl.RopePlan(d, sections, layout=layout)
    for inverse in (False, True):
        got = bl.rope(q, k, pos.cuda(), plan, inverse=inverse)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            ref = OB.rope(x, pos.numpy(), sections, plan.freqs, layout == "interleaved", inverse)
            mag = np.abs(OB._f64(x))
            P = plan.pairs
            pair = mag.copy()
            i, j = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if layout == "interleaved" else \
                (slice(0, P), slice(P, 2 * P))
            pair[..., i] = pair[..., j] = mag[..., i] + mag[..., j]
            _close(y, ref, 16 * F * pair, t)
            assert torch.equal(y[..., 2 * P:], x[..., 2 * P:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", [
    (2, 37, 4, 2, 80, (20,), "half"),                    # halves of 20 pairs: off 16-bit vectors, on fp32's
    (1, 37, 4, 2, 80, (40,), "half"),
    (1, 37, 4, 2, 80, (20,), "interleaved"),
    (3, 5, 6, 1, 96, (9, 10, 11), "half")], ids=lambda c: f"d{c[4]}p{sum(c[5])}{c[6]}")
def test_rope_of_a_part_of_other_heads(bl, case, dtype):
    test_rope_and_its_inverse(bl, case, dtype)


def test_rope_takes_views_and_works_in_place(bl):
    """Heads of a fused projection, rows that start anywhere, shared positions."""
    fused = _randn(2, 50, 3 * 4, 64, dtype=torch.bfloat16, seed=4)
    q, k = fused[:, :, :4], fused[:, :, 4:8]
    plan = bl.RopePlan(64, (20, 12), layout="interleaved")
    pos = torch.randint(0, 500, (50, 2), dtype=torch.int32, device="cuda")
    want = bl.rope(q.contiguous(), k.contiguous(), pos.expand(2, 50, 2).contiguous(), plan)
    got = bl.rope(q, k, pos, plan)
    assert all(torch.equal(a, b) and a.is_contiguous() for a, b in zip(got, want))
    rest = fused[:, :, 8:].clone()
    out = bl.rope(q, k, pos, plan, inplace=True)
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(fused[:, :, 8:], rest)
    # a view whose vectors are not aligned takes the element path: the same values
    odd = torch.empty(2 * 50 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 50, 4, 64)
    odd.copy_(want[0])
    assert torch.equal(bl.rope(odd, None, pos, plan, inverse=True)[0],
                       bl.rope(want[0], None, pos, plan, inverse=True)[0])
    # batches that do not follow one another, and heads before tokens
    long = _randn(2, 90, 4, 64, dtype=torch.bfloat16, seed=40)
    part = long[:, 20:70]
    ref = bl.rope(part.contiguous(), None, pos, plan)[0]
    assert torch.equal(bl.rope(part, None, pos, plan)[0], ref)
    before = long.clone()
    bl.rope(part, None, pos, plan, inplace=True)
    assert torch.equal(part, ref) and torch.equal(long[:, :20], before[:, :20])
    assert torch.equal(long[:, 70:], before[:, 70:])
    bhsd = _randn(2, 4, 50, 64, dtype=torch.bfloat16, seed=41)
    ref = bl.rope(bhsd.transpose(1, 2).contiguous(), None, pos, plan)[0]
    assert torch.equal(bl.rope(bhsd.transpose(1, 2), None, pos, plan)[0], ref)
    # packed tensors
    flat = bl.rope(want[0].flatten(0, 1), want[1].flatten(0, 1), pos.repeat(2, 1), plan)
    again = bl.rope(want[0], want[1], pos, plan)
    assert torch.equal(flat[0], again[0].flatten(0, 1)) and torch.equal(flat[1], again[1].flatten(0, 1))


def test_rope_passes_non_finite_values_of_other_dims_by(bl):
    """A NaN or an infinity stays within its pair; the dimensions behind pass through."""
    x = _randn(1, 3, 2, 64, dtype=torch.bfloat16, seed=5)
    x[0, 1, 0, 7] = float("inf")
    x[0, 1, 0, 60] = float("nan")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")[:, None]
    plan = bl.RopePlan(64, (25,), layout="interleaved")
    y = bl.rope(x, None, pos, plan)[0]
    bad = ~torch.isfinite(y)
    assert bad[0, 1, 0].nonzero().flatten().tolist() == [6, 7, 60] and int(bad.sum()) == 3


def test_rope_empty(bl):
    plan = bl.RopePlan(64, (32,))
    q = torch.empty(0, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(4, 1, dtype=torch.int32, device="cuda")
    assert bl.rope(q, q, pos, plan)[0].shape == q.shape
    q = torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert bl.rope(q, q, pos[:0], plan)[1].shape == q.shape


def test_rope_refusals(bl):
    plan = bl.RopePlan(64, (32,))
    q = _randn(2, 4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, lambda: bl.rope(q, q, pos.long(), plan)),
        (TypeError, lambda: bl.rope(q, q.float(), pos, plan)),
        (TypeError, lambda: bl.rope(q, q, pos.cpu(), plan)),
        (ValueError, lambda: bl.rope(q, q, pos[:3], plan)),
        (ValueError, lambda: bl.rope(q, q, pos.expand(4, 2).contiguous(), plan)),
        (ValueError, lambda: bl.rope(q, q[:, :3], pos, plan)),
        (ValueError, lambda: bl.rope(q[..., :32], None, pos, plan)),
        (ValueError, lambda: bl.rope(q.transpose(2, 3).contiguous().transpose(2, 3), None, pos, plan)),
        (ValueError, lambda: bl.rope(q, None, pos, bl.RopePlan(128, (64,)))),
        (bl.BLError, lambda: bl.rope(q[:, :, :1].expand(2, 4, 2, 64), None, pos, plan, inplace=True)),
        (bl.BLError, lambda: bl.rope(q, q, pos, plan, inplace=True)),
        (bl.BLError, lambda: bl.rope(q, q[:, :, 1:], pos, plan, inplace=True)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


def test_rope_in_place_and_autograd(bl):
    """In place, the rotation would be missing from the gradients of a tensor that wants them:
    refused. What autograd holds of a tensor that is then turned counts as changed."""
    plan = bl.RopePlan(64, (32,))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    q, k = (_randn(1, 4, 2, 64, dtype=torch.float32, seed=s) for s in (50, 51))
    before = q.clone()
    wants = q.clone().requires_grad_()
    for args in ((wants, k), (k, wants), (wants * 1, None), (wants[0], None)):
        with pytest.raises(ValueError):
            bl.rope(*args, pos, plan, inplace=True)
    assert torch.equal(wants.detach(), before)
    a = torch.ones_like(q).requires_grad_()
    product = a * q                                      # holds q for a's gradient
    bl.rope(q, k, pos, plan, inplace=True)
    assert torch.equal(q, bl.rope(before, None, pos, plan)[0])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.sum().backward()
    flat = before[0].clone()
    product = a[0] * flat                                # packed tensors too
    bl.rope(flat, None, pos, plan, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.sum().backward()
    with torch.no_grad():                                # as torch's own operations allow
        bl.rope(wants, None, pos, plan, inplace=True)
    assert torch.equal(wants.detach(), q)
    with torch.inference_mode():
        x = before.clone()
        bl.rope(x, None, pos, plan, inplace=True)
        assert torch.equal(x, q)


def test_rope_in_place_on_views_beside_each_other(bl):
    """q and k as other heads of one tensor, at steps of their own, batches inside the tokens,
    heads before them: the values of the call on copies, and nothing else changes."""
    plan = bl.RopePlan(64, (32,))
    pos = torch.randint(0, 500, (7, 1), dtype=torch.int32, device="cuda")
    views = [lambda x: (x[:, :, 0::2], x[:, :, 1::2]), lambda x: (x[:, :, 0:4:2], x[:, :, 4:]),
             lambda x: (x[:, :, 5:], x[:, :, 1:5:3]), lambda x: (x[:, :, :4], x[:, :, 4:5])]
    layouts = [(lambda t: t, (2, 7, 6, 64)), (lambda t: t.transpose(0, 1), (7, 2, 6, 64)),
               (lambda t: t.permute(0, 2, 1, 3), (2, 6, 7, 64)), (lambda t: t.permute(2, 1, 0, 3), (6, 7, 2, 64))]
    for i, view in enumerate(views):
        for layout, shape in layouts:
            x = _randn(*shape, dtype=torch.bfloat16, seed=60 + i)
            want = layout(x.clone())
            for t, turned in zip(view(want), bl.rope(*(t.contiguous() for t in view(want)), pos, plan)):
                t.copy_(turned)
            bl.rope(*view(layout(x)), pos, plan, inplace=True)
            assert torch.equal(layout(x), want)


# --- norm -----------------------------------------------------------------------

SHAPES = [(1, 1), (1, 64), (3, 7), (1000, 64), (517, 128), (33, 129), (5, 256), (9, 264), (7, 1000),
          (4, 1001), (6, 2048), (3, 5120), (2, 5123), (700, 7168), (2, 16384), (5000, 7), (3001, 129), (2000, 250), (900, 777), (1501, 1001), (800, 5123),
          (40, 16383)]


def _norm_inputs(rows, cols, dtype, wtype):
    x = _randn(rows, cols, dtype=dtype, seed=rows)
    r = _randn(rows, cols, dtype=dtype, seed=rows + 1, scale=3.0)
    w = (1 + 0.3 * _randn(cols, dtype=torch.float32, seed=cols)).to(wtype)
    return x, r, w


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_forward(bl, rows, cols, dtype):
    t = TYPES[dtype]
    for residual, w32 in ((True, False), (False, True)):
        x, r, w = _norm_inputs(rows, cols, t, torch.float32 if w32 else t)
        ry, rh, rr = OB.rms_norm(x, w, 1e-6, r if residual else None)
        y, h, rstd = bl.rms_norm_fwd(x, w, 1e-6, residual=r if residual else None)
        _close(y, ry, 64 * F * np.abs(ry), t)
        assert np.abs(_f64(rstd) / rr - 1).max() <= 64 * F
        if residual:
            _close(h, rh, 2 * F * np.abs(rh), t)
        else:
            assert h is x


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (257, 64), (65, 128), (33, 136), (9, 264),
                                       (5, 1000), (4, 1001), (3, 5120), (2, 16384), (3001, 129),
                                       (900, 777), (700, 2563)])
def test_norm_forward_in_8_bits(bl, rows, cols, group, fmt):
    """Codes stand for y within half a step of their format; y beside them is the plain call's."""
    t = torch.bfloat16
    x, r, w = _norm_inputs(rows, cols, t, torch.float32)
    ry, _, _ = OB.rms_norm(x, w, 1e-6, r)
    y, y8, h, rstd = bl.rms_norm_fwd_8bit(x, w, 1e-6, residual=r, fmt=fmt, group=group, with_y=True)
    plain = bl.rms_norm_fwd(x, w, 1e-6, residual=r)
    assert torch.equal(y, plain[0]) and torch.equal(h, plain[1]) and torch.equal(rstd, plain[2])
    only, h2, _ = bl.rms_norm_fwd_8bit(x, w, 1e-6, residual=r, fmt=fmt, group=group)
    assert torch.equal(only.codes.view(torch.uint8), y8.codes.view(torch.uint8))
    assert torch.equal(only.scales, y8.scales) and torch.equal(h2, h)
    codes = y8.codes.cpu().view(torch.uint8 if fmt == "e4m3" else torch.int8).numpy()
    scales = y8.scales.cpu().numpy()
    size = group or cols
    want = np.stack([np.abs(ry[:, j:j + size]).max(axis=1) for j in range(0, cols, size)], 1) / \
        (127.0 if fmt == "int8" else 448.0)
    assert np.abs(scales / want - 1).max() <= 66 * F
    s = np.repeat(scales, size, axis=1)[:, :cols].astype(np.float64)
    step = 0.5 * s if fmt == "int8" else np.maximum(np.abs(ry) / 16, s * 2.0 ** -10)
    back = OB.load8(codes, scales, group)
    assert (np.abs(back - ry) <= step * (1 + 1e-4) + 70 * F * np.abs(ry)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (257, 64), (33, 136), (9, 264), (4, 1001), (900, 777),
                                       (500, 1024), (700, 2563), (3, 5120), (2, 8192), (2, 16380), (2, 16384)])
@pytest.mark.parametrize("dtype,w32", [("fp16", False), ("fp16", True), ("fp32", True)])
def test_norm_forward_of_other_types_in_8_bits(bl, rows, cols, group, fmt, dtype, w32):
    """The bf16 test's bounds for fp16 and fp32, with a residual and without: aligned rows, rows too
    wide for the ring and rows that start anywhere."""
    t = TYPES[dtype]
    x, r, w = _norm_inputs(rows, cols, t, torch.float32 if w32 else t)
    for residual in (r, None):
        ry, _, _ = OB.rms_norm(x, w, 1e-6, residual)
        y, y8, h, rstd = bl.rms_norm_fwd_8bit(x, w, 1e-6, residual=residual, fmt=fmt, group=group, with_y=True)
        plain = bl.rms_norm_fwd(x, w, 1e-6, residual=residual)
        # fp32 rows that start anywhere: without 8 bits another order of the sum
        for a, b in zip((y, rstd), (plain[0], plain[2])):
            assert torch.equal(a, b) or (dtype == "fp32" and U.rel_l2(U.cpu(a), U.cpu(b)) <= 64 * F)
        _close(y, ry, 64 * F * np.abs(ry), t)
        assert torch.equal(h, plain[1])
        only, h2, _ = bl.rms_norm_fwd_8bit(x, w, 1e-6, residual=residual, fmt=fmt, group=group)
        assert torch.equal(only.codes.view(torch.uint8), y8.codes.view(torch.uint8))
        assert torch.equal(only.scales, y8.scales) and torch.equal(h2, h)
        codes, scales = _codes_np(y8), y8.scales.cpu().numpy()
        size = group or cols
        want = np.stack([np.abs(ry[:, j:j + size]).max(axis=1) for j in range(0, cols, size)], 1) / \
            (127.0 if fmt == "int8" else 448.0)
        assert np.abs(scales / want - 1).max() <= 66 * F
        s = np.repeat(scales, size, axis=1)[:, :cols].astype(np.float64)
        step = 0.5 * s if fmt == "int8" else np.maximum(np.abs(ry) / 16, s * 2.0 ** -10)
        back = OB.load8(codes, scales, group)
        assert (np.abs(back - ry) <= step * (1 + 1e-4) + 70 * F * np.abs(ry)).all()


@pytest.mark.parametrize("saved", ["same", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 128), (700, 5120)])
def test_norm_backward(bl, rows, cols, dtype, saved):
    t = TYPES[dtype]
    h, g_h, w = _norm_inputs(rows, cols, t, t)
    g_y = _randn(rows, cols, dtype=t, seed=rows + 2)
    rstd = torch.rsqrt((h.float() ** 2).mean(-1) + 1e-6)
    for group, with_h, weight in ((0, True, w), (64, False, w.float()), (128, True, None)):
        h8 = h if saved == "same" else bl.act_save(h, saved, group)
        if saved == "same":
            value = _f64(h)
        else:
            codes = h8.codes.cpu().view(torch.uint8 if saved == "e4m3" else torch.int8).numpy()
            value = OB.load8(codes, h8.scales.cpu().numpy(), group)
        ref_x, ref_w = OB.rms_norm_backward(g_y, value, rstd, weight, g_h if with_h else None)
        g_x, g_w = bl.rms_norm_bwd(g_y, h8, rstd, weight, g_h=g_h if with_h else None)
        u = np.abs(value * _f64(rstd)[:, None])
        gw = np.abs(_f64(g_y)) * (1 if weight is None else np.abs(_f64(weight)))
        mag = _f64(rstd)[:, None] * (gw + u * (gw * u).mean(axis=1, keepdims=True))
        if with_h:
            mag = mag + np.abs(_f64(g_h))
        _close(g_x, ref_x, 64 * F * mag, t)
        assert g_w.dtype == (torch.float32 if weight is None else weight.dtype)
        _close(g_w, ref_w, (rows + 64) * F * (np.abs(_f64(g_y)) * u).sum(axis=0), g_w.dtype)
        again = bl.rms_norm_bwd(g_y, h8, rstd, weight, g_h=g_h if with_h else None)
        assert torch.equal(again[0], g_x) and torch.equal(again[1], g_w)      # a fixed order
        only, none = bl.rms_norm_bwd(g_y, h8, rstd, weight, g_h=g_h if with_h else None,
                                     need_g_w=False)
        assert none is None and torch.equal(only, g_x)


@pytest.mark.parametrize("saved", ["same", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(9, 8), (13, 64), (7, 129), (5, 264), (300, 1001), (6, 1024), (4, 4096),
                                       (3, 5123), (2, 10000)])
def test_norm_backward_of_rows_of_any_size(bl, rows, cols, dtype, saved):
    """Rows around 1e-20, 1 and 1e18 beside each other, with gradients whose g_x has a place in
    the type: rstd^2 alone would leave fp32's range on either side."""
    t = TYPES[dtype]
    size = torch.tensor([1e-20, 1.0, 1e18], device="cuda")[torch.arange(rows, device="cuda") % 3][:, None]
    grad = torch.tensor([1.0, 1.0, 1e-12], device="cuda")[torch.arange(rows, device="cuda") % 3][:, None]
    h = (_randn(rows, cols, dtype=torch.float32, seed=rows) * size).to(t)
    g_y = (_randn(rows, cols, dtype=torch.float32, seed=rows + 1) * grad).to(t)
    w = 1 + 0.3 * _randn(cols, dtype=torch.float32, seed=cols)
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(-1))).float()
    h8, value = h, _f64(h)
    if saved != "same":
        h8 = bl.act_save(h, saved, 64)
        value = OB.load8(h8.codes.cpu().numpy(), h8.scales.cpu().numpy(), 64)
    ref_x, ref_w = OB.rms_norm_backward(g_y, value, rstd, w)
    g_x, g_w = bl.rms_norm_bwd(g_y, h8, rstd, w)
    u = np.abs(value * _f64(rstd)[:, None])
    gw = np.abs(_f64(g_y)) * np.abs(_f64(w))
    mag = _f64(rstd)[:, None] * (gw + u * (gw * u).mean(axis=1, keepdims=True))
    _close(g_x, ref_x, 64 * F * mag, t)
    _close(g_w, ref_w, (rows + 64) * F * (np.abs(_f64(g_y)) * u).sum(axis=0), torch.float32)


def test_norm_takes_views(bl):
    """Row strides, leading dims, unaligned bases: the contiguous call's values."""
    big = _randn(6, 10, 384, dtype=torch.bfloat16, seed=9)
    w = _randn(128, dtype=torch.float32, seed=10)
    x, r = big[..., :128], big[..., 128:256]
    want = bl.rms_norm_fwd(x.contiguous(), w, residual=r.contiguous())
    got = bl.rms_norm_fwd(x, w, residual=r)
    assert got[0].shape == (6, 10, 128) and got[2].shape == (6, 10)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    odd = torch.empty(60 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(6, 10, 128)
    odd.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(bl.rms_norm_fwd(odd, w, residual=r), want))
    with pytest.raises(ValueError):
        bl.rms_norm_fwd(big.transpose(0, 1)[..., :128], w)


@pytest.mark.parametrize("cols", [24, 136, 1000, 2568])
def test_norm_rows_that_start_anywhere(bl, cols):
    """Every misalignment of base and stride: the aligned call's values (codes bit for bit)."""
    rows = 37
    w = _randn(cols, dtype=torch.float32, seed=cols)
    x, r = _randn(rows, cols, dtype=torch.bfloat16, seed=1), _randn(rows, cols, dtype=torch.bfloat16, seed=2)
    want = bl.rms_norm_fwd(x, w, residual=r)
    want8 = bl.act_save(x, "int8", 32), bl.act_save(x, "e4m3", 0)
    for off in range(8):
        for pad in (0, 1, 3, 6):
            buf = torch.full((rows * (cols + pad) + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
            view = buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
            view.copy_(x)
            got = bl.rms_norm_fwd(view, w, residual=r)
            # sums of the odd layout's threads may run in another order
            for a, b in zip(got, want):
                assert U.rel_l2(U.cpu(a), U.cpu(b)) <= 2.0 ** -10 and torch.isfinite(a).all()
            for f, a in zip((("int8", 32), ("e4m3", 0)), want8):
                b = bl.act_save(view, *f)
                assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
                assert torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("cols", [1, 9, 129, 264, 1001, 1030, 5123])
@pytest.mark.parametrize("off", [0, 1, 3, 6])
def test_outputs_that_start_anywhere_keep_their_neighbours(bl, cols, off):
    """Through the C ABI, every output in the middle of a buffer: the bytes in front of it and
    behind it stay, and all of its own are written."""
    import ctypes
    from block_sparse_attention_fwd_gb300 import _lib
    lib = _lib.load()
    rows, dev = 21, "cuda"
    x, r = _randn(rows, cols, dtype=torch.bfloat16, seed=3), _randn(rows, cols, dtype=torch.bfloat16, seed=4)
    n = rows * cols

    def room(dtype, fill):
        whole = torch.full((n + 64,), fill, dtype=dtype, device=dev)
        return whole, whole[16 + off:16 + off + n]

    def untouched(whole, fill):
        return bool((whole[:16 + off] == fill).all() and (whole[16 + off + n:] == fill).all())

    y, h, g = (room(torch.bfloat16, 7.0) for _ in range(3))
    codes, saved = room(torch.int8, 77), room(torch.int8, 77)
    scales = torch.empty(rows, dtype=torch.float32, device=dev)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    act = _lib.Act8Struct(codes[1].data_ptr(), scales.data_ptr(), 1, 0)
    s = torch.cuda.current_stream().cuda_stream
    assert lib.bl_rms_norm_fwd(rows, cols, 0, x.data_ptr(), cols, r.data_ptr(), cols, None, 0, 1e-6,
                               y[1].data_ptr(), h[1].data_ptr(), rstd.data_ptr(), ctypes.byref(act), s) == 0
    ry, rh, rr = bl.rms_norm_fwd(x, None, residual=r)
    assert U.rel_l2(U.cpu(y[1]), U.cpu(ry).ravel()) <= 2.0 ** -10
    assert torch.equal(h[1], rh.flatten())
    assert untouched(y[0], 7.0) and untouched(h[0], 7.0) and untouched(codes[0], 77)
    value = U.cpu(codes[1]).reshape(rows, cols) * U.cpu(scales)[:, None]
    assert np.abs(value - U.cpu(ry)).max() <= 0.5 * U.cpu(scales).max() * 1.02 + 2.0 ** -8 * np.abs(U.cpu(ry)).max()
    assert lib.bl_rms_norm_bwd(rows, cols, 0, x.data_ptr(), h[1].data_ptr(), None, rstd.data_ptr(), None,
                               0, r.data_ptr(), g[1].data_ptr(), None, None, 0, s) == 0
    want = bl.rms_norm_bwd(x, rh, rstd, None, g_h=r, need_g_w=False)[0]
    assert U.rel_l2(U.cpu(g[1]), U.cpu(want).ravel()) <= 2.0 ** -9 and untouched(g[0], 7.0)
    own = torch.empty(rows, dtype=torch.float32, device=dev)
    act = _lib.Act8Struct(saved[1].data_ptr(), own.data_ptr(), 1, 0)
    assert lib.bl_act_save(rows, cols, 0, x.data_ptr(), cols, ctypes.byref(act), s) == 0
    ref = bl.act_save(x)
    assert torch.equal(saved[1], ref.codes.flatten()) and untouched(saved[0], 77)
    back = room(torch.bfloat16, 7.0)
    assert lib.bl_act_load(rows, cols, 0, ctypes.byref(act), back[1].data_ptr(), s) == 0
    assert torch.equal(back[1], bl.act_load(ref).flatten()) and untouched(back[0], 7.0)


def test_norm_edge_rows(bl):
    """A zero row, an infinity and a NaN stay within their rows; no rows at all."""
    x = _randn(4, 512, dtype=torch.bfloat16, seed=11)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    y, _, rstd = bl.rms_norm_fwd(x, None, 1e-6)
    assert (y[0] == 0).all() and float(rstd[0]) == pytest.approx(1000.0, rel=1e-6)
    assert torch.isnan(y[1, 5]) and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()
    y8, _, _ = bl.rms_norm_fwd_8bit(x, None, 1e-6, group=64)
    back = bl.act_load(y8)
    assert (back[0] == 0).all() and torch.isnan(back[2]).all() and torch.isfinite(back[3]).all()
    none = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = bl.rms_norm_fwd(none, None, residual=none)
    assert y.shape == h.shape == (0, 512) and rstd.shape == (0,)
    g_x, g_w = bl.rms_norm_bwd(none, none, rstd, None)
    assert g_x.shape == (0, 512) and (g_w == 0).all() and g_w.shape == (512,)


def test_norm_refusals(bl):
    x = _randn(4, 64, dtype=torch.bfloat16)
    w = _randn(64, dtype=torch.bfloat16)
    r = torch.ones(4, device="cuda")
    wide = torch.empty(1, 16385, dtype=torch.bfloat16, device="cuda")
    bad = [
        (TypeError, lambda: bl.rms_norm_fwd(x.double(), w)),
        (TypeError, lambda: bl.rms_norm_fwd(x, w.half())),
        (ValueError, lambda: bl.rms_norm_fwd(x, w[:32])),
        (ValueError, lambda: bl.rms_norm_fwd(x, w, residual=x.float())),
        (ValueError, lambda: bl.rms_norm_fwd(x, w, residual=x[:2])),
        (ValueError, lambda: bl.rms_norm_fwd(wide, None)),
        (bl.BLError, lambda: bl.rms_norm_fwd(x, w, eps=-1.0)),
        (bl.BLError, lambda: bl.rms_norm_fwd(x, w, eps=float("nan"))),
        (ValueError, lambda: bl.rms_norm_fwd_8bit(x, w, fmt="int4")),
        (ValueError, lambda: bl.rms_norm_fwd_8bit(x, w, group=16)),
        (ValueError, lambda: bl.rms_norm_bwd(x, x, r[:3], w)),
        (TypeError, lambda: bl.rms_norm_bwd(x, x.float(), r, w)),
        (ValueError, lambda: bl.rms_norm_bwd(x, x[:2], r, w)),
        (TypeError, lambda: bl.rms_norm_bwd(x, bl.act_save(x.float()), r, w)),
        (ValueError, lambda: bl.rms_norm_bwd(x.t().contiguous().t(), x, r, w)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


# --- 8 bits ---------------------------------------------------------------------

def _codes_np(a):
    c = a.codes.cpu()
    return (c.view(torch.uint8) if c.dtype == torch.float8_e4m3fn else c).numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 5), (300, 64), (77, 128), (1, 32), (5, 96), (33, 130),
                                       (4, 1000), (3, 1001), (2, 5120), (2, 20000), (3001, 129),
                                       (900, 777), (500, 2563), (2000, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_saved_codes_are_the_definition_bit_for_bit(bl, rows, cols, group, fmt, dtype):
    t = TYPES[dtype]
    x = _randn(rows, cols, dtype=t, seed=cols, scale=2.0)
    if rows > 1:
        x[1] = x[1] * 1e-4          # fp16 subnormals among them
    a = bl.act_save(x, fmt, group)
    codes, scales = OB.save8(x, fmt, group)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    assert np.array_equal(_codes_np(a), codes)
    back = bl.act_load(a)
    assert back.dtype == t and back.shape == x.shape
    ref = OB.load8(codes, scales, group)
    _close(back, ref, F * np.abs(ref), t)


def test_saved_edges(bl):
    """Zeros, the smallest and the largest values, NaN and infinities, no rows."""
    x = torch.zeros(6, 128, dtype=torch.float32, device="cuda")
    x[1, 3] = 1e-45                       # the smallest subnormal
    x[2] = 3.4028234e38
    x[2, ::2] = -3.4028234e38
    x[3, 70] = float("inf")
    x[4, 10] = float("nan")
    x[5, 0] = 1.2e-38
    for fmt in ("int8", "e4m3"):
        for group in (0, 64):
            a = bl.act_save(x, fmt, group)
            codes, scales = OB.save8(x, fmt, group)
            assert np.array_equal(a.scales.cpu().numpy(), scales, equal_nan=True)
            assert np.array_equal(_codes_np(a), codes)
            back = bl.act_load(a).cpu()
            assert (back[0] == 0).all() and torch.isfinite(back[[0, 1, 2, 5]]).all()
            assert torch.isnan(back[3, 64:]).all() and torch.isnan(back[4, :64]).all()
            assert torch.isnan(back[3, :64]).all() == (group == 0)
        none = bl.act_save(x[:0], fmt, 32)
        assert none.scales.shape == (0, 4) and bl.act_load(none).shape == (0, 128)


def test_saved_views(bl):
    big = _randn(5, 8, 200, dtype=torch.float16, seed=12)
    x = big[..., 8:136]
    for group in (0, 32):
        a, b = bl.act_save(x, "int8", group), bl.act_save(x.contiguous(), "int8", group)
        assert a.shape == x.shape and torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    odd = big[..., 3:131]                               # rows start off the vectors' alignment
    a, b = bl.act_save(odd, "e4m3", 64), bl.act_save(odd.contiguous(), "e4m3", 64)
    assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
    with pytest.raises(ValueError):
        bl.act_save(big.transpose(1, 2))
    with pytest.raises(ValueError):
        bl.act_save(big, "fp8")
    with pytest.raises(ValueError):
        bl.act_save(big, "int8", 16)


# --- the attention's backward from 8 bits -----------------------------------------

ATTN = [
    # B, n, H, Hk, d, causal, fmt, o in 8 bits
    (1, 1, 1, 1, 64, False, "int8", True),
    (1, 65, 2, 1, 64, False, "int8", False),
    (2, 300, 4, 2, 128, True, "e4m3", True),
    (1, 600, 3, 3, 128, False, "int8", True),
    (1, 129, 6, 2, 64, True, "e4m3", False),
    (1, 257, 2, 2, 128, False, "e4m3", False),
    (2, 513, 8, 2, 64, False, "int8", False),
    (1, 400, 5, 1, 128, True, "int8", True),
]


def _attn_case(bl, B, n, H, Hk, d, causal, fmt, seed=20):
    q = _randn(B, n, H, d, dtype=torch.bfloat16, seed=seed)
    k = _randn(B, n, Hk, d, dtype=torch.bfloat16, seed=seed + 1)
    v = _randn(B, n, Hk, d, dtype=torch.bfloat16, seed=seed + 2)
    g_o = _randn(B, n, H, d, dtype=torch.bfloat16, seed=seed + 3)
    shape = bl.make_shape(B, n, H, Hk, d, 128, 128, int(causal))
    o = torch.empty_like(q)
    lse = torch.empty((B, H, n), dtype=torch.float32, device="cuda")
    bl.attn_fwd(shape, q, k, v, d ** -0.5, o, lse)
    return shape, (q, k, v, o), g_o, lse, [bl.act_save(t, fmt) for t in (q, k, v, o)]


def _same_kv_gradients(got, ref, other_order):
    """G_K and G_V bit for bit; where few items make the call add the heads of a group in
    another order, fp32 sums that differ by their last bits round to another bf16 value
    now and then: with a share p of the elements one step (2^-8 at most) off, rel-L2 is
    2^-8 sqrt(p), and p stays below 2^-6 (sums of 2^6 F around a step of 2^16 F)."""
    for a, b in zip(got[1:], ref[1:]):
        if other_order:
            assert U.rel_l2(U.cpu(a), U.cpu(b)) <= 2.0 ** -11
        else:
            assert torch.equal(a, b)


@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"n{c[1]}d{c[4]}{c[6]}")
def test_attention_backward_from_8_bits(bl, case):
    B, n, H, Hk, d, causal, fmt, o_in8 = case
    scale = d ** -0.5
    shape, (q, k, v, o), g_o, lse, (q8, k8, v8, o8) = _attn_case(bl, B, n, H, Hk, d, causal, fmt)
    ws = torch.empty(bl.attn_bwd_act8_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)                                       # nothing may depend on what it held
    got = bl.attn_bwd_act8(shape, q8, k8, v8, o8 if o_in8 else o, g_o, lse, scale, workspace=ws)
    assert bl.bwd_check_status(shape, ws) == 0
    # the same call on the loaded tensors, with o as the values its codes stand for
    qb, kb, vb = (bl.act_load(t) for t in (q8, k8, v8))
    if not o_in8:
        ref = [torch.empty_like(t) for t in (qb, kb, vb)]
        w2 = torch.empty(bl.bwd_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
        bl.attn_bwd(shape, qb, kb, vb, o, g_o, lse, scale, None, *ref, w2)
        _same_kv_gradients(got, ref, H != Hk)
        assert U.rel_l2(U.cpu(got[0]), U.cpu(ref[0])) <= 1e-3 or n == 1
    if n == 1:
        # one key: P = exp(s q.k - lse) with the rounded q and k, G_V = P G_O, and G_Q and
        # G_K are roundings' remains; only G_V says anything
        p = np.exp(scale * (_f64(qb) * _f64(kb)).sum() - _f64(lse).item())
        assert U.rel_l2(U.cpu(got[2]), p * _f64(g_o)) <= U.REL_L2
        return
    value = o.float() if not o_in8 else o8.codes.float() * o8.scales
    rq, rk, rv = A.backward(qb.float().cpu(), kb.float().cpu(), vb.float().cpu(), value.cpu(),
                            g_o.float().cpu(), lse.cpu(), scale, None, 128, 128, causal=causal)
    for g, r in zip(got, (rq, rk, rv)):
        assert U.rel_l2(U.cpu(g), r) <= U.REL_L2


def test_attention_backward_from_8_bits_keeps_a_mask(bl):
    """With tile lists, dropped tiles add nothing: the same as the bf16 call on the loaded tensors."""
    from block_sparse_attention_fwd_gb300 import inputs
    w = inputs.custom("act8_mask", B=1, n=1000, H=4, Hk=2, d=128, run=48, clusters=8, alpha=3.0)
    q, k, v, g_o = (x.cuda() for x in inputs.generate(w, seed=3))
    shape = bl.make_shape(w.B, w.n, w.H, w.Hk, w.d, 128, 128)
    q, k, v, o, lse, stats = U.gpu_forward(shape, q, k, v, w.scale)
    lists = U.gpu_mask(shape, stats, lse, 0.05)
    assert 0 < int(lists["mask"].sum()) < lists["mask"].numel()
    q8, k8, v8 = (bl.act_save(t) for t in (q, k, v))
    got = bl.attn_bwd_act8(shape, q8, k8, v8, o, g_o, lse, w.scale, lists)
    ref = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(bl.bwd_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    bl.attn_bwd(shape, *(bl.act_load(t) for t in (q8, k8, v8)), o, g_o, lse, w.scale, lists, *ref, ws)
    _same_kv_gradients(got, ref, True)
    assert U.rel_l2(U.cpu(got[0]), U.cpu(ref[0])) <= 1e-3


@pytest.mark.parametrize("B,n,H,Hk,bq", [(1, 10000, 4, 2, 128), (1, 700, 4, 2, 64)])
def test_attention_backward_from_8_bits_of_kv_heads(bl, B, n, H, Hk, bq):
    """Grouped heads with an item for every SM, or tiles of 64: bf16's own order of sums."""
    _, (q, k, v, o), g_o, lse, (q8, k8, v8, _) = _attn_case(bl, B, n, H, Hk, 64, False, "int8")
    shape = bl.make_shape(B, n, H, Hk, 64, bq, bq)
    got = bl.attn_bwd_act8(shape, q8, k8, v8, o, g_o, lse, 0.125)
    ref = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(bl.bwd_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    bl.attn_bwd(shape, *(bl.act_load(t) for t in (q8, k8, v8)), o, g_o, lse, 0.125, None, *ref, ws)
    _same_kv_gradients(got, ref, False)
    assert U.rel_l2(U.cpu(got[0]), U.cpu(ref[0])) <= 1e-3


FEW = [
    # B, n, H, Hk, d, causal, window, tile, fmt, o in 8 bits, heads whose tile a mask drops (None: no lists)
    (1, 1, 1, 1, 64, False, 0, 128, "int8", True, None),
    (3, 1, 6, 2, 128, True, 0, 128, "e4m3", False, None),
    (2, 2, 4, 1, 64, True, 1, 128, "int8", False, None),
    (1, 15, 3, 3, 128, False, 0, 128, "int8", True, None),
    (2, 16, 4, 2, 128, True, 0, 128, "e4m3", True, None),
    (1, 17, 5, 1, 64, True, 0, 128, "int8", False, None),
    (2, 33, 6, 2, 128, True, 16, 128, "int8", True, None),
    (1, 48, 4, 4, 64, True, 17, 128, "e4m3", False, None),
    (2, 63, 6, 3, 64, False, 0, 64, "int8", True, (0, 3, 7)),
    (1, 64, 8, 2, 128, True, 0, 128, "int8", False, (0, 1, 2, 3)),
    (1, 64, 2, 1, 128, True, 40, 128, "e4m3", True, (1,)),
    (2, 64, 3, 1, 128, False, 0, 128, "int8", False, (0, 1, 2, 3, 4, 5)),
]


@pytest.mark.parametrize("case", FEW, ids=lambda c: f"n{c[1]}d{c[4]}{c[8]}")
def test_attention_backward_from_8_bits_of_few_tokens(bl, case):
    """Up to 64 tokens, element by element: half a step of bf16 and what fp32 can lose.

    A matrix instruction adds 16 exact products to an accumulator; with every of the 17
    terms cut at 2^-23 of the largest it is off by 17 * 2^-23 of the sum of their sizes,
    so d / 16 of them in a row by m * 2^-24, m = 2.125 d.  The sums over n G pairs take
    two parts, 4.25 (n G + 15) * 2^-24, and three additions of warps' sums; the parts
    leave 2^-16 of P and of dS.  P = 2^x with x = log2(e) (s S - LSE) is off, relative to
    it, by the error of s S and by 2^-21 of |s S| + |LSE| + 4 (three roundings of x, the
    constants', exp2's two units)."""
    B, n, H, Hk, d, causal, window, tile, fmt, o_in8, dropped = case
    scale, G, u = d ** -0.5, H // Hk, 2.0 ** -24
    q, g_o = (_randn(B, n, H, d, dtype=torch.bfloat16, seed=s) for s in (41, 42))
    k, v = (_randn(B, n, Hk, d, dtype=torch.bfloat16, seed=s) for s in (43, 44))
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    attends = (j <= i if causal else np.ones((n, n), bool)) & (i - j < (window or n))
    heads = lambda t: np.repeat(_f64(t).transpose(0, 2, 1, 3), G if t.shape[2] != H else 1, 1)  # noqa: E731
    S = np.where(attends, scale * heads(q) @ heads(k).swapaxes(2, 3), -np.inf)
    top = S.max(-1, keepdims=True)
    e = np.exp(S - top)
    o = (e / e.sum(-1, keepdims=True)) @ heads(v)
    lse = torch.from_numpy((top + np.log(e.sum(-1, keepdims=True)))[..., 0]).float().cuda()
    o = torch.from_numpy(o.transpose(0, 2, 1, 3)).to(torch.bfloat16).contiguous().cuda()
    q8, k8, v8, o8 = (bl.act_save(t, fmt) for t in (q, k, v, o))
    shape = bl.make_shape(B, n, H, Hk, d, tile, tile, int(causal), window)
    lists, on = None, np.ones((B, H))
    if dropped is not None:
        on.reshape(-1)[list(dropped)] = 0
        lists = bl.alloc_lists(shape, q.device)
        for name, t in lists.items():
            t.fill_(0)
        lists["q_cnt"].copy_(torch.from_numpy(on).to(torch.int32)[..., None])
        lists["q_idx"].masked_fill_(lists["q_cnt"][..., None] == 0, -7)        # never read
    ws = torch.full((bl.attn_bwd_act8_workspace_bytes(shape),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: bl.attn_bwd_act8(shape, q8, k8, v8, o8 if o_in8 else o, g_o, lse, scale, lists,  # noqa: E731
                                    workspace=ws)
    got = call()
    assert bl.bwd_check_status(shape, ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, call()))

    Q, K, V = (heads(bl.act_load(t)) for t in (q8, k8, v8))
    O = heads(o8.codes.float().double() * o8.scales.double()) if o_in8 else heads(o)
    dO, L = heads(g_o), _f64(lse)[..., None]
    use = attends * on[:, :, None, None]
    T = lambda x: x.swapaxes(2, 3)  # noqa: E731
    s = scale * Q @ T(K)
    P = np.where(use > 0, np.exp(np.where(use > 0, s - L, 0)), 0)
    D = (dO * O).sum(-1, keepdims=True)
    dP = dO @ T(V)
    dS = P * (dP - D)
    m = 2.125 * d
    eP = P * (scale * m * u * (abs(Q) @ T(abs(K))) + 2.0 ** -21 * (abs(s) + abs(L) + 4) + 2.0 ** -16)
    eD = (d + 4) * u * (abs(dO) * abs(O)).sum(-1, keepdims=True)
    edS = eP * abs(dP - D) + (P + eP) * (m * u * (abs(dO) @ T(abs(V))) + eD) + 2.0 ** -16 * abs(dS)
    terms = 4.25 * (n * G + 15) + 3
    sum_group = lambda x: x.reshape(B, Hk, G, n, d).sum(2)  # noqa: E731
    want = [(scale * dS @ K, scale * (edS + terms * u * abs(dS)) @ abs(K)),
            (sum_group(scale * T(dS) @ Q), sum_group(scale * T(edS + terms * u * abs(dS)) @ abs(Q))),
            (sum_group(T(P) @ dO), sum_group(T(eP + terms * u * P) @ abs(dO)))]
    for g, (ref, noise) in zip(got, want):
        err = abs(_f64(g).transpose(0, 2, 1, 3) - ref)
        assert np.all(err <= 2.0 ** -8 * (abs(ref) + noise) + noise + 2.0 ** -130)


def test_attention_backward_from_8_bits_of_few_tokens_reports_bad_lists(bl):
    shape, (q, k, v, o), g_o, lse, (q8, k8, v8, _) = _attn_case(bl, 1, 20, 3, 1, 64, False, "int8")
    lists = bl.alloc_lists(shape, q.device)
    for t in lists.values():
        t.fill_(0)
    lists["q_cnt"].copy_(torch.tensor([[[1], [2], [1]]], dtype=torch.int32))
    lists["q_idx"].copy_(torch.tensor([0, 0, 5], dtype=torch.int32).view(1, 3, 1, 1))
    ws = torch.empty(bl.attn_bwd_act8_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    got = bl.attn_bwd_act8(shape, q8, k8, v8, o, g_o, lse, 0.125, lists, workspace=ws)
    assert bl.bwd_check_status(shape, ws) != 0
    assert got[0][:, :, 0].any() and not got[0][:, :, 1:].any()       # only head 0's list stands


def test_attention_backward_from_8_bits_refusals(bl):
    shape, (q, k, v, o), g_o, lse, (q8, k8, v8, o8) = _attn_case(bl, 1, 130, 2, 1, 64, False, "int8")
    s = 0.125
    bad = [
        (TypeError, lambda: bl.attn_bwd_act8(shape, q, k8, v8, o, g_o, lse, s)),
        (TypeError, lambda: bl.attn_bwd_act8(shape, q8, bl.act_save(k, "e4m3"), v8, o, g_o, lse, s)),
        (ValueError, lambda: bl.attn_bwd_act8(shape, bl.act_save(q, "int8", 32), k8, v8, o, g_o, lse, s)),
        (ValueError, lambda: bl.attn_bwd_act8(shape, bl.act_save(q.float()), k8, v8, o, g_o, lse, s)),
        (ValueError, lambda: bl.attn_bwd_act8(shape, q8, q8, v8, o, g_o, lse, s)),
        (ValueError, lambda: bl.attn_bwd_act8(shape, q8, k8, v8, o[:, :5], g_o, lse, s)),
        (bl.BLError, lambda: bl.attn_bwd_act8(shape, q8, k8, v8, o, g_o, lse, 0.0)),
        (bl.BLError, lambda: bl.attn_bwd_act8(
            shape, q8, k8, v8, o, g_o, lse, s,
            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


# --- sizes past 32 bits ------------------------------------------------------------

def test_offsets_past_32_bits(bl):
    """More than 2^31 elements: the last rows are as if they stood alone."""
    rows = (2 ** 31) // 128 + 40000
    x = torch.empty(rows, 128, dtype=torch.bfloat16, device="cuda")
    x[:1000] = 1.0
    tail = _randn(1000, 128, dtype=torch.bfloat16, seed=30)
    x[1000:-1000] = 0.5
    x[-1000:] = tail
    a, b = bl.act_save(x), bl.act_save(tail)
    assert torch.equal(a.codes[-1000:], b.codes) and torch.equal(a.scales[-1000:], b.scales)
    back = bl.act_load(a)
    assert torch.equal(back[-1000:], bl.act_load(b))
    del back
    y, _, rstd = bl.rms_norm_fwd(x, None)
    y2, _, rstd2 = bl.rms_norm_fwd(tail, None)
    assert torch.equal(y[-1000:], y2) and torch.equal(rstd[-1000:], rstd2)
    g_x, _ = bl.rms_norm_bwd(y, a, rstd, None, need_g_w=False)
    assert torch.equal(g_x[-1000:], bl.rms_norm_bwd(y2, b, rstd2, None, need_g_w=False)[0])
    del y, g_x, a
    plan = bl.RopePlan(128, (64,))
    pos = torch.arange(rows // 8, dtype=torch.int32, device="cuda")[:, None]
    q = x[:rows // 8 * 8].view(1, rows // 8, 8, 128)
    got = bl.rope(q, None, pos, plan)[0]
    assert torch.equal(got[:, -100:], bl.rope(q[:, -100:], None, pos[-100:].contiguous(), plan)[0])
    del got
    got = bl.rope(q[..., 1:-1], None, pos, bl.RopePlan(126, (63,)))[0]      # element by element
    want = bl.rope(q[:, -100:, :, 1:-1], None, pos[-100:].contiguous(), bl.RopePlan(126, (63,)))[0]
    assert torch.equal(got[:, -100:], want)
