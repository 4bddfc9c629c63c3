"""Pins of the oracle of the operators around the attention (fp64, CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import block as OB


# --- rotary ---------------------------------------------------------------------

def _rope_case(seed=0, B=2, n=5, heads=3, d=24, sections=(3, 4, 2)):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, n, heads, d))
    pos = rng.integers(-50, 2000, size=(B, n, len(sections)))
    freqs = rng.uniform(1e-4, 1.0, size=sum(sections))
    return x, pos, sections, freqs


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product(interleaved):
    x, pos, sections, freqs = _rope_case()
    P = sum(sections)
    got = OB.rope(x, pos, sections, freqs, interleaved)
    angle = np.concatenate([pos[..., a:a + 1] * freqs[sum(sections[:a]):sum(sections[:a + 1])]
                            for a in range(3)], axis=-1)[:, :, None, :]
    a, b = (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])
    z = (a + 1j * b) * np.exp(1j * angle)
    ga, gb = (got[..., 0:2 * P:2], got[..., 1:2 * P:2]) if interleaved else \
        (got[..., :P], got[..., P:2 * P])
    assert np.abs(ga - z.real).max() < 1e-10 and np.abs(gb - z.imag).max() < 1e-10
    assert np.array_equal(got[..., 2 * P:], x[..., 2 * P:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(interleaved):
    """The inverse undoes the rotation, and is its transpose: <R x, g> = <x, R^-1 g>."""
    x, pos, sections, freqs = _rope_case(1)
    g = np.random.default_rng(2).standard_normal(x.shape)
    y = OB.rope(x, pos, sections, freqs, interleaved)
    assert np.abs(OB.rope(y, pos, sections, freqs, interleaved, inverse=True) - x).max() < 1e-12
    back = OB.rope(g, pos, sections, freqs, interleaved, inverse=True)
    assert abs((y * g).sum() - (x * back).sum()) < 1e-10


def test_rope_scores_depend_on_the_distance_only():
    """With one axis, q.k of rotated vectors is a function of the positions' difference."""
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 1, 1, 8))
    freqs = [10000.0 ** (-j / 4) for j in range(4)]

    def score(i, j):
        a = OB.rope(q, [[[i]]], (4,), freqs, False)
        b = OB.rope(k, [[[j]]], (4,), freqs, False)
        return float((a * b).sum())

    assert abs(score(17, 5) - score(100017, 100005)) < 1e-9
    assert abs(score(17, 5) - score(5, 17)) > 1e-3


# --- norm -----------------------------------------------------------------------

@pytest.mark.parametrize("residual", [False, True])
def test_norm_and_gradients_match_torch_autograd(residual):
    g = torch.Generator().manual_seed(4)
    x, r, gy, gh = (torch.randn(7, 33, dtype=torch.float64, generator=g) for _ in range(4))
    w = torch.randn(33, dtype=torch.float64, generator=g)
    for t in (x, r, w):
        t.requires_grad_()
    h = x + r if residual else x
    y = torch.nn.functional.rms_norm(h, (33,), w, eps=1e-5)
    loss = (y * gy).sum() + ((h * gh).sum() if residual else 0)
    loss.backward()
    oy, oh, rstd = OB.rms_norm(x, w, 1e-5, r if residual else None)
    assert np.abs(oy - y.detach().numpy()).max() < 1e-12
    gx, gw = OB.rms_norm_backward(gy, oh, rstd, w, gh if residual else None)
    assert np.abs(gx - x.grad.numpy()).max() < 1e-12
    assert np.abs(gw - w.grad.numpy()).max() < 1e-11
    if residual:
        assert np.abs(gx - r.grad.numpy()).max() < 1e-12


def test_norm_gradient_matches_differences():
    rng = np.random.default_rng(5)
    x, gy = rng.standard_normal((2, 3, 9))
    w = rng.standard_normal(9)
    _, h, rstd = OB.rms_norm(x, w, 1e-6)
    gx, gw = OB.rms_norm_backward(gy, h, rstd, w)
    e = 1e-6
    for at in np.ndindex(3, 9):
        d = np.zeros_like(x)
        d[at] = e
        f = [(OB.rms_norm(x + s * d, w, 1e-6)[0] * gy).sum() for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * e) - gx[at]) < 1e-7
    for c in range(9):
        d = np.zeros(9)
        d[c] = e
        f = [(OB.rms_norm(x, w + s * d, 1e-6)[0] * gy).sum() for s in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * e) - gw[c]) < 1e-7


# --- 8 bits ---------------------------------------------------------------------

def test_e4m3_values_and_rounding_match_torch():
    bits = torch.arange(256, dtype=torch.uint8)
    want = bits.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OB.e4m3_values(), want, equal_nan=True)
    v = OB.e4m3_values()[:127]
    mids = (v[1:] + v[:-1]) / 2                       # every tie
    rng = np.random.default_rng(6)
    x = np.concatenate([v, mids, -mids, np.nextafter(mids, 0), np.nextafter(mids, 500),
                        rng.uniform(-448, 448, 4000), rng.normal(size=4000) * 0.01])
    x = x.astype(np.float32)
    got = OB.round_e4m3(x)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32])
def test_saved_values_are_within_half_a_step(fmt, group):
    rng = np.random.default_rng(7)
    x = (rng.standard_normal((5, 77)) * np.exp(rng.normal(size=77))).astype(np.float32)
    codes, scales = OB.save8(x, fmt, group)
    assert scales.shape == (5, -(-77 // group) if group else 1)
    back = OB.load8(codes, scales, group)
    s = np.repeat(scales, group or 77, axis=1)[:, :77].astype(np.float64)
    if fmt == "int8":
        assert codes.min() >= -127 and np.abs(back - x).max() <= 0.5 * s.max() * (1 + 1e-5)
        assert (np.abs(back - x) <= 0.5 * s * (1 + 1e-5)).all()
    else:
        assert (np.abs(back - x) <= np.maximum(np.abs(x) / 16, s * 2.0 ** -10) * (1 + 1e-5)).all()
    # the largest of a group keeps its value up to the scale's rounding
    top = np.abs(x).argmax()
    assert math.isclose(back.flat[top], float(x.flat[top]), rel_tol=1e-6)


def test_saved_zeros_and_non_finite_groups():
    x = np.zeros((2, 70), dtype=np.float32)
    x[0, 3] = 2.0
    x[1, 40] = np.inf
    x[1, 65] = np.nan
    for fmt in ("int8", "e4m3"):
        codes, scales = OB.save8(x, fmt, 32)
        back = OB.load8(codes, scales, 32)
        assert back[0, 3] == pytest.approx(2.0) and np.count_nonzero(back[0]) == 1
        assert (back[1, :32] == 0).all() and np.isnan(back[1, 32:]).all()
        assert scales[0, 1] == np.float32(2.0 ** -126)
