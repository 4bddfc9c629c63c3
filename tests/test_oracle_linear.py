"""Pins of the oracle of the linear layers around the attention (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import linear as OL


# the known answers that the generator's authors publish with it
@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(counter, key, words):
    assert tuple(OL.philox(counter, key)) == words


def test_kept_share():
    """20000 draws at p = 0.3: the share is within 5 standard deviations, 0.0162."""
    k = OL.kept(20000, 0.3, seed=-5, offset=2 ** 40 + 3)
    assert abs(k.mean() - 0.7) < 0.0162
    assert OL.kept(64, 0.0, 1, 2).all() and not OL.kept(64, 1.0, 1, 2).any()
    assert (OL.kept(10, 0.5, 1, 2, first=5) == OL.kept(15, 0.5, 1, 2)[5:]).all()


def test_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = OL.e4m3_values(codes)
    finite = np.isfinite(want)
    assert (got[finite] == want[finite]).all() and finite.sum() == 254
    x = np.random.default_rng(0).standard_normal((300, 200)).astype(np.float32)
    s = OL.block_scales(x, 128, 128)
    assert s.shape == (3, 2)
    each = OL.spread(s, 128, 128, 300, 200)
    r = torch.from_numpy(x * (np.float32(1) / each)).to(torch.float8_e4m3fn).double().numpy()
    assert (OL.encode(x, each) == r).all()


def test_layer_norm_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    x, w, b, g, gh = (rng.standard_normal(s) for s in ((3, 7), 7, 7, (3, 7), (3, 7)))

    def loss(x, w, b):
        y, h, _, _ = OL.layer_norm(x, w, b, 1e-3)
        return (y * g).sum() + (h * gh).sum()

    _, h, mean, rstd = OL.layer_norm(x, w, b, 1e-3)
    got = OL.layer_norm_backward(g, h, mean, rstd, w, gh)
    for k, (t, gt) in enumerate(zip((x, w, b), got)):
        for at in np.ndindex(t.shape):
            d = np.zeros_like(t)
            d[at] = 1e-5
            args = [x, w, b]
            hi, lo = list(args), list(args)
            hi[k], lo[k] = t + d, t - d
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - gt[at]) < 1e-7
