"""The paged-cache oracle against properties that do not depend on how it is written."""
import numpy as np
import torch

from oracle import paged as P


def test_e4m3_values_are_torchs():
    t = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(P.e4m3_values(), t)


def test_nearest_is_nearest_with_ties_to_even():
    x = np.concatenate((np.linspace(0, 8, 4001), [.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0]))
    got = P.nearest(x, P.E2M1[:8])
    d = np.abs(P.E2M1[None, :8] - x[:, None])
    assert (d[np.arange(len(x)), got] == d.min(1)).all()
    assert P.nearest(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0]), P.E2M1[:8]).tolist() == [0, 2, 2, 4, 4, 6, 6]


def test_scales_match_torchs_rounding():
    x = np.random.default_rng(1).lognormal(0, 4, 5000).astype(np.float32).clip(0, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(P.nearest(x, P.e4m3_values()[:127]), want)


def test_quantised_values_are_within_half_a_step():
    """A code is off by at most half of e2m1's widest step (2) of its scale, plus what the scale's
    own rounding (2^-4 of itself) cuts off at 6."""
    x = np.random.default_rng(2).standard_normal((50, 128)).astype(np.float32)
    code, s = P.quantise_f32(x, 0.002)
    v = P.values(P.pack(code), s, 0.002)
    step = np.repeat(P.e4m3_values()[s] * 0.002, 16, -1)
    assert (np.abs(v - x) <= step * (1 + 6 / 16) + 1e-7).all()
    assert np.linalg.norm(v - x) / np.linalg.norm(x) < 0.15
    z, sz = P.quantise_f32(np.zeros((2, 32), np.float32), 1.0)
    assert not z.any() and not sz.any()


def test_rotation_keeps_lengths_and_adds_angles():
    rng = np.random.default_rng(3)
    for inter in (False, True):
        x = rng.standard_normal((3, 64))
        a, b = rng.uniform(0, 6, 16), rng.uniform(0, 6, 16)
        y = P.rotate(P.rotate(x, np.cos(a), np.sin(a), inter), np.cos(b), np.sin(b), inter)
        np.testing.assert_allclose(y, P.rotate(x, np.cos(a + b), np.sin(a + b), inter), atol=1e-12)
        np.testing.assert_allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))
        np.testing.assert_array_equal(y[:, 32:], x[:, 32:])


def test_attend_is_softmax():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((9, 64)), rng.standard_normal((9, 64))
    o, lse, _, _ = P.attend(q, k, v, 0.125, [9, 3, 0, 1])
    t = torch.from_numpy
    s = (t(q) @ t(k).T) * 0.125
    np.testing.assert_allclose(o[0], (torch.softmax(s[0], 0) @ t(v)).numpy())
    np.testing.assert_allclose(lse[1], torch.logsumexp(s[1, :3], 0).item())
    assert np.isneginf(lse[2]) and not o[2].any()
    np.testing.assert_allclose(o[3], v[0])
