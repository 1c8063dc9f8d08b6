"""Pins of the float64 oracle of rotary positions and of attention over a paged
cache, each against something that shares no formula with it."""
import math

import numpy as np
import pytest
import torch

from oracle import generate_oracle as O


def test_angles_are_exact_at_far_positions():
    """Small positions against the plain product; far ones by the sum of angles:
    t(2p) = 2 t(p) and t(p + r) = t(p) + t(r) modulo a turn."""
    freq = [1.0, 0.3, 1e-6, 3e5, -0.7]
    pos = [0, 1, 5, 1000]
    two = 2 * math.pi
    want = np.array([[math.fmod(p * f, two) % two for f in freq] for p in pos])
    got = O.angles(pos, freq)
    diff = np.abs(got - want)
    assert np.minimum(diff, two - diff).max() < 1e-6     # (3e5 x 1000 has an ulp of 4e-8)
    big = [2 ** 30 - 1, 2 ** 31 - 2, 2 ** 31 - 1, 1]
    t = O.angles(big, freq)

    def gap(x):
        x = np.abs(x) % two
        return np.minimum(x, two - x).max()

    assert gap(2 * t[0] - t[1]) < 1e-14
    assert gap(t[1] + t[3] - t[2]) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((5, 3, 64)), rng.uniform(0, 7, (5, 16))
    y = O.rotate(x, angle, interleaved)
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle)[:, None]
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-14)
    np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
    np.testing.assert_allclose(O.pair_size(x, 16, interleaved)[..., b],
                               np.abs(z.real * 0 + x[..., a]) + np.abs(x[..., b]))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (1, 1), (100, 2)])
def test_paged_attention_is_masked_attention(causal, window, sinks):
    """Against torch's attention in float64 with an explicit mask, the cache
    gathered by hand."""
    rng = np.random.default_rng(2)
    B, n, Hq, Hkv, d, page, per = 3, 4, 6, 2, 8, 4, 5
    pages = 20
    k, v = rng.standard_normal((2, pages, page, Hkv, d))
    q = rng.standard_normal((B, n, Hq, d))
    table = rng.permutation(pages)[:B * per].reshape(B, per)
    length = [19, 7, 4]
    got, lse, A, _ = O.paged_attention(q, k, v, table, length, page, causal, window, sinks, 0.3)
    for b in range(B):
        c = length[b]
        kb, vb = (x[table[b]].reshape(-1, Hkv, d)[:c].repeat(Hq // Hkv, 1) for x in (k, v))
        t, j = np.arange(c - n, c)[:, None], np.arange(c)[None]
        m = np.ones((n, c), bool)
        if causal:
            m = np.tril(np.ones((c, c), bool))[c - n:]
        if window:
            m &= (np.triu(np.ones((c, c), bool), 1 - window)[c - n:]) | (j < sinks)
        f = [torch.from_numpy(np.ascontiguousarray(x)).transpose(0, 1) for x in (q[b], kb, vb)]
        want = torch.nn.functional.scaled_dot_product_attention(
            *f, attn_mask=torch.from_numpy(m), scale=0.3).transpose(0, 1).numpy()
        np.testing.assert_allclose(got[b], want, atol=1e-13)
        s = np.einsum("ihd,jhd->hij", q[b], kb) * 0.3
        s[:, ~m] = -np.inf
        np.testing.assert_allclose(lse[b], np.log(np.exp(s).sum(-1)), atol=1e-13)
        assert (A[b] >= np.abs(got[b]) - 1e-12).all()


def test_rows_and_pages_that_hold_nothing():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 3, 4, 1, 8))
    q = rng.standard_normal((3, 2, 1, 8))
    table = np.array([[0, -1], [7, 1], [-5, 3]])
    o, lse, _, _ = O.paged_attention(q, k, v, table, [1, 8, 9], 4, True, 0, 0, 1.0)
    assert (o[0, 0] == 0).all() and lse[0, 0, 0] == -np.inf       # before the first key
    np.testing.assert_allclose(o[0, 1, 0], v[0, 0, 0])
    np.testing.assert_allclose(lse[1, 0, 1], np.log(np.exp(k[1, :, 0] @ q[1, 1, 0]).sum()))
    assert (o[2] == 0).all() and (lse[2] == -np.inf).all()        # no page is there
