"""Pins of the generation oracle against independent routines: torch's E4M3
conversion and SDPA in float64, hand-worked quantisation and verification."""
import numpy as np
import pytest
import torch

from oracle import generate_oracle as G


def test_e4m3_table_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(G.e4m3_table(), want)


@pytest.mark.parametrize("top,e", [(448, 0), (449, 1), (1.0, -8), (1.75, -8), (1.76, -7),
                                   (0, -127), (2.0 ** -133, -127), (2.0 ** -119, -127),
                                   (3.3e38, 120)])
def test_scale_is_the_smallest_that_fits(top, e):
    x = np.zeros(64)
    x[5] = top
    v, s = G.quantise(x)
    assert s[0] == e + 127 and s[1] == 0
    assert abs(v[5] - top) <= top / 16


def test_codes_round_as_torch_rounds():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((50, 96))).to(torch.bfloat16)
    v, s = G.quantise(x.double().numpy())
    e = np.repeat(s.astype(float) - 127, 32, -1)
    want = torch.from_numpy(x.double().numpy() / np.exp2(e)).float().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(v, want.double().numpy() * np.exp2(e))


def test_nan_and_infinity_become_nan():
    x = np.ones(32)
    x[3], x[4] = np.inf, np.nan
    v, s = G.quantise(x)
    assert np.isnan(v[[3, 4]]).all() and (np.delete(v, [3, 4]) == 1).all() and s[0] == 127 - 8


@pytest.mark.parametrize("causal", [False, True])
def test_prefix_attention_is_sdpa_over_the_joined_keys(causal):
    rng = np.random.default_rng(1)
    B, n, Lp, S, Hq, Hkv, d = 3, 4, 6, 5, 4, 2, 8
    q, ko, vo = (rng.standard_normal((B, m, h, d)) for m, h in ((n, Hq), (S, Hkv), (S, Hkv)))
    kp, vp = rng.standard_normal((2, Lp, Hkv, d))
    lens = [0, 3, 5]
    O, Z, A, _ = G.prefix_attention(q, kp, vp, ko, vo, lens, causal, 0.4)
    assert (A >= np.abs(O) - 1e-12).all()
    for b, c in enumerate(lens):
        k = np.concatenate([kp, ko[b, :c]]).repeat(Hq // Hkv, 1)
        v = np.concatenate([vp, vo[b, :c]]).repeat(Hq // Hkv, 1)
        mask = torch.ones(n, Lp + c, dtype=torch.bool)
        if causal:
            mask[:, Lp:] = torch.ones(n, c).tril(c - n).bool()
        t = [torch.from_numpy(x).transpose(0, 1) for x in (q[b], k, v)]
        want = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=mask, scale=0.4)
        np.testing.assert_allclose(O[b], want.transpose(0, 1).numpy(), atol=1e-12)
        s = (t[0] @ t[1].transpose(1, 2) * 0.4).masked_fill(~mask, -np.inf)
        np.testing.assert_allclose(Z[b], torch.logsumexp(s, -1).numpy(), atol=1e-12)


def test_a_query_without_keys():
    z = np.zeros
    O, Z, _, _ = G.prefix_attention(np.ones((1, 3, 1, 4)), z((0, 1, 4)), z((0, 1, 4)),
                                    np.ones((1, 2, 1, 4)), np.ones((1, 2, 1, 4)), [1], True, 1.0)
    assert (O[0, :2] == 0).all() and np.isneginf(Z[0, 0, :2]).all() and Z[0, 0, 2] == 4.0


def test_verification_by_hand():
    p = np.array([[.5, .5, 0], [.25, .25, .5], [0, 1, 0]], np.float32)
    q = np.array([[.25, .75, 0], [.75, .25, 0]], np.float32)
    # u q < p: .99 x .25 < .5; then .5 x .75 = .375 >= .25 fails; residual is all on token 2
    assert G.draft_verify(p, q, [0, 0], [.99, .5], .3, 2) == (1, [0, 2, -1])
    # equality is not acceptance: 1/3 does not divide, use u = 1/2, q = 1/2, p = 1/4
    p2 = np.array([[.25, .75], [.5, .5]], np.float32)
    q2 = np.array([[.5, .5]], np.float32)
    assert G.draft_verify(p2, q2, [0], [.5], 0, 1) == (0, [1, -1])
    # all accepted: the next token is drawn from the last row
    assert G.draft_verify(p, q, [0, 1], [.1, .1], .9, 2) == (2, [0, 1, 1])
    # a shorter draft draws from its own row; r exactly on a border takes the next token
    assert G.draft_verify(p, q, [0, 1], [.1, .1], .5, 0) == (0, [1, -1, -1])
    # p <= q everywhere after a rejection: p itself
    same = np.array([[.5, .5], [1, 0]], np.float32)
    assert G.draft_verify(same, same[:1], [5], [0.], .6, 1) == (0, [1, -1])
    assert G.draft_verify(np.zeros((1, 3), np.float32), np.zeros((0, 3)), [], [], .5, 0) == (0, [-1])


def test_accepted_and_resampled_tokens_follow_the_target():
    """Over draws of u, r and the draft, the first token has the target's
    distribution, whatever the drafter's: a grid of u and r instead of chance."""
    p = np.array([[.5, .125, .375], [1, 0, 0]], np.float32)
    q = np.array([[.25, .5, .25]], np.float32)
    got = np.zeros(3)
    n = 64
    for x in range(3):
        for i in range(n):
            u = (i + .5) / n
            for j in range(8):
                a, out = G.draft_verify(p, q, [x], [u], (j + .5) / 8, 1)
                got[out[0]] += q[0, x] / (n * 8)
    np.testing.assert_allclose(got, p[0], atol=1.0 / n)
