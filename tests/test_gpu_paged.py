"""GPU parity of serving from the quantised paged cache (append with rotation,
attention over the pages, window and sinks) with the float64 oracle.

Tolerances, derived from the arithmetic (half a rounding step is eps / 2):
 * append: scale bytes are equal; a code stands for the rotated value to half a
   step of E4M3, plus the rotation's fp32 error, below 2^-20 (|a| + |b|) for a pair
   (two products and a sum at 2^-24 each, sine and cosine within 2^-22 with their
   argument's rounding); a rotated query to 2^-8 |y| (bf16) plus the same;
 * attention: with A = sum_j p_j |v_j|, an O element is off by at most 2^-8 A
   (P rounded to bf16 or finer) + 2^-8 |O| (O rounded to bf16) + 2^-12 A (the
   exponential's 2^-21 and the sums' 2^-24 per step), and an exponent argument x
   carries 2 d 2^-24 T from its dot product on the tensor cores, which truncate
   (T the largest scale sum |q k| of the row), so 4 d 2^-24 T A more.  LSE: 2 d
   2^-24 T + 2^-21 + 2^-22 |LSE|, and 2^-24 for each of at most 2^8 sequential
   additions of a row's sum.  P below 2^-30 of a row's maximum may be held with an
   absolute error of 2^-40 of the largest |v|: 2^-40 Vmax for each key.
"""
import ctypes

import numpy as np
import pytest
import torch

from block_diffusion_lm_gb300 import csbp
from oracle import generate_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from block_diffusion_lm_gb300 import build
    build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(a, b):
    """Bit by bit (NaN included)."""
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b,
                                                                                     strict=True))


# ------------------------------------------------------------------- append
def dirty_cache(pages, page, Hkv, d, g):
    c = csbp.QuantCache(pages, page, Hkv, d)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.copy_(torch.randint(0, 120, t.shape, generator=g, device="cuda"))
    return c


def slots(table, start, count, rows, page, pages):
    """(b, i, slot) of every row that takes part; slot -1 when out of range."""
    out = []
    for b in range(table.shape[0]):
        for i in range(rows if count is None else min(rows, max(0, int(count[b])))):
            pos = int(start[b]) + i
            ok = 0 <= pos < table.shape[1] * page
            pg = int(table[b, pos // page]) if ok else -1
            out.append((b, i, pg * page + pos % page if 0 <= pg < pages else -1))
    return out


def half_step(x, e):
    """Half an E4M3 step at x under the scale 2^e."""
    a = np.maximum(np.abs(x) / np.exp2(e), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(a)) - 4 + e)


def check_append(c, before, q, out, k, v, table, start, count, freq, interleaved):
    """The cache and the rotated queries against the oracle; `before`: what the
    cache held, and `out` in rows that take no part."""
    pages, page, Hkv, d = c.k.shape
    B, rows = k.shape[:2]
    at = slots(table, start, count, rows, page, pages)
    half = len(freq)
    pos = np.array([[int(start[b]) + i for i in range(rows)] for b in range(B)]).reshape(-1)
    uniq, inv = np.unique(pos, return_inverse=True)
    angle = O.angles(uniq, freq)[inv]
    for x, codes, scales, old, old_s in ((k, c.k, c.k_scale, before[0], before[2]),
                                         (v, c.v, c.v_scale, before[1], before[3])):
        raw = f64(x).reshape(B * rows, Hkv, d)
        y, size = raw, np.zeros(raw.shape)
        if x is k:
            y = O.rotate(raw, angle, interleaved)
            size = O.pair_size(raw, half, interleaved)
            size[..., 2 * half:] = 0
        _, sb = O.quantise(y)
        want = O.dequantise(old.cpu().numpy(), old_s.cpu().numpy()).reshape(-1, Hkv, d)
        want_s = old_s.cpu().numpy().reshape(-1, Hkv, d // 32).copy()
        tol = np.zeros(want.shape)
        for b, i, s in at:
            if s >= 0:
                r = b * rows + i
                want[s], want_s[s] = np.where(np.isfinite(y[r]), y[r], np.nan), sb[r]
                e = np.repeat(sb[r].astype(int) - 127, 32, -1)
                tol[s] = half_step(y[r], e) * (1 + 1e-9) + 2.0 ** -20 * size[r]
        np.testing.assert_array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
        got = O.dequantise(codes.cpu().numpy(), scales.cpu().numpy()).reshape(want.shape)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        assert (np.abs(got - want)[fine] <= tol[fine]).all()
    if q is None:
        return
    raw = f64(q).reshape(B * rows, *q.shape[2:])
    y = O.rotate(raw, angle, interleaved).reshape(q.shape)
    size = O.pair_size(raw, half, interleaved)
    size[..., 2 * half:] = 0
    tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size.reshape(q.shape)
    got = f64(out)
    part = np.zeros((B, rows), bool)
    for b, i, _ in at:
        part[b, i] = True
    assert (np.abs(got - y)[part] <= tol[part]).all()
    if (~part).any():
        np.testing.assert_array_equal(got[~part], before[4][~part])


def freqs(rot, theta=1e4):
    return [theta ** (-2 * i / rot) for i in range(rot // 2)]


def stored(c):
    return [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]


APPENDS = [  # batch, rows, page, table entries, Hkv, d, Hq, rotary dim
    (1, 1, 1, 1, 1, 32, 1, 32), (3, 5, 16, 2, 2, 64, 14, 64), (2, 60, 64, 5, 3, 96, 0, 96),
    (4, 33, 7, 8, 8, 128, 40, 128), (1, 100, 128, 2, 1, 512, 3, 512), (65, 1, 16, 3, 4, 128, 5, 16),
    (2, 300, 48, 9, 2, 64, 4, 32), (3, 9, 4, 5, 2, 160, 2, 112), (2, 7, 16, 2, 8, 128, 32, 64),
    (700, 6, 16, 2, 1, 128, 1, 128)]


@pytest.mark.parametrize("B,rows,page,n,Hkv,d,Hq,rot", APPENDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_append(B, rows, page, n, Hkv, d, Hq, rot, interleaved, ragged):
    g = gen(B * 1000 + rows)
    pages = B * n + 2
    c = dirty_cache(pages, page, Hkv, d, g)
    before = stored(c)
    k, v = normal(g, B, rows, Hkv, d), normal(g, B, rows, Hkv, d) * 1e-3
    q = normal(g, B, rows, Hq, d) if Hq else None
    table = torch.randperm(pages, generator=g, device="cuda")[:B * n].view(B, n).int()
    start = torch.randint(0, n * page - rows + 1, (B,), generator=g, device="cuda").int()
    count = None
    if ragged:
        count = torch.randint(-1, rows + 2, (B,), generator=g, device="cuda").int()
    f = freqs(rot)
    out = c.append(k, v, table, start, count, rotary=csbp.Rotary(f, interleaved), q=q)
    assert (out is None) == (q is None)
    if q is not None:
        before.append(np.zeros(q.shape))
    check_append(c, before, q, out, k, v, table, start, count, f, interleaved)


def test_append_at_far_positions():
    """Up to the last position of 31 bits: page 2^16, 2^15 - 1 entries."""
    g = gen(3)
    c = dirty_cache(2, 65536, 1, 64, g)
    n = 32767
    table = torch.full((3, n), -1, dtype=torch.int32, device="cuda")
    table[0, -1], table[1, n // 3], table[2, 15] = 0, 1, 1
    start = i32([n * 65536 - 9, n // 3 * 65536 + 77, 15 * 65536 + 5000])
    k, v, q = (normal(g, 3, 9, h, 64) for h in (1, 1, 3))
    before = [*stored(c), None]
    f = freqs(64, 1e6)
    out = c.append(k, v, table, start, rotary=csbp.Rotary(f), q=q)
    check_append(c, before, q, out, k, v, table, start, None, f, False)


def test_append_rows_without_a_place():
    """Positions and pages out of range: nothing is written, queries are rotated
    all the same (from negative positions on)."""
    g = gen(4)
    c = dirty_cache(3, 8, 2, 64, g)
    table = i32([[0, 7], [-1, 1], [2, 5]])
    start = i32([5, 2, -3])
    k, v, q = (normal(g, 3, 8, h, 64) for h in (2, 2, 4))
    before = [*stored(c), None]
    f = freqs(48)
    out = c.append(k, v, table, start, rotary=csbp.Rotary(f), q=q)
    check_append(c, before, q, out, k, v, table, start, None, f, False)


def test_append_scales_next_to_where_they_change():
    """Groups whose largest rotated magnitude is 448 x 2^e but for a 10^-9th,
    above and below: the scale is that of the rotation itself."""
    d, n = 64, 32
    c = csbp.QuantCache(1, n, 1, d)
    x = torch.zeros((1, n, 1, d), dtype=torch.bfloat16, device="cuda")
    x[..., 0] = 2.0        # pairs (2, 0): cos t is 0.875 next to the border
    x[..., 5] = 1e-3
    want = []
    for sign in (-1, 1):
        # position p turns by p f: one frequency for each test of both sides
        f = [(np.arccos(0.875) + sign * 1e-9)] + [0.0] * 31
        c.append(x[:, :2], x[:, :2], i32([[0]]), i32([0]), rotary=csbp.Rotary(f))
        want.append(O.quantise(O.rotate(f64(x[0, :2]), O.angles([0, 1], f), False))[1])
        np.testing.assert_array_equal(c.k_scale.cpu().numpy()[0, :2], want[-1])
    assert want[0][1, 0, 0] != want[1][1, 0, 0]      # the two sides differ
    # and many random angles, near the border by chance
    g = gen(8)
    k = normal(g, 1, n, 1, d)
    k[..., ::2] *= 1e-2
    f = freqs(64, 1e6)
    before = [*stored(c)]
    v = k.clone()
    c.append(k, v, i32([[0]]), i32([0]), rotary=csbp.Rotary(f, True))
    check_append(c, before, None, None, k, v, i32([[0]]), i32([0]), None, f, True)


@pytest.mark.parametrize("B,Hkv,d", [(20000, 8, 128), (30000, 5, 64), (2000, 40, 512)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_codes_do_not_depend_on_other_heads(B, Hkv, d, interleaved):
    """A head whose scale lies next to where it changes alters no byte of the others."""
    g = gen(9)
    f = freqs(d)
    f[0] = float(np.arccos(0.875) + 1e-9)       # at position 1, (2, 0) turns to next to 1.75
    ro = csbp.Rotary(f, interleaved)
    table, start = torch.arange(B, device="cuda").int()[:, None], i32([1] * B)
    k = normal(g, B, 1, Hkv, d)
    got = []
    for first in (2.0, 1.5):
        k[:, :, 0] = 0
        k[:, :, 0, 0] = first
        c = csbp.QuantCache(B, 2, Hkv, d)
        c.append(k, k, table, start, rotary=ro)
        got.append(stored(c))
    # (in 64 bits the angle is above the border's, the magnitude below it)
    want = O.quantise(O.rotate(np.eye(1, d)[None] * 2.0, O.angles([1], f), interleaved))[1]
    assert (got[0][2][:, 1, 0, 0] == int(want[0, 0, 0])).all()
    assert same([t[:, :, 1:] for t in got[0]], [t[:, :, 1:] for t in got[1]])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_append_values_that_are_not_finite(value):
    """Both of a pair are stored as NaN, the group's scale is the others'."""
    g = gen(5)
    c = dirty_cache(2, 16, 2, 96, g)
    k, v = normal(g, 1, 20, 2, 96), normal(g, 1, 20, 2, 96)
    k[0, 3, 1, 7] = k[0, 4, 0, 90] = v[0, 5, 0, 95] = value
    k[0, 6] = value
    before = stored(c)
    f = freqs(64)
    start = i32([0])        # position 0 of the cache is row 0; angle 0 among them
    c.append(k, v, i32([[1, 0]]), start, rotary=csbp.Rotary(f))
    y = O.rotate(f64(k)[0], O.angles(range(20), f), False)
    assert not np.isfinite(y[3, 1, [7, 39]]).any()
    check_append(c, before, None, None, k, v, i32([[1, 0]]), start, None, f, False)


def test_append_strides_and_in_place():
    """Views into a packed projection, queries rotated where they lie; and an
    `out` of its own strides."""
    g = gen(6)
    B, rows, Hq, Hkv, d = 3, 7, 6, 2, 64
    packed = normal(g, B, rows + 2, Hq + 2 * Hkv + 1, d)[:, :rows]
    q, k, v = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:-1]
    table, start, count = i32([[0, 1]] * 3) + 2 * torch.arange(3, device="cuda").int()[:, None], i32(
        [0, 3, 8]), i32([7, 0, 5])
    f, ro = freqs(64), csbp.Rotary(freqs(64))
    c = dirty_cache(6, 8, Hkv, d, g)
    before = stored(c)
    room = torch.full((B, rows, Hq + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = c.append(k, v, table, start, count, rotary=ro, q=q, out=room[:, :, :Hq])
    assert out.data_ptr() == room.data_ptr()
    check_append(c, [*before, np.full(q.shape, 7.0)], q, out, k, v, table, start, count, f, False)
    assert (room[:, :, Hq:] == 7).all()
    want, kept = out.clone(), packed.clone()
    old = q.clone()
    c.append(k, v, table, start, count, rotary=ro, q=q, out=q)
    part = torch.arange(rows, device="cuda")[None] < count[:, None]
    assert torch.equal(q[part], want[part]) and torch.equal(q[~part], old[~part])
    assert torch.equal(packed[:, :, Hq:], kept[:, :, Hq:])


def test_append_without_rotation_is_write():
    g = gen(7)
    a, b = (csbp.QuantCache(9, 16, 3, 128) for _ in range(2))
    k, v = normal(g, 2, 50, 3, 128) * 3, normal(g, 2, 50, 3, 128)
    table, start = torch.randperm(9, generator=g, device="cuda")[:8].view(2, 4).int(), i32([0, 13])
    a.write(k, v, table, start)
    b.append(k, v, table, start, rotary=csbp.Rotary([0.0] * 64))
    assert same(stored(a), stored(b))


# ---------------------------------------------------------------- attention
def filled(pages, page, Hkv, d, g):
    """A cache full of keys and values, and what they stand for."""
    c = csbp.QuantCache(pages, page, Hkv, d)
    x = [normal(g, pages, page, Hkv, d) for _ in range(2)]
    table, zero = torch.arange(pages, device="cuda").int()[:, None], i32([0] * pages)
    c.write(*x, table, zero)
    return c


def values(c):
    return [O.dequantise(t.cpu().numpy(), s.cpu().numpy())
            for t, s in ((c.k, c.k_scale), (c.v, c.v_scale))]


def check_attn(out, q, c, table, length, causal, window, sinks, scale, rows=None):
    k, v = values(c)
    want, lse, A, T = O.paged_attention(f64(q), k, v, table.cpu().numpy(), length.tolist(),
                                        c.k.shape[1], causal, window, sinks, scale)
    d = q.shape[-1]
    Tr = T.transpose(0, 2, 1)[..., None]
    tiny = 2.0 ** -40 * np.nanmax(np.abs(np.where(np.isfinite(v), v, 0))) * max(length.tolist())
    tol = (2.0 ** -8 + 2.0 ** -12 + 4 * d * 2.0 ** -24 * Tr) * A + 2.0 ** -8 * np.abs(want) + tiny
    got = f64(out[0])
    worst = float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))
    assert worst <= 1, worst
    z = f64(out[1])
    none = lse == -np.inf
    np.testing.assert_array_equal(z == -np.inf, none)
    assert (got.transpose(0, 2, 1, 3)[none] == 0).all()
    tol = 2 * d * 2.0 ** -24 * T + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(none, 0, lse)) + 2.0 ** -16
    worst = float(np.max(np.abs(z[~none] - lse[~none]) / tol[~none], initial=0))
    assert worst <= 1, worst


def attn_case(B, n, per, page, Hq, Hkv, d, seed, lens=None):
    g = gen(seed)
    pages = B * per + 2
    c = filled(pages, page, Hkv, d, g)
    table = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).int()
    if lens is None:
        lens = torch.randint(0, per * page + 1, (B,), generator=g, device="cuda").tolist()
    return c, normal(g, B, n, Hq, d), table, i32(lens)


SHAPES = [  # batch, queries, table entries, page, Hq, Hkv, d, lengths
    (1, 1, 1, 1, 1, 1, 64, [1]), (1, 1, 1, 1, 1, 1, 128, [0]),
    (3, 1, 5, 16, 2, 2, 64, [80, 1, 17]), (2, 1, 9, 64, 32, 8, 128, [576, 129]),
    (4, 1, 40, 16, 8, 1, 128, [640, 0, 333, 16]), (2, 1, 3, 100, 32, 4, 128, None),
    (3, 1, 70, 7, 12, 4, 64, None), (2, 1, 11, 48, 14, 2, 64, [528, 47]),
    (2, 1, 20, 16, 9, 3, 128, None), (2, 1, 6, 16, 40, 5, 64, None),
    (1, 1, 4, 16, 24, 24, 64, [55]), (1, 1, 3, 32, 33, 11, 128, [90]),
    (2, 1, 4, 16, 64, 1, 128, None), (2, 1, 4, 16, 34, 2, 64, None),
    (5, 3, 6, 16, 8, 2, 64, [2, 96, 0, 1, 40]), (3, 9, 4, 64, 40, 8, 128, None),
    (2, 16, 8, 32, 14, 2, 64, [256, 5]), (2, 32, 5, 64, 40, 8, 128, [320, 100]),
    (1, 130, 3, 64, 4, 4, 128, [192]), (2, 70, 20, 16, 16, 2, 64, [300, 31]),
    (1, 200, 5, 64, 5, 1, 64, [260]), (17, 2, 3, 8, 3, 1, 128, None),
    (200, 1, 2, 16, 4, 2, 64, None), (1, 1, 1000, 1, 4, 1, 64, [777]),
    (900, 1, 2, 16, 4, 2, 64, None), (700, 30, 2, 16, 2, 1, 64, None),  # more than threads
    (2, 12, 4, 64, 4, 1, 128, [200, 77]), (1, 49, 4, 16, 3, 3, 64, [64]),
    (2, 129, 4, 64, 2, 1, 128, [256, 3]), (1, 257, 3, 64, 2, 2, 64, [150]),
]
MASKS = [(False, 0, 0), (True, 0, 0), (True, 37, 4), (False, 20, 0), (True, 1, 0), (False, 64, 70),
         (True, 10000, 3)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal,window,sinks", MASKS)
def test_attention(shape, causal, window, sinks):
    B, n, per, page, Hq, Hkv, d, lens = shape
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 11, lens)
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window, sinks=sinks)
    out = a.forward(q, c, table, length)
    check_attn(out, q, c, table, length, causal, window, sinks, d ** -0.5)
    # the same again, bit by bit
    assert same(a.forward(q, c, table, length), out)
    a.check()


@pytest.mark.parametrize("B,n,per,page,Hq,Hkv,d,causal,window,sinks", [
    (2, 1, 300, 64, 8, 2, 128, True, 0, 0),         # cut into many pieces
    (1, 1, 2000, 16, 4, 1, 64, False, 0, 0),
    (3, 1, 100, 64, 8, 8, 64, True, 5000, 130),
    (2, 4, 150, 64, 8, 2, 128, True, 0, 0),
    (1, 20, 200, 64, 10, 2, 64, False, 3000, 4),
    (1, 300, 60, 64, 4, 1, 128, True, 1000, 4),     # a chunk
    (1, 300, 60, 64, 4, 1, 128, True, 1000, 200),   # sinks end inside a tile
    (2, 100, 40, 48, 3, 1, 64, False, 300, 128),
    (2, 100, 40, 48, 3, 1, 64, True, 129, 127),
])
def test_attention_over_long_texts(B, n, per, page, Hq, Hkv, d, causal, window, sinks):
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 12,
                                    [per * page - 7 * b - 3 for b in range(B)])
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window, sinks=sinks)
    out = a.forward(q * 3, c, table, length)
    check_attn(out, q * 3, c, table, length, causal, window, sinks, d ** -0.5)


def test_attention_of_equal_weights_over_a_long_text():
    """q = 0 and V = 1: O is 1 and the LSE ln of the number of keys, however many
    are added up."""
    B, per, page, Hkv, d = 2, 16384, 64, 2, 64
    c = csbp.QuantCache(64, page, Hkv, d)
    one = torch.ones((64, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    c.write(one, one, torch.arange(64, device="cuda").int()[:, None], i32([0] * 64))
    table = torch.randint(0, 64, (B, per), device="cuda").int()
    length = i32([per * page, per * page - 12345])
    for n, Hq in ((1, 4), (40, 4)):
        q = torch.zeros((B, n, Hq, d), dtype=torch.bfloat16, device="cuda")
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d)
        o, lse = a.forward(q, c, table, length)
        # sums of up to 2^20 terms that lose 2^-23 each in a run of at most 2^13 steps
        assert (o.float() - 1).abs().max() <= 2.0 ** -8
        want = torch.log(length.double())[:, None, None]
        assert (lse.double() - want).abs().max() <= 2.0 ** -9


@pytest.mark.parametrize("n,Hq", [(1, 4), (6, 4), (40, 2)])
def test_accumulators_that_are_put_aside(n, Hq):
    """Texts that one CTA reads for itself, past what one accumulator takes in:
    with q = 0, O is the mean of V.  Half a rounding of O, 2^-8 of it; 2^-12 for
    sums of up to 2^11 MMAs that drop 2^-23 each.  LSE: 2^-13 for up to 2^11
    additions at 2^-24, and its own rounding."""
    B, page, per, d, n_pages = 304, 64, 10000, 64, 60
    g = gen(31)
    c = csbp.QuantCache(n_pages, page, 1, d)
    x = (torch.rand((n_pages, page, 1, d), generator=g, device="cuda") + 0.5).bfloat16()
    c.write(x, x, torch.arange(n_pages, device="cuda").int()[:, None], i32([0] * n_pages))
    table = torch.randint(0, n_pages, (B, per), generator=g, device="cuda").int()
    table[:, :per // 2] %= 7             # the first half has another mean
    length = i32([per * page - 1000 * b for b in range(B)])
    v = torch.from_numpy(values(c)[1]).cuda()[:, :, 0]       # [pages][page][d]
    a = csbp.PagedAttention(B, n, per, page, Hq, 1, d)
    q = torch.zeros((B, n, Hq, d), dtype=torch.bfloat16, device="cuda")
    o, lse = a.forward(q, c, table, length)
    a.check()
    whole = v.sum(1)
    for b in range(0, B, 19):
        m = int(length[b])
        want = whole[table[b, :m // page].long()].sum(0)
        want = (want + v[table[b, m // page].long(), :m % page].sum(0)) / m if m % page else want / m
        assert ((o[b].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want).all()
        z = float(np.log(m))
        assert (lse[b].double() - z).abs().max() <= 2.0 ** -12 + 2.0 ** -22 * z


def test_scale_bytes_at_odd_addresses():
    """A cache in storage of its user's whose scale bytes start anywhere."""
    for Hkv, n in ((4, 1), (4, 40)):
        c, q, table, length = attn_case(2, n, 5, 16, 8, Hkv, 128, 32, [80, 33])
        want = csbp.PagedAttention(2, n, 5, 16, 8, Hkv, 128).forward(q, c, table, length)
        room = [torch.zeros(t.numel() + 8, dtype=torch.uint8, device="cuda")
                for t in (c.k_scale, c.v_scale)]
        views = [r[x:x + t.numel()].view(t.shape).copy_(t)
                 for r, t, x in zip(room, (c.k_scale, c.v_scale), (1, 3))]
        odd = csbp.QuantCache(*c.k.shape, storage=(c.k, c.v, *views))
        a = csbp.PagedAttention(2, n, 5, 16, 8, Hkv, 128)
        assert same(a.forward(q, odd, table, length), want)
        k = normal(gen(33), 2, 3, Hkv, 128)
        for x in (c, odd):
            x.append(k, k, table, i32([7, 30]), rotary=csbp.Rotary(freqs(128)))
        assert same(stored(c)[2:], stored(odd)[2:])


def test_attention_strides_and_pages():
    """Queries in a packed projection; pages out of range are not read; the same
    page twice."""
    B, n, per, page, Hq, Hkv, d = 3, 2, 6, 16, 8, 2, 128
    c, _, table, _ = attn_case(B, n, per, page, Hq, Hkv, d, 13)
    g = gen(14)
    q = normal(g, B, n + 1, Hq + 3, d)[:, :n, :Hq]
    table[0, 2], table[1, 0], table[2, :] = -1, 1 << 30, -(1 << 31)
    table[1, 3] = table[1, 1]
    length = i32([90, 96, 50])
    for causal, window, sinks in MASKS:
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window,
                                sinks=sinks, scale=0.3)
        check_attn(a.forward(q, c, table, length), q, c, table, length, causal, window, sinks, 0.3)
    # lengths past the table, and below zero
    length = i32([1 << 30, -5, 97])
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d)
    check_attn(a.forward(q, c, table, length), q, c, table, i32([96, 0, 96]), False, 0, 0, d ** -0.5)


def test_attention_reads_pages_past_32_bits():
    pages, page, Hkv, d = 70000, 64, 8, 128      # 4.6e9 codes
    c = csbp.QuantCache(pages, page, Hkv, d)
    g = gen(15)
    ids = [69999, 3, 65536, 69998]
    x = [normal(g, 4, page, Hkv, d) for _ in range(2)]
    c.append(*x, i32(ids)[:, None], i32([0] * 4), rotary=csbp.Rotary([0.0] * 64))
    small = csbp.QuantCache(4, page, Hkv, d)
    small.write(*x, i32([[0], [1], [2], [3]]), i32([0] * 4))
    for n in (1, 40):
        q = normal(g, 1, n, 16, d)
        a = csbp.PagedAttention(1, n, 4, page, 16, Hkv, d)
        got = a.forward(q, c, i32([ids]), i32([250]))
        assert same(got, a.forward(q, small, i32([[0, 1, 2, 3]]), i32([250])))


@pytest.mark.parametrize("causal", [True, False])
def test_windows_next_to_31_bits(causal):
    """The longest table and the widest window that it allows, for more queries than a text
    has keys: positions run from below -1,500 on, and position less window past 32 bits."""
    n, page, per, lens = 1600, 62145, 34556, [100, 1700]
    assert 2 ** 31 - 1030 < page * per < 2 ** 31 - 1024
    c, q, table, _ = attn_case(2, n, 1, page, 1, 1, 64, 48, [0, 0])
    big = torch.full((2, per), -1, dtype=torch.int32, device="cuda")
    big[:, :1] = table
    length = i32(lens)
    small = csbp.PagedAttention(2, n, 1, page, 1, 1, 64, causal=causal)
    want = small.forward(q, c, table, length)
    check_attn(want, q, c, table, length, causal, 0, 0, 64 ** -0.5)
    for window in (page * per - 1, page * per - 400, 2 ** 31 - 1):
        a = csbp.PagedAttention(2, n, per, page, 1, 1, 64, causal=causal, window=window, sinks=3)
        assert same(a.forward(q, c, big, length), want)


# ------------------------------------- keys that are not read, not finite
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("kind", ["code", "scale"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,Hq,Hkv,causal,window,sinks,lens,where", [
    (2, 1, 4, 2, True, 0, 0, [60, 33], (1, 33)),         # just past the end
    (2, 1, 4, 2, True, 8, 4, [60, 33], (0, 30)),         # before the window
    (2, 5, 4, 2, True, 0, 0, [60, 33], (0, 58)),         # later than some queries
    (2, 5, 4, 2, True, 9, 2, [60, 33], (1, 21)),         # out of some queries' windows
    (2, 40, 4, 2, True, 0, 0, [60, 45], (0, 40)),        # the same, many rows
    (1, 40, 8, 1, True, 16, 3, [90], (0, 50)),
    (1, 40, 8, 1, False, 16, 3, [90], (0, 40)),
])
def test_keys_that_are_not_read_do_not_matter(B, n, Hq, Hkv, causal, window, sinks, lens, where, d,
                                              kind, name):
    """NaN in a key: rows that do not read it come out as without it, bit by bit;
    rows that do are NaN."""
    page, per = 16, 6
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 16, lens)
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window, sinks=sinks)
    clean = [x.clone() for x in a.forward(q, c, table, length)]
    check_attn(clean, q, c, table, length, causal, window, sinks, d ** -0.5)
    b, j = where
    pg = int(table[b, j // page])
    if kind == "code":
        getattr(c, name)[pg, j % page, 0, 5] = 0x7f
        getattr(c, name)[pg, j % page, Hkv - 1, d - 1] = 0xff
    else:
        getattr(c, name + "_scale")[pg, j % page, :, d // 32 - 1] = 255
    o, lse = a.forward(q, c, table, length)
    t = lens[b] - n + np.arange(n)
    reads = np.full(n, j < lens[b])
    if causal:
        reads &= j <= t
    if window:
        reads &= (t - j < window) | (j < sinks)
    G = Hq // Hkv
    for bb in range(B):
        for i in range(n):
            for h in range(Hq):
                bad = bb == b and reads[i] and (kind == "scale" or h // G in (0, Hkv - 1))
                x, want = o[bb, i, h], clean[0][bb, i, h]
                zx, zw = lse[bb, h, i], clean[1][bb, h, i]
                if not bad:
                    assert torch.equal(x, want) and torch.equal(zx, zw), (bb, i, h)
                elif name == "k":
                    assert x.isnan().all() and zx.isnan()
                else:
                    hit = [f for f in (5, d - 1) if kind == "code"
                           and h // G == (0 if f == 5 else Hkv - 1)]
                    hit = hit or list(range(d - 32, d))
                    nan = x.isnan().cpu().numpy()
                    assert nan[hit].all() and nan.sum() == len(hit)
                    assert torch.equal(zx, zw)


@pytest.mark.parametrize("n,Hq,Hkv,d", [(2, 8, 4, 64), (12, 8, 4, 128), (60, 8, 4, 128),
                                        (200, 4, 4, 64)])
def test_rows_do_not_depend_on_other_rows(n, Hq, Hkv, d):
    """Another query, or a key that only later queries read, changes nothing for a
    row, bit by bit: also where it changes the other rows' maxima by much."""
    B, page, per = 8, 64, 64              # several steps in a row for every CTA
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 34, [per * page] * 7 + [2000])
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    q[:, :, :, 3] = 1
    want = [x.clone() for x in a.forward(q, c, table, length)]
    for i, factor in ((1, 100.0), (n // 2, float("nan")), (n - 1, -7.0)):
        q2 = q.clone()
        q2[:, i] *= factor
        o, lse = a.forward(q2, c, table, length)
        others = [x for x in range(n) if x != i]
        assert same((o[:, others], lse[:, :, others]), (want[0][:, others], want[1][:, :, others]))
    later = 1 if n == 2 else n // 2       # a key of that query's own place
    for b in range(B):
        j = int(length[b]) - n + later
        pg = int(table[b, j // page])
        c.k_scale[pg, j % page] += 8
        c.k[pg, j % page, :, 3] = 0x7e    # 448 x the scale, where all queries are 1
        c.v_scale[pg, j % page] += 5
    o, lse = a.forward(q, c, table, length)
    assert same((o[:, :later], lse[:, :, :later]), (want[0][:, :later], want[1][:, :, :later]))
    assert not torch.equal(lse[:, :, later:], want[1][:, :, later:])


def test_values_far_apart():
    """Scales from 2^-100 to 2^100 beside one another."""
    B, n, per, page, Hq, Hkv, d = 1, 1, 8, 16, 4, 1, 64
    for n in (1, 40):
        c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 17, [128])
        g = gen(18)
        c.v_scale.copy_(torch.randint(27, 228, c.v_scale.shape, generator=g, device="cuda"))
        c.k_scale.copy_(torch.randint(100, 125, c.k_scale.shape, generator=g, device="cuda"))
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
        check_attn(a.forward(q, c, table, length), q, c, table, length, True, 0, 0, d ** -0.5)


def largest_terms(q, c, table, length, causal, window, sinks, scale):
    """Of each O element, the largest weight x scale of V's group among the keys that its
    query reads."""
    k, _ = values(c)
    page, Hkv = c.k.shape[1:3]
    scales = np.repeat(np.exp2(c.v_scale.cpu().numpy().astype(float) - 127), 32, -1)
    B, n, Hq, d = q.shape
    out = np.zeros(q.shape)
    for b in range(B):
        m = int(length[b])
        j = np.arange(m)
        at = table[b].cpu().numpy()[j // page], j % page
        for i in range(n):
            t = m - n + i
            ok = (j <= t) | (not causal)
            if window:
                ok &= (t - j < window) | (j < sinks)
            for h in range(Hq if ok.any() else 0):
                x = k[at][ok, h * Hkv // Hq] @ f64(q[b, i, h]) * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, i, h] = (w[:, None] * scales[at][ok, h * Hkv // Hq]).max(0)
    return out


def check_far(out, q, c, table, length, causal, window, sinks, scale):
    """As check_attn, but what is lost of P below f16's normal range is allowed for by the
    keys that a row reads: with p v 2^14 in units of 2^E, where E is at most 2^4 above
    (largest weight x scale) or taken from it, 2^-24 of a code up to 2^9 for each key, which
    is 2^-25 of that.  Scores are exact to their dot product's rounding, as there."""
    k, v = values(c)
    want, lse, A, T = O.paged_attention(f64(q), k, v, table.cpu().numpy(), length.tolist(),
                                        c.k.shape[1], causal, window, sinks, scale)
    d = q.shape[-1]
    M = largest_terms(q, c, table, length, causal, window, sinks, scale)
    tol = ((2.0 ** -8 + 2.0 ** -12 + 4 * d * 2.0 ** -24 * T.transpose(0, 2, 1)[..., None]) * A
           + 2.0 ** -8 * np.abs(want) + 2.0 ** -25 * M * max(length.tolist()))
    worst = float(np.max(np.abs(f64(out[0]) - want) / np.maximum(tol, 1e-300)))
    assert worst <= 1, worst
    z, none = f64(out[1]), lse == -np.inf
    np.testing.assert_array_equal(z == -np.inf, none)
    tol = 2 * d * 2.0 ** -24 * T + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(none, 0, lse)) + 2.0 ** -16
    assert (np.abs(z[~none] - lse[~none]) <= tol[~none]).all()


# query rows per KV head of up to 8, up to 16 and more
FAR = [(2, 8, 4, 64), (3, 8, 4, 128), (6, 4, 2, 128), (12, 8, 4, 64), (20, 4, 2, 128)]


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR)
@pytest.mark.parametrize("by", [16, 40, 100, 124])
def test_large_values_that_are_not_read(n, Hq, Hkv, d, by):
    """V of a key, 2^16 to 2^124 times the others', has no part in the rows that do not
    read it: drafts before it, or queries past its window."""
    B, page, per = 3, 16, 30
    lens = [470, 33, 257]
    for causal, window, sinks, back in ((True, 0, 0, 0), (True, 0, 0, n // 2), (True, 60, 3, 59),
                                        (True, 60, 3, 59 + n // 2), (False, 60, 0, 59 + n // 2)):
        c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 51, lens)
        for b in range(B):
            j = lens[b] - 1 - back
            if j >= 0:
                c.v_scale[int(table[b, j // page]), j % page, :, b % (d // 32)] += by
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window, sinks=sinks)
        check_far(a.forward(q, c, table, length), q, c, table, length, causal, window, sinks,
                  d ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR)
@pytest.mark.parametrize("by", [30, 45, 100])
def test_large_values_of_next_to_no_weight(n, Hq, Hkv, d, by):
    """V of a key, 2^30 to 2^100 times the others', with a weight of 2^-80 and less: the
    others are what O is made of, or both, or the key alone."""
    B, page, per = 2, 16, 20
    lens = [300, 130]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 52, lens)
    q[..., 3] = 8
    for b in range(B):
        for j in (0, 77, lens[b] - n):
            at = int(table[b, j // page]), j % page
            c.k[at][:] = 0
            c.k[at][:, 3] = 0xfe                      # -448
            c.k_scale[at][:, 0] = 127 - 6             # -7: a score of -56
            c.v_scale[at][:, 1] += by
    for causal in (True, False):
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, scale=1.0)
        check_far(a.forward(q, c, table, length), q, c, table, length, causal, 0, 0, 1.0)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR)
def test_values_far_apart_in_every_step(n, Hq, Hkv, d):
    """V's scales anywhere from 2^-100 to 2^100 and groups of zeros among them, in texts
    of many steps for each warp: against what each row's own keys allow."""
    B, page, per, pages = 24, 64, 256, 50
    g = gen(54)
    c = filled(pages, page, Hkv, d, g)
    table = torch.randint(0, pages, (B, per), generator=g, device="cuda").int()
    length = i32([page * per - 100 * b for b in range(B - 1)] + [n // 2])
    q = normal(g, B, n, Hq, d)
    c.v_scale.copy_(torch.randint(27, 228, c.v_scale.shape, generator=g, device="cuda"))
    empty = torch.rand(c.v_scale.shape, generator=g, device="cuda") < 0.1
    c.v_scale[empty] = 0
    c.v.view(*c.v_scale.shape, 32)[empty] = 0
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    out = a.forward(q, c, table, length)
    assert same(a.forward(q, c, table, length), out)
    for b in (0, 11, B - 1):
        for i in {0, n // 2, n - 1}:                 # a row as if it were alone
            at = slice(b, b + 1), slice(i, i + 1)
            few = out[0][at], out[1][at[0], :, at[1]]
            check_far(few, q[at], c, table[at[0]], (length[at[0]] - n + 1 + i).clamp(min=0), True,
                      0, 0, d ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR)
@pytest.mark.parametrize("kind", ["code", "scale"])
def test_nan_beside_values_far_apart(n, Hq, Hkv, d, kind):
    """A key with NaN in V among others whose values lie 2^60 apart: NaN for the rows that
    read it, in its features; the others as without it."""
    B, page, per = 2, 16, 20
    lens = [300, 130]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 55, lens)
    for b in range(B):
        for j, by in ((lens[b] - n, 60), (lens[b] - n - 2, 30), (lens[b] - n - 5, 90), (3, 70)):
            c.v_scale[int(table[b, j // page]), j % page, :, ::2] += by
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    clean = [x.clone() for x in a.forward(q, c, table, length)]
    bad = torch.zeros(clean[0].shape, dtype=torch.bool, device="cuda")
    for b in range(B):
        j = lens[b] - n + n // 2
        at = int(table[b, j // page]), j % page
        if kind == "code":
            c.v[at][:, 5] = 0x7f
            bad[b, n // 2:, :, 5] = True
        else:
            c.v_scale[at][:, 0] = 255
            bad[b, n // 2:, :, :32] = True
    o, lse = a.forward(q, c, table, length)
    assert torch.equal(lse, clean[1]) or kind == "scale"
    assert torch.equal(o.isnan(), bad)
    if kind == "code":
        assert torch.equal(torch.where(bad, 0, o), torch.where(bad, 0, clean[0]))
    i = n // 2
    check_far((o[:, :i].contiguous(), lse[:, :, :i].contiguous()), q[:, :i], c, table,
              length - n + i, True, 0, 0, d ** -0.5)


# more rows: 64, 160 and 256 + 44 per KV head
FAR_TILES = [(32, 4, 2, 64), (40, 8, 2, 128), (100, 6, 2, 64)]


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR_TILES)
@pytest.mark.parametrize("name,by", [("v", 16), ("v", 40), ("v", 124), ("k", 30), ("k", 100)])
def test_large_keys_and_values_that_are_not_read_by_many_rows(n, Hq, Hkv, d, name, by):
    """K or V of a key, 2^16 to 2^124 times the others', has no part in the rows that do
    not read it."""
    B, page, per = 3, 16, 30
    lens = [470, n - 3, 257]
    for causal, window, back in ((True, 0, 0), (True, 0, n // 2), (True, 60, 59 + n // 2),
                                 (False, 60, 59 + n // 2)):
        c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 56, lens)
        rows = np.ones((B, n), bool)             # those that do not read it
        for b in range(B):
            j, t = lens[b] - 1 - back, lens[b] - n + np.arange(n)
            if j >= 0:
                getattr(c, name + "_scale")[int(table[b, j // page]), j % page, :, b % (d // 32)] += by
                rows[b] = ((j > t) & causal) | ((t - j >= window) & bool(window))
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window)
        o, lse = a.forward(q, c, table, length)
        a.check()
        if name == "v":
            check_far((o, lse), q, c, table, length, causal, window, 0, d ** -0.5)
            continue
        # (a row that reads it has a score of 2^30 and more: all the others are nothing)
        k, v = values(c)
        want, z, A, T = O.paged_attention(f64(q), k, v, table.cpu().numpy(), lens, page, causal,
                                          window, 0, d ** -0.5)
        tol = ((2.0 ** -8 + 2.0 ** -12 + 4 * d * 2.0 ** -24 * T.transpose(0, 2, 1)[..., None]) * A
               + 2.0 ** -8 * np.abs(want))
        assert rows.any() and (np.abs(f64(o) - want)[rows] <= tol[rows]).all()
        z, T, got = (x.transpose(0, 2, 1)[rows] for x in (z, T, f64(lse)))
        none = z == -np.inf
        np.testing.assert_array_equal(got == -np.inf, none)
        tol = 2 * d * 2.0 ** -24 * T[~none] + 2.0 ** -15
        assert (np.abs(got[~none] - z[~none]) <= tol).all()


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR_TILES + FAR[1:4])
def test_large_keys_that_queries_are_zero_for(n, Hq, Hkv, d):
    """K of a key, 2^60 times the others', in a feature where all queries are 0: its score
    is 0, the others' are theirs."""
    B, page, per = 2, 16, 30
    lens = [470, 300]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 57, lens)
    q[..., 7] = 0
    for b in range(B):
        for j in (100, lens[b] - n):
            at = int(table[b, j // page]), j % page
            c.k[at][:, :32] = 0
            c.k[at][:, 7] = 0x7e
            c.k_scale[at][:, 0] = 127 + 50
    for causal in (True, False):
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal)
        check_far(a.forward(q, c, table, length), q, c, table, length, causal, 0, 0, d ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR_TILES)
@pytest.mark.parametrize("by", [30, 100])
def test_large_values_of_next_to_no_weight_for_many_rows(n, Hq, Hkv, d, by):
    """As for few rows; in a text that is cut among CTAs, in one piece of it."""
    B, page, per = 2, 64, 40
    lens = [2500, 130]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 58, lens)
    q[..., 3] = 8
    for b in range(B):
        j = lens[b] * 2 // 3
        at = int(table[b, j // page]), j % page
        c.k[at][:] = 0
        c.k[at][:, 3] = 0xfe
        c.k_scale[at][:, 0] = 127 - 6
        c.v_scale[at][:, 1] += by
    for causal in (True, False):
        a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, scale=1.0)
        check_far(a.forward(q, c, table, length), q, c, table, length, causal, 0, 0, 1.0)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR_TILES)
def test_scales_far_apart_and_near_again(n, Hq, Hkv, d):
    """V's and K's scales anywhere, groups of zeros and NaN among them, for some sequences
    of a call and not for others; the next call on the same handle finds them near."""
    B, page, per = 6, 64, 20
    lens = [1280, 1000, 64, 700, 1279, 0]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 59, lens)
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    want = [x.clone() for x in a.forward(q, c, table, length)]
    old = stored(c)
    g = gen(60)
    for b in (0, 3, 4):
        pages = table[b].long()
        for name, lo, hi in (("k_scale", 100, 123), ("v_scale", 27, 228)):
            t = getattr(c, name)
            t[pages] = torch.randint(lo, hi, t[pages].shape, generator=g, device="cuda").byte()
        empty = torch.rand(c.v_scale[pages].shape, generator=g, device="cuda") < 0.1
        c.v_scale[pages] = torch.where(empty, 0, c.v_scale[pages])
        codes = c.v[pages].view(*empty.shape, 32)
        c.v[pages] = torch.where(empty[..., None], 0, codes).view(c.v[pages].shape)
    o, lse = a.forward(q, c, table, length)
    assert same(a.forward(q, c, table, length), (o, lse))
    near = [1, 2, 5]
    assert same((o[near], lse[near]), (want[0][near], want[1][near]))
    for b in (0, 3, 4):
        for i in (0, n // 2, n - 1):
            at = slice(b, b + 1), slice(i, i + 1)
            check_far((o[at], lse[at[0], :, at[1]]), q[at], c, table[at[0]],
                      length[at[0]] - n + 1 + i, True, 0, 0, d ** -0.5)
    # NaN beside them
    clean = [o.clone(), lse.clone()]
    bad = torch.zeros(o.shape, dtype=torch.bool, device="cuda")
    for b in (0, 1, 3, 4):
        j = lens[b] - n // 2
        c.v[int(table[b, j // page]), j % page, :, 9] = 0xff
        bad[b, n - n // 2:, :, 9] = True
    o, lse = a.forward(q, c, table, length)
    assert torch.equal(lse, clean[1]) and torch.equal(o.isnan(), bad)
    assert torch.equal(torch.where(bad, 0, o), torch.where(bad, 0, clean[0]))
    for t, x in zip((c.k, c.v, c.k_scale, c.v_scale), old):
        t.copy_(x)
    assert same(a.forward(q, c, table, length), want)


@pytest.mark.parametrize("n,Hq,Hkv,d", [(1, 4, 1, 64), (1, 8, 8, 128), (3, 8, 2, 128), (24, 4, 2, 64),
                                        (32, 4, 2, 128), (110, 4, 2, 64)])
def test_weights_have_eleven_bits(n, Hq, Hkv, d):
    """V of one sign in half the features, of both in the others, where O is small beside
    A = sum p |v|: P as f16 costs 2^-11 A, the exponential, the sums and weights below f16's
    normal range (2^-25 of a row's largest) 2^-13 A more, and O's own rounding 2^-8 of it."""
    B, page, per = 3, 16, 40
    lens = [640, 37, 333]
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 62, lens)
    c.v[..., ::2] &= 0x7f
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    o, lse = a.forward(q, c, table, length)
    k, v = values(c)
    want, _, A, T = O.paged_attention(f64(q), k, v, table.cpu().numpy(), lens, page, True, 0, 0,
                                      d ** -0.5)
    tol = ((2.0 ** -11 + 2.0 ** -13 + 4 * d * 2.0 ** -24 * T.transpose(0, 2, 1)[..., None]) * A
           + 2.0 ** -8 * np.abs(want))
    assert (np.abs(f64(o) - want) <= tol).all()


@pytest.mark.parametrize("n", [1, 3, 12, 40])
def test_values_far_apart_under_scale_bytes_anywhere(n):
    """Scale bytes that are not loaded in words: at odd addresses, or of 3 heads of 64."""
    for Hkv, d in ((4, 128), (3, 64)):
        c, q, table, length = attn_case(3, n, 20, 16, 2 * Hkv, Hkv, d, 63, [320, 33, 200])
        g = gen(64)
        c.v_scale.copy_(torch.randint(60, 190, c.v_scale.shape, generator=g, device="cuda"))
        a = csbp.PagedAttention(3, n, 20, 16, 2 * Hkv, Hkv, d, causal=True)
        want = [x.clone() for x in a.forward(q, c, table, length)]
        check_far(want, q, c, table, length, True, 0, 0, d ** -0.5)
        room = [torch.zeros(t.numel() + 8, dtype=torch.uint8, device="cuda")
                for t in (c.k_scale, c.v_scale)]
        views = [r[x:x + t.numel()].view(t.shape).copy_(t)
                 for r, t, x in zip(room, (c.k_scale, c.v_scale), (1, 3))]
        odd = csbp.QuantCache(*c.k.shape, storage=(c.k, c.v, *views))
        assert same(a.forward(q, odd, table, length), want)


@pytest.mark.parametrize("n,Hq,Hkv,d", FAR_TILES + FAR)
def test_values_that_grow_step_by_step(n, Hq, Hkv, d):
    """V's scales rise by 2^40 every 256 keys, of keys without weight: what the first keys
    gave remains, in texts that a CTA takes as wholes."""
    B, page, per = 304, 64, 20
    c = filled(per, page, Hkv, d, gen(65))
    q = normal(gen(66), B, n, Hq, d)
    q[..., 3] = 8
    table = torch.arange(per, device="cuda").int().repeat(B, 1)
    length = i32([1280 - b % 7 for b in range(B)])
    c.v_scale.fill_(40)
    c.k[4:] = 0
    c.k[4:, :, :, 3] = 0xfe
    c.k_scale[4:, :, :, 0] = 127 - 4                  # -28: a score of -224
    for pg in range(4, per):
        c.v_scale[pg] = 40 + 40 * (pg // 4)
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, scale=1.0)
    o, lse = a.forward(q, c, table, length)
    for b in (0, 150, 303):
        at = slice(b, b + 1)
        check_far((o[at], lse[at]), q[at], c, table[at], length[at], False, 0, 0, 1.0)


def zeros_of_large_scale(c, name="v"):
    """Every 9th token of the cache: codes of 0 under a scale 2^60 above the others'.  It
    alters no value, only the path that is taken."""
    pages, page = c.k.shape[:2]
    at = (torch.arange(pages * page, device="cuda").view(pages, page) * 7 % 9 == 0)
    getattr(c, name)[at] = 0
    getattr(c, name + "_scale")[at] += 60


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal,window,sinks", MASKS)
def test_attention_where_scales_lie_far_apart(shape, causal, window, sinks):
    """All shapes and masks in the paths of scales far apart; V's for one half, K's for the
    other, where queries and pages are missing or not finite, too."""
    B, n, per, page, Hq, Hkv, d, lens = shape
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 71, lens)
    zeros_of_large_scale(c)
    table[::2, per // 2] = -1
    wide = normal(gen(72), B, n, Hq + 1, d)[:, :, :Hq]
    wide.copy_(q)
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=causal, window=window, sinks=sinks)
    out = a.forward(wide, c, table, length)
    check_attn(out, q, c, table, length, causal, window, sinks, d ** -0.5)
    assert same(a.forward(q, c, table, length), out)
    a.check()
    c2, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 73, lens)
    zeros_of_large_scale(c2, "k")
    out = a.forward(q, c2, table, length)
    check_attn(out, q, c2, table, length, causal, window, sinks, d ** -0.5)
    if n > 1:        # a query that is not finite has no part in the others
        bad = q.clone()
        bad[:, n // 2] = float("nan")
        o, lse = a.forward(bad, c2, table, length)
        others = [i for i in range(n) if i != n // 2]
        assert same((o[:, others], lse[:, :, others]), (out[0][:, others], out[1][:, :, others]))


@pytest.mark.parametrize("n", [4, 80])
def test_captured_call_meets_scales_far_apart(n):
    """One graph, replayed with scales that are near, far apart and near again."""
    c, q, table, length = attn_case(3, n, 12, 64, 4, 2, 128, 74, [768, 100, 500])
    far = csbp.QuantCache(*c.k.shape, storage=[t.clone() for t in stored(c)])
    zeros_of_large_scale(far)
    a = csbp.PagedAttention(3, n, 12, 64, 4, 2, 128, causal=True)
    want = [[x.clone() for x in a.forward(q, y, table, length)] for y in (c, far)]
    near = stored(c)
    out = a.alloc_outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward(q, c, table, length, out=out)
    for k in (0, 1, 1, 0):
        for t, x in zip((c.k, c.v, c.k_scale, c.v_scale), (near, stored(far))[k]):
            t.copy_(x)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[k])


def test_sums_in_parts_over_a_long_text():
    """q = 0 over a million keys of which some take the paths of scales far apart: O is the
    mean of V, to 2^-8 for its rounding and 2^-10 for the sums, LSE the number's ln."""
    page, per, Hkv, d = 64, 16384, 1, 64
    c = csbp.QuantCache(64, page, Hkv, d)
    x = (torch.rand((64, page, Hkv, d), generator=gen(75), device="cuda") + 0.5).bfloat16()
    c.write(x, x, torch.arange(64, device="cuda").int()[:, None], i32([0] * 64))
    zeros_of_large_scale(c)
    table = torch.randint(0, 64, (2, per), generator=gen(76), device="cuda").int()
    length = i32([per * page, 300000])
    v = torch.from_numpy(values(c)[1]).cuda()[:, :, 0]
    for n in (1, 50):
        a = csbp.PagedAttention(2, n, per, page, 1, Hkv, d)
        o, lse = a.forward(torch.zeros((2, n, 1, d), dtype=torch.bfloat16, device="cuda"), c, table,
                           length)
        a.check()
        for b in range(2):
            m = int(length[b])
            want = v.sum(1)[table[b, :m // page].long()].sum(0)
            want = (want + v[table[b, -(-m // page) - 1].long(), :m % page].sum(0)) / m
            assert ((o[b].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all()
            assert (lse[b].double() - np.log(m)).abs().max() <= 2.0 ** -10


def test_queries_far_apart():
    """Rows of very large and very small queries."""
    B, n, per, page, Hq, Hkv, d = 1, 8, 4, 16, 4, 2, 128
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 19, [64])
    q = q * torch.exp2(torch.arange(-100, 28, 4, device="cuda").float()).view(1, n, Hq, 1)
    q = q.bfloat16()
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, scale=2.0 ** -20)
    check_attn(a.forward(q, c, table, length), q, c, table, length, False, 0, 0, 2.0 ** -20)
    n = 30                               # 60 rows, on the tiles
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 19, [64])
    q = (q * torch.exp2(torch.arange(-100, 20, 1, device="cuda").float()).view(1, n, Hq, 1)).bfloat16()
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, scale=2.0 ** -20)
    check_attn(a.forward(q, c, table, length), q, c, table, length, False, 0, 0, 2.0 ** -20)
    c.k_scale.sub_(60)
    q2 = (q.float() * 2.0 ** 60).bfloat16()
    check_attn(a.forward(q2, c, table, length), q2, c, table, length, False, 0, 0, 2.0 ** -20)


# ------------------------------------------ pieces of several tiles of keys
@pytest.mark.parametrize("n,Hq,Hkv,d", [(32, 16, 8, 64), (30, 16, 4, 128)])
def test_queries_of_other_sizes_in_tiles_taken_in_turn(n, Hq, Hkv, d):
    """64 and 120 rows per KV head, whose tiles of keys go to two halves of a CTA in
    turn, four and more to a CTA: each row under its own power of two."""
    B, page, per = 8, 64, 16
    c, q, table, length = attn_case(B, n, per, page, Hq, Hkv, d, 41,
                                    [1024, 1000, 900, 1, 129, 128, 513, 1023])
    q = q * torch.exp2((torch.arange(n * Hq, device="cuda") % 11 - 8.0)).view(1, n, Hq, 1).bfloat16()
    a = csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, causal=True)
    out = a.forward(q, c, table, length)
    check_attn(out, q, c, table, length, True, 0, 0, d ** -0.5)
    assert same(a.forward(q, c, table, length), out)


@pytest.mark.parametrize("n,G,d,causal,lens", [
    (300, 1, 64, True, [513, 700, 385, 897, 640, 900]),   # 256 + 44 rows
    (92, 4, 128, False, [300, 513, 1000, 129, 640, 256]),  # 256 + 112
    (257, 1, 128, True, [200, 1000, 513, 650, 400, 900]),  # 256 + 1; rows without a key
    (200, 3, 64, True, [800, 100, 300, 1000, 500, 129]),   # 512 + 88
])
def test_pairs_of_row_tiles_before_a_single_one(n, G, d, causal, lens):
    """Rows that are some pairs of row tiles of 128 and a single one at the end, with so
    many heads that a CTA goes from the one to the other with several tiles of keys in
    each.  The heads hold the same and have the same scores, so their results differ by
    what the cuts of their keys change: at most half a step of O (2^-8 of it) and 2^-11 of
    the largest |v| (P's rounding and the exponential) each; LSE by the sums' 2^-18."""
    B, page, per, Hkv = 6, 64, 16, 19
    c, q, table, length = attn_case(B, n, per, page, G, 1, d, 42, lens)
    many = csbp.QuantCache(c.k.shape[0], page, Hkv, d)
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(many, name).copy_(getattr(c, name).expand_as(getattr(many, name)))
    qm = q.repeat(1, 1, Hkv, 1)
    a = csbp.PagedAttention(B, n, per, page, G * Hkv, Hkv, d, causal=causal)
    o, lse = a.forward(qm, many, table, length)
    a.check()
    assert same(a.forward(qm, many, table, length), (o, lse))
    # the first head against the oracle, the others against it
    check_attn((o[:, :, :G], lse[:, :G]), q, c, table, length, causal, 0, 0, d ** -0.5)
    k, v = values(c)
    tol = 2.0 ** -7 * o[:, :, :G].float().abs() + 2.0 ** -10 * float(np.abs(v).max())
    for h in range(1, Hkv):
        assert ((o[:, :, h * G:h * G + G].float() - o[:, :, :G].float()).abs() <= tol).all(), h
        z = lse[:, h * G:h * G + G]
        assert torch.equal(z.isinf(), lse[:, :G].isinf())
        assert ((z - lse[:, :G]).nan_to_num(0.0).abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("n,G,d", [(32, 2, 64), (40, 3, 128), (64, 2, 128), (150, 1, 64),
                                   (300, 1, 64), (200, 3, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_at_the_end_of_a_text(n, G, d, causal):
    """NaN in V's codes and scale bytes in the last, partial tile of one, two, three and
    four: single row tiles, pairs, and both.  Rows that read the key are NaN in its features
    and nowhere else, the others and all LSE stay as they are, bit by bit."""
    page, per, Hkv = 16, 32, 19
    lens = [70, 129, 200, 250, 300, 383, 400, 500, 510, 180, 255, 140]
    B = len(lens)
    c, q, table, length = attn_case(B, n, per, page, G * Hkv, Hkv, d, 43, lens)
    a = csbp.PagedAttention(B, n, per, page, G * Hkv, Hkv, d, causal=causal)
    clean = [x.clone() for x in a.forward(q, c, table, length)]
    bad = torch.zeros((B, n, G * Hkv, d), dtype=torch.bool, device="cuda")
    for b, m in enumerate(lens):
        j = m - 1 - b % 4 * (n // 5 if causal else 1)     # in the last tile of keys, as a rule
        pg = int(table[b, j // page])
        for h in range(b % 2, Hkv, 2):
            if h % 4 < 2:
                c.v[pg, j % page, h, 7 * h % d] = 0xff
                hit = slice(7 * h % d, 7 * h % d + 1)
            else:
                e = h % (d // 32)
                c.v_scale[pg, j % page, h, e] = 255
                hit = slice(32 * e, 32 * e + 32)
            first = max(0, j - m + n) if causal else 0    # the first query that reads it
            if j < 0:                                     # (a place behind the text: none)
                first = n
            bad[b, first:, h * G:h * G + G, hit] = True
    for _ in range(3):
        o, lse = a.forward(q, c, table, length)
        assert torch.equal(lse, clean[1])
        assert torch.equal(o.isnan(), bad)
        assert torch.equal(torch.where(bad, 0, o), torch.where(bad, 0, clean[0]))
    a.check()


def test_nan_in_tiles_of_all_kinds():
    """NaN in V at a window's edges, among sinks, beside a page that is not there, and in
    tiles that all rows read: NaN for the rows that read it, the same as before for the
    others."""
    page, per, Hkv, G, d, n = 16, 80, 19, 1, 64, 100
    B, m, window, sinks = 3, 1270, 700, 200
    t = m - n + np.arange(n)
    for causal in (True, False):
        for j in (3, 198, 199, 460, 471, 490, 569, 570, 571, 700, 900, 1000, 1169, 1170, 1200, 1269):
            c, q, table, length = attn_case(B, n, per, page, G * Hkv, Hkv, d, 44, [m] * B)
            table[:, 915 // page] = -1
            a = csbp.PagedAttention(B, n, per, page, G * Hkv, Hkv, d, causal=causal, window=window,
                                    sinks=sinks)
            clean = [x.clone() for x in a.forward(q, c, table, length)]
            for b in range(B):
                pg = int(table[b, j // page])
                c.v[pg, j % page, ::2, 40 + b] = 0x7f
                c.v_scale[pg, j % page, 1::2, 0] = 255
            reads = torch.from_numpy(((j <= t) | (not causal)) & ((t - j < window) | (j < sinks))).cuda()
            bad = torch.zeros((B, n, Hkv, d), dtype=torch.bool, device="cuda")
            for b in range(B):
                bad[b, :, ::2, 40 + b] = reads[:, None]
                bad[b, :, 1::2, :32] = reads[:, None, None]
            o, lse = a.forward(q, c, table, length)
            assert torch.equal(lse, clean[1]) and torch.equal(o.isnan(), bad), (causal, j)
            assert torch.equal(torch.where(bad, 0, o), torch.where(bad, 0, clean[0]))


def test_nan_does_not_make_a_long_text_slow():
    """A CTA with 150,000 keys of its own and NaN in the last of them works for as long as
    without (four times is allowed)."""
    page, per, B, n, Hkv, d = 64, 2400, 152, 64, 1, 128
    c = filled(B + 8, page, Hkv, d, gen(45))
    table = torch.randint(0, 8, (B, per), generator=gen(46), device="cuda").int()
    table[:, -1] = 8 + torch.arange(B, device="cuda").int()
    length = i32([per * page - 5] * B)
    q = normal(gen(47), B, n, 1, d)
    a = csbp.PagedAttention(B, n, per, page, 1, Hkv, d, causal=True)

    def ms():
        times = []
        for _ in range(4):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            o, lse = a.forward(q, c, table, length)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        a.check()
        return min(times), o, lse

    clean, want, z = ms()
    c.v[8:, page - 7, 0, 77] = 0xff          # read by the last two queries
    slow, o, lse = ms()
    assert o[:, -2:, 0, 77].isnan().all() and torch.equal(lse, z)
    o[:, -2:, 0, 77] = want[:, -2:, 0, 77]
    assert torch.equal(o, want)
    assert slow <= 4 * clean, (slow, clean)


# --------------------------------------------------------------- as one runs
def step_state(seed, B=3, n=4, Hq=8, Hkv=2, d=64, page=16, per=8, layers=2):
    g = gen(seed)
    s = dict(ro=csbp.Rotary(freqs(d)), q=normal(g, B, n, Hq, d), k=normal(g, B, n, Hkv, d),
             v=normal(g, B, n, Hkv, d),
             caches=[filled(B * per, page, Hkv, d, g) for _ in range(layers)],
             table=torch.randperm(B * per, generator=g, device="cuda").view(B, per).int(),
             start=i32([60, 0, 33][:B]), a=csbp.PagedAttention(B, n, per, page, Hq, Hkv, d, True),
             o=torch.empty((B, n, Hq, d), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((B, Hq, n), device="cuda"), rq=normal(g, B, n, Hq, d))
    s["length"] = s["start"] + n
    return s


def step(s, stream=None):
    """Each layer appends its tokens and reads its cache; returns what came out."""
    for c in s["caches"]:
        c.append(s["k"], s["v"], s["table"], s["start"], rotary=s["ro"], q=s["q"], out=s["rq"],
                 stream=stream)
        s["a"].forward(s["rq"], c, s["table"], s["length"], out=(s["o"], s["lse"]), stream=stream)
    return s["rq"], s["o"], s["lse"]


@pytest.mark.parametrize("n", [4, 20])
def test_step_against_read_and_prefix_attention(n):
    """append + paged attention = the write, read back and attention of the prefix
    operator, to the difference of their roundings."""
    s = step_state(20, n=n)
    rq, o, lse = step(s)
    c = s["caches"][-1]
    B, n, Hq, d = s["q"].shape
    rows = int(s["length"].max())
    ko, vo = c.read(s["table"], i32([0] * B), rows=rows)
    pre = csbp.PrefixAttention(B, n, 0, rows, Hq, c.Hkv, d, causal=True)
    o2, lse2 = pre.forward(rq, None, None, ko, vo, s["length"])
    A = vo.abs().float().max()
    assert (o.float() - o2.float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * A
    assert (lse - lse2).abs().max() <= 2.0 ** -14
    check_attn((o, lse), rq, c, s["table"], s["length"], True, 0, 0, d ** -0.5)


@pytest.mark.parametrize("n", [4, 20])
def test_captured_step_follows_its_inputs(n):
    """One graph of both operators in two layers, replayed with other values and
    other lengths."""
    s, t = step_state(21, n=n), step_state(22, n=n)
    want = []
    for x in (s, t):
        before = [stored(c) for c in x["caches"]]
        want.append([y.clone() for y in step(x)] + [y for c in x["caches"] for y in stored(c)])
        for c, old in zip(x["caches"], before):
            for dst, src in zip((c.k, c.v, c.k_scale, c.v_scale), old):
                dst.copy_(src)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = [stored(c) for c in s["caches"]]
    with torch.cuda.graph(graph):
        step(s)
    for x, w in ((s, want[0]), (t, want[1]), (s, None)):
        if w is None:
            break
        for name in ("q", "k", "v", "table", "start", "length"):
            s[name].copy_(x[name])
        for c, src in zip(s["caches"], keep if x is s else [stored(c) for c in t["caches"]]):
            for dst, y in zip((c.k, c.v, c.k_scale, c.v_scale), src):
                dst.copy_(y)
        s["o"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [s["rq"], s["o"], s["lse"]] + [y for c in s["caches"] for y in stored(c)]
        assert same(got, w)


@pytest.mark.parametrize("n", [4, 20])
def test_two_streams_at_once(n):
    a, b = step_state(23, n=n), step_state(24, n=n)
    want = [[x.clone() for x in step(s)] for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in zip((a, b), streams):
            step(s, stream=st)
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert same([s["rq"], s["o"], s["lse"]], w)


@pytest.mark.parametrize("n", [1, 10, 30])
def test_one_handle_many_calls_in_a_row(n):
    """Pieces of one call are not mistaken for those of another: lengths change
    from call to call on one workspace."""
    c, q, table, _ = attn_case(4, n, 200, 16, 8, 2, 128, 25)
    a = csbp.PagedAttention(4, n, 200, 16, 8, 2, 128, causal=True)
    lens = [[3200, 1, 0, 50], [16, 3000, 2900, 2800], [0, 0, 0, 0], [3200] * 4, [1, 2, 3, 4]]
    outs = [a.forward(q, c, table, i32(x)) for x in lens * 3]
    torch.cuda.synchronize()
    for k, x in enumerate(lens):
        check_attn(outs[k], q, c, table, i32(x), True, 0, 0, 128 ** -0.5)
        assert same(outs[k], outs[k + 5]) and same(outs[k], outs[k + 10])


@pytest.mark.parametrize("n", [3, 9, 50])
def test_rows_of_outputs_and_cache_behind_stay(n):
    """Outputs are written whole and nothing else is; the cache is only read."""
    c, q, table, length = attn_case(2, n, 4, 16, 4, 2, 64, 26, [30, 64])
    before = stored(c)
    a = csbp.PagedAttention(2, n, 4, 16, 4, 2, 64, True)
    o = torch.full((4, n, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 4, n), 7.0, device="cuda")
    want = a.forward(q, c, table, length)
    a.forward(q, c, table, length, out=(o[1:3], lse[1:3]))
    assert same(want, (o[1:3], lse[1:3]))
    assert (o[::3] == 7).all() and (lse[::3] == 7).all() and same(before, stored(c))


@pytest.mark.parametrize("n", [1, 20])
def test_on_a_named_stream(n):
    """Outputs made in a call on a named stream are there whatever the current one
    is busy with, zeros of rows that take no part among them."""
    s = step_state(28, n=n)
    x = torch.zeros((8192, 8192), dtype=torch.bfloat16, device="cuda")
    count = i32([n, 0, n - 1])

    def call(stream):
        rq = s["caches"][0].append(s["k"], s["v"], s["table"], s["start"], count, rotary=s["ro"],
                                   q=s["q"], stream=stream)
        return rq, *s["a"].forward(rq, s["caches"][0], s["table"], s["length"], stream=stream)

    want = [t.clone() for t in call(None)]
    assert (want[0][1] == 0).all()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in want]
    for _ in range(50):
        torch.mm(x, x)
    for t in old:
        t.fill_(7)
    del old, t
    side = torch.cuda.Stream()
    got = call(side)
    torch.cuda.synchronize()
    assert same(got, want)


def test_kernels_are_timed():
    s = step_state(27)
    step(s)
    torch.cuda.synchronize()
    ms, n = ctypes.c_double(), ctypes.c_int32()
    csbp.kernel_timing(True)
    try:
        step(s)
        torch.cuda.synchronize()
        for kind in (11, 13):
            assert csbp.lib().csbp_kernel_timing_read_kind(kind, ctypes.byref(ms),
                                                           ctypes.byref(n)) == 0
            assert n.value == 2 and 0.0 < ms.value < 1000.0
    finally:
        csbp.kernel_timing(False)
