"""GPU parity of the generation operators with the float64 oracle.

Tolerances, derived from the arithmetic (half a rounding step is eps / 2):
 * cache: bit-exact (the scale is a power of two, so the only rounding is
   E4M3's own, which both sides define);
 * attention: with A = sum_j p_j |v_j|, an O element is off by at most 2^-8 A
   (P rounded to bf16) + 2^-8 |O| (O rounded to bf16) + fp32 terms: the
   exponential's 2^-21 and the sums' 2^-24 per step, all below 2^-12 A here;
   an exponent argument x carries d 2^-24 T from its dot product (T the
   largest scale sum |q k| of the row), which changes p by that much
   relative, so 2 d 2^-24 T A more.  LSE: d 2^-24 T + 2^-21 + 2^-22 |LSE|, and
   2^-24 for each of at most 2^8 sequential additions of a row's sum;
 * verification: exact integers.
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


# ------------------------------------------------------------------- cache
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


def check_write(c, before, k, v, table, start, count):
    pages, page = c.k.shape[:2]
    at = slots(table, start, count, k.shape[1], page, pages)
    for x, codes, scales, old, old_s in ((k, c.k, c.k_scale, before[0], before[2]),
                                         (v, c.v, c.v_scale, before[1], before[3])):
        vals, sb = O.quantise(f64(x))
        want = O.dequantise(old.cpu().numpy(), old_s.cpu().numpy()).reshape(-1, *x.shape[2:])
        want_s = old_s.cpu().numpy().reshape(-1, *sb.shape[2:]).copy()
        for b, i, s in at:
            if s >= 0:
                want[s], want_s[s] = vals[b, i], sb[b, i]
        np.testing.assert_array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s)
        got = O.dequantise(codes.cpu().numpy(), scales.cpu().numpy()).reshape(want.shape)
        np.testing.assert_array_equal(got, want)


def check_read(c, out, table, start, count, fill):
    pages, page = c.k.shape[:2]
    for got, codes, scales in ((out[0], c.k, c.k_scale), (out[1], c.v, c.v_scale)):
        vals = torch.from_numpy(O.dequantise(codes.cpu().numpy(), scales.cpu().numpy()))
        vals = vals.to(torch.bfloat16).double().numpy().reshape(-1, *got.shape[2:])
        want = np.full(got.shape, fill)
        for b, i, s in slots(table, start, count, got.shape[1], page, pages):
            want[b, i] = vals[s] if s >= 0 else np.nan
        np.testing.assert_array_equal(f64(got), want)


CACHES = [  # batch, rows, page, table entries, Hkv, d
    (1, 1, 1, 1, 1, 32), (3, 5, 16, 2, 2, 64), (2, 200, 64, 5, 3, 96), (4, 33, 7, 8, 8, 128),
    (1, 700, 128, 6, 1, 1024), (65, 1, 16, 3, 4, 128)]


@pytest.mark.parametrize("B,rows,page,n,Hkv,d", CACHES)
@pytest.mark.parametrize("ragged", [False, True])
def test_cache_write_and_read(B, rows, page, n, Hkv, d, ragged):
    g = gen(B * 1000 + rows)
    pages = B * n + 2
    c = dirty_cache(pages, page, Hkv, d, g)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    k, v = normal(g, B, rows, Hkv, d), normal(g, B, rows, Hkv, d) * 1e-3
    table = torch.randperm(pages, generator=g, device="cuda")[:B * n].view(B, n).int()
    start = torch.randint(0, n * page - rows + 1, (B,), generator=g, device="cuda").int()
    count = None
    if ragged:
        count = torch.randint(-1, rows + 2, (B,), generator=g, device="cuda").int()
    c.write(k, v, table, start, count)
    check_write(c, before, k, v, table, start, count)
    out = tuple(torch.full_like(k, 7.0) for _ in range(2))
    assert c.read(table, start, count, out=out) is out
    check_read(c, out, table, start, count, 7.0)
    fresh = c.read(table, start, count, rows=rows)
    check_read(c, fresh, table, start, count, 0.0)


def test_cache_values_at_the_edges():
    """Zeros, subnormals, the largest bf16, ties, NaN and infinities."""
    v = torch.zeros(1, 16, 1, 64)
    x = v[0, :, 0]
    x[0, 3] = 2.0 ** -133
    x[1, :32] = torch.arange(32) * 2.0 ** -126
    x[2] = 3.3895e38
    x[3, 1], x[3, 2], x[3, 40] = float("inf"), 5.0, float("-inf")
    x[4, 0], x[4, 1] = float("nan"), -1.0
    x[5, :] = float("nan")
    x[6, :32] = torch.tensor([448., 432., 416., 400., 304., 17., 19., 0.0078125] * 4)  # ties
    x[6, 32:] = torch.tensor([448.] + [k * 2.0 ** -10 for k in range(31)])  # E4M3 subnormals
    x[7, 0] = 450.0
    x[8] = torch.linspace(-1, 1, 64)
    x[9, ::2] = -0.0
    v = v.to(torch.bfloat16).cuda()
    c = dirty_cache(2, 8, 1, 64, gen(1))
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    table, start = i32([[1, 0]]), i32([0])
    c.write(v, v, table, start)
    check_write(c, before, v, v, table, start, None)
    out = c.read(table, start, rows=16)
    check_read(c, out, table, start, None, 0.0)
    # every scale byte, the smallest and NaN among them
    c = dirty_cache(16, 16, 1, 64, gen(2))
    c.k_scale.copy_(torch.arange(256).view(16, 16, 1, 1).expand(16, 16, 1, 2))
    table = torch.arange(16, device="cuda").int()[None]
    out = c.read(table, start, rows=256)
    pages = c.k.shape[0]
    vals = torch.from_numpy(O.dequantise(c.k.cpu().numpy(), c.k_scale.cpu().numpy()))
    want = vals.to(torch.bfloat16).double().numpy().reshape(1, 256, 1, 64)
    np.testing.assert_array_equal(f64(out[0]), want)
    assert pages == 16


def test_cache_positions_and_pages_out_of_range():
    g = gen(3)
    c = dirty_cache(4, 8, 2, 64, g)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    k, v = normal(g, 4, 6, 2, 64), normal(g, 4, 6, 2, 64)
    # a negative start, past the table, pages -1 and 4, the largest position
    table, start = i32([[0, 1], [2, -1], [4, 3], [1, 1]]), i32([-3, 5, 6, 2147483647])
    c.write(k, v, table, start)
    check_write(c, before, k, v, table, start, None)
    out = tuple(torch.full_like(k, 3.0) for _ in range(2))
    c.read(table, start, out=out)
    check_read(c, out, table, start, None, 3.0)


def test_cache_strides():
    """k and v as views into one packed tensor, batch entries spaced out."""
    g = gen(4)
    packed = normal(g, 3, 11, 9, 64)[:, 2:9]
    k, v = packed[:, :, 2:4], packed[:, :, 4:6]
    c = dirty_cache(7, 4, 2, 64, g)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    table, start = i32([[0, 1], [2, 3], [4, 5]]), i32([0, 1, 0])
    c.write(k, v, table, start)
    check_write(c, before, k, v, table, start, None)
    dst = torch.full((3, 11, 9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    view = dst[:, 2:9]
    c.read(table, start, out=(view[:, :, 2:4], view[:, :, 4:6]))
    check_read(c, (view[:, :, 2:4], view[:, :, 4:6]), table, start, None, 5.0)
    rest = torch.ones(dst.shape, dtype=torch.bool)
    rest[:, 2:9, 2:6] = False
    assert (dst.cpu()[rest] == 5.0).all()


@pytest.mark.parametrize("rows", [5, 1500])
def test_cache_rows_on_16_bytes(rows):
    """Rows of the bf16 side that start on 16 bytes but not on 32."""
    B, H, d = 2, 3, 64
    g = gen(6)
    tok = H * d + 8

    def view():
        flat = normal(g, 8 + B * rows * tok)
        return flat.as_strided((B, rows, H, d), (rows * tok, tok, d, 1), 8)

    k, v = view(), view()
    n = -(-(rows + 2) // 16)
    c = dirty_cache(B * n, 16, H, d, g)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    table = torch.randperm(B * n, generator=g, device="cuda").int().view(B, n)
    start = i32([0, 2])
    c.write(k, v, table, start)
    check_write(c, before, k, v, table, start, None)
    out = view(), view()
    c.read(table, start, out=out)
    check_read(c, out, table, start, None, 0.0)


def test_rows_that_share_a_place_leave_bytes_of_either():
    g = gen(7)
    k, v = normal(g, 2, 40, 2, 64), normal(g, 2, 40, 2, 64) * 30
    alone = []
    for b in range(2):
        c = csbp.QuantCache(4, 16, 2, 64)
        c.write(k[b:b + 1], v[b:b + 1], i32([[0, 2, 1]]), i32([3]))
        alone.append([t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)])
    c = csbp.QuantCache(4, 16, 2, 64)
    c.write(k, v, i32([[0, 2, 1], [0, 2, 1]]), i32([3, 3]))
    for got, x, y in zip((c.k, c.v, c.k_scale, c.v_scale), *alone):
        assert ((got == x) | (got == y)).all()


def test_cache_beyond_32_bits():
    """Byte offsets past 2^32 in the codes."""
    pages, page = 70000, 64
    c = csbp.QuantCache(pages, page, 8, 128)
    g = gen(5)
    k, v = normal(g, 2, 70, 8, 128), normal(g, 2, 70, 8, 128)
    table, start = i32([[69999, 3], [69998, 65536]]), i32([1, 2])
    c.write(k, v, table, start)
    rk, rv = c.read(table, start, rows=70)
    for got, x in ((rk, k), (rv, v)):
        np.testing.assert_array_equal(f64(got), O.quantise(f64(x))[0])
    written = (c.k.view(pages, -1) != 0).any(1).nonzero()[:, 0].tolist()
    assert written == [3, 65536, 69998, 69999]


# --------------------------------------------------------------- attention
def attn_inputs(B, n, Lp, S, Hq, Hkv, d, seed, spread=1.0):
    g = gen(seed)
    return dict(q=normal(g, B, n, Hq, d) * spread, k_prefix=normal(g, Lp, Hkv, d),
                v_prefix=normal(g, Lp, Hkv, d), k_own=normal(g, B, S, Hkv, d),
                v_own=normal(g, B, S, Hkv, d))


def check_attn(got, t, own_len, causal, scale):
    o, lse = got
    c = [min(max(int(x), 0), t["k_own"].shape[1]) for x in own_len]
    ko, vo = f64(t["k_own"]), f64(t["v_own"])
    for b, m in enumerate(c):       # what lies past a sequence's end is not read
        ko[b, m:] = vo[b, m:] = 0
    want, Z, A, T = O.prefix_attention(f64(t["q"]), f64(t["k_prefix"]), f64(t["v_prefix"]), ko, vo,
                                       c, causal, scale)
    d = o.shape[-1]
    Tq = T.transpose(0, 2, 1)[..., None]
    tol = (2.0 ** -8 + 2.0 ** -12 + 2 * d * 2.0 ** -24 * Tq) * A + 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(o) - want)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-30)).max()
    got_z = f64(lse)
    empty = np.isneginf(Z)
    np.testing.assert_array_equal(np.isneginf(got_z), empty)
    ztol = d * 2.0 ** -24 * T + 2.0 ** -21 + 2.0 ** -16
    ok = ~empty
    assert (np.abs(got_z[ok] - Z[ok]) <= (ztol[ok] + 2.0 ** -22 * np.abs(Z[ok]))).all()
    assert (f64(o)[np.broadcast_to(empty.transpose(0, 2, 1)[..., None], o.shape)] == 0).all()


ATTN = [  # batch, queries, prefix, own_max, Hq, Hkv, d, causal, own_len
    (1, 1, 1, 0, 1, 1, 64, False, [0]),
    (1, 1, 0, 1, 1, 1, 128, False, [1]),
    (2, 3, 0, 0, 2, 1, 64, False, [0, 0]),                       # nothing to read
    (3, 2, 0, 9, 4, 2, 64, True, [0, 1, 9]),                     # some rows empty
    (2, 1, 128, 128, 8, 2, 128, False, [128, 0]),
    (3, 5, 1000, 77, 2, 2, 64, True, [77, 3, 0]),
    (2, 32, 257, 130, 10, 2, 128, False, [130, 129]),            # 5 heads per KV head
    (4, 16, 129, 64, 8, 1, 64, False, [64, 1, 999, -5]),         # clamped lengths
    (2, 33, 300, 200, 15, 3, 128, True, [150, 33]),
    (1, 300, 140, 300, 4, 2, 64, True, [300]),                   # many row tiles
    (1, 129, 1, 129, 1, 1, 128, False, [129]),
    (40, 1, 513, 20, 6, 2, 128, False, list(range(0, 40))),      # rows of many sequences
    (7, 3, 260, 140, 4, 4, 64, True, [140, 139, 2, 1, 0, 128, 129]),
    (2, 2, 200, 150, 256, 1, 64, False, [150, 7]),               # 256 heads per KV head
    (2, 1, 300, 3, 131, 1, 128, True, [3, 1]),                   # a prime head count
    (1, 1, 5000, 300, 4, 1, 128, False, [300]),                  # split along the keys
    (2, 1, 20011, 64, 4, 2, 64, True, [60, 64]),
    (17, 9, 640, 256, 4, 2, 128, False, [256 - 13 * i for i in range(17)]),
    (130, 1, 130, 5, 2, 1, 64, True, [i % 6 for i in range(130)]),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_prefix_attention(case):
    B, n, Lp, S, Hq, Hkv, d, causal, lens = ATTN[case]
    t = attn_inputs(B, n, Lp, S, Hq, Hkv, d, 100 + case)
    a = csbp.PrefixAttention(B, n, Lp, S, Hq, Hkv, d, causal=causal)
    got = a.forward(**t, own_len=i32(lens))
    a.check()
    check_attn(got, t, lens, causal, d ** -0.5)
    again = a.forward(**t, own_len=i32(lens))       # the workspace holds an old call's results
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("spread", [30.0, 0.0])
def test_sharp_and_flat_softmax(spread):
    """Scores of a hundred and more (the running maximum moves far) and
    scores that are all equal."""
    t = attn_inputs(3, 4, 700, 300, 8, 2, 128, 7, spread)
    a = csbp.PrefixAttention(3, 4, 700, 300, 8, 2, 128)
    check_attn(a.forward(**t, own_len=i32([300, 10, 150])), t, [300, 10, 150], False, 128 ** -0.5)


def test_growing_scores_rescale_exactly():
    """Keys whose scores climb along the prefix, so that the reference
    maximum moves in every tile."""
    t = attn_inputs(2, 2, 900, 130, 4, 2, 64, 8)
    t["q"].fill_(0.5)
    for x in (t["k_prefix"], t["k_own"]):
        L = x.shape[-3]
        ramp = torch.linspace(0, 6, L, device="cuda").view(L, 1, 1)
        x.copy_((x.float() * 0.1 + ramp).to(torch.bfloat16))
    a = csbp.PrefixAttention(2, 2, 900, 130, 4, 2, 64)
    check_attn(a.forward(**t, own_len=i32([130, 64])), t, [130, 64], False, 0.125)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_past_the_end_may_hold_anything(bad, causal):
    lens = [0, 1, 127, 128, 129, 200]
    t = attn_inputs(6, 2, 100, 260, 8, 2, 128, 9)
    for b, c in enumerate(lens):
        t["k_own"][b, c:] = bad
        t["v_own"][b, c:] = bad
    a = csbp.PrefixAttention(6, 2, 100, 260, 8, 2, 128, causal=causal)
    got = a.forward(**t, own_len=i32(lens))
    assert torch.isfinite(got[0].float()).all()
    check_attn(got, t, lens, causal, 128 ** -0.5)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,causal", [(1, False), (2, True), (40, False)])
def test_a_sequence_that_is_not_finite_stays_alone(value, n, causal):
    """K or V of one sequence that are not finite do not reach any other
    sequence's rows, also where they share row tiles."""
    B, Lp, S = 9, 150, 200
    lens = [200, 3, 129, 64, 200, 0, 128, 77, 200]
    t = attn_inputs(B, n, Lp, S, 8, 2, 128, 12)
    a = csbp.PrefixAttention(B, n, Lp, S, 8, 2, 128, causal=causal)
    others = [b for b in range(B) if b != 4]
    rest = {k: x if k.endswith("prefix") else x[others] for k, x in t.items()}
    for name in ("v_own", "k_own"):
        bad = {k: x.clone() for k, x in t.items()}
        bad[name][4, 131, 1, 5] = value
        o, lse = a.forward(**bad, own_len=i32(lens))
        a.check()
        check_attn((o[others], lse[others]), rest, [lens[b] for b in others], causal, 128 ** -0.5)
        # the sequence's own heads of that KV head do not hide it (its last query
        # reads key 131 in every case); an infinite K may give a score of -inf,
        # which weighs nothing
        if name == "v_own" or value != value:
            assert not torch.isfinite(o[4, -1, 4:].float()).all(-1).any(), name
        assert torch.isfinite(o[4, :, :4].float()).all()


@pytest.mark.parametrize("d", [64, 128])
def test_not_finite_where_jobs_are_cut(d):
    """Rows summed again from partial results, with both slots at work."""
    B, n, Lp, S = 16, 16, 5000, 300
    lens = [300, 1, 128, 0, 257, 300, 17, 129, 300, 64, 3, 200, 300, 255, 90, 300]
    t = attn_inputs(B, n, Lp, S, 8, 2, d, 19)
    t["v_own"][5, 140] = float("nan")
    t["v_own"][12, 2, 1, 7] = float("inf")
    a = csbp.PrefixAttention(B, n, Lp, S, 8, 2, d)
    o, lse = a.forward(**t, own_len=i32(lens))
    a.check()
    assert torch.isnan(o[5].float()).all()
    hit = o[12].float().view(n, 2, 4, d)[:, 1, :, 7]
    assert torch.isinf(hit).all()
    rest = [b for b in range(B) if b not in (5, 12)]
    part = {k: x if "prefix" in k else x[rest] for k, x in t.items()}
    check_attn((o[rest], lse[rest]), part, [lens[b] for b in rest], False, d ** -0.5)


def test_causal_queries_do_not_see_later_values():
    """The last key's V is read by the last query only, whatever it holds."""
    B, n, Lp, S = 3, 6, 300, 140
    lens = [140, 9, 128]
    t = attn_inputs(B, n, Lp, S, 4, 2, 64, 13)
    a = csbp.PrefixAttention(B, n, Lp, S, 4, 2, 64, causal=True)
    clean = {k: x.clone() for k, x in t.items()}
    for b, c in enumerate(lens):
        t["v_own"][b, c - 1] = float("nan")
        clean["v_own"][b, c - 1] = 0.0
    o, lse = a.forward(**t, own_len=i32(lens))
    assert torch.isnan(o[:, -1].float()).all()
    check_attn((torch.cat([o[:, :-1], a.forward(**clean, own_len=i32(lens))[0][:, -1:]], 1), lse),
               clean, lens, True, 0.125)


@pytest.mark.parametrize("d", [64, 128])
def test_row_tiles_without_a_key(d):
    """Every second row tile, and the last job, reads no key at all."""
    B, n = 160, 32
    t = attn_inputs(B, n, 0, 700, 16, 4, d, 17)
    lens = [0 if b % 2 or b >= 156 else 1 + 37 * b % 700 for b in range(B)]
    a = csbp.PrefixAttention(B, n, 0, 700, 16, 4, d)
    out = a.forward(**t, own_len=i32(lens))
    a.check()
    check_attn(out, t, lens, False, d ** -0.5)


@pytest.mark.parametrize("B,n,Lp,S,Hq,Hkv,d", [
    (16, 1, 1500, 3000, 8, 2, 128), (1, 1, 0, 5000, 2, 2, 64), (40, 3, 700, 1000, 6, 1, 64)])
@pytest.mark.parametrize("lens", ["none", "few", "one", "all"])
def test_room_for_more_keys(B, n, Lp, S, Hq, Hkv, d, lens):
    """Where the own tiles are cut by lengths that only the device knows."""
    lens = {"none": [0] * B, "few": [b % 7 for b in range(B)],
            "one": [0] * (B - 1) + [S], "all": [S - b for b in range(B)]}[lens]
    t = attn_inputs(B, n, Lp, S, Hq, Hkv, d, 23)
    a = csbp.PrefixAttention(B, n, Lp, S, Hq, Hkv, d)
    a.ws[256:] = 0x7f          # what a partial holds that nobody wrote
    out = a.forward(**t, own_len=i32(lens))
    a.check()
    check_attn(out, t, lens, False, d ** -0.5)


def test_attention_strides():
    """q, k and v as views into packed projections; the prefix as a slice of a
    longer cache."""
    B, n, Lp, S, Hq, Hkv, d = 3, 7, 200, 150, 6, 2, 64
    g = gen(10)
    qkv = normal(g, B, n + 3, Hq + 5, d)[:, 1:n + 1]
    pre = normal(g, Lp + 9, 2 * Hkv + 1, d)[4:Lp + 4]
    mine = normal(g, B, S + 2, 2 * Hkv, d)[:, 2:]
    t = dict(q=qkv[:, :, 2:Hq + 2], k_prefix=pre[:, :Hkv], v_prefix=pre[:, Hkv:2 * Hkv],
             k_own=mine[:, :, :Hkv], v_own=mine[:, :, Hkv:])
    lens = [150, 20, 0]
    a = csbp.PrefixAttention(B, n, Lp, S, Hq, Hkv, d, scale=0.2)
    got = a.forward(**t, own_len=i32(lens))
    check_attn(got, t, lens, False, 0.2)
    flat = {k: x.contiguous() for k, x in t.items()}
    want = a.forward(**flat, own_len=i32(lens))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_equals_the_library_merge_of_its_parts():
    """Prefix alone and own keys alone, merged exactly, are the whole."""
    B, n, Lp, S, H, d = 2, 3, 300, 100, 2, 64
    t = attn_inputs(B, n, Lp, S, H, H, d, 11)
    lens = i32([100, 41])
    whole = csbp.PrefixAttention(B, n, Lp, S, H, H, d).forward(**t, own_len=lens)
    pre = csbp.PrefixAttention(B, n, Lp, 0, H, H, d).forward(
        t["q"], t["k_prefix"], t["v_prefix"], None, None, None)
    mine = csbp.PrefixAttention(B, n, 0, S, H, H, d).forward(
        t["q"], None, None, t["k_own"], t["v_own"], lens)
    o = torch.empty((B * n, H, d), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((H, B * n), device="cuda")
    csbp.lse_merge([x[0].float().view(B * n, H, d) for x in (pre, mine)],
                   [x[1].permute(1, 0, 2).reshape(H, B * n).contiguous() for x in (pre, mine)],
                   o, z)
    ref = whole[0].float().view(B * n, H, d)
    # two bf16 roundings (each 2^-8 of P and of the partials) on either side
    assert (o.float() - ref).abs().max() <= 4 * 2.0 ** -8 * float(t["v_prefix"].abs().max())
    assert (z.view(H, B, n).transpose(0, 1) - whole[1]).abs().max() <= 2.0 ** -14


def test_attention_beyond_32_bits():
    """A prefix whose element offsets pass 2^31 and byte offsets 2^32: every
    key but one is orthogonal to the queries."""
    Lp, H, d = 2200000, 8, 128
    t = dict(k=torch.zeros((Lp, H, d), dtype=torch.bfloat16, device="cuda"))
    t["v"] = torch.zeros_like(t["k"])
    at = Lp - 5
    t["k"][at] = 4.0
    t["v"][at] = torch.arange(H * d, device="cuda").view(H, d).to(torch.bfloat16)
    q = torch.ones((1, 2, H, d), dtype=torch.bfloat16, device="cuda")
    a = csbp.PrefixAttention(1, 2, Lp, 0, H, H, d, scale=0.125)
    o, lse = a.forward(q, t["k"], t["v"], None, None, None)
    a.check()
    # scores: 64 at one key, 0 elsewhere; the others weigh Lp e^-64, nothing
    assert torch.equal(o, t["v"][at].expand(1, 2, H, d))
    assert (lse - 64.0).abs().max() <= 64 * 2.0 ** -22     # (scale log2 e) and ln 2 are rounded


# ------------------------------------------------------------ verification
def verify_inputs(B, K, V, seed, sharp=1.0):
    g = gen(seed)
    z = torch.randn((B, K + 1, V), generator=g, device="cuda") * sharp
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :K] + torch.randn((B, K, V), generator=g, device="cuda"), -1)
    x = torch.randint(0, V, (B, K), generator=g, device="cuda")
    if K:
        x = torch.multinomial(q.reshape(-1, V), 1, generator=g).view(B, K)
    u, r = (torch.rand(s, generator=g, device="cuda") for s in ((B, K), (B,)))
    return p, q, x.int(), u, r


def check_verify(got, p, q, x, u, r, length=None):
    acc, out = (t.cpu().numpy() for t in got)
    p, q, x, u, r = (t.cpu().numpy() for t in (p, q, x, u, r))
    for b in range(p.shape[0]):
        n = x.shape[1] if length is None else int(length[b])
        a, toks = O.draft_verify(p[b], q[b], x[b], u[b], r[b], n)
        assert acc[b] == a and out[b].tolist() == toks, b


VERIFY = [(1, 1, 2), (1, 0, 7), (5, 3, 100), (3, 4, 1001), (2, 2, 5000), (9, 16, 33),
          (40, 1, 257), (4, 2, 4099), (2, 1, 20000), (1, 1, 40000), (2, 2, 70001)]


@pytest.mark.parametrize("B,K,V", VERIFY)
@pytest.mark.parametrize("sharp", [1.0, 6.0])
def test_draft_verify(B, K, V, sharp):
    t = verify_inputs(B, K, V, 10 * B + K, sharp)
    check_verify(csbp.draft_verify(*t), *t)
    length = torch.randint(-1, K + 2, (B,), generator=gen(B), device="cuda").int()
    check_verify(csbp.draft_verify(*t, length), *t, length)


def test_verify_all_and_none_accepted():
    p, q, x, u, r = verify_inputs(4, 6, 300, 20)
    u0 = torch.zeros_like(u)
    acc, out = csbp.draft_verify(p, q, x, u0, r)
    assert (acc == 6).all() and torch.equal(out[:, :6], x)
    check_verify((acc, out), p, q, x, u0, r)
    p.scatter_(2, x.long()[..., None].expand(4, 6, 1).clone(), 0.0)
    acc, out = csbp.draft_verify(p, q, x, u0, r)
    assert (acc == 0).all() and (out[:, 1:] == -1).all()
    check_verify((acc, out), p, q, x, u0, r)


def test_verify_borders():
    """Ties of the acceptance test, r on borders of the cumulative sum,
    leading and trailing zeros, p <= q everywhere."""
    V = 5000
    p = torch.zeros((6, 2, V), device="cuda")
    q = torch.zeros((6, 1, V), device="cuda")
    p[:, 0, 100:104] = 0.25
    q[:, 0, 100] = 0.5
    p[:, 1, V - 1] = 1.0
    x = i32([[100]] * 6)
    u = torch.tensor([.5, .49999997, .5, .5, .5, .5], device="cuda")[:, None]
    r = torch.tensor([0., .5, 1 / 3, .6666667, .99999994, .33333334], device="cuda")
    check_verify(csbp.draft_verify(p, q, x, u, r), p, q, x, u, r)
    q[:, 0, 100:104] = 0.25            # nothing is left of p - q: p itself
    u = torch.full_like(u, 0.99)
    x = i32([[V]] * 5 + [[-1]])        # tokens that do not exist are not accepted
    check_verify(csbp.draft_verify(p, q, x, u, r), p, q, x, u, r)
    check_verify(csbp.draft_verify(p, q, x, u, r * 0), p, q, x, u, r * 0)


def test_verify_bad_numbers():
    """NaN and negative weights count as nothing; sums that are not finite,
    or nothing at all, give -1."""
    p, q, x, u, r = verify_inputs(5, 1, 700, 21)
    u.fill_(1.0)
    x[:, 0] = p[:, 0].argmin(-1).int()
    q.scatter_(2, x.long()[..., None], 1.0)      # rejected
    p[0, 0, 5], p[1, 0, 6] = float("nan"), -3.0
    p[2, 0, 7] = float("inf")
    p[3] = 0
    p[4] = float("nan")
    acc, out = csbp.draft_verify(p, q, x, u, r)
    assert (acc == 0).all() and out[2:, 0].tolist() == [-1, -1, -1]
    clean = p.nan_to_num(0.0, 0.0).clamp(min=0)
    check_verify((acc[:2], out[:2]), clean[:2], q[:2], x[:2], u[:2], r[:2])


def test_verify_strides():
    p, q, x, u, r = verify_inputs(4, 3, 501, 22)
    wide_p = torch.full((4, 6, 640), 9.0, device="cuda")
    wide_q = torch.full((4, 5, 509), 9.0, device="cuda")
    wide_p[:, 1:5, 3:504], wide_q[:, :3, 5:506] = p, q
    got = csbp.draft_verify(wide_p[:, 1:5, 3:504], wide_q[:, :3, 5:506], x, u, r)
    check_verify(got, p, q, x, u, r)
    buf = (torch.full((4,), 77, dtype=torch.int32, device="cuda"),
           torch.full((4, 4), 77, dtype=torch.int32, device="cuda"))
    assert csbp.draft_verify(p, q, x, u, r, out=buf) == buf
    assert torch.equal(buf[0], got[0]) and torch.equal(buf[1], got[1])


def test_verify_large_vocabulary_against_64_bit_sums():
    B, K, V = 16, 3, 131072
    p, q, x, u, r = verify_inputs(B, K, V, 23, 2.0)
    acc, out = csbp.draft_verify(p, q, x, u, r)
    P, Q = f64(p), f64(q)
    for b in range(B):
        a = K
        for i in range(K):
            t = int(x[b, i])
            if not float(u[b, i]) * Q[b, i, t] < P[b, i, t]:
                a = i
                break
        w = np.maximum(P[b, a] - Q[b, a], 0) if a < K else P[b, a]
        c = np.cumsum(w)
        assert acc[b] == a and out[b, a] == np.searchsorted(c, float(r[b]) * c[-1], "right")


# ------------------------------------------------- as a program uses them
def test_generation_step_end_to_end():
    """A block written to the cache, read back, attended to with the shared
    prefix (itself read from the cache), and its drafts verified."""
    B, M, Lp, S, Hq, Hkv, d, page, V = 3, 8, 200, 40, 4, 2, 64, 16, 500
    g = gen(30)
    nP, nS = -(-Lp // page), -(-S // page)
    c = csbp.QuantCache(nP + B * nS, page, Hkv, d)
    perm = torch.randperm(nP + B * nS, generator=g, device="cuda").int()
    tp, ts = perm[:nP].view(1, nP), perm[nP:].view(B, nS)
    pk, pv = normal(g, 1, Lp, Hkv, d), normal(g, 1, Lp, Hkv, d)
    c.write(pk, pv, tp, i32([0]))
    lens = [0, 13, 32]
    hk, hv = normal(g, B, 32, Hkv, d), normal(g, B, 32, Hkv, d)
    c.write(hk, hv, ts, i32([0] * B), i32(lens))            # what each generated so far
    nk, nv = normal(g, B, M, Hkv, d), normal(g, B, M, Hkv, d)
    c.write(nk, nv, ts, i32(lens))                          # the block of this step
    own_len = [x + M for x in lens]
    kp, vp = c.read(tp, i32([0]), rows=Lp)
    ko, vo = c.read(ts, i32([0] * B), i32(own_len), rows=S)
    q = normal(g, B, M, Hq, d)
    attn = csbp.PrefixAttention(B, M, Lp, S, Hq, Hkv, d)
    got = attn.forward(q, kp[0], vp[0], ko, vo, i32(own_len))
    attn.check()
    t = dict(q=q, k_prefix=torch.from_numpy(O.quantise(f64(pk))[0][0]),
             v_prefix=torch.from_numpy(O.quantise(f64(pv))[0][0]))
    for name, h, new in (("k_own", hk, nk), ("v_own", hv, nv)):
        x = np.zeros((B, S, Hkv, d))
        for b, n in enumerate(lens):
            x[b, :n], x[b, n:n + M] = O.quantise(f64(h))[0][b, :n], O.quantise(f64(new))[0][b]
        t[name] = torch.from_numpy(x)
    check_attn(got, t, own_len, False, d ** -0.5)
    ver = verify_inputs(B, M, V, 31)
    check_verify(csbp.draft_verify(*ver), *ver)


def step(s, stream=None):
    s["cache"].write(s["k"], s["v"], s["table"], s["start"], stream=stream)
    s["cache"].read(s["table"], s["zero"], s["len"], out=s["own"], stream=stream)
    o = s["attn"].forward(s["q"], s["kp"], s["vp"], *s["own"], s["len"], out=s["o"],
                          stream=stream)
    csbp.draft_verify(*s["ver"], out=s["acc"], stream=stream)
    return [*o, *s["acc"], *s["own"]]


def step_state(seed):
    B, M, Lp, S, Hq, Hkv, d, page = 4, 5, 333, 48, 8, 2, 128, 16
    g = gen(seed)
    s = dict(cache=csbp.QuantCache(12, page, Hkv, d), k=normal(g, B, M, Hkv, d),
             v=normal(g, B, M, Hkv, d), table=torch.arange(12, device="cuda").int().view(4, 3),
             start=i32([0, 9, 20, 43]), zero=i32([0] * 4), len=i32([5, 14, 25, 48]),
             kp=normal(g, Lp, Hkv, d), vp=normal(g, Lp, Hkv, d), q=normal(g, B, M, Hq, d),
             attn=csbp.PrefixAttention(B, M, Lp, S, Hq, Hkv, d, causal=True),
             ver=verify_inputs(B, M, 1000, seed))
    s["own"] = tuple(torch.zeros((B, S, Hkv, d), dtype=torch.bfloat16, device="cuda")
                     for _ in range(2))
    s["o"] = s["attn"].alloc_outputs()
    s["acc"] = (torch.zeros(B, dtype=torch.int32, device="cuda"),
                torch.zeros((B, M + 1), dtype=torch.int32, device="cuda"))
    return s


def test_other_streams_and_graph_replay_give_the_same():
    want = [x.clone() for x in step(step_state(40))]
    torch.cuda.synchronize()
    s = step_state(40)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(s, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    s = step_state(40)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    other = step_state(41)          # new inputs in the captured buffers
    for name in ("k", "v", "q", "kp", "vp"):
        s[name].copy_(other[name])
    for a, b in zip(s["ver"], other["ver"]):
        a.copy_(b)
    s["cache"].k.zero_(), s["cache"].v.zero_()
    s["cache"].k_scale.zero_(), s["cache"].v_scale.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    s["attn"].check()
    want = step(other)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_cut_attention_in_graphs_and_on_two_streams():
    """Calls that end with the joining of pieces, captured and at once."""
    shape = (2, 3, 4096, 130, 8, 2, 128)
    lens = i32([130, 7])
    calls, want = [], []
    for seed in (70, 71):
        t = attn_inputs(*shape, seed)
        first = csbp.PrefixAttention(*shape)
        want.append([x.clone() for x in first.forward(**t, own_len=lens)])
        calls.append((csbp.PrefixAttention(*shape), t, first.alloc_outputs()))
        first.check()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for a, t, out in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            a.forward(**t, own_len=lens, out=out)
            a.forward(**t, own_len=lens, out=out)
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (a, _, out), w in zip(calls, want):
        a.check()
        assert all(torch.equal(x, y) for x, y in zip(out, w))
        for x in out:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for (a, t, out), st in zip(calls, streams):
            a.forward(**t, own_len=lens, out=out, stream=st)
    torch.cuda.synchronize()
    for (_, _, out), w in zip(calls, want):
        assert all(torch.equal(x, y) for x, y in zip(out, w))


def test_two_streams_at_once():
    """Calls with workspaces of their own may overlap."""
    a, b = step_state(50), step_state(51)
    want = [[x.clone() for x in step(s)] for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in zip((a, b), streams):
            step(s, stream=st)
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(w, [*s["o"], *s["acc"], *s["own"]]))


def test_each_kernel_kind_is_timed():
    s = step_state(60)
    step(s)
    # (pieces to join: one token over keys that are cut up to fill the GPU)
    cut = csbp.PrefixAttention(1, 1, 4096, 0, 4, 2, 64)
    t = attn_inputs(1, 1, 4096, 0, 4, 2, 64, 61)
    args = t["q"], t["k_prefix"], t["v_prefix"], None, None, None
    cut.forward(*args)
    torch.cuda.synchronize()
    ms, n = ctypes.c_double(), ctypes.c_int32()
    read = csbp.lib().csbp_kernel_timing_read_kind
    csbp.kernel_timing(True)
    try:
        step(s)
        cut.forward(*args)
        torch.cuda.synchronize()
        for kind in range(11, 16):
            assert read(kind, ctypes.byref(ms), ctypes.byref(n)) == 0
            assert n.value >= 1 and 0.0 < ms.value < 1000.0, kind
        assert read(16, ctypes.byref(ms), ctypes.byref(n)) == -1
    finally:
        csbp.kernel_timing(False)


# ------------------------------------- rows without a key, keys not finite
@pytest.mark.parametrize("name", ["v_own", "k_own"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,S,Hq,Hkv,causal,lens,where", [
    (1, 4, 9, 2, 1, True, [2], (0, 0)),                     # queries before the first key
    (2, 3, 9, 4, 2, False, [0, 9], (1, 4)),                 # beside a neighbour of the tile
    (5, 40, 140, 4, 2, True, [30, 140, 0, 7, 0], (0, 0)),   # several row tiles
    (5, 40, 140, 4, 2, True, [30, 140, 0, 7, 0], (1, 139)),
    (3, 50, 300, 2, 1, False, [0, 300, 0], (1, 290)),       # the last row tile alone
    (1, 1000, 5000, 1, 1, True, [400], (0, 3)),             # far more room than keys
])
def test_rows_without_a_key_beside_keys_that_are_not_finite(B, n, S, Hq, Hkv, causal, lens, where,
                                                            d, value, name):
    """No prefix, so that some rows read no key at all: O = 0 and LSE = -inf
    whatever the keys of the tile hold, and other rows that do not read the key
    that is not finite come out as without it."""
    t = attn_inputs(B, n, 0, S, Hq, Hkv, d, 90)
    a = csbp.PrefixAttention(B, n, 0, S, Hq, Hkv, d, causal=causal)
    clean = [x.clone() for x in a.forward(**t, own_len=i32(lens))]
    check_attn(clean, t, lens, causal, d ** -0.5)
    b, j = where
    bad = dict(t)
    bad[name] = t[name].clone()
    bad[name][b, j] = value
    o, lse = a.forward(**bad, own_len=i32(lens))
    a.check()
    reads = torch.zeros((B, n), dtype=torch.bool, device="cuda")
    reads[b] = j <= lens[b] - n + torch.arange(n, device="cuda") if causal else True
    assert not reads.all() and reads.any()
    assert not torch.isfinite(o[reads].float()).all() or name == "k_own"
    o, lse = o.clone(), lse.clone()
    o[reads] = clean[0][reads]
    lse = torch.where(reads[:, None], clean[1], lse)
    check_attn((o, lse), t, lens, causal, d ** -0.5)


# ------------------------------------------------- sums of long vocabularies
@pytest.mark.parametrize("V", [131072, 1 << 27])
def test_verify_sums_beside_a_border(V):
    """r = 1/2 and w_0 + w_1 a little more or less than the rest R, so that token
    1 or 2 is next.  Two sums are compared: each may be off by 2^-42 of its
    value (see the kernel's comment), half of w_0 + w_1 + R and w_0 + w_1 by
    2^-42 R each, and half the gap has to be more: a gap of 2^-40 R does.  All
    weight lies where few threads read it, so that one thread adds thousands."""
    rng = np.random.default_rng(5)
    at = np.arange(max(512, V // 4096))
    at = (at // 4) * 128 + at % 4
    p, want = torch.zeros((6, 1, V), device="cuda"), []
    for b in range(6):
        w = np.exp(rng.standard_normal(len(at)) * 2).astype(np.float32)
        w = np.maximum(w, np.float32(2.0 ** -20))
        unit = 80                                      # exact sums in units of 2^-80
        R = sum(int(np.ldexp(float(x), 50)) for x in w[2:]) << (unit - 50)
        gap = R >> 40
        T = R + gap if b % 2 else R - gap
        hi = np.float32(T / 2.0 ** unit)
        hi = np.nextafter(np.nextafter(hi, np.float32(0)), np.float32(0))
        lo = np.float32((T - (int(np.ldexp(float(hi), 40)) << (unit - 40))) / 2.0 ** unit)
        w[0], w[1] = hi, lo
        T = sum(int(np.ldexp(float(x), 50)) for x in (hi, lo)) << (unit - 50)
        assert 0.9 * gap < abs(T - R) < 1.1 * gap
        p[b, 0, torch.from_numpy(at).cuda()] = torch.from_numpy(w).cuda()
        want.append(1 if T > R else int(at[2]))
    r = torch.full((6,), 0.5, device="cuda")
    acc, out = csbp.draft_verify(p, None, None, None, r)
    assert (acc == 0).all() and out[:, 0].tolist() == want


# --------------------------------------------------------- long key ranges
@pytest.mark.parametrize("d,Lp", [(64, 4_000_000), (128, 1_500_000)])
def test_sums_over_millions_of_keys(d, Lp):
    """Many rows and a long prefix, with values that all keys share: O is those
    values, whatever the weights.  Off by 2^-8 (P rounded to bf16), 2^-8 (O
    rounded) and 2^-9 at most for what the accumulator drops."""
    n, Hq = 912, 64
    g = gen(92)
    k = torch.empty((Lp, 1, d), dtype=torch.bfloat16, device="cuda")
    for x in k.split(1 << 20):
        x.copy_(normal(g, *x.shape) * 0.3)
    row = torch.linspace(0.25, 2.0, d, device="cuda").to(torch.bfloat16)
    row[1::2] *= -1
    v = row.expand(Lp, 1, d).contiguous()
    q = normal(g, 1, n, Hq, d)
    a = csbp.PrefixAttention(1, n, Lp, 0, Hq, 1, d)
    o, lse = a.forward(q, k, v, None, None, None)
    a.check()
    assert ((o.double() / row.double() - 1).abs() <= 2.0 ** -7 + 2.0 ** -9).all()
    for i, h in ((0, 0), (511, 63), (911, 7)):
        z = torch.logsumexp((k[:, 0].double() @ q[0, i, h].double()) * d ** -0.5, 0)
        assert abs(float(lse[0, h, i]) - float(z)) <= 2.0 ** -13


def row_by_row(t, got, own_len, causal, samples, scale):
    """Sampled rows against the definition in 64 bits, on the GPU."""
    o, lse = got
    n, Hq = t["q"].shape[1:3]
    G = Hq // t["k_prefix"].shape[1]
    d = o.shape[-1]
    for b, i, h in samples:
        c = min(max(own_len[b], 0), t["k_own"].shape[1])
        c = max(min(c, c - n + i + 1), 0) if causal else c
        k, v = (torch.cat([t[x + "_prefix"][:, h // G], t[x + "_own"][b, :c, h // G]]).double()
                for x in "kv")
        q = t["q"][b, i, h].double()
        s = (k @ q) * scale
        z = torch.logsumexp(s, 0)
        p = torch.exp(s - z)
        A, want = p @ v.abs(), p @ v
        T = float((k.abs() @ q.abs()).max()) * scale
        tol = (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12 + 2 * d * 2.0 ** -24 * T) * A + 2.0 ** -8 * want.abs()
        assert ((o[b, i, h].double() - want).abs() <= tol).all(), (b, i, h)
        ztol = d * 2.0 ** -24 * T + 2.0 ** -15 + 2.0 ** -22 * abs(float(z))
        assert abs(float(lse[b, h, i]) - float(z)) <= ztol, (b, i, h)


@pytest.mark.parametrize("d,S,Lp", [(64, 700, 300_000), (128, 700, 300_000), (64, 300_000, 700)])
@pytest.mark.parametrize("causal", [False, True])
def test_jobs_cut_into_runs(d, S, Lp, causal):
    """So many rows that jobs would stay whole, over so many keys that each is cut
    into runs; the last row tile is alone; one V is not finite."""
    B, n, Hq = 17, 127, 16
    if S > Lp:
        B, n = 4, 600
    t = attn_inputs(B, n, Lp, S, Hq, 1, d, 93)
    lens = [(S - 61 * b) if b % 5 else 3 * b for b in range(B)]
    a = csbp.PrefixAttention(B, n, Lp, S, Hq, 1, d, causal=causal)
    rows = B * n * Hq
    assert a.ws.numel() >= 2 * rows * d * 4             # partials
    got = a.forward(**t, own_len=i32(lens))
    a.check()
    rng = np.random.default_rng(94)
    some = [(0, 0, 0), (B - 1, n - 1, Hq - 1), (1, 5, 3)] + [
        tuple(int(x) for x in rng.integers(0, (B, n, Hq))) for _ in range(12)]
    row_by_row(t, got, lens, causal, some, d ** -0.5)
    again = a.forward(**t, own_len=i32(lens))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    want = [x.clone() for x in got]
    b, j = 1, lens[1] - 2                               # read by its sequence's last queries
    t["v_own"][b, j] = float("nan")
    o, lse = a.forward(**t, own_len=i32(lens))
    a.check()
    reads = torch.zeros((B, n), dtype=torch.bool, device="cuda")
    reads[b] = j <= lens[b] - n + torch.arange(n, device="cuda") if causal else True
    assert torch.isnan(o[reads].float()).all() and torch.equal(lse, want[1])
    assert torch.isfinite(o[~reads].float()).all()
    # rows beside it in a row tile are summed again
    other = ((o != want[0]).flatten(2).any(-1) & ~reads).nonzero().tolist()
    row_by_row(t, (o, lse), lens, causal, [(b, i, h) for b, i in other[::37] for h in (0, 9)],
               d ** -0.5)
