"""Float64 oracle of the generation operators (quantised cache, shared-prefix
attention, draft verification), from their definitions.  NumPy and Python
integers only; shares no code with the library."""
import numpy as np


# ------------------------------------------------------------ quantised cache
def e4m3_table():
    """Value of every E4M3 code (bias 7, 3 mantissa bits, no infinities)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = np.nan if (e, m) == (15, 7) else (
            m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -mag if c & 128 else mag
    return v


def quantise(x):
    """x float64 [..., d] -> (values the codes stand for, scale bytes
    [..., d / 32]); values are code times scale."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    finite = np.isfinite(g)
    top = np.where(finite, np.abs(g), 0).max(-1)
    e = np.full(top.shape, -127, np.int64)
    for idx in np.ndindex(top.shape):
        while top[idx] > 448 * 2.0 ** int(e[idx]):
            e[idx] += 1
    grid = np.sort(e4m3_table()[:127])            # nonnegative finite values, ascending
    s = np.exp2(e.astype(np.float64))[..., None]
    a = np.where(finite, np.abs(g), 0) / s
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.clip(hi - 1, 0, None)
    up, down = grid[hi] - a, a - grid[lo]
    # nearest; a tie goes to the even mantissa, whose index is even
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    v = np.where(finite, np.copysign(grid[pick], g), np.nan) * s
    return v.reshape(x.shape), (e + 127).astype(np.uint8)


def dequantise(codes, scales):
    """Values of uint8 codes [..., d] under scale bytes [..., d / 32]."""
    s = np.exp2(scales.astype(np.float64) - 127)
    s = np.where(scales == 255, np.nan, s)
    return e4m3_table()[codes] * np.repeat(s, 32, -1)


# ---------------------------------------------------- shared-prefix attention
def prefix_attention(q, kp, vp, ko, vo, own_len, causal, scale):
    """q [B][n][Hq][d], kp/vp [Lp][Hkv][d], ko/vo [B][S][Hkv][d].  Returns
    (O, LSE [B][Hq][n], A = sum_j p_j |v_j|, Smax [B][Hq][n], the largest
    scale * sum_c |q_c k_c| of a row's keys)."""
    B, n, Hq, d = q.shape
    Hkv, S = kp.shape[1], ko.shape[1]
    G = Hq // Hkv
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    Z = np.full((B, Hq, n), -np.inf)
    T = np.zeros((B, Hq, n))
    for b in range(B):
        c = min(max(int(own_len[b]), 0), S)
        for h in range(Hq):
            hk = h // G
            k = np.concatenate([kp[:, hk], ko[b, :c, hk]])
            v = np.concatenate([vp[:, hk], vo[b, :c, hk]])
            s = q[b, :, h] @ k.T * scale
            t = np.abs(q[b, :, h]) @ np.abs(k).T * scale
            ok = np.ones(s.shape, bool)
            if causal:
                j = np.arange(c)[None]
                ok[:, kp.shape[0]:] = j <= (c - n + np.arange(n))[:, None]
            for i in range(n):
                if not ok[i].any():
                    continue
                x = s[i, ok[i]]
                m = x.max()
                w = np.exp(x - m)
                O[b, i, h] = w @ v[ok[i]] / w.sum()
                A[b, i, h] = w @ np.abs(v[ok[i]]) / w.sum()
                Z[b, h, i] = m + np.log(w.sum())
                T[b, h, i] = t[i, ok[i]].max()
    return O, Z, A, T


# --------------------------------------------------------- draft verification
def _exact(x):
    """A finite float as an integer multiple of 2^-149 x 2^-900 (exact)."""
    n, d = float(x).as_integer_ratio()
    return n * ((1 << 1100) // d)


def draft_verify(p, q, token, u, r, length):
    """One sequence, exact arithmetic: p [K+1][V], q [K][V], token/u [K]."""
    K, V = len(p) - 1, p.shape[1]
    n = min(max(int(length), 0), K)
    one = _exact(1.0)
    a = n
    for i in range(n):
        x = int(token[i])
        if not (0 <= x < V and _exact(u[i]) * _exact(q[i, x]) < _exact(p[i, x]) * one):
            a = i
            break

    def draw(w):
        total = sum(w)
        if total <= 0:
            return None
        c = 0
        for v, x in enumerate(w):
            c += x
            if c * one > _exact(r) * total:
                return v
        return None

    pa = [max(_exact(x), 0) for x in p[a]]
    nxt = None
    if a < n:
        nxt = draw([max(_exact(x) - _exact(y), 0) for x, y in zip(p[a], q[a])])
    if nxt is None:
        nxt = draw(pa)
    nxt = -1 if nxt is None else nxt
    return a, [int(t) for t in token[:a]] + [nxt] + [-1] * (K - a)


# ------------------------------------------------------------ rotary positions
def _pi(digits):
    """pi x 10^digits, by Machin's formula in integers."""
    one = 10 ** (digits + 10)

    def arccot(x):
        total = term = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    return 4 * (4 * arccot(5) - arccot(239)) // 10 ** 10


_TWO_PI = 2 * _pi(60)      # x 10^60


def angles(pos, freq):
    """pos x freq modulo 2 pi, [len(pos)][len(freq)]: the product is exact."""
    out = np.empty((len(pos), len(freq)))
    for f, x in enumerate(freq):
        n, d = float(x).as_integer_ratio()
        for i, p in enumerate(pos):
            t = int(p) * n * 10 ** 60 // d % _TWO_PI
            out[i, f] = t / 10 ** 60
    return out


def rotate(x, angle, interleaved):
    """x float64 [rows][heads][d], angle [rows][dim / 2]."""
    half = angle.shape[-1]
    y = x.copy()
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
            (slice(0, half), slice(half, 2 * half)))
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    with np.errstate(invalid="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def pair_size(x, half, interleaved):
    """|a| + |b| of the pair that each feature is in, |x| beyond the pairs."""
    n = np.abs(x)
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
            (slice(0, half), slice(half, 2 * half)))
    both = n[..., a] + n[..., b]
    n[..., a] = n[..., b] = both
    return n


# --------------------------------------------------- attention over the pages
def paged_attention(q, k, v, table, length, page_size, causal, window, sinks, scale):
    """q [B][n][Hq][d]; k, v [pages][page_size][Hkv][d], the values that the
    cache stands for.  Returns (O, LSE [B][Hq][n], A = sum_j p_j |v_j|, Smax
    [B][Hq][n], the largest scale * sum_c |q_c k_c| of a row's keys)."""
    B, n, Hq, d = q.shape
    pages, _, Hkv = k.shape[:3]
    G = Hq // Hkv
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    Z = np.full((B, Hq, n), -np.inf)
    T = np.zeros((B, Hq, n))
    for b in range(B):
        c = min(max(int(length[b]), 0), table.shape[1] * page_size)
        j = np.arange(c)
        page = table[b, j // page_size].astype(np.int64)
        there = (page >= 0) & (page < pages)
        j, page = j[there], page[there]
        kb, vb = k[page, j % page_size], v[page, j % page_size]
        for i in range(n):
            t = c - n + i
            ok = np.ones(len(j), bool)
            if causal:
                ok &= j <= t
            if window:
                ok &= (t - j < window) | (j < sinks)
            if not ok.any():
                continue
            for h in range(Hq):
                x = kb[ok, h // G] @ q[b, i, h] * scale
                m = x.max()
                w = np.exp(x - m)
                vv = vb[ok, h // G]
                O[b, i, h] = w @ vv / w.sum()
                A[b, i, h] = w @ np.abs(vv) / w.sum()
                Z[b, h, i] = m + np.log(w.sum())
                T[b, h, i] = (np.abs(kb[ok, h // G]) @ np.abs(q[b, i, h])).max() * scale
    return O, Z, A, T
