"""Cases for measuring the operators that serve from the quantised paged cache:
appending keys and values with their position rotation, attention of a few new
tokens over the cache's pages, and the same with a sliding window and first
tokens that stay visible (sinks).

A step of generation computes q, k and v of its new tokens, rotates q and k by
their positions and keeps k and v in the E4M3 cache (`cache_append`), and lets
q read the cache where it lies (`attn_paged`): one token per sequence, the
drafts that a step verifies, a block that is denoised, or a chunk of a prompt.
Layers with a sliding window read their last `window` keys and the first
`sinks` ones (`attn_window`).

`run` computes the plain form with elementary torch operations, or, where
`own` is true, calls the framework.  `exact` computes the same outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

GROUP = 32          # features that share one power-of-two scale in the cache
E4M3_MAX = 448.0    # largest E4M3 magnitude


# ---------------------------------------------------------------- the cases
def _attn(name, B, n, S, page, Hq, Hkv, d, causal, window=0, sinks=0):
    return dict(name=name, op="attn_window" if window else "attn_paged", B=B, n=n, S=S, page=page,
                Hq=Hq, Hkv=Hkv, d=d, causal=causal, window=window, sinks=sinks)


def _append(name, B, rows, length, page, Hq, Hkv, d, rot, base, interleaved=False):
    return dict(name=name, op="cache_append", B=B, rows=rows, length=length, page=page, Hq=Hq,
                Hkv=Hkv, d=d, rot=rot, base=base, interleaved=interleaved)


def listed():
    return [
        # a small model's token, short texts: latency
        _attn("paged_token_small", 3, 1, 1000, 16, 2, 2, 64, True),
        # one token for each of a serving batch, medium texts (GQA 32/8)
        _attn("paged_token", 64, 1, 8192, 64, 32, 8, 128, True),
        # one token of a few sequences over a million tokens (GQA 32/4)
        _attn("paged_token_1m", 4, 1, 1048576, 64, 32, 4, 128, True),
        # eight drafted tokens and the one before them are verified (GQA 40/8)
        _attn("paged_drafts", 16, 9, 16000, 64, 40, 8, 128, True),
        # a denoising step of 32-token blocks at the dense 14B layer
        _attn("paged_block", 16, 32, 16384, 64, 40, 8, 128, False),
        # one token of many sequences in a layer with a window of 1,024
        _attn("window_token", 61, 1, 40000, 64, 32, 8, 128, True, 1024, 4),
        # a block is denoised in such a layer, heads of 64
        _attn("window_block", 24, 16, 20000, 16, 14, 2, 64, False, 1000, 64),
        # a chunk of a long prompt in such a layer
        _attn("window_chunk", 2, 2000, 16384, 64, 40, 8, 128, True, 1024, 4),
        # one new token for each of a few sequences is kept
        _append("append_token", 8, 1, 1000, 64, 32, 8, 128, 128, 1e6),
        # a small model: heads of 64, half of each rotated, in pairs of neighbours
        _append("append_small", 5, 200, 300, 16, 14, 2, 64, 32, 1e4, True),
        # the clean blocks of a batch are kept, far into their texts
        _append("append_block", 64, 32, 400000, 64, 40, 8, 128, 128, 5e5),
        # a prompt is kept, with its last page partly filled
        _append("append_prompt", 2, 65521, 65600, 64, 32, 8, 128, 128, 1e6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_paged", "attn_paged", "attn_window", "attn_window", "cache_append"])
    page = rng.choice([1, 16, 48, 64, 128])
    if op == "cache_append":
        Hq, Hkv, d = rng.choice([(0, 1, 128), (14, 2, 64), (32, 8, 128), (12, 3, 64), (40, 8, 128),
                                 (0, 4, 96)])
        B = _log(rng, 1, 64)
        rows = rng.choice([1, _log(rng, 2, max(2, 65536 // B))])
        case = _append("", B, rows, rows + rng.choice([_log(rng, 1, 200), _log(rng, 1, 400000)]),
                       page, Hq, Hkv, d, rng.choice([d, d // 2]), rng.choice([1e4, 5e5, 1e6]),
                       rng.random() < 0.3)
        # a page table of a sequence far into its text names few thousand pages
        if page < 16:
            case["length"] = rows + rng.randrange(1, 200)
    else:
        Hq, Hkv = rng.choice([(2, 2), (8, 1), (12, 4), (40, 8), (32, 8), (32, 4), (14, 2)])
        d = rng.choice([64, 128, 128])
        n = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64)])
        window = sinks = 0
        if op == "attn_window":
            window, sinks = _log(rng, 16, 4096), rng.choice([0, 4, _log(rng, 1, 128)])
            if rng.random() < 0.3:
                n = _log(rng, 64, 2000)
        B = _log(rng, 1, 64 if n <= 64 else 4)
        # keys x heads, and rows x keys, stay below the largest listed cases'
        most = min(1 << 20, (1 << 24) // (B * Hkv), (1 << 32) // (B * n * Hq))
        S = _log(rng, min(n, most) + 1, max(n + 2, most))
        case = _attn("", B, n, S, page, Hq, Hkv, d, rng.random() < 0.6, window, sinks)
    del case["name"]
    return case


# --------------------------------------------------------------- the inputs
def _power(frac, e):
    """The smallest e' with frac 2^e <= 448 x 2^e', 0.5 <= frac < 1 or 0."""
    e = torch.where(frac <= 0.875, e - 9, e - 8).clamp(min=-127)
    return torch.where(frac == 0, torch.full_like(e, -127), e)


def _quantise(x):
    """fp32 [rows, Hkv, d] -> E4M3 codes and scale bytes."""
    g = x.view(*x.shape[:-1], -1, GROUP)
    e = _power(*torch.frexp(g.abs().amax(-1)))
    codes = torch.ldexp(g, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(x.shape), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def whole(lo, hi, *shape):
        """Whole numbers lo .. hi."""
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.int32)

    s = dict(case)
    B, page, Hq, Hkv, d = (case[x] for x in ("B", "page", "Hq", "Hkv", "d"))
    append = case["op"] == "cache_append"
    if append:
        rows, length = case["rows"], case["length"]
        s["start"] = whole(0, length - rows, B)
        s["count"] = whole((rows + 1) // 2, rows, B)
        s["k"], s["v"] = normal(B, rows, Hkv, d).bfloat16(), normal(B, rows, Hkv, d).bfloat16()
        s["q"] = normal(B, rows, Hq, d).bfloat16() if Hq else None
        half = case["rot"] // 2
        s["freq"] = [case["base"] ** (-i / half) for i in range(half)]
        s["freq_t"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
        # pages that this call does not touch are few, however far the texts go
        per = -(-length // page)
        pages = B * (rows // page + 2) + 3
        s["table"] = torch.zeros((B, per), dtype=torch.int32, device="cuda")
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        first = s["start"].long() // page
        at = first[:, None] + torch.arange(rows // page + 2, device="cuda")[None]
        there = at < per
        b = torch.arange(B, device="cuda")[:, None].expand_as(at)
        s["table"][b[there], at[there]] = ids[:at.numel()].view(at.shape)[there]
    else:
        n, S = case["n"], case["S"]
        per = -(-S // page)
        pages = B * per + 3
        # pages are handed out in no order
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(
            B, per).to(torch.int32)
        s["len"] = whole(max(1, min(n, S), S // 2), S, B)
        # some features are larger than others, and weights are far from equal
        s["q"] = (1.5 * normal(B, n, Hq, d)).bfloat16()
    # what earlier tokens (and earlier users of the pages) left there
    for x in ("k", "v"):
        s["cache_" + x] = torch.empty((pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
        s["scale_" + x] = torch.empty((pages, page, Hkv, d // GROUP), dtype=torch.uint8,
                                      device="cuda")
        size = torch.exp(0.4 * normal(Hkv, d))
        step = max(1, (1 << 27) // (page * Hkv * d))
        for i in range(0, pages, step):
            m = min(step, pages - i)
            c, e = _quantise(normal(m * page, Hkv, d) * size)
            s["cache_" + x][i:i + m] = c.view(m, page, Hkv, d)
            s["scale_" + x][i:i + m] = e.view(m, page, Hkv, d // GROUP)
    if own:
        from block_diffusion_lm_gb300 import csbp
        s["cache"] = csbp.QuantCache(pages, page, Hkv, d, storage=(
            s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"]))
        if append:
            s["rotary"] = csbp.Rotary(s["freq"], interleaved=case["interleaved"])
        else:
            s["handle"] = csbp.PagedAttention(
                B, n, per, page, Hq, Hkv, d, causal=case["causal"], window=case["window"],
                sinks=case["sinks"])
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------ the operators
def run(s):
    if s["op"] == "cache_append":
        if not own:
            return _plain_append(s)
        q = s["cache"].append(s["k"], s["v"], s["table"], s["start"], s["count"],
                              rotary=s["rotary"], q=s["q"])
        return _cache_values(s, q)
    if not own:
        return _plain_attn(s)
    return s["handle"].forward(s["q"], s["cache"], s["table"], s["len"])


def _cache_values(s, q):
    """The cache's codes as the values they stand for, its scales' exponents and
    the rotated queries."""
    out = {"k": s["cache_k"].view(torch.float8_e4m3fn), "k_scale": s["scale_k"],
           "v": s["cache_v"].view(torch.float8_e4m3fn), "v_scale": s["scale_v"]}
    if q is not None:
        out["q"] = q
    return out


def _visible(s, b, device):
    """Places of the keys that some query of sequence b reads, and whether query
    i reads them: a whole number tensor and [n, keys]."""
    n, c = s["n"], int(s["len"][b])
    first = 0
    if s["window"]:
        first = max(0, c - n - s["window"] + 1)
    j = torch.arange(first, c, device=device)
    if s["window"]:
        j = torch.cat([torch.arange(min(s["sinks"], first), device=device), j])
    at = c - n + torch.arange(n, device=device)[:, None]
    reads = torch.ones((n, j.numel()), dtype=torch.bool, device=device)
    if s["causal"]:
        reads &= j <= at
    if s["window"]:
        reads &= (at - j < s["window"]) | (j < s["sinks"])
    return j, reads


def _plain_attn(s):
    B, n, page, Hq, Hkv, d = (s[x] for x in ("B", "n", "page", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.empty((B, n, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device="cuda")

    def keys(codes, scales, slot):
        x = codes.flatten(0, 1)[slot].view(torch.float8_e4m3fn).float()
        e = scales.flatten(0, 1)[slot].int() - 127
        x = torch.ldexp(x.view(-1, Hkv, d // GROUP, GROUP), e[..., None])
        return x.view(-1, Hkv, d).transpose(0, 1)                           # h j d

    for b in range(B):
        j, reads = _visible(s, b, "cuda")
        slot = s["table"][b].long()[j // page] * page + j % page
        k, v = (keys(s["cache_" + x], s["scale_" + x], slot) for x in ("k", "v"))
        q = s["q"][b].float().view(n, Hkv, G, d).transpose(0, 1).reshape(Hkv, n * G, d)
        x = torch.matmul(q, k.transpose(1, 2)) * d ** -0.5                  # h (i g) j
        x = x.view(Hkv, n, G, -1).masked_fill_(~reads[None, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        x = torch.exp(x - m)
        z = x.sum(-1, keepdim=True)
        r = torch.matmul(x.view(Hkv, n * G, -1), v).view(Hkv, n, G, d)
        r = torch.where(z > 0, r / z, torch.zeros_like(r))
        o[b] = r.transpose(0, 1).reshape(n, Hq, d).to(torch.bfloat16)
        lse[b] = (m + torch.log(z))[..., 0].transpose(1, 2).reshape(Hq, n)
    return o, lse


def _rotate(x, angle, interleaved):
    """x [rows, heads, d] in 64 bits, angle [rows, rot / 2]."""
    half = angle.shape[1]
    rot = x[..., :2 * half]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :half], rot[..., half:])
    c, t = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = a * c - b * t, a * t + b * c
    rot = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([rot, x[..., 2 * half:]], -1)


def _plain_append(s):
    """In 64 bits: angles of far positions, and magnitudes next to where the scale
    changes."""
    page, Hkv, d = s["page"], s["Hkv"], s["d"]
    t = torch.arange(s["rows"], device="cuda")
    b, t = torch.nonzero(t[None] < s["count"][:, None], as_tuple=True)
    pos = s["start"].long()[b] + t
    slot = s["table"].long()[b, pos // page] * page + pos % page
    angle = pos.double()[:, None] * s["freq_t"]
    q = None if s["q"] is None else torch.zeros_like(s["q"])
    for i in range(0, b.numel(), 16384):
        r = slice(i, i + 16384)
        for x, codes, scales in ((s["k"], s["cache_k"], s["scale_k"]),
                                 (s["v"], s["cache_v"], s["scale_v"])):
            x = x[b[r], t[r]].double()
            if codes is s["cache_k"]:
                x = _rotate(x, angle[r], s["interleaved"])
            x = x.view(-1, Hkv, d // GROUP, GROUP)
            e = _power(*torch.frexp(x.abs().amax(-1)))
            c = torch.ldexp(x, -e[..., None]).float().to(torch.float8_e4m3fn)
            codes.flatten(0, 1)[slot[r]] = c.view(torch.uint8).view(-1, Hkv, d)
            scales.flatten(0, 1)[slot[r]] = (e + 127).to(torch.uint8)
        if q is not None:
            q[b[r], t[r]] = _rotate(s["q"][b[r], t[r]].double(), angle[r],
                                    s["interleaved"]).to(torch.bfloat16)
    return _cache_values(s, q)


# ------------------------------------------------------------------ the work
def work(case):
    B, Hq, Hkv, d = (case[x] for x in ("B", "Hq", "Hkv", "d"))
    if case["op"] == "cache_append":
        rows = B * case["rows"] * (1 if case["rows"] == 1 else 0.75)  # counts: half to all
        # bf16 read, a code and 1/32 of a scale byte written; q read and written
        values = rows * d * (2 * Hkv * (3 + 1 / GROUP) + 4 * Hq)
        return {"bytes": values, "flops": rows * (Hkv + Hq) * case["rot"] * 3}
    n, length = case["n"], case["S"] * 0.75                           # lengths: half to all
    mine = length - (n / 2 if case["causal"] else 0)                  # keys of a query
    keys = length                                                     # and of any
    if case["window"]:
        # a query's window ends at itself, or with the block
        mine = min(mine, case["window"] + case["sinks"] + (0 if case["causal"] else n / 2))
        keys = min(keys, case["window"] + case["sinks"] + n)
    rows = B * n * Hq
    return {"bytes": B * keys * Hkv * d * 2 * (1 + 1 / GROUP) + rows * (4 * d + 4),
            "flops": 4.0 * d * rows * mine}


# ---------------------------------------------------- the definitions, 64 bits
def _e4m3_values(code):
    """The values of E4M3 codes, in 64 bits."""
    c = torch.arange(256, device=code.device)
    exp, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(exp == 0, man / 8 * 2.0 ** -6,
                      (1 + man / 8) * torch.exp2((exp - 7).double()))
    return torch.where(c >= 128, -mag, mag)[code.int()]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "cache_append" else _exact_attn(s)


def _exact_attn(s):
    B, n, page, Hq, Hkv, d = (s[x] for x in ("B", "n", "page", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.zeros((B, n, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64, device="cuda")
    for b, c in enumerate(s["len"].tolist()):
        at = (c - n + torch.arange(n, device="cuda")).repeat_interleave(G)[:, None]
        low = c - n - s["window"] + 1 if s["window"] else 0
        for h in range(Hkv):
            q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(n * G, d)
            # running maximum, sum and output over pieces of the keys
            m = torch.full((n * G, 1), -math.inf, dtype=torch.float64, device="cuda")
            z, acc = torch.zeros_like(m), torch.zeros_like(q)
            for j0 in range(0, c, 65536):
                j = torch.arange(j0, min(c, j0 + 65536), device="cuda")
                j = j[(j >= low) | (j < s["sinks"])]
                if j.numel() == 0:
                    continue
                pg = s["table"][b, j // page].long()
                k, v = (_e4m3_values(s["cache_" + x][pg, j % page, h]) * torch.exp2(
                    s["scale_" + x][pg, j % page, h].double() - 127).repeat_interleave(GROUP, -1)
                    for x in ("k", "v"))
                x = q @ k.T / math.sqrt(d)
                ok = (j >= 0).expand(x.shape)
                if s["causal"]:
                    ok = ok & (j <= at)
                if s["window"]:
                    ok = ok & ((j > at - s["window"]) | (j < s["sinks"]))
                x = x.masked_fill(~ok, -math.inf)
                top = torch.maximum(m, x.amax(-1, keepdim=True))
                ref = top.masked_fill(top == -math.inf, 0.0)
                old = torch.exp(m - ref)
                x = torch.exp(x - ref)
                z = z * old + x.sum(-1, keepdim=True)
                acc = acc * old + x @ v
                m = top
            some = z > 0
            res = torch.where(some, acc / z.masked_fill(~some, 1.0), 0.0)
            o[b, :, h * G:(h + 1) * G] = res.view(n, G, d)
            lse[b, h * G:(h + 1) * G] = (m + torch.log(z)).view(n, G).T
    return o, lse


def _exact_append(s):
    """Codes stand for x 2^-e before they are rounded; scales are whole numbers."""
    out = {"k_scale": None, "v_scale": None}
    page, Hkv, d, half = s["page"], s["Hkv"], s["d"], s["rot"] // 2
    pair = torch.arange(half, device="cuda")
    first, second = (2 * pair, 2 * pair + 1) if s["interleaved"] else (pair, pair + half)
    for x in ("k", "v", "q"):
        if s[x] is None:
            continue
        vals = torch.zeros_like(s["q"], dtype=torch.float64) if x == "q" else _e4m3_values(
            s["cache_" + x])
        for b in range(s["B"]):
            at, cnt = int(s["start"][b]), int(s["count"][b])
            pos = torch.arange(at, at + cnt, device="cuda")
            y = s[x][b, :cnt].double()
            if x != "v":
                z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                pos.double()[:, None] * s["freq_t"])[:, None]
                z = z * torch.complex(y[..., first], y[..., second])
                y[..., first], y[..., second] = z.real, z.imag
            if x == "q":
                vals[b, :cnt] = y
                continue
            slot = s["table"][b].long()[pos // page] * page + pos % page
            y = y.view(cnt, Hkv, d // GROUP, GROUP)
            top = y.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(min=-127)
            vals.view(-1, Hkv, d)[slot] = (y / torch.exp2(e)).view(cnt, Hkv, d)
        out[x] = vals
    return out
