"""Cases for measuring the generation operators: a quantised paged K/V cache,
attention of a batch that shares a prefix, and verification of drafted tokens.

A block-diffusion model generates block by block: a batch of continuations of
one prompt keeps its clean K/V in an E4M3 cache (`cache_write`), reads it back
to bf16 once per block (`cache_read`), runs every denoising step's M queries
against the shared prefix and the sequence's own keys (`attn_prefix`), and,
where a drafter proposed the block, keeps the drafts that the target's
probabilities accept (`draft_verify`).  A speculative step of one token per
sequence is the same with one query.

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
def _attn(name, B, n, Lp, S, Hq, Hkv, d, causal=False):
    return dict(name=name, op="attn_prefix", B=B, n=n, Lp=Lp, S=S, Hq=Hq, Hkv=Hkv, d=d,
                causal=causal)


def _cache(name, op, B, rows, length, page, Hkv, d):
    return dict(name=name, op=op, B=B, rows=rows, length=length, page=page, Hkv=Hkv, d=d)


def _verify(name, B, K, V):
    return dict(name=name, op="draft_verify", B=B, K=K, V=V)


def listed():
    return [
        # a small model, a few drafted tokens checked causally: latency
        _attn("attn_small_causal", 3, 5, 1000, 77, 2, 2, 64, causal=True),
        # one token per sequence after a medium prompt (GQA 32/8)
        _attn("attn_token", 8, 1, 8192, 256, 32, 8, 128),
        # one token per sequence, many sequences, a long prompt (GQA 32/4)
        _attn("attn_token_long", 61, 1, 131072, 500, 32, 4, 128),
        # a denoising step of 32-token blocks at the dense 14B layer (GQA 40/8)
        _attn("attn_block", 16, 32, 16384, 1024, 40, 8, 128),
        # the drafter's 16-token blocks over a million-token context
        _attn("attn_drafter_1m", 4, 16, 1048576, 64, 32, 8, 128),
        # one new token per sequence is written
        _cache("write_token", "cache_write", 8, 1, 1000, 64, 8, 128),
        # a prompt is written, with its last page partly filled
        _cache("write_prompt", "cache_write", 2, 65521, 65600, 64, 8, 128),
        # the keys of a few short sequences come back
        _cache("read_short", "cache_read", 5, 200, 300, 16, 2, 64),
        # a long shared prefix comes back once for a block
        _cache("read_prefix", "cache_read", 1, 131072, 131072, 64, 8, 128),
        # a few sequences, a 32K vocabulary
        _verify("verify_small", 3, 4, 32768),
        # a full serving batch: 16-token drafts, the 14B head's 128K vocabulary
        _verify("verify_batch", 96, 16, 131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_prefix", "attn_prefix", "cache_write", "cache_read", "draft_verify"])
    if op == "attn_prefix":
        Hq, Hkv = rng.choice([(2, 2), (8, 1), (12, 4), (40, 8), (32, 8), (32, 4), (14, 2)])
        d = rng.choice([64, 128, 128])
        n = rng.choice([1, 1, _log(rng, 2, 64)])
        B = _log(rng, 1, 64)
        most = 1 << 20
        # rows x keys stay below the largest listed case's
        most = max(16, min(most, (1 << 31) // (B * n * Hq)))
        case = _attn("", B, n, _log(rng, 1, most), _log(rng, 1, min(2048, most)), Hq, Hkv, d,
                     rng.random() < 0.4)
    elif op in ("cache_write", "cache_read"):
        Hkv, d = rng.choice([(1, 128), (2, 64), (4, 128), (8, 128), (3, 64)])
        B = _log(rng, 1, 64)
        rows = rng.choice([1, _log(rng, 2, max(2, 131072 // B))])
        length = rows + rng.randrange(1, 200)
        case = _cache("", op, B, rows, length, rng.choice([1, 16, 48, 64, 128]), Hkv, d)
    else:
        B, K = _log(rng, 1, 96), rng.randrange(1, 17)
        case = _verify("", B, K, _log(rng, 100, 131072))
    del case["name"]
    return case


# --------------------------------------------------------------- the inputs
def _pages(case):
    return -(-case["length"] // case["page"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def whole(lo, hi, *shape, dtype=torch.int32):
        """Whole numbers lo .. hi."""
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = dict(case)
    op = case["op"]
    if op == "attn_prefix":
        B, n, Lp, S, Hq, Hkv, d = (case[x] for x in ("B", "n", "Lp", "S", "Hq", "Hkv", "d"))
        s["q"] = normal(B, n, Hq, d)
        s["k_prefix"], s["v_prefix"] = normal(Lp, Hkv, d), normal(Lp, Hkv, d)
        s["k_own"], s["v_own"] = normal(B, S, Hkv, d), normal(B, S, Hkv, d)
        # every sequence has generated its own number of tokens
        s["own_len"] = whole(0, S, B)
        if own:
            from block_diffusion_lm_gb300 import csbp
            s["handle"] = csbp.PrefixAttention(B, n, Lp, S, Hq, Hkv, d, causal=case["causal"])
    elif op in ("cache_write", "cache_read"):
        B, rows, page, Hkv, d = (case[x] for x in ("B", "rows", "page", "Hkv", "d"))
        per = _pages(case)
        pages = B * per + 3
        # pages are handed out in no order; what earlier users wrote is still there
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * per].to(torch.int32)
        s["table"] = s["table"].view(B, per)
        for x in ("k", "v"):
            s["cache_" + x] = (whole(0, 119, pages, page, Hkv, d, dtype=torch.uint8)
                               | (whole(0, 1, pages, page, Hkv, d, dtype=torch.uint8) << 7))
            s["scale_" + x] = whole(117, 121, pages, page, Hkv, d // GROUP, dtype=torch.uint8)
        s["start"] = whole(0, case["length"] - rows, B)
        s["count"] = whole((rows + 1) // 2, rows, B)
        if op == "cache_write":
            s["k"], s["v"] = normal(B, rows, Hkv, d), normal(B, rows, Hkv, d)
        else:
            s["k"] = torch.zeros((B, rows, Hkv, d), dtype=torch.bfloat16, device="cuda")
            s["v"] = torch.zeros_like(s["k"])
        if own:
            from block_diffusion_lm_gb300 import csbp
            s["handle"] = csbp.QuantCache(pages, page, Hkv, d, storage=(
                s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"]))
    else:
        B, K, V = case["B"], case["K"], case["V"]
        logits = torch.randn((B, K + 1, V), generator=g, device="cuda") * 2.5
        s["p"] = torch.softmax(logits, -1)
        logits = logits[:, :K] + torch.randn((B, K, V), generator=g, device="cuda") * 0.7
        s["q"] = torch.softmax(logits, -1)
        del logits
        s["token"] = torch.multinomial(s["q"].view(B * K, V), 1, generator=g).view(B, K).to(
            torch.int32)
        s["u"], s["r"] = uniform(B, K), uniform(B)
        s["length"] = whole((K + 1) // 2, K, B)   # some sequences drafted fewer
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------ the operators
def run(s):
    op = s["op"]
    if own:
        from block_diffusion_lm_gb300 import csbp
        if op == "attn_prefix":
            return s["handle"].forward(s["q"], s["k_prefix"], s["v_prefix"], s["k_own"],
                                       s["v_own"], s["own_len"])
        if op == "cache_write":
            s["handle"].write(s["k"], s["v"], s["table"], s["start"], s["count"])
            return _cache_values(s)
        if op == "cache_read":
            return s["handle"].read(s["table"], s["start"], s["count"], out=(s["k"], s["v"]))
        return csbp.draft_verify(s["p"], s["q"], s["token"], s["u"], s["r"], s["length"])
    if op == "attn_prefix":
        return _plain_attn(s)
    if op == "cache_write":
        return _plain_write(s)
    if op == "cache_read":
        return _plain_read(s)
    return _plain_verify(s)


def _cache_values(s):
    """The cache's codes as the values they stand for, and its scales' exponents."""
    return {"k": s["cache_k"].view(torch.float8_e4m3fn), "k_scale": s["scale_k"],
            "v": s["cache_v"].view(torch.float8_e4m3fn), "v_scale": s["scale_v"]}


def _plain_attn(s):
    B, n, Lp, S, Hq, Hkv, d = (s[x] for x in ("B", "n", "Lp", "S", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    scale = d ** -0.5
    q = s["q"].float().view(B, n, Hkv, G, d).permute(2, 0, 1, 3, 4)        # h b i g d
    kp, vp = (s[x].float().permute(1, 0, 2) for x in ("k_prefix", "v_prefix"))   # h j d
    ko, vo = (s[x].float().permute(2, 0, 1, 3) for x in ("k_own", "v_own"))      # h b j d
    j = torch.arange(S, device=q.device)
    own_len = s["own_len"].long()
    end = own_len[:, None].expand(B, n)                                     # keys of a query
    if s["causal"]:
        end = own_len[:, None] - n + 1 + torch.arange(n, device=q.device)[None]
    reads = (j < end[..., None]) & (j < own_len[:, None, None])             # b i j
    reads = reads[None, :, :, None].expand(Hkv, B, n, G, S).reshape(Hkv, B, n * G, S)
    vo = torch.where((j < own_len[:, None])[None, :, :, None], vo, torch.zeros_like(vo))
    sp = torch.matmul(q.reshape(Hkv, B * n * G, d), kp.transpose(1, 2)) * scale
    so = torch.matmul(q.reshape(Hkv, B, n * G, d), ko.transpose(2, 3)) * scale
    so = torch.where(reads, so, torch.full_like(so, -math.inf)).view(Hkv, B * n * G, S)
    m = torch.maximum(sp.amax(-1), so.amax(-1)) if Lp else so.amax(-1)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)[..., None]
    sp, so = torch.exp(sp - base), torch.exp(so - base)
    total = sp.sum(-1) + so.sum(-1)
    o = torch.matmul(sp, vp) + torch.matmul(so.view(Hkv, B, n * G, S), vo).view(
        Hkv, B * n * G, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    lse = (base[..., 0] + torch.log(total)).view(Hkv, B, n, G)
    o = o.view(Hkv, B, n, G, d).permute(1, 2, 0, 3, 4).reshape(B, n, Hq, d)
    return o.to(torch.bfloat16), lse.permute(1, 0, 3, 2).reshape(B, Hq, n).contiguous()


def _slots(s):
    """(sequence, row) of every row that counts, and its page and place in it."""
    t = torch.arange(s["rows"], device="cuda")
    b, t = torch.nonzero(t[None] < s["count"][:, None], as_tuple=True)
    pos = s["start"].long()[b] + t
    return b, t, s["table"].long()[b, pos // s["page"]], pos % s["page"]


def _plain_write(s):
    b, t, page, place = _slots(s)
    Hkv, d = s["Hkv"], s["d"]

    def store(x, codes, scales):
        x = x[b, t].float().view(-1, Hkv, d // GROUP, GROUP)
        # the smallest power of two 2^e with max|x| <= 448 * 2^e
        frac, e = torch.frexp(x.abs().amax(-1))
        e = torch.where(frac <= 0.875, e - 9, e - 8).clamp(min=-127)
        e = torch.where(frac == 0, torch.full_like(e, -127), e)
        c = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[page, place] = c.view(-1, Hkv, d)
        scales[page, place] = (e + 127).to(torch.uint8)

    store(s["k"], s["cache_k"], s["scale_k"])
    store(s["v"], s["cache_v"], s["scale_v"])
    return _cache_values(s)


def _plain_read(s):
    b, t, page, place = _slots(s)
    Hkv, d = s["Hkv"], s["d"]

    def load(out, codes, scales):
        x = codes[page, place].view(torch.float8_e4m3fn).float().view(-1, Hkv, d // GROUP, GROUP)
        e = scales[page, place].int() - 127
        out[b, t] = torch.ldexp(x, e[..., None]).view(-1, Hkv, d).to(torch.bfloat16)

    load(s["k"], s["cache_k"], s["scale_k"])
    load(s["v"], s["cache_v"], s["scale_v"])
    return s["k"], s["v"]


def _plain_verify(s):
    B, K, V = s["B"], s["K"], s["V"]
    p, q, x = s["p"], s["q"], s["token"].long()
    i = torch.arange(K, device=p.device)
    px = torch.gather(p[:, :K], 2, x[..., None])[..., 0].double()
    qx = torch.gather(q, 2, x[..., None])[..., 0].double()
    fails = (s["u"].double() * qx >= px) | (i >= s["length"][:, None])
    a = torch.where(fails, i, torch.full_like(i, K)).amin(-1)              # accepted
    b = torch.arange(B, device=p.device)
    row = p[b, a].double()
    drafted = (a < s["length"])[:, None]
    w = torch.where(drafted, (row - q[b, a.clamp(max=K - 1)].double()).clamp(min=0), row)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, row)
    c = torch.cumsum(w, -1)
    nxt = (c <= s["r"].double()[:, None] * c[:, -1:]).sum(-1)
    j = torch.arange(K + 1, device=p.device)[None]
    x = torch.cat([x, x[:, :1]], -1)
    out = torch.where(j < a[:, None], x, torch.where(j == a[:, None], nxt[:, None], -1))
    return a.to(torch.int32), out.to(torch.int32)


# ------------------------------------------------------------------ the work
def work(case):
    op = case["op"]
    if op == "attn_prefix":
        B, n, Lp, S, Hq, Hkv, d = (case[x] for x in ("B", "n", "Lp", "S", "Hq", "Hkv", "d"))
        keys = Lp + S / 2                       # own lengths are uniform over 0 .. S
        rows = B * n * Hq
        bytes_ = (Lp + B * S / 2) * Hkv * d * 4 + rows * (4 * d + 4)
        return {"bytes": bytes_, "flops": 4.0 * d * rows * keys}
    if op in ("cache_write", "cache_read"):
        rows = case["B"] * case["rows"] * 0.75  # counts are uniform over rows / 2 .. rows
        rows = case["B"] if case["rows"] == 1 else rows
        values = 2 * rows * case["Hkv"] * case["d"]
        return {"bytes": values * (3 + 1 / GROUP), "flops": 3 * values}
    B, K, V = case["B"], case["K"], case["V"]
    # the first rejected position's two rows decide the next token
    return {"bytes": B * (8 * V + 16 * K + 8), "flops": 3 * B * V}


# ---------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn_prefix":
        return _exact_attn(s)
    if case["op"] == "cache_write":
        return _exact_write(s)
    if case["op"] == "cache_read":
        return _exact_read(s)
    return None  # whole numbers, held to the plain form alone


def _exact_attn(s):
    B, n, Lp, S, Hq, Hkv, d = (s[x] for x in ("B", "n", "Lp", "S", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.zeros((B, n, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["own_len"].tolist()
    for h in range(Hkv):
        q = s["q"][:, :, h * G:(h + 1) * G].double().reshape(B * n * G, d)
        # running maximum, sum and output of each row over pieces of the keys
        m = torch.full((B * n * G,), -math.inf, dtype=torch.float64, device="cuda")
        z = torch.zeros_like(m)
        acc = torch.zeros_like(q)

        def add(rows, k, v, ok=None):
            x = q[rows] @ k.T / math.sqrt(d)
            if ok is not None:
                x = x.masked_fill(~ok, -math.inf)
            top = torch.maximum(m[rows], x.amax(-1))
            ref = top.masked_fill(top == -math.inf, 0.0)
            old = torch.exp(m[rows] - ref)
            x = torch.exp(x - ref[:, None])
            z[rows] = z[rows] * old + x.sum(-1)
            acc[rows] = acc[rows] * old[:, None] + x @ v
            m[rows] = top

        for j in range(0, Lp, 65536):
            add(slice(None), s["k_prefix"][j:j + 65536, h].double(),
                s["v_prefix"][j:j + 65536, h].double())
        for b, c in enumerate(lens):
            if c == 0:
                continue
            ok = None
            if s["causal"]:
                last = c - n + torch.arange(n, device="cuda").repeat_interleave(G)
                ok = torch.arange(c, device="cuda")[None] <= last[:, None]
            add(slice(b * n * G, (b + 1) * n * G), s["k_own"][b, :c, h].double(),
                s["v_own"][b, :c, h].double(), ok)
        some = z > 0
        res = torch.where(some[:, None], acc / z.masked_fill(~some, 1.0)[:, None], 0.0)
        o[:, :, h * G:(h + 1) * G] = res.view(B, n, G, d)
        lse[:, h * G:(h + 1) * G] = (m + torch.log(z)).view(B, n, G).transpose(1, 2)
    return o, lse


def _e4m3_values(code):
    """The values of E4M3 codes, in 64 bits."""
    c = code.to(torch.int64)
    exp, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(exp == 0, man / 8 * 2.0 ** -6,
                      (1 + man / 8) * torch.exp2((exp - 7).double()))
    return torch.where(c >= 128, -mag, mag)


def _exact_write(s):
    out = {"k_scale": None, "v_scale": None}      # whole numbers
    Hkv, d, page = s["Hkv"], s["d"], s["page"]
    for x in ("k", "v"):
        vals = _e4m3_values(s["cache_" + x])
        for b in range(s["B"]):
            at, cnt = int(s["start"][b]), int(s["count"][b])
            pos = torch.arange(at, at + cnt, device="cuda")
            slot = s["table"][b].long()[pos // page] * page + pos % page
            a = s[x][b, :cnt].double().view(cnt, Hkv, d // GROUP, GROUP)
            top = a.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(min=-127)
            a = a / torch.exp2(e)
            # E4M3 keeps 3 bits after the leading one, and steps of 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
            vals.view(-1, Hkv, d)[slot] = (torch.round(a / step) * step).view(cnt, Hkv, d)
        out[x] = vals
    return out


def _exact_read(s):
    res = []
    page = s["page"]
    for x in ("k", "v"):
        out = torch.zeros_like(s[x], dtype=torch.float64)
        for b in range(s["B"]):
            at, cnt = int(s["start"][b]), int(s["count"][b])
            pos = torch.arange(at, at + cnt, device="cuda")
            slot = s["table"][b].long()[pos // page] * page + pos % page
            c = s["cache_" + x].flatten(0, 1)[slot]
            e = s["scale_" + x].flatten(0, 1)[slot].double() - 127
            out[b, :cnt] = _e4m3_values(c) * torch.exp2(e).repeat_interleave(GROUP, -1)
        res.append(out)
    return tuple(res)
