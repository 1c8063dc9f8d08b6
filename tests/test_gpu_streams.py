"""Calls on a stream that is named, while the current stream is busy: what the
binding allocates and fills belongs to the named stream, and what a handle
filled when it was made is there for any stream.

Every check is bit by bit against the same call on the current stream.  The
current stream is kept busy with matrix products, long enough (tens of
milliseconds) that a fill behind them would land after the kernel.
"""
import pytest
import torch

from block_diffusion_lm_gb300 import csbp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from block_diffusion_lm_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def busy():
    """Keeps the current stream busy for some tens of milliseconds."""
    x = torch.zeros((8192, 8192), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)

    def run():
        for _ in range(50):
            torch.mm(x, x, out=y)

    run()
    torch.cuda.synchronize()
    return run


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pending_blocks(like, busy):
    """Free memory of the sizes of `like` whose last user, a fill, waits behind
    the current stream's work."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in like]
    busy()
    for t in old:
        t.fill_(7)


def flat(x):
    """The tensors of an output (tuples, dicts, None)."""
    if x is None:
        return []
    if isinstance(x, dict):
        return [t for k in sorted(x) for t in flat(x[k])]
    return [x] if isinstance(x, torch.Tensor) else [t for y in x for t in flat(y)]


def on_a_named_stream(call, busy):
    """`call(stream)` allocates its outputs; compared with `call(None)`."""
    want = [t.clone() for t in flat(call(None))]
    pending_blocks(want, busy)
    side = torch.cuda.Stream()
    got = flat(call(side))
    torch.cuda.synchronize()
    for a, b in zip(want, got, strict=True):
        assert torch.equal(a, b)
    # and the memory stays with the reader on the current stream
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    busy()
    seen = [t.clone() for t in flat(got)]
    shapes = [t.shape for t in flat(got)]
    types = [t.dtype for t in flat(got)]
    del got
    with torch.cuda.stream(side):
        for s, d in zip(shapes, types):
            torch.empty(s, dtype=d, device="cuda").fill_(9)
    torch.cuda.synchronize()
    for a, b in zip(want, seen, strict=True):
        assert torch.equal(a, b)


# ------------------------------------------------------ generation operators
def filled_cache(B, rows, page, Hkv, d, seed):
    n = -(-rows // page)
    c = csbp.QuantCache(B * n, page, Hkv, d)
    table = torch.arange(B * n, device="cuda").int().view(B, n)
    c.write(normal(seed, B, rows, Hkv, d), normal(seed + 1, B, rows, Hkv, d), table, i32([0] * B))
    return c, table


@pytest.mark.parametrize("B,rows", [(3, 40), (2, 5000)])
def test_cache_read(B, rows, busy):
    c, table = filled_cache(B, rows, 16, 4, 128, 1)
    start, count = i32([0] * B), i32([rows - 3 * b for b in range(B)])
    on_a_named_stream(lambda st: c.read(table, start, count, rows=rows, stream=st), busy)


@pytest.mark.parametrize("B,n", [(2, 3), (16, 64)])
def test_prefix_attention(B, n, busy):
    Lp, S, Hq, Hkv, d = 2000, 100, 8, 2, 128
    a = csbp.PrefixAttention(B, n, Lp, S, Hq, Hkv, d)
    args = (normal(3, B, n, Hq, d), normal(4, Lp, Hkv, d), normal(5, Lp, Hkv, d),
            normal(6, B, S, Hkv, d), normal(7, B, S, Hkv, d), i32([S - b for b in range(B)]))
    on_a_named_stream(lambda st: a.forward(*args, stream=st), busy)


@pytest.mark.parametrize("B,K", [(3, 4), (700, 900)])
def test_draft_verify(B, K, busy):
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    V = 33
    p = torch.rand((B, K + 1, V), generator=g, device="cuda")
    q = torch.rand((B, K, V), generator=g, device="cuda")
    x = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
    u, r = (torch.rand(s, generator=g, device="cuda") for s in ((B, K), (B,)))
    on_a_named_stream(lambda st: csbp.draft_verify(p, q, x, u, r, stream=st), busy)


# ------------------------------------------------- handles made while busy
def test_a_new_cache_is_ready_for_another_stream(busy):
    k, v = normal(10, 2, 40, 2, 64), normal(11, 2, 40, 2, 64)
    table, start = torch.arange(6, device="cuda").int().view(2, 3), i32([0, 0])
    old = csbp.QuantCache(6, 16, 2, 64)
    old.write(k, v, table, start)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    new = csbp.QuantCache(6, 16, 2, 64)
    new.write(k, v, table, start, stream=side)
    torch.cuda.synchronize()
    for a, b in zip((old.k, old.v, old.k_scale, old.v_scale),
                    (new.k, new.v, new.k_scale, new.v_scale)):
        assert torch.equal(a, b)


def test_a_new_workspace_is_ready_for_another_stream(busy):
    """Its status word above all: the memory held something else before."""
    shape = (2, 3, 4096, 130, 8, 2, 128)
    args = (normal(12, 2, 3, 8, 128), normal(13, 4096, 2, 128), normal(14, 4096, 2, 128),
            normal(15, 2, 130, 2, 128), normal(16, 2, 130, 2, 128), i32([130, 7]))
    first = csbp.PrefixAttention(*shape)
    want = first.forward(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # (not the default stream: the status word is read behind its work anyway)
    with torch.cuda.stream(torch.cuda.Stream()):
        before = torch.full_like(first.ws, 1)
        torch.cuda.synchronize()
        del before
        busy()
        a = csbp.PrefixAttention(*shape)
        out = a.forward(*args, stream=side)
        a.check(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_a_handle_can_be_made_under_capture():
    q, k, v = normal(17, 1, 2, 2, 64), normal(18, 300, 2, 64), normal(19, 300, 2, 64)
    want = csbp.PrefixAttention(1, 2, 300, 0, 2, 2, 64).forward(q, k, v, None, None, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = csbp.PrefixAttention(1, 2, 300, 0, 2, 2, 64)
        got = a.forward(q, k, v, None, None, None)
    graph.replay()
    a.check()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


# ------------------------------------------------------- training operators
@pytest.fixture(scope="module")
def training():
    """One tile per copy: at most two addends per gradient, so results repeat."""
    shape = (1, 128, 64, 128)
    names = ("q_clean", "k_clean", "v_clean", "q_corr", "k_corr", "v_corr", "do_clean", "do_corr")
    t = {n: normal(30 + i, *shape) for i, n in enumerate(names)}
    return csbp.BlockDiffusionAttention(1, 128, 16, 64, 64, 128), t


def test_training_forward(training, busy):
    a, t = training
    on_a_named_stream(lambda st: a.forward(t, stream=st), busy)


def test_training_backward(training, busy):
    a, t = training
    out = a.forward(t)
    on_a_named_stream(lambda st: a.backward(t, out, stream=st), busy)


def test_vocab_cross_entropy(busy):
    N, Dm, V = 256, 256, 8192
    ce = csbp.VocabCrossEntropy(N, Dm, V)
    h, w = normal(40, N, Dm), normal(41, V, Dm)
    target = torch.arange(N, device="cuda").int() * 31
    on_a_named_stream(lambda st: ce(h, w, target, stream=st), busy)


def test_e4m3_decode(busy):
    x = (torch.arange(1 << 21, device="cuda") % 120).to(torch.uint8)
    on_a_named_stream(lambda st: csbp.e4m3_to_bf16(x, 0.5, stream=st), busy)


def test_a_new_training_workspace_is_ready_for_another_stream(training, busy):
    _, t = training
    want = training[0].forward(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(torch.cuda.Stream()):
        before = [torch.full_like(w, 1) for w in (training[0].ws_fwd, training[0].ws_bwd)]
        torch.cuda.synchronize()
        del before
        busy()
        a = csbp.BlockDiffusionAttention(1, 128, 16, 64, 64, 128)
        out = a.forward(t, stream=side)
        a.check(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(flat(want), flat(out), strict=True))
