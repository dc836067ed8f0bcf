"""GPU parity of the norms behind and before a block. h is the f64 definition's rounding: an
element may be the neighbour only where the f64 value lies within 2^-45 of the border between
the two (the sums' f64 rounding), so h is held to half a step of f32 (2^-24) and 2^-45; for a
16-bit type half a step of that after it. Codes and scales are compared bit for bit with the
rule on the h that the call returned."""
import numpy as np
import pytest

from oracle import layer
from test_gpu_norm_quant import EPS, TYPES, blocks, guarded, planes_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def call(gd, form, x, post, res, w, h, n, K, **kw):
    if form == "q8_0":
        a, whole, fill = guarded(n * (K // 32) * 34, torch.uint8)
        gd.rmsnorm_sandwich_q8_0(x, post, res, w, h, a, n, K, EPS, **kw)
        assert bool((whole[a.numel():] == fill).all())
        return (a,)
    p, whole, fill = guarded(n * 8 * (K // 32), torch.int32)
    s, sw, sf = guarded(n, torch.float32)
    gd.rmsnorm_sandwich_ternary_act(x, post, res, w, h, p, s, n, K, EPS, **kw)
    assert bool((whole[p.numel():] == fill).all()) and bool((sw[n:] == sf).all())
    return p, s


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def definition(x, post, res, gate, index, rs, bs):
    x, post, res, gate = f64(x), f64(post), f64(res), f64(gate)
    eps, rs, bs = (float(np.float32(v)) for v in (EPS, rs, bs))
    u = x
    if post is not None:
        u = x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * post
    if gate is not None:
        g = gate[index.clip(0, len(gate) - 1)] * ((index >= 0) & (index < len(gate)))[:, None]
        u = u * g
    return rs * res + bs * u


def check(form, got, h, w, T, want):
    hf = h.float().cpu().numpy()
    fi = torch.finfo(T)
    off = np.abs(want) * (2.0 ** -24 + 2.0 ** -45) + 2.0 ** -149
    if T != torch.float32:
        off = off + (np.abs(want) + off) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2
    assert (np.abs(hf - want) <= off).all()
    n, K = hf.shape
    codes, scale = layer.rmsnorm_codes(hf, w.cpu().numpy(), EPS, 32 if form == "q8_0" else K)
    if form == "q8_0":
        assert np.array_equal(got[0].cpu().numpy(), blocks(codes, scale))
    else:
        assert np.array_equal(got[0].cpu().numpy().view(np.uint32), planes_of(codes))
        assert np.array_equal(got[1].cpu().numpy(), scale[:, 0])


# One wave a row and eight, rows that fill the registers and rows past them.
@pytest.mark.parametrize("n,K", [(1, 32), (3, 96), (2, 4096), (5, 2560), (2, 4128), (3, 8192), (2, 8224), (1, 20000), (1030, 4096), (1024, 2560),
                                 (1025, 512), (1030, 992), (1024, 1056)])
@pytest.mark.parametrize("form", ["q8_0", "ternary"])
@pytest.mark.parametrize("T", TYPES)
def test_sandwich(gd, n, K, form, T):
    """Gates of each kind in turn, with and without the norm behind the block; h kept or not, in place of either input."""
    g = torch.Generator().manual_seed(n * 31 + K)
    x, res = (torch.randn(n, K, generator=g).mul(s).to(T).cuda() for s in (3, 1.5))
    w, post = (torch.randn(K, generator=g).mul(0.2).add(1).cuda() for _ in range(2))
    many = min(n, 3)
    kinds = [(post, None, None), (None, None, None), (post, 1, None), (post, n, None),
             (None, many, torch.randint(-1, many + 1, (n,), generator=g).int())]
    for i, (p, n_gates, index) in enumerate(kinds):
        gate = None if n_gates is None else torch.randn(n_gates, K, generator=g).to(T).cuda()
        rs, bs = ((1.0, 1.0), (0.75, -1.5), (0.0, 0.3))[i % 3]
        kw = dict(gate=gate, gate_index=None if index is None else index.cuda(), residual_scale=rs, block_scale=bs)
        which = index.numpy() if index is not None else np.zeros(n, int) if n_gates == 1 else np.arange(n)
        want = definition(x, p, res, gate, which, rs, bs)
        h, whole, fill = guarded(n * K, T)
        got = call(gd, form, x, p, res, w, h.view(n, K), n, K, **kw)
        assert bool((whole[n * K:] == fill).all())
        check(form, got, h.view(n, K), w, T, want)
        bare = call(gd, form, x, p, res, w, None, n, K, **kw)
        for place in (0, 1):
            both = [x.clone(), res.clone()]
            over = call(gd, form, both[0], p, both[1], w, both[place], n, K, **kw)
            assert torch.equal(both[place], h.view(n, K)) and torch.equal(both[1 - place], (res, x)[place])
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(got, bare, over))


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_plain_block_equals_the_norm_without_it(gd, form):
    """Without post_weight, gate and scales the codes, scales and h are those of the residual norm."""
    for T in TYPES:
        n, K = 7, 2560
        g = torch.Generator().manual_seed(4)
        x, res = (torch.randn(n, K, generator=g).to(T).cuda() for _ in range(2))
        w = torch.randn(K, generator=g).add(1).cuda()
        h, h2 = torch.empty_like(x), torch.empty_like(x)
        got = call(gd, form, x, None, res, w, h, n, K)
        if form == "q8_0":
            old = (torch.empty_like(got[0]),)
            gd.rmsnorm_q8_0(x, res, w, h2, old[0], n, K, EPS)
        else:
            old = torch.empty_like(got[0]), torch.empty_like(got[1])
            gd.rmsnorm_ternary_act(x, res, w, h2, *old, n, K, EPS)
        assert torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(got, old))


def test_zero_and_extreme_rows(gd):
    """Rows of zeros (scale 0, zero codes), magnitudes whose squares leave f32, blocks of zeros within a row."""
    n, K = 5, 512
    g = torch.Generator().manual_seed(9)
    x, res = torch.randn(n, K, generator=g), torch.randn(n, K, generator=g)
    x[0], res[0] = 0, 0
    x[1], res[1] = x[1] * 1e25, res[1] * 1e30
    x[2], res[2] = x[2] * 1e-30, res[2] * 1e-35
    x[3, :64], res[3, :64] = 0, 0
    x, res = x.cuda(), res.cuda()
    w, post = (torch.randn(K, generator=g).add(1).cuda() for _ in range(2))
    for form in ("q8_0", "ternary"):
        h = torch.empty_like(x)
        got = call(gd, form, x, post, res, w, h, n, K)
        check(form, got, h, w, torch.float32, definition(x, post, res, None, None, 1.0, 1.0))


def test_streams_and_graph(gd):
    n, K = 33, 1024
    g = torch.Generator().manual_seed(2)
    x, res = (torch.randn(n, K, generator=g).cuda() for _ in range(2))
    w, post = (torch.randn(K, generator=g).add(1).cuda() for _ in range(2))
    h, a = torch.empty_like(x), torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda")

    def run():
        gd.rmsnorm_sandwich_q8_0(x, post, res, w, h, a, n, K, EPS)
    run()
    want = h.clone(), a.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        h.zero_(), a.zero_()
        run()
    s.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(a, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        h.zero_(), a.zero_()
        graph.replay()
        assert torch.equal(h, want[0]) and torch.equal(a, want[1])


@pytest.mark.parametrize("K", [96, 4096, 8224, 20000])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_rows_that_take_nothing_of_their_block(gd, K, post, eps):
    """Whatever the block's output and the gates hold there: NaN, infinities, zeros (with eps = 0 too)."""
    n, T = 6, torch.float16
    g = torch.Generator().manual_seed(K)
    x, res = (torch.randn(n, K, generator=g).to(T) for _ in range(2))
    gate = torch.randn(2, K, generator=g).to(T)
    gate[0, 1] = float("inf")
    x[0], x[1, K - 1], x[2, 0], x[3] = float("nan"), float("inf"), -float("inf"), 0
    index = torch.tensor([-1, 2, -7, 1 << 30, 1, -1], dtype=torch.int32)
    x, res, gate, index = (t.cuda() for t in (x, res, gate, index))
    w = torch.ones(K, device="cuda")
    h, a = torch.empty_like(x), torch.empty(n * K // 32 * 34, dtype=torch.uint8, device="cuda")
    gd.rmsnorm_sandwich_q8_0(x, w if post else None, res, w, h, a, n, K, eps, gate=gate, gate_index=index, residual_scale=0.5)
    rows = [0, 1, 2, 3, 5]
    want = (res.double() * 0.5).to(T)
    assert torch.equal(h[rows], want[rows]) and not torch.equal(h[4], want[4]) and bool(h[4].isfinite().all())
    alone = torch.empty_like(a)
    gd.rmsnorm_q8_0(want, None, w, None, alone, n, K, eps)
    assert torch.equal(a.view(n, -1)[rows], alone.view(n, -1)[rows])


@pytest.mark.parametrize("n,K", [(3, 96), (3, 4096), (3, 8224), (1030, 512), (1030, 1056)])
@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_blocks_of_zeros_without_eps(gd, n, K, form):
    """A row whose block put out zeros adds nothing to the stream where eps is 0, as where it is not."""
    for T in TYPES:
        g = torch.Generator().manual_seed(n + K)
        x, res = (torch.randn(n, K, generator=g).to(T).cuda() for _ in range(2))
        w, post = (torch.randn(K, generator=g).add(1).cuda() for _ in range(2))
        gate = torch.randn(1, K, generator=g).to(T).cuda()
        x[1] = 0
        h = torch.empty_like(x)
        outs = []
        for h_out in (h, None):
            out = (torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda"),) if form == "q8_0" else \
                (torch.empty(n * 8 * (K // 32), dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda"))
            of = gd.rmsnorm_sandwich_q8_0 if form == "q8_0" else gd.rmsnorm_sandwich_ternary_act
            of(x, post, res, w, h_out, *out, n, K, 0.0, gate=gate, residual_scale=0.75)
            outs.append(out)
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        want = (res[1].double() * 0.75).float().to(T)
        assert torch.equal(h[1], want) and bool(h.isfinite().all())
        alone = [torch.empty(o.numel() // n, dtype=o.dtype, device="cuda") for o in outs[0]]
        (gd.rmsnorm_q8_0 if form == "q8_0" else gd.rmsnorm_ternary_act)(want, None, w, None, *alone, 1, K, 0.0)
        assert all(torch.equal(a.view(n, -1)[1], b) for a, b in zip(outs[0], alone))


@pytest.mark.parametrize("n,K", [(3, 96), (3, 4096), (3, 8224), (1030, 512), (1030, 1056)])
@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_rows_without_a_gate_take_nothing_of_the_weight_behind_the_block(gd, n, K, form):
    """h = residual_scale residual there, whatever post_weight holds (infinities and NaN)."""
    for T in TYPES:
        g = torch.Generator().manual_seed(n + K)
        x, res = (torch.randn(n, K, generator=g).to(T).cuda() for _ in range(2))
        w, post = (torch.randn(K, generator=g).add(1).cuda() for _ in range(2))
        post[1], post[K - 1] = float("inf"), float("nan")
        gate = torch.randn(1, K, generator=g).to(T).cuda()
        index = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        h = torch.empty_like(x)
        got = call(gd, form, x, post, res, w, h, n, K, gate=gate, gate_index=index, residual_scale=0.75)
        check(form, got, h, w, T, 0.75 * f64(res))
        bare = call(gd, form, x, post, res, w, None, n, K, gate=gate, gate_index=index, residual_scale=0.75)
        assert all(torch.equal(a, b) for a, b in zip(got, bare))
