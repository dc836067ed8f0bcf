"""GPU parity of the log probabilities against the f64 definition: values at the documented
2^-17 of their magnitude (2^-20 scale softcap more under a cap), tokens exactly: larger logits
first, of equal ones the lower token."""
import numpy as np
import pytest

from oracle import answer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def near(got, want, cap, scale):
    got = got.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    ok = np.isfinite(want)
    off = 2.0 ** -17 * np.abs(want[ok]) + 2.0 ** -100 + 2.0 ** -20 * scale * cap
    assert (np.abs(got[ok] - want[ok]) <= off).all(), (got[ok] - want[ok], off)


def run(gd, x, tokens, k, scale=1.0, cap=0.0, rows=None):
    """One call on x [n, V] (a device tensor, its rows possibly apart), compared row by row (all, or `rows`)."""
    n, V = x.shape
    m = tokens.shape[1]
    lp, ent = torch.full((n, m), 9.0, device="cuda"), torch.full((n + 8,), 9.0, device="cuda")
    ids = torch.full((n * k + 8,), 9, dtype=torch.int64, device="cuda")
    tops = torch.full((n * k + 8,), 9.0, device="cuda")
    gd.token_logprobs(x, tokens if m else None, lp if m else None, ent[:n], ids[:n * k].view(n, k) if k else None,
                      tops[:n * k].view(n, k) if k else None, n, V, scale=scale, softcap=cap)
    assert bool((ent[n:] == 9).all()) and bool((ids[n * k:] == 9).all()) and bool((tops[n * k:] == 9).all())
    xs, ts = x.float().cpu().numpy(), tokens.cpu().numpy()
    for r in range(n) if rows is None else rows:
        w_lp, w_ent, w_ids, w_tops = answer.logprobs(xs[r], ts[r], k, scale, cap)
        assert np.array_equal(ids[r * k:(r + 1) * k].cpu().numpy(), w_ids), r
        near(lp[r], w_lp, cap, scale)
        near(ent[r:r + 1], np.array([w_ent]), cap, scale)
        near(tops[r * k:(r + 1) * k], w_tops, cap, scale)
    return lp, ent[:n], ids[:n * k], tops[:n * k]


def given(n, V, m, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (n, m), generator=g)
    if m:
        t[0, 0] = V - 1
        t[-1, -1] = -1
        if m > 2:
            t[0, 1] = t[0, 0]        # the same token twice
            t[0, 2] = V              # one behind the vocabulary
    return t.cuda()


@pytest.mark.parametrize("V", [1, 2, 7, 63, 64, 65, 255, 1000, 2049, 8191, 8193, 16385, 50021, 131073])
@pytest.mark.parametrize("T", list(TYPES))
def test_lengths(gd, V, T):
    for n, m, k in ((1, 1, 1), (3, 4, 64), (2, 1, 0), (5, 0, 5), (1, 0, 64)):
        g = torch.Generator().manual_seed(V + n)
        x = torch.randn(n, V, generator=g).mul(3).to(TYPES[T]).cuda()
        run(gd, x, given(n, V, m, n), k)


@pytest.mark.parametrize("n,V,k", [(300, 4099, 20), (520, 33000, 5), (1500, 513, 64), (2100, 50, 3), (40, 100003, 20)])
def test_many_rows(gd, n, V, k):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, V, generator=g).mul(2).to(torch.bfloat16).cuda()
    run(gd, x, given(n, V, 1, 1), k, rows=[0, 1, n // 2, n - 1])


@pytest.mark.parametrize("V,k", [(37, 64), (5000, 64), (70001, 20), (70001, 1)])
@pytest.mark.parametrize("T", list(TYPES))
def test_orders_that_are_hard_on_a_selection(gd, V, k, T):
    """All alike, rising, falling, two values, one high run at the end, and zeros of both signs."""
    i = torch.arange(V, dtype=torch.float32)
    rows = torch.stack([torch.full((V,), 0.25), i / V * 8, -i / V * 8, (i % 2) * 3, torch.where(i > V - 40, 5.0, -1.0),
                        torch.where(i % 3 == 0, -0.0, 0.0), (i * 7919 % 64) / 8, torch.where(i % 512 < 16, 4.0, 0.0)])
    run(gd, rows.to(TYPES[T]).cuda(), given(8, V, 2, 3), k)


@pytest.mark.parametrize("T", list(TYPES))
@pytest.mark.parametrize("V", [70, 3001, 60007])
def test_banned_and_bad_logits(gd, T, V):
    """-infinity in most places, in all, in all but one; the type's lowest value as a mask, in all places too; NaN and infinities."""
    T = TYPES[T]
    g = torch.Generator().manual_seed(V)
    x = torch.randn(12, V, generator=g).to(T)
    low, inf = torch.finfo(T).min, float("inf")
    x[0, torch.rand(V, generator=g) < 0.99] = -inf
    x[1] = -inf
    x[2] = -inf
    x[2, V - 1] = -3.0
    x[3, torch.rand(V, generator=g) < 0.9] = low
    x[4] = low
    x[5] = low
    x[5, 3] = -inf
    x[6, V // 2] = float("nan")
    x[7, 0] = inf
    x[8, 1], x[8, 2] = inf, -inf
    x[9] = float("nan")
    x[10] = torch.finfo(T).max
    x[11, 5] = torch.finfo(T).max
    tokens = given(12, V, 3, 5)
    for cap, scale in ((0.0, 1.0), (30.0, 0.5)):
        run(gd, x.cuda(), tokens, 20, scale, cap)


@pytest.mark.parametrize("scale,cap", [(1.0, 0.0), (1.25, 0.0), (0.01, 0.0), (100.0, 0.0), (1.0, 30.0), (2.0, 5.0), (1.0, 1e30)])
def test_scales_and_caps(gd, scale, cap):
    for T in TYPES.values():
        g = torch.Generator().manual_seed(11)
        x = torch.randn(4, 20011, generator=g).mul(8).to(T).cuda()
        run(gd, x, given(4, 20011, 3, 2), 10, scale, cap)


def test_confident_rows(gd):
    """A token ahead of the others by 10 to 80: its log probability and the entropy keep their digits next to 0."""
    x = torch.zeros(8, 50000)
    for r in range(8):
        x[r, 777 * (r + 1)] = 10.0 * (r + 1)
    tokens = torch.tensor([[777 * (r + 1), 5] for r in range(8)]).cuda()
    run(gd, x.cuda(), tokens, 3)


@pytest.mark.parametrize("T", list(TYPES))
def test_rows_apart_and_unaligned(gd, T):
    """A vocabulary padded with NaN behind each row, rows that start at every alignment, one token's row from the middle."""
    T = TYPES[T]
    g = torch.Generator().manual_seed(3)
    for V, stride in ((5003, 5008), (5003, 5007), (64, 65), (8192, 8195), (9, 13)):
        pool = torch.full((6 * stride + 16,), float("nan"), dtype=T)
        for at in (0, 1, 3, 7):
            whole = pool.clone()
            rows = whole[at:at + 6 * stride].view(6, stride)[:, :V]
            rows.copy_(torch.randn(6, V, generator=g).to(T))
            d = whole.cuda()
            view = d[at:at + 6 * stride].view(6, stride)[:, :V]
            run(gd, view, given(6, V, 1, 1), 5)
            run(gd, view[4:5], given(1, V, 1, 1), 5)


def test_parts_that_are_asked_for(gd):
    """Each output alone equals the one of the whole call, bit for bit."""
    g = torch.Generator().manual_seed(8)
    for n, V in ((1, 50000), (70, 9001)):
        x, t = torch.randn(n, V, generator=g).cuda(), given(n, V, 2, 1)
        lp, ent, ids, tops = run(gd, x, t, 7, rows=[0])
        a, b = torch.empty_like(lp), torch.empty_like(ent)
        gd.token_logprobs(x, t, a, None, None, None, n, V)
        gd.token_logprobs(x, None, None, b, None, None, n, V)
        c, d = torch.empty(n, 7, dtype=torch.int64, device="cuda"), torch.empty(n, 7, device="cuda")
        gd.token_logprobs(x, None, None, None, c, d, n, V)
        assert torch.equal(a, lp) and torch.equal(b, ent) and torch.equal(c.view(-1), ids) and torch.equal(d.view(-1), tops)


def test_far_rows(gd):
    """Rows past 2^32 bytes of logits."""
    n, V = 36, 1 << 26
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    x.fill_(-2.0)
    x[:, 12345] = 20.0
    x[n - 1, V - 1] = 25.0
    t = torch.tensor([[12345]] * (n - 1) + [[V - 1]]).cuda()
    lp, ent = torch.empty(n, 1, device="cuda"), torch.empty(n, device="cuda")
    ids, tops = torch.empty(n, 2, dtype=torch.int64, device="cuda"), torch.empty(n, 2, device="cuda")
    gd.token_logprobs(x, t, lp, ent, ids, tops, n, V)
    s = (V - 1) * np.exp(-22.0)
    near(lp[0], np.array([-np.log1p(s)]), 0, 1)
    assert ids[0].tolist() == [12345, 0] and ids[n - 1].tolist() == [V - 1, 12345]
    s = (V - 2) * np.exp(-27.0) + np.exp(-5.0)
    near(lp[n - 1], np.array([-np.log1p(s)]), 0, 1)


def test_streams_and_graphs(gd):
    """On the user's stream, and captured twice on one workspace, replayed in turns with eager calls between."""
    g = torch.Generator().manual_seed(1)
    sizes = [(2, 60000), (9, 30000)]
    xs = [torch.randn(n, V, generator=g).cuda() for n, V in sizes]
    ts = [given(n, V, 1, 2) for n, V in sizes]
    need = max(gd.token_logprobs_workspace_bytes(n, V, 5) for n, V in sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    def outs(n):
        return (torch.zeros(n, 1, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, 5, dtype=torch.int64, device="cuda"),
                torch.zeros(n, 5, device="cuda"))

    def call(j, o):
        gd.token_logprobs(xs[j], ts[j], *o, *sizes[j], workspace=ws)
        return o
    want = [call(j, outs(sizes[j][0])) for j in range(2)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [call(j, outs(sizes[j][0])) for j in range(2)]
    s.synchronize()
    assert all(torch.equal(a, b) for o, w in zip(got, want) for a, b in zip(o, w))
    kept, graphs = [outs(sizes[j][0]) for j in range(2)], []
    for j in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(j, kept[j])
        graphs.append(graph)
    for i in range(6):
        for o in kept:
            for t in o:
                t.zero_()
        for j in ((0, 1) if i % 2 else (1, 0)):
            graphs[j].replay()
        assert all(torch.equal(a, b) for o, w in zip(kept, want) for a, b in zip(o, w)), i
        assert all(torch.equal(a, b) for a, b in zip(call(0, outs(2)), want[0]))


@pytest.mark.parametrize("scale,cap", [(1e30, 0.0), (1.0, 1e30), (1e-40, 0.0), (1.0, 1e-4), (1e30, 1e-4), (1e-30, 1e30)])
def test_scales_and_caps_at_their_limits(gd, scale, cap):
    """Ties, zeros, a banned token and wide logits; equal logits stay equally likely whatever the scale."""
    V = 5003
    x = torch.zeros(5, V)
    x[1, 7], x[1, 9] = 2.0, 2.0
    x[2] = torch.linspace(-30, 30, V)
    x[3] = -1e30
    x[3, 5] = 1e30
    x[4, ::2] = -float("inf")
    x = x.cuda()
    lp, ent = torch.empty(5, 1, device="cuda"), torch.empty(5, device="cuda")
    ids, tops = torch.empty(5, 3, dtype=torch.int64, device="cuda"), torch.empty(5, 3, device="cuda")
    gd.token_logprobs(x, torch.tensor([[7]] * 5, device="cuda"), lp, ent, ids, tops, 5, V, scale=scale, softcap=cap)
    for r in range(5):
        w_lp, w_ent, w_ids, w_tops = answer.logprobs(x[r].cpu().numpy(), np.array([7]), 3, scale, cap)
        assert np.array_equal(ids[r].cpu().numpy(), w_ids)
        # what lies past f32's range, 2 (1 - 2^-25) 2^127, is rounded to -infinity
        w_lp, w_tops = (np.where(w <= -(2 - 2.0 ** -24) * 2.0 ** 127, -np.inf, w) for w in (w_lp, w_tops))
        near(lp[r], w_lp, cap, scale)
        near(ent[r:r + 1], np.array([w_ent]), cap, scale)
        near(tops[r], w_tops, cap, scale)


@pytest.mark.parametrize("V", [1 << 18, 1 << 20, 1 << 22, 1 << 24])
@pytest.mark.parametrize("high", [3.5, 6.25])
def test_sums_of_long_rows(gd, V, high):
    """Rows that are not cut, equal logits below one that every wave meets first: their terms all round the same way. With a
    token 30 ahead of them, whose log probability is the sum itself, and without."""
    n = 257
    T = torch.float16
    x = torch.zeros(n, V, dtype=T, device="cuda")
    at = [100, 700, 1300, 1900]   # one of each wave's first vectors
    x[:, at] = high
    lp, ent = torch.empty(n, 1, device="cuda"), torch.empty(n, device="cuda")
    for ahead in (False, True):
        token = V // 2 + 1700 if ahead else at[0]
        if ahead:
            x[:, token] = 30.0
            s = (V - 5) * np.exp(-30.0) + 4 * np.exp(high - 30.0)
            d = 30 * (V - 5) * np.exp(-30.0) + (30 - high) * 4 * np.exp(high - 30.0)
        else:
            s, d = 3 + (V - 4) * np.exp(-high), high * (V - 4) * np.exp(-high)
        gd.token_logprobs(x, torch.full((n, 1), token, device="cuda"), lp, ent, None, None, n, V)
        for r in (0, n - 1):
            near(lp[r], np.array([-np.log1p(s)]), 0, 1)
            near(ent[r:r + 1], np.array([np.log1p(s) + d / (1 + s)]), 0, 1)


@pytest.mark.parametrize("scale", [1e-36, 1e-37, 1e-38])
def test_logits_whose_differences_leave_f32(gd, scale):
    """Scales so small that logits of both ends of f32's range are next to each other."""
    V = 5003
    g = torch.Generator().manual_seed(1)
    x = torch.empty(6, V)
    x[0], x[0, 4000] = -2.9e38, 3e38
    x[1], x[1, 7] = -3.4e38, 3.4e38
    x[2] = torch.rand(V, generator=g).mul(2).sub(1) * 3.4e38
    x[3] = torch.linspace(-3.4e38, 3.4e38, V)
    x[4], x[4, ::2] = 3.3e38, -float("inf")
    x[4, 1] = -3.3e38
    x[5] = -3.4e38
    run(gd, x.cuda(), given(6, V, 3, 2), 5, scale)
    run(gd, x[3:4].cuda(), given(1, V, 1, 2), 5, scale)


@pytest.mark.parametrize("cap,size,scale", [(cap, size, scale) for cap in (1e4, 1e6, 1e10, 1e30)
                                            for size, scale in ((50.0, 1.0), (50.0, 0.5), (3000.0, 0.01), (1e8, 1e-6), (1e9, 1e-7))
                                            if cap >= 20 * size])
def test_caps_far_above_the_logits(gd, cap, size, scale):
    """A cap of 20 times the logits and more: they are held to 2^-20 of the largest of them (every value in z comes from at most 8
    roundings, 2^-21 of itself, and is taken against the largest's)."""
    V = 9001
    g = torch.Generator().manual_seed(3)
    x = torch.rand(6, V, generator=g).mul(2).sub(1).mul(size)
    x[1, ::3] = -float("inf")
    x[2] = size
    x[3] = -size
    x[3, 5] = size
    x[4] = x[4].sort().values
    x[5, 7] = 2e30 if cap == 1e30 else x[5, 7]
    x = x.cuda()
    for n, rows in ((6, range(5 + (cap < 1e30))), (300, [0, 4, 299])):
        many = x.repeat(n // 6, 1).contiguous()
        lp, ent = torch.empty(n, 1, device="cuda"), torch.empty(n, device="cuda")
        gd.token_logprobs(many, torch.full((n, 1), 11, device="cuda"), lp, ent, None, None, n, V, scale=scale, softcap=cap)
        assert not bool(lp.isnan().any()) and not bool(ent.isnan().any())
        for r in rows:
            w_lp, w_ent, _, _ = answer.logprobs(many[r].cpu().numpy(), np.array([11]), 0, scale, cap)
            if r % 6 != 5 or cap < 1e30:
                near(lp[r], w_lp, size, scale)
                near(ent[r:r + 1], np.array([w_ent]), size, scale)


# Scales, leading logits and the others, 50 to 62 below in z: where f32's (x - top) c, c = f32(scale log2 e), is off by 0.95
# to 1.28 times the bound, in both directions.
FAR = [(1.0, 60.0, 0.0), (0.7123311758041382, 3.426105499267578, -66.76596069335938),
       (1.4191744327545166, 2.1121349334716797, -33.11961364746094), (0.7089429497718811, 8.91403579711914, -70.07681274414062),
       (1.486048698425293, 2.554197311401367, -35.12963104248047), (1.408717155456543, 3.893655776977539, -38.69828796386719),
       (1.456974983215332, 8.258298873901367, -32.92291259765625), (1.3893790245056152, 9.705148696899414, -34.919105529785156)]


@pytest.mark.parametrize("scale,top,rest", FAR)
def test_tokens_far_ahead(gd, scale, top, rest):
    """The leading token first, in the middle and last, of one wave's rows, rows cut into parts and long whole ones, banned
    tokens among them."""
    for n, V in ((1, 256), (1, 50000), (300, 50000)):
        for place in (0, V // 2, V - 1):
            x = torch.full((n + 1, V), rest, device="cuda")
            x[-1, 5::7] = -float("inf")
            x[:, place] = top
            tokens = torch.tensor([[place, 6]] * (n + 1), device="cuda")
            run(gd, x, tokens, 1, scale, rows=[0, n])


def test_rows_past_one_grid(gd):
    """More rows than a launch takes: all outputs beside the borders."""
    n, V, k, m = 2 * 65535 + 3, 37, 3, 2
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, V, generator=g).mul(3).half().cuda()
    tokens = torch.randint(-1, V, (n, m), generator=g).cuda()
    run(gd, x, tokens, k, rows=[0, 1, 65533, 65534, 65535, 65536, 131069, 131070, 131071, n - 1])


@pytest.mark.parametrize("m", [256, 257, 1000])
def test_many_tokens_of_a_row(gd, m):
    """More given tokens than a workgroup has threads, of whole rows and of rows cut into parts."""
    for n, V in ((3, 1000), (2, 50021), (300, 3001)):
        g = torch.Generator().manual_seed(m)
        x = torch.randn(n, V, generator=g).mul(3).cuda()
        run(gd, x, given(n, V, m, m), 2, rows=[0, n - 1])


@pytest.mark.parametrize("cap", [1e-4, 1e-3, 1.0, 4e3, 5e3, 1e5, 1e8, 1e12, 1e30])
def test_caps_next_to_the_logits(gd, cap):
    """Logits up to the cap and up to twice it, at every magnitude of both that is accepted."""
    V, scale = 9001, 10.0 / cap
    g = torch.Generator().manual_seed(6)
    for most in (0.1, 0.69, 2.0):
        x = torch.rand(3, V, generator=g).mul(2).sub(1).mul(most * cap).cuda()
        run(gd, x, given(3, V, 2, 2), 3, scale, cap)
        run(gd, x.repeat(100, 1).contiguous(), given(300, V, 2, 2), 3, scale, cap, rows=[0, 1, 2])


@pytest.mark.parametrize("V", [3, 5003, 50021])
def test_tokens_outside_the_vocabulary_are_padding(gd, V):
    """Of whole rows and of rows cut into parts, of rows that hold a NaN or an infinity too."""
    x = torch.zeros(5, V)
    x[1, 0], x[2, V - 1], x[3] = float("nan"), float("inf"), -float("inf")
    tokens = torch.tensor([[-1, V, 1, V + 1, 1 << 40, -(1 << 40)]] * 5).cuda()
    run(gd, x.cuda(), tokens, 2)
