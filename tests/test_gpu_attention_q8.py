"""GPU parity of attention over the 8-bit cache, against the f64 definition.

Bars. A score is computed to 4 * 2^-22 of S = scale * sum |q k| (22 bits of q,
f32 sums), which softmax turns into the same relative error of a weight, twice
over (numerator and denominator). f32: a weight keeps 21 bits and the sums over
the at most 5000 keys here round each partial result at most 160 times: 1e-5 of
the largest |v| covers both. f16 and bf16: a weight is rounded to f16, half a
step being 2^-11 of it (2^-12 of the largest in its binade), q may lose what is
below 2^-25 of its row's largest value, and the result is rounded once, half a
step of its type: eps / 2 of it."""
import numpy as np
import pytest

from oracle import layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def chain(t):
    return (1 << (t + 1)) - 1


class Case:
    """Sequences over a shared pool: codes and scales random, everything that no sequence holds filled with noise (NaN
    and infinite scales among it)."""

    def __init__(self, gd, lens, qs, H, Hkv, D, page=16, T=F32, seed=0, paged=True, words=None, qscale=1.0, max_len=None,
                 spare=2):
        rng = np.random.default_rng(seed)
        self.gd, self.lens, self.qs, self.H, self.Hkv, self.D, self.T = gd, lens, qs, H, Hkv, D, T
        B, self.page = len(lens), page
        self.max_len = max(max(lens), 1) if max_len is None else max_len
        self.max_q = max(max(qs), 1)
        per = -(-self.max_len // page)
        pages = (B * per if paged else B) + spare
        if not paged:
            self.page = page = per * page
            per = 1
        self.k, self.v = [], []
        codes = rng.integers(-127, 128, (2, pages, Hkv, page, D)).astype(np.int8)
        scales = rng.integers(0, 65536, (2, pages, Hkv, page, D // 32)).astype(np.uint16).view(np.float16)
        table = rng.permutation(pages)[:B * per].reshape(B, per) if paged else np.arange(B)[:, None]
        for b, n in enumerate(lens):
            x = np.zeros((2, Hkv, max(n, 1), D))
            for j in range(n):
                g, p = table[b, j // page], j % page
                scales[:, g, :, p] = (rng.uniform(0.3, 1.0, (2, Hkv, D // 32)) / 60).astype(np.float16)
                x[:, :, j] = codes[:, g, :, p] * np.repeat(scales[:, g, :, p].astype(np.float64), 32, -1)
            self.k.append(x[0][:, :n])
            self.v.append(x[1][:, :n])
        self.codes, self.scales, self.table = codes, scales, table
        self.cache = gd.KVCacheQ8(dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1]))
        self.page_table = dev(table.astype(np.int32)) if paged else None
        self.kv_lens = dev(np.array(lens, np.int32))
        self.start = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
        n_q = int(self.start[-1])
        self.q = torch.from_numpy((rng.standard_normal((n_q, H, D)) * qscale).astype(np.float32)).to(T)
        self.words = words
        self.tree = None if words is None else dev(np.array(words, np.uint64).view(np.int64))

    def run(self, scale=None, cap=0.0, out=None, q_start=True, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        out = torch.full(self.q.shape, float("nan"), dtype=self.T, device="cuda") if out is None else out
        self.gd.attn_decode_q8(self.q.cuda(), self.cache, self.page_table, self.kv_lens,
                               dev(self.start) if q_start else None, self.tree, out, self.H, self.max_q, self.max_len,
                               scale, softcap=cap, **kw)
        return out

    def want(self, scale=None, cap=0.0, gone=None):
        """(f64 rows, bar per row); gone[b]: positions of sequence b that nobody sees."""
        scale = self.D ** -0.5 if scale is None else scale
        outs, bars = [], []
        for b, (n, t) in enumerate(zip(self.lens, self.qs)):
            ctx = max(n - t, 0)
            sees = np.zeros((t, n), bool)
            sees[:, :ctx] = True
            for i in range(t):
                w = chain(i) if self.words is None else self.words[self.start[b] + i]
                for j in range(ctx, n):
                    sees[i, j] = w >> (j - ctx) & 1
            if gone is not None:
                sees[:, gone[b]] = False
            q = self.q[self.start[b]:self.start[b + 1]].double().numpy()
            o, vmax, smax = layer.attention_rows(q, self.k[b], self.v[b], sees, scale, cap)
            outs.append(o)
            bar = 1e-5 * vmax + 2.0 ** -19 * smax * vmax
            if self.T != F32:
                bar += 2.0 ** -11 * vmax
            bars.append(np.full(o.shape, bar) + (torch.finfo(self.T).eps / 2 * np.abs(o) if self.T != F32 else 0))
        return np.concatenate(outs), np.concatenate(bars)

    def check(self, got, want=None, **kw):
        want, bar = self.want(**kw) if want is None else want
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(np.isfinite(got.float().cpu().numpy()))
        worst = float(np.max(err - bar))
        assert worst <= 0, f"off by {err.max():.3e}, {worst:.3e} over the bar"


SHAPES = [  # lens, rows, H, Hkv, D, page
    ([1], [1], 4, 1, 128, 16), ([1], [1], 1, 1, 64, 16), ([15, 16, 17], [1, 1, 1], 8, 2, 64, 16),
    ([31, 32, 33], [1, 1, 1], 8, 8, 128, 16), ([127, 128, 129, 130], [1] * 4, 3, 1, 128, 48),
    ([700], [1], 32, 8, 128, 64), ([4097], [1], 16, 2, 64, 64), ([2500, 3, 900], [1, 1, 1], 10, 5, 128, 32),
    ([257], [1], 4, 2, 256, 16), ([40, 300], [3, 7], 8, 2, 128, 16), ([65, 64, 64], [64, 64, 5], 2, 1, 64, 16),
    ([600, 70], [33, 1], 6, 2, 256, 32), ([500], [17], 40, 5, 128, 16), ([1200, 5, 64], [2, 5, 16], 64, 4, 128, 16)]


@pytest.mark.parametrize("T", [F32, F16, BF16])
@pytest.mark.parametrize("lens,qs,H,Hkv,D,page", SHAPES)
def test_parity(gd, T, lens, qs, H, Hkv, D, page):
    c = Case(gd, lens, qs, H, Hkv, D, page, T, seed=sum(lens) + H)
    c.check(c.run())


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (5, 5, 64), (6, 1, 256)])
def test_trees(gd, T, H, Hkv, D):
    """Random trees, a row that sees nothing drafted, a word with bits past the drafted tokens and bits of later
    ones, and the last of 64."""
    rng = np.random.default_rng(D)
    qs, lens, words = [64, 9, 1], [200, 9, 33], []
    for t in qs:
        seen = []
        for i in range(t):
            seen.append((seen[rng.integers(0, i)] if i else 0) | 1 << i)
        words += seen
    words[3] = 0
    words[5] = (1 << 64) - 1
    words[64] = 0                       # the 9-token sequence has no context: this row sees no key at all
    words[66] = 0b101000110 | 1 << 40
    c = Case(gd, lens, qs, H, Hkv, D, 16, T, seed=5, words=words)
    got = c.run()
    c.check(got)
    assert not got[64].any()
    c.check(c.run(cap=2.0), cap=2.0)


@pytest.mark.parametrize("T", [F32, F16])
def test_softcap(gd, T):
    c = Case(gd, [300, 77], [2, 3], 8, 2, 128, 16, T, seed=3, qscale=8.0)
    for cap in (0.5, 30.0, 1e4):
        c.check(c.run(cap=cap), cap=cap)


def test_unpaged(gd):
    c = Case(gd, [130, 1, 95], [1, 1, 1], 8, 2, 128, 16, paged=False)
    c.check(c.run())
    c.check(c.run(q_start=False))
    assert torch.equal(c.run(), c.run(q_start=False))


def test_uniform_rows_without_starts(gd):
    c = Case(gd, [130, 61], [4, 4], 8, 2, 64, 16)
    assert torch.equal(c.run(), c.run(q_start=False))


@pytest.mark.parametrize("T", [F32, BF16])
def test_empty_sequences_and_rows_of_none(gd, T):
    """Lengths of zero, sequences without rows, a length shorter than its rows; rows behind the last stay as they were."""
    c = Case(gd, [0, 50, 3, 20], [2, 0, 5, 1], 8, 2, 64, 16, T, seed=2)
    n_q = int(c.start[-1])
    extra = torch.randn(6, 8, 64).to(T)
    q = torch.cat([c.q, extra])
    out = torch.full(q.shape, 5.0, dtype=T, device="cuda")
    gd.attn_decode_q8(q.cuda(), c.cache, c.page_table, c.kv_lens, dev(c.start), None, out, 8, 5, c.max_len, 0.125)
    assert not out[:2].any() and bool((out[n_q:] == 5).all())
    c.check(out[:n_q], scale=0.125)


def test_lengths_and_starts_out_of_range_are_clamped(gd):
    """Device values that the host cannot check never reach past the buffers: lengths above max_kv_len or below zero, starts
    above n_q, below zero and falling."""
    c = Case(gd, [40, 40, 40], [1, 1, 1], 4, 2, 64, 16)
    ref = c.run()
    out = torch.full_like(ref, 5.0)
    call = lambda lens, start, out: gd.attn_decode_q8(c.q.cuda(), c.cache, c.page_table, dev(np.array(lens, np.int32)),
                                                      dev(np.array(start, np.int32)), None, out, 4, 1, 40, 0.125)
    call([1 << 30, -5, 40], [0, 1, 2, 3], out)
    assert torch.equal(out[0], ref[0]) and not out[1].any() and torch.equal(out[2], ref[2])
    out.fill_(5.0)
    call([40, 40, 40], [0, 1, 1 << 30, 3], out)
    assert torch.equal(out[0], ref[0]) and bool((out[2] == 5).all())
    out.fill_(5.0)
    call([40, 40, 40], [-7, 1, 0, 0], out)
    assert torch.equal(out[0], ref[0]) and bool((out[1:] == 5).all())


def test_pages_outside_the_pool_are_not_seen(gd):
    c = Case(gd, [100, 64], [1, 1], 8, 2, 64, 16)
    t = c.table.astype(np.int32).copy()
    t[0, 2], t[0, 6] = -1, 1 << 30      # positions 32..47 and the last, 96..99
    t[1, :] = -9                        # everything: the row is empty
    c.page_table = dev(t)
    gone = [np.r_[32:48, 96:100], np.arange(64)]
    got = c.run()
    c.check(got, gone=gone)
    assert not got[1].any()


@pytest.mark.parametrize("T", [F32, BF16])
def test_drafted_keys_that_nobody_sees_may_be_unstored(gd, T):
    """Rows of a tree call whose words leave out a drafted key, whose row holds NaN scales and any codes."""
    words = [1 << 0, 1 << 0, 0b1001]
    c = Case(gd, [40], [3], 4, 2, 64, 16, T, words=words)
    for at in (38, 39):
        g, p = c.table[0, at // 16], at % 16
        for t in (c.cache.k_scales, c.cache.v_scales):
            t[g, :, p] = float("nan") if at == 38 else float("inf")
    c.check(c.run())


@pytest.mark.parametrize("T", [F32, F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [65504.0, -65504.0, -3.0, float("-inf"), float("nan")])
def test_unstored_drafted_keys_leave_the_others_alone(gd, T, D, bad):
    """A padded tree: drafted keys 1, 2 and 5 are seen by no row, and their rows hold scales far above the others',
    negative or infinite ones. The bar follows the values that are seen."""
    words = [1, 0, 0, 0b1001, 0b11001, 0, 0b1000001]
    c = Case(gd, [150, 30], [7, 1], 12, 2, D, 16, T, seed=11, words=words + [1])
    for i in (1, 2, 5):
        g, p = c.table[0, (143 + i) // 16], (143 + i) % 16
        for t in (c.cache.k_scales, c.cache.v_scales):
            t[g, :, p] = bad
        c.k[0][:, 143 + i] = c.v[0][:, 143 + i] = 0.0   # no row's bar takes it in
    c.check(c.run())


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(gd, scale):
    """Means, negative scales, and scores in the hundreds."""
    c = Case(gd, [333], [2], 8, 2, 128, 16, seed=9, qscale=4.0)
    c.check(c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("T,top", [(F32, 1e30), (F32, 1e-30), (BF16, 1e30), (F16, 6e4), (F16, 6e-8)])
def test_query_range(gd, T, top):
    """Rows of any finite size: the scale brings the scores back to ordinary ones."""
    c = Case(gd, [200], [1], 4, 2, 64, 16, T, seed=4)
    q = c.q.double()
    c.q = (q / q.abs().max() * top).to(T)
    c.check(c.run(scale=0.5 / top), scale=0.5 / top)


@pytest.mark.parametrize("T,D", [(F32, 64), (BF16, 64), (BF16, 128), (F32, 256)])
def test_value_scales_of_any_size(gd, T, D):
    """Value scales from f16's smallest to its largest, side by side: the bar follows the largest value seen."""
    c = Case(gd, [160], [1], 4, 2, D, 16, T, seed=6)
    rng = np.random.default_rng(1)
    for lo, hi in ((2.0 ** -24, 2.0 ** -20), (6e4, 65504.0), (2.0 ** -24, 65504.0)):
        s = np.exp(rng.uniform(np.log(lo), np.log(hi), c.scales[1].shape)).astype(np.float16)
        c.cache.v_scales.copy_(dev(s))
        for j in range(160):
            g, p = c.table[0, j // 16], j % 16
            c.v[0][:, j] = c.codes[1, g, :, p] * np.repeat(s[g, :, p].astype(np.float64), 32, -1)
        c.check(c.run())


def test_zero_values_and_queries(gd):
    c = Case(gd, [80], [1], 4, 2, 64, 16)
    ref = c.run()
    c.cache.v_scales.copy_(torch.where(c.cache.v_scales.isfinite(), 0.0, c.cache.v_scales))
    out = c.run()
    assert not out.any() and ref.any()
    c = Case(gd, [80], [1], 4, 2, 64, 16)
    c.q = torch.zeros_like(c.q)
    c.check(c.run())


def test_one_key_returns_its_value(gd):
    c = Case(gd, [1], [1], 4, 2, 128, 16)
    got = c.run().cpu().numpy().reshape(2, 2, 128)
    assert np.abs(got - c.v[0][:, None, 0]).max() <= 2.0 ** -20 * np.abs(c.v[0]).max()


def test_long_sequence_and_splits(gd):
    """Thousands of keys with a single row: many splits; and the same sequence beside 40 short ones."""
    c = Case(gd, [5000], [1], 8, 1, 128, 64, seed=8)
    c.check(c.run())
    c = Case(gd, [3000] + [5] * 40, [1] * 41, 4, 1, 64, 16, seed=8)
    c.check(c.run())


@pytest.mark.parametrize("T", [F32, BF16])
def test_pool_past_32_bit_offsets(gd, T):
    """A pool whose planes pass 4 GiB: a sequence on its first and last pages gives what the same rows give in a small pool."""
    heads, D, page = 8, 128, 64
    pages = (5 << 30) // (heads * D * page)
    big = gd.kv_q8_alloc(pages, page, heads, D)
    c = Case(gd, [150], [1], 16, heads, D, page, T, seed=12)
    where = [pages - 1, 0, pages - 2]
    for plane in ("k_codes", "k_scales", "v_codes", "v_scales"):
        for i, w in enumerate(where):
            getattr(big, plane)[w] = getattr(c.cache, plane)[c.table[0, i]]
    ref = c.run()
    c.cache, c.page_table = big, dev(np.array([where], np.int32))
    assert torch.equal(c.run(), ref)
    c.check(ref)


def test_many_sequences_and_rows(gd):
    """More blocks of rows than one grid holds beside its sequences (80 x 1024 > 65535), most of them empty."""
    B = 1024
    qs = [0] * B
    qs[3], qs[1000] = 64, 2
    lens = [0] * B
    lens[3], lens[1000] = 64, 9
    c = Case(gd, lens, qs, 40, 1, 64, 16, BF16, seed=13, max_len=64)
    c.check(c.run())


def test_workspace_contents_do_not_matter(gd):
    c = Case(gd, [900, 20], [2, 1], 8, 2, 128, 16)
    ref = c.run()
    need = gd.attn_decode_q8_workspace_bytes(2, 3, 8, 2, 128, 2, c.max_len)
    for fill in (0xFF, 0x00, 0x7F):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(c.run(workspace=ws[:need]), ref)
        assert bool((ws[need:] == fill).all())
    with pytest.raises(gd.GemmDecodeError, match="GD_ERANGE"):
        c.run(workspace=ws[:need - 1])


def test_graph_replays_and_two_graphs_on_one_workspace(gd):
    """Captured calls of two shapes that share a workspace, replayed in turn with changed inputs."""
    a = Case(gd, [700, 300], [1, 1], 8, 2, 128, 16, seed=1)
    b = Case(gd, [900], [5], 8, 2, 128, 16, BF16, seed=2)
    need = max(gd.attn_decode_q8_workspace_bytes(2, 2, 8, 2, 128, 1, 700),
               gd.attn_decode_q8_workspace_bytes(1, 5, 8, 2, 128, 5, 900))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        q, start, out = c.q.cuda(), dev(c.start), torch.empty(c.q.shape, dtype=c.T, device="cuda")
        call = lambda out, c=c, q=q, start=start: gd.attn_decode_q8(
            q, c.cache, c.page_table, c.kv_lens, start, None, out, 8, c.max_q, c.max_len, 0.1, workspace=ws)
        call(out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append((g, q, out, call, c))
    for i in range(4):
        for g, q, out, call, c in graphs:
            q.normal_()
            c.kv_lens.sub_(7)
            g.replay()
        torch.cuda.synchronize()
        for g, q, out, call, c in graphs:
            want = torch.empty_like(out)
            call(want)
            assert torch.equal(want, out), i


def test_side_stream(gd):
    c = Case(gd, [800], [2], 8, 2, 128, 16)
    ref = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [c.run() for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_repeats_are_equal(gd):
    c = Case(gd, [1500, 800, 9], [4, 2, 9], 16, 2, 128, 16, BF16)
    ref = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), ref)


def test_refusals(gd):
    c = Case(gd, [40, 40], [1, 1], 4, 2, 64, 16)
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        c.run(cap=-1.0)
    with pytest.raises(ValueError):
        c.run(out=torch.empty(3, 4, 64, device="cuda"))
    with pytest.raises(TypeError):
        c.run(out=torch.empty(2, 4, 64, dtype=F16, device="cuda"))
    c.max_len = 49
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        c.run()
    c.max_len, c.max_q = 40, 65
    with pytest.raises(gd.GemmDecodeError, match="GD_ERANGE"):
        c.run()
    c.max_q = 1
    c.page_table = c.page_table[:, :2]
    with pytest.raises(ValueError):
        c.run()
    c.page_table = c.page_table[:, :0].contiguous()
    with pytest.raises(ValueError, match="empty"):
        c.run()
    c.page_table = dev(c.table.astype(np.int32))[:, :2].contiguous()
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        c.run()


def test_one_workspace_for_every_smaller_call(gd):
    """A workspace made for a server's largest call takes every smaller one, and none writes past what it asks for itself."""
    H, Hkv, D, B, max_q, max_len = 8, 2, 64, 12, 6, 2000
    most = gd.attn_decode_q8_workspace_bytes(B, B * max_q, H, Hkv, D, max_q, max_len)
    ws = torch.empty(most, dtype=torch.uint8, device="cuda")
    for seqs, q, n in ((12, 6, 2000), (12, 6, 1000), (12, 1, 300), (1, 1, 2000), (1, 6, 1920), (3, 4, 129), (7, 5, 1100), (11, 1, 1999),
                       (1, 1, 128), (2, 3, 40)):
        c = Case(gd, [n] + [max(q, n - 7 * i) for i in range(1, seqs)], [q] * seqs, H, Hkv, D, 16, BF16, seed=n)
        need = gd.attn_decode_q8_workspace_bytes(seqs, seqs * q, H, Hkv, D, q, n)
        assert need <= most
        ws.fill_(0xA5)
        got = c.run(workspace=ws)
        assert bool((ws[need:] == 0xA5).all())
        c.check(got)
        assert torch.equal(got, c.run())


def overwrite(c, which, codes, scales):
    """Keys (0) or values (1) of every sequence of c as given: codes [len, D] and scales [len, D/32], the same in every head."""
    planes = ((c.cache.k_codes, c.cache.k_scales), (c.cache.v_codes, c.cache.v_scales))[which]
    for b, n in enumerate(c.lens):
        g, p = dev(c.table[b, np.arange(n) // c.page]), dev(np.arange(n) % c.page)
        planes[0][g, :, p] = dev(np.asarray(codes[:n], np.int8))[:, None]
        planes[1][g, :, p] = dev(np.asarray(scales[:n], np.float16))[:, None]
        x = np.asarray(codes[:n], np.float64) * np.repeat(np.asarray(scales[:n], np.float16).astype(np.float64), 32, -1)
        (c.k, c.v)[which][b][:] = x


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_cancel(gd, D):
    """Pairs of dims whose products nearly cancel: the bar goes by scale * sum |q k| (here some 10^5), which the 22
    bits of q are parts of, and not by the scores."""
    c = Case(gd, [300], [1], 4, 2, D, 16, seed=21, qscale=6e3)
    rng = np.random.default_rng(2)
    q = c.q.double().numpy()
    q[..., 1::2] = q[..., 0::2] * (1 + rng.uniform(-1, 1, q[..., 0::2].shape) * 2.0 ** -15)
    c.q = torch.from_numpy(q.astype(np.float32))
    codes = rng.integers(-127, 128, (300, D))
    codes[:, 1::2] = -codes[:, 0::2]
    overwrite(c, 0, codes, rng.uniform(0.3, 1.0, (300, D // 32)) / 60)
    c.check(c.run())


@pytest.mark.parametrize("T", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_worst_roundings_to_f16(gd, T, D):
    """Every weight but the first and every value lies just below the middle of two f16 numbers at the low end of a binade:
    each is off by nearly 2^-11 of itself, both downwards, 2^-10 of the result in all; half a step of the result's type is
    added. The sums of f32 add 1e-5, and the weights' scores (0 and one of 0.69) 2^-19."""
    n = 200
    c = Case(gd, [n], [1], 4, 2, D, 16, T, seed=3)
    w = 0.5 * (1 + 0.98 * 2.0 ** -11)
    low = lambda m: m / 2.0 ** np.floor(np.log2(m)) - 1          # over the binade's low end
    best = max(((x * y, x, y) for x in range(1, 128) for y in range(1024, 2048) if low(x * y) < 2.0 ** -11),
               key=lambda t: low(t[0]))
    k = np.zeros((n, D), np.int8)
    k[1:, 0] = -1
    overwrite(c, 0, k, np.ones((n, D // 32)))
    overwrite(c, 1, np.full((n, D), best[1]), np.full((n, D // 32), best[2] / 1024.0))
    c.q = torch.ones_like(c.q)
    scale = float(-np.log(w))
    got, (want, _) = c.run(scale=scale).double().cpu().numpy(), c.want(scale=scale)
    v = best[0] / 1024.0
    assert np.allclose(want, v, rtol=1e-12)
    bar = (2.0 ** -10 + 1e-5 + 2.0 ** -19 * scale) * v + torch.finfo(T).eps / 2 * v
    assert np.abs(got - want).max() <= bar


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("even", [False, True])
def test_long_parts(gd, T, even):
    """65536 keys in one part (512 sequences of 8 KV heads share one sequence's pages: a workgroup for each is enough). A
    lane's sum of weights is 2048 roundings of at most 2^-24 each, and a sum of values three matrix products for each of a
    wave's 512 steps, 1536: 3584 * 2^-24 is below 2^-28 per key. even: all weights but one are equal and all values too, so
    that the roundings have one sign."""
    B, Hkv, D, page, n = 512, 8, 64, 256, 65536
    assert gd.attn_decode_q8_workspace_bytes(B, B, Hkv, Hkv, D, 1, n) < B * Hkv * (D + 2) * 4 * 2   # one part
    rng = np.random.default_rng(31)
    pages = n // page
    codes = rng.integers(-127, 128, (2, pages, Hkv, page, D)).astype(np.int8)
    scales = (rng.uniform(0.3, 1.0, (2, pages, Hkv, page, D // 32)) / 60).astype(np.float16)
    q = torch.from_numpy(rng.standard_normal((1, Hkv, D)).astype(np.float32)).to(T)
    if even:
        codes[0], codes[1] = -10, 101
        codes[0, 0, :, 0] = 0
        scales[0], scales[1] = 0.01, 0.0101
        q = torch.full_like(q, 1.0)
    cache = gd.KVCacheQ8(dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1]))
    out = torch.empty(B, Hkv, D, dtype=T, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    scale = 0.1875
    gd.attn_decode_q8(q.cuda().expand(B, -1, -1).contiguous(), cache, table, lens, None, None, out, Hkv, 1, n, scale)
    assert bool((out == out[:1]).all())
    k, v = (np.repeat(scales[i].astype(np.float64), 32, -1) * codes[i] for i in range(2))
    k, v = (x.transpose(1, 0, 2, 3).reshape(Hkv, n, D) for x in (k, v))
    want, vmax, smax = layer.attention_rows(q.double().numpy(), k, v, np.ones((1, n), bool), scale)
    err = np.abs(out[:1].double().cpu().numpy() - want)
    bar = (1e-5 + 2.0 ** -28 * n + 2.0 ** -19 * smax) * vmax
    if T != F32:
        bar = bar + 2.0 ** -10 * vmax + torch.finfo(T).eps / 2 * np.abs(want)
    print(T, even, "off by", err.max() / vmax)
    assert np.all(err <= bar)


def test_rows_of_another_order_are_refused(gd):
    """Queries or outputs with the heads first have the right number of elements and would be read in the wrong order."""
    c = Case(gd, [40, 40, 40], [1, 1, 1], 4, 2, 64, 16)
    ref = c.run()
    first = torch.empty(4, 3, 64, device="cuda")
    with pytest.raises(ValueError, match="out must be"):
        c.run(out=first)
    assert torch.equal(c.run(out=torch.empty(3, 256, device="cuda")).view_as(ref), ref)
    c.q = c.q.transpose(0, 1).contiguous()
    with pytest.raises(ValueError, match="q must be"):
        c.run(out=torch.empty(3, 4, 64, device="cuda"))


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("scale,cap,top", [(1.0, 1e-39, 0.0), (1.0, 1e-39, 1.0), (1.0, 1e-30, 1e30), (3e38, 0.0, 0.0), (-3e38, 1e-3, 0.0),
                                           (3e38, 1e-3, 1e-3)])
def test_factors_past_f32(gd, T, scale, cap, top):
    """scale / softcap (or scale log2 e) past f32's range, with keys of zeros among the others: their scores are 0 and not
    NaN, and a cap of next to nothing leaves the mean of the values."""
    c = Case(gd, [90], [2], 4, 2, 64, 16, T, seed=14)
    c.q = (c.q.double() / c.q.double().abs().max() * top).to(T)
    codes = np.random.default_rng(3).integers(-127, 128, (90, 64))
    codes[::3] = 0
    overwrite(c, 0, codes, np.full((90, 2), 0.01))
    got, (want, _) = c.run(scale=scale, cap=cap).double().cpu().numpy(), c.want(scale=scale, cap=cap)
    vmax = np.abs(c.v[0]).max()
    if cap != 1e-3:
        mean = np.repeat(np.stack([c.v[0][:, :89].mean(1), c.v[0].mean(1)]), 2, axis=1)
        assert np.allclose(want, mean, atol=1e-12)
    assert np.abs(got - want).max() <= (1e-5 + (2.0 ** -10 + torch.finfo(T).eps / 2 if T != F32 else 0)) * vmax


@pytest.mark.parametrize("T", [F32, BF16])
@pytest.mark.parametrize("n", [8200, 9001, 17000])
@pytest.mark.parametrize("at", ["early", "late", "none"])
def test_more_than_64_parts(gd, T, n, at):
    """One sequence and KV head: 65, 71 and 133 parts, which the joining launch takes 64 at a time, the last batch partly
    filled. One key's score is far above the others' in the first batch or in the last part, so that the sums before (or
    behind) it are rescaled."""
    H, D = 3, 128
    c = Case(gd, [n], [1], H, 1, D, 16, T, seed=n)
    assert gd.attn_decode_q8_workspace_bytes(1, 1, H, 1, D, 1, n) >= 65 * H * (D + 2) * 4
    if at != "none":
        rng = np.random.default_rng(1)
        codes, scales = rng.integers(-127, 128, (n, D)), rng.uniform(0.3, 1.0, (n, D // 32)) / 60
        j = 130 if at == "early" else n - 2
        q0 = c.q[0, 0].double().numpy()
        codes[j] = np.where(q0 > 0, 127, -127)
        c.q = c.q[:, :1].expand(-1, H, -1).contiguous()
        overwrite(c, 0, codes, scales)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_trees_in_f16(gd, D):
    """Random trees of 64, 9 and 1 drafted tokens, capped and not, with rows that see nothing drafted or nothing at all."""
    rng = np.random.default_rng(D + 1)
    qs, lens, words = [64, 9, 1], [200, 9, 33], []
    for t in qs:
        seen = []
        for i in range(t):
            seen.append((seen[rng.integers(0, i)] if i else 0) | 1 << i)
        words += seen
    words[3] = words[64] = 0
    words[5] = (1 << 64) - 1
    c = Case(gd, lens, qs, 8, 2, D, 16, F16, seed=15, words=words)
    got = c.run()
    c.check(got)
    assert not got[64].any()
    c.check(c.run(cap=2.0), cap=2.0)
