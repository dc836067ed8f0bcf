"""GPU parity of the Q1_0 . q8_0 products with an epilogue, single and gated, against the
f64 definition at the documented bounds: sums within (K/128 + 9) 2^-23 of the sum of
magnitudes, carried through the activation, the gate's product and the residual, and half a
step of the output's type. The 8-bit output is compared bit for bit with the quantization
rule on the f32 output of the same call."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import answer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GUARD = 64


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def planes(gd, w):
    rows, K = w.shape[0], w.shape[1] * 128
    b, s = gd.q1_alloc_planes(rows, K)
    gd.q1_repack(dev(w.reshape(-1)), rows, K, b, s)
    return b, s


def guarded(shape, dtype):
    numel = int(np.prod(shape))
    fill = 0xA5 if dtype == torch.uint8 else 7.0
    whole = torch.full((numel + GUARD,), fill, dtype=dtype, device="cuda")
    return whole[:numel].view(shape), whole, fill


class Case:
    """Weights, activations and what stands around them, on both sides."""

    def __init__(self, gd, rows, K, n, sets=1, bias=True, seed=0):
        rng = np.random.default_rng(seed + 1000 * n + rows)
        self.rows, self.K, self.n = rows, K, n
        self.w = [wl.q1_weights_aos(rows, K, seed + i) for i in range(sets)]
        self.planes = [planes(gd, w) for w in self.w]
        self.a = wl.q8_acts_aos(K, seed + 7, n)
        self.a_dev = dev(self.a.reshape(-1))
        self.bias = [rng.standard_normal(rows).astype(np.float32) if bias else None for _ in range(sets)]
        self.bias_dev = [None if b is None else dev(b) for b in self.bias]
        self.residual = rng.standard_normal((n, rows)).astype(np.float32)

    def products(self, codes):
        a = answer.q8_values(self.a, self.n)
        return [answer.product(answer.q1_values(w), a, b, c) for w, b, c in zip(self.w, self.bias, codes)]

    def linear(self, gd, y, act=0, residual=None, **kw):
        gd.q1_q8_linear(*self.planes[0], self.a_dev, y, self.rows, self.K, self.n, bias=self.bias_dev[0], act=act,
                        residual=residual, **kw)
        return y

    def gated(self, gd, y, act=5, **kw):
        gd.q1_q8_gated(*self.planes[0], *self.planes[1], self.a_dev, y, self.rows, self.K, self.n, act=act,
                       gate_bias=self.bias_dev[0], up_bias=self.bias_dev[1], **kw)
        return y


def within(got, want, off, T):
    """off: how far the f32 value may be; the output's own rounding (half a step, or half of the smallest subnormal one)."""
    fi = torch.finfo(T)
    half = 0.0 if T == torch.float32 else (np.abs(want) + off) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2
    got = got.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - want) <= off + half)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], np.broadcast_to(off, got.shape)[bad][:5])


# Row counts beside 16, 32, 64 and 128, one block of K to many, columns beside 4, 16, 32 and 64.
SHAPES = [(1, 128, 1), (16, 256, 1), (33, 640, 1), (70, 1024, 1), (4096, 4096, 1), (130, 14336, 1), (257, 2176, 2),
          (64, 512, 3), (96, 384, 4), (50, 128, 4), (40, 16512, 1), (17, 33024, 3),
          (1, 128, 5), (31, 128, 7), (65, 384, 16), (127, 640, 31), (128, 1024, 32), (129, 896, 33), (600, 2560, 37),
          (515, 1152, 64), (200, 256, 65), (1030, 512, 130), (2085, 640, 300), (4200, 256, 1000), (64, 14336, 13), (96, 33024, 9),
          (14337, 4096, 1), (14340, 4096, 2), (28700, 1024, 3), (7201, 8192, 2), (8200, 1024, 1000), (2085, 14336, 300),
          (4096, 4096, 6), (3100, 14336, 7), (8200, 4096, 5), (2100, 14336, 14), (4000, 14336, 11), (2500, 14336, 16), (16500, 1664, 9),
          (32800, 1664, 9), (16400, 512, 8), (1030, 512, 500), (2200, 14336, 20), (4100, 8192, 40), (2085, 14336, 500),
          (8200, 2048, 1000)]


@pytest.mark.parametrize("rows,K,n", SHAPES)
def test_linear(gd, rows, K, n):
    """Every type, activations in turn, bias and residual; y in place of the residual."""
    c = Case(gd, rows, K, n, seed=rows + K)
    for i, (name, T) in enumerate(TYPES.items()):
        act = (rows + n + 2 * i) % 6
        (v, off), = c.products([act])
        res = dev(c.residual).to(T)
        r = res.float().cpu().numpy().astype(np.float64)
        y, whole, fill = guarded((n, rows), T)
        c.linear(gd, y, act, res)
        assert bool((whole[y.numel():] == fill).all())
        within(y, v + r, off + 2.0 ** -24 * np.abs(v + r) + 2.0 ** -24 * off, T)
        c.linear(gd, res, act, res)
        assert torch.equal(res, y)
    y = c.linear(gd, torch.empty(n, rows, device="cuda"))
    (v, off), = c.products([0])
    within(y, v, off, torch.float32)


@pytest.mark.parametrize("rows,K,n", [s for s in SHAPES if s[0] > 1])
def test_gated(gd, rows, K, n):
    c = Case(gd, rows, K, n, sets=2, bias=n % 2 == 1, seed=rows + K + 1)
    for i, (name, T) in enumerate(TYPES.items()):
        act = 1 + (rows + n + 2 * i) % 5
        (g, goff), (u, uoff) = c.products([act, 0])
        y, whole, fill = guarded((n, rows), T)
        c.gated(gd, y, act)
        assert bool((whole[y.numel():] == fill).all())
        off = np.abs(g) * uoff + np.abs(u) * goff + goff * uoff
        within(y, g * u, off + 2.0 ** -24 * (np.abs(g * u) + off), T)


@pytest.mark.parametrize("rows,K,n", [(32, 128, 1), (64, 640, 2), (4096, 1024, 1), (96, 384, 4), (32, 2176, 5),
                                      (160, 896, 33), (512, 256, 64), (1056, 640, 130), (4192, 128, 1000),
                                      (96, 4096, 1), (64, 8192, 4), (32, 14336, 2), (14336, 4096, 1), (160, 4096, 33),
                                      (2080, 14336, 300), (8224, 1024, 1000),
                                      (96, 4096, 8), (4096, 14336, 8), (2080, 4096, 16), (64, 8192, 12),
                                      (1056, 512, 500), (2208, 14336, 20), (2080, 14336, 500), (8224, 2048, 1000)])
@pytest.mark.parametrize("gated", [False, True])
def test_q8_output_is_the_quantized_f32_output(gd, rows, K, n, gated):
    """The blocks are those of the rule on v in f32, with and without y beside them, in any type; a row of zeros among them."""
    c = Case(gd, rows, K, n, sets=2, bias=False, seed=rows + 3)
    if n > 1:   # a column of zeros
        c.a[n - 1, :, 2:] = 0
        c.a_dev = dev(c.a.reshape(-1))
    call = c.gated if gated else c.linear
    y = torch.empty(n, rows, device="cuda")
    q, whole, fill = guarded((n * rows // 32 * 34,), torch.uint8)
    call(gd, y, act=5, y_q8=q)
    assert bool((whole[q.numel():] == fill).all())
    assert np.array_equal(q.cpu().numpy(), oracle.quantize_q8_0(y.cpu().numpy()))
    alone = torch.empty_like(q)
    call(gd, None, act=5, y_q8=alone)
    assert torch.equal(alone, q)
    for T in (torch.float16, torch.bfloat16):
        z = torch.empty(n, rows, dtype=T, device="cuda")
        alone.zero_()
        call(gd, z, act=5, y_q8=alone)
        assert torch.equal(alone, q) and torch.equal(z, y.to(T))


def edge_acts(K, n, seed):
    """Codes at both ends (-128 among them) and scales over f16's whole range: 65504, subnormal, zero, negative."""
    rng = np.random.default_rng(seed)
    a = wl.q8_acts_aos(K, seed, n)
    a[:, :, 2:] = rng.choice(np.array([-128, -127, -17, -16, -15, -1, 0, 1, 15, 16, 17, 126, 127], np.int8),
                             size=(n, K // 32, 32)).view(np.uint8)
    d = rng.choice(np.array([65504, 1, 2.0 ** -14, 2.0 ** -24, 1023 * 2.0 ** -24, 0, -0.37, 2047, 0.1], np.float16), size=(n, K // 32))
    a[:, :, :2] = d[..., None].view(np.uint8)
    return a


@pytest.mark.parametrize("rows,K,n", [(64, 512, 1), (80, 1280, 4), (48, 1408, 6), (300, 4096, 8), (90, 6400, 15), (200, 640, 40), (300, 384, 130), (2050, 8192, 600), (2050, 8192, 900)])
def test_edge_activations(gd, rows, K, n):
    c = Case(gd, rows, K, n, sets=2, bias=False, seed=5)
    c.a = edge_acts(K, n, rows)
    c.a_dev = dev(c.a.reshape(-1))
    (v, off), = c.products([0])[:1]
    within(c.linear(gd, torch.empty(n, rows, device="cuda")), v, off, torch.float32)


@pytest.mark.parametrize("rows,K,n", [(64, 512, 1), (64, 512, 4), (48, 640, 6), (40, 8192, 16), (300, 384, 70), (64, 4096, 40), (2050, 8192, 600), (2050, 8192, 900)])
def test_weight_scales_of_both_ends(gd, rows, K, n):
    """d0 of 65504, subnormal, zero, negative and, in one row alone, NaN and infinity."""
    c = Case(gd, rows, K, n, bias=False, seed=6)
    rng = np.random.default_rng(rows)
    d = rng.choice(np.array([65504, 2.0 ** -24, 2.0 ** -15, 0, -0.02, 0.3], np.float16), size=c.w[0].shape[:2])
    c.w[0][:, :, :2] = d[..., None].view(np.uint8)
    (v, off), = c.products([0])
    d[3, 1], d[17, 2] = np.nan, np.inf
    c.w[0][:, :, :2] = d[..., None].view(np.uint8)
    c.planes = [planes(gd, c.w[0])]
    y = c.linear(gd, torch.empty(n, rows, device="cuda"))
    sound = [r for r in range(rows) if r not in (3, 17)]
    within(y[:, sound], v[:, sound], off[:, sound], torch.float32)
    assert bool(y[:, 3].isnan().all()) and not bool(y[:, 17].isfinite().any())


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("rows,K,n", [(64, 512, 1), (64, 512, 4), (48, 640, 6), (40, 8192, 16), (300, 384, 70), (64, 4096, 40), (2050, 8192, 600), (2050, 8192, 900)])
def test_columns_do_not_touch_each_other(gd, rows, K, n, bad):
    """A column whose scale is no number is NaN, its neighbours keep every bit."""
    c = Case(gd, rows, K, n, bias=False, seed=8)
    y = c.linear(gd, torch.empty(n, rows, device="cuda"))
    at = n // 2
    a = c.a.copy()
    a[at, 3, :2] = np.array([bad], np.float16).view(np.uint8)
    c.a_dev = dev(a.reshape(-1))
    z = c.linear(gd, torch.empty(n, rows, device="cuda"))
    rest = [i for i in range(n) if i != at]
    assert bool(z[at].isnan().all()) and torch.equal(z[rest], y[rest])


def test_acts_at_their_ends(gd):
    """Sums from -1e6 to 1e6, through every activation: K = 128, one code set, so that the sum is exact."""
    vals = np.array([0.0, 1e-3, -1e-3, 0.5, -0.5, 1, -1, 3, -3, 6, -6, 9, -9, 13, -13, 20, -20, 60, -60, 88, -88, 104, -104, 200,
                     -200, 1e4, -1e4, 1e6, -1e6], np.float32)
    rows, n = len(vals), 3
    w = wl.q1_weights_aos(rows, 128, 1)
    for act in range(6):
        b = dev(vals)
        a = np.zeros((n, 4, 34), np.uint8)   # the sum is the bias
        y = torch.empty(n, rows, device="cuda")
        gd.q1_q8_linear(*planes(gd, w), dev(a.reshape(-1)), y, rows, 128, n, bias=b, act=act)
        want = np.tile(answer.act(vals, act), (n, 1))
        off = 2.0 ** -20 * np.abs(vals) if act > 2 else 2.0 ** -24 * np.abs(want)
        within(y, want, np.broadcast_to(off, want.shape), torch.float32)


def test_repeatable_and_apart_from_the_workspace(gd):
    """The same bits whatever the workspace held; a larger workspace than needed; one too small is refused."""
    c = Case(gd, 300, 1024, 37, sets=2, seed=2)
    need = gd.q1_q8_linear_workspace_bytes(1024, 37)
    assert need == 2 * 100 * 1024 + (16 << 20) and gd.q1_q8_linear_workspace_bytes(1024, 4) == 0
    y = c.gated(gd, torch.empty(37, 300, device="cuda"))
    for fill in (0, 0xFF):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        z = c.gated(gd, torch.full((37, 300), float("nan"), device="cuda"), workspace=ws)
        assert torch.equal(y, z)
        assert bool((ws[need:] == fill).all())
    with pytest.raises(gd.GemmDecodeError, match="GD_ERANGE"):
        c.gated(gd, y, workspace=ws[:need - 16])


def test_streams_and_graphs(gd):
    """On a stream of the user's, and captured twice on one workspace, replayed in turns with eager calls between."""
    c, d = Case(gd, 256, 768, 9, sets=2, seed=3), Case(gd, 96, 512, 3, seed=4)
    want = c.gated(gd, torch.empty(9, 256, device="cuda")), d.linear(gd, torch.empty(3, 96, device="cuda"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = c.gated(gd, torch.empty(9, 256, device="cuda")), d.linear(gd, torch.empty(3, 96, device="cuda"))
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ws = torch.empty(gd.q1_q8_linear_workspace_bytes(768, 9), dtype=torch.uint8, device="cuda")
    e = Case(gd, 512, 768, 6, seed=5)
    outs = [torch.empty(9, 256, device="cuda"), torch.empty(6, 512, device="cuda")]
    calls = [lambda y: c.gated(gd, y, workspace=ws), lambda y: e.linear(gd, y, workspace=ws)]
    eager = [f(torch.empty_like(o)) for f, o in zip(calls, outs)]
    graphs = []
    for f, o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(o)
        graphs.append(g)
    for i in range(6):
        for o in outs:
            o.fill_(float("nan"))
        for j in ((0, 1) if i % 2 else (1, 0)):
            graphs[j].replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, eager)), i
        assert torch.equal(c.gated(gd, torch.empty(9, 256, device="cuda"), workspace=ws), eager[0])
