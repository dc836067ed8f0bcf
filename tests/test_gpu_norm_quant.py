"""GPU parity of the norms with an 8-bit output and of the readers.

The rule fixes every step but the sum's order (in f64, 2^-53 a step), so h,
codes and scales are compared bit for bit with the f64 definition, and the
readers' values with f32(code) * scale rounded once."""
import numpy as np
import pytest

import oracle
from oracle import layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS = 1e-5
TYPES = [torch.float32, torch.float16, torch.bfloat16]
GUARD = 64


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def rows(n, K, T, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((n, K)) * scale).astype(np.float32)).to(T)


def blocks(codes, scale):
    """q8_0 bytes of codes [n, K] and f32 scales [n, K/32]."""
    n, K = codes.shape
    d = scale.astype(np.float16).reshape(n, K // 32, 1).view(np.uint8).reshape(n, K // 32, 2)
    return np.concatenate([d, codes.view(np.uint8).reshape(n, K // 32, 32)], -1).reshape(-1)


def planes_of(codes):
    n, K = codes.shape
    bits = np.unpackbits(codes.view(np.uint8).reshape(n, K, 1), axis=2, bitorder="little")   # [n, K, 8]
    words = np.packbits(np.ascontiguousarray(bits.transpose(0, 2, 1)), axis=2, bitorder="little")
    return np.ascontiguousarray(words).reshape(-1).view(np.uint32)


def guarded(numel, dtype):
    """A device view of numel elements with guard elements behind it."""
    fill = {torch.uint8: 0xA5, torch.int32: -7}.get(dtype, 7.0)
    whole = torch.full((numel + GUARD,), fill, dtype=dtype, device="cuda")
    return whole[:numel], whole, fill


def run(gd, form, x, res, w, h_out, n, K):
    """(activation bytes or (planes, scales)) of one call, guards checked."""
    if form == "q8_0":
        a, whole, fill = guarded(n * (K // 32) * 34, torch.uint8)
        gd.rmsnorm_q8_0(x, res, w, h_out, a, n, K, EPS)
        assert bool((whole[a.numel():] == fill).all())
        return a
    p, whole, fill = guarded(n * 8 * (K // 32), torch.int32)
    s, sw, sf = guarded(n, torch.float32)
    gd.rmsnorm_ternary_act(x, res, w, h_out, p, s, n, K, EPS)
    assert bool((whole[p.numel():] == fill).all()) and bool((sw[n:] == sf).all())
    return p, s


def check(form, got, h, w, n, K):
    codes, scale = layer.rmsnorm_codes(h, w, EPS, 32 if form == "q8_0" else K)
    if form == "q8_0":
        assert np.array_equal(got.cpu().numpy(), blocks(codes, scale))
    else:
        assert np.array_equal(got[0].cpu().numpy().view(np.uint32), planes_of(codes))
        assert np.array_equal(got[1].cpu().numpy(), scale[:, 0])


SHAPES = [(1, 32), (1, 64), (3, 96), (5, 1056), (2, 2560), (2, 4096), (7, 4128), (1, 6912), (3, 8192), (2, 8224),
          (1, 16416), (2, 20000), (300, 160), (5, 512), (4, 1024),
          (1030, 512), (1026, 544), (1025, 1024), (2050, 32)]   # the last four: a wave per row


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("n,K", SHAPES)
def test_parity(gd, form, T, n, K):
    x, res = rows(n, K, T, n * K), rows(n, K, T, n * K + 1, 3.0)
    w = rows(1, K, torch.float32, 5)[0] * 0.2 + 1
    h = (x.float() + res.float()).to(T)
    h_out = torch.full((n, K), float("nan"), dtype=T, device="cuda")
    got = run(gd, form, x.cuda(), res.cuda(), w.cuda(), h_out, n, K)
    assert torch.equal(h_out.cpu(), h)
    check(form, got, h.float().numpy(), w.numpy(), n, K)
    # without a residual the row itself is normed, with and without the copy
    for out in (None, torch.empty_like(h_out)):
        got = run(gd, form, h.cuda(), None, w.cuda(), out, n, K)
        check(form, got, h.float().numpy(), w.numpy(), n, K)
        assert out is None or torch.equal(out.cpu(), h)
    got = run(gd, form, x.cuda(), res.cuda(), w.cuda(), None, n, K)
    check(form, got, h.float().numpy(), w.numpy(), n, K)


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
@pytest.mark.parametrize("K", [96, 4096, 9216])
@pytest.mark.parametrize("T", [torch.float32, torch.bfloat16])
def test_in_place(gd, form, K, T):
    """The sum written over the residual, or over x."""
    n = 3
    x, res, w = rows(n, K, T, 1), rows(n, K, T, 2), torch.ones(K)
    h = (x.float() + res.float()).to(T)
    for which in (0, 1):
        t = [x.cuda(), res.cuda()]
        got = run(gd, form, t[0], t[1], w.cuda(), t[which], n, K)
        assert torch.equal(t[which].cpu(), h) and torch.equal(t[1 - which].cpu(), (res, x)[which])
        check(form, got, h.float().numpy(), w.numpy(), n, K)


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_extreme_rows(gd, form):
    """Zero rows and blocks, values at both ends of f32, products past f32's
    range, and rounding ties; a row of NaN leaves the others alone."""
    K = 128
    h = np.zeros((9, K), np.float32)
    w = np.ones(K, np.float32)
    h[1, 64:] = np.arange(64)                       # two zero blocks
    h[2] = 3e38
    h[3] = 1e-45                                    # f32's smallest
    h[4, :] = np.tile([127, 0.5, -0.5, 1.5, -1.5, 2.5, -63.5, 126.5], 16)   # exact halves: 127 sets the scale
    h[5, 0], h[5, 1] = 3e38, 1e-40
    h[6] = np.nan
    h[7] = np.linspace(-1, 1, K)
    h[8] = -h[4]
    w[:4] = [1, -2, 1e30, 1e-30]
    got = run(gd, form, torch.from_numpy(h).cuda(), None, torch.from_numpy(w).cuda(), None, 9, K)
    keep = [r for r in range(9) if r != 6]
    codes, scale = layer.rmsnorm_codes(h[keep], w, EPS, 32 if form == "q8_0" else K)
    if form == "q8_0":
        with np.errstate(over="ignore"):
            assert np.array_equal(got.cpu().numpy().reshape(9, -1)[keep], blocks(codes, scale).reshape(8, -1))
    else:
        assert np.array_equal(got[0].cpu().numpy().view(np.uint32).reshape(9, -1)[keep], planes_of(codes).reshape(8, -1))
        assert np.array_equal(got[1].cpu().numpy()[keep], scale[:, 0])


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_zero_rows_without_eps_and_zero_weights(gd, form):
    """A zero row with eps 0 (its root mean square is 0), a zero block and zero weights: zero codes and scales, no NaN."""
    K = 96
    h = np.zeros((3, K), np.float32)
    h[1] = np.arange(K) - 40
    h[2, 32:64] = 1e-30
    w = np.ones(K, np.float32)
    w[:32] = 0
    x, wd = torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda()
    if form == "q8_0":
        a = torch.full((3 * 3 * 34,), 0xA5, dtype=torch.uint8, device="cuda")
        gd.rmsnorm_q8_0(x, None, wd, None, a, 3, K, 0.0)
        a = a.cpu().numpy().reshape(3, 3, 34)
        assert not a[0].any() and not a[1, 0].any() and not a[2, [0, 2]].any()
        codes, scale = layer.rmsnorm_codes(h[1:], w, 0.0, 32)
        assert np.array_equal(a[1:].reshape(-1), blocks(codes, scale))
    else:
        p, s = torch.full((3 * 8 * 3,), -1, dtype=torch.int32, device="cuda"), torch.full((3,), -1.0, device="cuda")
        gd.rmsnorm_ternary_act(x, None, wd, None, p, s, 3, K, 0.0)
        codes, scale = layer.rmsnorm_codes(h[1:], w, 0.0, K)
        assert s[0] == 0 and not p[:24].any()
        assert np.array_equal(s[1:].cpu().numpy(), scale[:, 0])
        assert np.array_equal(p[24:].cpu().numpy().view(np.uint32), planes_of(codes))


def test_ties_go_up(gd):
    """Products at exact halves of a code step in every group: 127 in the group makes the step 1."""
    rng = np.random.default_rng(8)
    K = 4096
    h = (rng.integers(-126, 127, (2, K)) + 0.5).astype(np.float32)
    h[:, ::32] = 127
    w = np.ones(K, np.float32)
    for form in ("q8_0", "ternary"):
        check(form, run(gd, form, torch.from_numpy(h).cuda(), None, torch.from_numpy(w).cuda(), None, 2, K), h, w, 2, K)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("n,K", [(1, 32), (3, 96), (5, 4128), (129, 256)])
def test_readers(gd, T, n, K):
    x = rows(n, K, torch.float32, K + n)
    raw = oracle.quantize_q8_0(x.numpy())
    b = raw.reshape(n, K // 32, 34)
    d = b[:, :, :2].copy().view(np.float16).astype(np.float32)
    want = torch.from_numpy((b[:, :, 2:].view(np.int8).astype(np.float32) * d).reshape(n, K)).to(T)
    y, whole, fill = guarded(n * K, T)
    gd.q8_0_dequantize(torch.from_numpy(raw).cuda(), y, n, K)
    assert torch.equal(y.cpu().view(n, K), want) and bool((whole[n * K:] == fill).all())
    codes, s = oracle.quantize_absmax_int8(x.numpy())
    planes = torch.from_numpy(planes_of(codes).view(np.int32).copy()).cuda()
    y, whole, fill = guarded(n * K, T)
    gd.ternary_dequantize_act(planes, torch.from_numpy(s).cuda(), y, n, K)
    want = torch.from_numpy(codes.astype(np.float32) * s[:, None]).to(T)
    assert torch.equal(y.cpu().view(n, K), want) and bool((whole[n * K:] == fill).all())


def test_every_code_is_read(gd):
    codes = np.arange(-128, 128).astype(np.int8).reshape(1, 256)
    planes = torch.from_numpy(planes_of(codes).view(np.int32).copy()).cuda()
    y = torch.empty(256, device="cuda")
    gd.ternary_dequantize_act(planes, torch.ones(1, device="cuda"), y, 1, 256)
    assert np.array_equal(y.cpu().numpy(), codes[0].astype(np.float32))
    raw = blocks(codes, np.ones((1, 8), np.float32))
    gd.q8_0_dequantize(torch.from_numpy(raw).cuda(), y, 1, 256)
    assert np.array_equal(y.cpu().numpy(), codes[0].astype(np.float32))


def test_streams_and_graph(gd):
    """The call on a side stream, and captured: each replay equals the eager result on its inputs."""
    n, K = 4, 2560
    w = torch.ones(K, device="cuda")
    x, res = rows(n, K, torch.float32, 1).cuda(), rows(n, K, torch.float32, 2).cuda()
    h, a = torch.empty_like(x), torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda")
    y = torch.empty(n, K, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        gd.rmsnorm_q8_0(x, res, w, h, a, n, K, EPS)
        with torch.cuda.graph(graph, stream=side):
            gd.rmsnorm_q8_0(x, res, w, h, a, n, K, EPS)
            gd.q8_0_dequantize(a, y, n, K)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(rows(n, K, torch.float32, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        b, yy, hh = torch.empty_like(a), torch.empty_like(y), torch.empty_like(h)
        gd.rmsnorm_q8_0(x, res, w, hh, b, n, K, EPS)
        gd.q8_0_dequantize(b, yy, n, K)
        assert torch.equal(a, b) and torch.equal(y, yy) and torch.equal(h, hh)


def test_refusals_launch_nothing(gd):
    x = torch.zeros(2, 64, device="cuda")
    a = torch.zeros(136, dtype=torch.uint8, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(gd.GemmDecodeError, match="GD_ESHAPE"):
        gd.rmsnorm_q8_0(torch.zeros(2, 48, device="cuda"), None, w[:48], None, a, 2, 48, EPS)
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        gd.rmsnorm_q8_0(x, None, w, None, a, 2, 64, -1.0)
    with pytest.raises(ValueError):
        gd.rmsnorm_q8_0(x, None, w, None, a[:-1], 2, 64, EPS)
    with pytest.raises(TypeError):
        gd.rmsnorm_q8_0(x, x.half(), w, None, a, 2, 64, EPS)
    with pytest.raises(ValueError):
        gd.rmsnorm_q8_0(x.t(), None, w, None, a, 2, 64, EPS)
    assert not a.any()


@pytest.mark.parametrize("T", TYPES)
def test_codes_beside_those_of_the_quantizer(gd, T):
    """Rows of weight 1 against q8_0_quantize of the same values, and the cache's rows: other codes only at exact halves of a
    step (which bf16 rows have), by one; the cache's scales are the quantizer's."""
    n, K = 512, 1024
    x = rows(n, K, T, 77)
    x = torch.where(x.abs() < 2.0 ** -10, torch.full_like(x, 0.5), x)   # whole multiples of 2^-40, for exact arithmetic
    blocks_of = lambda a: a.cpu().numpy().reshape(-1, 34)
    plain = torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda")
    gd.q8_0_quantize(x.float().cuda(), plain, n, K)
    plain = blocks_of(plain)
    norm = blocks_of(run(gd, "q8_0", x.cuda(), None, torch.ones(K, device="cuda"), None, n, K))
    cache = gd.kv_q8_alloc(n // 16, 16, K // 64, 64)
    v = x.cuda().view(n, K // 64, 64)
    gd.kv_q8_store(cache, v, v, torch.arange(n, device="cuda"), n)
    stored = cache.v_codes.transpose(1, 2).reshape(-1, 32).cpu().numpy()
    scales = cache.v_scales.transpose(1, 2).reshape(-1).cpu().numpy()
    assert np.array_equal(scales, plain[:, :2].copy().view(np.float16)[:, 0])
    values, want = x.double().numpy().reshape(-1, 32), plain[:, 2:].view(np.int8)
    for got in (norm[:, 2:].view(np.int8), stored):
        at = np.argwhere(got != want)
        assert T != torch.bfloat16 or len(at)
        for r, i in at:
            val, top = (int(t * 2.0 ** 40) for t in (values[r, i], np.abs(values[r]).max()))
            lower = min(int(got[r, i]), int(want[r, i]))
            assert abs(int(got[r, i]) - int(want[r, i])) == 1 and 2 * 127 * val == (2 * lower + 1) * top
