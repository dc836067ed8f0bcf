"""Argument checks, on a host without a GPU, of the products with an epilogue, the norms
behind and before a block and the log probabilities: the documented status before any HIP call
(no compute is launched here)."""
import ctypes

import pytest

FAKE, FAR = 0x100000, 0x40000000000   # aligned addresses, far apart, that are never dereferenced: validation fails first
INVAL, SHAPE, ALIGN, RANGE = -1, -2, -3, -5
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 62


@pytest.fixture(scope="module")
def gd():
    import gemm_decode_amd
    return gemm_decode_amd


def test_linear_refusals(gd):
    L = gd.lib()

    def linear(b=FAKE, s=FAKE, a=FAKE, bias=FAKE, act=0, res=FAKE, y=FAR, q=None, rows=64, K=256, n=2, dt=F32, ws=None, wb=0):
        return L.q1_q8_linear(b, s, a, bias, act, res, y, q, rows, K, n, dt, ws, wb, None)

    def gated(b=FAKE, s=FAKE, a=FAKE, bias=FAKE, act=0, y=FAR, q=None, rows=64, K=256, n=2, dt=F32, ws=None, wb=0, second=False):
        two = (FAKE, FAKE, b, s) if second else (b, s, FAKE, FAKE)
        return L.q1_q8_gated(*two, a, FAKE if second else bias, bias if second else FAKE, act, y, q, rows, K, n, dt, ws, wb, None)
    for call in (linear, gated, lambda **k: gated(second=True, **k)):
        assert call(b=None) == INVAL and call(s=None) == INVAL and call(a=None) == INVAL
        assert call(y=None) == INVAL
        assert call(rows=0) == INVAL and call(K=0) == INVAL and call(n=0) == INVAL and call(n=-1) == INVAL
        assert call(dt=3) == INVAL and call(dt=-1) == INVAL and call(act=6) == INVAL and call(act=-1) == INVAL
        assert call(K=192) == SHAPE and call(q=2 * FAR, rows=63) == SHAPE
        assert call(b=FAKE + 8) == ALIGN and call(s=FAKE + 8) == ALIGN and call(a=FAKE + 1) == ALIGN
        assert call(bias=FAKE + 2) == ALIGN and call(y=FAR + 2) == ALIGN and call(y=FAR + 1, dt=F16) == ALIGN
        assert call(q=2 * FAR + 1) == ALIGN
        assert call(rows=(1 << 31) - 32) == RANGE and call(K=1 << 21) == RANGE and call(n=(1 << 20) + 1) == RANGE
        assert call(n=5) == INVAL and call(n=5, ws=FAKE, wb=100 * 256 + 5 * (1 << 19) - 1) == RANGE and call(n=5, ws=FAKE + 8, wb=1 << 24) == ALIGN
        assert call(rows=(1 << 26) + 32) == RANGE and call(rows=1 << 26, n=1025, ws=FAKE, wb=1 << 30) == RANGE
        assert call(rows=BIG) == RANGE and call(n=BIG) == RANGE and call(K=BIG) == RANGE
        assert call(y=FAKE) == INVAL and call(q=FAKE) == INVAL and call(q=FAR) == INVAL   # on top of what is read or written
    assert linear(res=FAKE + 2) == ALIGN
    assert linear(res=FAR + 4) == INVAL and linear(res=2 * FAR, q=2 * FAR + 64) == INVAL
    assert "overlap" in L.gemm_decode_last_error().decode()


def test_linear_workspace(gd):
    L, b = gd.lib(), ctypes.c_size_t(7)
    f = L.q1_q8_linear_workspace_bytes
    assert f(256, 4, ctypes.byref(b)) == 0 and b.value == 0
    assert f(256, 5, ctypes.byref(b)) == 0 and b.value == 100 * 256 + 5 * (1 << 19)
    assert f(256, 33, ctypes.byref(b)) == 0 and b.value == 200 * 256 + (1 << 24)
    assert f(256, 5, None) == INVAL and f(0, 5, ctypes.byref(b)) == INVAL and f(256, 0, ctypes.byref(b)) == INVAL
    assert f(130, 5, ctypes.byref(b)) == SHAPE and f(1 << 21, 5, ctypes.byref(b)) == RANGE and f(256, BIG, ctypes.byref(b)) == RANGE


def test_sandwich_refusals(gd):
    L = gd.lib()
    for fn, given in ((L.rmsnorm_sandwich_q8_0, (FAKE,)), (L.rmsnorm_sandwich_ternary_act, (FAKE, FAKE))):
        def call(x=FAKE, p=FAKE, g=FAKE, ng=2, gi=None, r=FAKE, rs=1.0, bs=1.0, w=FAKE, h=FAR, out=given, n=2, K=64, eps=1e-5,
                 dt=F32):
            return fn(x, p, g, ng, gi, r, rs, bs, w, h, *out, n, K, eps, dt, None)
        assert call(x=None) == INVAL and call(r=None) == INVAL and call(w=None) == INVAL
        assert call(out=(None,) * len(given)) == INVAL and call(out=(FAKE,) * (len(given) - 1) + (None,)) == INVAL
        assert call(n=0) == INVAL and call(K=0) == INVAL and call(dt=3) == INVAL
        for bad in (float("nan"), float("inf"), -float("inf")):
            assert call(eps=bad) == INVAL and call(rs=bad) == INVAL and call(bs=bad) == INVAL
        assert call(eps=-1e-6) == INVAL
        assert call(ng=0) == INVAL and call(ng=3) == INVAL and call(ng=-1, gi=FAKE) == INVAL
        assert call(g=None, gi=FAKE) == INVAL
        assert call(K=48) == SHAPE
        assert call(x=FAKE + 8) == ALIGN and call(p=FAKE + 4) == ALIGN and call(g=FAKE + 8) == ALIGN and call(r=FAKE + 8) == ALIGN
        assert call(w=FAKE + 8) == ALIGN and call(h=FAR + 8) == ALIGN and call(gi=FAKE + 2) == ALIGN
        assert call(out=tuple(p + 1 for p in given)) == ALIGN
        assert call(n=1 << 23, ng=1) == RANGE and call(K=(1 << 30) + 32) == RANGE and call(ng=1 << 23, gi=FAKE) == RANGE
        assert call(n=BIG) == RANGE and call(K=BIG) == RANGE and call(ng=BIG, gi=FAKE) == RANGE
        assert call(h=FAKE + 16) == INVAL and call(r=FAR, h=FAR + 256) == INVAL and call(g=2 * FAR, h=2 * FAR) == INVAL


def test_outputs_on_top_of_inputs_are_refused(gd):
    """Any output on any input, or on another output, by one byte."""
    L = gd.lib()
    n, K, A = 3, 64, [FAKE * (i + 1) for i in range(8)]
    ends = {"x": n * K * 4, "r": n * K * 4, "g": K * 4, "h": n * K * 4}
    for q8 in (True, False):
        def norm(**kw):
            at = dict(zip("xrghos", A), **kw)
            given = (at["o"],) if q8 else (at["o"], at["s"])
            fn = L.rmsnorm_sandwich_q8_0 if q8 else L.rmsnorm_sandwich_ternary_act
            return fn(at["x"], A[7], at["g"], 1, None, at["r"], 1.0, 1.0, A[7], at["h"], *given, n, K, 1e-5, F32, None)
        for name, bytes_ in ends.items():
            base = dict(zip("xrgh", A))[name]
            for out in ("o",) if q8 else ("o", "s"):
                assert norm(**{out: base}) == INVAL and norm(**{out: base + bytes_ - 4}) == INVAL
                assert "overlap" in L.gemm_decode_last_error().decode()
        if not q8:
            assert norm(s=A[4] + n * K - 4) == INVAL and "overlap" in L.gemm_decode_last_error().decode()

    V, m, k = 100, 2, 5

    def logprobs(**kw):
        at = dict(zip("xtleio", A), **kw)
        return L.token_logprobs(at["x"], 104, at["t"], m, at["l"], at["e"], at["i"], at["o"], k, n, V, 1.0, 0.0, F32, None, 0, None)
    outs = {"l": n * m * 4, "e": n * 4, "i": n * k * 8, "o": n * k * 4}
    for name in outs:
        for base, last in ((A[0], 2 * 104 * 4 + V * 4 - 8), (A[1], n * m * 8 - 8)):
            assert logprobs(**{name: base}) == INVAL and logprobs(**{name: base + last}) == INVAL
            assert "overlap" in L.gemm_decode_last_error().decode()
        for other, bytes_ in outs.items():
            if other != name:
                assert logprobs(**{name: dict(zip("xtleio", A))[other] + bytes_ // 8 * 8 - 8}) == INVAL
                assert "overlap" in L.gemm_decode_last_error().decode()


def test_logprobs_refusals(gd):
    L = gd.lib()

    def call(x=FAKE, st=100, t=FAKE, m=1, lp=FAKE, e=FAKE, i=FAKE, tl=FAKE, k=5, n=2, V=100, s=1.0, c=0.0, dt=F32, ws=None, wb=0):
        return L.token_logprobs(x, st, t, m, lp, e, i, tl, k, n, V, s, c, dt, ws, wb, None)
    assert call(x=None) == INVAL and call(t=None) == INVAL and call(lp=None) == INVAL and call(i=None) == INVAL
    assert call(tl=None) == INVAL and call(m=0, t=None, lp=None, e=None, i=None, tl=None, k=0) == INVAL
    assert call(n=0) == INVAL and call(V=0) == INVAL and call(k=-1) == INVAL and call(m=-1) == INVAL and call(st=99) == INVAL
    assert call(dt=3) == INVAL
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(s=bad) == INVAL
    for bad in (-1.0, float("nan"), float("inf"), 2e30, 9e-5, 1e-40):
        assert call(c=bad) == INVAL
    assert call(s=2e30) == INVAL and call(s=1e20, c=1e11) == INVAL
    assert call(x=FAKE + 2) == ALIGN and call(x=FAKE + 1, dt=BF16) == ALIGN and call(t=FAKE + 4) == ALIGN
    assert call(lp=FAKE + 2) == ALIGN and call(e=FAKE + 2) == ALIGN and call(i=FAKE + 4) == ALIGN and call(tl=FAKE + 2) == ALIGN
    assert call(k=65) == RANGE and call(n=1 << 23) == RANGE and call(V=(1 << 30) + 1, st=BIG) == RANGE
    assert call(st=(1 << 40) + 1) == RANGE and call(m=65537) == RANGE and call(m=65536, n=1 << 15) == RANGE
    assert call(n=BIG) == RANGE and call(V=BIG, st=BIG) == RANGE


def test_logprobs_workspace(gd):
    """Never less for a larger call."""
    L, b = gd.lib(), ctypes.c_size_t()
    f = L.token_logprobs_workspace_bytes
    assert f(1, 100, 5, None) == INVAL and f(0, 100, 5, ctypes.byref(b)) == INVAL and f(1, 0, 5, ctypes.byref(b)) == INVAL
    assert f(1, 100, 65, ctypes.byref(b)) == RANGE and f(1 << 23, 100, 5, ctypes.byref(b)) == RANGE
    sizes = {}
    grid = [(n, V, k) for n in (1, 2, 3, 7, 60, 300, 5000) for V in (1, 64, 5000, 33000, 50021, 131073, 1 << 22) for k in (0, 1, 20, 64)]
    for s in grid:
        assert f(*s, ctypes.byref(b)) == 0
        sizes[s] = b.value
    for s in grid:
        for t in grid:
            if all(x <= y for x, y in zip(s, t)):
                assert sizes[s] <= sizes[t], (s, t)
