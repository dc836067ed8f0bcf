"""Argument checks of the norm, rotary, 8-bit cache and attention entry points
on a host without a GPU: the documented status before any HIP call (no compute
is launched here)."""
import ctypes

import pytest

FAKE = 0x100000   # an aligned address that is never dereferenced: validation fails first
INVAL, SHAPE, ALIGN, RANGE = -1, -2, -3, -5
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def gd():
    import gemm_decode_amd
    return gemm_decode_amd


def test_norm_refusals(gd):
    L = gd.lib()
    for fn, out in ((L.rmsnorm_q8_0, (FAKE,)), (L.rmsnorm_ternary_act, (FAKE, FAKE))):
        def call(x=FAKE, r=FAKE, w=FAKE, h=FAKE, out=out, n=2, K=64, eps=1e-5, dt=F32):
            return fn(x, r, w, h, *out, n, K, eps, dt, None)
        assert call(x=None) == INVAL and call(w=None) == INVAL and call(out=(None,) * len(out)) == INVAL
        assert call(n=0) == INVAL and call(K=0) == INVAL and call(n=-1) == INVAL
        assert call(K=48) == SHAPE
        assert call(dt=3) == INVAL and call(dt=-1) == INVAL
        assert call(eps=-1e-6) == INVAL and call(eps=float("nan")) == INVAL and call(eps=float("inf")) == INVAL
        assert call(x=FAKE + 8) == ALIGN and call(r=FAKE + 4) == ALIGN and call(h=FAKE + 2) == ALIGN
        assert call(w=FAKE + 4) == ALIGN and call(out=tuple(p + 1 for p in out)) == ALIGN
        assert call(n=1 << 23) == RANGE and call(K=(1 << 30) + 32) == RANGE
        assert "large" in L.gemm_decode_last_error().decode()


def test_reader_refusals(gd):
    L = gd.lib()
    assert L.q8_0_dequantize(None, FAKE, 1, 32, F32, None) == INVAL
    assert L.q8_0_dequantize(FAKE, FAKE, 1, 33, F32, None) == SHAPE
    assert L.q8_0_dequantize(FAKE + 1, FAKE, 1, 32, F32, None) == ALIGN
    assert L.q8_0_dequantize(FAKE, FAKE + 8, 1, 32, F32, None) == ALIGN
    assert L.q8_0_dequantize(FAKE, FAKE, 1, 32, 9, None) == INVAL
    assert L.q8_0_dequantize(FAKE, FAKE, 1 << 30, 1 << 20, F32, None) == RANGE
    assert L.q8_0_dequantize(FAKE, FAKE, 1 << 62, 1 << 20, F32, None) == RANGE
    assert L.ternary_dequantize_act(FAKE, None, FAKE, 1, 32, F32, None) == INVAL
    assert L.ternary_dequantize_act(FAKE, FAKE + 2, FAKE, 1, 32, F32, None) == ALIGN
    assert L.ternary_dequantize_act(FAKE, FAKE, FAKE, 0, 32, F32, None) == INVAL


def test_rope_table_refusals(gd):
    L = gd.lib()

    def call(t=FAKE, n=16, rot=64, base=1e4, s=None):
        return L.rope_table(t, n, rot, base, None if s is None else ctypes.addressof(s), None)
    assert call(t=None) == INVAL and call(n=0) == INVAL and call(rot=0) == INVAL
    assert call(base=1.0) == INVAL and call(base=float("nan")) == INVAL and call(base=float("inf")) == INVAL
    assert call(rot=60) == SHAPE and call(rot=264) == RANGE and call(n=1 << 31) == RANGE
    assert call(n=(1 << 31) - 1, rot=8) == RANGE
    assert call(t=FAKE + 8) == ALIGN
    S = gd.RopeScaling
    assert call(s=S(7)) == INVAL and call(s=S(-1)) == INVAL
    assert call(s=S(gd.ROPE_LINEAR, 0.5)) == INVAL and call(s=S(gd.ROPE_NTK, float("nan"))) == INVAL
    assert call(s=S(gd.ROPE_YARN, 2.0, 0.0, 1, 32)) == INVAL
    assert call(s=S(gd.ROPE_YARN, 2.0, 4096, 32, 1)) == INVAL
    assert call(s=S(gd.ROPE_YARN, 2.0, 4096, 1, 32, -1.0)) == INVAL
    assert call(s=S(gd.ROPE_LLAMA3, 2.0, 4096, 0, 4)) == INVAL


def cache(gd, planes=(FAKE,) * 4, n_pages=4, page=32, heads=2, dim=64):
    from gemm_decode_amd import _KVQ8
    c = _KVQ8(*planes, n_pages, page, heads, dim)
    return c, ctypes.addressof(c)


BAD_CACHES = [
    (dict(planes=(None, FAKE, FAKE, FAKE)), INVAL), (dict(planes=(FAKE, FAKE, FAKE, None)), INVAL),
    (dict(planes=(FAKE, FAKE, FAKE + 8, FAKE)), ALIGN), (dict(n_pages=0), INVAL), (dict(page=0), INVAL),
    (dict(page=24), SHAPE), (dict(heads=0), INVAL), (dict(heads=4097), RANGE), (dict(dim=96), SHAPE),
    (dict(dim=512), SHAPE), (dict(n_pages=1 << 31), RANGE), (dict(n_pages=1 << 30, page=1 << 20), RANGE)]


def store(gd, ref, q=FAKE, qs=128, k=FAKE, ks=128, v=FAKE, vs=128, qo=FAKE, rope=FAKE, n_pos=8, rot=64, pos=FAKE,
          slots=FAKE, n=3, heads=2, dt=F32):
    return gd.lib().kv_q8_store(ref, q, qs, k, ks, v, vs, qo, rope, n_pos, rot, 0, pos, slots, n, heads, dt, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_refusals(gd, bad, status):
    keep, ref = cache(gd, **bad)
    L = gd.lib()
    assert store(gd, ref) == status
    assert L.kv_q8_load(ref, FAKE, FAKE, FAKE, 3, F32, None) == status
    assert attn(gd, ref) == status
    assert store(gd, None) == INVAL


def test_store_refusals(gd):
    keep, ref = cache(gd)
    assert store(gd, ref, k=None) == INVAL and store(gd, ref, v=None) == INVAL and store(gd, ref, slots=None) == INVAL
    assert store(gd, ref, q=None) == INVAL and store(gd, ref, qo=None) == INVAL
    assert store(gd, ref, n=0) == INVAL and store(gd, ref, heads=-1) == INVAL and store(gd, ref, dt=5) == INVAL
    assert store(gd, ref, rope=None) == INVAL and store(gd, ref, pos=None) == INVAL
    assert store(gd, ref, n_pos=0) == INVAL and store(gd, ref, rot=0) == INVAL
    assert store(gd, ref, rot=12) == SHAPE and store(gd, ref, rot=72) == SHAPE
    assert store(gd, ref, qs=127) == SHAPE and store(gd, ref, ks=126) == SHAPE and store(gd, ref, vs=130) == SHAPE
    assert store(gd, ref, vs=132, dt=BF16) == SHAPE          # 264 bytes are no multiple of 16
    assert store(gd, ref, k=FAKE + 8) == ALIGN and store(gd, ref, slots=FAKE + 4) == ALIGN
    assert store(gd, ref, rope=FAKE + 8) == ALIGN and store(gd, ref, qo=FAKE + 4) == ALIGN
    assert store(gd, ref, n=1 << 31, heads=64, qs=4096) == RANGE
    assert store(gd, ref, n=1 << 62) == RANGE
    big = (1 << 63) - 16
    assert store(gd, ref, heads=1 << 60, qs=big) == RANGE and store(gd, ref, heads=65537, qs=65537 * 64) == RANGE
    assert store(gd, ref, ks=big) == RANGE and store(gd, ref, vs=big) == RANGE and store(gd, ref, qs=big) == RANGE
    assert store(gd, ref, ks=-128) == SHAPE and store(gd, ref, n=-3) == INVAL


def test_store_refuses_rotation_in_place_of_strided_queries(gd):
    """q_out is contiguous: with q_out at q, the rows of a wider q would be overwritten before they are read."""
    keep, ref = cache(gd)
    assert store(gd, ref, q=FAKE, qo=FAKE, n=2, heads=2, qs=2 * 64 + 32) == INVAL
    assert "q_stride" in gd.lib().gemm_decode_last_error().decode()


def test_load_refusals(gd):
    keep, ref = cache(gd)
    L = gd.lib()
    assert L.kv_q8_load(ref, None, FAKE, FAKE, 3, F32, None) == INVAL
    assert L.kv_q8_load(ref, FAKE, None, None, 3, F32, None) == INVAL
    assert L.kv_q8_load(ref, FAKE, FAKE, FAKE, 0, F32, None) == INVAL
    assert L.kv_q8_load(ref, FAKE, FAKE, FAKE, 3, 4, None) == INVAL
    assert L.kv_q8_load(ref, FAKE + 4, FAKE, FAKE, 3, F32, None) == ALIGN
    assert L.kv_q8_load(ref, FAKE, FAKE + 4, FAKE, 3, F32, None) == ALIGN
    assert L.kv_q8_load(ref, FAKE, FAKE, FAKE, 1 << 31, F32, None) == RANGE


def attn(gd, ref, q=FAKE, out=FAKE, table=FAKE, max_pages=8, lens=FAKE, start=FAKE, tree=None, n_seqs=2, n_q=3,
         heads=4, max_q=2, max_len=200, scale=0.1, cap=0.0, dt=F32, ws=FAKE, ws_bytes=1 << 40):
    return gd.lib().attn_decode_q8(ref, q, out, table, max_pages, lens, start, tree, n_seqs, n_q, heads, max_q,
                                   max_len, scale, cap, dt, ws, ws_bytes, None)


def test_attention_refusals(gd):
    keep, ref = cache(gd)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(q=None), dict(out=None), dict(lens=None), dict(n_seqs=0), dict(n_q=0), dict(heads=0),
                dict(max_q=0), dict(max_len=0), dict(dt=3), dict(scale=nan), dict(scale=inf), dict(cap=-1.0),
                dict(cap=nan), dict(cap=inf), dict(cap=2e30), dict(ws=None), dict(max_pages=0), dict(max_len=257),
                dict(start=None), dict(table=None, max_len=33), dict(table=None, n_seqs=5, n_q=5, max_len=20)):
        assert attn(gd, ref, **bad) == INVAL, bad
    assert attn(gd, ref, heads=3) == SHAPE
    for bad in (dict(q=FAKE + 8), dict(out=FAKE + 4), dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(start=FAKE + 2),
                dict(tree=FAKE + 4), dict(ws=FAKE + 8)):
        assert attn(gd, ref, **bad) == ALIGN, bad
    for bad in (dict(max_q=65), dict(n_q=5), dict(heads=8192), dict(n_seqs=65536, n_q=3), dict(max_len=(1 << 30) + 1),
                dict(ws_bytes=8)):
        assert attn(gd, ref, **bad) == RANGE, bad


def test_attention_huge_sizes_do_not_overflow(gd):
    keep, ref = cache(gd)
    big = (1 << 63) - 1
    for bad in (dict(n_seqs=big), dict(n_q=big), dict(heads=big - 1), dict(max_q=big), dict(max_len=big)):
        assert attn(gd, ref, **bad) in (RANGE, SHAPE), bad
    assert attn(gd, ref, max_pages=big) == RANGE
    assert attn(gd, ref, max_pages=-1) == INVAL and attn(gd, ref, max_len=-1) == INVAL and attn(gd, ref, n_q=-1) == INVAL


def test_attention_workspace(gd):
    b = ctypes.c_size_t()
    L = gd.lib()
    assert L.attn_decode_q8_workspace_bytes(2, 3, 4, 2, 64, 2, 200, None) == INVAL
    assert L.attn_decode_q8_workspace_bytes(2, 3, 4, 2, 64, 2, 0, ctypes.byref(b)) == INVAL
    assert L.attn_decode_q8_workspace_bytes(2, 3, 4, 3, 64, 2, 200, ctypes.byref(b)) == SHAPE
    assert L.attn_decode_q8_workspace_bytes(2, 3, 4, 2, 80, 2, 200, ctypes.byref(b)) == SHAPE
    assert L.attn_decode_q8_workspace_bytes(2, 3, 4, 2, 64, 65, 200, ctypes.byref(b)) == RANGE
    # never more than a partial per split of 64 keys and query row
    for args in ((1, 1, 32, 8, 128, 1, 32768), (7, 100, 64, 8, 256, 64, 4097), (65535, 65535, 8, 8, 64, 1, 16)):
        assert L.attn_decode_q8_workspace_bytes(*args, ctypes.byref(b)) == 0
        n_q, heads, dim, length = args[1], args[2], args[4], args[6]
        assert 16 <= b.value <= 16 + n_q * heads * (dim + 2) * 4 * -(-length // 64)


def test_attention_workspace_of_the_largest_call_serves_the_smaller_ones(gd):
    """Fewer sequences, rows, query tokens or keys never need more (a plan may cut a smaller call into more parts)."""
    L, b = gd.lib(), ctypes.c_size_t()

    def need(*args):
        assert L.attn_decode_q8_workspace_bytes(*args, ctypes.byref(b)) == 0, args
        return b.value
    assert need(1, 1, 32, 8, 128, 1, 8192) <= need(1, 1, 32, 8, 128, 1, 8320)
    assert need(31, 31, 32, 8, 128, 1, 1024) <= need(32, 32, 32, 8, 128, 1, 1024)
    for heads, kv, dim in ((32, 8, 128), (8, 2, 64), (16, 1, 256), (40, 40, 128), (4096, 4096, 64)):
        for seqs in (1, 3, 32, 300):
            prev = 0
            for length in range(1, 40000, 517):
                now = need(seqs, seqs, heads, kv, dim, 1, length)
                assert now >= prev, (heads, kv, dim, seqs, length)
                prev = now
        for length in (300, 1024, 8192, 1 << 20):
            prev = 0
            for seqs in list(range(1, 70)) + [100, 255, 256, 257, 511, 512, 513, 1000, 4095, 4096, 5000, 65535]:
                now = need(seqs, seqs, heads, kv, dim, 1, length)
                assert now >= prev, (heads, kv, dim, seqs, length)
                prev = now
            for seqs in (1, 5, 40):
                prev = 0
                for max_q in range(1, 65):
                    now = need(seqs, seqs * max_q, heads, kv, dim, max_q, length)
                    assert now >= prev, (heads, kv, dim, seqs, max_q, length)
                    assert need(seqs, seqs * max_q - (max_q > 1), heads, kv, dim, max_q, length) <= now
                    prev = now


def test_outputs_that_overlap_inputs_are_refused(gd):
    """Rows are read and written by workgroups in any order: an output on top of an input is refused unless it is one of the
    documented in-place calls."""
    L = gd.lib()
    keep, ref = cache(gd)
    for at in (0, 16, -16, 3 * 4 * 64 * 4 - 16):      # three rows of 4 heads of 64 in f32
        assert attn(gd, ref, out=FAKE + at) == INVAL and "overlap" in L.gemm_decode_last_error().decode(), at
    for at in (16, -16, 2 * 64 * 4 - 16):             # two rows of 64
        for x, r in ((FAKE, None), (FAKE + (1 << 16), FAKE)):
            assert L.rmsnorm_q8_0(x, r, FAKE, FAKE + at, FAKE, 2, 64, 1e-5, F32, None) == INVAL
            assert L.rmsnorm_ternary_act(x, r, FAKE, FAKE + at, FAKE, FAKE, 2, 64, 1e-5, F32, None) == INVAL
            assert "h_out" in L.gemm_decode_last_error().decode()
    far, row = FAKE + (1 << 20), 2 * 64 * 4           # a token's two heads of 64 in f32: 512 bytes
    for q, qs, qo in ((FAKE, 128, FAKE + 16), (FAKE, 128, FAKE - 16), (FAKE, 192, FAKE + row), (FAKE, 4096, FAKE + 2 * 4096 * 4),
                      (FAKE, 4096, FAKE + row - 16), (FAKE, 4096, FAKE + 4096 * 4 - 3 * row + 16)):
        assert store(gd, ref, q=q, qs=qs, qo=qo, k=far, v=far, ks=128, vs=128) == INVAL, (q, qs, qo)
        assert "q_out" in L.gemm_decode_last_error().decode()
    for name in ("k", "v"):
        args = dict(q=FAKE, qo=FAKE + (1 << 16), k=far, v=far)
        args[name] = FAKE + (1 << 16) + 3 * row - 16
        assert store(gd, ref, **args) == INVAL and "k or v" in L.gemm_decode_last_error().decode()
