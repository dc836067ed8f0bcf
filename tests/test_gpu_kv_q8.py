"""GPU parity of the rotary table, the rotating cache write and the read back.

The rules fix every rounding (keys: sums of products to 2^-46 rounded to f32,
compared with f64's sums: a row differs if one of its values lies within 2^-46 of
a rounding border and next to a half of its code step, less than once in 10^11;
queries: the second product rounded to f32, then one fused step; the quantization rule, f32(code) * f32(scale)), so rows, codes and scales are
compared bit for bit."""
import numpy as np
import pytest

from oracle import layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 2.5},
            {"kind": "yarn", "factor": 8.0, "original_len": 4096, "low": 1, "high": 32},
            {"kind": "yarn", "factor": 2.0, "original_len": 64, "low": 1, "high": 32, "attention": 0.75},
            {"kind": "llama3", "factor": 8.0, "original_len": 8192, "low": 1, "high": 4}]


def scaling_of(gd, s):
    if s is None:
        return None
    kind = {"linear": gd.ROPE_LINEAR, "ntk": gd.ROPE_NTK, "yarn": gd.ROPE_YARN, "llama3": gd.ROPE_LLAMA3}[s["kind"]]
    return gd.RopeScaling(kind, **{k: v for k, v in s.items() if k != "kind"})


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("n_pos,rot,base", [(1, 8, 10000.0), (131, 64, 10000.0), (5000, 128, 500000.0), (77, 256, 1e6)])
def test_table(gd, scaling, n_pos, rot, base):
    """One f32 rounding of the f64 value: half a step (2^-24 of a value below 2, so 2^-24), and the f64 angle's own error,
    position * 2^-52 at most."""
    t = torch.full((n_pos, rot // 2, 2), float("nan"), device="cuda")
    gd.rope_table(t, n_pos, rot, base, scaling_of(gd, scaling))
    want = layer.rope_table(n_pos, rot, base, scaling)
    err = np.abs(t.cpu().numpy().astype(np.float64) - want)
    assert err.max() <= max(1.0, np.abs(want).max()) * (2.0 ** -24 + n_pos * 2.0 ** -50)


def test_table_far_positions(gd):
    """Positions where a f32 angle would be off by whole turns' fractions."""
    n_pos = 1 << 20
    t = torch.empty(n_pos, 4, 2, device="cuda")
    gd.rope_table(t, n_pos, 8, 10000.0)
    got = t[-3:].cpu().numpy().astype(np.float64)
    f, _ = layer.rope_freqs(8, 10000.0)
    a = np.arange(n_pos - 3, n_pos)[:, None] * f
    assert np.abs(got - np.stack([np.cos(a), np.sin(a)], -1)).max() <= 2.0 ** -24 + n_pos * 2.0 ** -50


def pool(gd, pages, page, heads, dim, seed=0):
    """A pool filled with noise, NaN scales among it: rows that are not stored must stay, and must not matter."""
    c = gd.kv_q8_alloc(pages, page, heads, dim)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k_codes, c.v_codes):
        t.random_(-128, 128, generator=g)
    for t in (c.k_scales, c.v_scales):
        t.view(torch.int16).random_(-32768, 32768, generator=g)
    return c


def bits(c):
    return [t.clone() for t in (c.k_codes, c.k_scales.view(torch.int16), c.v_codes, c.v_scales.view(torch.int16))]


CASES = [  # n_tok, heads, kv_heads, dim, rot, interleaved, page
    (1, 8, 2, 128, 128, False, 16), (1, 4, 4, 64, 64, True, 32), (37, 6, 2, 64, 32, False, 48), (19, 5, 5, 128, 64, True, 16),
    (1025, 3, 2, 64, 64, False, 32), (1030, 2, 1, 128, 40, True, 16), (13, 3, 1, 256, 256, False, 16), (9, 2, 2, 256, 24, True, 16), (5, 1, 1, 128, 8, False, 32), (70, 16, 8, 128, 128, True, 16)]


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("n,H,Hkv,D,rot,inter,page", CASES)
def test_store_and_load(gd, T, n, H, Hkv, D, rot, inter, page):
    rng = np.random.default_rng(n * D + rot)
    x = torch.from_numpy(rng.standard_normal((n, H + 2 * Hkv, D)).astype(np.float32) * 3).to(T)
    x[n // 2, H] = 0                                        # a zero key row
    table = layer.rope_table(50, rot, 10000.0).astype(np.float32)
    pos = rng.integers(0, 50, n).astype(np.int32)
    pages = -(-n // page) + 2
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    c = pool(gd, pages, page, Hkv, D)
    before = bits(c)
    rows = x.cuda()
    q, k, v = rows.split([H, Hkv, Hkv], dim=1)               # parts of one row, token-strided
    q_out = torch.full((n, H, D), float("nan"), dtype=T, device="cuda")
    gd.kv_q8_store(c, k, v, dev(slots), n, q=q, q_out=q_out, n_heads=H, rope=dev(table), positions=dev(pos),
                   interleaved=inter)
    xf = x.float().numpy()
    want_q = torch.from_numpy(layer.rotate(xf[:, :H], table, pos, inter, fused=True)).to(T)
    assert torch.equal(q_out.cpu(), want_q)
    turned = layer.rotate(xf[:, H:H + Hkv], table, pos, inter)
    for name, want in (("k", turned), ("v", xf[:, H + Hkv:])):
        codes, d = layer.q8_rows(want)
        at = (slots // page, slice(None), slots % page)
        got_c, got_d = getattr(c, name + "_codes").cpu().numpy(), getattr(c, name + "_scales").cpu().numpy()
        assert np.array_equal(got_c[at], codes) and np.array_equal(got_d[at], d)
    # nothing else was touched
    untouched = torch.ones(pages, page, dtype=torch.bool)
    untouched[torch.from_numpy(slots // page), torch.from_numpy(slots % page)] = False
    for b, a in zip(before, bits(c)):
        same = (b == a).all(-1).all(1).cpu()                 # [pages, page]
        assert bool(same[untouched].all())
    assert torch.equal(rows.cpu(), x)
    # and back, in another order, one slot twice, one outside the pool
    order = rng.permutation(n)
    ask = np.concatenate([slots[order], slots[:1], [-1, pages * page]])
    ko, vo = (torch.full((n + 3, Hkv, D), float("nan"), dtype=T, device="cuda") for _ in range(2))
    gd.kv_q8_load(c, dev(ask), ko, vo, n + 3)
    for got, want in ((ko, turned), (vo, xf[:, H + Hkv:])):
        codes, d = layer.q8_rows(want)
        val = codes.astype(np.float32) * np.repeat(d.astype(np.float32), 32, -1)
        val = np.concatenate([val[order], val[:1], np.zeros((2, Hkv, D), np.float32)])
        assert torch.equal(got.cpu(), torch.from_numpy(val).to(T))
    k1 = torch.empty_like(ko)
    gd.kv_q8_load(c, dev(ask), k1, None, n + 3)
    gd.kv_q8_load(c, dev(ask), None, vo, n + 3)
    assert torch.equal(k1, ko)


def test_padding_positions_and_no_rotation(gd):
    """Slots outside the pool are not stored, positions outside the table leave the token out, and without a table nothing
    is rotated; queries may be turned in place or be absent."""
    n, H, Hkv, D = 6, 4, 2, 64
    rng = np.random.default_rng(3)
    x = rng.standard_normal((n, H + 2 * Hkv, D)).astype(np.float32)
    q, k, v = dev(x[:, :H]), dev(x[:, H:H + Hkv]), dev(x[:, H + Hkv:])
    table = layer.rope_table(10, 64, 10000.0).astype(np.float32)
    slots = np.array([3, -1, 5, 64, 1 << 40, 7], np.int64)   # a pool of 64
    pos = np.array([1, 2, 10, 3, 4, -1], np.int32)
    c = pool(gd, 2, 32, Hkv, D)
    before = bits(c)
    q_out = torch.full((n, H, D), 9.0, device="cuda")
    gd.kv_q8_store(c, k, v, dev(slots), n, q=q, q_out=q_out, n_heads=H, rope=dev(table), positions=dev(pos))
    turned = layer.rotate(x[:, :H], table, np.clip(pos, 0, 9), False, fused=True)
    got = q_out.cpu().numpy()
    assert np.array_equal(got[[0, 1, 3, 4]], turned[[0, 1, 3, 4]]) and (got[[2, 5]] == 9).all()
    changed = [(b != a).any(-1).any(1).nonzero().tolist() for b, a in zip(before, bits(c))]
    assert all(p in ([[0, 3]], []) for p in changed) and changed[0] and changed[2]
    # in place, no table
    c = pool(gd, 2, 32, Hkv, D)
    gd.kv_q8_store(c, k, v, dev(np.arange(n)), n)
    assert np.array_equal(c.k_codes[0, :, :n].cpu().numpy().transpose(1, 0, 2), layer.q8_rows(x[:, H:H + Hkv])[0])
    gd.kv_q8_store(c, k, v, dev(np.arange(n)), n, q=q, q_out=q, n_heads=H, rope=dev(table),
                   positions=dev(np.arange(n, dtype=np.int32)))
    assert np.array_equal(q.cpu().numpy(), layer.rotate(x[:, :H], table, np.arange(n), False, fused=True))
    same = torch.empty_like(q)
    gd.kv_q8_store(c, k, v, dev(np.arange(n)), n, q=q, q_out=same, n_heads=H)
    assert torch.equal(same, q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", TYPES)
def test_rotation_in_place(gd, D, T):
    n, H = 33, 5
    rng = np.random.default_rng(D)
    x = torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float32)).to(T)
    table = layer.rope_table(64, D, 10000.0).astype(np.float32)
    pos = rng.integers(0, 64, n).astype(np.int32)
    kv = torch.zeros(n, 1, D, dtype=T, device="cuda")
    for inter in (False, True):
        q = x.cuda()
        c = pool(gd, 3, 16, 1, D)
        gd.kv_q8_store(c, kv, kv, dev(np.arange(n)), n, q=q, q_out=q, n_heads=H, rope=dev(table), positions=dev(pos),
                       interleaved=inter)
        assert torch.equal(q.cpu(), torch.from_numpy(layer.rotate(x.float().numpy(), table, pos, inter, fused=True)).to(T))


def test_values_next_to_ties(gd):
    """Rows whose codes fall on exact halves, and rows at both ends of f32's range."""
    rng = np.random.default_rng(5)
    D = 64
    v = (rng.integers(-126, 127, (40, 1, D)) + 0.5).astype(np.float32)
    v[:, :, ::32] = 127
    v[1] *= 2.0 ** -130
    v[2] *= 2.0 ** 10
    v[3] = 0
    v[4] = 1e-45
    c = pool(gd, 3, 16, 1, D)
    k = np.zeros_like(v)
    gd.kv_q8_store(c, dev(k), dev(v), dev(np.arange(40)), 40)
    codes, d = layer.q8_rows(v)
    assert np.array_equal(c.v_codes.view(-1, D)[:40].cpu().numpy(), codes[:, 0])
    assert np.array_equal(c.v_scales.view(-1, 2)[:40].cpu().numpy(), d[:, 0])
    assert not c.k_codes.view(-1, D)[:40].any() and not c.k_scales.view(-1, 2)[:40].any()


def test_graph_replays(gd):
    """One decode step's write and read captured: slots and positions move between replays."""
    n, H, Hkv, D = 3, 4, 2, 128
    rng = np.random.default_rng(6)
    table = dev(layer.rope_table(64, D, 10000.0).astype(np.float32))
    c = pool(gd, 4, 16, Hkv, D)
    q, k, v = (dev(rng.standard_normal((n, h, D)).astype(np.float32)) for h in (H, Hkv, Hkv))
    slots, pos = dev(np.arange(n)), dev(np.arange(n, dtype=np.int32))
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def step(c, qo, ko, vo):
        gd.kv_q8_store(c, k, v, slots, n, q=q, q_out=qo, n_heads=H, rope=table, positions=pos)
        gd.kv_q8_load(c, slots, ko, vo, n)
    step(c, qo, ko, vo)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, qo, ko, vo)
    for i in range(4):
        k.normal_()
        slots.add_(n)
        pos.add_(5)
        graph.replay()
        torch.cuda.synchronize()
        c2 = pool(gd, 4, 16, Hkv, D)
        want = [torch.empty_like(t) for t in (qo, ko, vo)]
        step(c2, *want)
        assert all(torch.equal(a, b) for a, b in zip((qo, ko, vo), want)), i


def test_long_pool_offsets(gd):
    """Rows whose byte offsets pass 2^32: the last page of a 5 GiB plane."""
    heads, D, page = 16, 128, 64
    pages = (5 << 30) // (heads * D * page)
    c = gd.kv_q8_alloc(pages, page, heads, D)
    rng = np.random.default_rng(7)
    x = rng.standard_normal((2, heads, D)).astype(np.float32)
    slots = dev(np.array([pages * page - 1, (pages - 2) * page], np.int64))
    gd.kv_q8_store(c, dev(x), dev(-x), slots, 2)
    ko, vo = (torch.empty(2, heads, D, device="cuda") for _ in range(2))
    gd.kv_q8_load(c, slots, ko, vo, 2)
    codes, d = layer.q8_rows(x)
    want = codes.astype(np.float32) * np.repeat(d.astype(np.float32), 32, -1)
    assert np.array_equal(ko.cpu().numpy(), want)
    codes, d = layer.q8_rows(-x)
    assert np.array_equal(vo.cpu().numpy(), codes.astype(np.float32) * np.repeat(d.astype(np.float32), 32, -1))


def test_refusals(gd):
    c = pool(gd, 2, 16, 1, 64)
    k = torch.zeros(2, 1, 64, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        gd.kv_q8_store(c, k, k.half(), slots, 2)
    with pytest.raises(TypeError):
        gd.kv_q8_store(c, k, k, slots.int(), 2)
    with pytest.raises(ValueError):
        gd.kv_q8_store(c, k, k, slots[:1], 2)
    with pytest.raises(ValueError):
        gd.kv_q8_store(c, k, k, slots, 2, q=k)
    with pytest.raises(ValueError):
        gd.kv_q8_store(c, k[:, :, ::2], k, slots, 2)
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        gd.kv_q8_store(c, k, k, slots, 2, positions=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(gd.GemmDecodeError, match="GD_ESHAPE"):
        gd.kv_q8_store(c, k, k, slots, 2, rope=torch.zeros(4, 36, 2, device="cuda"),
                       positions=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="empty"):
        gd.kv_q8_store(c, k, k, slots, 2, rope=torch.zeros(0, 32, 2, device="cuda"))
    with pytest.raises(TypeError):
        gd.kv_q8_load(c, slots, None, None, 2)
    with pytest.raises(gd.GemmDecodeError, match="GD_ESHAPE"):
        gd.kv_q8_load(gd.kv_q8_alloc(2, 20, 1, 64), slots, k, k, 2)


def test_outputs_beside_the_inputs(gd):
    """q_out right behind q, between the rows of a wide projection, and (one token) at q inside a fused row: none of them
    overlaps what is read."""
    n, H, D = 2, 2, 64
    rng = np.random.default_rng(12)
    table = layer.rope_table(8, D, 10000.0).astype(np.float32)
    pos, slots = np.array([3, 5], np.int32), dev(np.arange(n))
    c = pool(gd, 1, 16, 1, D)
    x = rng.standard_normal((n, H + 2, D)).astype(np.float32)
    want = layer.rotate(x[:, :H], table, pos, False, fused=True)
    buf = torch.full((n, 16, D), 7.0, device="cuda")         # a token's row, with room behind its heads
    buf[:, :H + 2] = dev(x)
    room = buf.view(-1)[(H + 2) * D:(H + 2) * D + n * H * D].view(n, H, D)
    q, k, v = buf[:, :H], buf[:, H:H + 1], buf[:, H + 1:H + 2]
    gd.kv_q8_store(c, k, v, slots, n, q=q, q_out=room, n_heads=H, rope=dev(table), positions=dev(pos))
    assert np.array_equal(room.cpu().numpy(), want)
    assert np.array_equal(buf[:, :H + 2].cpu().numpy(), x) and bool((buf.view(-1)[(H + 2 + n * H) * D:16 * D] == 7).all())
    both = torch.cat([dev(x[:, :H]).view(-1), torch.zeros(n * H * D, device="cuda")]).view(2, n, H, D)
    gd.kv_q8_store(c, k, v, slots, n, q=both[0], q_out=both[1], n_heads=H, rope=dev(table), positions=dev(pos))
    assert np.array_equal(both.cpu().numpy(), np.stack([x[:, :H], want]))
    one = dev(x[:1])
    gd.kv_q8_store(c, one[:, H:H + 1], one[:, H + 1:], slots[:1], 1, q=one[:, :H], q_out=one[:, :H], n_heads=H, rope=dev(table),
                   positions=dev(pos[:1]))
    assert np.array_equal(one.cpu().numpy()[:, :H], want[:1]) and np.array_equal(one.cpu().numpy()[:, H:], x[:1, H:])
    with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
        gd.kv_q8_store(c, k, v, slots, n, q=both[0], q_out=both.view(-1)[64:64 + n * H * D].view(n, H, D), n_heads=H)
