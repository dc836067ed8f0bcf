"""Offsets past 32 bits in the products with an epilogue, the norms around a block and the log
probabilities, and calls on two streams at once."""
import numpy as np
import pytest

import workloads as wl
from oracle import answer
from q1_layout import element_position
from test_gpu_answer_path import K, Half, dev
from test_gpu_logprobs import near
from test_gpu_norm_quant import EPS
from test_gpu_norm_sandwich import check, definition
from test_gpu_q1_linear import within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    yield gemm_decode_amd
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gated", [False, True])
def test_outputs_past_2_31_elements(gd, gated):
    """65600 rows of 33000 columns: the first, the last and what lies around 2^31 elements and 2^32 bytes."""
    rows, K, n = 65600, 128, 33000
    rng = np.random.default_rng(11)
    w = [wl.q1_weights_aos(rows, K, 11 + i) for i in range(2)]
    a = wl.q8_acts_aos(K, 18, n)
    p = []
    for x in w:
        b, s = gd.q1_alloc_planes(rows, K)
        gd.q1_repack(dev(x.reshape(-1)), rows, K, b, s)
        p += [b, s]
    y = torch.full((n, rows), 9.0, dtype=torch.bfloat16, device="cuda")
    if gated:
        gd.q1_q8_gated(*p, dev(a.reshape(-1)), y, rows, K, n)
    else:
        gd.q1_q8_linear(*p[:2], dev(a.reshape(-1)), y, rows, K, n)
    cols = [0, 1, 31, (1 << 31) // rows, (1 << 31) // rows + 1, (1 << 30) // rows, n - 2, n - 1] + list(rng.integers(0, n, 4))
    v = answer.q8_values(a[cols], len(cols))
    t, off = answer.product(answer.q1_values(w[0]), v, None, 5 if gated else 0)
    if gated:
        u, uoff = answer.product(answer.q1_values(w[1]), v, None, 0)
        off = np.abs(t) * uoff + np.abs(u) * off + off * uoff
        t = t * u
        off = off + 2.0 ** -24 * (np.abs(t) + off)
    within(y[cols], t, off, torch.bfloat16)


def signs_of(bits, rows, K):
    """+1 and -1 of the given rows of a bit plane (int32 [R64/64, K/128, 2, 64, 2]), f64 [len(rows), K]."""
    r = torch.tensor(rows, device="cuda")
    words = bits[r // 64, :, :, r % 64, :].cpu().numpy().view(np.uint32)   # [rows, K/128, half, word]
    out = np.empty((len(rows), K // 128, 128))
    for e in range(128):
        h, m, at = element_position(e)
        out[:, :, e] = 2.0 * (words[:, :, h, m] >> np.uint32(at) & 1) - 1
    return out.reshape(len(rows), K)


@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 40, 600])
def test_weights_past_4_gib(gd, n):
    """A bit plane of 8.6 GB, random signs with scales of 1: rows at its start, around 2^32 bytes and at its end."""
    rows, K = (1 << 21) + 40, 32768
    bb, sb = gd.q1_planes_bytes(rows, K)
    bits = torch.randint(-1 << 63, (1 << 63) - 1, (bb // 8,), dtype=torch.int64, device="cuda").view(torch.uint8)
    scales = torch.full((sb // 2,), 1.0, dtype=torch.float16, device="cuda").view(torch.uint8)
    a = wl.q8_acts_aos(K, 5, n)
    y = torch.empty(n, rows, device="cuda")
    gd.q1_q8_linear(bits, scales, dev(a.reshape(-1)), y, rows, K, n)
    edge = (1 << 32) // (K // 8)
    some = [0, 1, 63, 64, edge - 1, edge, edge + 1, edge + 65, rows // 2 + 77, rows - 64, rows - 40, rows - 2, rows - 1]
    cols = sorted({0, 1 % n, n // 2, n - 1})
    w = signs_of(bits.view(torch.int32).view(-1, K // 128, 2, 64, 2), some, K)
    want, off = answer.product(w, answer.q8_values(a[cols], len(cols)), None, 0)
    within(y[cols][:, some], want, off, torch.float32)


@pytest.mark.parametrize("form", ["q8_0", "ternary"])
def test_norms_past_2_31_elements(gd, form):
    n, K, T = 525000, 4128, torch.bfloat16
    x, res = (torch.randn(n, K, dtype=T, device="cuda") for _ in range(2))
    post, w = (torch.randn(K, device="cuda") * 0.1 + 1 for _ in range(2))
    gate = torch.randn(3, K, device="cuda").to(T)
    index = torch.randint(-1, 4, (n,), device="cuda", dtype=torch.int32)
    h = torch.empty_like(x)
    if form == "q8_0":
        out = (torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda"),)
        gd.rmsnorm_sandwich_q8_0(x, post, res, w, h, *out, n, K, EPS, gate=gate, gate_index=index)
    else:
        out = torch.empty(n * 8 * (K // 32), dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
        gd.rmsnorm_sandwich_ternary_act(x, post, res, w, h, *out, n, K, EPS, gate=gate, gate_index=index)
    for rows in (slice(0, 2), slice((1 << 31) // K - 1, (1 << 31) // K + 2), slice(n - 2, n)):
        part = [o.view(n, -1)[rows].reshape(-1) for o in out]
        i = index[rows].cpu().numpy()
        check(form, part, h[rows], w, T, definition(x[rows], post, res[rows], gate, i, 1.0, 1.0))


def test_logits_past_2_31_elements(gd):
    n, V, k = 2200, 1000003, 5
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    for r in range(0, n, 200):
        x[r:r + 200] = torch.randn(200, V, device="cuda") * 2
    tokens = torch.randint(0, V, (n, 1), device="cuda")
    lp, ent = torch.empty(n, 1, device="cuda"), torch.empty(n, device="cuda")
    ids, tops = torch.empty(n, k, dtype=torch.int64, device="cuda"), torch.empty(n, k, device="cuda")
    gd.token_logprobs(x, tokens, lp, ent, ids, tops, n, V)
    for r in (0, (1 << 31) // V, (1 << 31) // V + 1, n - 1):
        w_lp, w_ent, w_ids, w_tops = answer.logprobs(x[r].float().cpu().numpy(), tokens[r].cpu().numpy(), k)
        assert np.array_equal(ids[r].cpu().numpy(), w_ids)
        near(lp[r], w_lp, 0.0, 1.0)
        near(ent[r:r + 1], np.array([w_ent]), 0.0, 1.0)
        near(tops[r], w_tops, 0.0, 1.0)


def test_two_streams_at_once(gd):
    """Steps of different sizes, enqueued in turn on two streams with workspaces of their own, give what they give alone."""
    m = Half(gd, torch.bfloat16)
    rng = np.random.default_rng(4)
    sizes, args = (40, 9), []
    for n in sizes:
        args.append((dev(rng.standard_normal((n, K)).astype(np.float32)), dev(rng.standard_normal((n, K)).astype(np.float32)).bfloat16(),
                     dev(rng.integers(-1, 3, n).astype(np.int32)), dev(rng.integers(0, 1000, (n, 1)))))
    want = [m.step(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got = []
    for _ in range(12):
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(m.step(*a))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for k, v in want[i % 2].items():
            assert torch.equal(o[k], v), (i, k)
