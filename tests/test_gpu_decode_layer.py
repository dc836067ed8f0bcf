"""The operators around a decode layer's products run together, as a decode loop runs
them: norm with 8-bit output -> fused Q1_0 projection -> rotary cache write -> attention
over the cache (a prompt chunk, single tokens, a drafted tree) -> q8_0 quantization ->
Q1_0 output projection -> residual norm into ternary planes -> ternary GEMV. Each step is compared
with the oracle on the inputs it had, with its own bar; then the loop is captured and replayed."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
H, HKV, D, PAGE = 4, 2, 64, 16
K = H * D
ROWS = (H + 2 * HKV) * D
EPS = 1e-5


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


class Layer:
    def __init__(self, gd, seqs, capacity):
        self.gd = gd
        self.w_qkv, self.w_o = wl.q1_weights_aos(ROWS, K, 1), wl.q1_weights_aos(K, K, 2)
        self.planes = []
        for w, rows in ((self.w_qkv, ROWS), (self.w_o, K)):
            b, s = gd.q1_alloc_planes(rows, K)
            gd.q1_repack(dev(w.reshape(-1)), rows, K, b, s)
            self.planes.append((b, s))
        rng = np.random.default_rng(3)
        self.g1, self.g2 = (dev((1 + 0.1 * rng.standard_normal(K)).astype(np.float32)) for _ in range(2))
        self.tern = wl.ternary_inputs(96, K, 4)
        per = capacity // PAGE
        self.table = dev(rng.permutation(seqs * per).reshape(seqs, per).astype(np.int32))
        self.cache = gd.kv_q8_alloc(seqs * per, PAGE, HKV, D)
        self.rope = torch.empty(capacity, D // 2, 2, device="cuda")
        gd.rope_table(self.rope, capacity, D, 10000.0, gd.RopeScaling(gd.ROPE_LINEAR, 2.0))
        self.capacity = capacity

    def slots(self, seq, at):
        """Slots of position at[i] of sequence seq[i] (device tensors)."""
        return self.table[seq, at // PAGE].long() * PAGE + at % PAGE

    def step(self, x, residual, seq, at, positions, lens, start, tree, max_q, max_len):
        """One layer for n tokens; returns every intermediate."""
        gd, n = self.gd, x.shape[0]
        o = {"h": torch.empty_like(x), "a": torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device="cuda")}
        gd.rmsnorm_q8_0(x, residual, self.g1, o["h"], o["a"], n, K, EPS)
        o["qkv"] = torch.empty(n, H + 2 * HKV, D, device="cuda")
        gd.q1_q8_gemv(*self.planes[0], o["a"], o["qkv"], ROWS, K, n)
        q, k, v = o["qkv"].split([H, HKV, HKV], dim=1)
        o["q"] = torch.empty(n, H, D, device="cuda")
        gd.kv_q8_store(self.cache, k, v, self.slots(seq, at), n, q=q, q_out=o["q"], n_heads=H, rope=self.rope,
                       positions=positions)
        o["attn"] = torch.empty(n, H, D, device="cuda")
        gd.attn_decode_q8(o["q"], self.cache, self.table, lens, start, tree, o["attn"], H, max_q, max_len, D ** -0.5)
        o["a2"] = torch.empty_like(o["a"])
        gd.q8_0_quantize(o["attn"], o["a2"], n, K)
        o["y"] = torch.empty(n, K, device="cuda")
        gd.q1_q8_gemv(*self.planes[1], o["a2"], o["y"], K, K, n)
        o["h2"] = torch.empty_like(x)
        o["planes"] = torch.empty(n, 8 * (K // 32), dtype=torch.int32, device="cuda")
        o["scale"] = torch.empty(n, device="cuda")
        gd.rmsnorm_ternary_act(o["y"], o["h"], self.g2, o["h2"], o["planes"], o["scale"], n, K, EPS)
        return o


def q8_bytes(codes, scale):
    n, k = codes.shape
    d = scale.astype(np.float16).reshape(n, k // 32, 1).view(np.uint8).reshape(n, k // 32, 2)
    return np.concatenate([d, codes.view(np.uint8).reshape(n, k // 32, 32)], -1).reshape(-1)


def test_prompt_decode_and_draft(gd):
    """Two sequences: prompt chunks of 20 and 7 tokens, three single tokens, then a drafted tree of 4 beside one token; the
    dequantized cache is compared along the way."""
    cap, max_q = 64, 20
    m = Layer(gd, 2, cap)
    rng = np.random.default_rng(9)
    keys = [np.zeros((HKV, 0, D)) for _ in range(2)], [np.zeros((HKV, 0, D)) for _ in range(2)]
    lens = [0, 0]
    tree4 = [0b1, 0b11, 0b101, 0b1011]       # token 3 below 1, tokens 1 and 2 below 0
    table = m.rope.cpu().numpy()
    for qs, words in (([20, 7], None), ([1, 1], None), ([1, 0], None), ([0, 1], None), ([4, 1], tree4 + [1])):
        n = sum(qs)
        seq = np.repeat([0, 1], qs)
        at = np.concatenate([np.arange(lens[b], lens[b] + qs[b]) for b in range(2)]).astype(np.int64)
        depth = at if words is None else np.concatenate(
            [[lens[0] + bin(w).count("1") - 1 for w in words[:4]], at[4:]])
        for b in range(2):
            lens[b] += qs[b]
        start = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
        x, res = (rng.standard_normal((n, K)).astype(np.float32) for _ in range(2))
        o = m.step(dev(x), dev(res), dev(seq), dev(at), dev(depth.astype(np.int32)), dev(np.array(lens, np.int32)), dev(start),
                   None if words is None else dev(np.array(words, np.int64)), max_q, cap)
        g = {k: v.cpu().numpy() for k, v in o.items()}
        # norm and projection, bit for bit
        h = x + res
        assert np.array_equal(g["h"], h)
        codes, s = layer.rmsnorm_codes(h, m.g1.cpu().numpy(), EPS, 32)
        assert np.array_equal(g["a"], q8_bytes(codes, s))
        want = oracle.q1_q8_gemv_aos(m.w_qkv, g["a"].reshape(n, -1), ROWS, K, n)
        assert np.array_equal(g["qkv"].reshape(n, ROWS).view(np.uint32), np.asarray(want).reshape(n, ROWS).view(np.uint32))
        # rotation, bit for bit, and what the cache now holds
        q, k, v = g["qkv"][:, :H], g["qkv"][:, H:H + HKV], g["qkv"][:, H + HKV:]
        assert np.array_equal(g["q"], layer.rotate(q, table, depth, False, fused=True))
        for store, rows in zip(keys, (layer.rotate(k, table, depth, False), v)):
            c, d = layer.q8_rows(rows)
            val = c * np.repeat(d.astype(np.float64), 32, -1)
            for b in range(2):
                store[b] = np.concatenate([store[b], val[seq == b].transpose(1, 0, 2)], axis=1)
        back = [torch.empty(sum(lens), HKV, D, device="cuda") for _ in range(2)]
        all_seq = np.repeat([0, 1], lens)
        all_at = np.concatenate([np.arange(t) for t in lens])
        gd.kv_q8_load(m.cache, m.slots(dev(all_seq), dev(all_at)), back[0], back[1], sum(lens))
        for got, store in zip(back, keys):
            val = np.concatenate([store[b].transpose(1, 0, 2) for b in range(2)]).astype(np.float32)
            assert np.array_equal(got.cpu().numpy(), val)
        # attention: its own bar
        for b in range(2):
            sees = np.zeros((qs[b], lens[b]), bool)
            for t in range(qs[b]):
                w = (1 << (t + 1)) - 1 if words is None else words[start[b] + t]
                sees[t, :lens[b] - qs[b]] = True
                for i in range(qs[b]):
                    sees[t, lens[b] - qs[b] + i] = w >> i & 1
            want, vmax, smax = layer.attention_rows(g["q"][start[b]:start[b + 1]], keys[0][b], keys[1][b], sees, D ** -0.5)
            err = np.abs(g["attn"][start[b]:start[b + 1]] - want)
            assert err.max(initial=0) <= 1e-5 * vmax + 2.0 ** -19 * smax * vmax
        # output projection and the residual norm, bit for bit
        assert np.array_equal(g["a2"], oracle.quantize_q8_0(g["attn"].reshape(n, K)))
        want = np.asarray(oracle.q1_q8_gemv_aos(m.w_o, g["a2"].reshape(n, -1), K, K, n)).reshape(n, K)
        assert np.array_equal(g["y"].view(np.uint32), want.view(np.uint32))
        assert np.array_equal(g["h2"], g["y"] + g["h"])
        codes, s = layer.rmsnorm_codes(g["h2"], m.g2.cpu().numpy(), EPS, K)
        assert np.array_equal(g["scale"], s[:, 0])
        # the planes feed the ternary GEMV: its exact dot is that of the codes
        P, N, w_scale = m.tern[0], m.tern[1], float(m.tern[2])
        y, dot = torch.empty(96, device="cuda"), torch.empty(96, dtype=torch.int32, device="cuda")
        for t in range(n):
            problems = gd.make_ternary_problems([(dev(P.view(np.int32)), dev(N.view(np.int32)), o["planes"][t], y, dot, w_scale,
                                                  o["scale"][t:t + 1])])
            gd.ternary_gemv_grouped(problems, 1, 96, K)
            assert np.array_equal(dot.cpu().numpy(), oracle.ternary_dot_direct(P, N, codes[t]))


def test_captured_decode_steps(gd):
    """A decode step of three sequences captured once and replayed, positions and lengths moving on the device, equals the eager
    loop on a cache of its own, step by step."""
    seqs, cap = 3, 48
    a, b = Layer(gd, seqs, cap), Layer(gd, seqs, cap)
    rng = np.random.default_rng(5)
    x, res = (torch.empty(seqs, K, device="cuda") for _ in range(2))
    seq, start = dev(np.arange(seqs)), dev(np.arange(seqs + 1, dtype=np.int32))
    at = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    pos, lens = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.ones(seqs, dtype=torch.int32, device="cuda")
    data = [dev(rng.standard_normal((seqs, K)).astype(np.float32)) for _ in range(2 * 40)]

    def run(m):
        return m.step(x, res, seq, at, pos, lens, start, None, 1, cap)

    x.copy_(data[0])
    res.copy_(data[1])
    run(a)                       # once before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(a)
    for i in range(40):
        x.copy_(data[2 * i])
        res.copy_(data[2 * i + 1])
        graph.replay()
        torch.cuda.synchronize()
        want = run(b)
        for k in want:
            assert torch.equal(out[k], want[k]), (i, k)
        at.add_(1)
        pos.add_(1)
        lens.add_(1)
