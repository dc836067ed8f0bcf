"""The operators behind the attention run together, as a decode layer's second half and the end
of a decode step run them: output projection -> norms behind and before the feed-forward block
-> gated products straight into q8_0 -> down projection onto the residual -> last norm ->
vocabulary product -> log probabilities. Each step is compared with its definition on the
inputs it had; then a greedy loop that feeds its own tokens is captured and replayed."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import answer, layer
from test_gpu_logprobs import near
from test_gpu_norm_quant import blocks
from test_gpu_norm_sandwich import check, definition
from test_gpu_q1_linear import dev, planes, within

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
K, FF, V, TOP = 256, 640, 1003, 5
EPS, CAP, BLOCK = 1e-5, 20.0, 0.5
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def gd():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a visible HIP device")
    import gemm_decode_amd
    return gemm_decode_amd


class Half:
    """Weights of the layer's second half and of the model's end."""

    def __init__(self, gd, T):
        self.gd, self.T = gd, T
        rng = np.random.default_rng(1)
        self.w = {name: wl.q1_weights_aos(rows, cols, i) for i, (name, rows, cols) in
                  enumerate((("o", K, K), ("gate", FF, K), ("up", FF, K), ("down", K, FF), ("vocab", V, K)))}
        self.planes = {name: planes(gd, w) for name, w in self.w.items()}
        self.bias = dev((0.1 * rng.standard_normal(K)).astype(np.float32))
        self.post, self.pre, self.last = (dev((1 + 0.1 * rng.standard_normal(K)).astype(np.float32)) for _ in range(3))
        self.gate = dev(rng.standard_normal((2, K)).astype(np.float32)).to(T)
        self.embed = dev(rng.standard_normal((V, K)).astype(np.float32)).to(T)

    def step(self, attn, residual, index, tokens):
        """attn f32 [n, K]; every intermediate is returned."""
        gd, n, T = self.gd, attn.shape[0], self.T
        blocks_of = lambda width: torch.empty(n * (width // 32) * 34, dtype=torch.uint8, device="cuda")
        o = {"a0": blocks_of(K), "o": torch.empty(n, K, dtype=T, device="cuda"), "h": torch.empty(n, K, dtype=T, device="cuda"),
             "a1": blocks_of(K), "f": blocks_of(FF), "d": torch.empty(n, K, dtype=T, device="cuda"), "a2": blocks_of(K),
             "logits": torch.empty(n, V, dtype=T, device="cuda"), "lp": torch.empty(n, 1, device="cuda"),
             "entropy": torch.empty(n, device="cuda"), "ids": torch.empty(n, TOP, dtype=torch.int64, device="cuda"),
             "tops": torch.empty(n, TOP, device="cuda")}
        gd.q8_0_quantize(attn, o["a0"], n, K)
        gd.q1_q8_linear(*self.planes["o"], o["a0"], o["o"], K, K, n, bias=self.bias)
        gd.rmsnorm_sandwich_q8_0(o["o"], self.post, residual, self.pre, o["h"], o["a1"], n, K, EPS, gate=self.gate,
                                 gate_index=index, block_scale=BLOCK)
        gd.q1_q8_gated(*self.planes["gate"], *self.planes["up"], o["a1"], None, FF, K, n, y_q8=o["f"])
        gd.q1_q8_linear(*self.planes["down"], o["f"], o["d"], K, FF, n, residual=o["h"])
        gd.rmsnorm_q8_0(o["d"], None, self.last, None, o["a2"], n, K, EPS)
        gd.q1_q8_linear(*self.planes["vocab"], o["a2"], o["logits"], V, K, n)
        gd.token_logprobs(o["logits"], tokens, o["lp"], o["entropy"], o["ids"], o["tops"], n, V, softcap=CAP)
        return o


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("T", TYPES)
def test_each_step(gd, T, n):
    m = Half(gd, T)
    rng = np.random.default_rng(n)
    attn = rng.standard_normal((n, K)).astype(np.float32)
    res = dev(rng.standard_normal((n, K)).astype(np.float32)).to(T)
    index = dev(rng.integers(-1, 3, n).astype(np.int32))
    tokens = dev(rng.integers(-1, V, (n, 1)))
    o = m.step(dev(attn), res, index, tokens)
    values = {name: answer.q1_values(w) for name, w in m.w.items()}
    codes = lambda name: answer.q8_values(o[name].cpu().numpy(), n)
    f64 = lambda t: t.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(o["a0"].cpu().numpy(), oracle.quantize_q8_0(attn))
    want, off = answer.product(values["o"], codes("a0"), m.bias.cpu().numpy(), 0)
    within(o["o"], want, off, T)
    check("q8_0", (o["a1"],), o["h"], m.pre, T, definition(o["o"], m.post, res, m.gate, index.cpu().numpy(), 1.0, BLOCK))
    # the gated products' blocks are those of the call's own f32 output
    y = torch.empty(n, FF, device="cuda")
    gd.q1_q8_gated(*m.planes["gate"], *m.planes["up"], o["a1"], y, FF, K, n)
    assert np.array_equal(o["f"].cpu().numpy(), oracle.quantize_q8_0(y.cpu().numpy()))
    (g, goff), (u, uoff) = (answer.product(values[w], codes("a1"), None, c) for w, c in (("gate", 5), ("up", 0)))
    bound = np.abs(g) * uoff + np.abs(u) * goff + goff * uoff
    within(y, g * u, bound + 2.0 ** -24 * (np.abs(g * u) + bound), torch.float32)
    want, off = answer.product(values["down"], codes("f"), None, 0)
    total = want + f64(o["h"])
    within(o["d"], total, off + 2.0 ** -24 * (np.abs(total) + off), T)
    c, s = layer.rmsnorm_codes(f64(o["d"]), m.last.cpu().numpy(), EPS, 32)
    assert np.array_equal(o["a2"].cpu().numpy(), blocks(c, s))
    want, off = answer.product(values["vocab"], codes("a2"), None, 0)
    within(o["logits"], want, off, T)
    x, t = o["logits"].float().cpu().numpy(), tokens.cpu().numpy()
    for r in range(n):
        lp, entropy, ids, tops = answer.logprobs(x[r], t[r], TOP, 1.0, CAP)
        assert np.array_equal(o["ids"][r].cpu().numpy(), ids)
        near(o["lp"][r], lp, CAP, 1.0)
        near(o["entropy"][r:r + 1], np.array([entropy]), CAP, 1.0)
        near(o["tops"][r], tops, CAP, 1.0)


@pytest.mark.parametrize("seqs", [1, 6])
def test_captured_greedy_loop(gd, seqs):
    """A step whose most likely tokens are the next step's input, captured once and replayed, equals the eager loop: every
    intermediate of every step, with eager calls of other sizes between the replays."""
    m = Half(gd, torch.bfloat16)
    index = dev((np.arange(seqs) % 3 - 1).astype(np.int32))
    asked = dev(np.arange(seqs)[:, None] * 7)

    def run(now):
        x = m.embed[now]
        return m.step(x.float(), x, index, asked)

    first = dev(np.arange(seqs) * 100 + 3)
    now = first.clone()
    run(now)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(now)
        now.copy_(out["ids"][:, 0])
    now.copy_(first)
    token = first.clone()
    for i in range(24):
        graph.replay()
        m.step(torch.ones(9, K, device="cuda"), m.embed[:9], dev(np.zeros(9, np.int32)), dev(np.zeros((9, 1), np.int64)))
        want = run(token)
        for k in want:
            assert torch.equal(out[k], want[k]), (i, k)
        token = want["ids"][:, 0].clone()
        assert torch.equal(token, now)
