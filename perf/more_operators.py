"""What is measured of the operators that finish a decode layer and a decode step: the Q1_0 . q8_0 product with bias,
activation and residual in its epilogue, the gated feed-forward block's two products in one, the norms behind and before a
block with its gate and residual scale, and the log probabilities of given tokens with entropy and top alternatives.

`own` picks who computes: the plain torch forms below, or the library's entry points on the same inputs. What is held in 8
bits is returned as the values it stands for, through the library's own readers (`q8_0_dequantize`,
`ternary_dequantize_act`), which are part of the timed call. A product's 8-bit output is read in bf16, as the next block's
stream holds it: its codes are those of a sum in 32 bits, where one that falls on the border of two codes may take either."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 2.0 ** -17   # about 1e-5, and the same number in 32 and in 64 bits
ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]   # in the order of the library's ACT_ codes


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the attention's output projection of one decode token, added to the residual stream
        {"name": "linear, one token", "op": "linear", "n": 1, "rows": 4096, "K": 4096, "act": "none", "bias": False,
         "residual": True, "form": "y", "type": "f32"},
        # the feed-forward's down projection of a ragged decode batch, with a bias
        {"name": "linear, batch of 13", "op": "linear", "n": 13, "rows": 4096, "K": 14336, "act": "none", "bias": True,
         "residual": True, "form": "y", "type": "bf16"},
        # the down projection of a whole prompt
        {"name": "linear, prompt", "op": "linear", "n": 2039, "rows": 4096, "K": 14336, "act": "none", "bias": False,
         "residual": True, "form": "y", "type": "bf16"},
        # gate and up projection of one decode token, written as the down projection reads it
        {"name": "gated, one token", "op": "gated", "n": 1, "rows": 14336, "K": 4096, "act": "silu", "bias": False,
         "form": "q8_0", "type": "bf16"},
        # the squared-ReLU block of the smaller shape, a batch of drafted tokens
        {"name": "gated, 37 tokens", "op": "gated", "n": 37, "rows": 6912, "K": 2560, "act": "relu2", "bias": False,
         "form": "y", "type": "f16"},
        # gate and up projection of a prompt
        {"name": "gated, prompt", "op": "gated", "n": 509, "rows": 14336, "K": 4096, "act": "silu", "bias": False,
         "form": "q8_0", "type": "bf16"},
        # behind the attention and before the feed-forward block of one decode token
        {"name": "norms q8_0, one token", "op": "norms", "form": "q8_0", "n": 1, "K": 4096, "post": True, "gates": 0,
         "type": "f32"},
        # a ragged batch with a scale for each channel, written for the ternary products
        {"name": "norms ternary, 61 tokens", "op": "norms", "form": "ternary", "n": 61, "K": 2560, "post": True,
         "gates": 1, "type": "f16"},
        # a prompt chunk of several sequences, each with gates of its own
        {"name": "norms q8_0, prompt", "op": "norms", "form": "q8_0", "n": 4099, "K": 4096, "post": True, "gates": 7,
         "type": "bf16"},
        # the answer's token with its alternatives
        {"name": "logprobs, one token", "op": "logprobs", "n": 1, "V": 49152, "given": 1, "k": 8, "cap": 0.0, "scale": 1.0,
         "banned": 0.0, "type": "f32"},
        # a serving batch under a grammar that bans half of the tokens, temperature 0.8
        {"name": "logprobs, 61 tokens", "op": "logprobs", "n": 61, "V": 50021, "given": 1, "k": 20, "cap": 0.0,
         "scale": 1.25, "banned": 0.5, "type": "f16"},
        # the log probabilities of a prompt's own tokens
        {"name": "logprobs, prompt", "op": "logprobs", "n": 2039, "V": 100003, "given": 1, "k": 5, "cap": 30.0, "scale": 1.0,
         "banned": 0.0, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["linear", "gated", "norms", "logprobs"])
    t = rng.choice(["f32", "bf16", "f16"])
    if op == "norms":
        K = 32 * _log(rng, 8, 450)
        n = _log(rng, 1, max(1, 2 ** 24 // K))
        return {"op": op, "form": rng.choice(["q8_0", "ternary"]), "n": n, "K": K, "post": rng.random() < 0.8,
                "gates": rng.choice([0, 1, min(n, 5), n]), "type": t}
    if op == "logprobs":
        V = _log(rng, 1000, 160000)
        return {"op": op, "n": _log(rng, 1, 2 ** 26 // V), "V": V, "given": rng.choice([1, 1, 3]),
                "k": rng.choice([0, 1, 5, 20, 64]), "cap": rng.choice([0.0, 0.0, 30.0]), "scale": rng.choice([1.0, 1.25, 0.7]),
                "banned": rng.choice([0.0, 0.0, 0.5]), "type": t}
    K = 128 * _log(rng, 2, 112)
    form = rng.choice(["y", "q8_0"])
    rows = 32 * _log(rng, 2, 448) if form == "q8_0" else _log(rng, 33, 14336)
    n = rng.choice([1, _log(rng, 1, min(2048, 2 ** 36 // (rows * K)))])
    c = {"op": op, "n": n, "rows": rows, "K": K, "act": rng.choice(ACTS if op == "linear" else ACTS[1:]),
         "bias": rng.random() < 0.5}
    if op == "linear":
        c["residual"] = rng.random() < 0.5
    return {**c, "form": form, "type": t}


def work(c):
    b, n = SIZE[c["type"]], c["n"]
    if c["op"] == "norms":
        e, K = n * c["K"], c["K"]
        code = e * 34 // 32 if c["form"] == "q8_0" else e + 4 * n
        read = 2 * b * e + 4 * K + (4 * K if c["post"] else 0) + c["gates"] * K * b
        return {"bytes": read + b * e + code + 4 * e, "flops": 20 * e}
    if c["op"] == "logprobs":
        return {"bytes": n * (c["V"] * b + c["given"] * 12 + 4 + c["k"] * 12), "flops": 6 * n * c["V"]}
    rows, K, sets = c["rows"], c["K"], 2 if c["op"] == "gated" else 1
    read = sets * (rows * K // 128 * 18 + (4 * rows if c["bias"] else 0)) + n * K // 32 * 34
    if c.get("residual"):
        read += n * rows * b
    # an 8-bit output is written as codes and as the values that they stand for
    written = n * rows * b if c["form"] == "y" else n * rows * 34 // 32 + 2 * n * rows
    return {"bytes": read + written, "flops": 2 * sets * n * rows * K}


# ----------------------------------------------------------------- inputs

def _weights(rows, K, g, dev):
    """Q1_0 blocks of a rows x K matrix: 18 bytes for 128 weights, an f16 scale and 128 sign bits."""
    w = torch.empty((rows, K // 128, 18), dtype=torch.uint8, device=dev)
    w.random_(0, 256, generator=g)
    d = torch.rand((rows, K // 128), generator=g, device=dev) * 0.03 + 0.005
    w[:, :, :2] = d.half()[..., None].view(torch.uint8)
    return w


def _acts(n, K, g, dev):
    """q8_0 blocks of n activations, a few channels of them loud: 34 bytes for 32 values, an f16 scale and 32 codes."""
    x = torch.randn((n, K), generator=g, device=dev)
    x *= torch.where(torch.rand(K, generator=g, device=dev) < 0.01, 10.0, 1.0)
    b = x.view(n, K // 32, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    a = torch.empty((n, K // 32, 34), dtype=torch.uint8, device=dev)
    a[:, :, :2] = d.half().view(torch.uint8)
    a[:, :, 2:] = (b / d.clamp(min=1e-20)).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return a


def _planes(w, rows, K):
    """The weights as a program holds them: repacked once when the model is loaded."""
    import gemm_decode_amd as gd
    bits, scales = gd.q1_alloc_planes(rows, K)
    gd.q1_repack(w.reshape(-1), rows, K, bits, scales)
    return bits, scales


def prepare(case, seed):
    dev = "cuda"
    c, T, n = case, TYPES[case["type"]], case["n"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] in ("linear", "gated"):
        rows, K = c["rows"], c["K"]
        s = {"c": c, "a": _acts(n, K, g, dev), "w": [_weights(rows, K, g, dev) for _ in range(2 if c["op"] == "gated" else 1)]}
        s["bias"] = [randn(rows) if c["bias"] else None for _ in s["w"]]
        s["residual"] = randn(n, rows).to(T) if c.get("residual") else None
        s["a_q8"] = s["a"].view(-1)
        # where the product goes: the stream's type, or 8 bits and the values read from them
        s["y"] = torch.empty((n, rows), dtype=T if c["form"] == "y" else torch.bfloat16, device=dev)
        s["y_q8"] = None if c["form"] == "y" else torch.empty(n * (rows // 32) * 34, dtype=torch.uint8, device=dev)
        if own:
            s["planes"] = [_planes(w, rows, K) for w in s["w"]]
        return s
    if c["op"] == "norms":
        K = c["K"]
        loud = torch.where(torch.rand(K, generator=g, device=dev) < 0.01, 20.0, 1.0)   # a few loud channels
        s = {"c": c, "x": (randn(n, K) * 3).to(T), "residual": (randn(n, K) * 2 * loud).to(T),
             "weight": 1 + 0.2 * randn(K), "post": 0.3 + 0.1 * randn(K) if c["post"] else None,
             "gate": (0.5 * randn(c["gates"], K)).to(T) if c["gates"] else None, "gate_index": None,
             "h": torch.empty((n, K), dtype=T, device=dev), "y": torch.empty((n, K), device=dev)}
        if 1 < c["gates"] < n:   # sequences of several tokens, each with its own gates
            s["gate_index"] = (torch.arange(n, device=dev) * c["gates"] // n).int()
        if c["form"] == "q8_0":
            s["a_q8"] = torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device=dev)
        else:
            s["planes"] = torch.empty(n * 8 * (K // 32), dtype=torch.int32, device=dev)
            s["x_scale"] = torch.empty(n, device=dev)
        return s
    V, m, k = c["V"], c["given"], c["k"]
    x = randn(n, V).mul_(2.5)
    sharp = torch.randint(0, V, (n, 4), generator=g, device=dev)   # what the model would say
    x.scatter_add_(1, sharp, 12 * torch.rand((n, 4), generator=g, device=dev))
    if c["banned"]:
        x.masked_fill_(torch.rand((n, V), generator=g, device=dev) < c["banned"], float("-inf"))
        if n > 3:
            x[2] = float("-inf")   # a grammar that has come to a dead end
    s = {"c": c, "logits": x.to(T)}
    tokens = torch.randint(0, V, (n, m), generator=g, device=dev)
    tokens[:, 0] = torch.where(torch.rand(n, generator=g, device=dev) < 0.7, sharp[:, 0], tokens[:, 0])
    if n > 1:
        tokens[-1] = -1   # the batch's padding
    s["tokens"] = tokens
    s["logprobs"], s["entropy"] = torch.empty((n, m), device=dev), torch.empty(n, device=dev)
    s["top_ids"] = torch.empty((n, k), dtype=torch.int64, device=dev) if k else None
    s["top_logprobs"] = torch.empty((n, k), device=dev) if k else None
    return s


# -------------------------------------------------------------- plain forms

def _codes(p, a):
    """8-bit codes of p for the largest magnitudes a: p * (127 / a) to the nearest whole number, halves upwards (in 64 bits:
    a value next to a half must not change sides)."""
    v = p.double() * torch.where(a > 0, 127 / a.double(), 0.0)
    f = v.floor()
    return (f + (v - f >= 0.5)).clamp(-127, 127)


def _dense(w):
    """The values of Q1_0 blocks [rows, K / 128, 18], in 32 bits."""
    rows = w.shape[0]
    d = w[:, :, :2].contiguous().view(torch.float16).float()
    bits = w[:, :, 2:, None] >> torch.arange(8, dtype=torch.uint8, device=w.device) & 1
    return ((bits.float() * 2 - 1).view(rows, -1, 128) * d).view(rows, -1)


def _act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "relu2":
        return x.clamp(min=0).square()
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x / (1 + torch.exp(-x)) if name == "silu" else x


def _plain_product(s):
    c, n = s["c"], s["c"]["n"]
    d = s["a"][:, :, :2].contiguous().view(torch.float16).float()
    a = (s["a"][:, :, 2:].contiguous().view(torch.int8).float() * d).view(n, -1)
    y = torch.matmul(a, _dense(s["w"][0]).t())
    if c["bias"]:
        y = y + s["bias"][0]
    y = _act(y, c["act"])
    if c["op"] == "gated":
        up = torch.matmul(a, _dense(s["w"][1]).t())
        y = y * (up + s["bias"][1] if c["bias"] else up)
    elif c["residual"]:
        y = y + s["residual"].float()
    if c["form"] == "y":
        return {"y": y.to(TYPES[c["type"]])}
    b = y.view(n, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    d = (top.double() / 127).float().half().float()
    return {"y": (_codes(b, top).float() * d).view(n, -1).to(torch.bfloat16)}


def _plain_norms(s):
    c = s["c"]
    n, K = c["n"], c["K"]
    u = s["x"].double()
    if c["post"]:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["post"].double()
    if c["gates"]:
        gate = s["gate"] if s["gate_index"] is None else s["gate"][s["gate_index"].long()]
        u = u * gate.double()
    h = (0.75 * s["residual"].double() + 1.5 * u).float().to(TYPES[c["type"]])
    hd = h.double()
    rstd = torch.rsqrt((hd * hd).mean(-1, keepdim=True) + EPS)
    p = hd * s["weight"].double()
    if c["form"] == "q8_0":
        p = p.view(n, K // 32, 32)
        a = p.abs().amax(-1, keepdim=True)
        d = (a * rstd[:, :, None] / 127).float().half().float()
    else:
        a = p.abs().amax(-1, keepdim=True)
        d = (a * rstd / 127).float()
    return {"h": h, "y": (_codes(p, a).float() * d).view(n, K)}


def _plain_logprobs(s):
    c, x = s["c"], s["logits"].float()
    z = (c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x) * c["scale"]
    z = z.masked_fill(x == float("-inf"), float("-inf"))   # what is banned stays so under a cap
    m = z.amax(-1, keepdim=True)
    some = m > float("-inf")   # rows that have a token left
    d = torch.where(z > float("-inf"), z - m, float("-inf"))
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    lse = torch.log(total)
    mean = (e * d.clamp(min=-200)).sum(-1, keepdim=True, dtype=torch.float64) / total   # exp(-200) is 0 in 32 bits
    entropy = torch.where(some, lse - mean, 0.0).float().squeeze(-1)

    def of(ids):
        return torch.where(ids >= 0, (torch.gather(d, 1, ids.clamp(min=0)) - lse).float(), 0.0)

    out = {"entropy": entropy, "logprobs": torch.where(some | (s["tokens"] < 0), of(s["tokens"]), float("-inf"))}
    if c["k"]:
        # one whole number that orders by value, and by place where values are alike: no two are equal
        i = (x + 0.0).view(torch.int32)
        order = torch.where(i < 0, i ^ 0x7FFFFFFF, i).long() * 2 ** 32 + (2 ** 32 - 1 - torch.arange(c["V"], device=x.device))
        ids = torch.topk(order, min(c["k"], c["V"]), dim=-1).indices
        left = torch.gather(x, 1, ids) > float("-inf")
        out["top_logprobs"] = torch.where(left, of(ids), float("-inf"))
        out["top_ids"] = torch.where(left, ids, -1)
    return out


# -------------------------------------------------------- the library's calls

def _own_product(s):
    import gemm_decode_amd as gd
    c = s["c"]
    n, rows, K = c["n"], c["rows"], c["K"]
    act = ACTS.index(c["act"])
    y = s["y"] if c["form"] == "y" else None
    if c["op"] == "linear":
        gd.q1_q8_linear(*s["planes"][0], s["a_q8"], y, rows, K, n, bias=s["bias"][0], act=act, residual=s["residual"],
                        y_q8=s["y_q8"])
    else:
        gd.q1_q8_gated(*s["planes"][0], *s["planes"][1], s["a_q8"], y, rows, K, n, act=act, gate_bias=s["bias"][0],
                       up_bias=s["bias"][1], y_q8=s["y_q8"])
    if y is None:
        gd.q8_0_dequantize(s["y_q8"], s["y"], n, rows)
    return {"y": s["y"]}


def _own_norms(s):
    import gemm_decode_amd as gd
    n, K = s["c"]["n"], s["c"]["K"]
    more = {"gate": s["gate"], "gate_index": s["gate_index"], "residual_scale": 0.75, "block_scale": 1.5}
    if s["c"]["form"] == "q8_0":
        gd.rmsnorm_sandwich_q8_0(s["x"], s["post"], s["residual"], s["weight"], s["h"], s["a_q8"], n, K, EPS, **more)
        gd.q8_0_dequantize(s["a_q8"], s["y"], n, K)
    else:
        gd.rmsnorm_sandwich_ternary_act(s["x"], s["post"], s["residual"], s["weight"], s["h"], s["planes"], s["x_scale"], n, K,
                                        EPS, **more)
        gd.ternary_dequantize_act(s["planes"], s["x_scale"], s["y"], n, K)
    return {"h": s["h"], "y": s["y"]}


def _own_logprobs(s):
    import gemm_decode_amd as gd
    c = s["c"]
    gd.token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"], c["n"], c["V"],
                      scale=c["scale"], softcap=c["cap"])
    out = {"entropy": s["entropy"], "logprobs": s["logprobs"]}
    return {**out, "top_logprobs": s["top_logprobs"], "top_ids": s["top_ids"]} if c["k"] else out


def run(state):
    op = state["c"]["op"]
    if own:
        return {"linear": _own_product, "gated": _own_product, "norms": _own_norms, "logprobs": _own_logprobs}[op](state)
    return {"linear": _plain_product, "gated": _plain_product, "norms": _plain_norms, "logprobs": _plain_logprobs}[op](state)


# -------------------------------------------------- from the definitions, in 64 bits

def _exact_codes(g):
    """Codes of rows of 64-bit values, the largest magnitude of a row as 127 (halves upwards), and those magnitudes."""
    top = g.abs().max(dim=1).values
    v = g * torch.where(top > 0, 127.0 / top, torch.zeros_like(top))[:, None]
    low = torch.floor(v)
    return torch.where(v - low >= 0.5, low + 1, low).clamp(-127, 127), top


def _exact_product(c, s):
    n, rows, K = c["n"], c["rows"], c["K"]
    signs = torch.tensor([[1.0 if byte >> j & 1 else -1.0 for j in range(8)] for byte in range(256)], dtype=torch.float64,
                         device="cuda")
    blocks = s["a"].view(-1, 34)
    a = blocks[:, 2:].contiguous().view(torch.int8).double()
    a = (a * blocks[:, :2].contiguous().view(torch.float16).double()).view(n, K)
    sums = []
    for w in s["w"]:
        out = torch.empty((n, rows), dtype=torch.float64, device="cuda")
        for r in range(0, rows, 2048):
            part = w[r:r + 2048]
            dense = signs[part[:, :, 2:].reshape(-1).int()].view(-1, 128)
            dense = dense * part[:, :, :2].reshape(-1, 2).view(torch.float16).double()
            out[:, r:r + 2048] = a @ dense.view(part.shape[0], K).t().contiguous()
        sums.append(out)
    if c["bias"]:
        sums = [t + b.double() for t, b in zip(sums, s["bias"])]
    t = sums[0]
    y = {"none": lambda: t, "relu": lambda: torch.relu(t), "relu2": lambda: torch.relu(t).pow(2),
         "gelu": lambda: t * torch.special.ndtr(t),
         "gelu_tanh": lambda: t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t.pow(3))),
         "silu": lambda: t * torch.sigmoid(t)}[c["act"]]()
    if c["op"] == "gated":
        y = y * sums[1]
    elif c["residual"]:
        y = y + s["residual"].double()
    if c["form"] == "y":
        return {"y": y}
    code, top = _exact_codes(y.view(-1, 32))
    return {"y": (code * (top / 127.0).float().half().double()[:, None]).view(n, rows)}


def _exact_norms(c, s):
    def inv(t):
        return (t.pow(2).sum(1, keepdim=True) / c["K"] + EPS).sqrt().reciprocal()

    n, K = c["n"], c["K"]
    block = s["x"].double()
    if c["post"]:
        block = block * (inv(block) * s["post"].double()[None])
    if c["gates"]:
        which = torch.zeros(n, dtype=torch.int64, device="cuda") if c["gates"] == 1 else torch.arange(n, device="cuda")
        block = block * s["gate"].double()[which if s["gate_index"] is None else s["gate_index"].long()]
    h = (block * 1.5 + s["residual"].double() * 0.75).float().to(TYPES[c["type"]]).double()
    p = h * s["weight"].double()[None]
    if c["form"] == "q8_0":
        code, top = _exact_codes(p.view(-1, 32))
        d = (top * inv(h).expand(n, K // 32).reshape(-1) / 127.0).float().half().double()
        return {"h": h, "y": (code * d[:, None]).view(n, K)}
    code, top = _exact_codes(p)
    return {"h": h, "y": code * (top[:, None] * inv(h) / 127.0).float().double()}


def _exact_logprobs(c, s):
    outs = {"entropy": [], "logprobs": [], "top_logprobs": [], "top_ids": []}
    for r in range(0, c["n"], 128):
        x, tokens = s["logits"][r:r + 128].double(), s["tokens"][r:r + 128]
        z = x
        if c["cap"]:
            z = torch.tanh(z / c["cap"]) * c["cap"] + torch.where(torch.isneginf(x), x, 0.0)
        lp = torch.log_softmax(z * c["scale"], dim=1)
        dead = torch.isneginf(x).all(dim=1)
        lp[dead] = float("-inf")
        outs["entropy"].append(torch.special.entr(lp.exp()).sum(1))
        given = torch.gather(lp, 1, tokens.clamp(min=0))
        given[tokens < 0] = 0
        outs["logprobs"].append(given)
        if c["k"]:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]]
            outs["top_logprobs"].append(torch.gather(lp, 1, ids))
            ids[torch.isneginf(torch.gather(x, 1, ids))] = -1
            outs["top_ids"].append(ids)
    return {name: torch.cat(v) for name, v in outs.items() if v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_product, "gated": _exact_product, "norms": _exact_norms, "logprobs": _exact_logprobs}[case["op"]](case, s)
