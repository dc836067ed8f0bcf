"""What is measured of the operators around a decode layer's products: the norm with an 8-bit output, rotary positions with
the write of the 8-bit cache, the cache read back, and attention over that cache for one token or a tree of drafted tokens
of each of several sequences.

`own` picks who computes: the plain torch forms below, or the library's entry points on the same inputs. What is held in 8
bits is returned as the values it stands for, through the library's own readers (`q8_0_dequantize`,
`ternary_dequantize_act`, `kv_q8_load`), which are part of the timed call."""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 2.0 ** -17   # about 1e-5, and the same number in 32 and in 64 bits


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before the projections of one decode token (hidden size 4096, the 8B-class shape)
        {"name": "norm q8_0, one token", "op": "norm", "form": "q8_0", "n": 1, "K": 4096, "type": "f32"},
        # a ragged batch of decode tokens before the ternary projections (hidden size 2560)
        {"name": "norm ternary, 37 tokens", "op": "norm", "form": "ternary", "n": 37, "K": 2560, "type": "f32"},
        # a prefill chunk, residual stream in bf16
        {"name": "norm q8_0, prefill", "op": "norm", "form": "q8_0", "n": 4099, "K": 4096, "type": "bf16"},
        # one decode token: rotate q and k, append to the cache
        {"name": "store, one token", "op": "store", "n": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 64, "pos": 32768, "skip": 0, "type": "f32"},
        # a padded batch of decode tokens of a model that rotates half of each head, pairs interleaved
        {"name": "store, padded batch", "op": "store", "n": 61, "heads": 16, "kv_heads": 16, "dim": 64, "rot": 32,
         "interleaved": True, "page": 16, "pos": 131072, "skip": 5, "type": "f16"},
        # a prefill chunk of 8 thousand tokens
        {"name": "store, prefill", "op": "store", "n": 8191, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 64, "pos": 32768, "skip": 0, "type": "bf16"},
        # a short shared prefix read back for a prefill's own attention
        {"name": "load, short prefix", "op": "load", "n": 211, "kv_heads": 8, "dim": 128, "page": 16, "type": "bf16"},
        # a long prefix read back in full precision
        {"name": "load, long prefix", "op": "load", "n": 65521, "kv_heads": 8, "dim": 128, "page": 64, "type": "f32"},
        # three young sequences, a prompt's last and first tokens: where latency counts
        {"name": "attention, short", "op": "attn", "seqs": 3, "q": 1, "heads": 8, "kv_heads": 2, "dim": 64, "len": 300,
         "page": 16, "tree": False, "cap": 0.0, "type": "f32"},
        # the single decode token of the 8B-class shape at 4096 positions
        {"name": "attention, one sequence", "op": "attn", "seqs": 1, "q": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "len": 4096, "page": 64, "tree": False, "cap": 0.0, "type": "f32"},
        # trees of up to 13 drafted tokens for five sequences, capped scores
        {"name": "attention, drafted trees", "op": "attn", "seqs": 5, "q": 13, "heads": 32, "kv_heads": 8, "dim": 128,
         "len": 5003, "page": 32, "tree": True, "cap": 50.0, "type": "bf16"},
        # a serving batch of 32 long sequences
        {"name": "attention, long batch", "op": "attn", "seqs": 32, "q": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "len": 32768, "page": 64, "tree": False, "cap": 0.0, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "store", "load", "attn"])
    t = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        K = 32 * _log(rng, 8, 450)
        return {"op": op, "form": rng.choice(["q8_0", "ternary"]), "n": _log(rng, 1, max(1, 2 ** 24 // K)), "K": K, "type": t}
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([16, 32, 48, 64, 256])
    if op == "load":
        return {"op": op, "n": _log(rng, 1, 2 ** 26 // (kv * dim)), "kv_heads": kv, "dim": dim, "page": page, "type": t}
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    if op == "store":
        n = _log(rng, 1, 2 ** 25 // (heads * dim))
        return {"op": op, "n": n, "heads": heads, "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 16]), "interleaved": rng.random() < 0.5, "page": page,
                "pos": rng.choice([4096, 32768, 131072]), "skip": rng.randint(0, n // 4), "type": t}
    seqs = _log(rng, 1, 48)
    q = rng.choice([1, 1, 1, _log(rng, 2, 64)])
    top = max(64, min(32768, 2 ** 28 // (seqs * kv * dim), 2 ** 31 // (seqs * q * heads * dim)))
    return {"op": op, "seqs": seqs, "q": q, "heads": heads, "kv_heads": kv, "dim": dim, "len": _log(rng, 1, top) + q,
            "page": page, "tree": q > 1 and rng.random() < 0.7, "cap": rng.choice([0.0, 0.0, 30.0]), "type": t}


def _lens(c):
    """(total lengths, query tokens) of a case's sequences: the first is the longest, the others spread below it."""
    rng = random.Random(c["seqs"] * 1000003 + c["len"] * 101 + c["q"])
    qs = [c["q"]] + [rng.randint(1, c["q"]) for _ in range(c["seqs"] - 1)]
    lens = [c["len"]] + [rng.randint(max(n, c["len"] // 2), c["len"]) for n in qs[1:]]
    return lens, qs


def work(c):
    b = SIZE[c["type"]]
    if c["op"] == "norm":
        e = c["n"] * c["K"]
        code = e * 34 // 32 if c["form"] == "q8_0" else e + 4 * c["n"]
        return {"bytes": 3 * b * e + 4 * c["K"] + code + 4 * e, "flops": 12 * e}
    row = c["dim"] + c["dim"] // 16   # codes and scales of one position of one head
    if c["op"] == "load":
        e = 2 * c["n"] * c["kv_heads"]
        return {"bytes": e * (row + c["dim"] * b) + 8 * c["n"], "flops": e * c["dim"]}
    if c["op"] == "store":
        q, kv = c["n"] * c["heads"] * c["dim"], 2 * c["n"] * c["kv_heads"]
        return {"bytes": 2 * q * b + kv * (c["dim"] * b * 2 + row) + c["n"] * (4 * c["rot"] + 12),
                "flops": 3 * (q + kv * c["dim"])}
    lens, qs = _lens(c)
    return {"bytes": 2 * sum(lens) * c["kv_heads"] * row + 2 * sum(qs) * c["heads"] * c["dim"] * b,
            "flops": sum(4 * t * n * c["heads"] * c["dim"] for t, n in zip(qs, lens))}


# ----------------------------------------------------------------- inputs

def _pool(pages, c, g, dev):
    """A cache pool as a server holds it: codes that fill their range, scales of values near one."""
    codes, scales = [], []
    for _ in range(2):
        x = torch.empty((pages, c["kv_heads"], c["page"], c["dim"]), dtype=torch.int8, device=dev)
        x.random_(-127, 128, generator=g)
        codes.append(x)
        d = torch.rand((pages, c["kv_heads"], c["page"], c["dim"] // 32), generator=g, device=dev)
        scales.append(((0.5 + d) * 0.014).to(torch.float16))
    return {"k_codes": codes[0], "k_scales": scales[0], "v_codes": codes[1], "v_scales": scales[1]}


def _cache(s):
    """The handle that a program keeps with its pool (it checks the four planes once and holds no data)."""
    if own:
        import gemm_decode_amd as gd
        s["cache"] = gd.KVCacheQ8(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return s


def _slots(n, pages, page, g, dev):
    """Places of n consecutive tokens in a pool whose pages were handed out in a random order."""
    order = torch.randperm(pages, generator=g, device=dev)
    t = torch.arange(n, device=dev)
    return order[t // page] * page + t % page


def prepare(case, seed):
    dev = "cuda"
    c, T = case, TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] == "norm":
        n, K = c["n"], c["K"]
        loud = torch.where(torch.rand(K, generator=g, device=dev) < 0.01, 20.0, 1.0)   # a few loud channels
        s = {"c": c, "x": randn(n, K).to(T), "residual": (randn(n, K) * 2 * loud).to(T),
             "weight": 1 + 0.2 * randn(K), "h": torch.empty((n, K), dtype=T, device=dev),
             "y": torch.empty((n, K), device=dev)}
        if c["form"] == "q8_0":
            s["a_q8"] = torch.empty(n * (K // 32) * 34, dtype=torch.uint8, device=dev)
        else:
            s["planes"] = torch.empty(n * 8 * (K // 32), dtype=torch.int32, device=dev)
            s["x_scale"] = torch.empty(n, device=dev)
        return s
    if c["op"] == "load":
        pages = -(-c["n"] // c["page"]) + 3
        s = _cache({"c": c, **_pool(pages, c, g, dev)})
        s["slots"] = _slots(c["n"], pages, c["page"], g, dev)
        s["k"] = torch.empty((c["n"], c["kv_heads"], c["dim"]), dtype=T, device=dev)
        s["v"] = torch.empty_like(s["k"])
        return s
    if c["op"] == "store":
        n, D = c["n"], c["dim"]
        pages = -(-n // c["page"]) + 3
        s = _cache({"c": c, **_pool(pages, c, g, dev)})
        # q, k and v are parts of one row, as the fused projection leaves them
        rows = randn(n, c["heads"] + 2 * c["kv_heads"], D).to(T)
        s["q"], s["k"], s["v"] = rows.split([c["heads"], c["kv_heads"], c["kv_heads"]], dim=1)
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = torch.arange(c["pos"], dtype=torch.float64, device=dev)[:, None] * freq
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()
        first = int(torch.randint(0, max(1, c["pos"] - n), (1,), generator=g, device=dev))
        s["positions"] = ((first + torch.arange(n, device=dev)) % c["pos"]).int()
        s["slots"] = _slots(n, pages, c["page"], g, dev)
        if c["skip"]:
            s["slots"][n - c["skip"]:] = -1   # the padding of the batch is not stored
        s["q_out"] = torch.empty((n, c["heads"], D), dtype=T, device=dev)
        s["k_back"] = torch.empty((n, c["kv_heads"], D), dtype=torch.float32, device=dev)
        s["v_back"] = torch.empty_like(s["k_back"])
        return s
    lens, qs = _lens(c)
    per = -(-c["len"] // c["page"])
    pages = sum(-(-n // c["page"]) for n in lens) + 2
    s = _cache({"c": c, **_pool(pages, c, g, dev)})
    order = torch.randperm(pages, generator=g, device=dev).int()
    need = torch.tensor([-(-n // c["page"]) for n in lens], device=dev)
    at = (torch.cumsum(need, 0) - need)[:, None] + torch.minimum(torch.arange(per, device=dev), need[:, None] - 1)
    s["page_table"] = order[at].contiguous()
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["q_start"] = torch.tensor([sum(qs[:i]) for i in range(len(qs) + 1)], dtype=torch.int32, device=dev)
    total = sum(qs)
    s["q"] = (randn(total, c["heads"], c["dim"]) * 1.5).to(T)
    s["out"] = torch.empty_like(s["q"])
    s["tree_mask"] = None
    if c["tree"]:
        rng, words = random.Random(seed), []
        for t in qs:   # each drafted token hangs below an earlier one, and sees what that one sees and itself
            seen = []
            for i in range(t):
                w = (seen[rng.randrange(max(0, i - 4), i)] if i else 0) | 1 << i
                seen.append(w)
            words += [w - (1 << 64) if w >> 63 else w for w in seen]
        s["tree_mask"] = torch.tensor(words, dtype=torch.int64, device=dev)
    return s


# -------------------------------------------------------------- plain forms

def _codes(p, a):
    """8-bit codes of p for the largest magnitudes a: p * (127 / a) to the nearest whole number, halves upwards (in 64 bits:
    a value next to a half must not change sides)."""
    v = p.double() * torch.where(a > 0, 127 / a.double(), 0.0)
    f = v.floor()
    return (f + (v - f >= 0.5)).clamp(-127, 127)


def _plain_norm(s):
    c = s["c"]
    n, K = c["n"], c["K"]
    h = (s["x"].float() + s["residual"].float()).to(TYPES[c["type"]])
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


def _rotate(x, s):
    """x [n, heads, D] turned by its tokens' angles, in 64 bits."""
    c = s["c"]
    rot = c["rot"]
    cs = s["rope"].double()[s["positions"].long()][:, None]   # [n, 1, rot / 2, 2]
    co, si = cs[..., 0], cs[..., 1]
    x = x.double()
    t = x[..., :rot]
    x1, x2 = (t[..., 0::2], t[..., 1::2]) if c["interleaved"] else (t[..., :rot // 2], t[..., rot // 2:])
    y1, y2 = x1 * co - x2 * si, x2 * co + x1 * si
    y = torch.stack([y1, y2], -1).flatten(-2) if c["interleaved"] else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _write(x, codes, scales, page, at):
    x = x[:page.shape[0]]
    n, h, D = x.shape
    b = x.reshape(n, h, D // 32, 32)
    a = b.abs().amax(-1, keepdim=True)
    q = _codes(b, a).to(torch.int8).view(n, h, D)
    d = (a.double() / 127).float().half().squeeze(-1)
    codes[page, :, at] = q
    scales[page, :, at] = d


def _read(codes, scales, page, at, live, T):
    q, d = codes[page, :, at].float(), scales[page, :, at].float()
    x = q * d.repeat_interleave(32, -1)
    return (x * live[:, None, None]).to(T)


def _plain_store(s):
    c = s["c"]
    live = s["slots"] >= 0
    stored = s["slots"][:c["n"] - c["skip"]]   # the batch's padding is behind its tokens
    page, at = stored // c["page"], stored % c["page"]
    q = _rotate(s["q"], s).to(TYPES[c["type"]])
    _write(_rotate(s["k"], s).float(), s["k_codes"], s["k_scales"], page, at)
    _write(s["v"].float(), s["v_codes"], s["v_scales"], page, at)
    page, at = s["slots"].clamp(min=0) // c["page"], s["slots"].clamp(min=0) % c["page"]
    return {"q": q, "k": _read(s["k_codes"], s["k_scales"], page, at, live, torch.float32),
            "v": _read(s["v_codes"], s["v_scales"], page, at, live, torch.float32)}


def _plain_load(s):
    c = s["c"]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    live, T = s["slots"] >= 0, TYPES[c["type"]]
    return {"k": _read(s["k_codes"], s["k_scales"], page, at, live, T),
            "v": _read(s["v_codes"], s["v_scales"], page, at, live, T)}


def _rows(codes, scales, table):
    """[sequences, heads, positions, D] of the pages of a table, in 32 bits."""
    x = codes[table.long()].float().unflatten(-1, (-1, 32)) * scales[table.long()].float()[..., None]
    x = x.flatten(-2).permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _plain_attn(s):
    c = s["c"]
    B, T, Hq, Hkv, D = c["seqs"], c["q"], c["heads"], c["kv_heads"], c["dim"]
    G = Hq // Hkv
    start, total = s["q_start"].long(), s["q"].shape[0]
    count = start[1:] - start[:-1]
    t = torch.arange(T, device=start.device)
    row = (start[:-1, None] + t).clamp(max=total - 1)   # rows past a sequence's own are computed and not used
    q = s["q"].float()[row].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    k = _rows(s["k_codes"], s["k_scales"], s["page_table"])
    sc = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    del k
    if c["cap"]:
        sc = c["cap"] * torch.tanh(sc / c["cap"])
    lens = s["kv_lens"].long()
    ctx = lens - count
    j = torch.arange(sc.shape[-1], device=start.device)
    i = j - ctx[:, None]   # place of a key among the drafted ones
    words = s["tree_mask"][row] if c["tree"] else None
    if words is None:
        own_keys = i[:, None] <= t[:, None]
    else:
        own_keys = (words[:, :, None] >> i.clamp(0, 63)[:, None] & 1) == 1
    sees = ((i < 0)[:, None] | own_keys) & (j < lens[:, None])[:, None]
    sees = sees[:, None, :, None].expand(B, 1, T, G, -1).reshape(B, 1, T * G, -1)
    sc = sc.masked_fill(~sees, float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _rows(s["v_codes"], s["v_scales"], s["page_table"])) / den
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    r = torch.arange(total, device=start.device)
    b = torch.searchsorted(start, r, right=True) - 1
    return {"out": o[b, r - start[b]].to(TYPES[c["type"]])}


# -------------------------------------------------------- the library's calls

def _own_norm(s):
    import gemm_decode_amd as gd
    n, K = s["c"]["n"], s["c"]["K"]
    if s["c"]["form"] == "q8_0":
        gd.rmsnorm_q8_0(s["x"], s["residual"], s["weight"], s["h"], s["a_q8"], n, K, EPS)
        gd.q8_0_dequantize(s["a_q8"], s["y"], n, K)
    else:
        gd.rmsnorm_ternary_act(s["x"], s["residual"], s["weight"], s["h"], s["planes"], s["x_scale"], n, K, EPS)
        gd.ternary_dequantize_act(s["planes"], s["x_scale"], s["y"], n, K)
    return {"h": s["h"], "y": s["y"]}


def _own_store(s):
    import gemm_decode_amd as gd
    c = s["c"]
    gd.kv_q8_store(s["cache"], s["k"], s["v"], s["slots"], c["n"], q=s["q"], q_out=s["q_out"], n_heads=c["heads"],
                   rope=s["rope"], positions=s["positions"], interleaved=c["interleaved"])
    gd.kv_q8_load(s["cache"], s["slots"], s["k_back"], s["v_back"], c["n"])
    return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}


def _own_load(s):
    import gemm_decode_amd as gd
    gd.kv_q8_load(s["cache"], s["slots"], s["k"], s["v"], s["c"]["n"])
    return {"k": s["k"], "v": s["v"]}


def _own_attn(s):
    import gemm_decode_amd as gd
    c = s["c"]
    gd.attn_decode_q8(s["q"], s["cache"], s["page_table"], s["kv_lens"], s["q_start"], s["tree_mask"], s["out"],
                      c["heads"], c["q"], c["len"], 1 / math.sqrt(c["dim"]), softcap=c["cap"])
    return {"out": s["out"]}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"norm": _own_norm, "store": _own_store, "load": _own_load, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "store": _plain_store, "load": _plain_load, "attn": _plain_attn}[op](state)


# -------------------------------------------------- from the definitions, in 64 bits

def _exact_q8(x):
    """The values that 8-bit codes of x stand for, 32 to a group: the scale is the largest magnitude over 127 in 32 bits and
    then in 16, a code the nearest whole number (halves upwards) of x times 127 over that magnitude."""
    g = x.reshape(-1, 32)
    top = g.abs().max(dim=1).values
    code = torch.zeros_like(g)
    some = top > 0
    v = g[some] * (127.0 / top[some])[:, None]
    code[some] = torch.where(v - torch.floor(v) >= 0.5, torch.floor(v) + 1, torch.floor(v)).clamp(-127, 127)
    return code, top


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = (s["x"].float() + s["residual"].float()).to(TYPES[c["type"]]).double()
        inv = (h.pow(2).sum(1) / c["K"] + EPS).sqrt().reciprocal()
        p = h * s["weight"].double()[None]
        if c["form"] == "q8_0":
            code, top = _exact_q8(p)
            d = (top * inv.repeat_interleave(c["K"] // 32) / 127.0).float().half().double()
            return {"h": h, "y": (code * d[:, None]).view(c["n"], c["K"])}
        top = p.abs().max(dim=1).values
        v = p * (127.0 / top)[:, None]
        code = torch.where(v - torch.floor(v) >= 0.5, torch.floor(v) + 1, torch.floor(v)).clamp(-127, 127)
        return {"h": h, "y": code * (top * inv / 127.0).float().double()[:, None]}
    if c["op"] == "load":
        out = {}
        for name in ("k", "v"):
            x = s[name + "_codes"].double().view(-1, 32) * s[name + "_scales"].double().view(-1, 1)
            x = x.view(-1, c["kv_heads"], c["page"], c["dim"]).transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])
            out[name] = x[s["slots"]]
        return out
    if c["op"] == "store":
        half = c["rot"] // 2
        if c["interleaved"]:
            first = 2 * torch.arange(half, device="cuda")
            second = first + 1
        else:
            first = torch.arange(half, device="cuda")
            second = first + half
        table = s["rope"][s["positions"].long()].double()

        def turned(x):
            y = x.double().clone()
            z = torch.view_as_complex(torch.stack([y[..., first], y[..., second]], -1))
            z = z * torch.view_as_complex(table)[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        out = {"q": turned(s["q"])}
        for name, x in (("k", turned(s["k"]).float().double()), ("v", s["v"].double())):
            code, top = _exact_q8(x)
            d = (top / 127.0).float().half().double()
            out[name] = (code * d[:, None]).view(x.shape)
            out[name][s["slots"] < 0] = 0
        return out
    lens, qs = _lens(c)
    G, D, rows, outs = c["heads"] // c["kv_heads"], c["dim"], 0, []
    for b in range(c["seqs"]):
        pages = s["page_table"][b, :-(-lens[b] // c["page"])].long()

        def cached(name):
            x = s[name + "_codes"][pages].double().unflatten(-1, (D // 32, 32)) * s[name + "_scales"][pages].double()[..., None]
            return x.flatten(-2).transpose(0, 1).reshape(c["kv_heads"], -1, D)[:, :lens[b]]

        k, v, before = cached("k"), cached("v"), lens[b] - qs[b]
        for t in range(qs[b]):
            word = (1 << (t + 1)) - 1 if s["tree_mask"] is None else int(s["tree_mask"][rows])
            see = torch.ones(lens[b], dtype=torch.bool, device="cuda")
            see[before:] = torch.tensor([bool(word >> i & 1) for i in range(qs[b])], device="cuda")
            q = s["q"][rows].double().view(c["kv_heads"], G, D)
            z = torch.matmul(k, q.transpose(1, 2).contiguous()) / math.sqrt(D)   # [heads, keys, G]
            if c["cap"]:
                z = torch.tanh(z / c["cap"]) * c["cap"]
            z = torch.softmax(z.masked_fill(~see[None, :, None], float("-inf")), dim=1)
            outs.append(torch.matmul(z.transpose(1, 2).contiguous(), v).reshape(c["heads"], D))
            rows += 1
    return {"out": torch.stack(outs)}
