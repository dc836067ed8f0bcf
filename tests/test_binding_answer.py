"""The binding's own refusals for the products with an epilogue, the norms behind and before a
block and the log probabilities, and the statuses behind them (CPU tensors; no compute is launched here)."""
import pytest

torch = pytest.importorskip("torch")
ROWS, K = 64, 256


@pytest.fixture()
def gd(monkeypatch):
    import gemm_decode_amd
    # a CPU tensor's index: what is checked is the rest (a wrong type may end in the refusal of the device, which comes first)
    monkeypatch.setattr(gemm_decode_amd, "_current", lambda: (-1, 0))
    return gemm_decode_amd


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


def weight(gd):
    return [u8(b) for b in gd.q1_planes_bytes(ROWS, K)]


def test_products(gd):
    w, a, y = weight(gd), u8(2 * K // 32 * 34), torch.zeros(2, ROWS)

    def linear(a=a, y=y, n=2, **kw):
        gd.q1_q8_linear(*kw.pop("w", w), a, y, ROWS, kw.pop("K", K), n, **kw)

    def gated(a=a, y=y, n=2, **kw):
        gd.q1_q8_gated(*kw.pop("w", w), *w, a, y, ROWS, kw.pop("K", K), n, **kw)
    for call in (linear, gated):
        for bad in (dict(a=a[:-1]), dict(y=torch.zeros(ROWS)), dict(w=(w[0][:-1], w[1])), dict(w=(w[0], w[1][1:])),
                    dict(y_q8=u8(2 * ROWS // 32 * 34 - 1))):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in (dict(y=y.double()), dict(a=a.to(torch.int8)), dict(y_q8=torch.zeros(136)), dict(workspace=torch.zeros(4))):
            with pytest.raises((TypeError, ValueError)):
                call(**bad)
        with pytest.raises(gd.GemmDecodeError):
            call(K=192)
        with pytest.raises(gd.GemmDecodeError, match="null pointer"):
            call(y=None)
        with pytest.raises(gd.GemmDecodeError, match="GD_ERANGE"):   # five columns need more
            call(a=u8(5 * K // 32 * 34), y=torch.zeros(5, ROWS), n=5, workspace=u8(4096))
        with pytest.raises(gd.GemmDecodeError, match="activation"):
            call(act=9)
    for bad in (dict(bias=torch.zeros(ROWS + 1)), dict(residual=torch.zeros(ROWS))):
        with pytest.raises(ValueError):
            linear(**bad)
    with pytest.raises((TypeError, ValueError)):
        linear(residual=y.half())
    with pytest.raises(ValueError):
        gated(up_bias=torch.zeros(1))
    with pytest.raises(ValueError):
        linear(y=torch.zeros(ROWS, 2).t())


def test_norms(gd):
    n = 3
    x, res, w = torch.zeros(n, K), torch.zeros(n, K), torch.ones(K)

    def q8(x=x, post=w, res=res, w=w, h=None, out=u8(n * K // 32 * 34), **kw):
        gd.rmsnorm_sandwich_q8_0(x, post, res, w, h, out, n, K, 1e-5, **kw)

    def ternary(x=x, post=w, res=res, w=w, h=None, out=torch.zeros(n * 8 * K // 32, dtype=torch.int32), **kw):
        gd.rmsnorm_sandwich_ternary_act(x, post, res, w, h, out, torch.zeros(n), n, K, 1e-5, **kw)
    for call in (q8, ternary):
        for bad in (dict(x=x[:2]), dict(post=w[1:]), dict(res=res[1:]), dict(w=torch.ones(1)), dict(h=torch.zeros(K)),
                    dict(gate=torch.zeros(K - 1)), dict(gate=torch.zeros(K, n)), dict(gate=torch.zeros(0, K)),
                    dict(gate=x, gate_index=torch.zeros(2, dtype=torch.int32))):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in (dict(res=res.half()), dict(post=w.half()), dict(h=x.bfloat16()), dict(gate=x.half()),
                    dict(gate=x, gate_index=torch.zeros(n, dtype=torch.int64)), dict(x=x.double())):
            with pytest.raises((TypeError, ValueError)):
                call(**bad)
        with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
            call(gate=torch.zeros(2, K))   # two gates for three rows, and no index
        with pytest.raises(gd.GemmDecodeError, match="GD_EINVAL"):
            call(block_scale=float("nan"))


def test_logprobs(gd):
    n, V = 2, 50
    x, t, lp = torch.zeros(n, V), torch.zeros(n, 3, dtype=torch.int64), torch.zeros(n, 3)
    ids, tops, ent = torch.zeros(n, 4, dtype=torch.int64), torch.zeros(n, 4), torch.zeros(n)

    def call(x=x, t=t, lp=lp, ent=ent, ids=ids, tops=tops, n=n, **kw):
        gd.token_logprobs(x, t, lp, ent, ids, tops, n, V, **kw)
    for bad in (dict(x=x[:, :-1]), dict(x=torch.zeros(V, n).t()), dict(x=x[0]), dict(x=x[:1]), dict(t=None), dict(lp=None),
                dict(ids=None), dict(tops=None), dict(t=t[:1], lp=lp[:1]), dict(lp=lp[:, :2]), dict(ids=ids[:, :0], tops=tops[:, :0]),
                dict(ent=ent[:1]), dict(t=t.reshape(-1), lp=lp.reshape(-1))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(t=t.int()), dict(lp=lp.half()), dict(ids=ids.int()), dict(tops=tops.double()), dict(x=x.double()),
                dict(ent=ent.double())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad, name in ((dict(scale=0.0), "GD_EINVAL"), (dict(softcap=-1.0), "GD_EINVAL"), (dict(x=x[:1].expand(n, V)), "GD_EINVAL"),
                      (dict(t=None, lp=None, ent=None, ids=None, tops=None), "GD_EINVAL")):
        with pytest.raises(gd.GemmDecodeError, match=name):
            call(**bad)
    with pytest.raises(gd.GemmDecodeError, match="GD_E"):
        gd.token_logprobs(x, None, None, None, torch.zeros(n, 65, dtype=torch.int64), torch.zeros(n, 65), n, V)
