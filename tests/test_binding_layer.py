"""The binding's own refusals for the norm, rotary, 8-bit cache and attention
calls, and the strides it takes (CPU tensors; no compute is launched here)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gd():
    import gemm_decode_amd
    return gemm_decode_amd


def test_binding_refuses_what_is_not_on_a_device(gd, monkeypatch):
    """CPU tensors, other types, other sizes and other devices are refused before the library is called."""
    t = torch.zeros(2, 64)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        gd.rmsnorm_q8_0(t, None, torch.ones(64), None, torch.zeros(136, dtype=torch.uint8), 2, 64, 1e-5)
    with pytest.raises(TypeError):
        gd.rmsnorm_q8_0(t.double(), None, torch.ones(64), None, torch.zeros(136, dtype=torch.uint8), 2, 64, 1e-5)
    with pytest.raises(ValueError):
        gd.kv_q8_alloc(2, 16, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        gd.KVCacheQ8(torch.zeros(4), None, None, None)
    with pytest.raises(TypeError):
        monkeypatch.setattr(gd, "_current", lambda: (0, 0))
        gd.rope_table(torch.zeros(4, 4, 2), 4, 8, scaling={"kind": 1})


def test_binding_token_rows(gd):
    """The strides that a token-strided input may have (checked on the CPU: the device index of a CPU tensor is -1)."""
    rows = torch.zeros(5, 6, 64)
    q, k, v = rows.split([4, 1, 1], dim=1)
    assert gd._token_rows(-1, q, torch.float32, 5, 256, "q") == (rows.data_ptr(), 384)
    assert gd._token_rows(-1, k, torch.float32, 5, 64, "k") == (rows.data_ptr() + 4 * 256, 384)
    assert gd._token_rows(-1, rows.view(5, 384)[:, 64:192], torch.float32, 5, 128, "x")[1] == 384
    assert gd._token_rows(-1, rows[:1, :4], torch.float32, 1, 256, "q")[1] == 256
    with pytest.raises(ValueError):
        gd._token_rows(-1, rows.transpose(0, 1), torch.float32, 6, 320, "x")
    with pytest.raises(ValueError):
        gd._token_rows(-1, rows[:, :, ::2], torch.float32, 5, 192, "x")
    with pytest.raises(ValueError):
        gd._token_rows(-1, rows, torch.float32, 4, 384, "x")
    with pytest.raises(ValueError):
        gd._token_rows(0, rows, torch.float32, 5, 384, "x")
    with pytest.raises(TypeError):
        gd._token_rows(-1, rows, torch.bfloat16, 5, 384, "x")


def test_cache_planes_of_another_order_are_refused(gd):
    """Planes with the right number of elements in another order of the axes, or in fewer axes (refused by shape, before the
    device is asked for)."""
    def planes():
        codes = lambda: torch.zeros(3, 2, 32, 64, dtype=torch.int8)
        scales = lambda: torch.zeros(3, 2, 32, 2, dtype=torch.float16)
        return [codes(), scales(), codes(), scales()]
    for i, name in ((1, "k_scales"), (2, "v_codes"), (3, "v_scales")):
        for other in (lambda t: t.transpose(1, 2).contiguous(), lambda t: t.reshape(-1), lambda t: t.reshape(3, 2, 16, -1),
                      lambda t: t[:2]):
            p = planes()
            p[i] = other(p[i])
            with pytest.raises(ValueError, match=name + r" must be \["):
                gd.KVCacheQ8(*p)
        p = planes()
        p[i] = None
        with pytest.raises(TypeError, match=name):
            gd.KVCacheQ8(*p)
    with pytest.raises(ValueError, match="device"):
        gd.KVCacheQ8(*planes())


def test_rows_of_another_order_are_refused(gd):
    """Rows with the heads first or the dims before the heads (on the CPU: the device index of a CPU tensor is -1); the axes that
    say the same, joined or split, are taken."""
    t = torch.zeros(5, 6, 64)
    for same in (t, t.view(5, 384), t.view(30, 64), t.view(-1), t.view(1, 5, 6, 64), t.view(5, 1, 384)):
        assert gd._rows_on(-1, same, torch.float32, 5, 6, 64, "x") == t.data_ptr()
    for other in (t.view(6, 5, 64), t.view(5, 64, 6), t.view(64, 30), t.view(6, 320), t.view(5, 12, 32), t[:4].contiguous(),
                  torch.zeros(4, 8, 60)):
        with pytest.raises(ValueError, match="x must be"):
            gd._rows_on(-1, other, torch.float32, 5, 6, 64, "x")
    assert gd._token_rows(-1, t, torch.float32, 5, 384, "k", 64)[1] == 384
    assert gd._token_rows(-1, t.view(5, 1, 384), torch.float32, 5, 384, "k", 64)[1] == 384
    for other in (t.view(5, 64, 6), t.view(5, 12, 32), t.view(5, 3, 128)):
        with pytest.raises(ValueError, match="k must be"):
            gd._token_rows(-1, other, torch.float32, 5, 384, "k", 64)


@pytest.mark.parametrize("private", [True, False])
def test_current_device_and_stream_without_private_calls(gd, monkeypatch, private):
    """The device and stream come from torch's public functions where the quick ones are not there."""
    asked = []
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: asked.append("public") or 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: type("S", (), {"cuda_stream": 40 + i}))
    for name, value in (("_cuda_getDevice", lambda: 5), ("_cuda_getCurrentRawStream", lambda i: 70 + i)):
        if private:
            monkeypatch.setattr(torch._C, name, value, raising=False)
        else:
            monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(gd, "_device_and_stream", [])
    assert gd._current() == ((5, 75) if private else (3, 43))
    assert gd._current() == ((5, 75) if private else (3, 43))   # asked anew, not kept
    assert len(asked) == (0 if private else 2)
