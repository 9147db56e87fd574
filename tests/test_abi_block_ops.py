"""Host-side checks of the norm, the 4-bit products and the balance loss: refused before the GPU
is touched, so these run without one."""
import ctypes

import pytest
import torch

from mixture_experts_layer_50_b200 import _native as nat

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100004)
lib = nat.lib


def w4(q=FAKE, scale=FAKE, mats=1, parts=1, rows=64, cols=128, group=64):
    return nat.moe_w4(q, scale, mats, parts, rows, cols, group)


def cfg(**kw):
    return nat.make_config(**{**dict(N=16, d=128, E=4, k=2, F=64), **kw})


def norm(N=4, d=256, dtype=0, x=FAKE, residual=None, weight=None, eps=1e-6, y=FAKE, residual_out=None,
         y8=None, y8_scale=None, group=128):
    return lib.moe_rms_norm(N, d, dtype, x, residual, weight, eps, y, residual_out, y8, y8_scale, group, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 1), (dict(d=0), 1), (dict(dtype=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(group=64), 1), (dict(residual_out=FAKE), 1), (dict(y8=FAKE), 1), (dict(y8_scale=FAKE), 1),
    (dict(y=None), 1), (dict(x=None), 1), (dict(d=12), 2), (dict(d=32776), 2), (dict(d=6, dtype=1), 2),
    (dict(d=16388, dtype=1), 2), (dict(N=2 ** 31), 2), (dict(x=ODD), 2), (dict(y=ODD), 2),
    (dict(residual=ODD), 2), (dict(weight=ODD), 2), (dict(y8=ODD, y8_scale=FAKE), 2),
    (dict(residual=FAKE, residual_out=ODD), 2)])
def test_norm_refuses(kw, code):
    assert norm(**kw) == code
    assert lib.moe_last_error()


def test_norm_without_rows_is_nothing():
    assert norm(N=0, x=None, y=None) == 0


BAD_W4 = [(dict(mats=0), 1), (dict(parts=3), 1), (dict(rows=0), 1), (dict(cols=0), 1), (dict(group=16), 1),
          (dict(cols=100), 2), (dict(mats=1026), 2), (dict(rows=2 ** 25), 2)]


@pytest.mark.parametrize("kw,code", BAD_W4 + [(dict(q=None), 1), (dict(scale=None), 1), (dict(q=ODD), 2),
                                              (dict(scale=ODD), 2)])
def test_w4_matrices_are_checked(kw, code):
    w = w4(**kw)
    call = lambda: lib.moe_w4_matmul(ctypes.byref(w), FAKE, None, 128, 8, None, None, 8, 0.0, FAKE, 0, None, None)
    assert call() == code and lib.moe_last_error()
    assert lib.moe_w4_quantize(ctypes.byref(w), FAKE, None) == code
    if (kw, code) in BAD_W4:
        assert lib.moe_w4_size(ctypes.byref(w), None) == 0


def test_w4_size():
    sc = ctypes.c_size_t()
    # 3 x 2 matrices of 33 x 72: 3 blocks of rows, 2 of columns, 3 groups
    assert lib.moe_w4_size(ctypes.byref(w4(None, None, 3, 2, 33, 72, 32)), ctypes.byref(sc)) == 3 * 2 * 3 * 2 * 512
    assert sc.value == 3 * 2 * 3 * 3 * 32
    assert lib.moe_w4_size(None, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(x_rows=-1), 1), (dict(x_rows=7), 1), (dict(x_scale=FAKE, x_group=64), 1),
    (dict(clamp=float("nan")), 1), (dict(out_dtype=3), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(x=ODD), 2), (dict(out=ODD), 2), (dict(rows=2 ** 30 + 1, x_rows=2 ** 30 + 1), 2), (dict(ws=ODD), 1)])
def test_w4_matmul_refuses(kw, code):
    a = {**dict(x=FAKE, x_scale=None, x_group=128, x_rows=8, offsets=None, rows=8, clamp=0.0, out=FAKE,
                out_dtype=0, ws=None), **kw}
    st = lib.moe_w4_matmul(ctypes.byref(w4()), a["x"], a["x_scale"], a["x_group"], a["x_rows"], a["offsets"], None,
                           a["rows"], a["clamp"], a["out"], a["out_dtype"], a["ws"], None)
    assert st == code and lib.moe_last_error()


def test_w4_matmul_needs_offsets_for_several_matrices():
    w = w4(mats=2)
    assert lib.moe_w4_matmul(ctypes.byref(w), FAKE, None, 128, 8, None, None, 8, 0.0, FAKE, 0, None, None) == 1


def test_w4_matmul_needs_a_row_to_read():
    call = lambda rows: lib.moe_w4_matmul(ctypes.byref(w4()), FAKE, None, 128, 0, None, FAKE, rows, 0.0, FAKE, 0, None,
                                          None)
    assert call(8) == 1 and b"no rows" in lib.moe_last_error()
    assert call(0) == 0


GU = dict(mats=4, parts=2, rows=64, cols=128)
DOWN = dict(mats=4, parts=1, rows=128, cols=64)


def ffn(c=None, gu=None, down=None, x=FAKE, offsets=FAKE, row_token=FAKE, ye=FAKE, ws=FAKE):
    c, gu, down = c or cfg(), w4(**{**GU, **(gu or {})}), w4(**{**DOWN, **(down or {})})
    return lib.moe_expert_ffn_w4(ctypes.byref(c), x, None, offsets, row_token, ctypes.byref(gu), ctypes.byref(down),
                                 ye, ws, None)


def forward(c=None, gu=None, down=None, x=FAKE, x8=None, x8_scale=None, W_g=FAKE, bias=None, y=FAKE, ws=FAKE):
    c, gu, down = c or cfg(), w4(**{**GU, **(gu or {})}), w4(**{**DOWN, **(down or {})})
    return lib.moe_forward_w4(ctypes.byref(c), x, x8, x8_scale, W_g, None, bias, None, ctypes.byref(gu),
                              ctypes.byref(down), y, None, ws, None)


@pytest.mark.parametrize("call", [ffn, forward])
@pytest.mark.parametrize("kw,code", [
    (dict(gu=dict(mats=5)), 1), (dict(gu=dict(parts=1)), 1), (dict(gu=dict(rows=72)), 1), (dict(gu=dict(cols=64)), 1),
    (dict(down=dict(mats=3)), 1), (dict(down=dict(parts=2)), 1), (dict(down=dict(rows=64)), 1),
    (dict(down=dict(cols=128)), 1), (dict(c=cfg(n_shared=1)), 1), (dict(c=cfg(k=5)), 1), (dict(c=cfg(dtype=1)), 2),
    (dict(x=None), 1), (dict(x=ODD), 2), (dict(ws=None), 1), (dict(ws=ODD), 1)])
def test_layers_with_4_bit_experts_refuse(call, kw, code):
    assert call(**kw) == code and lib.moe_last_error()


def test_more_refusals_of_the_layer():
    assert ffn(offsets=None) == 1 and ffn(row_token=None) == 1 and ffn(ye=None) == 1
    assert forward(x8=FAKE) == 1 and forward(x8_scale=FAKE) == 1 and forward(W_g=None) == 1
    assert forward(y=None) == 1 and forward(bias=FAKE) == 1 and forward(x8=ODD, x8_scale=FAKE) == 2


def test_balance_loss_refuses():
    c = cfg()
    def loss(c=c, logits=FAKE, ids=FAKE, alpha=1.0, ws=FAKE):
        return lib.moe_balance_loss(ctypes.byref(c), logits, ids, None, alpha, None, FAKE, FAKE, FAKE, FAKE, ws, None)
    def back(c=c, logits=FAKE, ids=FAKE, alpha=1.0, dlogits=FAKE, accumulate=0, ws=FAKE):
        return lib.moe_balance_loss_backward(ctypes.byref(c), logits, ids, None, alpha, None, dlogits, accumulate, ws,
                                             None)
    for call in (loss, back):
        assert call(logits=None) == 1 and call(ids=None) == 1 and call(alpha=float("nan")) == 1
        assert call(ws=None) == 1 and call(ws=ODD) == 1 and call(c=cfg(k=5)) == 1 and call(c=cfg(E=2000)) == 2
    assert back(dlogits=None) == 1 and back(accumulate=2) == 1


def test_binding_checks_types_and_shapes():
    with pytest.raises(ValueError):
        nat.moe_rms_norm(x=torch.zeros(2, 8, dtype=torch.float16), y=torch.zeros(2, 8, dtype=torch.float16))
    with pytest.raises(ValueError):          # host tensors
        nat.moe_rms_norm(x=torch.zeros(2, 8), y=torch.zeros(2, 8))
    with pytest.raises(ValueError):
        nat.W4Matrix.quantize(torch.zeros(1, 33, 64, dtype=torch.bfloat16), parts=2)
    with pytest.raises(nat.MoeError):
        nat.W4Matrix(torch.zeros(1, 1, 1, 1, 512, dtype=torch.uint8), torch.zeros(1), rows=16, cols=60, group=64)


class ElsewhereMatrix:
    """Stands for a W4Matrix on a device that is not the current one."""
    class q:
        get_device = staticmethod(lambda: 7)
    mats, parts, rows, cols, group = 4, 1, 64, 128, 64
    c = w4()


class Uncalled:
    def __getattr__(self, name):
        return lambda *a: pytest.fail(f"{name} was called")


def test_4_bit_matrices_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(nat.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(nat, "_typed", lambda t, *a: 0)
    monkeypatch.setattr(nat, "_stream", lambda s: None)
    monkeypatch.setattr(nat, "_ptr", lambda t: 0)
    monkeypatch.setattr(nat, "lib", Uncalled())
    m, x = ElsewhereMatrix(), torch.zeros(16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda:7"):
        nat.moe_w4_matmul(m, x=x, out=torch.zeros(16, 64))
    with pytest.raises(ValueError, match="cuda:7"):
        nat.moe_expert_ffn_w4(cfg(), x=x, offsets=None, row_token=None, W_gu=m, W_down=m, ye=None, ws=None)
    with pytest.raises(ValueError, match="cuda:7"):
        nat.moe_forward_w4(cfg(), x=x, W_g=None, W_gu=m, W_down=m, y=x, ws=None)
