"""The calls around the layer refuse memory of another device, and arrays too small or of another
type, before the library is called (no GPU needed: the tensors are stand-ins)."""
import pytest
import torch

from mixture_experts_layer_50_b200 import _native as nat


class Stand:
    """What the binding asks of a device tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


class Uncalled:
    def __getattr__(self, name):
        return lambda *a: pytest.fail(f"{name} was called")


@pytest.fixture(autouse=True)
def _stand_ins(monkeypatch):
    monkeypatch.setattr(nat.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(nat, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(nat, "_stream", lambda s: None)
    monkeypatch.setattr(nat, "lib", Uncalled())


I32, BF, U8 = torch.int32, torch.bfloat16, torch.uint8
CFG = nat.make_config(N=16, d=128, E=4, k=2, F=64, n_bias_sets=2)


class Matrix:
    """Stands for a W4Matrix of the current device."""
    def __init__(self, mats, parts, rows, cols):
        self.q = Stand(mats, dtype=U8)
        self.mats, self.parts, self.rows, self.cols, self.group = mats, parts, rows, cols, 64
        self.c = nat.moe_w4(None, None, mats, parts, rows, cols, 64)


GU, DOWN = Matrix(4, 2, 64, 128), Matrix(4, 1, 128, 64)
AWAY = Stand(1 << 20, dtype=U8, device=1)
CALLS = [
    lambda ws: nat.moe_balance_loss(CFG, logits=Stand(16, 4), ids=Stand(16, 2, dtype=I32), alpha=1.0, ws=ws),
    lambda ws: nat.moe_balance_loss_backward(CFG, logits=Stand(16, 4), ids=Stand(16, 2, dtype=I32), alpha=1.0,
                                             dlogits=Stand(16, 4), ws=ws),
    lambda ws: nat.moe_w4_matmul(Matrix(1, 1, 64, 128), x=Stand(16, 128, dtype=BF), out=Stand(16, 64), ws=ws),
    lambda ws: nat.moe_expert_ffn_w4(CFG, x=Stand(16, 128, dtype=BF), offsets=Stand(5, dtype=I32),
                                     row_token=Stand(32, dtype=I32), W_gu=GU, W_down=DOWN,
                                     ye=Stand(32, 128, dtype=BF), ws=ws),
    lambda ws: forward(ws=ws),
]


def forward(ws=None, **kw):
    return nat.moe_forward_w4(CFG, x=Stand(16, 128, dtype=BF), W_g=Stand(4, 128, dtype=BF), W_gu=GU, W_down=DOWN,
                              y=Stand(16, 128, dtype=BF), ws=Stand(1 << 20, dtype=U8) if ws is None else ws, **kw)


@pytest.mark.parametrize("call", CALLS)
def test_workspace_of_another_device(call):
    with pytest.raises(ValueError, match="ws is on cuda:1"):
        call(AWAY)


GOOD = dict(logit_offset=Stand(4), bias=Stand(2, 4), modality=Stand(16, dtype=U8))
ROUTE = dict(logits=Stand(16, 4), ids=Stand(16, 2, dtype=I32), gates=Stand(16, 2), counts=Stand(4, dtype=I32),
             demand=Stand(4, dtype=I32), drop_mask=Stand(16, 2, dtype=U8), offsets=Stand(5, dtype=I32))


@pytest.mark.parametrize("name", list(GOOD) + list(ROUTE))
@pytest.mark.parametrize("fault", ["device", "size", "type"])
def test_other_arrays_of_the_layer(name, fault):
    good = GOOD.get(name) or ROUTE[name]
    bad = {"device": Stand(*good.shape, dtype=good.dtype, device=1),
           "size": Stand(good.numel() - 1, dtype=good.dtype),
           "type": Stand(*good.shape, dtype=torch.float16)}[fault]
    with pytest.raises(ValueError, match=name):
        forward(**{name: bad}) if name in GOOD else forward(route_out={name: bad})


def test_the_right_arrays_reach_the_library(monkeypatch):
    class Called(Exception):
        pass

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise Called(name)
            return call
    monkeypatch.setattr(nat, "lib", Lib())
    with pytest.raises(Called, match="moe_forward_w4"):
        forward(route_out=ROUTE, **GOOD)
    with pytest.raises(Called):                        # longer ones are fine too
        forward(route_out=dict(ids=Stand(64, 2, dtype=I32)), modality=Stand(99, dtype=torch.bool))
    for call in CALLS:
        with pytest.raises(Called):
            call(Stand(1 << 20, dtype=U8))
