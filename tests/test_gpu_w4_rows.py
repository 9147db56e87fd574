"""GPU tests: the experts of a 4-bit layer read the norm's bf16 rows, or its 8-bit ones on request."""
import pytest
import torch

from mixture_experts_layer_50_b200 import MoELayer, W4MoELayer
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 20])
def test_rows_of_the_experts(cuda_dev, N):
    shape = W.PRESETS["dsv3-n64"].replace(N=N, d=264, E=8, k=2, F=128)
    t = W.make_inputs(shape, device="cuda")
    w4 = W4MoELayer.from_layer(MoELayer.from_workload(shape, t), group=32)
    res = torch.randn(N, 264, device="cuda").to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(264, device="cuda")).to(torch.bfloat16)
    h, h8 = torch.empty_like(res), torch.empty(N, 264, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(N, 3, device="cuda")
    nat.moe_rms_norm(x=t["x"], residual=res, weight=w, y=h, y8=h8, y8_scale=sc)
    total = (t["x"].float() + res.float()).to(torch.bfloat16)
    want = {False: w4.forward(h), True: w4.forward(h, x8=h8, x8_scale=sc)}
    assert not torch.equal(want[False], want[True])
    for rows8 in want:
        got, s = w4.forward_normed(t["x"], res, w, rows8=rows8)
        assert torch.equal(got, want[rows8]) and torch.equal(s, total)
    assert torch.equal(w4.forward_normed(t["x"], res, w)[0], want[False])  # no fewer bits unless asked for
    assert w4.check_status() == 0
