"""GPU tests: a host thread's first CUDA work may be any of the library's calls, and calls on
workspaces of their own run beside one another."""
import threading

import pytest
import torch

from mixture_experts_layer_50_b200 import MoELayer, W4MoELayer
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def in_thread(f):
    """f's result, or its exception, from a thread that has done nothing yet."""
    got = []

    def run():
        try:
            got.append(f())
        except Exception as e:
            got.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


SHAPE = W.PRESETS["dsv3-n64"].replace(N=20, d=256, E=8, k=2, F=128)


def layers():
    t = W.make_inputs(SHAPE, device="cuda")
    layer = MoELayer.from_workload(SHAPE, t)
    return layer, W4MoELayer.from_layer(layer, group=32), t["x"]


@pytest.mark.parametrize("which", [0, 1])
def test_a_layer_is_the_first_work_of_a_thread(which):
    *both, x = layers()
    want = both[which].forward(x)
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    in_thread(lambda: both[which].forward(x, y=y))
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_the_operators_around_it_are_the_first_work_of_a_thread():
    _, w4, x = layers()
    s = torch.cuda.current_stream()
    y, y1 = torch.empty_like(x), torch.empty_like(x)
    out, out1 = (torch.empty(20, 128, device="cuda") for _ in range(2))
    one = nat.W4Matrix(w4.W_gu.q[:1], w4.W_gu.scale[:1], rows=128, cols=256, group=32)
    z, ids = torch.randn(20, 8, device="cuda"), torch.zeros(20, 2, dtype=torch.int32, device="cuda")
    cfg = nat.make_config(20, 256, 8, 2, 128)
    ws, (d, d1) = nat.alloc_workspace(cfg), (torch.empty(20, 8, device="cuda") for _ in range(2))
    calls = [lambda o: nat.moe_rms_norm(x=x, y=o, stream=s), lambda o: nat.moe_w4_matmul(one, x=x, out=o, stream=s),
             lambda o: nat.moe_balance_loss(cfg, logits=z, ids=ids, alpha=1.0, dlogits=o, ws=ws, stream=s)]
    for call, a, b in zip(calls, (y, out, d), (y1, out1, d1)):
        call(a)
        in_thread(lambda: call(b))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_threads_with_layers_of_their_own():
    layer, first, x = layers()
    second = W4MoELayer.from_layer(layer, group=32)
    want = first.forward(x)
    torch.cuda.synchronize()
    results = [[], []]

    def run(w4, out):
        for _ in range(50):
            out.append(w4.forward(x))
    threads = [threading.Thread(target=run, args=a) for a in zip((first, second), results)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(r) for r in results] == [50, 50] and all(torch.equal(y, want) for r in results for y in r)
