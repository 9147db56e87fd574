"""GPU tests: 4-bit layers and matrices whose stream is given as a raw handle, or is not the
current one, take their memory from that stream."""
import pytest
import torch

from mixture_experts_layer_50_b200 import MoELayer, W4MoELayer
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def layer():
    shape = W.PRESETS["dsv3-n64"].replace(N=20, d=256, E=8, k=2, F=128)
    t = W.make_inputs(shape, device="cuda")
    return W4MoELayer.from_layer(MoELayer.from_workload(shape, t)), t["x"]


def given_back(like, n=6):
    """Places that the current stream has given back, and may still be writing."""
    freed = [torch.empty_like(like) for _ in range(n)]
    return {f.data_ptr() for f in freed}


@pytest.mark.parametrize("raw", [False, True])
def test_layer(raw):
    w4, x = layer()
    want, total = w4.forward_normed(x, x)
    plain = w4.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = side.cuda_stream if raw else side
    places = given_back(want)
    got, got_total = w4.forward_normed(x, x, stream=stream)
    got_plain = w4.forward(x, stream=stream)
    torch.cuda.synchronize()
    assert not places & {g.data_ptr() for g in (got, got_total, got_plain)}
    assert torch.equal(got, want) and torch.equal(got_total, total) and torch.equal(got_plain, plain)


@pytest.mark.parametrize("raw", [False, True])
def test_host_buffers(raw):
    w4, x = layer()
    want = w4.forward(x).cpu()
    xh = [x.cpu().pin_memory() for _ in range(3)]
    yh = [torch.zeros(20, 256, dtype=torch.bfloat16).pin_memory() for _ in range(3)]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    assert torch.equal(w4.forward_host(xh[0], yh[0], stream=stream), want)
    yh[0].zero_()
    w4.forward_host_batches(xh, yh, stream=stream)
    assert all(torch.equal(y, want) for y in yh)


def test_the_null_stream_and_its_other_handle():
    w4, x = layer()
    want = w4.forward(x)
    for handle in (0, 1):                   # NULL and cudaStreamLegacy
        got, _ = w4.forward_normed(x, torch.zeros_like(x), stream=handle)
        assert torch.equal(w4.forward(x, stream=handle), want)
        torch.cuda.synchronize()
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("raw", [False, True])
def test_quantize(raw):
    Wt = torch.randn(2, 64, 256, device="cuda").to(torch.bfloat16)
    want = nat.W4Matrix.quantize(Wt, parts=2, group=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    places = given_back(want.q) | given_back(want.scale)
    got = nat.W4Matrix.quantize(Wt, parts=2, group=64, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert not places & {got.q.data_ptr(), got.scale.data_ptr()}
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


BUSY = 200_000_000                          # clock cycles: a tenth of a second


def taken_anew(places, stream, make, n=6):
    """Whether memory at ``places`` is handed out while ``stream`` is at work (an allocation that
    has to wait for the device may find it done)."""
    new = []
    for _ in range(n):
        new.append(make())
        if new[-1].data_ptr() in places and not stream.query():
            return True
    return False


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_inputs_given_back_while_the_other_stream_still_reads_them(raw, normed):
    w4, x = layer()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    t, u, g = x.clone(), x.clone(), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    places = {t.data_ptr()} | ({u.data_ptr(), g.data_ptr()} if normed else set())
    want = w4.forward_normed(t, u, g)[0] if normed else w4.forward(t)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = w4.forward_normed(t, u, g, stream=stream)[0] if normed else w4.forward(t, stream=stream)
    del t, u, g
    assert not taken_anew(places, side, lambda: torch.zeros_like(x))
    assert not taken_anew(places, side, lambda: torch.zeros(256, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_outputs_given_back_while_the_current_stream_still_reads_them():
    w4, x = layer()
    side = torch.cuda.Stream()
    for f in (lambda: w4.forward(x, stream=side), lambda: w4.forward_normed(x, x, stream=side)):
        got = f()
        torch.cuda.synchronize()
        got = got if isinstance(got, tuple) else (got,)
        places = {g.data_ptr() for g in got}
        torch.cuda._sleep(BUSY)
        read = [g + 0 for g in got]
        del got
        current = torch.cuda.current_stream()
        with torch.cuda.stream(side):
            assert not taken_anew(places, current, lambda: torch.empty_like(x))
        torch.cuda.synchronize()
        assert all(torch.isfinite(r).all() for r in read)


def test_quantised_weights_given_back_while_the_other_stream_still_reads_them():
    Wt = torch.randn(2, 64, 256, device="cuda").to(torch.bfloat16)
    want = nat.W4Matrix.quantize(Wt, parts=2, group=64)
    side, place, like = torch.cuda.Stream(), Wt.data_ptr(), torch.zeros_like(Wt)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = nat.W4Matrix.quantize(Wt, parts=2, group=64, stream=side)
    del Wt
    assert not taken_anew({place}, side, lambda: torch.zeros_like(like))
    torch.cuda.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


@pytest.mark.parametrize("raw", [False, True])
def test_captured_on_a_stream_that_is_given(raw):
    w4, x = layer()
    want, (want_n, total) = w4.forward(x), w4.forward_normed(x, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        stream = side.cuda_stream if raw else side
        y = w4.forward(x, stream=stream)
        n, t = w4.forward_normed(x, x, stream=stream)
    for _ in range(2):
        for o in (y, n, t):
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(n, want_n) and torch.equal(t, total)
