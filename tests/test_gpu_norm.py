"""GPU tests of moe_rms_norm against the float64 definition.

Tolerances.  A row's sum of squares is added in fp32: at most 32 terms in a thread, 5 steps in a
warp, 5 over the warps, each rounding by 2^-24 of a sum of positive terms; the square root halves
that; rsqrtf (2 ulp), the division, two products and the rounding of s add 8 more roundings.
42 / 2 + 2 * 2 + 8 roundings are below 64 * 2^-24 = 2^-18, relative to y.  Rounding to bf16 adds
2^-8, to e4m3 2^-4 (or half of the smallest step, 2^-10, of the scaled value)."""
import numpy as np
import pytest
import torch

import block_ref as R
from gpu_util import host
from mixture_experts_layer_50_b200 import _native as nat

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -18


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def make(N, d, dtype, seed, residual=True, weight=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = r(N, d).to(dtype)
    res = (r(N, d) * 3).to(dtype) if residual else None
    w = (1 + 0.3 * r(d)).to(dtype) if weight else None
    return x, res, w


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def run(x, res, w, group, eps=EPS, y=None, residual_out=None):
    N, d = x.shape
    out = dict(y=torch.empty_like(x) if y is None else y,
               residual_out=None if res is None else (torch.empty_like(x) if residual_out is None
                                                      else residual_out),
               y8=torch.full((N, d), 0x55, dtype=torch.uint8, device="cuda"),
               y8_scale=torch.full((N, -(-d // 128) if group else 1), -1.0, device="cuda"))
    nat.moe_rms_norm(x=x, residual=res, weight=w, eps=eps, group=group, **out)
    return out


def check(x, res, w, out, group, ref=None, eps=EPS):
    s, y = R.rms_norm(f64(x), f64(res), f64(w), eps) if ref is None else ref
    step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0
    got = f64(out["y"])
    assert (np.abs(got - y) <= np.abs(y) * (step * 1.001 + F32) + 1e-38).all()
    if out["residual_out"] is not None:
        step_s = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(f64(out["residual_out"]) - s) <= np.abs(s) * (step_s * 1.001 + 2.0 ** -24)).all()
    q, sc = R.e4m3_to_f64(host(out["y8"])), f64(out["y8_scale"])
    for i, (a, b) in enumerate(R.groups(x.shape[1], group)):
        amax = np.abs(y[:, a:b]).max(1)
        assert (np.abs(sc[:, i] - amax / 448) <= amax / 448 * (F32 + 2.0 ** -22)).all()
        err = np.abs(q[:, a:b] * sc[:, i:i + 1] - y[:, a:b])
        tol = np.abs(y[:, a:b]) * (2.0 ** -4 + F32) + sc[:, i:i + 1] * 2.0 ** -10 * (1 + F32)
        assert (err <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("N,d", [(1, 8), (1, 7168), (3, 120), (9, 136), (17, 264), (5, 504),
                                 (7, 1032), (33, 1408), (130, 2048), (2, 5120), (6, 10008),
                                 (2, 16384)])
def test_norm_against_float64(N, d, dtype, group):
    x, res, w = make(N, d, dtype, seed=N * 7 + d)
    check(x, res, w, run(x, res, w, group), group)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 32768), (torch.float32, 4), (torch.float32, 12)])
def test_largest_and_smallest_rows(dtype, d):
    x, res, w = make(3, d, dtype, seed=d)
    check(x, res, w, run(x, res, w, 128), 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_residual_or_weight(dtype):
    x, _, _ = make(10, 1160, dtype, 3, residual=False, weight=False)
    check(x, None, None, run(x, None, None, 128), 128)
    # the 8-bit output alone, and the norm alone
    y8 = torch.empty(10, 1160, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(10, 10, device="cuda")
    nat.moe_rms_norm(x=x, eps=EPS, y8=y8, y8_scale=sc)
    both = run(x, None, None, 128)
    assert torch.equal(y8.view(torch.uint8), both["y8"]) and torch.equal(sc, both["y8_scale"])
    y = torch.empty_like(x)
    nat.moe_rms_norm(x=x, eps=EPS, y=y)
    assert torch.equal(y, both["y"])


def test_in_place():
    x, res, w = make(21, 4096, torch.bfloat16, 5)
    want = run(x, res, w, 128)
    xi, ri = x.clone(), res.clone()
    got = run(xi, ri, w, 128, y=xi, residual_out=ri)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_zero_rows_and_groups():
    x, _, w = make(4, 512, torch.bfloat16, 6, residual=False)
    x[1] = 0
    x[2, 128:256] = 0
    out = run(x, None, w, 128)
    check(x, None, w, out, 128)
    assert (host(out["y8_scale"])[1] == 0).all() and (host(out["y8"])[1] & 127 == 0).all()
    assert host(out["y8_scale"])[2, 1] == 0
    row = run(x, None, w, 0)
    assert host(row["y8_scale"])[1, 0] == 0


def test_tiny_values_keep_a_finite_scale():
    # y = 1e-40 (subnormal): amax / 448 would be below 2^-126
    x = torch.full((1, 256), 1e-30, dtype=torch.float32, device="cuda")
    w = torch.full((256,), 1e-7, dtype=torch.float32, device="cuda")
    out = run(x, None, w, 128, eps=1e6)
    s, y = R.rms_norm(f64(x), None, f64(w), 1e6)
    assert (host(out["y8_scale"]) >= 2.0 ** -126).all()
    q = R.e4m3_to_f64(host(out["y8"])) * np.repeat(f64(out["y8_scale"]), 128, 1)
    assert (np.abs(q - y) <= 2.0 ** -126 * 2.0 ** -9).all()


def test_non_finite_values_stay_in_their_row():
    x, _, w = make(5, 1408, torch.bfloat16, 7, residual=False)
    clean = run(x, None, w, 128)
    x[1, 700] = float("nan")
    x[3, 5] = float("inf")
    out = run(x, None, w, 128)
    y = host(out["y"])
    assert np.isnan(y[1]).all()
    assert np.isnan(y[3, 5]) and (np.delete(y[3], 5) == 0).all()      # finite / infinite = 0
    sc, q = host(out["y8_scale"]), R.e4m3_to_f64(host(out["y8"]))
    assert np.isnan(sc[1]).all() and np.isnan(q[1]).all()
    assert not np.isfinite(sc[3, 0]) and (sc[3, 1:] == 0).all()
    for n in ("y", "y8", "y8_scale"):
        assert torch.equal(out[n][[0, 2, 4]], clean[n][[0, 2, 4]])
    x[3, 5] = 0
    assert np.isnan(host(run(x, None, w, 0)["y8_scale"])[1]).all()


def test_rows_do_not_touch_each_other_or_their_surroundings():
    # N not a multiple of the rows of a block; canaries behind the last row
    N, d = 13, 72
    x, res, w = make(N, d, torch.bfloat16, 8)
    buf = torch.full((N + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    nat.moe_rms_norm(x=x, residual=res, weight=w, eps=EPS, y=buf[:N])
    assert (buf[N:] == 7).all()
    one = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    for i in (0, 7, 8, 12):
        nat.moe_rms_norm(x=x[i:i + 1], residual=res[i:i + 1], weight=w, eps=EPS, y=one)
        assert torch.equal(one[0], buf[i])


def test_no_rows():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    nat.moe_rms_norm(x=e, y=e)


def test_stream_and_graph_replay():
    x, res, w = make(64, 2048, torch.bfloat16, 9)
    out = run(x, res, w, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nat.moe_rms_norm(x=x, residual=res, weight=w, eps=EPS, **out)
    x2, res2, _ = make(64, 2048, torch.bfloat16, 10)
    x.copy_(x2)
    res.copy_(res2)
    g.replay()
    torch.cuda.synchronize()
    want = run(x2, res2, w, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = {n: torch.empty_like(v) for n, v in out.items()}
    nat.moe_rms_norm(x=x2, residual=res2, weight=w, eps=EPS, stream=s, **side)
    s.synchronize()
    for n in want:
        assert torch.equal(out[n], want[n]) and torch.equal(side[n], want[n]), n
