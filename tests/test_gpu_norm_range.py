"""GPU tests of moe_rms_norm for finite rows whose squares leave fp32's range, and for tiny eps.

Tolerances: those of test_gpu_norm.  Where a row is rescaled, it is by a power of two, which is
exact, and what its squares lose below 2^-149 is below 2^-60 of their sum."""
import numpy as np
import pytest
import torch

import block_ref as R
from gpu_util import host
from test_gpu_norm import check, f64, make, run

pytestmark = pytest.mark.gpu
BF, F4 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


# each way of sharing out a row: a warp with 1, 2 and 4 vectors a thread, a block with 1, 2 and 4
SHAPES = [(9, 136, BF), (5, 504, BF), (3, 1000, BF), (2, 7168, BF), (520, 1032, BF), (515, 5120, BF), (2, 16384, BF),
          (9, 68, F4), (3, 500, F4), (2, 2048, F4), (520, 1408, F4), (3, 16384, F4)]


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("N,d,dtype", SHAPES)
def test_squares_above_the_range(N, d, dtype, group):
    x, res, w = make(N, d, dtype, seed=d)
    scale = torch.tensor([2.0 ** e for e in (62, 1, 70, 100, 120)], device="cuda")[torch.arange(N, device="cuda") % 5]
    xs, rs = ((t.double() * scale[:, None]).to(dtype) for t in (x, res))
    out = run(xs, rs, w, group)
    check(xs, rs, w, out, group)
    plain = run((x.double() * 2).to(dtype), (res.double() * 2).to(dtype), w, group)
    for n in out:                                                  # rows of the ordinary kind are as they were
        assert torch.equal(out[n][1::5], plain[n][1::5]), n


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 1e-30, 2.0 ** -81, 2.0 ** -79, 1e-20])
@pytest.mark.parametrize("N,d,dtype", SHAPES)
def test_squares_below_the_range(N, d, dtype, eps):
    x, _, w = make(N, d, dtype, seed=d + 1, residual=False)
    # (fp32 down to 2^-120: below that the inputs themselves would have fewer digits)
    scale = torch.tensor([2.0 ** e for e in (-45, 0, -55, -70, -100, -120)], device="cuda")[
        torch.arange(N, device="cuda") % 6]
    xs = (x.double() * scale[:, None]).to(dtype)
    out = run(xs, None, w, 128, eps=float(np.float32(eps)))
    s, y = R.rms_norm(f64(xs), None, f64(w), float(np.float32(eps)))
    keep = np.abs(y).max(1) > 2.0 ** -100                          # (rows that eps swallows whole have tiny y)
    sel = lambda t: None if t is None else t[torch.from_numpy(np.flatnonzero(keep)).cuda()].contiguous()
    check(sel(xs), None, w, {n: sel(t) for n, t in out.items()}, 128, ref=(s[keep], y[keep]), eps=eps)
    got = host(out["y"])
    assert np.isfinite(got).all() and (np.abs(got[~keep]) <= 2.0 ** -99).all()


@pytest.mark.parametrize("N,d,dtype", SHAPES)
def test_largest_values_of_the_type(N, d, dtype):
    big = torch.finfo(dtype).max
    x = torch.full((N, d), big, dtype=dtype, device="cuda")
    x[:, 1::2] = -big
    out = run(x, None, None, 128)
    check(x, None, None, out, 128)
    # rsqrtf is off by 2 ulp: 2^-22 (and nothing is left of that in bf16)
    assert (np.abs(np.abs(host(out["y"])) - 1) <= (0 if dtype == BF else 2.0 ** -18)).all()


def test_a_sum_that_is_infinite_stays_infinite():
    x = torch.full((2, 1408), 2.0 ** 127, dtype=BF, device="cuda")
    x[1] = 1.0
    out = run(x, x.clone(), None, 128)
    y = host(out["y"])
    assert np.isnan(y[0]).all() and np.isinf(host(out["residual_out"])[0]).all()
    assert (y[1] == 1).all()


def test_zero_rows_with_and_without_eps():
    x = torch.zeros(4, 1032, dtype=F4, device="cuda")
    x[2] = 1e-25
    y = host(run(x, None, None, 128, eps=1e-30)["y"])
    assert (y[[0, 1, 3]] == 0).all()
    want = 1e-25 / np.sqrt(1e-50 + 1e-30)
    assert (np.abs(y[2] - want) <= want * 2.0 ** -18).all()
    y = host(run(x, None, None, 128, eps=0.0)["y"])
    assert np.isnan(y[[0, 1, 3]]).all() and (np.abs(y[2] - 1) <= 2.0 ** -18).all()      # 0 / 0
