"""GPU tests of the 4-bit products: rows of large numbers of one sign.

Tolerances.  The kernel multiplies codes 0..15, two rows of weights in one sum (code + 16 code'),
starts from -8 (and -136) times the sum of x, and takes the second row's sum as a difference: so
its roundings go with B = scale * sum |x|, whatever the codes are.  The magnitudes in a sum are at
most (255 + 136) sum |x| for both rows and (15 + 8) sum |x| for the one, 26 sum |x| after the
division by 16.  An mma's error is below 2^-22 of them for each 16 columns, the sum of x is added
with 7 roundings of 2^-24 (8 to 136 times), and the groups' sums join as in test_gpu_w4, each at
most 8 B.  So the error is at most ((group / 16) * 26 + 16 + (columns / group + 12) * 2) * 2^-22 * sum B."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_50_b200 import _native as nat
from test_gpu_w4 import f64, make_w, make_x, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def biased_bound(w, cols, group, x):
    """The bound above for rows x [n][cols] and the scales that w [rows][cols] was made with."""
    return (group / 16 * 26 + 16 + (cols / group + 12) * 2) * 2.0 ** -22 * (np.abs(x) @ w.T)


def scales_of(w, rows, cols):
    """[mats, parts, rows, cols]: each weight's scale."""
    s = w.scale.double().cpu().numpy()
    r, c = np.arange(rows)[:, None], np.arange(cols)[None]
    return s[:, :, r // 16, c // w.group, r % 8, r % 16 // 8]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,rows,cols", [(3, 40, 512), (17, 64, 1032), (1, 16, 8)])
def test_rows_of_one_sign_up_to_the_largest(n, rows, cols, group, sign):
    w, wv = make_w(1, 1, rows, cols, group, seed=31)
    sv = scales_of(w, rows, cols)[0, 0]
    rng = np.random.default_rng(32)
    for e in (0, 56, 57, 58, 60, 62):
        x = torch.from_numpy(sign * (1 + rng.random((n, cols)) * 0.9) * 2.0 ** e).to(torch.bfloat16).cuda()
        xv = f64(x)
        out = torch.empty(n, rows, device="cuda")
        nat.moe_w4_matmul(w, x=x, out=out)
        v = xv @ wv[0, 0].T
        assert within(f64(out), v, biased_bound(sv, cols, group, xv) + np.abs(v) * 2.0 ** -24), e
    same = torch.full((n, cols), sign * 2.0 ** 57, dtype=torch.bfloat16, device="cuda")
    nat.moe_w4_matmul(w, x=same, out=out)
    v = f64(same) @ wv[0, 0].T
    assert within(f64(out), v, biased_bound(sv, cols, group, f64(same)) + np.abs(v) * 2.0 ** -24)


@pytest.mark.parametrize("value", [2.0 ** 63, -2.0 ** 63, float("inf"), float("-inf"), float("nan"), 3e38])
def test_rows_with_a_number_that_counts_as_infinite(value):
    w, _ = make_w(1, 1, 64, 520, 64, seed=33)
    x, _, _, _ = make_x(11, 520, "bf16", seed=34)
    clean, got = torch.empty(11, 64, device="cuda"), torch.empty(11, 64, device="cuda")
    nat.moe_w4_matmul(w, x=x, out=clean)
    x[4, 77] = value
    x[9, 519] = value
    x[9, 0] = -value
    nat.moe_w4_matmul(w, x=x, out=got)
    bad = torch.zeros(11, dtype=torch.bool, device="cuda")
    bad[[4, 9]] = True
    assert torch.equal(got[~bad], clean[~bad])
    assert not torch.isfinite(got[bad]).any()
