"""GPU tests of the 4-bit products' accuracy where the codes are small or at the ends of their range.

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

import block_ref as R
from mixture_experts_layer_50_b200 import _native as nat
from test_gpu_w4 import f64, make_x, within
from test_gpu_w4_range import biased_bound, scales_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("codes", [[8], [7, 8, 9], [0], [15], [0, 15]])
@pytest.mark.parametrize("n,rows,cols,group", [(3, 40, 520, 128), (20, 64, 1032, 32), (1, 4112, 4096, 64)])
def test_small_codes_and_the_ends_of_their_range(n, rows, cols, group, codes, kind):
    rng = np.random.default_rng(len(codes) + rows)
    shape = (1, 1, -(-rows // 16), -(-cols // 64), 512)
    pick = lambda: np.array(codes, np.uint8)[rng.integers(0, len(codes), shape)]
    q = pick() | pick() << 4
    s = torch.from_numpy((rng.random(shape[:3] + (-(-cols // group), 8, 2)) * 0.02 + 0.01).astype(np.float32))
    s = s.to(torch.bfloat16)
    w = nat.W4Matrix(torch.from_numpy(q).cuda(), s.cuda(), rows=rows, cols=cols, group=group)
    wv = R.w4_values(q, s.double().numpy(), rows, cols, group)[0, 0]
    x, xs, xg, xv = make_x(n, cols, kind, seed=rows)
    out = torch.empty(n, rows, device="cuda")
    nat.moe_w4_matmul(w, x=x, x_scale=xs, x_group=xg, out=out)
    v = xv @ wv.T
    finite = np.where(np.isnan(xv), 0, xv)
    tol = biased_bound(scales_of(w, rows, cols)[0, 0], cols, group, finite)
    assert within(f64(out), v, tol + np.abs(np.where(np.isnan(v), 0, v)) * 2.0 ** -24)
