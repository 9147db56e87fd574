"""GPU tests of the 4-bit products' groups of rows where the offsets contradict each other."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from mixture_experts_layer_50_b200 import _native as nat
from test_gpu_w4 import expect, f64, make_w, make_x

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def test_bad_indices_behind_a_bad_offset_read_zeros():
    # group 0 has 100 rows, group 1 would have -50: only group 0 runs, and all its indices are checked
    w, wv = make_w(2, 1, 32, 128, 64, seed=41)
    x, _, _, xv = make_x(20, 128, "bf16", seed=42)
    idx = np.random.default_rng(43).integers(0, 20, 100).astype(np.int32)
    wrong = [50, 60, 77, 99]
    idx[wrong] = [20, -1, 10 ** 6, -2 ** 31]
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    out = torch.full((100, 32), -3.0, device="cuda")
    nat.moe_w4_matmul(w, x=x, offsets=dev(np.array([0, 100, 50], np.int32)), row_index=dev(idx), out=out, ws=ws)
    assert nat.moe_check_status(ws) == nat.MOE_ERR_INVALID_INPUT
    got = f64(out)
    assert (got[wrong] == 0).all()
    keep = np.setdiff1d(np.arange(100), wrong)
    v, tol = expect(wv[0], xv[idx[keep]], 128, 64)
    assert (np.abs(got[keep] - v) <= tol + np.abs(v) * 2.0 ** -24).all()


def test_the_same_row_in_two_groups_of_decreasing_offsets():
    # 0..40 and 10..50 overlap; what each writes is its own product, or the other's
    w, wv = make_w(3, 1, 32, 128, 64, seed=44)
    x, _, _, xv = make_x(50, 128, "bf16", seed=45)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    out = torch.full((50, 32), -3.0, device="cuda")
    nat.moe_w4_matmul(w, x=x, offsets=dev(np.array([0, 40, 10, 50], np.int32)), out=out, ws=ws)
    assert nat.moe_check_status(ws) == nat.MOE_ERR_INVALID_INPUT
    got = f64(out)
    near = []
    for e in (0, 2):
        v, tol = expect(wv[e], xv, 128, 64)
        near.append(np.abs(got - v) <= tol + np.abs(v) * 2.0 ** -24)
    assert near[0][:10].all() and near[1][40:].all() and (near[0] | near[1])[10:40].all()
