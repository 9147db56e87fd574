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


@pytest.mark.parametrize("wrong", [[], [5, 6, 4000, 8989], [0, 4, 8990, 9000]])
def test_more_row_indices_than_are_looked_over_at_the_start(wrong):
    # beyond 8192 rows every tile looks at its own; indices outside the groups are nobody's
    w, wv = make_w(2, 1, 64, 264, 64, seed=46)
    x, _, _, xv = make_x(300, 264, "bf16", seed=47)
    idx = np.random.default_rng(48).integers(0, 300, 9001).astype(np.int32)
    idx[wrong] = 300
    off = np.array([5, 4000, 8990], np.int32)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    out = torch.full((9001, 64), -3.0, device="cuda")
    nat.moe_w4_matmul(w, x=x, offsets=dev(off), row_index=dev(idx), out=out, ws=ws)
    inside = [r for r in wrong if 5 <= r < 8990]
    assert nat.moe_check_status(ws) == (nat.MOE_ERR_INVALID_INPUT if inside else 0)
    got = f64(out)
    assert (got[inside] == 0).all() and (got[:5] == -3).all() and (got[8990:] == -3).all()
    for e in range(2):
        rows = np.setdiff1d(np.arange(off[e], off[e + 1]), np.array(inside, int))
        v, tol = expect(wv[e], xv[idx[rows]], 264, 64)
        assert (np.abs(got[rows] - v) <= tol + np.abs(v) * 2.0 ** -24).all()
