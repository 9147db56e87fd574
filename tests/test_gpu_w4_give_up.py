"""GPU tests of the 4-bit products where a wait inside the kernel runs out: the status word says
so, no output that may lack rows is passed off as a number, the kernel ends and the next call is
right.  (The library's self-test lets one warp start as if its wait had run out; nothing waits for
it in vain.)"""
import pytest
import torch

from gpu_util import check_status
from mixture_experts_layer_50_b200 import _native as nat
from test_gpu_w4 import make_w, make_x

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def workspace():
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    return ws[(-ws.data_ptr()) % 256:][:256]


# whole rounds of items, items cut into units, clusters of blocks; one and several tiles of rows
SHAPES = [(1, 7176, 2056, 2, 128), (3, 2064, 14336, 1, 64), (16, 4104, 1800, 2, 64), (33, 1032, 7176, 1, 128),
          (200, 512, 1160, 1, 64), (2, 48, 264, 1, 32), (3, 520, 14344, 1, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("warp", [0, 5, 15, 16 + 3, 32, 7 * 16 + 9])
@pytest.mark.parametrize("n,rows,cols,parts,group", SHAPES)
def test_one_warp_gives_up(n, rows, cols, parts, group, warp, kind):
    w, _ = make_w(1, parts, rows, cols, group, seed=rows)
    x, xs, xg, _ = make_x(n, cols, kind, seed=n)
    x = x if kind == "bf16" else torch.where(x.float().isnan(), torch.zeros_like(x.float()), x.float()).to(x.dtype)
    a = dict(x=x, x_scale=xs, x_group=xg)
    want = torch.empty(n, rows, device="cuda")
    nat.moe_w4_matmul(w, out=want, **a)
    assert torch.isfinite(want).all()
    for ws in (workspace(), None):
        out = torch.full((n + 1, rows), -3.0, device="cuda")
        nat.moe_selftest_w4_give_up(w, out=out[:n], ws=ws, warp=warp, **a)
        torch.cuda.synchronize()
        gone = torch.isnan(out[:n])
        assert torch.equal(out[:n][~gone], want[~gone]) and bool((out[n] == -3).all())
        if ws is not None:
            # (a small product has fewer blocks, or some without outputs)
            st = nat.moe_check_status(ws)
            assert st == nat.MOE_ERR_TIMEOUT or (st == 0 and not gone.any() and warp >= 16)
        assert bool(gone.any()) or warp >= 16
    ws = workspace()
    nat.moe_w4_matmul(w, out=out[:n], ws=ws, **a)
    check_status(ws)
    assert torch.equal(out[:n], want)


def test_other_blocks_are_as_always():
    w, _ = make_w(1, 1, 40000, 512, 64, seed=1)              # more items than blocks
    x, _, _, _ = make_x(5, 512, "bf16", seed=2)
    want, out = torch.empty(5, 40000, device="cuda"), torch.empty(5, 40000, device="cuda")
    nat.moe_w4_matmul(w, x=x, out=want)
    nat.moe_selftest_w4_give_up(w, x=x, out=out, warp=3)
    gone = torch.isnan(out)
    assert gone.any() and not gone.all() and torch.equal(out[~gone], want[~gone])


def test_it_shows_in_bf16_and_behind_swiglu():
    w, _ = make_w(1, 2, 64, 256, 64, seed=3)
    x, _, _, _ = make_x(4, 256, "bf16", seed=4)
    out = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    nat.moe_selftest_w4_give_up(w, x=x, out=out, warp=0)
    assert torch.isnan(out).all()
    with pytest.raises(nat.MoeError):
        nat.moe_selftest_w4_give_up(w, x=x, out=out, warp=-1)
