"""Host-side limits of the 4-bit products, without a GPU: the kernel numbers tiles of rows in 32
bits, for the groups that contradicting offsets can describe too (each up to all rows of out)."""
import ctypes

import pytest

from mixture_experts_layer_50_b200 import _native as nat

FAKE = ctypes.c_void_p(0x100000)
lib = nat.lib


def matmul(rows, mats):
    w = nat.moe_w4(FAKE, FAKE, mats, 1, 8, 64, 64)
    return lib.moe_w4_matmul(ctypes.byref(w), FAKE, None, 128, 16, FAKE, FAKE, rows, 0.0, FAKE, 0, None, None)


@pytest.mark.parametrize("rows,mats", [(2 ** 24 + 2 ** 15, 1025), (2 ** 27, 1025), (2 ** 28, 64)])
def test_rows_times_matrices(rows, mats):
    assert (rows // 8 + 1) * mats >= 2 ** 31
    assert matmul(rows, mats) == nat.MOE_ERR_UNSUPPORTED
    assert b"too many rows" in lib.moe_last_error()


def test_rows_times_experts():
    c = nat.make_config(N=2 ** 25, d=64, E=1024, k=1, F=64)
    gu, down = nat.moe_w4(FAKE, FAKE, 1024, 2, 64, 64, 64), nat.moe_w4(FAKE, FAKE, 1024, 1, 64, 64, 64)
    st = lib.moe_expert_ffn_w4(ctypes.byref(c), FAKE, None, FAKE, FAKE, ctypes.byref(gu), ctypes.byref(down), FAKE,
                               FAKE, None)
    assert st == nat.MOE_ERR_UNSUPPORTED and b"too many rows" in lib.moe_last_error()
