"""GPU tests of the balance loss for tokens whose logits are all far below zero, where sigmoids
underflow but their shares are as good as any.

Tolerances: those of test_gpu_balance_loss (2^-17), and as much again for the rounding of an
exponent's argument: a difference of two logits is off by 2^-24 of itself, so a probability
e^-x by x e^-x 2^-24 (at most 2^-25) of the largest, and by 2^-17 of itself up to x = 128; where x is
more, the probability is below 1e-55 and meets the absolute term alone."""
import numpy as np
import pytest
import torch

from gpu_util import check_status, dev, host
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W
from test_gpu_balance_loss import call

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -16
LOWEST = float(np.finfo(np.float32).min)
LEVELS = [0.0, -14.0, -16.0, -17.0, -20.0, -60.0, -88.0, -91.0, -95.0, -100.0, -104.0, -120.0, -200.0, -5000.0, -3e30,
          LOWEST]


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def reference(z, ids, mask, k, alpha):
    """loss, counts, P, dlogits and the magnitudes it is the difference of; sigmoids by their
    logarithms, so that no share is lost."""
    N, E = z.shape
    live = np.ones(N, bool) if mask is None else mask != 0
    T = max(1, int(live.sum()))
    counts = np.bincount(ids[live].ravel(), minlength=E)
    f = counts / (T * k)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        log_s = np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))
        top = log_s.max(1, keepdims=True)
        a = np.where(np.isfinite(top), np.exp(log_s - top), 0.0)
        u = np.where(z > 0, np.exp(-np.abs(z)), 1.0) / (1 + np.exp(-np.abs(z)))
    total = a.sum(1, keepdims=True)
    p = np.divide(a, total, out=np.zeros_like(a), where=total > 0)
    p[~live] = 0
    P = p.sum(0) / T
    f0 = np.abs(f - 1 / E)
    d = alpha * E / T * p * u * (f - (p * f).sum(1, keepdims=True))
    mag = alpha * E / T * p * u * (f0 + (p * f0).sum(1, keepdims=True))
    return alpha * E * (f * P).sum(), counts, P, d, mag


def check(out, z, ids, mask, alpha=0.01, g=1.0):
    E, k = z.shape[1], ids.shape[1]
    loss, counts, P, d, mag = reference(z.astype(np.float64), ids, mask, k, alpha)
    np.testing.assert_array_equal(host(out["counts"]), counts)
    assert (np.abs(host(out["P"]) - P) <= P * TOL + 1e-30).all()
    assert abs(float(out["loss"]) - loss) <= abs(loss) * TOL
    # 2^-50: as there
    err = np.abs(host(out["dlogits"]).astype(np.float64) - g * d)
    assert (err <= abs(g) * mag * TOL + abs(g) * alpha * E * 2.0 ** -50).all()


def make(N, E, k, seed, spread=2.0, masked=False):
    rng = np.random.default_rng(seed)
    level = np.array(LEVELS)[rng.integers(0, len(LEVELS), N)][:, None]
    z = np.maximum(level + rng.standard_normal((N, E)) * spread, LOWEST).astype(np.float32)
    ids = np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)
    return z, ids, (rng.random(N) < 0.7).astype(np.uint8) if masked else None


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,E,k", [(1, 8, 2), (300, 8, 2), (257, 13, 3), (100, 16, 1), (200, 32, 4), (130, 64, 2), (90, 100, 8),
                                   (300, 256, 8), (120, 250, 8), (777, 384, 6), (90, 500, 32), (70, 1024, 8), (5001, 256, 8),
                                   (3601, 384, 6)])
def test_far_negative_rows(N, E, k, masked):
    z, ids, mask = make(N, E, k, seed=N + E, masked=masked)
    out, _, ws = call(z, ids, mask, W.SIGMOID)
    check_status(ws)
    check(out, z, ids, mask)
    again, _, _ = call(z, ids, mask, W.SIGMOID)
    assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.parametrize("level", LEVELS)
@pytest.mark.parametrize("E", [8, 32, 256])
def test_every_row_at_one_level(level, E):
    rng = np.random.default_rng(E)
    z = np.maximum(level + rng.standard_normal((40, E)), LOWEST).astype(np.float32)
    ids = np.argsort(-z, 1, kind="stable")[:, :2].astype(np.int32)
    out, _, _ = call(z, ids, None, W.SIGMOID)
    check(out, z, ids, None)
    assert abs(float(host(out["P"]).astype(np.float64).sum()) - 1) <= 2.0 ** -16


def test_one_expert_ahead_of_far_ones():
    # the largest sigmoid is ordinary or not, the others underflow beside it
    rng = np.random.default_rng(3)
    z = (-95 + rng.standard_normal((60, 24))).astype(np.float32)
    z[np.arange(60), rng.integers(0, 24, 60)] = np.linspace(-110, 10, 60).astype(np.float32)
    z[:, 23] = -np.inf
    z[30] = -np.inf                                       # no probabilities at all
    ids = np.argsort(-z, 1, kind="stable")[:, :2].astype(np.int32)
    out, _, _ = call(z, ids, None, W.SIGMOID)
    check(out, z, ids, None)
    d = host(out["dlogits"])
    assert (d[:, 23] == 0).all() and (d[30] == 0).all()


@pytest.mark.parametrize("E", [8, 40])
def test_ordinary_rows_do_not_depend_on_far_neighbours(E):
    rng = np.random.default_rng(4)
    z = rng.standard_normal((64, E)).astype(np.float32)
    ids = np.tile(np.arange(min(E, 8), dtype=np.int32), (64, 1))     # the same counts, whatever the logits
    near, _, _ = call(z, ids, None, W.SIGMOID)
    far = z.copy()
    far[1::2] -= 100
    got, _, _ = call(far, ids, None, W.SIGMOID)
    assert torch.equal(got["dlogits"][::2], near["dlogits"][::2])


def test_backward_call_of_far_rows():
    z, ids, mask = make(333, 40, 4, seed=12, masked=True)
    g = torch.tensor([-2.5], device="cuda")
    out, cfg, ws = call(z, ids, mask, W.SIGMOID, grad_loss=g)
    check(out, z, ids, mask, g=-2.5)
    base = torch.randn(333, 40, device="cuda")
    acc = base.clone()
    nat.moe_balance_loss_backward(cfg, logits=dev(z), ids=dev(ids), token_mask=dev(mask), alpha=0.01, grad_loss=g,
                                  dlogits=acc, accumulate=True, ws=ws)
    assert torch.equal(acc, base + out["dlogits"])


@pytest.mark.parametrize("score", [W.SOFTMAX, W.SIGMOID])
def test_infinite_logits(score):
    z, ids, _ = make(40, 24, 2, seed=5)
    z[:] = np.random.default_rng(6).standard_normal((40, 24))
    z[11, 3] = np.inf
    out, _, _ = call(z, ids, None, score)
    if score == W.SIGMOID:                 # a sigmoid of 1
        check(out, z, ids, None)
    else:                                  # no probabilities: it shows
        assert np.isnan(float(out["loss"])) and np.isnan(host(out["P"])).all()
        assert np.isnan(host(out["dlogits"])[11]).all()
        assert np.isfinite(np.delete(host(out["dlogits"]), 11, 0)).all()
