"""GPU tests of moe_balance_loss and moe_balance_loss_backward against the float64 definition.

Tolerances.  A probability is two expf (2 ulp each at most), a sum of at most 1024 terms over a
tree of 32 adds and 5 shuffles, a reciprocal and a product: below 2^-18 relative.  P adds at most
16384 of them over sums of positive terms in chains of at most 32 adds per team (fp32), then in
fixed point: below 2^-17.  The gradient is a difference of two terms of that accuracy."""
import numpy as np
import pytest
import torch

import block_ref as R
from gpu_util import check_status, dev, host
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -17


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def make(N, E, k, seed, masked=False, scale=1.5):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((N, E)) * scale + rng.standard_normal(E) * 0.7).astype(np.float32)
    ids = np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)
    mask = (rng.random(N) < 0.7).astype(np.uint8) if masked else None
    return z, ids, mask


def call(z, ids, mask, score, alpha=0.01, grad_loss=None, ws=None, cfg=None):
    N, E = z.shape
    k = ids.shape[1]
    cfg = cfg or nat.make_config(N, 8, E, k, 8, score_fn=score)
    ws = nat.alloc_workspace(cfg) if ws is None else ws
    out = dict(loss=torch.full((1,), 9.0, device="cuda"),
               counts=torch.full((E,), -5, dtype=torch.int32, device="cuda"),
               P=torch.full((E,), 9.0, device="cuda"),
               dlogits=torch.full((N, E), 9.0, device="cuda"))
    nat.moe_balance_loss(cfg, logits=dev(z), ids=dev(ids), token_mask=None if mask is None else dev(mask),
                         alpha=alpha, grad_loss=grad_loss, ws=ws, **out)
    return out, cfg, ws


def check(out, z, ids, mask, score, alpha=0.01, g=1.0):
    E, k = z.shape[1], ids.shape[1]
    loss, counts, P, d, mag = R.balance(z.astype(np.float64), ids, mask, E, k, alpha, score == W.SIGMOID)
    np.testing.assert_array_equal(host(out["counts"]), counts)
    assert (np.abs(host(out["P"]) - P) <= P * TOL + 1e-30).all()
    assert abs(float(out["loss"]) - loss) <= abs(loss) * TOL
    # 2^-50: the last bits of the float64 reference where all f are equal
    assert (np.abs(host(out["dlogits"]).astype(np.float64) - g * d) <= abs(g) * mag * TOL
            + abs(g) * alpha * E * 2.0 ** -50).all()


@pytest.mark.parametrize("score", [W.SOFTMAX, W.SIGMOID])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (1, 4, 2), (3, 5, 5), (31, 8, 2), (100, 13, 3),
                                   (257, 32, 4), (500, 33, 2), (64, 64, 1), (129, 100, 8),
                                   (300, 256, 8), (777, 384, 6), (90, 500, 32), (70, 1024, 8),
                                   (16384, 64, 2)])
def test_loss_counts_and_gradient(N, E, k, masked, score):
    z, ids, mask = make(N, E, k, seed=N + E, masked=masked)
    out, _, ws = call(z, ids, mask, score)
    check_status(ws)
    check(out, z, ids, mask, score)


@pytest.mark.parametrize("score", [W.SOFTMAX, W.SIGMOID])
def test_gradient_against_differences(score):
    z, ids, mask = make(12, 7, 2, seed=4, masked=True)
    out, _, _ = call(z, ids, mask, score, alpha=1.0)
    got = host(out["dlogits"]).astype(np.float64)
    z64, h = z.astype(np.float64), 1e-5
    f = lambda v: R.balance(v, ids, mask, 7, 2, 1.0, score == W.SIGMOID)[0]
    for t in range(12):
        for e in range(7):
            up, dn = z64.copy(), z64.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central difference: h^2 times the third derivative (below 1), and 1e-16 / h
            assert abs((f(up) - f(dn)) / (2 * h) - got[t, e]) <= 1e-9 + 1e-6 * np.abs(got).max()


def test_masked_tokens_may_hold_anything():
    z, ids, mask = make(200, 48, 4, seed=6, masked=True)
    clean, _, _ = call(z, ids, mask, W.SOFTMAX)
    z2, ids2 = z.copy(), ids.copy()
    z2[mask == 0] = np.nan
    ids2[mask == 0] = 10 ** 6
    dirty, _, ws = call(z2, ids2, mask, W.SOFTMAX)
    check_status(ws)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    assert (host(dirty["dlogits"])[mask == 0] == 0).all()


def test_no_token_left():
    z, ids, _ = make(40, 16, 2, seed=7)
    out, _, _ = call(z, ids, np.zeros(40, np.uint8), W.SIGMOID)
    for n in out:
        assert (host(out[n]) == 0).all(), n


def test_no_tokens_at_all():
    cfg = nat.make_config(0, 8, 16, 2, 8)
    ws = nat.alloc_workspace(cfg)
    loss = torch.full((1,), 9.0, device="cuda")
    counts = torch.full((16,), 9, dtype=torch.int32, device="cuda")
    nat.moe_balance_loss(cfg, logits=torch.empty(0, 16, device="cuda"),
                         ids=torch.empty(0, 2, dtype=torch.int32, device="cuda"), alpha=1.0,
                         loss=loss, counts=counts, ws=ws)
    assert float(loss) == 0 and (counts == 0).all()


def test_excluded_experts_and_empty_rows():
    # -inf logits: experts that a mask forbids; one token may use none
    z, ids, _ = make(50, 24, 2, seed=8)
    z[:, 20:] = -np.inf
    z[7] = -np.inf
    ids = np.argsort(-z, 1, kind="stable")[:, :2].astype(np.int32)
    out, _, _ = call(z, ids, None, W.SOFTMAX)
    check(out, z, ids, None, W.SOFTMAX)
    d = host(out["dlogits"])
    assert (d[:, 20:] == 0).all() and (d[7] == 0).all() and np.isfinite(d).all()
    low = np.where(np.isinf(z), np.finfo(np.float32).min, z).astype(np.float32)
    out2, _, _ = call(low, ids, None, W.SOFTMAX)   # masks of the type's lowest value
    keep = np.arange(50) != 7
    np.testing.assert_array_equal(host(out2["dlogits"])[keep], d[keep])


def test_nan_is_not_hidden():
    z, ids, _ = make(50, 24, 2, seed=9)
    z[11, 3] = np.nan
    for score in (W.SOFTMAX, W.SIGMOID):
        out, _, _ = call(z, ids, None, score)
        assert np.isnan(host(out["dlogits"])[11]).all() and np.isnan(float(out["loss"]))
        assert np.isfinite(np.delete(host(out["dlogits"]), 11, 0)).all()
        if score == W.SOFTMAX:
            assert np.isnan(host(out["P"])).all()


def test_extreme_logits():
    z, ids, _ = make(64, 32, 3, seed=10, scale=60.0)
    out, _, _ = call(z, ids, None, W.SOFTMAX)
    E, k = 32, 3
    loss, _, P, d, mag = R.balance(z.astype(np.float64), ids, None, E, k, 0.01, False)
    # expf's argument is rounded: 2^-24 of a difference up to 500 moves a probability by 2^-15
    assert (np.abs(host(out["P"]) - P) <= P * 2.0 ** -14 + 1e-30).all()
    assert np.isfinite(host(out["dlogits"])).all()


def test_invalid_ids_are_reported_and_count_nowhere():
    z, ids, _ = make(30, 16, 2, seed=11)
    ids[4, 1], ids[9, 0] = 16, -1
    out, _, ws = call(z, ids, None, W.SOFTMAX)
    assert nat.moe_check_status(ws) == nat.MOE_ERR_INVALID_INPUT
    ok = ids[(ids >= 0) & (ids < 16)]
    np.testing.assert_array_equal(host(out["counts"]), np.bincount(ok, minlength=16))


@pytest.mark.parametrize("score", [W.SOFTMAX, W.SIGMOID])
def test_backward_call_scales_and_accumulates(score):
    z, ids, mask = make(333, 40, 4, seed=12, masked=True)
    g = torch.tensor([-2.5], device="cuda")
    out, cfg, ws = call(z, ids, mask, score, grad_loss=g)
    check(out, z, ids, mask, score, g=-2.5)
    d = torch.full((333, 40), 3.0, device="cuda")
    args = dict(logits=dev(z), ids=dev(ids), token_mask=dev(mask), alpha=0.01, grad_loss=g, ws=ws)
    nat.moe_balance_loss_backward(cfg, dlogits=d, **args)
    assert torch.equal(d, out["dlogits"])
    base = torch.randn(333, 40, device="cuda")
    acc = base.clone()
    nat.moe_balance_loss_backward(cfg, dlogits=acc, accumulate=True, **args)
    assert torch.equal(acc, base + out["dlogits"])


def test_same_bits_every_time_and_after_other_calls():
    a = make(5000, 96, 4, seed=13, masked=True)
    b = make(5000, 96, 4, seed=14)
    first, cfg, ws = call(*a, W.SOFTMAX)
    ws.fill_(0xAB)                       # the scratch needs no preparation
    nat.moe_workspace_init(ws)
    for _ in range(3):
        call(*b, W.SOFTMAX, ws=ws, cfg=cfg)
        again, _, _ = call(*a, W.SOFTMAX, ws=ws, cfg=cfg)
        for n in first:
            assert torch.equal(first[n], again[n]), n


def test_agrees_with_the_statistic():
    z, ids, _ = make(2000, 64, 6, seed=15)
    out, cfg, ws = call(z, ids, None, W.SIGMOID, alpha=1.0)
    aux = torch.empty(1, device="cuda")
    load = torch.empty(64, dtype=torch.int32, device="cuda")
    nat.moe_balance(cfg, logits=dev(z), ids=dev(ids), aux=aux, set_load=load, ws=ws)
    assert torch.equal(load, out["counts"])
    assert abs(float(aux) - float(out["loss"])) <= 1e-5 * float(aux)


def test_graph_replay_and_side_stream():
    z, ids, mask = make(700, 48, 4, seed=16, masked=True)
    want, cfg, ws = call(z, ids, mask, W.SOFTMAX)
    zd, idd, md = dev(z), dev(ids), dev(mask)
    out = {n: torch.zeros_like(v) for n, v in want.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nat.moe_balance_loss(cfg, logits=zd, ids=idd, token_mask=md, alpha=0.01, ws=ws, **out)
    for _ in range(2):
        for v in out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), n
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = {n: torch.empty_like(v) for n, v in want.items()}
    ws2 = nat.alloc_workspace(cfg)
    torch.cuda.synchronize()
    nat.moe_balance_loss(cfg, logits=zd, ids=idd, token_mask=md, alpha=0.01, ws=ws2, stream=s, **other)
    s.synchronize()
    for n in want:
        assert torch.equal(other[n], want[n]), n


@pytest.mark.parametrize("score", [W.SOFTMAX, W.SIGMOID])
@pytest.mark.parametrize("N,E,k", [(5001, 256, 8), (4999, 250, 2), (3601, 384, 6), (3700, 383, 1), (2500, 512, 4),
                                   (2501, 509, 3)])
def test_more_tokens_than_the_gpu_holds(N, E, k, score):
    z, ids, mask = make(N, E, k, seed=N + E, masked=True)
    out, _, ws = call(z, ids, mask, score)
    check(out, z, ids, mask, score)
    check_status(ws)
    again, _, _ = call(z, ids, mask, score)
    assert all(torch.equal(out[n], again[n]) for n in ("loss", "counts", "P", "dlogits"))


def test_logits_written_just_before_the_call():
    # (the row pass loads its first logits while the assignments are still being counted)
    sets = [make(4000, 64, 2, seed=s, masked=False) for s in (1, 2)]
    want = [call(z, ids, None, W.SOFTMAX)[0] for z, ids, _ in sets]
    zs, idss = [dev(z) for z, _, _ in sets], [dev(i) for _, i, _ in sets]
    z, ids = torch.empty_like(zs[0]), torch.empty_like(idss[0])
    cfg = nat.make_config(4000, 8, 64, 2, 8)
    ws = nat.alloc_workspace(cfg)
    got = [dict(loss=torch.zeros(1, device="cuda"), dlogits=torch.zeros_like(z)) for _ in range(40)]
    def run():
        for i, g in enumerate(got):
            z.copy_(zs[i % 2])
            ids.copy_(idss[i % 2])
            nat.moe_balance_loss(cfg, logits=z, ids=ids, alpha=0.01, ws=ws, **g)
    def right():
        torch.cuda.synchronize()
        return all(torch.equal(g[n], want[i % 2][n]) for i, g in enumerate(got) for n in g)
    run()
    assert right()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for g in got:
        g["dlogits"].zero_()
    graph.replay()
    assert right()
