"""GPU tests of the products with 4-bit weights (moe_w4_quantize, moe_w4_matmul,
moe_expert_ffn_w4, moe_forward_w4) against float64.

Tolerances.  Codes times rows are exact; an mma adds 16 exact products to an fp32 sum with an
error below 2^-22 of the sum of their magnitudes, so a group's sum is off by group / 16 times
that; scaling it adds three roundings of 2^-24 (two scales and the product), adding it to the
others one for each group, and adding up to eight partial sums eight.  With A = sum |w x| that is
at most (group / 16 + (columns / group + 12) / 4) * 2^-22 * A.  SiLU(g) u moves by at most 1.1 |u| dg +
|SiLU(g)| du, and its own evaluation by 2^-20.  Rounding to bf16 is 2^-8 relative."""
import ctypes

import numpy as np
import pytest
import torch

import block_ref as R
import oracle as O
from gpu_util import assert_close_layer, check_status, dev, host
from mixture_experts_layer_50_b200 import _native as nat
from mixture_experts_layer_50_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


@pytest.fixture(autouse=True)
def _needs_cuda(cuda_dev):
    yield


def f64(t):
    return t.double().cpu().numpy()


def make_w(mats, parts, rows, cols, group, seed):
    """Random codes (the whole range) and scales; returns the W4Matrix and its values."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (mats, parts, -(-rows // 16), -(-cols // 64), 512), dtype=np.uint8)
    s = (rng.random((mats, parts, -(-rows // 16), -(-cols // group), 8, 2)) * 0.02 + 0.01).astype(np.float32)
    st = torch.from_numpy(s).to(torch.bfloat16)
    w = nat.W4Matrix(torch.from_numpy(q).cuda(), st.cuda(), rows=rows, cols=cols, group=group)
    return w, R.w4_values(q, st.double().numpy(), rows, cols, group)


def make_x(n, cols, kind, seed):
    """(x, x_scale, x_group, float64 values)"""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((n, cols)).astype(np.float32)
    if kind == "bf16":
        x = torch.from_numpy(v).to(torch.bfloat16)
        return x.cuda(), None, 128, x.double().numpy()
    group = 128 if kind == "e4m3" else 0
    x = torch.from_numpy(v * 100).to(torch.float8_e4m3fn)
    ng = len(R.groups(cols, group))
    sc = (rng.random((n, ng)) * 0.02 + 0.005).astype(np.float32)
    val = x.double().numpy() * np.repeat(sc.astype(np.float64), group or cols, 1)[:, :cols]
    return x.cuda(), dev(sc), group, val


def bound(w, cols, group, x):
    return (group / 16 + (cols / group + 12) / 4) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T)


def within(got, v, tol):
    """Every finite expected value is met within tol; a NaN row of the 8-bit inputs (a draw beyond
    the type's range) gives NaN."""
    nan = np.isnan(v)
    return np.array_equal(nan, np.isnan(got)) and (np.abs(got - v)[~nan] <= np.broadcast_to(tol, v.shape)[~nan]).all()


def expect(w, x, cols, group, clamp=0.0):
    """(value, tolerance) of one group's rows x through parts w [parts][rows][cols], fp32."""
    z = [x @ m.T for m in w]
    t = [bound(m, cols, group, x) for m in w]
    if len(z) == 1:
        return z[0], t[0]
    v = R.swiglu(z[0], z[1], clamp)
    up = np.abs(z[1]) if clamp <= 0 else np.minimum(np.abs(z[1]), clamp)
    return v, 1.1 * (up + t[1]) * t[0] + (np.abs(R.silu(z[0])) + t[0]) * t[1] + 2.0 ** -20 * np.abs(v)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3 row"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,rows,cols,parts", [
    (1, 16, 64, 1), (1, 8, 8, 1), (1, 40, 72, 2), (2, 33, 136, 1), (8, 160, 1032, 2),
    (9, 48, 2056, 1), (17, 24, 320, 2), (32, 100, 520, 1), (33, 17, 4096, 1), (70, 64, 264, 2),
    (5, 4112, 192, 1)])
def test_one_matrix(n, rows, cols, parts, group, kind):
    w, wv = make_w(1, parts, rows, cols, group, seed=rows + cols)
    x, xs, xg, xv = make_x(n, cols, kind, seed=n)
    v, tol = expect(wv[0], xv, cols, group)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((n + 2, rows), -3.0, dtype=dt, device="cuda")
        nat.moe_w4_matmul(w, x=x, x_scale=xs, x_group=xg, out=buf[:n])
        step = BF if dt == torch.bfloat16 else 2.0 ** -24
        assert within(f64(buf[:n]), v, tol + (np.abs(v) + tol) * step + 1e-37)
        assert (buf[n:] == -3).all()


def test_codes_are_read_where_the_layout_says():
    # one code differs from 8 at a time: the output is that weight's column of x
    rows, cols, group = 40, 136, 32
    x = torch.arange(1, cols + 1, dtype=torch.float32).to(torch.bfloat16).reshape(1, cols).cuda()
    rng = np.random.default_rng(0)
    for _ in range(40):
        r, c, code = int(rng.integers(rows)), int(rng.integers(cols)), int(rng.integers(16))
        q = np.full((1, 1, 3, 3, 512), 0x88, np.uint8)
        g, half = r % 8, (r % 16) // 8
        byte = 16 * (4 * g + (c % 32) // 8) + 4 * (2 * ((c % 64) // 32) + (c % 8) // 4) + 2 * (c % 2) + (c % 4) // 2
        q[0, 0, r // 16, c // 64, byte] = (code | 0x80) if half == 0 else (0x08 | code << 4)
        sc = torch.ones(1, 1, 3, 5, 8, 2, dtype=torch.bfloat16)
        sc[0, 0, r // 16, c // group, g, half] = 0.5
        w = nat.W4Matrix(torch.from_numpy(q).cuda(), sc.cuda(), rows=rows, cols=cols, group=group)
        out = torch.empty(1, rows, device="cuda")
        nat.moe_w4_matmul(w, x=x, out=out)
        want = np.zeros(rows)
        want[r] = 0.5 * (code - 8) * float(x[0, c])
        np.testing.assert_array_equal(host(out)[0], want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes", [[3, 0, 1, 40, 0, 8], [0, 0, 0, 0, 0, 0], [1, 1, 1, 1, 1, 1],
                                   [0, 0, 100, 0, 0, 0], [7, 9, 16, 17, 32, 33]])
def test_groups_and_row_index(sizes, kind):
    mats, rows, cols, group = 6, 72, 328, 64
    w, wv = make_w(mats, 1, rows, cols, group, seed=5)
    x, xs, xg, xv = make_x(50, cols, kind, seed=6)
    R_ = sum(sizes)
    idx = np.random.default_rng(7).integers(0, 50, R_ + 9).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    out = torch.full((R_ + 9, rows), -3.0, device="cuda")
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    nat.moe_w4_matmul(w, x=x, x_scale=xs, x_group=xg, offsets=dev(off), row_index=dev(idx), out=out, ws=ws)
    check_status(ws)
    got = f64(out)
    for e in range(mats):
        s = slice(off[e], off[e + 1])
        v, tol = expect(wv[e], xv[idx[s]], cols, group)
        assert within(got[s], v, tol + np.abs(v) * 2.0 ** -24)
    assert (got[R_:] == -3).all()                        # behind the last group


def test_many_groups():
    mats = 1025
    w, wv = make_w(mats, 1, 16, 64, 64, seed=8)
    sizes = np.random.default_rng(9).integers(0, 3, mats)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    x, _, _, xv = make_x(int(off[-1]), 64, "bf16", seed=10)
    out = torch.empty(int(off[-1]), 16, device="cuda")
    nat.moe_w4_matmul(w, x=x, offsets=dev(off), out=out)
    e = np.repeat(np.arange(mats), sizes)
    v = np.einsum("rc,rwc->rw", xv, wv[e, 0])
    tol = (64 / 16 + 13 / 4) * 2.0 ** -22 * np.einsum("rc,rwc->rw", np.abs(xv), np.abs(wv[e, 0]))
    assert (np.abs(f64(out) - v) <= tol + np.abs(v) * 2.0 ** -24).all()


def test_bad_offsets_and_indices_are_reported():
    w, wv = make_w(3, 1, 32, 128, 128, seed=11)
    x, _, _, xv = make_x(6, 128, "bf16", seed=12)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:256]
    out = torch.full((6, 32), -3.0, device="cuda")
    nat.moe_w4_matmul(w, x=x, offsets=dev(np.array([0, 2, 9, 6], np.int32)), out=out, ws=ws)
    assert nat.moe_check_status(ws) == nat.MOE_ERR_INVALID_INPUT
    assert (out[2:] == -3).all() and (out[:2] != -3).all()
    idx = dev(np.array([0, 6, -1, 3, 4, 5], np.int32))
    nat.moe_w4_matmul(w, x=x, offsets=dev(np.array([0, 2, 4, 6], np.int32)), row_index=idx, out=out, ws=ws)
    assert nat.moe_check_status(ws) == nat.MOE_ERR_INVALID_INPUT
    assert (out[1:3] == 0).all() and (out[3:] != 0).any()


def test_swiglu_clamp_and_large_preactivations():
    w, wv = make_w(1, 2, 64, 256, 64, seed=13)
    x, _, _, xv = make_x(6, 256, "bf16", seed=14)
    x = x * 64
    xv = xv * 64
    out = torch.empty(6, 64, device="cuda")
    for clamp in (0.0, 10.0):
        nat.moe_w4_matmul(w, x=x, clamp=clamp, out=out)
        v, tol = expect(wv[0], xv, 256, 64, clamp)
        assert np.isfinite(host(out)).all()
        assert (np.abs(f64(out) - v) <= tol + np.abs(v) * 2.0 ** -22 + 1e-30).all()


def test_non_finite_rows_stay_their_own():
    w, _ = make_w(1, 1, 48, 192, 64, seed=15)
    x, _, _, _ = make_x(12, 192, "bf16", seed=16)
    clean, got = torch.empty(12, 48, device="cuda"), torch.empty(12, 48, device="cuda")
    nat.moe_w4_matmul(w, x=x, out=clean)
    x[3, 100] = float("nan")
    x[9, 0] = float("inf")
    nat.moe_w4_matmul(w, x=x, out=got)
    keep = [i for i in range(12) if i not in (3, 9)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[9]).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("mats,parts,rows,cols", [(1, 1, 16, 64), (2, 2, 40, 200), (3, 1, 17, 1032)])
def test_quantize(mats, parts, rows, cols, group):
    rng = np.random.default_rng(rows)
    Wt = torch.from_numpy((rng.standard_normal((mats, parts * rows, cols)) * 0.02).astype(np.float32)).to(torch.bfloat16)
    Wt[0, 3, :min(group, cols)] = 0
    w = nat.W4Matrix.quantize(Wt.cuda(), parts=parts, group=group)
    wv = Wt.double().numpy().reshape(mats, parts, rows, cols)
    ng = -(-cols // group)
    pad = np.zeros((mats, parts, rows, ng * group))
    pad[..., :cols] = wv
    amax = np.abs(pad).reshape(mats, parts, rows, ng, group).max(-1)
    r = np.arange(rows)
    sc = w.scale.double().cpu().numpy()[:, :, r // 16][:, :, np.arange(rows), :, r % 8, (r % 16) // 8]
    sc = np.moveaxis(sc, 0, 2)             # [mats, parts, rows, ng]
    assert (np.abs(sc - amax / 7) <= amax / 7 * (BF * 1.001)).all()
    got = R.w4_values(w.q.cpu().numpy(), w.scale.double().cpu().numpy(), rows, cols, group)
    full = np.repeat(sc, group, -1)[..., :cols]
    # half a step, or up to a bf16 rounding of the scale beyond the last code
    assert (np.abs(got - wv) <= full * (0.5 + 7 * BF) * 1.0001).all()
    # padding is code 8 (zero)
    if cols % 64:
        codes = w.q.cpu().numpy()[..., -1, :].reshape(mats, parts, -1, 8, 4, 2, 2, 2, 2)
        first_pad = cols % 64              # a multiple of 8
        for h in range(2):
            for t in range(4):
                if 32 * h + 8 * t >= first_pad:
                    assert (codes[:, :, :, :, t, h] == 0x88).all()


def ffn_case(N, d, F, E, k, S, group, kind, act=W.SWIGLU, clamp=0.0, seed=0, drop=0):
    rng = np.random.default_rng(seed)
    parts = 2 if act == W.SWIGLU else 1
    gu, guv = make_w(E + S, parts, F, d, group, seed + 1)
    dn, dnv = make_w(E + S, 1, d, F, group, seed + 2)
    x, xs, _, xv = make_x(N, d, kind, seed + 3)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(N)]).astype(np.int32)
    cfg = nat.make_config(N, d, E, k, F, n_shared=S, act=act, clamp=clamp)
    pairs = [[t for t in range(N) if e in ids[t]] for e in range(E)]
    if drop:
        pairs = [p[:drop] for p in pairs]
    off = np.concatenate([[0], np.cumsum([len(p) for p in pairs])]).astype(np.int32)
    tok = np.zeros(N * k, np.int32)
    tok[:off[-1]] = np.concatenate(pairs)
    return cfg, gu, guv, dn, dnv, x, xs, xv, off, tok


def ffn_expect(guv, dnv, xv, d, F, group, act, clamp):
    if act == W.SWIGLU:
        h, th = expect(guv, xv, d, group, clamp)
    else:
        z, th = expect(guv, xv, d, group)
        h = np.maximum(z, 0)
    th = th + (np.abs(h) + th) * BF                        # h is stored as bf16
    y = h @ dnv[0].T
    return y, th @ np.abs(dnv[0]).T + bound(dnv[0], F, group, np.abs(h) + th)


@pytest.mark.parametrize("N,d,F,E,k,S,group,kind,act,clamp,drop", [
    (1, 128, 64, 4, 2, 0, 64, "bf16", W.SWIGLU, 0.0, 0),
    (1, 264, 200, 5, 5, 1, 128, "e4m3", W.SWIGLU, 0.0, 0),
    (7, 200, 136, 9, 3, 1, 32, "bf16", W.SWIGLU, 0.1, 0),
    (40, 512, 328, 6, 2, 1, 128, "e4m3", W.SWIGLU, 0.0, 0),
    (64, 256, 128, 3, 2, 0, 64, "bf16", W.SWIGLU, 0.0, 20),
    (33, 136, 72, 16, 4, 1, 64, "bf16", W.RELU, 0.0, 0),
    (150, 64, 48, 4, 1, 1, 32, "e4m3", W.SWIGLU, 0.0, 5)])
def test_expert_ffn(N, d, F, E, k, S, group, kind, act, clamp, drop):
    cfg, gu, guv, dn, dnv, x, xs, xv, off, tok = ffn_case(N, d, F, E, k, S, group, kind, act, clamp,
                                                          seed=N, drop=drop)
    ye = torch.full((N * k + S * N, d), -3.0, dtype=torch.bfloat16, device="cuda")
    ws = nat.alloc_workspace(cfg)
    nat.moe_expert_ffn_w4(cfg, x=x, x_scale=xs, offsets=dev(off), row_token=dev(tok), W_gu=gu,
                          W_down=dn, ye=ye, ws=ws)
    check_status(ws)
    assert nat.moe_last_launch_count() == 2
    got = f64(ye)
    for e in range(E + S):
        s = slice(off[e], off[e + 1]) if e < E else slice(N * k, N * k + N)
        rows = xv[tok[s]] if e < E else xv
        y, tol = ffn_expect(guv[e], dnv[e], rows, d, F, group, act, clamp)
        assert within(got[s], y, tol + (np.abs(y) + tol) * BF)
    assert (got[off[E]:N * k] == -3).all()


@pytest.mark.parametrize("name,N,kw", [("mixtral-n16", 16, dict(d=256, F=512)),
                                       ("dsv3-n64", 5, dict(d=384, E=16, k=4, F=256)),
                                       ("v41flash-n64", 130, dict(d=256, E=12, k=3, F=136)),
                                       ("v41flash-n64", 1, dict(d=256, E=12, k=3, F=136))])
@pytest.mark.parametrize("rows8", [False, True])
def test_layer_with_norm(name, N, kw, rows8):
    """The operators together as a decode step uses them: residual norm (with the 8-bit rows),
    4-bit layer, balance loss on its logits; against the oracle on the quantised weights."""
    shape = W.PRESETS[name].replace(N=N, **kw)
    t = W.make_inputs(shape, device="cuda")
    gu = nat.W4Matrix.quantize(t["W_gu"], parts=2, group=64)
    dn = nat.W4Matrix.quantize(t["W_down"], group=64)
    C = O.capacity(N, shape.k, shape.E, 1.25) if N > 100 else 0
    cfg = nat.config_from_shape(shape, capacity=C)
    ws = nat.alloc_workspace(cfg)
    d, E, k = shape.d, shape.E, shape.k
    res = torch.randn(N, d, device="cuda").to(torch.bfloat16)
    x, y = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    x8 = torch.empty(N, d, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(N, -(-d // 128), device="cuda")
    nat.moe_rms_norm(x=t["x"], residual=res, y=x, residual_out=res, y8=x8, y8_scale=sc)
    ro = dict(logits=torch.empty(N, E, device="cuda"),
              ids=torch.empty(N, k, dtype=torch.int32, device="cuda"),
              gates=torch.empty(N, k, device="cuda"),
              counts=torch.empty(E, dtype=torch.int32, device="cuda"),
              drop_mask=torch.empty(N, k, dtype=torch.uint8, device="cuda"))
    nat.moe_forward_w4(cfg, x=x, x8=x8 if rows8 else None, x8_scale=sc if rows8 else None, W_g=t["W_g"],
                       W_gu=gu, W_down=dn, y=y, bias=t.get("bias"), modality=t.get("modality"),
                       route_out=ro, ws=ws)
    check_status(ws)
    ids, gates = host(ro["ids"]), host(ro["gates"]).astype(np.float64)
    want = O.dispatch(ids, E, C)
    np.testing.assert_array_equal(host(ro["counts"]), want["counts"])
    np.testing.assert_array_equal(host(ro["drop_mask"]), want["drop_mask"])
    guv = R.w4_values(gu.q.cpu().numpy(), f64(gu.scale), shape.F, d, 64)
    dnv = R.w4_values(dn.q.cpu().numpy(), f64(dn.scale), d, shape.F, 64)
    xv = f64(x8) * np.repeat(f64(sc), 128, 1)[:, :d] if rows8 else f64(x)
    ref = np.zeros((N, d))
    for tok in range(N):
        slots = [(ids[tok, j], gates[tok, j]) for j in range(k) if not want["drop_mask"][tok, j]]
        for e, g in slots + [(E, 1.0)] * shape.n_shared:
            h = R.swiglu(guv[e, 0] @ xv[tok], guv[e, 1] @ xv[tok], shape.clamp)
            ref[tok] += g * (dnv[e, 0] @ h)
    assert_close_layer(host(y), ref)
    # the router's loss on the same batch counts what the router demanded
    out = dict(loss=torch.empty(1, device="cuda"), counts=torch.empty(E, dtype=torch.int32, device="cuda"))
    nat.moe_balance_loss(cfg, logits=ro["logits"], ids=ro["ids"], alpha=1.0, ws=ws, **out)
    np.testing.assert_array_equal(host(out["counts"]), want["demand"])
    check_status(ws)


def test_layer_follows_the_bf16_layer():
    """With weights that 4 bits hold exactly, the two layers route alike and agree."""
    shape = W.PRESETS["dsv3-n64"].replace(N=24, d=256, E=8, k=2, F=128)
    t = W.make_inputs(shape, device="cuda")
    for n in ("W_gu", "W_down"):
        codes = torch.randint(-7, 8, t[n].shape, device="cuda").to(torch.bfloat16)
        codes[..., ::32] = 7                   # every group's largest magnitude is 7 steps
        t[n] = codes * 2.0 ** -7
    gu = nat.W4Matrix.quantize(t["W_gu"], parts=2, group=32)
    dn = nat.W4Matrix.quantize(t["W_down"], group=32)
    cfg = nat.config_from_shape(shape)
    ws = nat.alloc_workspace(cfg)
    y, y4 = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    ro = [dict(ids=torch.empty(24, 2, dtype=torch.int32, device="cuda")) for _ in range(2)]
    nat.moe_forward(cfg, x=t["x"], W_g=t["W_g"], W_gu=t["W_gu"], W_down=t["W_down"], y=y, bias=t["bias"],
                    route_out=ro[0], ws=ws)
    nat.moe_forward_w4(cfg, x=t["x"], W_g=t["W_g"], W_gu=gu, W_down=dn, y=y4, bias=t["bias"],
                       route_out=ro[1], ws=ws)
    check_status(ws)
    assert torch.equal(ro[0]["ids"], ro[1]["ids"])
    assert_close_layer(host(y4), host(y).astype(np.float64))


def test_same_bits_in_graphs_and_on_streams():
    cfg, gu, _, dn, _, x, xs, _, off, tok = ffn_case(33, 512, 256, 6, 2, 1, 64, "e4m3", seed=3)
    args = dict(x=x, x_scale=xs, offsets=dev(off), row_token=dev(tok), W_gu=gu, W_down=dn)
    ws = nat.alloc_workspace(cfg)
    ye = torch.empty(99, 512, dtype=torch.bfloat16, device="cuda")
    nat.moe_expert_ffn_w4(cfg, ye=ye, ws=ws, **args)
    got = torch.zeros_like(ye)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nat.moe_expert_ffn_w4(cfg, ye=got, ws=ws, **args)
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), ye.view(torch.int16))
    ws2 = nat.alloc_workspace(cfg)
    torch.cuda.synchronize()
    two = [torch.zeros_like(ye) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, o, w in zip(streams, two, (ws, ws2)):           # two calls at once, a workspace each
        nat.moe_expert_ffn_w4(cfg, ye=o, ws=w, stream=s, **args)
    torch.cuda.synchronize()
    for o in two:
        assert torch.equal(o.view(torch.int16), ye.view(torch.int16))


def test_empty_batch():
    cfg = nat.make_config(0, 64, 4, 2, 64)
    gu, _ = make_w(4, 2, 64, 64, 64, seed=1)
    dn, _ = make_w(4, 1, 64, 64, 64, seed=2)
    ws = nat.alloc_workspace(cfg)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    nat.moe_expert_ffn_w4(cfg, x=e, offsets=torch.zeros(5, dtype=torch.int32, device="cuda"),
                          row_token=torch.empty(0, dtype=torch.int32, device="cuda"), W_gu=gu,
                          W_down=dn, ye=e, ws=ws)
    one, _ = make_w(1, 1, 64, 64, 64, seed=3)
    nat.moe_w4_matmul(one, x=e, out=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))


def values_on_gpu(w):
    """R.w4_values in float64 on the device, for the large shapes."""
    r, c = torch.arange(w.rows, device="cuda")[:, None], torch.arange(w.cols, device="cuda")[None]
    byte = 16 * (4 * (r % 8) + c % 32 // 8) + 4 * (2 * (c % 64 // 32) + c % 8 // 4) + 2 * (c % 2) + c % 4 // 2
    both = w.q[:, :, r // 16, c // 64, byte]
    code = torch.where(r % 16 < 8, both & 15, both >> 4).double()
    return (code - 8) * w.scale[:, :, r // 16, c // w.group, r % 8, r % 16 // 8].double()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,rows,cols,parts,group", [
    (1, 7176, 2056, 2, 128),      # whole rounds of items and a cut rest
    (3, 2064, 14336, 1, 64),      # few items, many columns: clusters
    (9, 520, 8200, 1, 32),        # a cluster whose last run is ragged
    (16, 4104, 1800, 2, 64),
    (33, 1032, 7176, 1, 128),     # three tiles
    (48, 264, 4360, 2, 32),
    (200, 512, 1160, 1, 64),      # thirteen tiles
    (2, 48, 264, 1, 32)])
def test_large_shapes(n, rows, cols, parts, group, kind):
    g = torch.Generator(device="cuda").manual_seed(rows)
    shape = (1, parts, -(-rows // 16))
    q = torch.randint(0, 256, shape + (-(-cols // 64), 512), generator=g, device="cuda", dtype=torch.uint8)
    sc = (torch.rand(shape + (-(-cols // group), 8, 2), generator=g, device="cuda") * 0.02 + 0.01).to(torch.bfloat16)
    w = nat.W4Matrix(q, sc, rows=rows, cols=cols, group=group)
    x, xs, xg, xv = make_x(n, cols, kind, seed=n)
    wv, xt = values_on_gpu(w)[0], torch.from_numpy(xv).cuda()
    z = [xt @ m.t() for m in wv]
    t = [(group / 16 + (cols / group + 12 + 8) / 4) * 2.0 ** -22 * (xt.abs() @ m.abs().t()) for m in wv]
    if parts == 2:
        s = z[0] * torch.sigmoid(z[0])
        v = s * z[1]
        tol = 1.1 * (z[1].abs() + t[1]) * t[0] + (s.abs() + t[0]) * t[1] + 2.0 ** -20 * v.abs()
    else:
        v, tol = z[0], t[0]
    out = [torch.empty(n, rows, device="cuda") for _ in range(2)]
    for o in out:
        nat.moe_w4_matmul(w, x=x, x_scale=xs, x_group=xg, out=o)
    assert torch.equal(out[0].view(torch.int32), out[1].view(torch.int32))      # the same bits again
    assert within(f64(out[0]), v.cpu().numpy(), (tol + v.abs() * 2.0 ** -24 + 1e-37).cpu().numpy())


@pytest.mark.parametrize("N,E,k,S,C", [(1, 64, 8, 1, 0), (24, 40, 4, 1, 0), (90, 5, 2, 0, 30), (300, 9, 2, 1, 0)])
def test_large_ffn_against_the_bf16_layer(N, E, k, S, C):
    """Many groups, tiles and units: the 4-bit experts against the bf16 experts on the values that
    the codes stand for (those of multiples of 2^-7 up to 7 are bf16 numbers)."""
    d, F = 1032, 520
    g = torch.Generator(device="cuda").manual_seed(N)
    codes = [torch.randint(-7, 8, s, generator=g, device="cuda").to(torch.bfloat16)
             for s in ((E + S, 2 * F, d), (E + S, d, F))]
    for c in codes:
        c[..., ::32] = 7
    Wgu, Wdn = (c * 2.0 ** -7 for c in codes)
    cfg = nat.make_config(N, d, E, k, F, n_shared=S, capacity=C)
    x = torch.randn(N, d, generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn(N, E, generator=g, device="cuda")
    ws = nat.alloc_workspace(cfg)
    ids, gates = torch.empty(N, k, dtype=torch.int32, device="cuda"), torch.empty(N, k, device="cuda")
    counts, demand = (torch.empty(E, dtype=torch.int32, device="cuda") for _ in range(2))
    drop = torch.empty(N, k, dtype=torch.uint8, device="cuda")
    nat.moe_route(cfg, logits=z, ids=ids, gates=gates, counts=counts, demand=demand, drop_mask=drop, ws=ws)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    tok, slot = torch.full((N * k,), -7, dtype=torch.int32, device="cuda"), torch.empty(N, k, dtype=torch.int32, device="cuda")
    xp = torch.empty(N * k, d, dtype=torch.bfloat16, device="cuda")
    nat.moe_permute(cfg, ids=ids, drop_mask=drop, x=x, offsets=off, row_token=tok, slot_row=slot, xp=xp, ws=ws)
    ye, y4 = (torch.zeros(N * k + S * N, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nat.moe_expert_ffn(cfg, xp=xp, offsets=off, x=x, W_gu=Wgu, W_down=Wdn, ye=ye, ws=ws)
    nat.moe_expert_ffn_w4(cfg, x=x, offsets=off, row_token=tok, W_gu=nat.W4Matrix.quantize(Wgu, parts=2, group=32),
                          W_down=nat.W4Matrix.quantize(Wdn, group=32), ye=y4, ws=ws)
    check_status(ws)
    assert_close_layer(host(y4), host(ye).astype(np.float64))


def test_small_and_large_numbers():
    w, wv = make_w(1, 1, 64, 512, 128, seed=21)
    x, _, _, xv = make_x(5, 512, "bf16", seed=22)
    out = torch.empty(5, 64, device="cuda")
    for e in (-45, 40, 58):
        nat.moe_w4_matmul(w, x=(x.double() * 2.0 ** e).to(torch.bfloat16), out=out)
        v, tol = expect(wv[0], xv * 2.0 ** e, 512, 128)
        assert within(f64(out), v, tol + np.abs(v) * 2.0 ** -24)
    nat.moe_w4_matmul(w, x=(x.double() * 2.0 ** -100).to(torch.bfloat16), out=out)
    assert np.abs(f64(out)).max() <= 2.0 ** -75              # nothing but what is left of 2^-100
    nat.moe_w4_matmul(w, x=torch.full_like(x, 2.0 ** 63), out=out)
    assert not torch.isfinite(out).any()


def test_layer_class():
    shape = W.PRESETS["dsv3-n64"].replace(N=20, d=256, E=8, k=2, F=128)
    t = W.make_inputs(shape, device="cuda")
    from mixture_experts_layer_50_b200 import MoELayer, W4MoELayer
    layer = MoELayer.from_workload(shape, t)
    w4 = W4MoELayer.from_layer(layer, group=32)
    y = w4.forward(t["x"])
    want = torch.empty_like(y)
    nat.moe_forward_w4(w4.config(20), x=t["x"], W_g=t["W_g"], W_gu=w4.W_gu, W_down=w4.W_down, y=want, bias=t["bias"],
                       ws=w4.ws)
    assert torch.equal(y, want) and w4.check_status() == 0
    # 4 bits: the largest of 32 normal weights is 7 steps, some 2.2 sigma, so a step is 0.31 sigma
    # and its rounding 0.09 sigma rms; three matrices in a product: 16 %
    assert np.sqrt(((host(y) - host(layer.forward(t["x"]))) ** 2).mean()) <= 0.2 * np.sqrt((host(y) ** 2).mean())
    got = torch.empty_like(y)
    for _ in range(2):
        assert torch.equal(w4.forward_graphed(t["x"], got), want)
    xh, yh = t["x"].cpu().pin_memory(), torch.empty(20, 256, dtype=torch.bfloat16).pin_memory()
    assert torch.equal(w4.forward_host(xh, yh), want.cpu())
    res = torch.randn(20, 256, device="cuda").to(torch.bfloat16)
    yn, total = w4.forward_normed(t["x"], res, weight=torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(total, (t["x"].float() + res.float()).to(torch.bfloat16))
    h = torch.empty_like(y)
    nat.moe_rms_norm(x=t["x"], residual=res, y=h)
    # the same rows in bf16: e4m3 is off by 2^-4 at most, 2.6 % rms, in both factors of SwiGLU
    bf = w4.forward(h)
    assert np.sqrt(((host(yn) - host(bf)) ** 2).mean()) <= 0.1 * np.sqrt((host(bf) ** 2).mean())
    with pytest.raises(ValueError):
        w4.forward(torch.empty(21, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        W4MoELayer.from_layer(MoELayer.from_workload(shape, t, overflow="reroute"))


def test_two_graphs_share_a_workspace():
    cases = [ffn_case(n, 256, 128, 5, 2, 1, 64, "bf16", seed=n) for n in (7, 30)]
    ws = nat.alloc_workspace(cases[1][0])
    graphs = []
    for cfg, gu, _, dn, _, x, xs, _, off, tok in cases:
        a = dict(x=x, x_scale=xs, offsets=dev(off), row_token=dev(tok), W_gu=gu, W_down=dn)
        want = torch.empty(cfg.N * 3, 256, dtype=torch.bfloat16, device="cuda")
        nat.moe_expert_ffn_w4(cfg, ye=want, ws=nat.alloc_workspace(cfg), **a)
        got, g = torch.zeros_like(want), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            nat.moe_expert_ffn_w4(cfg, ye=got, ws=ws, **a)
        graphs.append((g, got, want, a))
    for _ in range(3):
        for g, got, _, _ in graphs:
            got.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in graphs:
        assert torch.equal(got, want)


def test_layer_on_another_stream_takes_its_own_memory():
    shape = W.PRESETS["dsv3-n64"].replace(N=20, d=256, E=8, k=2, F=128)
    t = W.make_inputs(shape, device="cuda")
    from mixture_experts_layer_50_b200 import MoELayer, W4MoELayer
    w4 = W4MoELayer.from_layer(MoELayer.from_workload(shape, t))
    want, total = w4.forward_normed(t["x"], t["x"])
    plain = w4.forward(t["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # memory that the current stream has given back, and may still be writing
    freed = [torch.empty_like(want) for _ in range(6)]
    places = {f.data_ptr() for f in freed}
    del freed
    got, got_total = w4.forward_normed(t["x"], t["x"], stream=side)
    got_plain = w4.forward(t["x"], stream=side)
    torch.cuda.synchronize()
    assert not places & {g.data_ptr() for g in (got, got_total, got_plain)}
    assert torch.equal(got, want) and torch.equal(got_total, total) and torch.equal(got_plain, plain)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,rows,cols,parts", [
    (16, 7176, 1288, 2), (3, 1544, 5128, 2),                            # clusters of 3
    (3, 520, 7176, 1),                                                  # 4
    (7, 2568, 7176, 2), (3, 1032, 14344, 2),                            # 5
    (16, 4104, 5128, 2), (7, 1544, 5128, 2), (3, 520, 5128, 1),         # 6
    (16, 3592, 5128, 2),                                                # 7
    (3, 520, 14344, 1), (31, 7176, 1288, 2)])                           # 8; 2
def test_clusters_of_every_size(n, rows, cols, parts, kind):
    test_large_shapes(n, rows, cols, parts, 64, kind)


@pytest.mark.parametrize("sizes", [[20, 3, 40, 0, 16, 17, 1, 8, 9, 33] * 5, [16] * 40 + [1] * 60, [5] * 30 + [31] * 20])
def test_costly_and_cheap_tiles_in_rounds(sizes):
    # more items than blocks: every row of every group still has its own expert's outputs
    E, cols, rows, n = len(sizes), 264, 1032, sum(sizes)
    w, wv = make_w(E, 1, rows, cols, 64, seed=E)
    x, xs, xg, xv = make_x(n, cols, "bf16", seed=n)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    out = torch.full((n + 2, rows), 7.0, device="cuda")
    nat.moe_w4_matmul(w, x=torch.cat([x, x[:2]]), offsets=dev(off), out=out)
    assert bool((out[n:] == 7.0).all())
    got = f64(out)
    for e in range(E):
        a, b = off[e], off[e + 1]
        v, tol = expect(wv[e], xv[a:b], cols, 64)
        assert within(got[a:b], v, tol + np.abs(v) * 2.0 ** -24 + 1e-37), e
