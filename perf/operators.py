"""Cases of the operators around a layer's router and experts: the residual RMS norm that feeds
them (with an 8-bit output), the experts' products with 4-bit weights, and the router's balance
loss with its gradient.

``run(state)`` computes an operator in plain torch operations (``own`` false) or through the
package's entry points (``own`` true); ``exact`` is the definition in float64.

4-bit matrices are stored as the package stores them.  A matrix of ``rows`` x ``cols`` is cut
into blocks of 16 rows and 64 columns; a block is 512 bytes, 16 for each of 32 lanes.  Lane
4 g + t holds rows g and g + 8 and, of each half h of the columns, columns 32 h + 8 t ... + 7:
byte 4 (2 h + j) + 2 e + p has the codes of column 32 h + 8 t + 4 j + 2 p + e, row g in its low
and row g + 8 in its high four bits.  A code c stands for (c - 8) times the scale of its row and
group of columns; the scales of a block of rows are [groups][8][2] (rows g and g + 8), bf16.
"""
import math

import torch

own = False

NORM_EPS = 1e-6


# ---- the cases ---------------------------------------------------------------------------
def listed():
    return [
        # one token enters a decode step of the 7168-wide layer: latency
        dict(name="norm 1x7168", op="norm", N=1, d=7168, dtype="bf16", residual=True, bits8=True, group=128),
        # a ragged batch in 32 bits, one 8-bit scale for a row
        dict(name="norm 3001x1408 f32", op="norm", N=3001, d=1408, dtype="f32", residual=False, bits8=True, group=0),
        # a prefill batch of the 5120-wide layer
        dict(name="norm 16384x5120", op="norm", N=16384, d=5120, dtype="bf16", residual=True, bits8=True, group=128),
        # one token through a gate/up pair of the 4096-wide layer: the smallest product
        dict(name="w4 1x4096 swiglu", op="w4", R=1, cols=4096, rows=14336, parts=2, group=128, x8=False, x_group=128, out="bf16"),
        # a ragged decode batch of 8-bit rows through a down projection, fine groups, 32-bit output
        dict(name="w4 33x14336 8-bit", op="w4", R=33, cols=14336, rows=4096, parts=1, group=32, x8=True, x_group=0, out="f32"),
        # one token, top-8 of the 32 experts that one of eight ranks holds, and the shared expert
        dict(name="ffn 1 token 7168", op="ffn", N=1, d=7168, F=2048, E=32, k=8, shared=1, group=128, clamp=0.0, x8=False),
        # a small decode batch on all eight experts of the 4096-wide layer
        dict(name="ffn 16 tokens 4096", op="ffn", N=16, d=4096, F=14336, E=8, k=2, shared=0, group=128, clamp=0.0, x8=False),
        # a decode batch of 8-bit rows on a rank's 32 experts and the shared expert
        dict(name="ffn 64 tokens 7168 8-bit", op="ffn", N=64, d=7168, F=2048, E=32, k=8, shared=1, group=128, clamp=0.0, x8=True),
        # a ragged decode batch, clipped SwiGLU, groups of 64
        dict(name="ffn 37 tokens 5120", op="ffn", N=37, d=5120, F=2304, E=48, k=6, shared=1, group=64, clamp=10.0, x8=False),
        # a small batch of a fine-tuning step, sigmoid scores: latency
        dict(name="balance 64x256", op="balance", N=64, E=256, k=8, score="sigmoid", masked=False),
        # a training batch on eight experts, an odd number of tokens, no padding
        dict(name="balance 8191x8", op="balance", N=8191, E=8, k=2, score="softmax", masked=False),
        # a padded training batch on 384 experts
        dict(name="balance 16384x384", op="balance", N=16384, E=384, k=6, score="softmax", masked=True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "w4", "ffn", "balance"])
    if op == "norm":
        f32 = rng.random() < 0.3
        d = _log(rng, 64, 8192, 4 if f32 else 8)
        N = _log(rng, 1, min(16384, 16384 * 5120 // (d * (2 if f32 else 1))))
        return dict(op="norm", N=N, d=d, dtype="f32" if f32 else "bf16", residual=rng.random() < 0.6,
                    bits8=rng.random() < 0.7, group=rng.choice([128, 128, 0]))
    if op == "w4":
        parts = rng.choice([1, 2])
        cols = _log(rng, 256, 14336, 8)
        rows = _log(rng, 256, 14336, 8)
        return dict(op="w4", R=_log(rng, 1, 48), cols=cols, rows=rows, parts=parts, group=rng.choice([32, 64, 128]),
                    x8=rng.random() < 0.5, x_group=rng.choice([128, 0]), out="bf16" if parts == 2 else rng.choice(["bf16", "f32"]))
    if op == "ffn":
        d = _log(rng, 1024, 7168, 8)
        F = _log(rng, 512, 8192, 8)
        E = min(48, max(4, int(1.3e9 / (3 * d * F))))
        E = _log(rng, 4, max(4, E))
        k, S = rng.randint(1, min(8, E)), rng.randint(0, 1)
        N = _log(rng, 1, min(96, int(5e10 / (6 * (k + S) * d * F))))
        return dict(op="ffn", N=N, d=d, F=F, E=E, k=k, shared=S, group=rng.choice([32, 64, 128]), clamp=rng.choice([0.0, 10.0]), x8=rng.random() < 0.5)
    E = _log(rng, 4, 384)
    return dict(op="balance", N=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E // 2)),
                score=rng.choice(["softmax", "sigmoid"]), masked=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------
def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _w4(gen, mats, parts, rows, cols, group):
    """Codes of normally distributed weights and their scales, in the stored layout."""
    rb, ku, ng = -(-rows // 16), -(-cols // 64), -(-cols // group)
    q = torch.empty((mats, parts, rb, ku, 512), dtype=torch.uint8, device=gen.device)
    for m in range(mats):
        v = torch.randn((2, parts, rb, ku, 512), generator=gen, device=gen.device)
        c = v.mul_(2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        q[m] = c[0] | (c[1] << 4)
    s = torch.rand((mats, parts, rb, ng, 8, 2), generator=gen, device=gen.device) * 0.3 + 0.85
    return q, (s * (0.02 / 2.6)).to(torch.bfloat16)


def _rows8(x, group):
    """8-bit rows and their scales, as a quantising producer hands them over."""
    n, d = x.shape
    g = group or d
    ng = -(-d // g)
    p = torch.nn.functional.pad(x, (0, ng * g - d)).view(n, ng, g)
    s = p.abs().amax(2) / 448
    return (p / s[:, :, None]).reshape(n, ng * g)[:, :d].contiguous().to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = _dev()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    randn = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "norm":
        N, d = case["N"], case["d"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # a few channels are much larger than the others, as in a trained residual stream
        big = 1 + 7 * (torch.rand(d, generator=gen, device=dev) < 0.01)
        s["x"] = randn(N, d).to(dt)
        s["residual"] = (randn(N, d) * 2 * big).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * randn(d)).to(dt)
        s["y"] = torch.empty_like(s["x"])
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["bits8"]:
            ng = -(-d // case["group"]) if case["group"] else 1
            s["y8"] = torch.empty((N, d), dtype=torch.float8_e4m3fn, device=dev)
            s["y8_scale"] = torch.empty((N, ng), device=dev)
    elif case["op"] == "w4":
        R, cols, rows, parts = case["R"], case["cols"], case["rows"], case["parts"]
        s["q"], s["scale"] = _w4(gen, 1, parts, rows, cols, case["group"])
        x = randn(R, cols)
        s["x"], s["x_scale"] = _rows8(x, case["x_group"]) if case["x8"] else (x.to(torch.bfloat16), None)
        s["out"] = torch.empty((R, rows), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=dev)
    elif case["op"] == "ffn":
        N, d, F, E, k, S = (case[n] for n in ("N", "d", "F", "E", "k", "shared"))
        s["q_gu"], s["s_gu"] = _w4(gen, E + S, 2, F, d, case["group"])
        s["q_dn"], s["s_dn"] = _w4(gen, E + S, 1, d, F, case["group"])
        x = randn(N, d)
        s["x"], s["x_scale"] = _rows8(x, 128) if case["x8"] else (x.to(torch.bfloat16), None)
        # the batch's routing: skewed experts, k different ones a token, in token order
        score = randn(N, E) + 0.5 * randn(E)
        ids = score.topk(k, dim=1).indices
        chosen = torch.zeros((E, N), dtype=torch.bool, device=dev)
        chosen[ids.reshape(-1), torch.arange(N, device=dev).repeat_interleave(k)] = True
        where = chosen.nonzero()
        s["row_token"] = where[:, 1].to(torch.int32).contiguous()
        counts = chosen.sum(1)
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["most"] = int(counts.max())
        s["ye"] = torch.zeros((N * k + S * N, d), dtype=torch.bfloat16, device=dev)
    else:
        N, E, k = case["N"], case["E"], case["k"]
        s["logits"] = randn(N, E) * 1.5 + randn(E) * 0.7
        s["ids"] = s["logits"].topk(k, dim=1).indices.to(torch.int32)
        if case["masked"]:
            # the batch's sequences fill 60 to 100 % of their places; padding holds anything
            n = torch.rand(-(-N // 512), generator=gen, device=dev) * 0.4 + 0.6
            place = torch.arange(N, device=dev)
            s["mask"] = (place % 512 < (n * 512)[place // 512]).to(torch.uint8)
            s["logits"][s["mask"] == 0] = float("nan")
        else:
            s["mask"] = None
        s["alpha"] = 0.01
        for name, shape, dt in (("loss", 1, torch.float32), ("counts", E, torch.int32), ("P", E, torch.float32)):
            s[name] = torch.empty(shape, dtype=dt, device=dev)
        s["dlogits"] = torch.empty((N, E), device=dev)
    return s


# ---- one pass ----------------------------------------------------------------------------
def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_norm(s):
    case = s["case"]
    if own:
        from mixture_experts_layer_50_b200 import moe_rms_norm
        moe_rms_norm(x=s["x"], residual=s["residual"], weight=s["weight"], eps=NORM_EPS, y=s["y"],
                     residual_out=s["residual_out"], y8=s.get("y8"), y8_scale=s.get("y8_scale"), group=case["group"])
        return {n: s[n] for n in ("y", "residual_out", "y8", "y8_scale") if s.get(n) is not None}
    dt = s["x"].dtype
    v = s["x"].float()
    out = {}
    if s["residual"] is not None:
        v = v + s["residual"].float()
        out["residual_out"] = v.to(dt)
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + NORM_EPS) * s["weight"].float()
    out["y"] = y.to(dt)
    if case["bits8"]:
        n, d = y.shape
        g = case["group"] or d
        ng = -(-d // g)
        p = torch.nn.functional.pad(y, (0, ng * g - d)).view(n, ng, g)
        sc = p.abs().amax(2) / 448
        v8 = torch.where(sc[:, :, None] == 0, p, p / sc[:, :, None]).reshape(n, ng * g)[:, :d]
        out["y8"], out["y8_scale"] = v8.contiguous().to(torch.float8_e4m3fn), sc
    return out


def _plain_w4(q, scale, rows, cols, group):
    """The matrices [mats, parts, rows, cols] that codes and scales stand for, in 32 bits."""
    m, p, rb, ku = q.shape[:4]
    c = torch.stack((q & 15, q >> 4), -1).view(m, p, rb, ku, 8, 4, 2, 2, 2, 2, 2)  # g t h j e p r
    c = c.permute(0, 1, 2, 10, 4, 3, 6, 5, 7, 9, 8).reshape(m, p, rb * 16, ku * 64)[:, :, :rows, :cols]
    s = scale.permute(0, 1, 2, 5, 4, 3).reshape(m, p, rb * 16, -1)[:, :, :rows]
    return (c.float() - 8) * s.float().repeat_interleave(group, 3)[..., :cols]


def _plain_rows(x, x_scale, group):
    v = x.float()
    if x_scale is not None:
        v = v * (x_scale.repeat_interleave(group, 1)[:, :v.shape[1]] if group else x_scale)
    return v


def _plain_swiglu(z, clamp):
    """z [..., 2, rows, columns of rows' products]: SiLU(gate) * up."""
    gate, up = z.unbind(-3)
    if clamp > 0:
        gate, up = gate.clamp(-clamp, clamp), up.clamp(-clamp, clamp)
    return gate * torch.sigmoid(gate) * up


def _run_w4(s):
    case = s["case"]
    if own:
        from mixture_experts_layer_50_b200 import W4Matrix, moe_w4_matmul
        if "w" not in s:
            s["w"] = W4Matrix(s["q"], s["scale"], rows=case["rows"], cols=case["cols"], group=case["group"])
        moe_w4_matmul(s["w"], x=s["x"], x_scale=s["x_scale"], x_group=case["x_group"], out=s["out"])
        return s["out"]
    w = _plain_w4(s["q"], s["scale"], case["rows"], case["cols"], case["group"])[0]
    z = w @ _plain_rows(s["x"], s["x_scale"], case["x_group"]).t()
    z = _plain_swiglu(z, 0.0) if case["parts"] == 2 else z[0]
    return z.t().to(s["out"].dtype).contiguous()


def _run_ffn(s):
    case = s["case"]
    N, d, F, E, k, S = (case[n] for n in ("N", "d", "F", "E", "k", "shared"))
    if own:
        from mixture_experts_layer_50_b200 import W4Matrix, alloc_workspace, make_config, moe_expert_ffn_w4
        if "cfg" not in s:
            s["cfg"] = make_config(N, d, E, k, F, n_shared=S, clamp=case["clamp"])
            s["ws"] = alloc_workspace(s["cfg"])
            s["w_gu"] = W4Matrix(s["q_gu"], s["s_gu"], rows=F, cols=d, group=case["group"])
            s["w_dn"] = W4Matrix(s["q_dn"], s["s_dn"], rows=d, cols=F, group=case["group"])
        moe_expert_ffn_w4(s["cfg"], x=s["x"], x_scale=s["x_scale"], offsets=s["offsets"], row_token=s["row_token"],
                          W_gu=s["w_gu"], W_down=s["w_dn"], ye=s["ye"], ws=s["ws"])
        return s["ye"]
    hit = (s["offsets"][1:] > s["offsets"][:-1]).nonzero()[:, 0]  # the experts that have rows
    at = torch.zeros(E, dtype=torch.long, device=hit.device).index_put((hit,), torch.arange(len(hit), device=hit.device))
    if S:
        hit = torch.cat((hit, hit.new_full((1,), E)))
    wg = _plain_w4(s["q_gu"][hit], s["s_gu"][hit], F, d, case["group"])
    wd = _plain_w4(s["q_dn"][hit], s["s_dn"][hit], d, F, case["group"])[:, 0]
    x = _plain_rows(s["x"], s["x_scale"], 128)
    r = torch.arange(N * k, device=x.device, dtype=torch.int32)
    e = torch.searchsorted(s["offsets"], r, right=True) - 1
    c = r - s["offsets"][e]
    e, n = at[e], len(hit) - S
    xe = torch.zeros((n, s["most"], d), device=x.device)
    xe[e, c] = x[s["row_token"]]
    h = _plain_swiglu((wg[:n] @ xe.transpose(1, 2)[:, None]), case["clamp"])
    y = (wd[:n] @ h).transpose(1, 2)[e, c]
    if S:
        hs = _plain_swiglu(wg[n] @ x.t(), case["clamp"])
        y = torch.cat((y, (wd[n] @ hs).t()))
    return y.to(torch.bfloat16)


def _run_balance(s):
    case = s["case"]
    N, E, k = case["N"], case["E"], case["k"]
    if own:
        from mixture_experts_layer_50_b200 import alloc_workspace, make_config, moe_balance_loss
        if "cfg" not in s:
            s["cfg"] = make_config(N, 8, E, k, 8, score_fn=int(case["score"] == "sigmoid"))
            s["ws"] = alloc_workspace(s["cfg"])
        moe_balance_loss(s["cfg"], logits=s["logits"], ids=s["ids"], token_mask=s["mask"], alpha=s["alpha"],
                         loss=s["loss"], counts=s["counts"], P=s["P"], dlogits=s["dlogits"], ws=s["ws"])
        return {n: s[n] for n in ("loss", "counts", "P", "dlogits")}
    z, keep = s["logits"], s["mask"]
    if keep is not None:
        z = torch.where(keep[:, None] != 0, z, 0.0)
    if case["score"] == "softmax":
        a = torch.exp(z - z.amax(1, keepdim=True))
        slope = torch.ones_like(a)
    else:
        a = 1 / (1 + torch.exp(-z))
        slope = 1 / (1 + torch.exp(z))
    p = a / a.sum(1, keepdim=True)
    w = torch.ones(N, device=z.device) if keep is None else (keep != 0).float()
    n = w.double().sum().clamp(min=1)
    counts = torch.zeros(E, device=z.device, dtype=torch.float64)
    counts = counts.index_add(0, s["ids"].reshape(-1).long(), w.double().repeat_interleave(k))
    f = counts / (n * k)
    P = (p * w[:, None]).sum(0, dtype=torch.float64) / n
    loss = s["alpha"] * E * (f * P).sum()
    f0 = (f - 1 / E).float()  # the sum of p is 1, so any constant may be taken off f
    dz = (s["alpha"] * E / n).float() * (w[:, None] * p * slope * (f0 - (p * f0).sum(1, keepdim=True)))
    return {"loss": loss.float().reshape(1), "counts": counts.to(torch.int32), "P": P.float(), "dlogits": dz}


_RUN = {"norm": _run_norm, "w4": _run_w4, "ffn": _run_ffn, "balance": _run_balance}


# ---- what a pass cannot do without -------------------------------------------------------
def _w4_bytes(rows, cols, group):
    return rows * cols / 2 + rows * -(-cols // group) * 2


def work(case):
    if case["op"] == "norm":
        N, d, el = case["N"], case["d"], 4 if case["dtype"] == "f32" else 2
        b = N * d * el * (4 if case["residual"] else 2) + d * el
        if case["bits8"]:
            b += N * d + 4 * N * (-(-d // case["group"]) if case["group"] else 1)
        return {"bytes": b, "flops": 6 * N * d}
    if case["op"] == "w4":
        R, cols, rows, parts = case["R"], case["cols"], case["rows"], case["parts"]
        x = R * cols + 4 * R * (-(-cols // 128) if case["x_group"] else 1) if case["x8"] else 2 * R * cols
        return {"bytes": parts * _w4_bytes(rows, cols, case["group"]) + x + R * rows * (4 if case["out"] == "f32" else 2),
                "flops": 2 * R * cols * rows * parts}
    if case["op"] == "ffn":
        N, d, F, E, k, S = (case[n] for n in ("N", "d", "F", "E", "k", "shared"))
        # experts that a batch of N tokens reaches when its experts are spread evenly
        hit = k if N == 1 else E * (1 - (1 - k / E) ** N)
        per = 2 * _w4_bytes(F, d, case["group"]) + _w4_bytes(d, F, case["group"])
        rows = N * (k + S)
        x = N * d + 4 * N * -(-d // 128) if case["x8"] else 2 * N * d
        return {"bytes": (hit + S) * per + x + 4 * (N * k + E + 1) + 2 * rows * d, "flops": 6 * rows * d * F}
    N, E, k = case["N"], case["E"], case["k"]
    return {"bytes": 8 * N * E + 4 * N * k + (N if case["masked"] else 0) + 8 * E + 4, "flops": 10 * N * E}


# ---- the definitions in 64 bits ----------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + NORM_EPS) * s["weight"].double()
        out = {"y": y}
        if s["residual"] is not None:
            out["residual_out"] = v
        if case["bits8"]:
            parts = y.split(case["group"] or y.shape[1], 1)
            sc = [t.abs().max(1, keepdim=True).values / 448 for t in parts]
            out["y8"] = torch.cat([t / u for t, u in zip(parts, sc)], 1)
            out["y8_scale"] = torch.cat(sc, 1)
        return out
    if case["op"] == "w4":
        x = _exact_rows(s["x"], s["x_scale"], case["x_group"])
        w = [_exact_w4(s["q"][0, i], s["scale"][0, i], case["rows"], case["cols"], case["group"]) for i in range(case["parts"])]
        z = [x @ m.t() for m in w]
        return z[0] if case["parts"] == 1 else z[0] / (1 + torch.exp(-z[0])) * z[1]
    if case["op"] == "ffn":
        N, d, F, E, k, S = (case[n] for n in ("N", "d", "F", "E", "k", "shared"))
        x = _exact_rows(s["x"], s["x_scale"], 128)
        at, token = s["offsets"].tolist(), s["row_token"].long()
        rows = [(x[token[at[e]:at[e + 1]]], e) for e in range(E)] + [(x, E)] * S
        got = []
        for xe, e in rows:
            g, u = (xe @ _exact_w4(s["q_gu"][e, i], s["s_gu"][e, i], F, d, case["group"]).t() for i in (0, 1))
            if case["clamp"] > 0:
                g, u = (torch.clip(t, -case["clamp"], case["clamp"]) for t in (g, u))
            got.append((g / (1 + torch.exp(-g)) * u) @ _exact_w4(s["q_dn"][e, 0], s["s_dn"][e, 0], d, F, case["group"]).t())
        return torch.cat(got)
    E, k = case["E"], case["k"]
    live = torch.ones(case["N"], dtype=torch.bool, device=s["logits"].device) if s["mask"] is None else s["mask"] != 0
    z = s["logits"][live].double().requires_grad_()
    n = max(1, z.shape[0])
    counts = torch.bincount(s["ids"][live].reshape(-1).long(), minlength=E)
    p = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
    P = p.sum(0) / n
    loss = s["alpha"] * E * (counts.double() / (n * k) * P).sum()
    dz = torch.zeros(s["logits"].shape, dtype=torch.float64, device=z.device)
    dz[live] = torch.autograd.grad(loss, z)[0]
    return {"loss": loss.detach().reshape(1), "counts": None, "P": P.detach(), "dlogits": dz}


def _exact_rows(x, x_scale, group):
    v = x.double()
    if x_scale is None:
        return v
    return torch.cat([t * x_scale[:, i:i + 1].double() for i, t in enumerate(v.split(group or v.shape[1], 1))], 1)


def _exact_w4(q, scale, rows, cols, group):
    """One stored matrix by its definition: the code and the scale of every (row, column)."""
    r, c = torch.arange(rows, device=q.device)[:, None], torch.arange(cols, device=q.device)[None]
    byte = 16 * (4 * (r % 8) + c % 32 // 8) + 4 * (c % 64 // 32 * 2 + c % 8 // 4) + 2 * (c % 2) + c % 4 // 2
    both = q[r // 16, c // 64, byte]
    code = torch.where(r % 16 < 8, both & 15, both >> 4)
    return (code.double() - 8) * scale[r // 16, c // group, r % 8, r % 16 // 8].double()
