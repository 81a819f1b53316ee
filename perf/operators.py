"""Cases for measuring the router, the experts' products and the combine's backward pass.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()``
makes what a user's program holds before the call, and ``run()`` makes one pass:
through the library's operators where ``own`` is true, and through the same formulas
in elementary torch operations, in 32 bits and rounded once at the end, where it is
false. ``exact()`` states the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
NEAR = 4e-6  # choice scores closer than this (and not equal) may be ordered either way in 32 bits


def listed():
    return [
        # One token of a decoding user: the call's latency. DeepSeek-V3's router shape:
        # 256 experts in 8 groups, the best 4 groups kept, a balance bias on the choice.
        dict(name="route_one_token", op="route", T=1, E=256, k=8, scoring="sigmoid", biased=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5, dtype="f32", masked=False),
        # The same router over a prefill batch.
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, scoring="sigmoid", biased=True,
             groups=8, keep=4, group_score="top2", renorm=True, scale=2.5, dtype="f32", masked=False),
        # Softmax routing with experts masked out (capacity, dead experts), rows that
        # keep none, and lowest-value masks; an odd batch of bf16 logits.
        dict(name="route_softmax_masked", op="route", T=4097, E=64, k=6, scoring="softmax",
             biased=False, groups=1, keep=1, group_score="max", renorm=True, scale=1.0,
             dtype="bf16", masked=True),
        # The router's backward pass of a training step, an odd batch.
        dict(name="route_backward", op="route_bwd", T=16383, E=256, k=8, scoring="softmax",
             biased=False, groups=1, keep=1, group_score="max", renorm=True, scale=1.0,
             dtype="f32", masked=True),
        # Decode step: 128 tokens in the low-latency rectangles, a few rows per expert, so
        # every touched expert's e4m3 weights are read for them (gate and up, SwiGLU).
        dict(name="experts_fp8_decode", op="experts", T=128, E=256, k=8, K=7168, N=2048,
             act="swiglu", dtype="fp8", rect=128, bias=False, residual=False, preact=False),
        # Prefill over the expert-contiguous buffer of the same model shape.
        dict(name="experts_fp8_prefill", op="experts", T=8192, E=256, k=8, K=7168, N=2048,
             act="swiglu", dtype="fp8", rect=0, bias=False, residual=False, preact=False),
        # Training forward in bf16: bias, SwiGLU, and the pre-activations kept for backward.
        dict(name="experts_bf16_train", op="experts", T=4096, E=64, k=6, K=4096, N=2048,
             act="swiglu", dtype="bf16", rect=0, bias=True, residual=False, preact=True),
        # A small ragged batch: odd sizes, experts with few rows or none, the whole epilogue.
        dict(name="experts_bf16_ragged", op="experts", T=77, E=20, k=3, K=1000, N=1304,
             act="gelu", dtype="bf16", rect=0, bias=True, residual=True, preact=False),
        # Backward of the second product of the training layer, down to the gradient of
        # the pre-activations (SwiGLU), with the weights' and the bias's gradients.
        dict(name="experts_backward", op="experts_bwd", T=4096, E=64, k=6, K=2048, N=4096,
             act="swiglu"),
        # The same on a ragged batch with odd sizes and experts without rows.
        dict(name="experts_backward_ragged", op="experts_bwd", T=333, E=24, k=2, K=520, N=904,
             act="gelu"),
        # Backward of the combine over a prefill batch.
        dict(name="combine_backward", op="combine_bwd", T=8192, H=7168, k=8, drop=0.0),
        # The same for a small odd batch with dropped picks.
        dict(name="combine_backward_small", op="combine_bwd", T=129, H=1032, k=5, drop=0.1),
    ]


def _log_size(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))))
    v = max(lo, min(hi, v // step * step))
    return v + step if v in (1536, 3072) else v


def draw(rng):
    op = rng.choice(["route", "route_bwd", "experts", "experts", "experts_bwd", "combine_bwd"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log_size(rng, 8, 512 // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(12, E // groups * keep))
        scoring = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, T=_log_size(rng, 1, 16384), E=E, k=k, scoring=scoring,
                    biased=scoring == "sigmoid" and rng.random() < 0.7, groups=groups, keep=keep,
                    group_score=rng.choice(["max", "top2"]), renorm=k > 1 and rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.random() < 0.5)
    if op == "experts" and rng.random() < 0.5:
        E = _log_size(rng, 4, 128)
        T = _log_size(rng, 1, 4096)
        rect = rng.random() < 0.5 and T <= 512
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)),
                    K=_log_size(rng, 256, 7168, 128), N=_log_size(rng, 128, 2048, 128),
                    act=rng.choice(["swiglu", "swiglu", "none"]), dtype="fp8",
                    rect=T if rect else 0, bias=rng.random() < 0.3, residual=False, preact=False)
    if op == "experts":
        E = _log_size(rng, 1, 64)
        act = rng.choice(["swiglu", "gelu", "silu", "relu", "none"])
        return dict(op=op, T=_log_size(rng, 1, 4096), E=E, k=rng.randint(1, min(6, E)),
                    K=_log_size(rng, 64, 4096, 8), N=_log_size(rng, 64, 2048, 16 if act == "swiglu" else 8),
                    act=act, dtype="bf16", rect=0, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.3, preact=rng.random() < 0.5)
    if op == "experts_bwd":
        E = _log_size(rng, 1, 64)
        return dict(op=op, T=_log_size(rng, 1, 4096), E=E, k=rng.randint(1, min(6, E)),
                    K=_log_size(rng, 64, 2048, 16), N=_log_size(rng, 64, 4096, 8),
                    act=rng.choice(["swiglu", "gelu", "silu", "relu", "none"]))
    return dict(op=op, T=_log_size(rng, 1, 8192), H=_log_size(rng, 64, 7168, 8),
                k=rng.randint(1, 8), drop=rng.choice([0.0, 0.05]))


# ------------------------------------------------------------------------------- inputs
def _choice64(s, case):
    """Choice scores and group scores in 64 bits of logits s["logits"]."""
    l = s["logits"].double()
    live = l > -math.inf
    score = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    c = score + s["bias"].double() if case["biased"] else score
    c = torch.where(live, c, -math.inf)
    T, E = l.shape
    g = c.view(T, case["groups"], E // case["groups"])
    if case["group_score"] == "max" or g.shape[2] == 1:
        gs = g.amax(2)
    else:
        two = g.topk(2, 2).values
        gs = torch.where(two[..., 0] > -math.inf, two.clamp(min=-1e300).masked_fill(two == -math.inf, 0).sum(2), -math.inf)
    return score, c, gs


def _close_rows(v):
    """Rows of v with two values that differ by less than NEAR without being equal."""
    if v.shape[1] < 2:
        return torch.zeros(v.shape[0], dtype=torch.bool, device=v.device)
    v = torch.sort(v, dim=1, descending=True).values
    gap = v[:, :-1] - v[:, 1:]
    return ((gap > 0) & (gap < NEAR)).any(1)


def _route_logits(case, g, rows):
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    l = (1.5 * torch.randn(rows, case["E"], generator=g, device=DEV)).to(dt)
    if case["masked"]:
        u = torch.rand(rows, case["E"], generator=g, device=DEV)
        l = torch.where(u < 0.08, torch.tensor(-math.inf, dtype=dt, device=DEV), l)
        l = torch.where(u > 0.98, torch.tensor(torch.finfo(dt).min, dtype=dt, device=DEV), l)
        none = torch.rand(rows, 1, generator=g, device=DEV) < 0.02
        l = torch.where(none, torch.tensor(-math.inf, dtype=dt, device=DEV), l)
    return l


def _regions(case, g):
    """Rows per expert of uniform top-k routing, their starts, and the fullest expert's count."""
    T, E, k = case["T"], case["E"], case["k"]
    picks = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices
    count = torch.bincount(picks.reshape(-1), minlength=E)
    start = torch.cumsum(count, 0) - count
    return count.to(torch.int32), start.to(torch.int32), max(1, int(count.max()))


def _rows_fp8(x, block=128):
    """e4m3 rows and one fp32 scale per 128 columns (amax / 448)."""
    b = x.view(*x.shape[:-1], x.shape[-1] // block, block)
    amax = b.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (b / scale.unsqueeze(-1)).clamp_(-448, 448).to(torch.float8_e4m3fn).view(x.shape), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * std

    if case["op"] in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["biased"] else None
        s["logits"] = _route_logits(case, g, T)
        # Rows whose choice 32 bits cannot decide are drawn again: either order is right there.
        # Softmax without a bias chooses by the logits themselves and has no such rows, but
        # for groups scored by sums.
        for _ in range(12):
            score, c, gs = _choice64(s, case)
            bad = _close_rows(gs) if case["groups"] > 1 and case["keep"] < case["groups"] else \
                torch.zeros(T, dtype=torch.bool, device=DEV)
            if case["scoring"] == "sigmoid" or case["biased"]:
                top = torch.sort(c, dim=1, descending=True).values
                # with groups the picks can lie deep in the order
                bad |= _close_rows(top if case["groups"] > 1 and E <= 64 else top[:, : min(E, 4 * k + 1)])
            n = int(bad.sum())
            if n == 0:
                break
            s["logits"][bad] = _route_logits(case, g, n)
        s["topk_idx"] = torch.empty(T, k, dtype=torch.int64, device=DEV)
        s["topk_weights"] = torch.empty(T, k, device=DEV)
        if case["op"] == "route_bwd":
            s["topk_idx"] = _route_plain(s, case)[0]
            s["grad_weights"] = torch.randn(T, k, generator=g, device=DEV)
            s["grad_logits"] = torch.empty_like(s["logits"])
    elif case["op"] == "experts":
        E, K, N = case["E"], case["K"], case["N"]
        NW = 2 * N if case["act"] == "swiglu" else N
        s["count"], s["start"], s["most"] = _regions(case, g)
        M = case["T"] * case["k"]
        if case["dtype"] == "fp8":
            s["w"] = torch.empty(E, NW, K, dtype=torch.float8_e4m3fn, device=DEV)
            s["w_scale"] = torch.empty(E, NW // 128, K // 128, device=DEV)
            for e in range(E):  # weights in 128 x 128 blocks of one scale each
                b = torch.randn(NW // 128, 128, K // 128, 128, generator=g, device=DEV).div_(math.sqrt(K))
                s["w_scale"][e] = b.abs().amax((1, 3)) / 448.0
                s["w"][e] = b.div_(s["w_scale"][e][:, None, :, None]).clamp_(-448, 448).to(
                    torch.float8_e4m3fn).view(NW, K)
            lead = (E, case["rect"]) if case["rect"] else (M,)
            s["x"], s["x_scale"] = _rows_fp8(torch.randn(*lead, K, generator=g, device=DEV))
            if case["rect"]:
                s["x_scale"] = s["x_scale"].transpose(1, 2).contiguous()
        else:
            s["w"] = normal(E, NW, K, std=1 / math.sqrt(K))
            s["x"] = normal(M, K)
        lead = s["x"].shape[:-1]
        s["bias"] = 0.5 * torch.randn(E, NW, generator=g, device=DEV) if case["bias"] else None
        s["residual"] = normal(*lead, N) if case["residual"] else None
        s["y"] = torch.zeros(*lead, N, dtype=torch.bfloat16, device=DEV)
        s["z"] = torch.zeros(*lead, NW, dtype=torch.bfloat16, device=DEV) if case["preact"] else None
    elif case["op"] == "experts_bwd":
        E, K, N = case["E"], case["K"], case["N"]
        s["count"], s["start"], s["most"] = _regions(case, g)
        M = case["T"] * case["k"]
        s["w"] = normal(E, N, K, std=1 / math.sqrt(K))
        s["x"], s["dy"] = normal(M, K), normal(M, N)
        KZ = 2 * K if case["act"] == "swiglu" else K
        s["z"] = normal(M, KZ) if case["act"] != "none" else None
        s["dz"] = torch.zeros(M, KZ, dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
        s["db"] = torch.empty(E, N, device=DEV)
    else:
        T, H, k = case["T"], case["H"], case["k"]
        live = torch.rand(T, k, generator=g, device=DEV) >= case["drop"]
        slot = torch.randperm(T * k, generator=g, device=DEV).view(T, k).to(torch.int32)
        s["index"] = torch.where(live, slot, -1)
        s["weights"] = torch.where(live, torch.rand(T, k, generator=g, device=DEV), 0.0)
        s["eo"], s["dy"] = normal(T * k, H), normal(T, H)
        s["deo"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)
        s["dweights"] = torch.empty(T, k, device=DEV)
    return s


# ------------------------------------------------------------------------- plain forms
def _route_plain(s, case):
    l = s["logits"].float()
    T, E = l.shape
    G, k = case["groups"], case["k"]
    live = l > -math.inf
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        p = torch.where(live, torch.exp(l - torch.where(m > -math.inf, m, 0.0)), 0.0)
        score = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    if case["biased"]:
        c = score + s["bias"]
    else:  # a softmax is ordered as its logits are
        c = score if case["scoring"] == "sigmoid" else l
    c = torch.where(live, c, -math.inf)
    if G > 1:
        if case["group_score"] == "max" or E == G:
            gs = c.view(T, G, E // G).amax(2)
        else:
            by = score if case["scoring"] == "softmax" and not case["biased"] else c
            two = torch.where(live, by, -math.inf).view(T, G, E // G).sort(dim=2, descending=True).values[..., :2]
            gs = torch.where(two[..., 0] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2), -math.inf)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, : case["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = torch.where(kept.repeat_interleave(E // G, 1), c, -math.inf)
    top = c.sort(dim=1, descending=True, stable=True)
    ok = top.values[:, :k] > -math.inf
    idx = torch.where(ok, top.indices[:, :k], -1)
    w = torch.where(ok, score.gather(1, top.indices[:, :k]), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return idx, w * case["scale"]


def _route_grad(l, idx, gw, case):
    """Gradient of the logits, in the type of l."""
    live = l > -math.inf
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        p = torch.where(live, torch.exp(l - torch.where(m > -math.inf, m, 0.0)), 0.0)
        score = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    ok = idx >= 0
    at = idx.clamp(min=0)
    sel = torch.where(ok, score.gather(1, at), 0.0)
    gs = torch.where(ok, gw, 0.0) * case["scale"]
    if case["renorm"]:
        total = sel.sum(1, keepdim=True)
        inv = torch.where(total > 0, 1.0 / total, 0.0)
        apart = gs.unsqueeze(2) - gs.unsqueeze(1)  # g_j - g_i: a lone pick's gradient is exactly zero
        gs = torch.where(ok, (apart * (sel * inv).unsqueeze(1)).sum(2) * inv, 0.0)
    ds = torch.zeros_like(score).scatter_add_(1, at, gs)
    if case["scoring"] == "sigmoid":
        return ds * score * (1.0 - score)
    return score * (ds - (ds * score).sum(1, keepdim=True))


def _act(z, act):
    if act == "swiglu":
        a, b = z.chunk(2, -1)
        return a / (1.0 + torch.exp(-a)) * b
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z / math.sqrt(2.0)))
    return z.clamp(min=0.0) if act == "relu" else z


def _act_grad(d, z, act):
    """Gradient of the pre-activations from that of the activations."""
    if act == "none":
        return d
    if act == "relu":
        return torch.where(z > 0, d, 0.0)
    if act == "gelu":
        return d * (0.5 * (1.0 + torch.erf(z / math.sqrt(2.0))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    a, b = z.chunk(2, -1) if act == "swiglu" else (z, None)
    sg = 1.0 / (1.0 + torch.exp(-a))
    da = sg * (1.0 + a * (1.0 - sg))
    return d * da if b is None else torch.cat([d * b * da, d * a * sg], -1)


def _padded(s, rows):
    """Row numbers [E, most] of the experts' regions and which of them are real."""
    r = torch.arange(s["most"], device=DEV)
    real = r < s["count"].unsqueeze(1)
    return torch.where(real, s["start"].long().unsqueeze(1) + r, rows), real


def _gather(x, at):
    """Rows of x in 32 bits at the places `at`; the row past the last is zero."""
    return torch.cat([x.float(), torch.zeros(1, x.shape[1], device=DEV)])[at]


def _put(like, v, at, real):
    out = torch.zeros(like.shape, device=DEV)
    out[at[real]] = v[real]
    return out.to(like.dtype)


def _experts_plain(s, case):
    E, NW, K = s["w"].shape
    w = s["w"].float()
    if case["dtype"] == "fp8":
        w.view(E, NW // 128, 128, K // 128, 128).mul_(s["w_scale"][:, :, None, :, None])
    if case["rect"]:
        n = s["most"]
        scale = s["x_scale"][:, :, :n].transpose(1, 2).unsqueeze(-1)
        x = (s["x"][:, :n].float().view(E, n, K // 128, 128) * scale).view(E, n, K)
    else:
        x = s["x"].float()
        if case["dtype"] == "fp8":
            x = (x.view(-1, K // 128, 128) * s["x_scale"].unsqueeze(-1)).view(-1, K)
        at, real = _padded(s, x.shape[0])
        x = _gather(x, at)
    z = torch.bmm(x, w.transpose(1, 2))
    del w, x
    if s["bias"] is not None:
        z = z + s["bias"].unsqueeze(1)
    y = _act(z, case["act"])
    if case["rect"]:
        real = torch.arange(s["most"], device=DEV) < s["count"].unsqueeze(1)
        out = torch.zeros(s["y"].shape, dtype=s["y"].dtype, device=DEV)
        out[:, : s["most"]] = torch.where(real.unsqueeze(-1), y, 0.0).to(out.dtype)
        return {"y": out}
    if s["residual"] is not None:
        y = y + _gather(s["residual"], at)
    out = {"y": _put(s["y"], y, at, real)}
    if s["z"] is not None:
        out["z"] = _put(s["z"], z, at, real)
    return out


def _experts_backward_plain(s, case):
    at, real = _padded(s, s["x"].shape[0])
    dy, x, w = _gather(s["dy"], at), _gather(s["x"], at), s["w"].float()
    dw = torch.bmm(dy.transpose(1, 2), x)
    dx = torch.bmm(dy, w)
    dz = _act_grad(dx, None if s["z"] is None else _gather(s["z"], at), case["act"])
    return {"dz": _put(s["dz"], dz, at, real), "dw": dw.to(torch.bfloat16), "db": dy.sum(1)}


def _combine_backward_plain(s):
    ok = s["index"] >= 0
    at = s["index"].clamp(min=0).long()
    dy = s["dy"].float()
    dweights = torch.where(ok, (s["eo"].float()[at] * dy.unsqueeze(1)).sum(2), 0.0)
    deo = torch.zeros(s["deo"].shape, device=DEV)
    deo[at[ok]] = (s["weights"].unsqueeze(2) * dy.unsqueeze(1))[ok]
    return {"deo": deo.to(torch.bfloat16), "dweights": dweights}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "route":
            idx, w = _route_plain(s, case)
            return {"idx": idx, "weights": w}
        if op == "route_bwd":
            d = _route_grad(s["logits"].float(), s["topk_idx"], s["grad_weights"], case)
            return {"dlogits": d.to(s["logits"].dtype)}
        if op == "experts":
            return _experts_plain(s, case)
        if op == "experts_bwd":
            return _experts_backward_plain(s, case)
        return _combine_backward_plain(s)

    import unpermute_ep_dispatch_gb300 as epd
    if op == "route":
        idx, w = epd.ep_route(
            s["logits"], case["k"], s["status"], scoring=case["scoring"], bias=s["bias"],
            num_groups=case["groups"], topk_groups=case["keep"], group_score=case["group_score"],
            renormalize=case["renorm"], routed_scale=case["scale"], topk_idx=s["topk_idx"],
            topk_weights=s["topk_weights"])
        return {"idx": idx, "weights": w}
    if op == "route_bwd":
        return {"dlogits": epd.ep_route_backward(
            s["grad_weights"], s["logits"], s["topk_idx"], s["status"], scoring=case["scoring"],
            renormalize=case["renorm"], routed_scale=case["scale"], grad_logits=s["grad_logits"])}
    if op == "experts":
        fp8 = case["dtype"] == "fp8"
        y, z = epd.ep_expert_matmul(
            s["x"], s["w"], s["count"], s["status"],
            expert_start_loc=None if case["rect"] else s["start"],
            x_scale=s["x_scale"] if fp8 else None, w_scale=s["w_scale"] if fp8 else None,
            bias=s["bias"], activation=case["act"], residual=s["residual"], y=s["y"],
            preact=s["z"])
        return {"y": y} if z is None else {"y": y, "z": z}
    if op == "experts_bwd":
        dz = epd.ep_expert_matmul_dgrad(
            s["dy"], s["w"], s["count"], s["status"], expert_start_loc=s["start"],
            activation=case["act"], preact=s["z"], dx=s["dz"])
        dw, db = epd.ep_expert_matmul_wgrad(
            s["dy"], s["x"], s["count"], s["status"], expert_start_loc=s["start"], dw=s["dw"],
            dbias=s["db"])
        return {"dz": dz, "dw": dw, "db": db}
    deo, dweights = epd.ep_unpermute_backward(
        s["dy"], s["eo"], s["index"], s["weights"], s["status"], grad_expert_out=s["deo"],
        grad_weights=s["dweights"])
    return {"deo": deo, "dweights": dweights}


# --------------------------------------------------------------------------- what it needs
def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        item = 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return {"bytes": T * E * item + T * k * 12 + (4 * E if case["biased"] else 0),
                    "flops": T * E * 4}
        return {"bytes": 2 * T * E * item + T * k * 12, "flops": T * E * 6}
    if op == "combine_bwd":
        T, H, k = case["T"], case["H"], case["k"]
        pairs = T * k * (1 - case["drop"])
        return {"bytes": 2 * T * H + 4 * pairs * H + 12 * T * k, "flops": 3 * pairs * H}
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    touched = E * (1 - (1 - k / E) ** T)
    M = T * k
    if op == "experts":
        NW = 2 * N if case["act"] == "swiglu" else N
        item = 1 if case["dtype"] == "fp8" else 2
        scales = (M * K + touched * NW * K / 128) / 128 * 4 if case["dtype"] == "fp8" else 0
        return {"bytes": touched * NW * K * item + M * K * item + scales + M * N * 2
                + (touched * NW * 4 if case["bias"] else 0) + (M * N * 2 if case["residual"] else 0)
                + (M * NW * 2 if case["preact"] else 0), "flops": 2.0 * M * NW * K}
    KZ = 2 * K if case["act"] == "swiglu" else K
    return {"bytes": touched * N * K * 2 + E * N * K * 2 + 2 * M * (N + K)
            + 2 * M * KZ * (1 if case["act"] == "none" else 2) + 4 * E * N, "flops": 4.0 * M * N * K}


# ---------------------------------------------------------------------- in 64 bits
def _exact_route(s, case):
    score, c, gs = _choice64(s, case)
    T, E = score.shape
    G, k = case["groups"], case["k"]
    if case["scoring"] == "softmax" and not case["biased"]:
        c = s["logits"].double()
    if G > 1:
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices
        rank = torch.argsort(order, 1)
        c = c.masked_fill((rank >= case["keep"]).repeat_interleave(E // G, 1), -math.inf)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    gone = order.values[:, :k] == -math.inf
    w = score.gather(1, order.indices[:, :k]).masked_fill(gone, 0)
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return {"idx": order.indices[:, :k].masked_fill(gone, -1), "weights": w * case["scale"]}


def _exact_route_backward(s, case):
    """By the Jacobian of the weights, through torch's own differentiation in 64 bits."""
    l = s["logits"].double().requires_grad_()
    idx = s["topk_idx"]
    live = (l > -math.inf).any(1)
    if case["scoring"] == "sigmoid":
        score = torch.sigmoid(l)
    else:
        score = torch.softmax(torch.where(live.unsqueeze(1), l, 0.0), 1)
    w = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0)), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    d, = torch.autograd.grad((w * s["grad_weights"].double()).sum() * case["scale"], l)
    return {"dlogits": torch.where(live.unsqueeze(1), torch.nan_to_num(d), 0.0)}


def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    op = case["op"]
    if op in ("experts", "experts_bwd") and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if op == "route":
        return _exact_route(s, case)
    if op == "route_bwd":
        return _exact_route_backward(s, case)
    act = case.get("act")
    if op == "experts":
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        z = None if s["z"] is None else torch.zeros(s["z"].shape, dtype=torch.float64, device=DEV)
        for e, (c, o) in enumerate(zip(s["count"].tolist(), s["start"].tolist())):
            if c == 0:
                continue
            w = s["w"][e].double()
            at = (e, slice(0, c)) if case["rect"] else slice(o, o + c)
            x = s["x"][at].double()
            if case["dtype"] == "fp8":
                xs = s["x_scale"][e, :, :c].t() if case["rect"] else s["x_scale"][at]
                x = x * xs.double().repeat_interleave(128, 1)
                w = w * s["w_scale"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            v = torch.mm(x, w.t())
            if s["bias"] is not None:
                v += s["bias"][e].double()
            if z is not None:
                z[at] = v
            if act == "swiglu":
                half = v.shape[1] // 2
                v = v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:]
            elif act == "silu":
                v = v * torch.sigmoid(v)
            elif act == "gelu":
                v = v * _phi(v)
            elif act == "relu":
                v = torch.relu(v)
            y[at] = v + (0 if s["residual"] is None else s["residual"][at].double())
        return {"y": y} if z is None else {"y": y, "z": z}
    if op == "experts_bwd":
        dz = torch.zeros(s["dz"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)
        db = torch.zeros(s["db"].shape, dtype=torch.float64, device=DEV)
        for e, (c, o) in enumerate(zip(s["count"].tolist(), s["start"].tolist())):
            at = slice(o, o + c)
            dy = s["dy"][at].double()
            dw[e], db[e] = torch.mm(dy.t(), s["x"][at].double()), dy.sum(0)
            d = torch.mm(dy, s["w"][e].double())
            if act != "none":
                z = s["z"][at].double()
            if act == "swiglu":
                a, b = z.chunk(2, 1)
                sg = torch.sigmoid(a)
                d = torch.cat([d * b * (sg + a * sg * (1 - sg)), d * a * sg], 1)
            elif act == "silu":
                sg = torch.sigmoid(z)
                d = d * (sg + z * sg * (1 - sg))
            elif act == "gelu":
                d = d * (_phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            elif act == "relu":
                d = d * (z > 0)
            dz[at] = d
        return {"dz": dz, "dw": dw, "db": db}
    dw = torch.zeros(s["dweights"].shape, dtype=torch.float64, device=DEV)
    deo = torch.zeros(s["deo"].shape, dtype=torch.float64, device=DEV)
    dy = s["dy"].double()
    for j in range(case["k"]):
        t = torch.nonzero(s["index"][:, j] >= 0).squeeze(1)
        slot = s["index"][t, j].long()
        dw[t, j] = torch.einsum("th,th->t", s["eo"][slot].double(), dy[t])
        deo[slot] = dy[t] * s["weights"][t, j].double().unsqueeze(1)
    return {"deo": deo, "dweights": dw}
