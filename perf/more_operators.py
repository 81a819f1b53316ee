"""Cases for measuring the norm, its gradient, rotary positions, the paged cache and decode attention.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()``
makes what a user's program holds before the call, and ``run()`` makes one pass:
through the library's operators where ``own`` is true, and through the same formulas
in elementary torch operations, in 32 bits (angles in 64) and rounded once at the end,
where it is false. ``exact()`` states the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # One decoding user's token ahead of the router: the call's latency.
        dict(name="norm_one_token", op="norm", T=1, H=7168, kind="rms", dtype="bf16", residual=True, bias=False,
             out="bf16", stats=False),
        # A prefill batch ahead of the router and the fp8 dispatch: the residual joins, the router reads
        # bf16 rows and the dispatch e4m3 rows with their scales.
        dict(name="norm_prefill_fp8", op="norm", T=8192, H=7168, kind="rms", dtype="bf16", residual=True, bias=False,
             out="both", stats=False),
        # The norm of a training step, its statistics kept, over an odd batch of a 32-bit residual stream.
        dict(name="norm_train_f32", op="norm", T=4097, H=4096, kind="layer", dtype="f32", residual=False, bias=True,
             out="bf16", stats=True),
        # Its backward pass in a training step of bf16 rows, the residual's gradient joined.
        dict(name="norm_backward", op="norm_bwd", T=8192, H=7168, kind="layer", dtype="bf16", bias=True, joined=True),
        # The same on a small ragged batch of a narrow layer, 32-bit rows.
        dict(name="norm_backward_small", op="norm_bwd", T=333, H=1032, kind="rms", dtype="f32", bias=False,
             joined=False),
        # Rotation of a training batch's queries and keys (32 + 8 heads), backward.
        dict(name="rotary_backward", op="rotary", T=8192, N=40, D=128, R=128, interleaved=False, far=8192,
             inverse=True),
        # Part of an odd head, interleaved pairs, far positions of a long context, an odd batch.
        dict(name="rotary_partial", op="rotary", T=1021, N=20, D=80, R=32, interleaved=True, far=1000000,
             inverse=False),
        # A decode batch's keys and values into the paged cache, queries rotated on the way.
        dict(name="append_decode", op="append", B=128, T=128, QH=32, KH=8, D=128, R=128, interleaved=False, page=64,
             far=8192, cache="bf16"),
        # A ragged prefill's keys and values into an e4m3 cache of small pages.
        dict(name="append_prefill_fp8", op="append", B=5, T=16384, QH=64, KH=8, D=128, R=64, interleaved=True, page=16,
             far=4096, cache="fp8"),
        # One user's next token over a short context: the call's latency.
        dict(name="attention_one", op="attention", B=1, lo=1000, hi=1000, QH=32, KH=8, D=128, page=64, cache="bf16",
             window=0, lse=False),
        # A serving batch of ragged lengths (an empty sequence among them).
        dict(name="attention_batch", op="attention", B=128, lo=0, hi=8191, QH=32, KH=8, D=128, page=64, cache="bf16",
             window=0, lse=True),
        # One long context in an e4m3 cache of small pages, wide groups.
        dict(name="attention_long_fp8", op="attention", B=2, lo=131072, hi=200001, QH=64, KH=4, D=128, page=16,
             cache="fp8", window=0, lse=False),
    ]


def _log_size(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rotary", "append", "attention", "attention"])
    if op == "norm":
        out = rng.choice(["bf16", "bf16", "fp8", "both"])
        return dict(op=op, T=_log_size(rng, 1, 8192), H=_log_size(rng, 128, 7168, 8 if out == "bf16" else 128),
                    kind=rng.choice(["layer", "rms"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.5, bias=rng.random() < 0.5, out=out, stats=rng.random() < 0.5)
    if op == "norm_bwd":
        return dict(op=op, T=_log_size(rng, 1, 8192), H=_log_size(rng, 64, 7168, 8), kind=rng.choice(["layer", "rms"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5, joined=rng.random() < 0.5)
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    R = rng.choice([D, D, D // 2])
    if op == "rotary":
        return dict(op=op, T=_log_size(rng, 1, 8192), N=_log_size(rng, 1, 20), D=D, R=R,
                    interleaved=rng.random() < 0.5, far=_log_size(rng, 64, 1000000), inverse=rng.random() < 0.5)
    KH = rng.choice([1, 2, 4, 8])
    QH = KH * rng.choice([1, 2, 4, 7, 8, 16])
    page = rng.choice([1, 16, 24, 64, 128])
    cache = rng.choice(["bf16", "bf16", "fp8"])
    if op == "append":
        B = _log_size(rng, 1, 64)
        T = max(B, _log_size(rng, 1, 16384 * 64 // max(64, QH * D // 128)))
        return dict(op=op, B=B, T=T, QH=QH, KH=KH, D=D, R=R, interleaved=rng.random() < 0.5, page=page,
                    far=_log_size(rng, 16, 4096), cache=cache)
    B = _log_size(rng, 1, 128)
    hi = _log_size(rng, 1, min(300000, max(16, 400000000 // (B * KH * D))))
    return dict(op=op, B=B, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, QH=QH, KH=KH, D=D, page=page, cache=cache,
                window=rng.choice([0, 0, 0, 1 + hi // 3]), lse=rng.random() < 0.5)


# ------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Lengths spread evenly from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _runs(case):
    """Tokens that each sequence of an append gets: one at least, the rest in uneven shares."""
    B, T = case["B"], case["T"]
    ends = [i + 1 + (T - B) * (i + 1) * (i + 2) // (B * (B + 1)) for i in range(B)]
    return [e - s for s, e in zip([0] + ends, ends)]


def _inv_freq(R):
    return 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)


def _fp8_cache(x):
    """e4m3 values [.., D] of x and one fp32 scale for each token and head (amax / 448)."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale.unsqueeze(-1)).clamp_(-448, 448).to(FP8), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 29)
    op = case["op"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # a residual stream: features of their own offsets and sizes, a few of them large
        size = torch.exp(0.5 * normal(H, dtype=torch.float32))
        size[torch.rand(H, generator=g, device=DEV) < 0.01] *= 8.0
        s["x"] = (normal(T, H, dtype=torch.float32) * size + 0.3 * normal(H, dtype=torch.float32)).to(dt)
        s["weight"] = 1.0 + 0.2 * normal(H, dtype=torch.float32)
        s["bias"] = 0.1 * normal(H, dtype=torch.float32) if case["bias"] else None
        if op == "norm":
            s["residual"] = normal(T, H, dtype=dt) if case["residual"] else None
            s["sum"] = torch.empty(T, H, dtype=dt, device=DEV) if case["residual"] else None
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if case["out"] != "fp8" else None
            s["q"] = torch.empty(T, H, dtype=FP8, device=DEV) if case["out"] != "bf16" else None
            s["q_scale"] = torch.empty(T, H // 128, device=DEV) if case["out"] != "bf16" else None
            s["mean"] = torch.empty(T, device=DEV) if case["stats"] and case["kind"] == "layer" else None
            s["rstd"] = torch.empty(T, device=DEV) if case["stats"] else None
        else:
            x = s["x"].double()
            mean = x.mean(1) if case["kind"] == "layer" else torch.zeros(T, dtype=torch.float64, device=DEV)
            s["rstd"] = ((x - mean.unsqueeze(1)).square().mean(1) + 1e-5).rsqrt().float()
            s["mean"] = mean.float() if case["kind"] == "layer" else None
            s["dy"] = normal(T, H)
            s["grad_sum"] = normal(T, H, dtype=dt) if case["joined"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(H, device=DEV)
            s["dbias"] = torch.empty(H, device=DEV) if case["bias"] else None
            if own:
                import unpermute_ep_dispatch_gb300 as epd
                s["workspace"] = epd.new_norm_workspace(H)
        return s
    if op == "rotary":
        T, N, D = case["T"], case["N"], case["D"]
        s["inv_freq"] = _inv_freq(case["R"])
        s["x"] = normal(T, N, D)
        s["out"] = torch.empty_like(s["x"])
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    elif op == "append":
        B, T, QH, KH, D, page = (case[n] for n in ("B", "T", "QH", "KH", "D", "page"))
        s["inv_freq"] = _inv_freq(case["R"])
        n = torch.tensor(_runs(case), device=DEV)
        s["seq"] = torch.repeat_interleave(torch.arange(B, device=DEV, dtype=torch.int32), n)
        first = torch.randint(0, case["far"], (B,), generator=g, device=DEV)
        inside = torch.arange(T, device=DEV) - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
        s["positions"] = (torch.repeat_interleave(first, n) + inside).to(torch.int32)
        s["qkv"] = normal(T, QH + 2 * KH, D)  # one projection's rows
        # Pages for the new tokens alone: what lies before them is on pages of the table's own
        # numbers, which other sequences of the batch may share (a common prompt).
        most = (case["far"] + max(_runs(case)) + page - 1) // page + 1
        table = torch.zeros(B, most, dtype=torch.int64, device=DEV)
        at = torch.arange(most, device=DEV).unsqueeze(0)
        new = (at >= (first // page).unsqueeze(1)) & (at <= ((first + n - 1) // page).unsqueeze(1))
        pages = sum(-(-r // page) + 1 for r in _runs(case))  # a run may end on one page more
        table[new] = torch.randperm(pages, generator=g, device=DEV)[: int(new.sum())]
        s["table"] = table.to(torch.int32)
        for c in ("k", "v"):
            if case["cache"] == "fp8":
                s[c], s[c + "_scale"] = _fp8_cache(normal(pages, page, KH, D, dtype=torch.float32))
            else:
                s[c], s[c + "_scale"] = normal(pages, page, KH, D), None
        s["q_out"] = torch.empty(T, QH, D, dtype=torch.bfloat16, device=DEV)
    else:
        B, QH, KH, D, page = (case[n] for n in ("B", "QH", "KH", "D", "page"))
        lens = torch.tensor(_lengths(case), device=DEV)[torch.randperm(B, generator=g, device=DEV)]
        s["lengths"] = lens.to(torch.int32)
        most = max(1, -(-case["hi"] // page))
        need = torch.arange(most, device=DEV).unsqueeze(0) < ((lens + page - 1) // page).unsqueeze(1)
        pages = max(1, int(need.sum()))
        table = torch.zeros(B, most, dtype=torch.int64, device=DEV)
        table[need] = torch.randperm(pages, generator=g, device=DEV)[: int(need.sum())]
        s["table"] = table.to(torch.int32)
        s["q"] = normal(B, QH, D) * 1.5
        for c in ("k", "v"):
            if case["cache"] == "fp8":
                s[c], s[c + "_scale"] = _fp8_cache(normal(pages, page, KH, D).float())
            else:
                s[c], s[c + "_scale"] = normal(pages, page, KH, D), None
        s["out"] = torch.empty(B, QH, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, QH, device=DEV) if case["lse"] else None
        if own:
            import unpermute_ep_dispatch_gb300 as epd
            s["workspace"] = epd.new_attention_workspace(B, QH, KH, D)
    if own and op in ("rotary", "append"):
        import unpermute_ep_dispatch_gb300 as epd
        s["steps"] = epd.rotary_steps(s["inv_freq"])
    return s


# ------------------------------------------------------------------------- plain forms
def _norm_plain(s, case):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    mean = x.mean(1, keepdim=True) if case["kind"] == "layer" else torch.zeros(x.shape[0], 1, device=DEV)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
    y = c * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    out = {}
    if s["sum"] is not None:
        out["sum"] = x.to(s["x"].dtype)
    if s["y"] is not None:
        out["y"] = y.to(torch.bfloat16)
    if s["q"] is not None:
        b = y.view(y.shape[0], -1, 128)
        amax = b.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        out["q"] = (b / scale.unsqueeze(-1)).clamp(-448, 448).to(FP8).view(y.shape)
        out["q_scale"] = scale
    if s["mean"] is not None:
        out["mean"] = mean.squeeze(1)
    if s["rstd"] is not None:
        out["rstd"] = rstd.squeeze(1)
    return out


def _norm_backward_plain(s):
    dy, x, rstd = s["dy"].float(), s["x"].float(), s["rstd"].unsqueeze(1)
    if s["mean"] is not None:
        x = x - s["mean"].unsqueeze(1)
    xhat = x * rstd
    g = dy * s["weight"]
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if s["mean"] is not None:
        d = d - g.mean(1, keepdim=True)
    d = d * rstd
    if s["grad_sum"] is not None:
        d = d + s["grad_sum"].float()
    out = {"dx": d.to(s["x"].dtype), "dweight": (dy * xhat).sum(0)}
    if s["dbias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _rotate_plain(x, positions, inv_freq, interleaved, inverse=False):
    """The rotation of x [T, N, D] in 32 bits, of angles taken in 64."""
    R = 2 * inv_freq.shape[0]
    angle = positions.double().unsqueeze(1) * inv_freq
    c, n = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    if inverse:
        n = -n
    x = x.float()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        turned = torch.cat([a * c - b * n, a * n + b * c], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _append_plain(s, case):
    QH, KH, page = case["QH"], case["KH"], case["page"]
    qkv, pos = s["qkv"], s["positions"].long()
    turned = _rotate_plain(qkv[:, : QH + KH], s["positions"], s["inv_freq"], case["interleaved"])
    at = s["table"].long()[s["seq"].long(), pos // page]
    for name, rows in (("k", turned[:, QH:]), ("v", qkv[:, QH + KH:].float())):
        if case["cache"] == "fp8":
            rows, scale = _fp8_cache(rows)
            s[name].view(torch.uint8)[at, pos % page] = rows.view(torch.uint8)
            s[name + "_scale"][at, pos % page] = scale
        else:
            s[name][at, pos % page] = rows.to(torch.bfloat16)
    return {"q": turned[:, :QH].to(torch.bfloat16), "k": s["k"], "v": s["v"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _attention_plain(s, case):
    B, QH, KH, D, page = (case[n] for n in ("B", "QH", "KH", "D", "page"))
    table, lens = s["table"].long(), s["lengths"].long()
    L = table.shape[1] * page

    def rows(name):  # [B, KH, L, D]
        x = s[name][table] if case["cache"] == "bf16" else s[name].view(torch.uint8)[table].view(FP8)
        x = x.float()
        if case["cache"] == "fp8":
            x = x * s[name + "_scale"][table].unsqueeze(-1)
        return x.view(B, L, KH, D).transpose(1, 2)

    at = torch.arange(L, device=DEV)
    live = at < lens.unsqueeze(1)
    if case["window"]:
        live = live & (at >= (lens - case["window"]).unsqueeze(1))
    live = live.view(B, 1, 1, L)
    q = s["q"].float().view(B, KH, QH // KH, D) / math.sqrt(D)
    score = torch.where(live, torch.matmul(q, rows("k").transpose(2, 3)), -math.inf)
    m = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, rows("v")) / torch.where(total > 0, total, 1.0)
    out = {"o": o.reshape(B, QH, D).to(torch.bfloat16)}
    if s["lse"] is not None:
        out["lse"] = (m + torch.log(total)).view(B, QH)
    return out


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "norm":
            return _norm_plain(s, case)
        if op == "norm_bwd":
            return _norm_backward_plain(s)
        if op == "rotary":
            x = _rotate_plain(s["x"], s["positions"], s["inv_freq"], case["interleaved"], case["inverse"])
            return {"x": x.to(torch.bfloat16)}
        if op == "append":
            return _append_plain(s, case)
        return _attention_plain(s, case)

    import unpermute_ep_dispatch_gb300 as epd
    if op == "norm":
        r = epd.ep_layer_norm(
            s["x"], s["weight"], bias=s["bias"], residual=s["residual"], eps=1e-5, kind=case["kind"], sum=s["sum"],
            y=s["y"], with_y=s["y"] is not None, y_q=s["q"], y_scale=s["q_scale"], mean=s["mean"], rstd=s["rstd"])
        names = {"sum": "sum", "y": "y", "q": "y_q", "q_scale": "y_scale", "mean": "mean", "rstd": "rstd"}
        return {n: r[m] for n, m in names.items() if r[m] is not None}
    if op == "norm_bwd":
        dx, dweight, dbias = epd.ep_layer_norm_backward(
            s["dy"], s["x"], s["weight"], s["rstd"], mean=s["mean"], kind=case["kind"], grad_sum=s["grad_sum"],
            workspace=s["workspace"], dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])
        return {"dx": dx, "dweight": dweight} if dbias is None else {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "rotary":
        return {"x": epd.ep_rotary(s["x"], s["positions"], s["steps"], interleaved=case["interleaved"],
                                   inverse=case["inverse"], out=s["out"])}
    if op == "append":
        QH, KH = case["QH"], case["KH"]
        q = epd.ep_cache_append(
            s["qkv"][:, QH: QH + KH], s["qkv"][:, QH + KH:], s["k"], s["v"], s["table"], s["positions"], s["status"],
            token_seq=s["seq"], q=s["qkv"][:, :QH], steps=s["steps"], interleaved=case["interleaved"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"])
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    o, lse = epd.ep_decode_attention(
        s["q"], s["k"], s["v"], s["table"], s["lengths"], s["workspace"], s["status"], k_scale=s["k_scale"],
        v_scale=s["v_scale"], window=case["window"], out=s["out"], lse=s["lse"])
    return {"o": o} if lse is None else {"o": o, "lse": lse}


# --------------------------------------------------------------------------- what it needs
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        item = 4 if case["dtype"] == "f32" else 2
        if op == "norm":
            wide = {"bf16": 2, "fp8": 1 + 4 / 128, "both": 3 + 4 / 128}[case["out"]]
            return {"bytes": T * H * (item * (3 if case["residual"] else 1) + wide) + 4 * H * (1 + case["bias"])
                    + (8 * T if case["stats"] else 0), "flops": 8 * T * H}
        return {"bytes": T * H * (2 + item * (3 if case["joined"] else 2)) + 4 * H * (2 + case["bias"]) + 8 * T,
                "flops": 12 * T * H}
    if op == "rotary":
        T, N, D, R = case["T"], case["N"], case["D"], case["R"]
        return {"bytes": 4 * T * N * D + 4 * T, "flops": 3 * T * N * R}
    QH, KH, D = case["QH"], case["KH"], case["D"]
    held = 2 * D if case["cache"] == "bf16" else D + 4  # a token's bytes for one head
    if op == "append":
        T = case["T"]
        return {"bytes": T * (4 * QH * D + 4 * KH * D + 2 * KH * held + 8), "flops": 3 * T * (QH + KH) * case["R"]}
    lens = _lengths(case)
    tokens = sum(min(n, case["window"]) for n in lens) if case["window"] else sum(lens)
    return {"bytes": 2 * tokens * KH * held + 4 * case["B"] * QH * D, "flops": 4.0 * tokens * QH * D}


# ---------------------------------------------------------------------- in 64 bits
def _exact_norm(s, case):
    x = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    n = x.shape[1]
    mean = x.sum(1) / n if case["kind"] == "layer" else torch.zeros(x.shape[0], dtype=torch.float64, device=DEV)
    var = torch.einsum("th,th->t", x - mean[:, None], x - mean[:, None]) / n
    rstd = torch.pow(var + 1e-5, -0.5)
    y = torch.addcmul(torch.zeros_like(x), (x - mean[:, None]) * s["weight"].double(), rstd[:, None])
    if s["bias"] is not None:
        y += s["bias"].double()
    out = {"sum": x, "y": y, "mean": mean, "rstd": rstd}
    if s["q"] is not None:
        top = torch.nn.functional.max_pool1d(y.abs().unsqueeze(1), 128).squeeze(1) / 448.0
        top[top == 0] = 1.0
        out["q"], out["q_scale"] = y / top.repeat_interleave(128, 1), top
    return {k: v for k, v in out.items() if s[k] is not None}


def _exact_norm_backward(s, case):
    """By torch's own differentiation of the norm in 64 bits."""
    x = s["x"].double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    mean = x.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0
    y = (x - mean) * torch.rsqrt((x - mean).pow(2).mean(1, keepdim=True) + 1e-5) * w
    dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
    out = {"dx": dx + (0 if s["grad_sum"] is None else s["grad_sum"].double()), "dweight": dw}
    if s["dbias"] is not None:
        out["dbias"] = s["dy"].double().sum(0)
    return out


def _exact_turn(x, positions, inv_freq, interleaved, sign):
    """As a product of complex numbers."""
    R = 2 * inv_freq.shape[0]
    x = x.double()
    head = x[..., :R]
    pairs = head.unflatten(-1, (R // 2, 2)) if interleaved else head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), sign * torch.outer(positions.double(), inv_freq))
    pairs = torch.view_as_real(z * turn.unsqueeze(1))
    head = (pairs if interleaved else pairs.transpose(-1, -2)).flatten(-2)
    return torch.cat([head, x[..., R:]], -1)


def _exact_append(s, case):
    QH, KH, page = case["QH"], case["KH"], case["page"]
    x = s["qkv"]
    turned = _exact_turn(x[:, : QH + KH], s["positions"], s["inv_freq"], case["interleaved"], 1.0)
    pos = s["positions"].long()
    slot = s["table"].long()[s["seq"].long(), pos // page] * page + pos % page
    out = {"q": turned[:, :QH]}
    for name, rows in (("k", turned[:, QH:]), ("v", x[:, QH + KH:].double())):
        held = s[name].double().flatten(0, 1)
        if case["cache"] == "fp8":
            top = rows.abs().amax(-1) / 448.0
            top[top == 0] = 1.0
            rows = rows / top.unsqueeze(-1)
            out[name + "_scale"] = s[name + "_scale"].double().flatten(0, 1).index_copy(0, slot, top).view(
                s[name + "_scale"].shape)
        out[name] = held.index_copy(0, slot, rows).view(s[name].shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s, case)
    if op == "norm_bwd":
        return _exact_norm_backward(s, case)
    if op == "rotary":
        return {"x": _exact_turn(s["x"], s["positions"], s["inv_freq"], case["interleaved"],
                                 -1.0 if case["inverse"] else 1.0)}
    if op == "append":
        return _exact_append(s, case)
    KH, D, page = case["KH"], case["D"], case["page"]
    B, QH = case["B"], case["QH"]
    o = torch.zeros(B, QH, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, QH), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        at = s["table"][b, first // page: (n + page - 1) // page].long()
        cut = slice(first % page, first % page + n - first)
        for h in range(KH):
            k, v = (s[c][:, :, h].view(torch.uint8)[at].view(s[c].dtype).double() if case["cache"] == "fp8"
                    else s[c][at, :, h].double() for c in ("k", "v"))
            if case["cache"] == "fp8":
                k, v = (x * s[c][at, :, h].double().unsqueeze(-1) for x, c in ((k, "k_scale"), (v, "v_scale")))
            k, v = k.flatten(0, 1)[cut], v.flatten(0, 1)[cut]
            g = slice(h * QH // KH, (h + 1) * QH // KH)
            score = s["q"][b, g].double() @ k.t() * D ** -0.5
            o[b, g] = torch.softmax(score, 1) @ v
            lse[b, g] = torch.logsumexp(score, 1)
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
