"""ep_route, ep_expert_matmul, their gradients and ep_unpermute_backward against plain
definitions in 64 bits.

Tolerances: a bf16 output is rounded once, at most 2^-9 of its value from the exact
result; 2^-8 is allowed. Sums of n products accumulated in fp32 in any order, each step
rounded or truncated, are within n * 2^-23 of the sum of the products' magnitudes. An
activation passes an error on with its largest slope (1.13 for silu and gelu)."""
import math

import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd

pytestmark = pytest.mark.gpu

DEV = "cuda"
INF = math.inf


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def check_ok(status):
    torch.cuda.synchronize()
    epd.check_status(status, "test")


# ------------------------------------------------------------------------------ routing
def route_ref(l, k, scoring, bias, groups, keep, group_score, renorm, scale):
    """Token by token, with Python sorting: (value descending, index ascending)."""
    l = l.double().cpu()
    T, E = l.shape
    size = E // groups
    idx = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = [v if v < INF else -INF for v in l[t].tolist()]
        m = max(row)
        if m == -INF:
            continue
        if scoring == "sigmoid":
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        else:
            ex = [math.exp(v - m) for v in row]
            s = [v / sum(ex) for v in ex]
        b = [0.0] * E if bias is None else bias.double().cpu().tolist()
        c = [s[e] + b[e] for e in range(E)]
        rank = row if scoring == "softmax" and bias is None else c
        live = [e for e in range(E) if row[e] > -INF]
        score = []
        for g in range(groups):
            own = sorted((c[e] for e in live if e // size == g), reverse=True)
            two = own[:2] if group_score == "top2" else own[:1]
            score.append(sum(two) if two else -INF)
        best = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
        order = sorted((e for e in live if e // size in best), key=lambda e: (-rank[e], e))[:k]
        total = sum(s[e] for e in order)
        for j, e in enumerate(order):
            idx[t, j] = e
            w[t, j] = (s[e] / total if total > 0 else 0.0) * scale if renorm else s[e] * scale
    return idx, w


def route_inputs(T, E, dtype, seed, masked):
    """Logits on a grid of 1/8 whose scores are far apart in 32 bits or exactly equal (ties)."""
    g = gen(seed)
    l = (torch.randint(-24, 25, (T, E), generator=g, device=DEV).float() / 8).to(dtype)
    if masked:
        u = torch.rand(T, E, generator=g, device=DEV)
        l[u < 0.2] = -INF
        l[u > 0.95] = torch.finfo(dtype).min
        l[0] = -INF                                    # nothing left
        if T > 2:
            l[1] = torch.finfo(dtype).min              # lowest everywhere: an ordinary row
            l[2] = -INF
            l[2, E // 2] = 0.5                         # one expert left
    return l


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,groups,keep,gs", [
    (1, 256, 8, 8, 4, "top2"), (5, 1, 1, 1, 1, "max"), (37, 8, 8, 1, 1, "max"), (33, 60, 6, 6, 2, "max"),
    (64, 160, 6, 8, 3, "top2"), (130, 33, 33, 1, 1, "max"), (17, 600, 40, 40, 7, "top2"),
    (9, 4096, 64, 64, 16, "max"), (4, 64, 3, 64, 5, "top2"), (21, 96, 7, 3, 3, "top2"),
    (3, 1030, 9, 2, 1, "top2")])
@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("masked", [False, True])
def test_route(dtype, T, E, k, groups, keep, gs, scoring, biased, masked):
    l = route_inputs(T, E, dtype, T * 7 + E, masked)
    # biases of whole numbers: sums of a score and a bias are equal only where both are
    bias = torch.randint(-2, 3, (E,), generator=gen(E), device=DEV).float() if biased else None
    if gs == "top2" and scoring == "softmax":
        l = (l.float() * 1.0).to(dtype)
    status = epd.new_status()
    k = min(k, E)
    idx, w = epd.ep_route(l, k, status, scoring=scoring, bias=bias, num_groups=groups,
                          topk_groups=keep, group_score=gs, renormalize=True, routed_scale=2.5)
    check_ok(status)
    ri, rw = route_ref(l, k, scoring, bias, groups, keep, gs, True, 2.5)
    if gs == "top2" and keep < groups:
        # sums of two scores may tie in 32 bits only: a row may differ where the kept groups'
        # scores are that close; the weights' sum still has to be the scale
        same = (idx.cpu() == ri).all(1)
        assert same.float().mean() > 0.9
        got, want = w.cpu().double()[same], rw[same]
    else:
        assert torch.equal(idx.cpu(), ri)
        got, want = w.cpu().double(), rw
    # exp, a division and a sum of up to k terms: a few units in the last place of 32 bits
    assert (got - want).abs().max() <= (k + 16) * 2 ** -23 * 2.5


def test_route_without_renormalize_and_scores():
    l = route_inputs(50, 48, torch.float32, 3, True)
    status = epd.new_status()
    idx, w = epd.ep_route(l, 5, status, scoring="softmax", renormalize=False)
    check_ok(status)
    ri, rw = route_ref(l, 5, "softmax", None, 1, 1, "max", False, 1.0)
    assert torch.equal(idx.cpu(), ri)
    assert (w.cpu().double() - rw).abs().max() <= 70 * 2 ** -23


def test_route_reports_nonfinite_logits():
    l = torch.randn(6, 16, device=DEV)
    l[2, 3] = math.nan
    l[4, 5] = INF
    status = epd.new_status()
    idx, w = epd.ep_route(l, 4, status)
    torch.cuda.synchronize()
    assert int(status.item()) == epd.EPD_ERR_NONFINITE
    clean = torch.where(torch.isnan(l) | (l == INF), -INF, l)
    ri, _ = route_ref(clean, 4, "softmax", None, 1, 1, "max", True, 1.0)
    assert torch.equal(idx.cpu(), ri)
    assert torch.isfinite(w).all()


def route_weights64(l, idx, scoring, renorm, scale):
    live = (l > -INF).any(1, keepdim=True)
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(torch.where(live, l, 0.0), 1)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return w * scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (7, 1, 1), (65, 60, 6), (33, 300, 40), (5, 4096, 64), (2, 1030, 3)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(dtype, T, E, k, scoring, renorm):
    l = route_inputs(T, E, dtype, E + T, T > 3 and E > 8)
    status = epd.new_status()
    idx, _ = epd.ep_route(l, k, status, scoring=scoring)
    g = torch.randn(T, k, generator=gen(T), device=DEV)
    d = epd.ep_route_backward(g, l, idx, status, scoring=scoring, renormalize=renorm, routed_scale=1.5)
    check_ok(status)
    x = l.double().requires_grad_()
    w = route_weights64(x, idx, scoring, renorm, 1.5)
    want, = torch.autograd.grad((w * g.double()).sum(), x)
    want = torch.where((l > -INF).any(1, keepdim=True), torch.nan_to_num(want), 0.0)
    # slopes of the weights are at most 1 / S per pick; S >= the largest pick's score
    s = torch.sigmoid(l.double()) if scoring == "sigmoid" else \
        torch.softmax(torch.where((l > -INF).any(1, keepdim=True), l.double(), 0.0), 1)
    sel = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    S = sel.sum(1, keepdim=True).clamp(min=1e-30) if renorm else torch.ones(T, 1, device=DEV, dtype=torch.float64)
    tol = (k + 24) * 2 ** -23 * 1.5 * 2 * g.abs().double().amax(1, keepdim=True) * \
        torch.minimum(s / S, torch.ones_like(s))
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2 ** -8
    assert ((d.double() - want).abs() <= tol + 1e-37).all()


def test_route_backward_against_differences():
    """Central differences of the 64-bit weights along random directions."""
    T, E, k = 12, 40, 5
    l = torch.randn(T, E, generator=gen(1), device=DEV)
    status = epd.new_status()
    for scoring in ("softmax", "sigmoid"):
        idx, _ = epd.ep_route(l, k, status, scoring=scoring)
        g = torch.randn(T, k, generator=gen(2), device=DEV)
        d = epd.ep_route_backward(g, l, idx, status, scoring=scoring)
        v = torch.randn(T, E, generator=gen(3), device=DEV).double()
        h = 1e-5
        up = (route_weights64(l.double() + h * v, idx, scoring, True, 1.0) * g).sum(1)
        dn = (route_weights64(l.double() - h * v, idx, scoring, True, 1.0) * g).sum(1)
        diff = (up - dn) / (2 * h)
        assert torch.allclose((d.double() * v).sum(1), diff, rtol=1e-5, atol=1e-5)
    check_ok(status)


def test_route_backward_repeated_and_invalid_picks():
    l = torch.randn(3, 10, device=DEV)
    idx = torch.tensor([[2, 2, 5], [1, -1, 0], [4, 99, 3]], device=DEV)
    g = torch.randn(3, 3, device=DEV)
    status = epd.new_status()
    d = epd.ep_route_backward(g, l, idx, status, scoring="sigmoid", renormalize=False)
    torch.cuda.synchronize()
    assert int(status.item()) == epd.EPD_ERR_INVALID_EXPERT
    s = torch.sigmoid(l.double())
    want = torch.zeros(3, 10, dtype=torch.float64, device=DEV)
    for t in range(3):
        for j in range(3):
            e = int(idx[t, j])
            if 0 <= e < 10:
                want[t, e] += g[t, j].double() * s[t, e] * (1 - s[t, e])
    assert (d.double() - want).abs().max() < 1e-6


# ------------------------------------------------------------------------- products
def act64(z, act):
    if act == "swiglu":
        a, b = z.chunk(2, -1)
        return a * torch.sigmoid(a) * b
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z.relu() if act == "relu" else z


def regions(counts, gaps, rect=0):
    """Starts of regions with gaps between them, in an order that is not the experts'."""
    E = len(counts)
    if rect:
        return [e * rect for e in range(E)], E * rect
    order = sorted(range(E), key=lambda e: (e * 7 + 3) % E)
    start, at = [0] * E, 0
    for e in order:
        start[e] = at
        at += counts[e] + gaps
    return start, at + 2


COUNTS = {
    "one": [1], "empty": [0], "none_and_some": [0, 5, 0, 0, 3, 1, 0], "ragged": [33, 1, 0, 127, 128, 129, 64, 7],
    "long": [700, 3, 255, 256, 257], "forty": [(i * 37) % 23 for i in range(40)],
}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rows_of(start, counts):
    return torch.tensor([s + r for s, c in zip(start, counts) for r in range(c)], dtype=torch.int64, device=DEV)


def forward_case(counts, K, N, act, seed, fp8=False, bias=False, residual=False, rect=0, col_major=False, gaps=0):
    g = gen(seed)
    E = len(counts)
    NW = 2 * N if act == "swiglu" else N
    start, M = regions(counts, gaps, rect)
    x = torch.randn(M, K, generator=g, device=DEV)
    w = torch.randn(E, NW, K, generator=g, device=DEV) / math.sqrt(K)
    real = rows_of(start, counts)
    dead = torch.ones(M, dtype=torch.bool, device=DEV)
    dead[real] = False
    kw = {}
    if fp8:
        C = K // 128
        xs = 0.5 + torch.rand(M, C, generator=g, device=DEV)
        ws = 0.5 + torch.rand(E, (NW + 127) // 128, C, generator=g, device=DEV)
        x, w = x.to(torch.float8_e4m3fn), (w * 8).to(torch.float8_e4m3fn)
        xd = x.double() * xs.double().repeat_interleave(128, 1)
        wd = w.double() * ws.double().repeat_interleave(128, 1)[:, :NW].repeat_interleave(128, 2)
        x.view(torch.uint8)[dead] = 0x7f                       # NaN in rows of no expert
        xs[dead] = math.nan
        if rect:
            kw["x_scale"] = xs.view(E, rect, C).transpose(1, 2).contiguous()
        elif col_major:
            ld = M + 5
            kw["x_scale"] = torch.full((C, ld), math.nan, device=DEV)
            kw["x_scale"][:, :M] = xs.t()
            kw["scale_col_major"] = True
        else:
            kw["x_scale"] = xs
        kw["w_scale"] = ws
    else:
        x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
        xd, wd = x.double(), w.double()
        x[dead] = math.nan
    b = 0.5 * torch.randn(E, NW, generator=g, device=DEV) if bias else None
    r = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16) if residual else None
    z = torch.full((M, NW), math.nan, dtype=torch.float64, device=DEV)
    mag = torch.full((M, NW), math.nan, dtype=torch.float64, device=DEV)
    for e, (s, c) in enumerate(zip(start, counts)):
        z[s:s + c] = xd[s:s + c] @ wd[e].t() + (0 if b is None else b[e].double())
        mag[s:s + c] = xd[s:s + c].abs() @ wd[e].abs().t() + (0 if b is None else b[e].double().abs())
    y = act64(z, act) + (0 if r is None else r.double())
    zerr = (K + 16) * 2.0 ** -23 * mag + 1e-30
    if act == "swiglu":
        a, u = z.chunk(2, 1)
        ea, eu = zerr.chunk(2, 1)
        yerr = 1.13 * ea * (u.abs() + eu) + eu * (a * torch.sigmoid(a)).abs()
        yerr = yerr + 16 * 2.0 ** -23 * (a.abs() * u.abs())
    else:
        yerr = 1.13 * zerr + 16 * 2.0 ** -23 * z.abs()
    kw |= dict(bias=b, activation=act)
    if rect:
        x = x.view(E, rect, K)
        r = None if r is None else r.view(E, rect, N)
    else:
        kw["expert_start_loc"] = i32(start)
    return x, w, i32(counts), kw | dict(residual=r), real, y, z, yerr + y.abs() * 2 ** -8, zerr + z.abs() * 2 ** -8


def run_forward(counts, K, N, act, seed=0, preact=False, **opts):
    x, w, cnt, kw, real, y, z, ty, tz = forward_case(counts, K, N, act, seed, **opts)
    status = epd.new_status()
    lead = x.shape[:-1]
    fill = 7.0
    out = torch.full((*lead, N), fill, dtype=torch.bfloat16, device=DEV)
    pre = torch.full((*lead, z.shape[1]), fill, dtype=torch.bfloat16, device=DEV) if preact else None
    got, gz = epd.ep_expert_matmul(x, w, cnt, status, y=out, preact=pre, **kw)
    check_ok(status)
    assert got is out and gz is pre
    got = got.view(-1, N)
    assert ((got[real].double() - y[real]).abs() <= ty[real]).all()
    dead = torch.ones(got.shape[0], dtype=torch.bool, device=DEV)
    dead[real] = False
    assert (got[dead] == fill).all(), "rows of no expert were written"
    if preact:
        gz = gz.view(got.shape[0], -1)
        assert ((gz[real].double() - z[real]).abs() <= tz[real]).all()
        assert (gz[dead] == fill).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", [(64, 64), (8, 8), (520, 272), (72, 136), (1000, 1304)])
def test_expert_matmul_bf16(counts, K, N):
    run_forward(COUNTS[counts], K, N, "none", seed=K + N, gaps=3)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias,residual,preact", [(True, False, False), (False, True, True), (True, True, True)])
def test_expert_matmul_epilogue(act, bias, residual, preact):
    run_forward(COUNTS["ragged"], 200, 304, act, seed=5, bias=bias, residual=residual, preact=preact, gaps=1)
    run_forward(COUNTS["forty"], 136, 16, act, seed=6, bias=bias, residual=residual, preact=preact)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,act", [(128, 128, "none"), (256, 384, "swiglu"), (640, 200, "gelu"), (1152, 128, "swiglu")])
@pytest.mark.parametrize("col_major", [False, True])
def test_expert_matmul_fp8(counts, K, N, act, col_major):
    run_forward(COUNTS[counts], K, N, act, seed=K, fp8=True, bias=act != "none", preact=act == "swiglu",
                col_major=col_major, gaps=2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rect", [130, 257])
def test_expert_matmul_rectangles(fp8, rect):
    run_forward(COUNTS["ragged"], 384, 256, "swiglu", fp8=fp8, rect=rect, bias=True)
    run_forward([min(c, rect) for c in COUNTS["long"]], 128, 128, "none", fp8=fp8, rect=rect, residual=True)


def test_expert_matmul_one_expert_is_a_linear_layer():
    run_forward([1000], 1024, 512, "gelu", bias=True, residual=True)


@pytest.mark.parametrize("N", [8, 24, 40, 72, 200])
def test_expert_matmul_gated_odd_widths(N):
    run_forward(COUNTS["ragged"], 72, N, "swiglu", seed=N, bias=True, residual=True, preact=True)


def test_expert_matmul_long_reduction_and_many_rows():
    run_forward([2000, 0, 311], 4096, 640, "swiglu", seed=2)
    run_forward([900, 20], 4096, 1024, "none", seed=3, fp8=True)


def test_expert_matmul_infinities_stay_in_their_row():
    x, w, cnt, kw, real, y, *_ = forward_case([40, 90], 256, 128, "none", 1)
    x[7, 3] = INF
    x[50, 9] = math.nan
    status = epd.new_status()
    got, _ = epd.ep_expert_matmul(x, w, cnt, status, **kw)
    check_ok(status)
    bad = ~torch.isfinite(got[real]).all(1)
    assert set(real[bad].tolist()) <= {7, 50} and 50 in real[bad].tolist()


def test_expert_rows_out_of_range_are_reported_and_cut():
    w = torch.randn(3, 64, 64, device=DEV).to(torch.bfloat16)
    x = torch.randn(100, 64, device=DEV).to(torch.bfloat16)
    for counts, start, code in (([10, 90, 5], [0, 10, 99], epd.EPD_ERR_CAPACITY),
                                ([10, -4, 5], [0, 10, 20], epd.EPD_ERR_INVALID_ARG),
                                ([10, 4, 5], [0, -3, 20], epd.EPD_ERR_INVALID_ARG),
                                ([10, 4, 5], [0, 200, 20], epd.EPD_ERR_CAPACITY)):
        status = epd.new_status()
        y = torch.full((101, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        epd.ep_expert_matmul(x, w, i32(counts), status, expert_start_loc=i32(start), y=y[:100])
        torch.cuda.synchronize()
        assert int(status.item()) == code
        assert (y[100] == 7).all()
        assert torch.allclose(y[:10].float(), x[:10].float() @ w[0].float().t(), rtol=0.02, atol=0.02)
    status = epd.new_status()
    epd.ep_expert_matmul(x[:30].view(3, 10, 64), w, i32([3, 11, 2]), status)
    torch.cuda.synchronize()
    assert int(status.item()) == epd.EPD_ERR_CAPACITY


def backward_case(counts, K, N, act, seed, gaps, rect=0):
    g = gen(seed)
    E = len(counts)
    start, M = regions(counts, gaps, rect)
    KZ = 2 * K if act == "swiglu" else K
    dy = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(E, N, K, generator=g, device=DEV) / math.sqrt(N)).to(torch.bfloat16)
    z = torch.randn(M, KZ, generator=g, device=DEV).to(torch.bfloat16)
    real = rows_of(start, counts)
    dead = torch.ones(M, dtype=torch.bool, device=DEV)
    dead[real] = False
    for t in (dy, x, z):
        t[dead] = math.nan
    return E, start, M, KZ, dy, x, w, z, real, dead


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,act", [(64, 64, "none"), (8, 16, "relu"), (264, 520, "swiglu"), (136, 72, "gelu"),
                                     (1000, 200, "silu"), (304, 1304, "none")])
def test_dgrad(counts, K, N, act):
    E, start, M, KZ, dy, x, w, z, real, dead = backward_case(COUNTS[counts], K, N, act, K, 3)
    status = epd.new_status()
    dx = torch.full((M, KZ), 7.0, dtype=torch.bfloat16, device=DEV)
    epd.ep_expert_matmul_dgrad(dy, w, i32(COUNTS[counts]), status, expert_start_loc=i32(start), activation=act,
                               preact=None if act == "none" else z, dx=dx)
    check_ok(status)
    d = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(d)
    for e, (s, c) in enumerate(zip(start, COUNTS[counts])):
        d[s:s + c] = dy[s:s + c].double() @ w[e].double()
        mag[s:s + c] = dy[s:s + c].double().abs() @ w[e].double().abs()
    zz = z.double().requires_grad_()
    a = act64(zz, act)
    slope, = torch.autograd.grad(a, zz, torch.where(dead.unsqueeze(1), 0.0, d)) if act != "none" else (d,)
    big, = torch.autograd.grad(act64(zz, act), zz, torch.ones_like(a)) if act != "none" else (torch.ones_like(d),)
    m2 = torch.cat([mag, mag], 1) if act == "swiglu" else mag
    d2 = torch.cat([d, d], 1) if act == "swiglu" else d
    tol = (N + 16) * 2.0 ** -23 * m2 * big.abs() + 2 ** -8 * slope.abs() + 16 * 2.0 ** -23 * d2.abs() * (1 + torch.cat([z, z], 1)[:, :KZ].double().abs()) ** 2 + 1e-30
    assert ((dx[real].double() - slope[real]).abs() <= tol[real]).all()
    assert (dx[dead] == 7).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", [(64, 64), (8, 16), (264, 520), (136, 72), (1000, 200), (512, 768)])
@pytest.mark.parametrize("with_dbias", [False, True])
def test_wgrad(counts, K, N, with_dbias):
    E, start, M, KZ, dy, x, w, z, real, dead = backward_case(COUNTS[counts], K, N, "none", N, 5)
    status = epd.new_status()
    dw, db = epd.ep_expert_matmul_wgrad(dy, x, i32(COUNTS[counts]), status, expert_start_loc=i32(start),
                                        with_dbias=with_dbias)
    check_ok(status)
    assert (db is not None) == with_dbias
    for e, (s, c) in enumerate(zip(start, COUNTS[counts])):
        a, b = dy[s:s + c].double(), x[s:s + c].double()
        want = a.t() @ b
        tol = (c + 8) * 2.0 ** -23 * (a.abs().t() @ b.abs()) + 2 ** -8 * want.abs()
        assert ((dw[e].double() - want).abs() <= tol).all()
        if with_dbias:
            assert ((db[e].double() - a.sum(0)).abs() <= (c + 1) * 2.0 ** -23 * a.abs().sum(0)).all()


# Few tiles and a long reduction: several pairs of blocks share it.
FEW = dict(one=[1], sixteen=[16], two=[40, 7], wide=[130, 3], rows=[200], full=[256], gap=[3, 0, 90], eight=[1] * 8,
           second=[257])


@pytest.mark.parametrize("counts", FEW)
@pytest.mark.parametrize("K,N,act", [(1544, 200, "none"), (4096, 512, "gelu"), (2000, 136, "swiglu"), (3592, 2304, "none")])
def test_shared_reduction_bf16(counts, K, N, act):
    run_forward(FEW[counts], K, N, act, seed=K, bias=act != "none", residual=act == "swiglu", preact=act == "gelu", gaps=1)


@pytest.mark.parametrize("counts", FEW)
@pytest.mark.parametrize("K,N,act", [(1536, 200, "none"), (4096, 512, "gelu"), (2176, 128, "swiglu"), (3200, 2304, "none")])
def test_shared_reduction_fp8(counts, K, N, act):
    run_forward(FEW[counts], K, N, act, seed=K, fp8=True, bias=act != "none", residual=act == "swiglu",
                preact=act == "gelu", gaps=1)


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_reduction_of_rectangles(fp8):
    run_forward([3, 0, 20], 2048, 256, "swiglu", fp8=fp8, rect=24, bias=True)


@pytest.mark.parametrize("counts", FEW)
@pytest.mark.parametrize("K,N,act", [(200, 1544, "none"), (512, 4104, "swiglu"), (136, 2000, "silu"), (2304, 3592, "none")])
def test_shared_reduction_dgrad(counts, K, N, act):
    E, start, M, KZ, dy, x, w, z, real, dead = backward_case(FEW[counts], K, N, act, K, 1)
    status = epd.new_status()
    dx = torch.full((M, KZ), 7.0, dtype=torch.bfloat16, device=DEV)
    epd.ep_expert_matmul_dgrad(dy, w, i32(FEW[counts]), status, expert_start_loc=i32(start), activation=act,
                               preact=None if act == "none" else z, dx=dx)
    check_ok(status)
    d = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(d)
    for e, (s, c) in enumerate(zip(start, FEW[counts])):
        d[s:s + c] = dy[s:s + c].double() @ w[e].double()
        mag[s:s + c] = dy[s:s + c].double().abs() @ w[e].double().abs()
    zz = z.double().requires_grad_()
    a = act64(zz, act)
    slope, = torch.autograd.grad(a, zz, torch.where(dead.unsqueeze(1), 0.0, d)) if act != "none" else (d,)
    big, = torch.autograd.grad(act64(zz, act), zz, torch.ones_like(a)) if act != "none" else (torch.ones_like(d),)
    m2 = torch.cat([mag, mag], 1) if act == "swiglu" else mag
    d2 = torch.cat([d, d], 1) if act == "swiglu" else d
    tol = (N + 16) * 2.0 ** -23 * m2 * big.abs() + 2 ** -8 * slope.abs() + 16 * 2.0 ** -23 * d2.abs() * (1 + torch.cat([z, z], 1)[:, :KZ].double().abs()) ** 2 + 1e-30
    assert ((dx[real].double() - slope[real]).abs() <= tol[real]).all()
    assert (dx[dead] == 7).all()


@pytest.mark.parametrize("counts", [[1600], [3000, 70], [1537, 0, 1599], [5, 4000], [6145]])
@pytest.mark.parametrize("K,N", [(64, 72), (264, 256), (1000, 520)])
def test_shared_reduction_wgrad(counts, K, N):
    E, start, M, _, dy, x, w, z, real, dead = backward_case(counts, K, N, "none", K, 1)
    status = epd.new_status()
    dw, db = epd.ep_expert_matmul_wgrad(dy, x, i32(counts), status, expert_start_loc=i32(start), with_dbias=True)
    check_ok(status)
    for e, (s, c) in enumerate(zip(start, counts)):
        d, v = dy[s:s + c].double(), x[s:s + c].double()
        want = d.t() @ v
        tol = (c + 16) * 2.0 ** -23 * (d.abs().t() @ v.abs()) + 2 ** -8 * want.abs() + 1e-30
        assert ((dw[e].double() - want).abs() <= tol).all()
        assert ((db[e].double() - d.sum(0)).abs() <= (c + 16) * 2.0 ** -23 * d.abs().sum(0) + 1e-30).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [256, 2304])
def test_shared_reduction_with_more_tiles_than_clusters(fp8, N):
    """Regions may lie over one another, and then there are more tiles than rows in the buffer
    account for; both experts have the same weights, so that the order of their writes is no matter."""
    x, w, cnt, kw, real, y, z, ty, tz = forward_case([300], 4096, N, "none", 11, fp8=fp8)
    kw |= dict(expert_start_loc=i32([0, 0]))
    if fp8:
        kw["w_scale"] = kw["w_scale"].repeat(2, 1, 1)
    got = []
    for _ in range(2):
        status = epd.new_status()
        got.append(epd.ep_expert_matmul(x, w.repeat(2, 1, 1), i32([300, 300]), status, **kw)[0])
        check_ok(status)
        assert ((got[-1].double() - y).abs() <= ty)[real].all()
    again = []
    for _ in range(2):
        status = epd.new_status()
        again.append(epd.ep_expert_matmul(x, w, cnt, status, **(kw | dict(expert_start_loc=i32([0])) | (
            dict(w_scale=kw["w_scale"][:1].contiguous()) if fp8 else {})))[0])
        check_ok(status)
    assert torch.equal(again[0][real], again[1][real]), "the parts are added in a fixed order"


def test_backward_rectangles():
    counts, rect = [3, 0, 70, 128], 130
    E, start, M, KZ, dy, x, w, z, real, dead = backward_case(counts, 64, 96, "silu", 1, 0, rect)
    status = epd.new_status()
    dx = epd.ep_expert_matmul_dgrad(dy.view(E, rect, -1), w, i32(counts), status, activation="silu",
                                    preact=z.view(E, rect, -1))
    dw, _ = epd.ep_expert_matmul_wgrad(dy.view(E, rect, -1), x.view(E, rect, -1), i32(counts), status)
    flat = epd.ep_expert_matmul_dgrad(dy, w, i32(counts), status, expert_start_loc=i32(start), activation="silu", preact=z)
    fw, _ = epd.ep_expert_matmul_wgrad(dy, x, i32(counts), status, expert_start_loc=i32(start))
    check_ok(status)
    assert torch.equal(dx.view(M, -1)[real], flat[real]) and torch.equal(dw, fw)


def test_gradients_match_central_differences():
    """dgrad, wgrad and dbias of a layer against central differences of its 64-bit loss along
    random directions. The loss is linear in each argument, so the differences are exact but for
    64-bit rounding; each bf16 gradient is within 2^-9 of its exact value (and a 64-term fp32
    sum within 2^-17), so along v the two differ by at most 2^-8 of the sum of |gradient| |v|."""
    K, N, counts = 64, 64, [9, 0, 30]
    start, M = regions(counts, 0)
    g = gen(4)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(3, N, K, generator=g, device=DEV) / 8).to(torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    status = epd.new_status()
    dx = epd.ep_expert_matmul_dgrad(dy, w, i32(counts), status, expert_start_loc=i32(start))
    dw, db = epd.ep_expert_matmul_wgrad(dy, x, i32(counts), status, expert_start_loc=i32(start), with_dbias=True)
    check_ok(status)
    real = rows_of(start, counts)

    def loss(xx, ww, bb):
        return sum((dy[s:s + c].double() * (xx[s:s + c] @ ww[e].t() + bb[e])).sum()
                   for e, (s, c) in enumerate(zip(start, counts)))
    at = [x.double(), w.double(), torch.zeros(3, N, dtype=torch.float64, device=DEV)]
    for i, got in enumerate((dx, dw, db)):
        v = torch.randn(at[i].shape, generator=g, device=DEV).double()
        h = 1e-3
        up = loss(*[a + h * v if j == i else a for j, a in enumerate(at)])
        dn = loss(*[a - h * v if j == i else a for j, a in enumerate(at)])
        prod = got.double() * v
        prod = prod[real] if i == 0 else prod
        assert abs(float(prod.sum() - (up - dn) / (2 * h))) <= (2 ** -8 if i < 2 else 2 ** -17) * float(prod.abs().sum()) + 1e-6


def test_many_experts():
    """4096 experts of a few rows each: the walk over the counts goes in batches of 32."""
    counts = [(i * 2654435761 >> 7) % 4 for i in range(4096)]
    run_forward(counts, 64, 24, "gelu", seed=11, bias=True, gaps=1)
    run_forward(counts, 128, 128, "swiglu", seed=12, fp8=True)


def sampled(rows, n, seed):
    return torch.randint(0, rows, (n,), generator=gen(seed), device=DEV)


def test_offsets_beyond_32_bits():
    """Row buffers and weights of more than 2^32 elements: sampled rows of the last regions."""
    bf = dict(dtype=torch.bfloat16, device=DEV)
    M, K, N = 1_100_000, 64, 4096                       # y: 4.5e9 elements
    g = gen(21)
    x, w = torch.randn(M, K, generator=g, **bf), torch.randn(2, N, K, generator=g, **bf) / 8
    counts, start = [M - 300, 300], [300, 0]
    status = epd.new_status()
    y, z = epd.ep_expert_matmul(x, w, i32(counts), status, expert_start_loc=i32(start), with_preact=True,
                                activation="relu")
    check_ok(status)
    at = torch.cat([sampled(300, 8, 1), M - 1 - sampled(1000, 40, 2), 300 + sampled(M - 300, 40, 3)])
    want = torch.where((at < 300).unsqueeze(1), x[at].double() @ w[1].double().t(), x[at].double() @ w[0].double().t())
    tol = 2 ** -8 * want.abs() + 80 * 2.0 ** -23 * (x[at].double().abs() @ w[0].double().abs().t()) * 4
    assert ((z[at].double() - want).abs() <= tol).all() and ((y[at].double() - want.relu()).abs() <= tol).all()
    # the same buffer as dy: dx over 4096 columns, and the weights' gradients of 1.1 million rows
    dx = epd.ep_expert_matmul_dgrad(x, w.transpose(1, 2).contiguous(), i32(counts), status,
                                    expert_start_loc=i32(start), activation="relu", preact=z)
    check_ok(status)
    want = torch.where(z[at] > 0, want, 0.0)
    assert ((dx[at].double() - want).abs() <= tol).all()
    del y, z, dx
    E, K, N = 17, 16392, 16384                           # w: 4.6e9 elements
    w = torch.randn(E, N, K, generator=g, **bf) / 128
    x = torch.randn(E * 3, K, generator=g, **bf)
    y, _ = epd.ep_expert_matmul(x, w, i32([3] * E), status, expert_start_loc=i32([3 * e for e in range(E)]))
    check_ok(status)
    want = x[-3:].double() @ w[-1].double().t()
    mag = x[-3:].double().abs() @ w[-1].double().abs().t()
    assert ((y[-3:].double() - want).abs() <= 2 ** -8 * want.abs() + K * 2.0 ** -23 * mag).all()
    dw, _ = epd.ep_expert_matmul_wgrad(y, x, i32([3] * E), status, expert_start_loc=i32([3 * e for e in range(E)]))
    check_ok(status)
    rows = sampled(N, 64, 5)
    want = y[-3:, rows].double().t() @ x[-3:].double()
    assert ((dw[-1, rows].double() - want).abs() <= 2 ** -8 * want.abs() + 1e-4).all()


# ------------------------------------------------------------------------- combine backward
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (3, 1032, 5), (130, 2048, 8), (17, 7168, 8), (9, 264, 64), (4, 4104, 11)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_unpermute_backward(T, H, k, drop):
    g = gen(T + H)
    M = T * k + 3
    live = torch.rand(T, k, generator=g, device=DEV) >= drop
    index = torch.where(live, torch.randperm(M, generator=g, device=DEV)[:T * k].view(T, k).to(torch.int32), -1)
    w = torch.rand(T, k, generator=g, device=DEV)
    eo = torch.randn(M, H, generator=g, device=DEV).to(torch.bfloat16)
    gy = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    status = epd.new_status()
    geo = torch.full((M, H), 7.0, dtype=torch.bfloat16, device=DEV)
    _, gw = epd.ep_unpermute_backward(gy, eo, index, w, status, grad_expert_out=geo)
    check_ok(status)
    filled = torch.zeros(M, dtype=torch.bool, device=DEV)
    for t in range(T):
        for j in range(k):
            s = int(index[t, j])
            if s < 0:
                assert float(gw[t, j]) == 0
                continue
            filled[s] = True
            want = w[t, j].double() * gy[t].double()
            assert ((geo[s].double() - want).abs() <= 2 ** -8 * want.abs()).all()
            a, b = gy[t].double(), eo[s].double()
            assert abs(float(gw[t, j].double() - a @ b)) <= (H + 1) * 2.0 ** -24 * float(a.abs() @ b.abs())
    assert (geo[~filled] == 7).all()


def test_unpermute_backward_offsets_beyond_32_bits():
    T, H, k = 300, 8192, 2
    M = 530_000                                          # 4.3e9 elements
    eo = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
    index = (M - 1 - torch.randperm(T * k, generator=gen(1), device=DEV)).view(T, k).to(torch.int32)
    eo[M - T * k:] = torch.randn(T * k, H, generator=gen(2), device=DEV).to(torch.bfloat16)
    gy = torch.randn(T, H, generator=gen(3), device=DEV).to(torch.bfloat16)
    w = torch.rand(T, k, generator=gen(4), device=DEV)
    status = epd.new_status()
    geo, gw = epd.ep_unpermute_backward(gy, eo, index, w, status)
    check_ok(status)
    at = index.long()
    want = w.double().unsqueeze(2) * gy.double().unsqueeze(1)
    assert ((geo[at].double() - want).abs() <= 2 ** -8 * want.abs()).all()
    dot = (eo[at].double() * gy.double().unsqueeze(1)).sum(2)
    mag = (eo[at].double() * gy.double().unsqueeze(1)).abs().sum(2)
    assert ((gw.double() - dot).abs() <= (H + 1) * 2.0 ** -24 * mag).all()


def test_unpermute_backward_reports_slots_outside():
    index = torch.tensor([[0, 5], [-2, 1]], dtype=torch.int32, device=DEV)
    eo = torch.randn(3, 64, device=DEV).to(torch.bfloat16)
    gy = torch.randn(2, 64, device=DEV).to(torch.bfloat16)
    status = epd.new_status()
    _, gw = epd.ep_unpermute_backward(gy, eo, index, torch.ones(2, 2, device=DEV), status)
    torch.cuda.synchronize()
    assert int(status.item()) == epd.EPD_ERR_CAPACITY
    assert gw[0, 1] == 0 and gw[1, 0] == 0 and gw[0, 0] != 0


# ------------------------------------------------------------------------- streams, graphs, refusals
def test_operators_on_another_stream_and_in_a_graph():
    counts, K, N = [40, 0, 90], 256, 128
    x, w, cnt, kw, real, y, z, ty, tz = forward_case(counts, K, N, "swiglu", 9, bias=True)
    l = torch.randn(64, 16, device=DEV)
    status = epd.new_status()
    out = torch.zeros(x.shape[0], N, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(64, 2, dtype=torch.int64, device=DEV)
    wt = torch.zeros(64, 2, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    epd.ep_expert_matmul(x, w, cnt, status, y=out, stream=side, **kw)
    epd.ep_route(l, 2, status, topk_idx=idx, topk_weights=wt, stream=side)
    side.synchronize()
    first, first_idx = out.clone(), idx.clone()
    assert ((first[real].double() - y[real]).abs() <= ty[real]).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        epd.ep_route(l, 2, status, topk_idx=idx, topk_weights=wt)
        epd.ep_expert_matmul(x, w, cnt, status, y=out, **kw)
    out.zero_()
    idx.zero_()
    for _ in range(3):
        graph.replay()
    check_ok(status)
    assert torch.equal(out[real], first[real]) and torch.equal(idx, first_idx)


def test_refusals():
    s = epd.new_status()
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, w = torch.zeros(16, 64, **bf), torch.zeros(2, 32, 64, **bf)
    c, o = i32([4, 4]), i32([0, 8])
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x, w, c, s)                                      # no starts
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x, w, c, s, expert_start_loc=o, activation="tanh")
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x.float(), w, c, s, expert_start_loc=o)
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x, w[:, :, :56].contiguous(), c, s, expert_start_loc=o)
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x.t().contiguous().t(), w, c, s, expert_start_loc=o)   # strided rows
    with pytest.raises(epd.EpdError):                                         # N % 8
        epd.ep_expert_matmul(x, torch.zeros(2, 24, 64, **bf), c, s, expert_start_loc=o, activation="swiglu")
    with pytest.raises(epd.EpdError):                                         # K % 8
        epd.ep_expert_matmul(torch.zeros(16, 60, **bf), torch.zeros(2, 32, 60, **bf), c, s, expert_start_loc=o)
    with pytest.raises(ValueError):
        epd.ep_expert_matmul(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), c, s, expert_start_loc=o)
    with pytest.raises(ValueError):
        epd.ep_expert_matmul_dgrad(torch.zeros(16, 32, **bf), w, c, s, expert_start_loc=o, preact=x)
    with pytest.raises(TypeError):
        epd.ep_expert_matmul_dgrad(torch.zeros(16, 32, **bf), w, c, s, expert_start_loc=o, activation="silu")
    with pytest.raises(ValueError):
        epd.ep_expert_matmul_wgrad(torch.zeros(15, 32, **bf), x, c, s, expert_start_loc=o)
    l = torch.zeros(4, 12, device=DEV)
    for kw in (dict(num_topk=13), dict(num_topk=0), dict(num_topk=2, num_groups=5),
               dict(num_topk=2, num_groups=4, topk_groups=5)):
        with pytest.raises(epd.EpdError):
            epd.ep_route(l, status=s, **kw)
    with pytest.raises(ValueError):
        epd.ep_route(l, 2, s, scoring="tanh")
    with pytest.raises(ValueError):
        epd.ep_route(l.half(), 2, s)
    with pytest.raises(ValueError):
        epd.ep_route_backward(torch.zeros(4, 3, device=DEV), l, torch.zeros(4, 2, dtype=torch.int64, device=DEV), s)
    with pytest.raises(ValueError):
        epd.ep_unpermute_backward(torch.zeros(3, 64, **bf), x, i32([[0], [1]]), torch.zeros(2, 1, device=DEV), s)
    torch.cuda.synchronize()
    assert int(s.item()) == 0


def test_no_rows_at_all():
    s = epd.new_status()
    bf = dict(dtype=torch.bfloat16, device=DEV)
    y, _ = epd.ep_expert_matmul(torch.zeros(0, 64, **bf), torch.ones(2, 32, 64, **bf), i32([0, 0]), s,
                                expert_start_loc=i32([0, 0]))
    assert y.shape == (0, 32)
    dw, db = epd.ep_expert_matmul_wgrad(torch.zeros(0, 32, **bf), torch.zeros(0, 64, **bf), i32([0, 0]), s,
                                        expert_start_loc=i32([0, 0]), with_dbias=True)
    assert (dw == 0).all() and (db == 0).all()
    idx, w = epd.ep_route(torch.zeros(0, 8, device=DEV), 2, s)
    assert idx.shape == (0, 2)
    assert epd.ep_route_backward(w, torch.zeros(0, 8, device=DEV), idx, s).shape == (0, 8)
    check_ok(s)
