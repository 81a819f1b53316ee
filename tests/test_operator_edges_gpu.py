"""The router, the products and their gradients at the ends of their ranges, against plain
definitions in 64 bits."""
import math

import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd
from test_operators_gpu import (DEV, INF, backward_case, check_ok, forward_case, gen, i32, route_inputs,
                                route_ref)

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23     # of a 32-bit value, at most
TINY = 2.0 ** -149   # spacing of 32-bit values near zero
TINY_BF16 = 2.0 ** -133


def uniform(shape, lo, hi, seed):
    return lo + (hi - lo) * torch.rand(shape, generator=gen(seed), device=DEV)


# Where a sigmoid's rows lie: near one, where 1 - s is far smaller than s, near zero, where s falls
# below the smallest normal number, and rows with both.
SATURATED = {"high": (8.0, 20.0), "very high": (20.0, 60.0), "low": (-100.0, -80.0), "lowest": (-103.0, -88.5),
             "wide": (-100.0, 20.0)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", SATURATED)
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(70, 24, 4), (9, 600, 40), (5, 8, 1)])
def test_route_backward_of_saturated_sigmoids(dtype, rows, renorm, T, E, k):
    """Within a few units in the last place of dl = ds s (1 - s), and finite. s, 1 - s and a
    weight p are each within 8 units; a weight of picks that differ by d in their logits within
    d / 2 units more (the rounding of the difference), and its sum over the picks adds k."""
    l = uniform((T, E), *SATURATED[rows], T).to(dtype)
    idx = torch.rand(T, E, generator=gen(E), device=DEV).topk(k, 1).indices
    g = 1.5 * torch.sign(torch.randn(T, k, generator=gen(k), device=DEV)) + 0.25 * torch.randn(T, k, generator=gen(3), device=DEV)
    status = epd.new_status()
    d = epd.ep_route_backward(g, l, idx, status, scoring="sigmoid", renormalize=renorm, routed_scale=2.0)
    check_ok(status)
    x = l.double().gather(1, idx)
    s, c, g = torch.sigmoid(x), torch.sigmoid(-x), 2.0 * g.double()
    if renorm:
        p = s / s.sum(1, keepdim=True)
        apart = g.unsqueeze(2) - g.unsqueeze(1)
        pick = (apart * p.unsqueeze(1)).sum(2) * p * c
        far = x.amax(1, keepdim=True) - x
        bound = (apart.abs() * p.unsqueeze(1)).sum(2) * p * c * (k + 32 + far + far.amax(1, keepdim=True)) * ULP
        bound = bound + 8 * apart.abs().amax(2) * TINY   # a weight below the smallest normal number
    else:
        pick = g * s * c
        bound = pick.abs() * 24 * ULP + 4 * g.abs() * TINY
    want = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter(1, idx, pick)
    tol = torch.zeros_like(want).scatter(1, idx, bound + 2 * TINY)
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2 ** -8 + TINY_BF16 * (want != 0)
    assert torch.isfinite(d).all()
    assert ((d.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ahead", [0.0, 6.0, 12.0, 18.0, 40.0])
@pytest.mark.parametrize("T,E,k", [(40, 256, 1), (33, 64, 6), (6, 1030, 40), (9, 5, 5)])
def test_route_backward_of_confident_softmax(dtype, ahead, T, E, k):
    """One logit of every row lies `ahead` of the others: 1 - s of it is far smaller than s.
    dl_e = sum over i of s_e s_i (ds_e - ds_i), each product within the roundings of its two
    scores (16 units, and half a unit for each unit that the logit lies below the row's largest)
    and of the sum of E terms in the order of a tree and per lane (E / 32 + k + 8)."""
    l = torch.randn(T, E, generator=gen(T), device=DEV)
    top = torch.randint(0, E, (T, 1), generator=gen(E), device=DEV)
    l = l.scatter_add(1, top, torch.full((T, 1), ahead, device=DEV)).to(dtype)
    # the confident expert first among the picks of even rows, left out of the others'
    order = torch.rand(T, E, generator=gen(7), device=DEV)
    order = order.scatter(1, top, torch.where(torch.arange(T, device=DEV) % 2 == 0, 2.0, -1.0).unsqueeze(1))
    idx = order.topk(k, 1).indices
    if k > 2:
        idx[:, 2] = idx[:, 0]      # picked twice
        idx[1::3, 1] = -1
    g = torch.randn(T, k, generator=gen(k), device=DEV)
    status = epd.new_status()
    d = epd.ep_route_backward(g, l, idx, status, scoring="softmax", renormalize=False)
    check_ok(status)
    x = l.double()
    s = torch.softmax(x, 1)
    ds = torch.zeros_like(s).scatter_add(1, idx.clamp(min=0), torch.where(idx >= 0, g.double(), 0.0))
    want, bound = torch.zeros_like(s), torch.zeros_like(s)
    for e in range(E):
        term = s[:, e:e + 1] * s * (ds[:, e:e + 1] - ds)
        want[:, e], bound[:, e] = term.sum(1), term.abs().sum(1)
    # duplicate picks are summed first, in 32 bits
    dup = torch.zeros_like(s).scatter_add(1, idx.clamp(min=0), torch.where(idx >= 0, g.double().abs(), 0.0)).amax(1, keepdim=True)
    far = (x.amax(1, keepdim=True) - x).amax(1, keepdim=True)
    others = torch.stack([s[:, torch.arange(E, device=DEV) != e].sum(1) for e in range(E)], 1)
    tol = bound * (E / 32 + k + 40 + far) * ULP + 2 * ULP * dup * s * others + 4 * TINY
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2 ** -8 + TINY_BF16
    assert ((d.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows", ["low", "lowest", "wide"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k", [(70, 24, 4), (9, 600, 40), (5, 8, 1)])
def test_route_weights_of_low_sigmoids(rows, renorm, biased, T, E, k):
    """Scores below the smallest normal number are numbers all the same, and so are their shares."""
    l = uniform((T, E), *SATURATED[rows], T)
    bias = 2.0 * torch.randperm(E, generator=gen(E), device=DEV).float() if biased else None
    status = epd.new_status()
    idx, w = epd.ep_route(l, k, status, scoring="sigmoid", bias=bias, renormalize=renorm)
    check_ok(status)
    x = l.double()
    order = (torch.sigmoid(x) + bias.double() if biased else x).sort(dim=1, descending=True, stable=True).indices
    assert torch.equal(idx, order[:, :k])
    s = torch.sigmoid(x).gather(1, idx)
    if renorm:
        s = s / s.sum(1, keepdim=True)
        # the roundings of a score and of the sum, and half a unit for each unit that a logit lies
        # below the largest (no more than 120)
        tol = s * (k + 24 + 64) * ULP + 6 * TINY
    else:
        tol = s * 8 * ULP + 3 * TINY
    assert ((w.double() - s).abs() <= tol).all()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [2, 3, 8])
def test_route_ranks_groups_of_low_scores(scoring, size):
    """A group's score is within a few units in the last place of the sum of its two best scores,
    however low: of two groups with one expert each the one whose logit is the next larger
    number is kept. (That is sixteen units of the score or more from 16 on.)"""
    low = torch.cat([uniform((400,), -80, -16, 1), -torch.arange(17, 80, device=DEV).float()])
    T = low.shape[0]
    up = torch.nextafter(low, torch.zeros_like(low))
    l = torch.full((T, 4 * size), -INF, device=DEV)
    l[:, 0] = 0.0                        # the row's largest, kept always
    l[:, size], l[:, 2 * size + 1] = low, up
    status = epd.new_status()
    idx, _ = epd.ep_route(l, 2, status, scoring=scoring, num_groups=4, topk_groups=2, group_score="top2")
    check_ok(status)
    assert (idx[:, 0] == 0).all()
    assert (idx[:, 1] == 2 * size + 1).all()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_chooses_by_exact_scores(scoring):
    """With a bias of zero the choice goes by the 32-bit scores, which tell logits apart that
    differ by sixteen units of their score or more."""
    low = uniform((300,), -80, -16, 2)
    l = torch.full((300, 12), -INF, device=DEV)
    l[:, 3], l[:, 4], l[:, 9] = low, torch.nextafter(low, torch.zeros_like(low)), 0.0
    status = epd.new_status()
    idx, _ = epd.ep_route(l, 2, status, scoring=scoring, bias=torch.zeros(12, device=DEV))
    check_ok(status)
    assert (idx == torch.tensor([9, 4], device=DEV)).all()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,gs", [(1, "max"), (4, "top2"), (3, "top2"), (6, "max")])
@pytest.mark.parametrize("E", [24, 48, 312])
def test_route_reports_nan_bias(scoring, groups, gs, E):
    """A NaN bias is reported, and its expert cannot be chosen nor count for its group."""
    l = torch.randn(50, E, generator=gen(E), device=DEV)
    bias = torch.randint(-2, 3, (E,), generator=gen(2), device=DEV).float()
    gone = torch.arange(E, device=DEV) % 5 == 0
    keep = max(1, groups // 2)
    want_status, status = epd.new_status(), epd.new_status()
    opts = dict(scoring=scoring, num_groups=groups, topk_groups=keep, group_score=gs)
    want, ww = epd.ep_route(l, 4, want_status, bias=torch.where(gone, -INF, bias), **opts)
    check_ok(want_status)
    got, gw = epd.ep_route(l, 4, status, bias=torch.where(gone, math.nan, bias), **opts)
    torch.cuda.synchronize()
    assert int(status.item()) == epd.EPD_ERR_NONFINITE
    assert not (got % 5 == 0).any()
    assert torch.equal(got, want) and torch.equal(gw, ww)


LOWEST = torch.finfo(torch.bfloat16).min


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
def test_dgrad_of_lowest_preactivations(act):
    """A pre-activation of the type's lowest value has no slope, whatever it is multiplied by."""
    counts, K, N = [5, 0, 20], 64, 64
    E, start, M, KZ, dy, x, w, z, real, dead = backward_case(counts, K, N, act, 3, 0)
    z[:, 0:KZ:3] = LOWEST                       # gates, and for swiglu up features too
    if act == "swiglu":
        z[:, K:2 * K:4] = -LOWEST
        z[:, 1] = LOWEST
        z[:, K + 1] = LOWEST
    dy = (dy.float() * 8).to(torch.bfloat16)
    status = epd.new_status()
    dx = epd.ep_expert_matmul_dgrad(dy, w, i32(counts), status, expert_start_loc=i32(start), activation=act, preact=z)
    check_ok(status)
    gate = z[real][:, :K].float() == LOWEST
    assert (dx[real][:, :K][gate] == 0).all()
    if act == "swiglu":
        assert (dx[real][:, K:][gate] == 0).all()
    assert not torch.isnan(dx[real].float()).any()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("fp8", [False, True])
def test_product_of_lowest_preactivations(act, fp8):
    counts, K, N = [5, 0, 20], 128, 128
    x, w, cnt, kw, real, *_ = forward_case(counts, K, N, act, 4, fp8=fp8, bias=True)
    kw["bias"][:, :N] = torch.finfo(torch.float32).min
    status = epd.new_status()
    y, _ = epd.ep_expert_matmul(x, w, cnt, status, **kw)
    check_ok(status)
    assert (y[real] == 0).all()


def choice64(l, scoring, bias):
    """One row in 64 bits: logits, scores, and what the choice goes by (-inf: cannot be chosen)."""
    row = [v if v < INF else -INF for v in l.double().tolist()]
    m = max(row)
    if scoring == "sigmoid":
        s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in row]
    else:
        ex = [math.exp(v - m) if m > -INF else 0.0 for v in row]
        s = [v / max(sum(ex), 1e-300) for v in ex]
    c = [-INF if v == -INF else a + b for v, a, b in zip(row, s, bias or [0.0] * len(row))]
    return row, s, c


@pytest.mark.parametrize("T,E,k,groups,keep,gs", [
    (64, 256, 8, 8, 4, "top2"), (33, 60, 6, 6, 2, "max"), (17, 600, 40, 40, 7, "top2"), (21, 96, 7, 3, 3, "top2"),
    (5, 1030, 9, 2, 1, "top2")])
@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked,dtype", [(False, torch.float32), (True, torch.float32), (True, torch.bfloat16)])
def test_route_every_row(T, E, k, groups, keep, gs, scoring, biased, renorm, masked, dtype):
    """Every row's picks are right to within the roundings of the 32-bit scores, and its weights
    are those of its picks. A score is within 8 units, so two sums of two differ by 32 at most;
    a whole bias of up to 2 makes a value of up to 3, and a sum of up to 6, which round by 2^-23
    and 2^-22: 2^-20 for the two. Values nearer than `near` may come in either order, and where
    none are the picks are the 64-bit ones exactly."""
    l = route_inputs(T, E, dtype, T * 5 + E, masked)
    bias = torch.randint(-2, 3, (E,), generator=gen(E), device=DEV).float() if biased else None
    status = epd.new_status()
    idx, w = epd.ep_route(l, k, status, scoring=scoring, bias=bias, num_groups=groups, topk_groups=keep,
                          group_score=gs, renormalize=renorm, routed_scale=1.5)
    check_ok(status)
    ri, _ = route_ref(l, k, scoring, bias, groups, keep, gs, renorm, 1.5)
    l, idx, w = l.cpu(), idx.cpu(), w.cpu()
    bias = None if bias is None else bias.double().tolist()
    size, exact = E // groups, 0
    for t in range(T):
        row, s, c = choice64(l[t], scoring, bias)
        near = (2.0 ** -20 if biased else 0.0) + 32 * ULP * max(s)
        got = idx[t].tolist()
        n = sum(e >= 0 for e in got)
        assert all(e == -1 for e in got[n:]) and len(set(got[:n])) == n
        assert all(0 <= e < E and c[e] > -INF for e in got[:n])
        two = []
        for g in range(groups):
            own = sorted((v for v in c[g * size:(g + 1) * size] if v > -INF), reverse=True)
            two.append(sum(own[:2] if gs == "top2" else own[:1]) if own else -INF)
        cut = sorted(two, reverse=True)[keep - 1]
        sure = [g for g in range(groups) if two[g] > cut + near] if keep < groups else range(groups)
        used = {e // size for e in got[:n]}
        assert len(used) <= keep and all(two[g] >= cut - near for g in used)
        order = row if scoring == "softmax" and not biased else c
        assert all(order[a] >= order[b] - near for a, b in zip(got[:n], got[1:n]))
        kept = [e for g in sure for e in range(g * size, (g + 1) * size) if c[e] > -INF]
        assert n >= min(k, len(kept))
        if n == k:
            assert all(e in got or order[e] <= order[got[-1]] + near for e in kept)
        close = keep < groups and any(0 < abs(v - cut) <= near for v in two)
        live = sorted(order)
        if not close and not any(0 < b - a <= near for a, b in zip(live, live[1:])):
            assert got == ri[t].tolist()
            exact += 1
        total = sum(s[e] for e in got[:n])
        for j, e in enumerate(got):
            want = 0.0 if e < 0 or (renorm and total == 0) else s[e] * 1.5 / (total if renorm else 1.0)
            assert abs(float(w[t, j]) - want) <= (k + 24) * ULP * 1.5
    if scoring == "softmax" and not biased and (gs == "max" or keep == groups):
        assert exact == T


@pytest.mark.parametrize("few,many", [(1600, 8 * 1600), (300, 40 * 300)])
def test_the_same_rows_in_a_larger_buffer(few, many):
    """A call repeats itself to the bit; the same rows in a buffer of another size may be added up
    in other parts, and are within the roundings of the sums."""
    K, N = 4096, 512
    g = gen(few)
    x = torch.randn(few, K, generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn(few, N, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(1, N, K, generator=g, device=DEV) / 64).to(torch.bfloat16)
    out = []
    for cap in (few, few, many):
        xx, yy = torch.full((cap, K), math.nan, dtype=x.dtype, device=DEV), torch.full((cap, N), math.nan, dtype=x.dtype, device=DEV)
        xx[:few], yy[:few] = x, dy
        status, rows = epd.new_status(), dict(expert_start_loc=i32([0]))
        y, _ = epd.ep_expert_matmul(xx, w, i32([few]), status, **rows)
        dx = epd.ep_expert_matmul_dgrad(yy, w, i32([few]), status, **rows)
        dw, db = epd.ep_expert_matmul_wgrad(yy, xx, i32([few]), status, with_dbias=True, **rows)
        check_ok(status)
        out.append((y[:few], dx[:few], dw, db))
    assert all(torch.equal(a, b) for a, b in zip(out[0], out[1]))
    X, D, W = x.double(), dy.double(), w[0].double()
    for got in (out[0], out[2]):
        for v, a, b, n in ((got[0], X, W.t(), K), (got[1], D, W, N), (got[2][0], D.t(), X, few)):
            want = a @ b
            assert ((v.double() - want).abs() <= 2 ** -8 * want.abs() + (n + 16) * ULP * (a.abs() @ b.abs())).all()
        assert ((got[3][0].double() - D.sum(0)).abs() <= (few + 16) * ULP * D.abs().sum(0)).all()


@pytest.mark.parametrize("counts", [[16], [0], [3, 0, 5000, 70, 1], [1500, 1600, 24 * 64 - 1, 24 * 64]])
@pytest.mark.parametrize("K,N", [(64, 64), (256, 256)])
def test_wgrad_of_few_rows_in_a_large_buffer(counts, K, N):
    """Whether an expert's reduction is shared goes by the rows it has, not by the buffer's: experts
    that share theirs beside some that do not, and tiles past the first."""
    g = gen(sum(counts))
    cap = max(sum(counts), 4096 * len(counts))
    start = [sum(counts[:e]) for e in range(len(counts))]
    x = torch.full((cap, K), math.nan, dtype=torch.bfloat16, device=DEV)
    dy = torch.full((cap, N), math.nan, dtype=torch.bfloat16, device=DEV)
    n = sum(counts)
    x[:n], dy[:n] = torch.randn(n, K, generator=g, device=DEV), torch.randn(n, N, generator=g, device=DEV)
    status = epd.new_status()
    dw, db = epd.ep_expert_matmul_wgrad(dy, x, i32(counts), status, expert_start_loc=i32(start), with_dbias=True)
    check_ok(status)
    for e, (s, c) in enumerate(zip(start, counts)):
        a, b = dy[s:s + c].double(), x[s:s + c].double()
        want = a.t() @ b
        assert ((dw[e].double() - want).abs() <= (c + 16) * ULP * (a.abs().t() @ b.abs()) + 2 ** -8 * want.abs()).all()
        assert ((db[e].double() - a.sum(0)).abs() <= (c + 16) * ULP * a.abs().sum(0)).all()


def test_as_many_rows_as_a_buffer_may_have():
    """2^31 - 1 rows of one expert: row numbers of the last steps and tiles reach 2^31. All but a
    few rows are zero, and the values are whole, so that every sum is exact."""
    M, K, N = 2 ** 31 - 1, 8, 8
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("needs 103 GB on the device")
    g = gen(31)
    at = torch.cat([torch.tensor([0, 1, 63, 12_345_678, 2 ** 30], device=DEV), torch.arange(M - 300, M, device=DEV)])
    x, dy = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    x[at] = torch.randint(-4, 5, (len(at), K), generator=g, device=DEV).to(torch.bfloat16)
    dy[at] = torch.randint(-4, 5, (len(at), N), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randint(-4, 5, (1, N, K), generator=g, device=DEV).to(torch.bfloat16)
    status, rows = epd.new_status(), dict(expert_start_loc=i32([0]))
    dw, db = epd.ep_expert_matmul_wgrad(dy, x, i32([M]), status, with_dbias=True, **rows)
    check_ok(status)
    assert torch.equal(dw[0], (dy[at].double().t() @ x[at].double()).to(torch.bfloat16))
    assert torch.equal(db[0].double(), dy[at].double().sum(0))
    y, _ = epd.ep_expert_matmul(x, w, i32([M]), status, **rows)
    check_ok(status)
    assert torch.equal(y[at], (x[at].double() @ w[0].double().t()).to(torch.bfloat16))
    assert (y[2 ** 20:2 ** 20 + 4096] == 0).all() and (y[M - 5000:M - 300] == 0).all()
