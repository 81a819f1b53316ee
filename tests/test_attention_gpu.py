"""Decode attention over the paged cache on the GPU against the formula in 64 bits.

Tolerances: half a step of bf16 for the output, and the weights' relative error times the sum of
weight * |value|. The weights: a score's fp32 sum over D products of size |q| |k| (below 2^4 after
the scale, 2^-24 for each of D / 16 + 4 additions in a chain: 2^-15.6 at most), the exponential 2^-22,
the weights' two bf16 parts 2^-15 (what is left of the first is below 2^-7 of the weight, and half a
step of the second is 2^-8 of that), 2^-14.3 together. In an e4m3 cache they are one fp16 part instead:
half a step is finfo(float16).eps / 2 = 2^-11 of the weight, and that comes on top.
lse: the same 2^-14, and its own rounding."""
import math

import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd
from cache_formulas import attend, paged, values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(999 + seed)
    return g


def check(lengths, page, KH, G, D, fp8=False, window=0, scale=None, order="page,row,head", seed=0, workspace=None,
          q_scale=1.0, garbage=True, v_spread=False, v_power=0):
    g = gen(seed)
    B, QH = len(lengths), KH * G
    most = max(1, -(-max(lengths) // page))
    pages = B * most
    k, v, ks, vs = paged(pages, page, KH, D, fp8, DEV, g, order)
    if v_spread:  # values' scales over ten powers of two
        vs *= torch.exp2(10 * torch.rand(vs.shape, generator=g, device=DEV) - 5)
    if v_power:  # very small or large values
        (vs if fp8 else v).mul_(2.0 ** v_power)
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, most)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    # one projection's rows: the queries are slices of them
    q = (torch.randn(B, QH + 2, D, generator=g, device=DEV) * q_scale).to(torch.bfloat16)[:, 1:QH + 1]
    want, lse = attend(q, values(k, ks), values(v, vs), table, lens, scale, window)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), table, lens, scale, window)
    if garbage:  # what is not live may hold anything
        at = torch.arange(most * page, device=DEV)
        dead = (at >= lens[:, None]) | ((at < lens[:, None] - window) if window else False)
        where = table[:, at // page].long()[dead], (at % page).expand(B, -1)[dead]
        for t in (k, v):
            if fp8:
                t.view(torch.uint8)[where] = 0x7F
            else:
                t[where] = float("nan")
        if fp8:
            ks[where], vs[where] = float("nan"), float("inf")
        table[(at[::page] >= lens[:, None])] = 10**9
    status = epd.new_status(DEV)
    if workspace is None:
        workspace = epd.new_attention_workspace(B, QH, KH, D, DEV)
    kw = dict(k_scale=ks, v_scale=vs, softmax_scale=scale, window=window, with_lse=True)
    out, got_lse = epd.ep_decode_attention(q, k, v, table, lens, workspace, status, **kw)
    assert int(status) == 0
    # (2^-134: half a step of the smallest bf16)
    tol = 2.0 ** -134 + 2.0 ** -8 * want.abs() + (2.0 ** -14 + (2.0 ** -11 if fp8 else 0)) * size
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
    empty = lens <= 0
    assert bool((out[empty] == 0).all()) and bool((got_lse[empty] == -float("inf")).all())
    live = ~empty
    assert bool(((got_lse[live].double() - lse[live]).abs() <= 2.0 ** -14 + 2.0 ** -23 * lse[live].abs()).all())
    again, lse2 = epd.ep_decode_attention(q, k, v, table, lens, workspace, status, **kw)
    assert torch.equal(out, again) and torch.equal(got_lse, lse2)
    return workspace


RAGGED = [0, 1, 15, 16, 17, 127, 128, 129, 1000, 2, 0, 333]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("KH,G", [(1, 1), (2, 4), (3, 7), (1, 16), (2, 17), (1, 40), (8, 8)])
def test_heads(KH, G, D, fp8):
    check(RAGGED, 16, KH, G, D, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order", ["page,row,head", "page,head,row"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 500])
def test_pages(page, order, fp8):
    check(RAGGED, page, 2, 8, 128, fp8, order=order, seed=page)


def test_odd_head():
    check(RAGGED, 5, 2, 3, 8)
    check(RAGGED, 5, 2, 3, 200)
    check(RAGGED, 5, 2, 3, 112, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 5000])
def test_window(window, fp8):
    check(RAGGED + [5000], 16, 2, 4, 128, fp8, window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 0], [5], [16 * 128], [100_003], [70_000, 3, 0, 20_001], [4097] * 3])
def test_lengths(lengths, fp8):
    check(lengths, 64, 2, 8, 128, fp8)
    check(lengths, 64, 1, 4, 64 if fp8 else 256, fp8)


@pytest.mark.parametrize("B", [151, 152, 153, 256, 257, 700])
def test_many_sequences(B):
    check([(i * 37) % 300 for i in range(B)], 16, 2, 4, 64, seed=B)


MIXED = {  # of few and many tiles, between lengths that no block takes alone
    "short": [(i * 97) % 200 for i in range(60)],
    "one long": [5] * 20 + [3001] + [0, 700] * 12,
    "long first": [3900, 1, 2, 3] + [600] * 36,
    "equal": [513] * 41,
    "few": [2000, 100, 511, 512, 513, 0, 1, 33],
}


@pytest.mark.parametrize("order", ["page,row,head", "page,head,row"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("KH,G,D", [(8, 4, 128), (8, 16, 64), (8, 1, 256), (4, 12, 256), (6, 8, 128), (16, 2, 80), (12, 9, 128)])
@pytest.mark.parametrize("lengths", list(MIXED))
def test_heads_together(lengths, KH, G, D, fp8, order):
    """Several kv heads of a sequence at once, in one block and shared by many."""
    check(MIXED[lengths], 16, KH, G, D, fp8, order=order, seed=KH)


@pytest.mark.parametrize("fp8", [False, True])
def test_heads_together_paged(fp8):
    for page in (1, 7, 64):
        check(MIXED["one long"], page, 8, 4, 128, fp8, window=333 if page == 7 else 0, seed=page)
        check(MIXED["long first"], page, 8, 8, 64, fp8, window=2500 if page == 64 else 0, seed=page)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_of_heads_together(fp8):
    g = gen(12)
    B, KH, G, D, page = 48, 8, 4, 128, 16
    k, v, ks, vs = paged(4 * B, page, KH, D, fp8, DEV, g)
    table = torch.randperm(4 * B, generator=g, device=DEV).int().view(B, 4)
    lens = torch.full((B,), 64, dtype=torch.int32, device=DEV)
    q = torch.randn(B, KH * G, D, generator=g, device=DEV).bfloat16()
    ws, st = epd.new_attention_workspace(B, KH * G, KH, D, DEV), epd.new_status(DEV)
    full, _ = epd.ep_decode_attention(q, k, v, table, lens, ws, st, k_scale=ks, v_scale=vs)
    assert int(st) == 0
    table[7, 2], table[40, 0] = 4 * B, -5
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, ws, st, k_scale=ks, v_scale=vs)
    assert int(st) == epd.EPD_ERR_CAPACITY
    good = torch.ones(B, dtype=torch.bool, device=DEV)
    good[[7, 40]] = False
    assert torch.equal(out[good], full[good])
    # as if the page's positions were not there
    for b, rest in ((7, [0, 1, 3]), (40, [1, 2, 3])):
        want, _ = attend(q[b:b + 1], values(k, ks), values(v, vs), table[b:b + 1, rest], lens[:1] - page)
        size, _ = attend(q[b:b + 1], values(k, ks), values(v, vs).abs(), table[b:b + 1, rest], lens[:1] - page)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -14 + (2.0 ** -11 if fp8 else 0)) * size
        assert bool(((out[b].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("power", [-125, -60, 60])
def test_values_of_all_sizes(power):
    """Values, and the scales of an e4m3 cache's, down to numbers below the smallest normal one."""
    check([700, 33, 4000], 16, 2, 4, 128, True, v_power=power)
    check([700, 33, 4000], 16, 2, 4, 128, False, v_power=power)


def test_queries_of_all_sizes():
    for fp8 in (False, True):
        check([700, 33], 16, 2, 4, 128, fp8, q_scale=2.0 ** 115, scale=2.0 ** -118)
        check([700, 33], 16, 2, 4, 128, fp8, q_scale=2.0 ** -115, scale=2.0 ** 112)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [8, 16])
def test_heads_of_a_group_stand_alone(G, fp8):
    """Queries of infinities, NaN and of very different sizes beside one another, over the same keys."""
    g = gen(13)
    KH, D, n = 2, 128, 300
    k, v, ks, vs = paged(n, 1, KH, D, fp8, DEV, g)
    k[..., 0] = 0
    q = torch.randn(1, KH * G, D, generator=g, device=DEV).bfloat16()
    q[0, 1] = float("inf")
    q[0, 2, 7] = float("nan")
    q[0, 3, 0] = 2.0 ** 100  # of no weight: the keys are 0 there
    q[0, 5] *= 2.0 ** -60
    q[0, G + 4, 5] = -float("inf")
    table, lens = torch.arange(n, dtype=torch.int32, device=DEV).view(1, n), torch.tensor([n], dtype=torch.int32, device=DEV)
    st = epd.new_status(DEV)
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, epd.new_attention_workspace(1, KH * G, KH, D, DEV), st, k_scale=ks, v_scale=vs)
    bad = [1, 2, G + 4]
    good = [h for h in range(KH * G) if h not in bad + [3]]
    assert int(st) == 0 and bool(out[0, bad].isnan().all())
    want, _ = attend(q, values(k, ks), values(v, vs), table, lens)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), table, lens)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -14 + (2.0 ** -11 if fp8 else 0)) * size
    assert bool(((out.double() - want).abs() <= tol)[0, good].all())


def test_many_small_weights():
    """One token of weight one among 2^17 of 2^-25.5 whose values count for more: the fp16 weights hold
    them (to half a step, 2^-34 of the largest weight, times their number and value)."""
    n, D = 2 ** 17, 64
    k = torch.zeros(n // 64 + 1, 64, 1, D, device=DEV)
    k[0, 0, 0, 0] = 448.0
    v = torch.ones(n // 64 + 1, 64, 1, D, device=DEV)
    v[0, 0] = 2.0 ** -6
    k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    one = torch.ones(n // 64 + 1, 64, 1, device=DEV)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    q[0, 0, 0] = 1.0
    table, lens = torch.arange(n // 64 + 1, dtype=torch.int32, device=DEV).view(1, -1), torch.tensor([n + 1], dtype=torch.int32, device=DEV)
    scale = 25.5 * math.log(2) / 448
    st = epd.new_status(DEV)
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, epd.new_attention_workspace(1, 1, 1, D, DEV), st, k_scale=one, v_scale=one,
                                     softmax_scale=scale)
    want, _ = attend(q, k.double(), v.double(), table, lens, scale)
    tol = (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -11) * want.abs() + n * 2.0 ** -34
    assert int(st) == 0 and bool(((out.double() - want).abs() <= tol).all())


def test_scores_of_all_sizes():
    """Nearly one-hot and flat softmaxes, given scales, values of very different scales."""
    for fp8 in (False, True):
        check([700, 33], 16, 2, 4, 128, fp8, scale=0.0)
        check([700, 33], 16, 2, 4, 128, fp8, scale=-0.05)
        check([700, 33], 16, 2, 4, 128, fp8, q_scale=2.0 ** -30)
    check([700, 33, 4000], 16, 2, 4, 128, True, v_spread=True)


def test_large_scores():
    """Scores in the thousands: the largest takes all, whatever was summed before it."""
    D, n = 128, 1000
    k = torch.zeros(1, 1000, 1, D, dtype=torch.bfloat16, device=DEV)
    k[0, :, 0, 0] = torch.arange(n, device=DEV).bfloat16()  # rounded: 256 steps of 4 at the end
    v = torch.randn(1, 1000, 1, D, device=DEV).bfloat16()
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16, device=DEV)
    q[0, :, 0] = torch.tensor([16.0, -16.0, 1e30, 0.0], device=DEV)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    status = epd.new_status(DEV)
    ws = epd.new_attention_workspace(1, 4, 1, D, DEV)
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, ws, status, softmax_scale=1.0)
    want, _ = attend(q, k.double(), v.double(), table, lens, 1.0)
    # scores are exact; weights other than the largest are 0 but for ties and for head 3
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14).all())


def test_nonfinite_stays_in_its_sequence():
    g = gen(1)
    k, v, _, _ = paged(4, 64, 2, 64, False, DEV, g)
    table, lens = torch.arange(4, dtype=torch.int32, device=DEV).view(4, 1), torch.tensor([64, 50, 64, 10], dtype=torch.int32, device=DEV)
    q = torch.randn(4, 8, 64, generator=g, device=DEV).bfloat16()
    ws, status = epd.new_attention_workspace(4, 8, 2, 64, DEV), epd.new_status(DEV)
    want, _ = epd.ep_decode_attention(q, k, v, table, lens, ws, status)
    k[1, 3, 0, 5] = float("nan")
    v[2, 7, 1, 9] = float("inf")
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, ws, status)
    assert bool(out[1, :4].isnan().all()) and torch.equal(out[1, 4:], want[1, 4:])
    assert bool((out[2, 4:, 9] == float("inf")).all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, :4] = False
    keep[2, 4:, 9] = False
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths(fp8):
    g = gen(2)
    k, v, ks, vs = paged(6, 16, 2, 64, fp8, DEV, g)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    q = torch.randn(2, 4, 64, generator=g, device=DEV).bfloat16()
    ws = epd.new_attention_workspace(2, 4, 2, 64, DEV)

    def run(table, lens):
        status = epd.new_status(DEV)
        out, _ = epd.ep_decode_attention(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV), ws, status,
                                         k_scale=ks, v_scale=vs)
        return out, int(status)
    full, code = run(table, [48, 48])
    assert code == 0
    for page in (-1, 6, 2**31 - 1):
        bad = table.clone()
        bad[1, 1] = page
        out, code = run(bad, [48, 48])
        assert code == epd.EPD_ERR_CAPACITY and torch.equal(out[0], full[0])
        # as if the page's positions were not there
        lens = torch.tensor([32], dtype=torch.int32, device=DEV)
        want, _ = attend(q[1:], values(k, ks), values(v, vs), table[1:, [0, 2]], lens)
        assert float((out[1:].double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 2.0 ** -11
    out, code = run(table, [48, 49])
    assert code == epd.EPD_ERR_CAPACITY and torch.equal(out, full)
    out, code = run(table, [48, -3])
    assert code == epd.EPD_ERR_INVALID_ARG and torch.equal(out[0], full[0]) and bool((out[1] == 0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_tables_and_caches_with_other_strides(fp8):
    """One table row for all sequences, a table that is a part of a wider one, kv heads that share their rows."""
    g = gen(14)
    B, KH, D, page, n = 5, 2, 64, 16, 70
    k, v, ks, vs = paged(8, page, KH, D, fp8, DEV, g)
    wide = torch.stack([torch.randperm(8, generator=g, device=DEV) for _ in range(B)]).int()
    q = torch.randn(B, 4, D, generator=g, device=DEV).bfloat16()
    lens = torch.tensor([n, 3, 0, 80, 17], dtype=torch.int32, device=DEV)
    ws, st = epd.new_attention_workspace(B, 4, KH, D, DEV), epd.new_status(DEV)

    def f(table, k=k, v=v, ks=ks, vs=vs):
        return epd.ep_decode_attention(q, k, v, table, lens, ws, st, k_scale=ks, v_scale=vs)[0]
    one = wide[:1].expand(B, 8)
    assert torch.equal(f(one), f(one.contiguous()))
    assert torch.equal(f(wide[:, 1:6]), f(wide[:, 1:6].contiguous()))
    half = [None if t is None else t[:, :, :1].expand(t.shape) for t in (k, v, ks, vs)]
    whole = [None if t is None else t.contiguous() for t in half]
    assert torch.equal(f(wide, *half), f(wide, *whole)) and int(st) == 0
    # and appending through a shared row; not into rows that heads share
    new = torch.randn(2, KH, D, generator=g, device=DEV).bfloat16()
    at = torch.tensor([2, 40], dtype=torch.int32, device=DEV)
    got, want = [[None if t is None else t.clone() for t in (k, v, ks, vs)] for _ in range(2)]
    for (a, b, c, d), table in ((got, one), (want, one.contiguous())):
        epd.ep_cache_append(new, new, a, b, table, at, st, k_scale=c, v_scale=d)
    assert int(st) == 0 and all(x is None or torch.equal(x.float(), y.float()) for x, y in zip(got, want))
    assert not torch.equal(got[0].float(), k.float())
    with pytest.raises(epd.EpdError):
        epd.ep_cache_append(new, new, half[0], half[1], one, at, st, k_scale=half[2], v_scale=half[3])
    with pytest.raises(epd.EpdError):
        f(torch.as_strided(wide, (B, 5), (2, 1)))


def test_one_workspace_for_many_shapes():
    ws = epd.new_attention_workspace(64, 64, 8, 256, DEV)
    for i, (lengths, KH, G, D, fp8) in enumerate([([3000] * 3, 8, 8, 128, False), ([17], 1, 1, 64, True), ([900] * 60, 2, 4, 256, False),
                                                  ([50_000], 1, 16, 128, True), ([5] * 64, 8, 8, 80, False)]):
        check(lengths, 16, KH, G, D, fp8, workspace=ws, seed=i)


def test_offsets_beyond_32_bits():
    KH, D, page = 8, 128, 64
    pages = 36_000  # 2.36e9 elements
    g = gen(5)
    small_k, small_v, _, _ = paged(4, page, KH, D, False, DEV, g)
    k = torch.empty(pages, page, KH, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    at = torch.tensor([pages - 1, 5, pages - 2, 33_000], device=DEV)
    k[at], v[at] = small_k, small_v
    q = torch.randn(1, 32, D, generator=g, device=DEV).bfloat16()
    lens = torch.tensor([250], dtype=torch.int32, device=DEV)
    ws, status = epd.new_attention_workspace(1, 32, KH, D, DEV), epd.new_status(DEV)
    out, _ = epd.ep_decode_attention(q, k, v, at.int().view(1, 4), lens, ws, status)
    want, _ = epd.ep_decode_attention(q, small_k, small_v, torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4), lens, ws, status)
    assert int(status) == 0 and torch.equal(out, want)


def test_graph_and_stream():
    g = gen(6)
    k, v, _, _ = paged(40, 16, 2, 128, False, DEV, g)
    table = torch.randperm(40, generator=g, device=DEV).int().view(4, 10)
    lens = torch.tensor([160, 3, 77, 0], dtype=torch.int32, device=DEV)
    q = torch.randn(4, 8, 128, generator=g, device=DEV).bfloat16()
    ws, status = epd.new_attention_workspace(4, 8, 2, 128, DEV), epd.new_status(DEV)

    def step():
        return epd.ep_decode_attention(q, k, v, table, lens, ws, status, with_lse=True)
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in step()]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    lens += 0
    lens.copy_(torch.tensor([5, 160, 0, 100], dtype=torch.int32, device=DEV))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step())) and int(status) == 0


def test_refusals():
    g = gen(7)
    k, v, ks, vs = paged(4, 16, 2, 64, True, DEV, g)
    kb, vb = k.bfloat16(), v.bfloat16()
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    q = torch.randn(2, 4, 64, device=DEV).bfloat16()
    ws, st = epd.new_attention_workspace(2, 4, 2, 64, DEV), epd.new_status(DEV)
    f = epd.ep_decode_attention
    for bad in (lambda: f(q.float(), kb, vb, table, lens, ws, st), lambda: f(q[:1], kb, vb, table, lens, ws, st),
                lambda: f(q[:, :3], kb, vb, table, lens, ws, st), lambda: f(q[..., :32], kb, vb, table, lens, ws, st),
                lambda: f(q, k, v, table, lens, ws, st), lambda: f(q, kb, vb, table, lens, ws, st, k_scale=ks, v_scale=vs),
                lambda: f(q, kb, v, table, lens, ws, st), lambda: f(q, kb, vb, table, lens.long(), ws, st),
                lambda: f(q, kb, vb, table, lens[:1], ws, st), lambda: f(q, kb, vb, table, lens, ws[:100], st),
                lambda: f(q, kb, vb, table.long(), lens, ws, st), lambda: f(q, kb, vb, table, lens, ws, st, out=q.float()),
                lambda: f(q, kb, vb, table, lens, ws, st, lse=ws), lambda: f(q.cpu(), kb, vb, table, lens, ws, st)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(epd.EpdError):
        f(q, kb, vb, table, lens, ws, st, window=-1)
    with pytest.raises(epd.EpdError):
        f(q, kb, vb, table, lens, ws, st, softmax_scale=float("nan"))
    with pytest.raises(epd.EpdError):
        epd.new_attention_workspace(2, 4, 3, 64, DEV)
    assert int(st) == 0


FAR = {  # values' scales far apart: what a token's row and its scale are replaced by
    "zero rows": (3, 0, 0.0),       # as the append holds a row of zeros: scale 1
    "one zero row": (10**6, 0, 0.0),
    "large rows": (50, 1, 0.0),     # 2^30 times the others' scale, in one column
    "no weight": (50, 2, -60.0),    # 2^30 times the others' scale, with next to no weight
    "spread": (1, 3, 0.0),          # from 2^-30 to 2^30 times the others' scale
}


@pytest.mark.parametrize("power", [0, -10, -20, -30, -70])
@pytest.mark.parametrize("what", list(FAR))
@pytest.mark.parametrize("KH,G,D", [(2, 4, 128), (1, 16, 128), (8, 8, 64), (2, 12, 256), (1, 1, 80)])
def test_values_of_far_scales(KH, G, D, what, power):
    """Rows of an e4m3 cache beside rows of very different scales, each held to the bound of the others:
    half a step of the output, and 2^-11 and 2^-14 of the sum of |weight value| in its own column."""
    g = gen(40 + D)
    lengths, page = [700, 33, 2500, 1, 17, 0, 128], 16
    B, most = len(lengths), -(-max(lengths) // page)
    k, v, ks, vs = paged(B * most, page, KH, D, True, DEV, g)
    table = torch.randperm(B * most, generator=g, device=DEV).int().view(B, most)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    q = torch.randn(B, KH * G, D, generator=g, device=DEV).bfloat16()
    vs *= 2.0 ** power
    every, kind, score = FAR[what]
    at = torch.arange(0, most * page, every, device=DEV)
    where = table[:, at // page].long(), (at % page).expand(B, -1)
    codes = v.view(torch.uint8)
    if kind == 0:
        codes[where] = 0
        vs[where] = 1.0
    elif kind == 3:
        vs *= torch.exp2(60 * torch.rand(vs.shape, generator=g, device=DEV) - 30)
    else:
        codes[where] &= torch.where(torch.arange(D, device=DEV) == 3, 255, 0).to(torch.uint8)
        vs[where] *= 2.0 ** 30
    if score:  # (keys against every query of the sequence's first head; for the others they are as any)
        away = -q[:, 0].float() / q[:, 0].float().abs().amax(-1, keepdim=True)
        k.view(torch.uint8)[where[0], where[1], 0] = (448 * away).to(torch.float8_e4m3fn).view(torch.uint8)[:, None]
        ks[where[0], where[1], 0] = 60.0 * D ** 0.5 / (q[:, 0].float() * 448 * -away).sum(-1)[:, None]
    want, lse = attend(q, values(k, ks), values(v, vs), table, lens)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), table, lens)
    st = epd.new_status(DEV)
    f = lambda: epd.ep_decode_attention(q, k, v, table, lens, epd.new_attention_workspace(B, KH * G, KH, D, DEV), st,  # noqa: E731
                                        k_scale=ks, v_scale=vs, with_lse=True)
    out, got = f()
    tol = 2.0 ** -134 + 2.0 ** -8 * want.abs() + (2.0 ** -14 + 2.0 ** -11) * size
    err = (out.double() - want).abs()
    assert int(st) == 0 and bool((err <= tol).all()), (float((err / size.clamp(min=1e-300)).max()), float((err - tol).max()))
    live = lens > 0
    assert bool(((got[live].double() - lse[live]).abs() <= 2.0 ** -14 + 2.0 ** -23 * lse[live].abs()).all())
    again = f()
    assert torch.equal(out, again[0]) and torch.equal(got, again[1])


def test_scales_of_either_sign_and_zero():
    """A value is e4m3 * scale, whatever the scale is."""
    g = gen(41)
    k, v, ks, vs = paged(20, 16, 2, 128, True, DEV, g)
    vs *= torch.where(torch.rand(vs.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    vs[:, 3] = 0.0
    vs[4:6] = 0.0
    vs[7] *= -2.0 ** 12
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(1, 20)
    lens = torch.tensor([311], dtype=torch.int32, device=DEV)
    q = torch.randn(1, 16, 128, generator=g, device=DEV).bfloat16()
    st = epd.new_status(DEV)
    out, _ = epd.ep_decode_attention(q, k, v, table, lens, epd.new_attention_workspace(1, 16, 2, 128, DEV), st, k_scale=ks, v_scale=vs)
    want, _ = attend(q, values(k, ks), values(v, vs), table, lens)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), table, lens)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -14 + 2.0 ** -11) * size
    assert int(st) == 0 and bool(((out.double() - want).abs() <= tol).all())
    # an infinite or NaN scale makes its own kv head's output so, and no other's
    for bad in (float("inf"), float("nan")):
        vs[9, 2, 1] = bad
        got, _ = epd.ep_decode_attention(q, k, v, table, lens, epd.new_attention_workspace(1, 16, 2, 128, DEV), st, k_scale=ks, v_scale=vs)
        assert torch.equal(got[0, :8], out[0, :8]) and not bool(got[0, 8:].isfinite().any())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 17, 33, 129, 300, 513, 5000])
def test_lse_of_nan_scores(n, fp8):
    """A NaN key makes its kv head's output and lse NaN, wherever its tile is joined."""
    g = gen(n)
    for at in (0, n - 1):
        k, v, ks, vs = paged(-(-n // 16), 16, 2, 64, fp8, DEV, g)
        if fp8:
            ks[at // 16, at % 16, 1] = float("nan")
        else:
            k[at // 16, at % 16, 1, 5] = float("nan")
        table = torch.arange(-(-n // 16), dtype=torch.int32, device=DEV).view(1, -1)
        q = torch.randn(1, 8, 64, generator=g, device=DEV).bfloat16()
        st = epd.new_status(DEV)
        out, lse = epd.ep_decode_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                                           epd.new_attention_workspace(1, 8, 2, 64, DEV), st, k_scale=ks, v_scale=vs, with_lse=True)
        assert bool(out[0, 4:].isnan().all()) and bool(lse[0, 4:].isnan().all())
        assert bool(out[0, :4].isfinite().all()) and bool(lse[0, :4].isfinite().all())


def test_windows_of_any_size():
    """A window past 2^31 - 1 is the whole context, and no remainder of it."""
    g = gen(42)
    k, v, _, _ = paged(20, 16, 2, 64, False, DEV, g)
    table, lens = torch.arange(20, dtype=torch.int32, device=DEV).view(1, 20), torch.tensor([300], dtype=torch.int32, device=DEV)
    q = torch.randn(1, 4, 64, generator=g, device=DEV).bfloat16()
    ws, st = epd.new_attention_workspace(1, 4, 2, 64, DEV), epd.new_status(DEV)

    def f(window):
        return epd.ep_decode_attention(q, k, v, table, lens, ws, st, window=window)[0]
    whole = f(0)
    for window in (300, 2**31 - 1, 2**31, 2**32, 2**32 + 5, 2**63 + 7):
        assert torch.equal(f(window), whole), window
    for window in (-1, -2**31, -2**32, -2**32 + 5):
        with pytest.raises(epd.EpdError):
            f(window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("KH,G,D", [(8, 4, 128), (8, 12, 64), (4, 8, 256), (4, 16, 256)])
def test_long_runs_of_one_warp(KH, G, D, fp8):
    """A sequence for every block, of so many tokens that the matrix instructions' sums, which are cut off and
    not rounded, would lose more than the output's own rounding: its pages are a few, over and over."""
    g = gen(50 + D)
    page, few, times, B = 64, 48, 500, 152
    k, v, ks, vs = paged(few, page, KH, D, fp8, DEV, g)
    if fp8:
        x = (values(v, vs) * 0.25 + 1).float()
        vs = x.abs().amax(-1) / 448
        v = (x / vs.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        v = (v.float() * 0.25 + 1).bfloat16()
    q = torch.randn(1, KH * G, D, generator=g, device=DEV).bfloat16()
    once = torch.randperm(few, generator=g, device=DEV).int().view(1, few)
    want, lse = attend(q, values(k, ks), values(v, vs), once, torch.tensor([few * page]))
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), once, torch.tensor([few * page]))
    table, n = once.repeat(1, times).expand(B, few * times), few * page * times
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    st = epd.new_status(DEV)
    f = lambda: epd.ep_decode_attention(q.expand(B, KH * G, D), k, v, table, lens, epd.new_attention_workspace(B, KH * G, KH, D, DEV),  # noqa: E731
                                        st, k_scale=ks, v_scale=vs, with_lse=True)
    out, got = f()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -14 + (2.0 ** -11 if fp8 else 0)) * size
    assert int(st) == 0 and bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want) / size).mean())
    assert bool(((got.double() - lse - math.log(times)).abs() <= 2.0 ** -14 + 2.0 ** -23 * lse.abs()).all())
    again = f()
    assert torch.equal(out, again[0]) and torch.equal(got, again[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_long_runs_whose_maxima_and_scales_move(fp8):
    """What a run has put aside is brought to the maxima and scales that came after it: scores that rise and
    fall by hundreds, and values' scales by 2^20, along the sequence."""
    g = gen(60)
    KH, G, D, page, pages, B = 8, 2, 64, 64, 1200, 152
    k, v, ks, vs = paged(pages, page, KH, D, fp8, DEV, g)
    q = torch.randn(1, KH * G, D, generator=g, device=DEV).bfloat16()
    n = pages * page - 17
    at = torch.arange(pages * page, device=DEV).view(pages, page) / (pages * page)
    rise = (300 * torch.sin(9 * at) * at).unsqueeze(-1)  # of the scores of every kv head's first query
    unit = q[0].float().view(KH, G, D)[:, 0]
    along = unit / unit.square().sum(-1, keepdim=True)
    if fp8:
        vs *= torch.exp2(torch.round(20 * torch.cos(23 * at))).unsqueeze(-1)
        x = along * rise.unsqueeze(-1) + values(k, ks).float() * 0.1
        ks = x.abs().amax(-1) / 448
        k = (x / ks.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        k = (along * rise.unsqueeze(-1) + k.float() * 0.1).bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, pages)
    want, lse = attend(q, values(k, ks), values(v, vs), table, torch.tensor([n]), 1.0)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), table, torch.tensor([n]), 1.0)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    st = epd.new_status(DEV)
    out, got = epd.ep_decode_attention(q.expand(B, KH * G, D), k, v, table.expand(B, pages), lens,
                                       epd.new_attention_workspace(B, KH * G, KH, D, DEV), st, k_scale=ks, v_scale=vs,
                                       softmax_scale=1.0, with_lse=True)
    # scores up to 2^8.3 and products up to some 2^10: 2^-24 of that for each of D / 16 + 4 additions, 2^-11
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + (2.0 ** -11 if fp8 else 0)) * size
    assert int(st) == 0 and bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() / size).max())
    assert bool(((got.double() - lse).abs() <= 2.0 ** -11 + 2.0 ** -23 * lse.abs()).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,KH,G,D", [(3, 1, 4, 128), (2, 2, 16, 64), (5, 1, 9, 256)])
def test_long_runs_shared_by_blocks(B, KH, G, D, fp8):
    """Millions of tokens of a sequence, in the runs of many warps of many blocks, all joined."""
    g = gen(70 + D)
    page, few, times = 64, 48, 2000
    k, v, ks, vs = paged(few, page, KH, D, fp8, DEV, g)
    q = torch.randn(B, KH * G, D, generator=g, device=DEV).bfloat16()
    once = torch.stack([torch.randperm(few, generator=g, device=DEV) for _ in range(B)]).int()
    lens = torch.full((B,), few * page, dtype=torch.int32, device=DEV)
    want, lse = attend(q, values(k, ks), values(v, vs), once, lens)
    size, _ = attend(q, values(k, ks), values(v, vs).abs(), once, lens)
    st = epd.new_status(DEV)
    out, got = epd.ep_decode_attention(q, k, v, once.repeat(1, times), lens * times, epd.new_attention_workspace(B, KH * G, KH, D, DEV),
                                       st, k_scale=ks, v_scale=vs, with_lse=True)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -14 + (2.0 ** -11 if fp8 else 0)) * size
    assert int(st) == 0 and bool(((out.double() - want).abs() <= tol).all())
    assert bool(((got.double() - lse - math.log(times)).abs() <= 2.0 ** -14 + 2.0 ** -23 * lse.abs()).all())
