"""Rotary positions and the paged cache's append on the GPU against the formulas in 64 bits.

Tolerances: half a step of the output (bf16 2^-8, e4m3 2^-4 of the value or 2^-10 of the scale below
its smallest normal number) and 2^-19 of the larger of |a|, |b| for each of the two products in fp32
arithmetic: the angle is within pi 2^-24, the hardware's sines within 2^-20.5, roundings of 2^-24 each."""
import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd
from cache_formulas import paged, turn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
FP8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(4321 + seed)
    return g


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device=DEV).to(torch.bfloat16)


def slack(x, D):
    """2^-20 of the pair's size, bounded by the head's largest element."""
    return 2.0 ** -19 * x.double().abs().amax(-1, keepdim=True).expand(*x.shape[:-1], D)


def near(got, want, more, half=2.0 ** -8):
    err = (got.double() - want).abs()
    assert bool((err <= half * want.abs() + more).all()), float((err - half * want.abs() - more).max())


SHAPES = [(128, 128), (64, 64), (80, 32), (80, 80), (96, 48), (96, 24), (8, 8), (8, 2), (256, 256), (256, 128), (192, 66), (40, 36), (128, 6)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", SHAPES)
@pytest.mark.parametrize("T,N", [(1, 1), (37, 5), (3, 40), (700, 33)])
def test_rotary(T, N, D, R, interleaved):
    x = rand(T, N, D)
    f, _ = epd.rotary_frequencies(R)
    steps = epd.rotary_steps(f, DEV)
    pos = torch.randint(0, 5000, (T,), generator=gen(1), device=DEV, dtype=torch.int32)
    want = turn(x, pos, f, interleaved, 1.25)
    kw = dict(interleaved=interleaved, rotary_scale=1.25)
    got = epd.ep_rotary(x, pos, steps, **kw)
    near(got, want, slack(x, D) * 2)
    assert torch.equal(got[..., R:], x[..., R:])
    # in place, and heads and tokens in the other order
    y = x.clone()
    assert epd.ep_rotary(y, pos, steps, out=y, **kw) is y and torch.equal(y, got)
    z = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(epd.ep_rotary(z, pos, steps, **kw), got)
    # the inverse turns the gradient back: rotation by minus the angle, times the same scale
    near(epd.ep_rotary(x, pos, steps, inverse=True, **kw), turn(x, pos, f, interleaved, 1.25, True), slack(x, D) * 2)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 64), (80, 24), (40, 10)])
def test_rest_of_a_head_is_carried_over(D, R, interleaved):
    """Infinities, negative zeros and NaN beside one another too, each for itself."""
    def same(a, b):
        return bool(((a.contiguous().view(torch.int16) == b.contiguous().view(torch.int16)) | (a.isnan() & b.isnan())).all())
    x = torch.zeros(3, 2, D, dtype=torch.bfloat16, device=DEV)
    odd = torch.tensor([float("inf"), 1.0, float("nan"), -0.0, -float("inf"), 3.0, 0.0, 2.0 ** -133], device=DEV).bfloat16()
    x[..., R:] = odd.repeat(D)[:D - R]
    x[1, :, R:] = odd.flip(0).repeat(D)[1:D - R + 1]
    steps = epd.rotary_steps(epd.rotary_frequencies(R)[0], DEV)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    got = epd.ep_rotary(x, pos, steps, interleaved=interleaved, rotary_scale=1.5)
    assert same(got[..., R:], x[..., R:])
    # queries and keys on the way into a cache; the values are carried over whole
    k, v = (torch.zeros(3, 1, 2, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, st = torch.arange(3, dtype=torch.int32, device=DEV).view(3, 1), epd.new_status(DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    q = epd.ep_cache_append(x, x, k, v, table, pos, st, q=x, steps=steps, interleaved=interleaved, rotary_scale=1.5)
    assert int(st) == 0
    assert same(q[..., R:], x[..., R:]) and same(k[:, 0, :, R:], x[..., R:]) and same(v[:, 0], x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient(interleaved):
    """<dy, rotate(x)> has the gradient rotate_inverse(dy): by the formula's own derivative and by differences."""
    x, dy, d = rand(9, 3, 64), rand(9, 3, 64, seed=1), rand(9, 3, 64, seed=2)
    f, _ = epd.rotary_frequencies(32)
    pos = torch.arange(9, device=DEV, dtype=torch.int32) * 1000
    got = epd.ep_rotary(dy, pos, epd.rotary_steps(f, DEV), interleaved=interleaved, inverse=True)
    leaf = x.double().requires_grad_()
    grad, = torch.autograd.grad(turn(leaf, pos, f, interleaved), leaf, dy.double())
    near(got, grad, slack(dy, 64))

    def loss(h):
        return (turn(x.double() + h * d.double(), pos, f, interleaved) * dy.double()).sum()
    slope = float(loss(1.0) - loss(-1.0)) / 2  # the rotation is linear
    assert abs(float((got.double() * d.double()).sum()) - slope) <= 2.0 ** -8 * float((grad * d.double()).abs().sum())


def test_rotary_far_positions():
    x = rand(6, 4, 128)
    pos = torch.tensor([0, 1, 10**6, 2**31 - 1, -1, -(2**31)], device=DEV, dtype=torch.int32)
    f, _ = epd.rotary_frequencies(128)
    # 64 bits keep 2^31 * f to 2^-22: the test's own angles are good to 2^-21
    near(epd.ep_rotary(x, pos, epd.rotary_steps(f, DEV)), turn(x, pos, f), 4 * slack(x, 128))


def test_frequencies():
    f, s = epd.rotary_frequencies(64)
    assert s == 1.0 and torch.allclose(f, 10000.0 ** (-torch.arange(32).double() / 32))
    g, s = epd.rotary_frequencies(64, scaling="linear", factor=4)
    assert s == 1.0 and torch.equal(g, f / 4)
    g, s = epd.rotary_frequencies(64, scaling="ntk", factor=4)
    assert float(g[0]) == 1.0 and abs(float(g[-1] * 4 / f[-1]) - 1) < 1e-12
    g, s = epd.rotary_frequencies(64, scaling="yarn", factor=4, original_length=4096)
    assert abs(s - 1.138629436111989) < 1e-12
    turns = f * 4096 / 6.283185307179586
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.8], f[turns < 0.8] / 4)
    assert bool(((g <= f) & (g >= f / 4)).all())
    assert epd.rotary_frequencies(64, scaling="yarn")[1] == 1.0
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="x"), dict(rotary_dim=8, factor=0.5)):
        with pytest.raises(ValueError):
            epd.rotary_frequencies(**bad)
    assert epd.rotary_steps([0.0, 3.141592653589793, -1.5707963267948966], DEV).tolist() == [0, -(1 << 63), -(1 << 62)]
    with pytest.raises(ValueError):
        epd.rotary_steps([float("inf")], DEV)


def check_append(T, S, page, KH, QH, D, R, interleaved, fp8, order, padded=False, seed=0):
    g = gen(seed)
    most = 7
    per = [T // S + (i < T % S) for i in range(S)]
    seq, pos = [], []
    for s, n in enumerate(per):
        first = (s * 5) % max(1, most * page - n + 1)
        seq += [s] * n
        pos += list(range(first, first + n))
    order_of = torch.randperm(T, generator=g, device=DEV)
    seq = torch.tensor(seq, dtype=torch.int32, device=DEV)[order_of]
    pos = torch.tensor(pos, dtype=torch.int32, device=DEV)[order_of]
    if padded:
        seq[::3] = -1
        pos[::3] = 10**9
    table = torch.randperm(S * most, generator=g, device=DEV).to(torch.int32).view(S, most)
    k, v, ks, vs = paged(S * most, page, KH, D, fp8, DEV, g, order)
    before = [None if t is None else t.clone() for t in (k, v, ks, vs)]
    qkv = torch.randn(T, QH + 2 * KH, D, generator=g, device=DEV).to(torch.bfloat16)
    f = epd.rotary_frequencies(R)[0] if R else []
    status = epd.new_status(DEV)
    q_out = torch.full((T, QH, D), 7.0, dtype=torch.bfloat16, device=DEV)
    if QH:
        q = epd.ep_cache_append(qkv[:, QH:QH + KH], qkv[:, QH + KH:], k, v, table, pos, status, token_seq=seq,
                                q=qkv[:, :QH], steps=epd.rotary_steps(f, DEV) if R else None, interleaved=interleaved,
                                rotary_scale=1.1, k_scale=ks, v_scale=vs, q_out=q_out)
        assert q is q_out
    else:
        assert epd.ep_cache_append(qkv[:, :KH], qkv[:, KH:], k, v, table, pos, status, token_seq=seq,
                                   steps=epd.rotary_steps(f, DEV) if R else None, interleaved=interleaved,
                                   rotary_scale=1.1, k_scale=ks, v_scale=vs) is None
    assert int(status) == 0
    live = seq >= 0
    turned = turn(qkv[:, :QH + KH], pos, f, interleaved, 1.1) if R else qkv[:, :QH + KH].double()
    if QH:
        near(q_out[live], turned[live, :QH], 2 * slack(qkv[live, :QH], D))
        assert bool((q_out[~live] == 7).all())
    at = table[seq.clamp(min=0).long(), pos.long().clamp(max=most * page - 1) // page].long()[live], pos.long()[live] % page
    for cache, scale, rows, old, old_scale in ((k, ks, turned[:, QH:], before[0], before[2]),
                                               (v, vs, qkv[:, QH + KH:].double(), before[1], before[3])):
        rows = rows[live]
        size = 2 * slack(qkv[live, :1], 1) if R else torch.zeros(1, device=DEV)
        size = 2 * 2.0 ** -19 * 6.0  # of values up to 6
        if fp8:
            amax = rows.abs().amax(-1)
            near(scale[at], amax / 448, size / 448, 2.0 ** -23)
            near(cache[at].double() * scale[at].double().unsqueeze(-1), rows,
                 2.0 ** -10 * scale[at].double().unsqueeze(-1) + 2 * size, 2.0 ** -4)
        else:
            near(cache[at], rows, size)
        # nothing else was touched
        mask = torch.ones(cache.shape[:2], dtype=torch.bool, device=DEV)
        mask[at] = False
        assert torch.equal(cache.view(torch.uint8)[mask] if fp8 else cache[mask], old.view(torch.uint8)[mask] if fp8 else old[mask])
        if fp8:
            assert torch.equal(scale[mask], old_scale[mask])


@pytest.mark.parametrize("order", ["page,row,head", "page,head,row"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (64, 32, True), (80, 80, False), (96, 48, False), (256, 64, True), (16, 0, False), (48, 6, False), (48, 6, True), (256, 250, False), (192, 192, False)])
def test_append(D, R, interleaved, fp8, order):
    check_append(29, 5, 3, 2, 6, D, R, interleaved, fp8, order, padded=True)
    check_append(5, 5, 16, 1, 0, D, R, interleaved, fp8, order)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,S,page,KH,QH", [(1, 1, 1, 1, 1), (1, 1, 64, 8, 32), (130, 130, 1, 3, 21), (2500, 9, 64, 8, 64), (300, 60, 5, 1, 71)])
def test_append_sizes(T, S, page, KH, QH, fp8):
    check_append(T, S, page, KH, QH, 128, 128, False, fp8, "page,row,head", seed=T)


def test_append_in_place_and_zero_rows():
    g = gen(0)
    k, v, ks, vs = paged(4, 8, 2, 32, True, DEV, g)
    x = torch.zeros(4, 2, 32, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(4, 1)
    pos = torch.tensor([0, 3, 7, 1], dtype=torch.int32, device=DEV)
    status = epd.new_status(DEV)
    q = rand(4, 5, 32)
    f = epd.rotary_frequencies(32)[0]
    steps = epd.rotary_steps(f, DEV)
    want = epd.ep_cache_append(x, x, k, v, table, pos, status, q=q, steps=steps, k_scale=ks, v_scale=vs)
    assert epd.ep_cache_append(x, x, k, v, table, pos, status, q=q, q_out=q, steps=steps, k_scale=ks, v_scale=vs) is q
    assert torch.equal(q, want)
    rows = torch.arange(4, device=DEV)
    assert float(k[rows, pos.long()].float().abs().max()) == 0 and bool((ks[rows, pos.long()] == 1).all())
    assert int(status) == 0


@pytest.mark.parametrize("what", ["page", "negative page", "position", "negative position", "sequence", "negative sequence"])
def test_append_out_of_range(what):
    g = gen(0)
    k, v, _, _ = paged(6, 4, 2, 64, False, DEV, g)
    old = k.clone(), v.clone()
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    pos = torch.tensor([0, 5, 11], dtype=torch.int32, device=DEV)
    seq = torch.tensor([0, 1, 1], dtype=torch.int32, device=DEV)
    if "page" in what:
        table[1, 1] = -1 if "negative" in what else 6
    elif "position" in what:
        pos[1] = -1 if "negative" in what else 12
    else:
        seq[1] = -2 if "negative" in what else 2
    x, q = rand(3, 2, 64), rand(3, 4, 64, seed=1)
    q_out = torch.full_like(q, 7.0)
    status = epd.new_status(DEV)
    epd.ep_cache_append(x, x, k, v, table, pos, status, token_seq=seq, q=q, q_out=q_out)
    assert int(status) == epd.EPD_ERR_CAPACITY
    assert torch.equal(k[0, 0], x[0]) and torch.equal(v[5, 3], x[2]) and torch.equal(q_out[0], q[0])
    assert bool((q_out[1] == 7).all())
    rest = torch.ones(6, 4, dtype=torch.bool, device=DEV)
    rest[0, 0] = rest[5, 3] = False
    assert torch.equal(k[rest], old[0][rest]) and torch.equal(v[rest], old[1][rest])


def test_append_offsets_beyond_32_bits():
    KH, D, page = 8, 128, 64
    pages = 36_000  # 2.36e9 elements
    k = torch.empty(pages, page, KH, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    table = torch.tensor([[3, pages - 1]], dtype=torch.int32, device=DEV)
    x = rand(2, KH, D)
    status = epd.new_status(DEV)
    epd.ep_cache_append(x, -x, k, v, table, torch.tensor([1, 127], dtype=torch.int32, device=DEV), status,
                        token_seq=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert int(status) == 0
    assert torch.equal(k[pages - 1, 63], x[1]) and torch.equal(v[pages - 1, 63], -x[1]) and torch.equal(k[3, 1], x[0])


def test_rotary_offsets_beyond_32_bits():
    T, N, D = 600_000, 32, 128  # 2.46e9 elements
    x = torch.ones(T, N, D, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, T // 2, T - 1], device=DEV)
    x[rows] = rand(3, N, D)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    steps = epd.rotary_steps(epd.rotary_frequencies(D)[0], DEV)
    want = epd.ep_rotary(x[rows], pos[rows], steps)
    assert torch.equal(epd.ep_rotary(x, pos, steps, out=x)[rows], want)


def test_nothing_to_do():
    steps = epd.rotary_steps(epd.rotary_frequencies(64)[0], DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert epd.ep_rotary(rand(0, 4, 64), none, steps).shape == (0, 4, 64)
    assert epd.ep_rotary(rand(2, 0, 64), torch.zeros(2, dtype=torch.int32, device=DEV), steps).shape == (2, 0, 64)
    k, v, _, _ = paged(1, 4, 2, 64, False, DEV, gen(0))
    status = epd.new_status(DEV)
    epd.ep_cache_append(rand(0, 2, 64), rand(0, 2, 64), k, v, torch.zeros(0, 1, dtype=torch.int32, device=DEV), none, status)
    assert int(status) == 0


def test_refusals():
    steps = epd.rotary_steps(epd.rotary_frequencies(64)[0], DEV)
    x, pos = rand(4, 2, 64), torch.zeros(4, dtype=torch.int32, device=DEV)
    k, v, ks, vs = paged(4, 8, 2, 64, True, DEV, gen(0))
    kb, vb = k.bfloat16(), v.bfloat16()
    table = torch.zeros(4, 1, dtype=torch.int32, device=DEV)
    st = epd.new_status(DEV)
    f = epd.ep_cache_append
    for bad in (lambda: epd.ep_rotary(x.float(), pos, steps), lambda: epd.ep_rotary(x, pos.long(), steps),
                lambda: epd.ep_rotary(x, pos[:3], steps), lambda: epd.ep_rotary(x[..., :32], pos, steps),
                lambda: epd.ep_rotary(x.transpose(1, 2), pos, steps), lambda: epd.ep_rotary(x, pos, steps.int()),
                lambda: epd.ep_rotary(x, pos, steps, out=x[:3]), lambda: epd.ep_rotary(x.cpu(), pos, steps),
                lambda: f(x, x, k, v, table, pos, st), lambda: f(x, x, kb, vb, table, pos, st, k_scale=ks, v_scale=vs),
                lambda: f(x, x, kb, vb[:3], table, pos, st), lambda: f(x, x, kb, vb, table.long(), pos, st),
                lambda: f(x, x, kb, vb, table[:3], pos, st), lambda: f(x[..., :32], x, kb, vb, table, pos, st),
                lambda: f(x.transpose(0, 1), x, kb, vb, table, pos, st), lambda: f(x, x, kb, vb.transpose(1, 2), table, pos, st),
                lambda: f(x, x, kb, vb, table, pos, st, q_out=x), lambda: f(x, x, kb, vb, table, pos, st, token_seq=pos[:1]),
                lambda: f(x, x, k, v, table, pos, st, k_scale=ks[:3], v_scale=vs), lambda: f(x, x, kb.float(), vb.float(), table, pos, st),
                lambda: f(x, x, kb, vb, table, pos, st, q=x[:3]), lambda: f(x, x, kb[0], vb[0], table, pos, st)):
        with pytest.raises(ValueError):
            bad()
    wide = rand(4, 2, 264)
    with pytest.raises(epd.EpdError):
        epd.ep_rotary(wide, pos, steps)
    with pytest.raises(epd.EpdError):  # strides that are no multiples of 16 bytes
        epd.ep_rotary(rand(4, 2, 68)[..., :64], pos, steps)
    assert int(st) == 0


def test_graph_and_stream():
    g = gen(3)
    k, v, ks, vs = paged(8, 4, 2, 64, True, DEV, g)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    pos = torch.tensor([0, 3, 5, 6], dtype=torch.int32, device=DEV)
    steps = epd.rotary_steps(epd.rotary_frequencies(64)[0], DEV)
    st = epd.new_status(DEV)
    qkv = rand(4, 8, 64)

    def step():
        x = epd.ep_rotary(qkv, pos, steps)
        q = epd.ep_cache_append(qkv[:, 4:6], qkv[:, 6:], k, v, table, pos, st, q=qkv[:, :4], steps=steps, k_scale=ks, v_scale=vs)
        return x, q, k.view(torch.uint8), vs
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
    pos += 1
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (128, 64, True), (64, 0, False), (80, 24, False), (48, 6, True), (256, 256, False)])
def test_append_carries_values_over(D, R, interleaved):
    """Values (and keys that are not rotated) are written as they are, or as e4m3 numbers of the quotients by
    their scale: both to the last bit."""
    T, KH, page = 1500, 4, 16
    qkv = rand(T, 2 * KH, D, seed=D)
    pages = -(-T // page) + 3
    table = torch.randperm(pages, generator=gen(D), device=DEV).int().view(1, pages)
    pos = torch.randperm(pages * page, generator=gen(D + 1), device=DEV)[:T].int()
    seq = torch.zeros(T, dtype=torch.int32, device=DEV)
    seq[::5] = -1
    live = seq == 0
    at = table[0, pos.long() // page].long()[live], pos.long()[live] % page
    steps = epd.rotary_steps(epd.rotary_frequencies(R)[0], DEV) if R else None
    for fp8 in (False, True):
        k, v, ks, vs = paged(pages, page, KH, D, fp8, DEV, gen(1))
        st = epd.new_status(DEV)
        epd.ep_cache_append(qkv[:, :KH], qkv[:, KH:], k, v, table, pos, st, token_seq=seq, steps=steps, interleaved=interleaved,
                            k_scale=ks, v_scale=vs)
        assert int(st) == 0
        for cache, scale, rows in ((v, vs, qkv[live, KH:]),) + (() if R else ((k, ks, qkv[live, :KH]),)):
            if not fp8:
                assert torch.equal(cache[at], rows)
                continue
            rows = rows.float()
            want = rows.abs().amax(-1) / torch.full(rows.shape[:2], 448.0, device=DEV)
            assert torch.equal(scale[at], want)
            codes = (rows / want.unsqueeze(-1).expand_as(rows)).clamp(-448, 448).to(FP8)
            assert torch.equal(cache.view(torch.uint8)[at], codes.view(torch.uint8))


def test_append_of_rows_below_448_of_the_smallest_number():
    """A rotary scale may take keys below 2^-141, where amax / 448 rounds to 0: their scale is the smallest
    number there is then, never 0."""
    k, v, ks, vs = paged(4, 8, 2, 64, True, DEV, gen(0))
    x = rand(4, 2, 64)
    x[..., ::3] = 0
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(4, 1)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    st = epd.new_status(DEV)
    steps = epd.rotary_steps(epd.rotary_frequencies(64)[0], DEV)
    for power in (-120, -140, -146):
        epd.ep_cache_append(x, x, k, v, table, pos, st, steps=steps, rotary_scale=2.0 ** power, k_scale=ks, v_scale=vs)
        rows, scale = x.double() * 2.0 ** power, ks[:, 0].double()
        assert bool((scale > 0).all())
        # half a step of e4m3, a step of the products (2^-149 each), half a step of the scale times 448
        got = k[:, 0].double() * scale.unsqueeze(-1)
        tol = 2.0 ** -4 * rows.abs() + 2.0 ** -10 * scale.unsqueeze(-1) + 226 * 2.0 ** -149
        assert bool(((got - rows).abs() <= tol).all())
    assert int(st) == 0


def test_sizes_past_32_bits_are_refused():
    """The C entry points take 32-bit sizes: a larger one is an error, not its remainder."""
    few = torch.zeros(8, dtype=torch.int32, device=DEV)
    many = 2 ** 32 + 8
    rows = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV).expand(many, 8)
    heads = torch.zeros(1, 1, 8, dtype=torch.bfloat16, device=DEV).expand(many, 1, 8)
    steps, st = epd.rotary_steps([1.0, 0.5, 0.2, 0.1], DEV), epd.new_status(DEV)
    cache = torch.zeros(2, 4, 1, 8, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    for bad in (lambda: epd.ep_layer_norm(rows), lambda: epd.ep_layer_norm_backward(rows, rows, None, few, kind="rms"),
                lambda: epd.ep_rotary(heads, few, steps), lambda: epd.ep_rotary(heads.transpose(0, 1), few, steps),
                lambda: epd.ep_cache_append(heads, heads, cache, cache, table, few, st, token_seq=few),
                lambda: epd.ep_decode_attention(heads, cache, cache, table.expand(many, 2), few, few.view(torch.uint8), st)):
        with pytest.raises(ValueError, match="2147483647"):
            bad()
