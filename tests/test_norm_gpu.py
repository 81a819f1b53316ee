"""The norm and its gradients on the GPU against the formulas in 64 bits.

Tolerances: half a step of the output's type (bf16 2^-8, e4m3 2^-4, relative) for its one rounding,
and 64 units of 2^-24 of the terms' sizes for fp32 arithmetic (a row's sums have at most 32 + 11
additions in a chain: 8 or 32 columns a thread, two trees over 32)."""
import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32 = 64 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def rand(*shape, seed=0, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(1234 + seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale + shift).to(dtype)


def near(got, want, slack, dtype):
    assert got.dtype == dtype
    err = (got.double() - want).abs()
    tol = HALF[dtype] * want.abs() + slack
    assert bool((err <= tol).all()), float((err - tol).max())


def formula(x, residual, w, b, eps, kind):
    s = x.double() + (0 if residual is None else residual.double())
    mean = s.mean(1, keepdim=True) if kind == "layer" else torch.zeros(s.shape[0], 1, dtype=torch.float64, device=DEV)
    rstd = ((s - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (s - mean) * rstd
    y = y * (1 if w is None else w.double()) + (0 if b is None else b.double())
    big = s.abs().amax(1, keepdim=True) * rstd * (1 if w is None else w.double().abs()) + (0 if b is None else b.double().abs())
    return s, mean, rstd, y, big.expand_as(y)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (700, 264), (33, 1000), (1, 7168), (350, 7168), (5, 8192), (4, 8200), (170, 16384)])
def test_norm(T, H, dtype, kind):
    x, r = rand(T, H, dtype=dtype, scale=2.0, shift=0.7), rand(T, H, seed=1, dtype=dtype)
    w, b = rand(H, seed=2, scale=0.3, shift=1.0), rand(H, seed=3)
    for residual, ww, bb in ((None, w, b), (r, w, None), (r, None, None)):
        fp8 = H % 128 == 0
        d = epd.ep_layer_norm(x, ww, bias=bb, residual=residual, eps=1e-5, kind=kind, with_fp8=fp8, with_stats=True)
        s, mean, rstd, y, big = formula(x, residual, ww, bb, 1e-5, kind)
        near(d["y"], y, F32 * big, torch.bfloat16)
        near(d["rstd"], rstd.squeeze(1), F32 * rstd.squeeze(1), torch.float32)
        if kind == "layer":
            near(d["mean"], mean.squeeze(1), F32 * s.abs().amax(1), torch.float32)
        else:
            assert d["mean"] is None
        if residual is None:
            assert d["sum"] is None
        else:
            near(d["sum"], s, 0.0 if dtype is torch.float32 else 2.0 ** -24 * s.abs(), dtype)
        if fp8:
            blocks, bigs = y.view(T, -1, 128).abs().amax(2), big.reshape(T, -1, 128).amax(2)
            near(d["y_scale"], blocks / 448, F32 * bigs / 448 + 2.0 ** -24 * blocks / 448, torch.float32)
            got = d["y_q"].double() * d["y_scale"].double().repeat_interleave(128, 1)
            # a step of e4m3 is absolute below 2^-6: half of 2^-9 of the scale
            scale = d["y_scale"].double().repeat_interleave(128, 1)
            tol = HALF[torch.float8_e4m3fn] * y.abs() + 2.0 ** -10 * scale + 2 * F32 * big
            assert bool(((got - y).abs() <= tol).all())
        else:
            assert d["y_q"] is None


def test_rows_of_zeros_and_large_offsets():
    x = torch.zeros(3, 256, device=DEV)
    x[1] = 1e4 + rand(256)  # the mean is 10^4 standard deviations: the centred values keep their digits
    d = epd.ep_layer_norm(x, with_fp8=True)
    assert float(d["y"][0].float().abs().max()) == 0 and bool((d["y_scale"][0] == 1).all())
    _, _, _, y, _ = formula(x, None, None, None, 1e-5, "layer")
    # x itself is exact; its mean is off by at most 64 units of 2^-24 of 10^4
    near(d["y"][1], y[1], F32 * 1e4 * 2, torch.bfloat16)


@pytest.mark.parametrize("shift", [0.0, 0.9, 1.1, 3.0, 100.0])
def test_means_around_the_deviation(shift):
    """The variance by the squares' mean and, where the row's mean is above its deviation, by centred values."""
    x = rand(64, 1000, shift=shift)
    x[::2] -= 2 * shift
    d = epd.ep_layer_norm(x, with_stats=True)
    _, mean, rstd, y, big = formula(x, None, None, None, 1e-5, "layer")
    near(d["y"], y, F32 * big, torch.bfloat16)
    near(d["rstd"], rstd.squeeze(1), F32 * rstd.squeeze(1), torch.float32)


def test_tiny_rows():
    """e4m3 rows whose scale is below the smallest normal number: its reciprocal overflows."""
    x, w = rand(5, 256), torch.full((256,), 1e-37, device=DEV)
    d = epd.ep_layer_norm(x, w, with_fp8=True)
    y = formula(x, None, w, None, 1e-5, "layer")[3]
    scale = d["y_scale"].double().repeat_interleave(128, 1)
    # the scale itself has steps of 2^-149, up to 2^-20 of it here
    assert bool(((d["y_q"].double() * scale - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * scale + 2.0 ** -19 * 448 * scale).all())


def test_nonfinite_rows_stay_alone():
    x = rand(64, 1024, dtype=torch.bfloat16)
    want = epd.ep_layer_norm(x)["y"].clone()
    y2 = x.clone()
    y2[5, 17], y2[9, 1000] = float("nan"), float("inf")
    got = epd.ep_layer_norm(y2)["y"]
    keep = torch.ones(64, dtype=torch.bool, device=DEV)
    keep[[5, 9]] = False
    assert torch.equal(got[keep], want[keep])
    assert bool(got[5].isnan().all()) and bool(got[9].isnan().any())


def test_outputs_in_place():
    x, r, w = rand(300, 1032, dtype=torch.bfloat16), rand(300, 1032, seed=1, dtype=torch.bfloat16), rand(1032, seed=2)
    want = epd.ep_layer_norm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = epd.ep_layer_norm(x2, w, residual=r2, sum=r2, y=x2)
    assert torch.equal(got["sum"], want["sum"]) and torch.equal(got["y"], want["y"])
    assert got["sum"].data_ptr() == r2.data_ptr() and got["y"].data_ptr() == x2.data_ptr()
    st = epd.ep_layer_norm(x, w, with_stats=True)
    dy, gs = rand(300, 1032, seed=4, dtype=torch.bfloat16), rand(300, 1032, seed=5, dtype=torch.bfloat16)
    want = epd.ep_layer_norm_backward(dy, x, w, st["rstd"], mean=st["mean"], grad_sum=gs)
    for k in range(3):
        a = [dy.clone(), x.clone(), gs.clone()]
        dx, dw, _ = epd.ep_layer_norm_backward(a[0], a[1], w, st["rstd"], mean=st["mean"], grad_sum=a[2], dx=a[k])
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def grads(dy, x, w, mean, rstd, gs):
    dy, x, rstd = dy.double(), x.double(), rstd.double().unsqueeze(1)
    xh = (x - (0 if mean is None else mean.double().unsqueeze(1))) * rstd
    g = dy * (1 if w is None else w.double())
    mg = 0 if mean is None else g.mean(1, keepdim=True)
    dx = rstd * (g - mg - xh * (g * xh).mean(1, keepdim=True)) + (0 if gs is None else gs.double())
    big = rstd * (g.abs().amax(1, keepdim=True) * 2 + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
        + (0 if gs is None else gs.double().abs())
    return dx, big, dy * xh, dy


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 8), (5, 72), (5000, 64), (33, 1000), (333, 1032), (1, 7168), (400, 7168), (6, 8200), (170, 16384)])
def test_norm_backward(T, H, dtype, kind):
    x, dy = rand(T, H, dtype=dtype, scale=2.0, shift=0.7), rand(T, H, seed=1, dtype=torch.bfloat16)
    w, gs = rand(H, seed=2, scale=0.3, shift=1.0), rand(T, H, seed=3, dtype=dtype)
    st = epd.ep_layer_norm(x, w, kind=kind, with_stats=True)
    for ww, joined, bias in ((w, None, True), (None, gs, False), (w, gs, True)):
        args = (dy, x, ww, st["rstd"])
        kw = dict(mean=st["mean"], kind=kind, grad_sum=joined, with_dbias=bias)
        dx, dw, db = epd.ep_layer_norm_backward(*args, **kw)
        want, big, per_w, per_b = grads(dy, x, ww, st["mean"], st["rstd"], joined)
        near(dx, want, F32 * big, dtype)
        # sums over T rows: at most T additions in a chain, and their random walk well below that
        for got, terms in ((dw, per_w), (db, per_b)):
            if got is None:
                assert not bias
                continue
            s, total = terms.sum(0), terms.abs().sum(0)
            assert bool(((got.double() - s).abs() <= 2.0 ** -24 * (T + 16) * total).all())
            assert float((got.double() - s).norm()) <= 1e-5 * float(s.norm())
        again = epd.ep_layer_norm_backward(*args, **kw)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and (db is None or torch.equal(db, again[2]))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_against_differences(kind):
    """The kernel's gradients along a direction against central differences of the norm in 64 bits."""
    T, H = 4, 136
    x, w, b, dy = rand(T, H), rand(H, seed=1, shift=1.0), rand(H, seed=2), rand(T, H, seed=3, dtype=torch.bfloat16)
    st = epd.ep_layer_norm(x, w, bias=b, kind=kind, with_stats=True)
    dx, dw, db = epd.ep_layer_norm_backward(dy, x, w, st["rstd"], mean=st["mean"], kind=kind, with_dbias=True)
    d = [rand(*t.shape, seed=9 + i).double() for i, t in enumerate((x, w, b))]

    def loss(h):
        return (formula(x.double() + h * d[0], None, w.double() + h * d[1], b.double() + h * d[2], 1e-5, kind)[3]
                * dy.double()).sum()
    h = 1e-4  # the differences' own error: h^2 times third derivatives, 1e-8 times a few hundred
    slope = float((loss(h) - loss(-h)) / (2 * h))
    got = float((dx.double() * d[0]).sum() + (dw.double() * d[1]).sum() + (db.double() * d[2]).sum())
    terms = float((dx.double() * d[0]).abs().sum() + (dw.double() * d[1]).abs().sum() + (db.double() * d[2]).abs().sum())
    assert abs(got - slope) <= F32 * terms + 1e-4


def test_no_rows():
    x = torch.empty(0, 256, device=DEV)
    assert epd.ep_layer_norm(x)["y"].shape == (0, 256)
    dw, db = torch.ones(256, device=DEV), torch.ones(256, device=DEV)
    epd.ep_layer_norm_backward(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV), x, None, torch.empty(0, device=DEV),
                               mean=torch.empty(0, device=DEV), dweight=dw, dbias=db)
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_offsets_beyond_32_bits():
    T, H = 300_000, 7232  # 2.17e9 elements
    x = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    rows = [0, 1, T // 2, T - 2, T - 1]
    x[rows] = rand(len(rows), H, dtype=torch.bfloat16)
    d = epd.ep_layer_norm(x, with_stats=True)
    small = epd.ep_layer_norm(x[rows].contiguous(), with_stats=True)
    assert torch.equal(d["y"][rows], small["y"]) and torch.equal(d["rstd"][rows], small["rstd"])
    dy = d["y"]
    dx, dw, _ = epd.ep_layer_norm_backward(dy, x, None, d["rstd"], mean=d["mean"])
    few = epd.ep_layer_norm_backward(dy[rows].contiguous(), x[rows].contiguous(), None, small["rstd"], mean=small["mean"])
    assert torch.equal(dx[rows], few[0])
    assert float((dw - few[1]).abs().max()) <= 1e-4 * float(few[1].abs().max())  # rows of ones give none


def test_graph_and_stream():
    x, w, dy = rand(97, 2048, dtype=torch.bfloat16), rand(2048, seed=1), rand(97, 2048, seed=2, dtype=torch.bfloat16)
    ws = epd.new_norm_workspace(2048, DEV)
    side = torch.cuda.Stream()

    def step():
        d = epd.ep_layer_norm(x, w, with_stats=True, with_fp8=True)
        return [d["y"], d["y_q"].view(torch.uint8), *epd.ep_layer_norm_backward(
            dy, x, w, d["rstd"], mean=d["mean"], workspace=ws, with_dbias=True)]
    want = [t.clone() for t in step()]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in step()]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(rand(97, 2048, seed=7, dtype=torch.bfloat16))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_own_workspace_on_a_given_stream(monkeypatch):
    """A workspace made by the call stays its own until the given stream has read it."""
    from unpermute_ep_dispatch_gb300 import _binding
    H = 8192
    x, w, dy = rand(300, H, dtype=torch.bfloat16), rand(H, seed=1), rand(300, H, seed=2, dtype=torch.bfloat16)
    rstd = rand(300, seed=3).abs()
    want = epd.ep_layer_norm_backward(dy, x, w, rstd, kind="rms")
    made = []

    def new(*args):
        t = torch.empty(epd.epd_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)
        made.append(t.data_ptr())
        return t
    monkeypatch.setattr(_binding, "new_norm_workspace", new)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
    got = epd.ep_layer_norm_backward(dy, x, w, rstd, kind="rms", stream=side)
    other = torch.empty(epd.epd_norm_workspace_bytes(H), dtype=torch.uint8, device=DEV)
    assert other.data_ptr() not in made and len(made) == 1
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want[:2]))


def test_refusals():
    x, w = rand(4, 256), rand(256)
    st = rand(4)
    dy = rand(4, 256, dtype=torch.bfloat16)
    for bad in (lambda: epd.ep_layer_norm(x.half()), lambda: epd.ep_layer_norm(x[0]), lambda: epd.ep_layer_norm(x.t()),
                lambda: epd.ep_layer_norm(x, w[:-1]), lambda: epd.ep_layer_norm(x, w.bfloat16()),
                lambda: epd.ep_layer_norm(x, residual=x.bfloat16()), lambda: epd.ep_layer_norm(x, kind="batch"),
                lambda: epd.ep_layer_norm(x, sum=x), lambda: epd.ep_layer_norm(x, with_y=False),
                lambda: epd.ep_layer_norm(x[:, :136].contiguous(), with_fp8=True),
                lambda: epd.ep_layer_norm(x, kind="rms", mean=st), lambda: epd.ep_layer_norm(x.cpu()),
                lambda: epd.ep_layer_norm_backward(dy, x, w, st, kind="rms", mean=st),
                lambda: epd.ep_layer_norm_backward(dy, x, w, st, mean=st, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
                lambda: epd.ep_layer_norm_backward(x, x, w, st, mean=st),
                lambda: epd.ep_layer_norm_backward(dy, x, w, st[:3], mean=st)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        epd.ep_layer_norm_backward(dy, x, w, st)
    with pytest.raises(epd.EpdError):
        epd.ep_layer_norm(rand(4, 250))
    with pytest.raises(epd.EpdError):
        epd.ep_layer_norm(rand(1, 16392))
    with pytest.raises(epd.EpdError):
        epd.ep_layer_norm(x, eps=-1.0)


def test_own_workspace_belongs_to_the_given_stream(monkeypatch):
    """What a call on the current stream still has to write is not handed to a call on another one."""
    from unpermute_ep_dispatch_gb300 import _binding
    H = 8192
    args = [(rand(300, H, seed=i, dtype=torch.bfloat16), rand(300, H, seed=i + 5, dtype=torch.bfloat16), rand(H, seed=i + 10),
             rand(300, seed=i + 15).abs()) for i in range(2)]
    want = [epd.ep_layer_norm_backward(*a, kind="rms") for a in args]
    made, plain = [], _binding.new_norm_workspace

    def new(*a):
        made.append(plain(*a))
        return made[-1]
    monkeypatch.setattr(_binding, "new_norm_workspace", new)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some ten milliseconds of the current stream
    first = epd.ep_layer_norm_backward(*args[0], kind="rms")
    places = [made.pop().data_ptr()]
    second = epd.ep_layer_norm_backward(*args[1], kind="rms", stream=side)
    places.append(made.pop().data_ptr())
    torch.cuda.synchronize()
    assert places[0] != places[1]
    for got, ref in zip((first, second), want):
        assert all(torch.equal(a, b) for a, b in zip(got[:2], ref[:2]))


@pytest.mark.parametrize("dtype,size,deviation", [(torch.float32, 2.0 ** 57, 1e14), (torch.float32, 1e18, 1e15), (torch.bfloat16, 1e18, 1e17),
                                                  (torch.float32, 1e20, 1e17), (torch.float32, 1e25, 0.0), (torch.bfloat16, 1e25, 0.0)])
def test_means_whose_squares_overflow(size, deviation, dtype):
    """The squares' sum is infinite; the centred values' is not."""
    T, H = 5, 7168
    x = (size + deviation * rand(T, H)).to(dtype)
    w, b = rand(H, seed=2, scale=0.3, shift=1.0), rand(H, seed=3)
    if deviation == 0.0:  # every centred value is the mean's error, at most the root of the mean of their squares
        d = epd.ep_layer_norm(x, with_stats=True)
        near(d["mean"], x.double().mean(1), F32 * x.double().abs().amax(1), torch.float32)
        assert bool((d["y"].float().abs() <= 1).all())
        return
    d = epd.ep_layer_norm(x, w, bias=b, with_stats=True)
    s, mean, rstd, y, big = formula(x, None, w, b, 1e-5, "layer")
    near(d["mean"], mean.squeeze(1), F32 * s.abs().amax(1), torch.float32)
    # the mean's error adds its square to the variance: half of (F32 mean rstd)^2 of the root
    off = F32 + (F32 * s.abs().amax(1, keepdim=True) * rstd).square() / 2
    near(d["rstd"], rstd.squeeze(1), (off * rstd).squeeze(1), torch.float32)
    near(d["y"], y, F32 * big + off * (y - b.double()).abs(), torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [128, 512, 1152, 7168, 8320])
def test_e4m3_rows_are_the_rounded_quotients(H, dtype):
    """x = 1 or -1 is its own root-mean-square norm: the rows are the weights, whose e4m3 numbers are those
    of the quotients by the scale, to the last one."""
    T = 700
    x = torch.where(rand(T, H) < 0, -1.0, 1.0).to(dtype)
    for seed in range(20):
        w = rand(H, seed=seed, scale=2.0 ** (seed - 10))
        if seed % 2:
            w = w.bfloat16().float()
        d = epd.ep_layer_norm(x, w, eps=0.0, kind="rms", with_fp8=True)
        b = w.view(-1, 128)
        scale = b.abs().amax(1) / torch.full((H // 128,), 448.0, device=DEV)
        assert torch.equal(d["y_scale"], scale.expand(T, -1))
        want = (x.float() * w).view(T, -1, 128) / scale[:, None].expand(T, -1, 128)
        want = want.clamp(-448, 448).to(torch.float8_e4m3fn).view(T, H)
        assert torch.equal(d["y_q"].float(), want.float())


@pytest.mark.parametrize("power", [-126, -139, -143, -147])
def test_rows_below_448_of_the_smallest_number(power):
    """amax / 448 rounds to 0 below 2^-141: the scale is the smallest number there is then, never 0."""
    x = torch.where(rand(9, 512) < 0, -1.0, 1.0)
    w = rand(512).abs() * 2.0 ** power
    w[::7] = 0.0
    d = epd.ep_layer_norm(x, w, eps=0.0, kind="rms", with_fp8=True)
    y = x.double() * w.double()
    scale = d["y_scale"].double().repeat_interleave(128, 1)
    assert bool((scale > 0).all())
    # half a step of e4m3, and 448 half steps of the scale's own 2^-149
    tol = 2.0 ** -4 * y.abs() + 2.0 ** -10 * scale + 224 * 2.0 ** -149
    assert bool(((d["y_q"].double() * scale - y).abs() <= tol).all())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(700, 128), (5000, 256), (9000, 512), (33, 640), (1300, 1152), (5, 8320), (400, 8320), (170, 16256)])
def test_e4m3_rows_of_ragged_widths(T, H, dtype, residual):
    """Blocks that walk over many rows, and widths whose last groups of 128 some of a block's lanes have and others have not."""
    x, r = rand(T, H, dtype=dtype, scale=2.0, shift=0.7), rand(T, H, seed=1, dtype=dtype) if residual else None
    w, b = rand(H, seed=2, scale=0.3, shift=1.0), rand(H, seed=3)
    d = epd.ep_layer_norm(x, w, bias=b, residual=r, with_fp8=True)
    s, _, _, y, big = formula(x, r, w, b, 1e-5, "layer")
    near(d["y"], y, F32 * big, torch.bfloat16)
    blocks, bigs = y.view(T, -1, 128).abs().amax(2), big.reshape(T, -1, 128).amax(2)
    near(d["y_scale"], blocks / 448, F32 * bigs / 448 + 2.0 ** -24 * blocks / 448, torch.float32)
    scale = d["y_scale"].double().repeat_interleave(128, 1)
    tol = HALF[torch.float8_e4m3fn] * y.abs() + 2.0 ** -10 * scale + 2 * F32 * big
    assert bool(((d["y_q"].double() * scale - y).abs() <= tol).all())
    only = epd.ep_layer_norm(x, w, bias=b, residual=r, with_y=False, with_fp8=True)
    assert torch.equal(only["y_q"].view(torch.uint8), d["y_q"].view(torch.uint8)) and torch.equal(only["y_scale"], d["y_scale"])
