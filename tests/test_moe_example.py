"""The example layer: routing, dispatch, products, combine and all their gradients together,
against the same layer in 64 bits."""
import math

import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd

pytestmark = pytest.mark.gpu


def layer64(x, router, w1, b1, w2, b2, idx):
    """y of the layer in 64 bits for the given picks (differentiable)."""
    T, k = idx.shape
    p = torch.softmax(x @ router.t(), 1).gather(1, idx)
    p = p / p.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        a, u = (x[t] @ w1[e].t() + b1[e]).chunk(2, 1)
        h = a * torch.sigmoid(a) * u
        y = y.index_add(0, t, (h @ w2[e].t() + b2[e]) * p[t, j].unsqueeze(1))
    return y


@pytest.mark.parametrize("T,H,N,E,k", [(200, 256, 128, 12, 3), (33, 520, 136, 40, 2), (1, 64, 32, 4, 4)])
def test_training_layer(T, H, N, E, k):
    from examples.moe_layer import MoELayer
    torch.manual_seed(T)
    layer = MoELayer(H, N, E, k)
    with torch.no_grad():
        layer.b1.normal_(std=0.3)
        layer.b2.normal_(std=0.3)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16).requires_grad_()
    dy = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    y = layer(x)
    y.backward(dy)
    torch.cuda.synchronize()
    epd.check_status(layer.status, "layer")
    # the picks, as the layer's own logits give them
    idx, _ = epd.ep_route(x.detach().float() @ layer.router.detach().t(), k, layer.status)
    args = [t.detach().double().requires_grad_() for t in (x, layer.router, layer.w1, layer.b1, layer.w2, layer.b2)]
    want = layer64(*args, idx)
    want.backward(dy.double())
    # z, h, the experts' rows, their gradients and the results are rounded to bf16 on the way, each
    # by at most 2^-9 of its value; five such roundings in a row, taken as independent of sign at
    # worst, are 5 * 2^-9 of the norms that they pass through; twice that is allowed
    tol = 10 * 2 ** -9
    assert (y.double() - want).norm() <= tol * want.norm()
    for got, a, name in zip((x, layer.router, layer.w1, layer.b1, layer.w2, layer.b2), args,
                            ("x", "router", "w1", "b1", "w2", "b2")):
        assert (got.grad.double() - a.grad).norm() <= tol * a.grad.norm() + 1e-6, name


def test_decode_step():
    from examples.moe_layer import decode_step, quantize_blocks
    T, H, N, E, k = 50, 512, 256, 24, 4
    torch.manual_seed(3)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w1 = torch.randn(E, 2 * N, H, device="cuda") / math.sqrt(H)
    w2 = (torch.randn(E, H, N, device="cuda") / math.sqrt(N)).to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda")
    q, s = quantize_blocks(w1)
    status = epd.new_status()
    ws = epd.new_workspace(T, k, E, 1, 1)
    y = decode_step(x, logits, q, s, w2, k, ws, status)
    torch.cuda.synchronize()
    epd.check_status(status, "decode")
    idx, _ = epd.ep_route(logits, k, status)
    wd = q.double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    # the cast of the low-latency dispatch: per 128 columns, amax / 448
    b = x.float().view(T, H // 128, 128)
    xs = b.abs().amax(2, keepdim=True) / 448
    xd = ((b / xs).to(torch.float8_e4m3fn).double() * xs.double()).view(T, H)
    p = torch.softmax(logits.double(), 1).gather(1, idx)
    p = p / p.sum(1, keepdim=True)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            a, u = (wd[e] @ xd[t]).chunk(2)
            want[t] += p[t, j] * (w2[e].double() @ (a * torch.sigmoid(a) * u))
    # three roundings to bf16 (h, the experts' rows, y), as above
    assert (y.double() - want).norm() <= 6 * 2 ** -9 * want.norm()
