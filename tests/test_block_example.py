"""The example's block: norms, projections, rotary positions, the paged cache, decode attention and the
layer together, against the same block in 64 bits."""
import math

import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd
from cache_formulas import attend, paged, turn, values

pytestmark = pytest.mark.gpu


def rms(x, w, eps=1e-5):
    return x * (x.square().mean(1, keepdim=True) + eps).rsqrt() * w.double()


def parts(B, H, QH, KH, D, page, length, fp8, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, by=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * by
    pages = -(-(length + 4) // page)
    k, v, ks, vs = paged(B * pages, page, KH, D, fp8, "cuda", g)
    cache = dict(k_cache=k, v_cache=v,
                 page_table=torch.randperm(B * pages, generator=g, device="cuda").int().view(B, pages))
    if fp8:
        cache.update(k_scale=ks, v_scale=vs)
    positions = torch.randint(0, length, (B,), generator=g, device="cuda", dtype=torch.int32)
    f, _ = epd.rotary_frequencies(D)
    return f, dict(norm_weight=1 + 0.2 * normal(H), w_qkv=normal((QH + 2 * KH) * D, H, by=1 / math.sqrt(H)).bfloat16(),
                   w_o=normal(H, QH * D, by=1 / math.sqrt(QH * D)).bfloat16(), heads=QH, kv_heads=KH, cache=cache,
                   positions=positions, lengths=positions + 1, steps=epd.rotary_steps(f, "cuda"),
                   workspace=epd.new_attention_workspace(B, QH, KH, D), status=epd.new_status())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,H,QH,KH,D,page,length", [(5, 256, 8, 2, 64, 16, 300), (1, 512, 4, 4, 128, 64, 1000), (33, 136, 7, 1, 80, 8, 40)])
def test_attention_step(B, H, QH, KH, D, page, length, fp8):
    from examples.moe_layer import attention_step
    f, a = parts(B, H, QH, KH, D, page, length, fp8)
    x = torch.randn(B, H, device="cuda").bfloat16()
    for _ in range(3):  # three tokens one after another
        cache = a["cache"]
        k, v = (values(cache[n + "_cache"], cache.get(n + "_scale")) for n in ("k", "v"))
        qkv = (rms(x.double(), a["norm_weight"]) @ a["w_qkv"].double().t()).view(B, QH + 2 * KH, D)
        turned = turn(qkv[:, :QH + KH], a["positions"], f)
        at = cache["page_table"][torch.arange(B), a["positions"].long() // page].long(), a["positions"].long() % page
        k[at], v[at] = turned[:, QH:], qkv[:, QH + KH:]
        o, _ = attend(turned[:, :QH], k, v, cache["page_table"], a["lengths"])
        want = o.reshape(B, -1) @ a["w_o"].double().t()
        y = attention_step(x, **a)
        epd.check_status(a["status"])
        # y, qkv, q and k, o and the result are rounded to bf16 on the way, each by 2^-9 of its value on
        # average at most (e4m3 keys and values of one of the positions by 2^-5): five in a row and a
        # softmax between, twice over; the last also rounds the residual's part
        tol = (10 * 2 ** -9 + (2 ** -5 if fp8 else 0)) * want.norm() + 2 ** -9 * x.double().norm()
        assert (y.double() - x.double() - want).norm() <= tol
        a["positions"] += 1
        a["lengths"] += 1
        x = y


def test_block_decode_step_in_a_graph():
    """Every operator of a block captured once, then replayed for one token after another."""
    from examples.moe_layer import attention_step, block_decode_step, decode_step, quantize_blocks
    B, H, QH, KH, D, E, N, topk = 16, 256, 8, 2, 64, 8, 128, 2
    torch.manual_seed(3)
    w1, scale = quantize_blocks(torch.randn(E, 2 * N, H, device="cuda") / 16)
    w2 = (torch.randn(E, H, N, device="cuda") / 16).bfloat16()
    router, weight = torch.randn(E, H, device="cuda") / 16, torch.ones(H, device="cuda")
    x = torch.randn(B, H, device="cuda").bfloat16()
    results = []
    for captured in (False, True):
        _, a = parts(B, H, QH, KH, D, 16, 100, True, seed=7)
        experts = dict(w1_q=w1, w1_scale=scale, w2=w2, topk=topk, status=a["status"], workspace=epd.new_workspace(B, topk, E, 1, 1))
        state, out = x.clone(), []
        step = lambda: block_decode_step(state, a, weight, router, experts)  # noqa: E731
        if captured:
            fresh = [t.clone() for t in (a["cache"]["k_cache"].view(torch.uint8), a["cache"]["v_cache"].view(torch.uint8))]
            step()
            a["cache"]["k_cache"].view(torch.uint8).copy_(fresh[0])
            a["cache"]["v_cache"].view(torch.uint8).copy_(fresh[1])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = step()
        for _ in range(4):
            if captured:
                graph.replay()
            else:
                y = step()
            out.append(y.clone())
            state.copy_(y)
            a["positions"] += 1
            a["lengths"] += 1
        epd.check_status(a["status"])
        results.append(torch.stack(out))
    assert torch.equal(results[0], results[1]) and bool(results[0].isfinite().all())
    # the block is its halves
    _, a = parts(B, H, QH, KH, D, 16, 100, True, seed=7)
    mid = attention_step(x, **a)
    y = epd.ep_layer_norm(mid, weight, kind="rms")["y"]
    moe = decode_step(y, y.float() @ router.t(), w1, scale, w2, topk, epd.new_workspace(B, topk, E, 1, 1), a["status"])
    assert torch.equal(mid + moe, results[0][0])


def test_training_block():
    """y + stream of the norm with its residual and the layer, and all gradients."""
    from examples.moe_layer import MoEBlock
    from test_moe_example import layer64
    torch.manual_seed(5)
    T, H, N, E, k = 150, 256, 128, 12, 3
    block = MoEBlock(H, N, E, k)
    with torch.no_grad():
        block.weight.normal_(1.0, 0.2)
        block.layer.b1.normal_(std=0.3)
        block.layer.b2.normal_(std=0.3)
    x, r = (torch.randn(T, H, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    dy, ds = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(2))
    y, stream = block(x, r)
    torch.autograd.backward((y, stream), (dy, ds))
    epd.check_status(block.layer.status)
    normed = epd.ep_layer_norm(x.detach(), block.weight.detach(), residual=r.detach(), kind="rms")["y"]
    idx, _ = epd.ep_route(normed.float() @ block.layer.router.detach().t(), k, block.layer.status)
    p = (x, r, block.weight, block.layer.router, block.layer.w1, block.layer.b1, block.layer.w2, block.layer.b2)
    a = [t.detach().double().requires_grad_() for t in p]
    s = a[0] + a[1]
    want = layer64(s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt() * a[2], *a[3:], idx)
    torch.autograd.backward((want, s), (dy.double(), ds.double()))
    # the layer's five roundings of bf16, the norm's and its gradient's two each, twice over
    tol = 18 * 2 ** -9
    assert (y.double() - want).norm() <= tol * want.norm()
    assert (stream.double() - s).norm() <= 2 ** -9 * s.norm()
    for got, v, name in zip(p, a, ("x", "residual", "weight", "router", "w1", "b1", "w2", "b2")):
        assert (got.grad.double() - v.grad).norm() <= tol * v.grad.norm() + 1e-6, name


def test_training_block_second_derivative_is_an_error():
    from examples.moe_layer import MoEBlock
    block = MoEBlock(64, 32, 4, 2)
    x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_()
    y, _ = block(x, x.detach())
    g, = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        g.float().sum().backward()


def test_captured_training_pass_of_the_norm():
    """Forward and backward in one CUDA graph. (Torch ties a leaf's gradient to the stream of the graph
    that first used it: no eager graph of the captured leaves may be alive, with any operators.)"""
    from examples.moe_layer import _Norm
    x, r = (torch.randn(40, 256, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(256, device="cuda")
    dy = torch.randn(40, 256, device="cuda").bfloat16()

    def grads(*leaves):
        leaves = [t.detach().requires_grad_() for t in leaves]
        return torch.autograd.grad(_Norm.apply(*leaves, 1e-5)[0], leaves, dy)
    want = [t.clone() for t in grads(x, r, w)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(x, r, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads(x, r, w)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
