"""A Mixture-of-Experts layer on one GPU, from router logits to the combined rows.

``MoELayer`` is a training layer: routing, dispatch, the experts' two products (SwiGLU
between them), the combine, and the backward pass of all of it, in libepd's operators
(the router's own projection is a plain matrix product). ``decode_step`` is a serving step
for a small batch: the low-latency dispatch casts the tokens to e4m3 rectangles, the first
product reads them with their scales, the second runs in bf16.

Around them: ``MoEBlock`` puts a norm (with the residual in it) ahead of the training layer,
and ``attention_step`` is the other half of a block's decode step -- norm, projection, rotary
positions and the append to the paged cache, attention over it, output projection and residual --
so that ``block_decode_step`` is a whole block in the library's operators.

    python examples/moe_layer.py [--tokens 4096] [--hidden 4096] [--experts 64] [--topk 6]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unpermute_ep_dispatch_gb300 as epd  # noqa: E402


class _NoSecondDerivative(torch.autograd.Function):
    """Passes gradients on; a derivative of them is an error. (``once_differentiable`` sees only
    what depends on the incoming gradient, and these depend on the layer's inputs as well.)"""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of the expert operators have no derivative")


class _Norm(torch.autograd.Function):
    """(norm(x + residual), x + residual): root-mean-square norm with fp32 weights."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        d = epd.ep_layer_norm(x, weight, residual=residual, eps=eps, kind="rms", with_stats=True)
        ctx.save_for_backward(d["sum"], weight, d["rstd"])
        return d["y"], d["sum"]

    @staticmethod
    def backward(ctx, dy, dsum):
        s, weight, rstd = ctx.saved_tensors
        dx, dweight, _ = epd.ep_layer_norm_backward(dy.contiguous(), s, weight, rstd, kind="rms",
                                                    grad_sum=dsum.contiguous())
        grads = dx, dweight
        if torch.is_grad_enabled():  # create_graph
            grads = _NoSecondDerivative.apply(torch.empty(0, requires_grad=True), *grads)
        return grads[0], grads[0], grads[1], None


class _Experts(torch.autograd.Function):
    """y = combine(experts(permute(x))), weighted by the router's top-k weights."""

    @staticmethod
    def forward(ctx, x, logits, w1, b1, w2, b2, layer):
        E, k, status = w1.shape[0], layer.topk, layer.status
        idx, weights = epd.ep_route(logits, k, status, **layer.routing, **layer.choice)
        # a workspace serves one stream at a time: every pass takes its own, from the allocator of
        # the stream that it runs on, and gives it back there
        ws = epd.new_workspace(x.shape[0], k, E, 1, 1, x.device)
        d = epd.ep_dispatch(x, None, idx, E, 1, 1, ws, status, with_is_token_in_rank=False)
        rows = dict(tokens_per_expert=d["tokens_per_expert"], status=status,
                    expert_start_loc=d["expert_start_loc"])
        h, z = epd.ep_expert_matmul(d["out"], w1, bias=b1, activation="swiglu", with_preact=True,
                                    **rows)
        eo, _ = epd.ep_expert_matmul(h, w2, bias=b2, **rows)
        y = epd.ep_unpermute(eo, d["output_index"], weights, status)
        ctx.save_for_backward(logits, w1, w2, idx, weights, d["out"], h, z, eo, d["output_index"],
                              d["tokens_per_expert"], d["expert_start_loc"])
        ctx.layer = layer
        return y

    @staticmethod
    def backward(ctx, dy):
        logits, w1, w2, idx, weights, xp, h, z, eo, index, counts, start = ctx.saved_tensors
        layer, status = ctx.layer, ctx.layer.status
        rows = dict(tokens_per_expert=counts, status=status, expert_start_loc=start)
        deo, dweights = epd.ep_unpermute_backward(dy.contiguous(), eo, index, weights, status)
        dz = epd.ep_expert_matmul_dgrad(deo, w2, activation="swiglu", preact=z, **rows)
        dw2, db2 = epd.ep_expert_matmul_wgrad(deo, h, with_dbias=True, **rows)
        dxp = epd.ep_expert_matmul_dgrad(dz, w1, **rows)
        dw1, db1 = epd.ep_expert_matmul_wgrad(dz, xp, with_dbias=True, **rows)
        # a token's gradient is the sum of its rows': the combine with weights of one
        dx = epd.ep_unpermute(dxp, index, torch.ones_like(weights), status)
        dlogits = epd.ep_route_backward(dweights, logits, idx, status, **layer.routing)
        grads = dx, dlogits, dw1, db1, dw2, db2
        if torch.is_grad_enabled():  # create_graph
            grads = _NoSecondDerivative.apply(torch.empty(0, requires_grad=True), *grads)
        return *grads, None


class MoELayer(torch.nn.Module):
    """bf16 weights and rows, fp32 router logits and biases. ``choice_bias`` [E] steers the
    choice of experts towards balance and is not trained by gradient."""

    def __init__(self, hidden, intermediate, num_experts, topk, scoring="softmax", num_groups=1,
                 topk_groups=1, group_score="max", choice_bias=None, device="cuda"):
        super().__init__()

        def weight(*shape):
            return torch.nn.Parameter(torch.randn(*shape, device=device, dtype=torch.bfloat16)
                                      / math.sqrt(shape[-1]))
        self.router = torch.nn.Parameter(torch.randn(num_experts, hidden, device=device)
                                         / math.sqrt(hidden))
        self.w1 = weight(num_experts, 2 * intermediate, hidden)
        self.b1 = torch.nn.Parameter(torch.zeros(num_experts, 2 * intermediate, device=device))
        self.w2 = weight(num_experts, hidden, intermediate)
        self.b2 = torch.nn.Parameter(torch.zeros(num_experts, hidden, device=device))
        self.topk = topk
        self.routing = dict(scoring=scoring, renormalize=True)
        self.choice = dict(bias=choice_bias, num_groups=num_groups, topk_groups=topk_groups,
                           group_score=group_score)
        self.status = epd.new_status(device)

    def forward(self, x):
        logits = x.float() @ self.router.t()
        return _Experts.apply(x, logits, self.w1, self.b1, self.w2, self.b2, self)


class MoEBlock(torch.nn.Module):
    """The MoE half of a block: the residual stream joined and normed, then the layer. Returns the
    layer's rows and the residual stream, which the next norm adds up."""

    def __init__(self, hidden, *args, eps=1e-5, device="cuda", **kw):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device))
        self.eps = eps
        self.layer = MoELayer(hidden, *args, device=device, **kw)

    def forward(self, x, residual):
        y, stream = _Norm.apply(x, residual, self.weight, self.eps)
        return self.layer(y), stream


def quantize_blocks(w):
    """e4m3 weights [E, N, K] with one fp32 scale per 128 x 128 block (N, K multiples of 128)."""
    E, N, K = w.shape
    b = w.float().view(E, N // 128, 128, K // 128, 128)
    scale = b.abs().amax((2, 4)).clamp(min=1e-12) / 448.0
    q = (b / scale[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(E, N, K), scale


def decode_step(x, logits, w1_q, w1_scale, w2, topk, workspace, status, rows_per_expert=None,
                **routing):
    """One serving step: x [T, H] bf16, w1_q [E, 2N, H] e4m3 with its block scales, w2 [E, H, N]
    bf16. Every expert has a rectangle of rows_per_expert rows (T always suffices)."""
    T, H = x.shape
    E = w1_q.shape[0]
    rows = T if rows_per_expert is None else rows_per_expert
    idx, weights = epd.ep_route(logits, topk, status, **routing)
    q, scale, count, index, _ = epd.ep_dispatch_lowlatency(x, idx, E, 1, 1, rows, workspace,
                                                           status, with_src_token=False)
    h, _ = epd.ep_expert_matmul(q, w1_q, count, status, x_scale=scale, w_scale=w1_scale,
                                activation="swiglu")
    eo, _ = epd.ep_expert_matmul(h, w2, count, status)
    return epd.ep_unpermute(eo.view(E * rows, H), index, weights, status)


def attention_step(x, norm_weight, w_qkv, w_o, heads, kv_heads, cache, lengths, positions, steps,
                   workspace, status, eps=1e-5):
    """The attention half of a block for one new token of every sequence: x [B, H] bf16, the
    residual stream. w_qkv [(heads + 2 kv_heads) D, H] and w_o [H, heads D] bf16; cache: a dict of
    k_cache, v_cache, page_table (and the scales of an e4m3 cache); positions [B] int32 of the new
    tokens, lengths = positions + 1. Returns x + attention(norm(x)) [B, H]."""
    B, H = x.shape
    y = epd.ep_layer_norm(x, norm_weight, eps=eps, kind="rms")["y"]
    # one expert over all rows is an ordinary linear layer
    rows = dict(tokens_per_expert=torch.full((1,), B, dtype=torch.int32, device=x.device),
                expert_start_loc=torch.zeros(1, dtype=torch.int32, device=x.device), status=status)
    qkv, _ = epd.ep_expert_matmul(y, w_qkv.unsqueeze(0), **rows)
    qkv = qkv.view(B, heads + 2 * kv_heads, -1)
    q = epd.ep_cache_append(qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:],
                            positions=positions, status=status, q=qkv[:, :heads], steps=steps, **cache)
    o, _ = epd.ep_decode_attention(q, lengths=lengths, workspace=workspace, status=status, **cache)
    return epd.ep_expert_matmul(o.view(B, -1), w_o.unsqueeze(0), residual=x, **rows)[0]


def block_decode_step(x, attention, norm_weight, router, experts, eps=1e-5):
    """A whole block for one new token of every sequence: `attention` are attention_step's
    arguments after x, `experts` decode_step's after the logits. Returns the residual stream."""
    x = attention_step(x, **attention)
    y = epd.ep_layer_norm(x, norm_weight, eps=eps, kind="rms")["y"]
    return x + decode_step(y, y.float() @ router.t(), **experts)


def _time(f, n=10):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--intermediate", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    args = ap.parse_args()
    T, H, N, E, k = args.tokens, args.hidden, args.intermediate, args.experts, args.topk
    layer = MoELayer(H, N, E, k)
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    dy = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)

    def train():
        layer.zero_grad(set_to_none=True)
        x.grad = None
        layer(x).backward(dy)
    ms = _time(train)
    epd.check_status(layer.status, "training step")
    flops = 3 * 2 * T * k * 3 * H * N
    print(f"training step: T={T} H={H} N={N} E={E} k={k}: {ms:.3f} ms, "
          f"{flops / ms / 1e9:.0f} TFLOP/s over forward and backward")

    t = min(T, 128)
    w1_q, w1_scale = quantize_blocks(layer.w1.detach())
    ws = epd.new_workspace(t, k, E, 1, 1)
    xs = x.detach()[:t].contiguous()
    with torch.no_grad():
        logits = xs.float() @ layer.router.t()
        ms = _time(lambda: decode_step(xs, logits, w1_q, w1_scale, layer.w2.detach(), k, ws,
                                       layer.status))
    epd.check_status(layer.status, "decode step")
    print(f"decode step: T={t}: {ms * 1e3:.1f} us")

    QH, KH, D, page, length = 32, 8, 128, 64, 4096
    pages = -(-length // page)
    kv = [torch.randn(t * pages, page, KH, D, device="cuda").bfloat16() for _ in range(2)]
    positions = torch.full((t,), length - 1, dtype=torch.int32, device="cuda")
    attention = dict(
        norm_weight=torch.ones(H, device="cuda"), heads=QH, kv_heads=KH,
        w_qkv=(torch.randn((QH + 2 * KH) * D, H, device="cuda") / math.sqrt(H)).bfloat16(),
        w_o=(torch.randn(H, QH * D, device="cuda") / math.sqrt(QH * D)).bfloat16(),
        cache=dict(k_cache=kv[0], v_cache=kv[1], page_table=torch.randperm(
            t * pages, device="cuda").int().view(t, pages)),
        positions=positions, lengths=positions + 1, status=layer.status,
        steps=epd.rotary_steps(epd.rotary_frequencies(D)[0], "cuda"),
        workspace=epd.new_attention_workspace(t, QH, KH, D))
    experts = dict(w1_q=w1_q, w1_scale=w1_scale, w2=layer.w2.detach(), topk=k, workspace=ws,
                   status=layer.status)
    with torch.no_grad():
        ms = _time(lambda: block_decode_step(xs, attention, torch.ones(H, device="cuda"),
                                             layer.router, experts))
    epd.check_status(layer.status, "block decode step")
    print(f"block decode step: T={t}, {QH} / {KH} heads of {D}, {length} positions: {ms * 1e3:.1f} us")


if __name__ == "__main__":
    main()
