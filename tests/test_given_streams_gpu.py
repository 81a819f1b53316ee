"""Calls on a given stream whose outputs the call allocates: their memory is the given stream's, none that the
current stream may still have work on."""
import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
T, H, E, k = 300, 256, 8, 2


def rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(77 + seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def operators():
    status, x = epd.new_status(DEV), rand(T, H)
    logits, weight = rand(T, E, dtype=torch.float32, seed=1), rand(H, dtype=torch.float32, seed=2)
    idx, top = epd.ep_route(logits, k, status)
    ws = epd.new_workspace(T, k, E, 1, 1, DEV)
    d = epd.ep_dispatch(x, None, idx, E, 1, 1, ws, status)
    w = rand(E, 128, H, seed=3)
    rows = dict(tokens_per_expert=d["tokens_per_expert"], status=status, expert_start_loc=d["expert_start_loc"])
    dy = rand(d["out"].shape[0], 128, seed=4)
    rstd = rand(T, dtype=torch.float32, seed=5).abs()
    heads, pos = rand(T, 4, 64, seed=6), torch.arange(T, dtype=torch.int32, device=DEV)
    steps = epd.rotary_steps(epd.rotary_frequencies(64)[0], DEV)
    kv = [torch.zeros(T, 1, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table, one = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1), torch.ones(T, dtype=torch.int32, device=DEV)
    aws = epd.new_attention_workspace(T, 4, 2, 64, DEV)
    kw = dict(workspace=ws, status=status)
    return {
        "route": lambda **s: epd.ep_route(logits, k, status, **s),
        "route_backward": lambda **s: epd.ep_route_backward(top, logits, idx, status, **s),
        "dispatch": lambda **s: epd.ep_dispatch(x, None, idx, E, 1, 1, ws, status, **s),
        "layout": lambda **s: epd.ep_dispatch_layout(idx, E, 1, 1, **kw, **s),
        "unpermute": lambda **s: epd.ep_unpermute(d["out"], d["output_index"], top, status, **s),
        "unpermute_backward": lambda **s: epd.ep_unpermute_backward(x, d["out"], d["output_index"], top, status, **s),
        "matmul": lambda **s: epd.ep_expert_matmul(d["out"], w, with_preact=True, **rows, **s),
        "dgrad": lambda **s: epd.ep_expert_matmul_dgrad(dy, w, **rows, **s),
        "wgrad": lambda **s: epd.ep_expert_matmul_wgrad(dy, d["out"], with_dbias=True, **rows, **s),
        "norm": lambda **s: epd.ep_layer_norm(x, weight, residual=x, with_fp8=True, with_stats=True, **s),
        "norm_backward": lambda **s: epd.ep_layer_norm_backward(x, x, weight, rstd, kind="rms", with_dbias=True, **s),
        "rotary": lambda **s: epd.ep_rotary(heads, pos, steps, **s),
        "append": lambda **s: epd.ep_cache_append(heads[:, :2], heads[:, 2:], *kv, table, pos * 0, status, q=heads, steps=steps, **s),
        "attention": lambda **s: epd.ep_decode_attention(heads, *kv, table, one, aws, status, with_lse=True, **s),
    }


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


@pytest.mark.parametrize("name", ["route", "route_backward", "dispatch", "layout", "unpermute", "unpermute_backward", "matmul", "dgrad",
                                  "wgrad", "norm", "norm_backward", "rotary", "append", "attention"])
def test_outputs_belong_to_the_given_stream(name):
    op = operators()[name]
    side = torch.cuda.Stream()
    op(), op(stream=side)
    torch.cuda.synchronize()
    out = tensors(op())
    want = [t.clone() for t in out]
    torch.cuda.synchronize()
    places = {t.data_ptr() for t in out}
    torch.cuda._sleep(2_000_000)  # the current stream is behind, and what it holds is let go
    del out
    got = tensors(op(stream=side))
    assert len(got) == len(want) and not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        if name not in ("dispatch", "matmul", "unpermute_backward", "dgrad"):  # (rows past the last are no one's)
            assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


@pytest.mark.parametrize("name", ["dispatch", "norm", "norm_backward", "append", "attention"])
def test_given_streams_in_a_graph(name):
    """A captured call on a stream that the capture forks to, its outputs used on the first one."""
    op = operators()[name]
    side = torch.cuda.Stream()
    op(stream=side)
    torch.cuda.synchronize()
    want = [t.clone() for t in tensors(op())]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = tensors(op(stream=side))
        torch.cuda.current_stream().wait_stream(side)
        got = [t.clone() for t in out]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        if name != "dispatch":  # (rows past the last are no one's)
            assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
