"""The example layer under several streams and a second derivative."""
import pytest
import torch

import unpermute_ep_dispatch_gb300 as epd

pytestmark = pytest.mark.gpu


def test_passes_on_two_streams_share_no_workspace(monkeypatch):
    """A workspace serves one stream at a time (epd.h): passes of one layer that may run at the
    same time must not meet in one."""
    from examples.moe_layer import MoELayer
    torch.manual_seed(0)
    layer = MoELayer(256, 128, 12, 3)
    x = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    want = layer(x)
    used, dispatch = [], epd.ep_dispatch

    def watched(rows, scale, idx, E, R, N, workspace, *args, **kw):
        start = workspace.data_ptr()
        used.append((torch.cuda.current_stream().cuda_stream, start, start + workspace.numel()))
        return dispatch(rows, scale, idx, E, R, N, workspace, *args, **kw)

    monkeypatch.setattr(epd, "ep_dispatch", watched)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [[], []]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[i].append(layer(x))
    torch.cuda.synchronize()
    epd.check_status(layer.status, "layer")
    assert len(used) == 8
    for a in used:
        for b in used:
            assert a[0] == b[0] or a[2] <= b[1] or b[2] <= a[1], "two streams in one workspace"
    for y in out[0] + out[1]:
        assert torch.equal(y, want)


def test_batches_of_many_sizes_leave_nothing_behind():
    from examples.moe_layer import MoELayer
    layer = MoELayer(64, 32, 16, 2)

    def run(tokens):
        with torch.no_grad():
            layer(torch.zeros(tokens, 64, device="cuda", dtype=torch.bfloat16))
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated()
    first = run(1)
    assert all(run(t) <= first for t in range(2, 40))


def test_second_derivative_is_refused():
    """The gradients have none of their own: a loss that needs it is an error, not a wrong number."""
    from examples.moe_layer import MoELayer
    layer = MoELayer(64, 32, 16, 2)
    x = torch.randn(20, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    dx, = torch.autograd.grad(layer(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        (layer(x).float().sum() + dx.float().pow(2).sum()).backward()
