"""Layer calls on a stream other than the caller's own: whose memory results and workspaces are, and
when it is given back.  A stream is held back by a sleeping kernel, so that the order of what follows on
it is known."""
import pytest
import torch

from tests.test_mxfp4_gpu import Case
from tests.test_mxfp4_streams_gpu import _hold, other  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

KW = dict(d=512, E=16, k=4, f=256)


def _calls(layer):
    """name: call(x, stream) -> list of results, for a layer of either kind."""
    return dict(
        forward=lambda x, s: [layer.forward(x, stream=s)],
        forward_few=lambda x, s: [layer.forward_few(x[:16], stream=s)],
        route=lambda x, s: list(layer.route(x=x, want_logits=True, stream=s).values()),
        router_logits_static=lambda x, s: [layer.router_logits_static(x[:16], stream=s)])


NAMES = ["forward", "forward_few", "route", "router_logits_static"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("mx", [False, True])
def test_results_on_another_stream(other, name, mx):  # noqa: F811
    """No result takes a block that the caller's stream still uses; none dropped early, or read by the
    caller and dropped, is given to anyone else too soon."""
    c = Case(T=100, **KW)
    layer = c.layer(mx)
    call = _calls(layer)[name]
    want = [t.clone() for t in call(c.x, None)]
    torch.cuda.synchronize()
    # in use on the caller's stream
    blocks = [torch.empty_like(t) for t in want for _ in range(2)]
    torch.cuda.synchronize()
    _hold()
    for b in blocks:
        b.fill_(1)
    del b, blocks
    got = call(c.x, other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # dropped before it is written
    del got
    _hold(other)
    call(c.x, other)
    fresh = [torch.empty_like(t).fill_(3) for t in want for _ in range(3)]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in fresh)
    # read by the caller, who has waited for it, and dropped while the read is held back
    got = call(c.x, other)
    torch.cuda.current_stream().wait_stream(other)
    _hold()
    read = [t.clone() for t in got]
    del got
    x2 = Case(T=100, seed=1, **KW).x
    again = call(x2, other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
    assert not all(torch.equal(a, b) for a, b in zip(again, want))
    assert layer.device_status() == 0


@pytest.mark.parametrize("T1,T2", [(4, 60), (60, 300), (200, 300)])
@pytest.mark.parametrize("mx", [False, True])
def test_workspace_replaced_while_in_use(other, mx, T1, T2):  # noqa: F811
    """A larger call replaces the workspace that a call on another stream still uses: its memory is not
    handed out before that call is done."""
    c = Case(T=T2, **KW)
    x1 = c.x[:T1].contiguous()
    want1 = c.layer(mx).forward(x1).clone()
    want2 = c.layer(mx).forward(c.x).clone()
    layer = c.layer(mx)
    size = layer.workspace(T1).numel()
    torch.cuda.synchronize()
    out1 = torch.empty_like(x1)
    _hold(other)
    layer.forward(x1, out=out1, stream=other)
    out2 = layer.forward(c.x)
    assert layer.ws.numel() > size
    fresh = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out1, want1) and torch.equal(out2, want2)
    assert all((t == 255).all() for t in fresh)
    assert layer.device_status() == 0


@pytest.mark.parametrize("mx", [False, True])
def test_workspace_reserved_for_another_stream(other, mx):  # noqa: F811
    """workspace(T) on the caller's stream, which is held back, then the first call on another."""
    c = Case(T=70, **KW)
    want = c.layer(mx).forward(c.x).clone()
    layer = c.layer(mx)
    torch.cuda.synchronize()
    _hold()
    layer.workspace(70)
    out = torch.empty_like(c.x)
    layer.forward(c.x, out=out, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and layer.device_status() == 0


def test_training_calls_on_another_stream(other):  # noqa: F811
    """The first forward_save and backward of a layer, on a stream beside a held-back caller's."""
    c = Case(T=40, **KW)
    layer, dout = c.layer(False), c.x.flip(0).contiguous()
    out, saved = layer.forward_save(c.x)
    want = [out, *layer.backward(c.x, dout, saved=saved).values()]
    stats = layer.router_stats(*(layer.route(x=c.x, want_logits=True)[n] for n in ("logits", "idx")),
                               n_groups=4)
    health = layer.expert_health(40)
    torch.cuda.synchronize()
    layer = c.layer(False)
    _hold()
    out, saved = layer.forward_save(c.x, stream=other)
    got = [out, *layer.backward(c.x, dout, saved=saved, stream=other).values()]
    h = layer.expert_health(40, stream=other)
    r = layer.route(x=c.x, want_logits=True, stream=other)
    s = layer.router_stats(r["logits"], r["idx"], n_groups=4, stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip((*h, *s), (*health, *stats)))
    assert layer.device_status() == 0


def _capture(call):
    """The call in a graph, after one of the same on a side stream."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [16, 100])
def test_graph_replayed_after_a_larger_call(cuda_ok, mx, T):
    """The workspace of a captured call outlives its replacement by a larger call's."""
    c = Case(T=300, **KW)
    x = c.x[:T].contiguous()
    layer, out = c.layer(mx), torch.empty_like(x)
    want, want_big = c.layer(mx).forward(x).clone(), c.layer(mx).forward(c.x).clone()
    g = _capture(lambda: layer.forward(x, out=out))
    size = layer.ws.numel()
    assert torch.equal(layer.forward(c.x), want_big)
    assert layer.ws.numel() > size
    fresh = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(layer.forward(c.x), want_big)
    assert all((t == 255).all() for t in fresh)
    assert layer.device_status() == 0


def test_backward_graph_replayed_after_a_larger_call(cuda_ok):
    c = Case(T=100, **KW)
    x, dout = c.x[:8].contiguous(), c.x[8:16].contiguous()
    layer = c.layer(False)
    grads = {n: t for n, t in layer.backward(x, dout).items() if n != "dx"}
    want = {n: t.clone() for n, t in grads.items()}
    res = {}

    def step():
        res["g"] = layer.backward(x, dout, grads=grads, overwrite=True)

    g = _capture(step)
    size = layer.bw_ws.numel()
    layer.backward(c.x, c.x)
    assert layer.bw_ws.numel() > size
    fresh = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
    for t in grads.values():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(grads[n], want[n]) for n in want)
    assert all((t == 255).all() for t in fresh)
    assert layer.device_status() == 0


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [16, 100])
def test_first_call_of_a_layer_captured(cuda_ok, mx, T):
    """A workspace allocated by a captured call is cleared in every replay, and by the first call outside
    the graph; whatever its memory held before."""
    c = Case(T=T, **KW)
    want = c.layer(mx).forward(c.x).clone()
    layer, out = c.layer(mx), torch.empty_like(c.x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(c.x, out=out)
    layer.ws.fill_(0xAB)
    assert torch.equal(layer.forward(c.x), want)
    layer.ws.fill_(0xAB)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(layer.forward(c.x), want)
    assert layer.device_status() == 0


@pytest.mark.parametrize("T", [10, 200])
def test_layer_dropped_while_a_call_runs(other, T):  # noqa: F811
    """A converted layer holds the only references to its codes and scales: dropped while a call on another
    stream is still to run, it gives them (and the workspace) back only after that call."""
    c = Case(T=T, **KW)
    trained = c.layer(False)
    want = trained.to_mxfp4().forward(c.x).clone()
    served = trained.to_mxfp4()
    shapes = [t.shape for w in served.tensors[2:] for t in w]
    out = torch.empty_like(c.x)
    torch.cuda.synchronize()
    _hold(other)
    served.forward(c.x, out=out, stream=other)
    del served
    fresh = [torch.empty(s, dtype=torch.uint8, device="cuda").fill_(255) for s in shapes
             for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all((t == 255).all() for t in fresh)


@pytest.mark.parametrize("mx", [False, True])
def test_workspace_of_a_captured_call_reserved_for_another_stream(other, mx):  # noqa: F811
    """workspace(T) on the caller's stream, held back, after a layer's first call was captured; then the
    first call outside the graph on another stream."""
    c = Case(T=70, **KW)
    want = c.layer(mx).forward(c.x).clone()
    layer, out = c.layer(mx), torch.empty_like(c.x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(c.x, out=out)
    got = torch.empty_like(c.x)
    layer.ws.fill_(0xAB)
    _hold()
    layer.workspace(70)
    layer.forward(c.x, out=got, stream=other)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want)
    assert layer.device_status() == 0
