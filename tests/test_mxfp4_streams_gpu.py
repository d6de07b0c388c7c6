"""Calls on a stream other than the caller's own: whose memory results, inputs and workspaces are, and
when it is given back.  A stream is held back by a sleeping kernel, so that the order of what follows on
it is known."""
import pytest
import torch

from sparse_moe_layer_warp_b200 import mxfp4_dequantize, mxfp4_quantize

pytestmark = pytest.mark.gpu

HOLD = 40_000_000  # clocks: 20 ms or more


def _hold(stream=None):
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        torch.cuda._sleep(HOLD)


def _matrix(seed, rows=512, cols=1024):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=gen, device="cuda").to(torch.bfloat16)


@pytest.fixture
def other(cuda_ok):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    yield torch.cuda.Stream()
    torch.cuda.synchronize()


def test_result_is_not_a_block_in_use_on_the_callers_stream(other):
    """A block freed on the caller's stream, which still writes it, is not handed out for a result on
    another."""
    w = _matrix(0)
    want = mxfp4_quantize(w)
    want_back = mxfp4_dequantize(*want)
    blocks = [torch.empty_like(t) for t in (*want, want_back)]
    torch.cuda.synchronize()
    _hold()
    for b in blocks:
        b.fill_(1)
    del b, blocks
    got = mxfp4_quantize(w, stream=other)
    back = mxfp4_dequantize(*got, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(back, want_back)


def test_result_dropped_before_it_is_written(other):
    w = _matrix(1)
    torch.cuda.synchronize()
    _hold(other)
    shapes = [(t.shape, t.dtype) for t in mxfp4_quantize(w, stream=other)]  # dropped at once
    fresh = [torch.empty(s, dtype=d, device="cuda").fill_(3) for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in fresh)


def test_input_dropped_before_it_is_read(other):
    w = _matrix(2)
    want = mxfp4_quantize(w)
    torch.cuda.synchronize()
    _hold(other)
    got = mxfp4_quantize(w, stream=other)
    shape = w.shape
    del w
    fresh = [torch.empty(shape, dtype=torch.bfloat16, device="cuda").fill_(7) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all((t == 7).all() for t in fresh)


def test_result_read_by_the_caller_then_dropped(other):
    """The caller's stream waits for the other, reads a result and drops it: the next call's result may
    not take its place before that."""
    a, b = _matrix(3), _matrix(4)
    want_a, want_b = mxfp4_quantize(a), mxfp4_quantize(b)
    torch.cuda.synchronize()
    got = mxfp4_quantize(a, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    _hold()
    read = [t.clone() for t in got]
    del got
    got_b = mxfp4_quantize(b, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(read[0], want_a[0]) and torch.equal(read[1], want_a[1])
    assert torch.equal(got_b[0], want_b[0]) and torch.equal(got_b[1], want_b[1])


def test_external_stream(other):
    w = _matrix(5)
    want = mxfp4_quantize(w)
    torch.cuda.synchronize()
    got = mxfp4_quantize(w, stream=torch.cuda.ExternalStream(other.cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
