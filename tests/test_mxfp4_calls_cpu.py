"""What the Python calls of the MXFP4 operators refuse before anything reaches the library.  No GPU."""
import pytest
import torch

from sparse_moe_layer_warp_b200 import binding


def test_dequantise_refuses_strided_scales():
    """The library reads the scales as dense memory, as it does the codes."""
    codes = torch.zeros(4, 32, dtype=torch.uint8)
    wide = torch.zeros(4, 4, dtype=torch.uint8)
    for scales in (wide[:, :2], wide[:, ::2], torch.zeros(2, 4, dtype=torch.uint8).t(),
                   torch.zeros(1, 2, dtype=torch.uint8).expand(4, 2)):
        assert scales.shape == (4, 2)
        with pytest.raises(ValueError, match="contiguous"):
            binding.mxfp4_dequantize(codes, scales)
    with pytest.raises(ValueError, match="contiguous"):
        binding.mxfp4_dequantize(torch.zeros(32, 4, dtype=torch.uint8).t(), wide[:, :2].contiguous())


def _layer_tensors(mx, E=4, d=256, f=128):
    """Arguments of a layer, on the CPU."""
    def pair(rows, cols):
        return (torch.zeros(E + 1, rows, cols // 2, dtype=torch.uint8),
                torch.zeros(E + 1, rows, cols // 32, dtype=torch.uint8))

    def dense(rows, cols):
        return torch.zeros(E + 1, rows, cols, dtype=torch.bfloat16)

    make = pair if mx else dense
    return dict(w_router=torch.zeros(E, d, dtype=torch.bfloat16), router_bias=torch.zeros(E),
                w_gate=make(f, d), w_up=make(f, d), w_down=make(d, f))


@pytest.mark.parametrize("mx", [False, True])
def test_layer_refuses_weights_on_different_devices(mx):
    """The kernels run on one device: a tensor of another would be read through an address that means
    nothing there."""
    cls, good = binding.MoELayerMXFP4 if mx else binding.MoELayer, _layer_tensors(mx)
    for name, t in good.items():
        if name == "w_router":
            continue
        parts = range(len(t)) if isinstance(t, tuple) else [None]
        for i in parts:
            if i is None:
                bad = t.to("meta")
            else:
                bad = tuple(p.to("meta") if j == i else p for j, p in enumerate(t))
            with pytest.raises(ValueError, match="on meta"):
                cls(**dict(good, **{name: bad}), top_k=2, max_tokens=8)


@pytest.fixture
def devices(monkeypatch):
    """torch.cuda with device 0 and its stream 7 current; the contexts entered are recorded."""
    entered = []

    class Stream:
        def __init__(self, handle, index):
            self.cuda_stream, self.device = handle, torch.device("cuda", index)

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            entered.append(self.what)

        def __exit__(self, *exc):
            entered.append(None)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 7, raising=False)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: "caller's")
    return Stream, entered


class Tensor:
    is_cuda = True

    def __init__(self):
        self.on = []

    def record_stream(self, s):
        self.on.append(s)


def test_call_runs_on_its_tensors_device_and_stream(devices):
    Stream, entered = devices
    mine, other, far = Stream(7, 0), Stream(9, 0), Stream(9, 1)
    for stream in (None, mine):  # nothing to switch
        t = Tensor()
        with binding._on(0, stream, t) as on:
            assert on.new(t) is t
        assert entered == [] and t.on == []
    with binding._on(1, None):  # another device than the current one
        assert entered == [1]
    x, r = Tensor(), Tensor()
    with binding._on(0, other, x, None) as on:  # another stream
        assert entered[-1] is other and on.new(r) is r
    assert entered[-1] is None and x.on == [other] and r.on == ["caller's"]
    with binding._on(1, far, x):
        assert entered[-1] is far
    for dev, stream in ((1, other), (0, far)):
        with pytest.raises(ValueError, match="stream: of cuda"):
            binding._on(dev, stream)


def test_layer_calls_check_their_tensors_device(devices, monkeypatch):
    """A layer on device 1, the current device 0: calls run there, and refuse tensors of another."""
    _, entered = devices
    layer = object.__new__(binding.MoELayer)
    layer.handle = None
    layer.cfg = binding.moe_config(8, 256, 4, 2, 128, 1, binding.MOE_BF16, 1.0)

    class Fake:
        """A tensor's shape, type and device."""

        def __init__(self, shape, dtype, index):
            self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", index)

        def dim(self):
            return len(self.shape)

        def get_device(self):
            return self.device.index

    layer._start(Fake((4, 256), torch.bfloat16, 1))
    there, here = (Fake((3, 256), torch.bfloat16, i) for i in (1, 0))
    calls = []
    monkeypatch.setattr(binding, "moe_forward", lambda *a: calls.append(list(entered)))
    monkeypatch.setattr(binding, "moe_forward_few", lambda *a: calls.append(list(entered)))
    monkeypatch.setattr(binding.MoELayer, "_workspace", lambda self, n: None)
    for call in (layer.forward, layer.forward_few):
        for x, out in ((here, there), (there, here), (here, here)):
            with pytest.raises(ValueError, match="on cuda:0, the layer on cuda:1"):
                call(x, out=out)
        call(there, out=there)
    assert calls == [[1], [1, None, 1]]
    logits, idx = Fake((3, 4), torch.float32, 0), Fake((3, 2), torch.int32, 0)
    with pytest.raises(ValueError, match="on cuda:0"):
        layer.route(logits=logits)
    with pytest.raises(ValueError, match="on cuda:0"):
        layer.router_stats(logits, idx, 2)
    with pytest.raises(ValueError, match="on cuda:0"):
        layer.router_logits_static(here)
    with pytest.raises(ValueError, match="on cuda:0"):
        layer.forward_save(here)
    with pytest.raises(ValueError, match="on cuda:0"):
        layer.backward(there, here)


def test_conversion_calls_check_sizes_and_types():
    """The calls that take their results' tensors: one of another size would be written past its end."""
    w = torch.zeros(4, 128, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    q, d, t = (binding.moe_mxfp4_quantize, binding.moe_mxfp4_dequantize,
               binding.moe_mxfp4_tile_scales)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        q(w.half(), codes, scales)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        d(codes, scales, w.half())
    for c, s, name in ((codes[:3], scales, "codes"), (codes.int(), scales, "codes"),
                       (codes, scales[:3], "scales"), (codes, scales.int(), "scales"),
                       (codes.to("meta"), scales, "codes"), (codes, scales.to("meta"), "scales")):
        with pytest.raises(ValueError, match=name):
            q(w, c, s)
        with pytest.raises(ValueError, match=name):
            d(c, s, w)
    for tiled in (scales[:3], scales.int(), scales.to("meta")):
        with pytest.raises(ValueError, match="tiled"):
            t(scales, tiled)
    with pytest.raises(ValueError, match="scales"):
        t(scales.int(), scales)
    for call in (lambda: q(w, codes, scales), lambda: d(codes, scales, w),
                 lambda: t(scales, scales.clone())):  # consistent: the pointers are looked at next
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
