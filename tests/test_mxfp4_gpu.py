"""MXFP4 quantisation, the layer over MXFP4 experts and the one-launch layer, against 64-bit forms
(tests/mxfp4_reference.py, which also derives the bounds)."""
import ctypes

import pytest
import torch

from sparse_moe_layer_warp_b200 import (MoEError, MoELayer, MoELayerMXFP4, binding,
                                        moe_forward_launch_count, mxfp4_dequantize,
                                        mxfp4_quantize)
from tests import mxfp4_reference as ref

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ quantisation
def _matrix(rows, cols, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(rows, cols, generator=gen, dtype=torch.float64)
    # blocks of every magnitude, far below and above 1
    w *= torch.exp2(torch.randint(-120, 120, (rows, cols // 32), generator=gen).double()
                    ).repeat_interleave(32, dim=1)
    return w.to(dtype)


def _check_quantise(w):
    codes, scales = mxfp4_quantize(w.cuda())
    want_c, want_s = ref.quantize(w)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want_c)
    for dt in (torch.float32, torch.bfloat16):
        got = mxfp4_dequantize(codes, scales, dtype=dt).cpu()
        want = ref.values(want_c, want_s).to(dt)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        # zeros keep their sign
        assert torch.equal(torch.signbit(got.nan_to_num()), torch.signbit(want.nan_to_num()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (7, 32), (129, 160), (1013, 1312),
                                       (33, 4096)])
def test_quantise_equals_the_definition(cuda_ok, rows, cols, dtype):
    _check_quantise(_matrix(rows, cols, dtype, rows * cols))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_at_borders(cuda_ok, dtype):
    """Ties, saturation, zeros of both signs, the type's smallest and largest values, and blocks that
    hold an infinity or a NaN."""
    edges = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0]
    row = torch.tensor(edges + [-e for e in edges], dtype=torch.float64)
    rows = [row * 2.0 ** s for s in (-126, -20, 0, 20, 124)]
    fin = torch.finfo(dtype)
    for special in (fin.max, fin.tiny, 2.0 ** -133, float("inf"), float("-inf"), float("nan")):
        r = torch.zeros(32, dtype=torch.float64)
        r[5], r[6] = special, -0.0
        r[7] = 1.0 if special != special or abs(special) > 1 else special / 2
        rows.append(r)
    rows.append(torch.zeros(32, dtype=torch.float64))
    rows.append(-torch.zeros(32, dtype=torch.float64))
    _check_quantise(torch.stack(rows).to(dtype))


def test_quantise_all_bf16_values(cuda_ok):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    w = bits.view(torch.bfloat16).reshape(-1, 32)       # neighbours share an exponent mostly
    _check_quantise(w)
    _check_quantise(w.t().reshape(-1, 32).contiguous())  # and blocks that do not


def test_dequantise_every_code_and_scale(cuda_ok):
    codes = torch.arange(256, dtype=torch.uint8).repeat(16, 1)        # [16, 512 values]
    scales = torch.arange(256, dtype=torch.uint8).reshape(16, 16)
    for dt in (torch.float32, torch.bfloat16):
        got = mxfp4_dequantize(codes.cuda(), scales.cuda(), dtype=dt).cpu()
        want = ref.values(codes, scales).to(dt)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())


def test_quantise_empty_and_leading_dimensions(cuda_ok):
    for shape in ((0, 64), (3, 0), (0, 0)):
        c, s = mxfp4_quantize(torch.empty(shape, device="cuda"))
        assert c.shape == (shape[0], shape[1] // 2) and s.shape == (shape[0], shape[1] // 32)
        assert mxfp4_dequantize(c, s).shape == shape
    w = _matrix(30, 64, torch.bfloat16, 3)
    flat = mxfp4_quantize(w.cuda())
    cube = mxfp4_quantize(w.reshape(2, 3, 5, 64).cuda())
    assert torch.equal(flat[0], cube[0].reshape(30, 32)) and torch.equal(flat[1],
                                                                        cube[1].reshape(30, 2))


def test_quantise_on_another_stream(cuda_ok):
    w = _matrix(257, 512, torch.bfloat16, 9).cuda()
    want = mxfp4_quantize(w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mxfp4_quantize(w, stream=s)
    back = mxfp4_dequantize(*got, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(back, mxfp4_dequantize(*want))


@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 384), (640, 1280)])
def test_tile_scales(cuda_ok, rows, cols):
    gen = torch.Generator().manual_seed(rows)
    s = torch.randint(0, 256, (rows, cols // 32), generator=gen, dtype=torch.uint8)
    out = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    binding.moe_mxfp4_tile_scales(s.cuda(), out)
    assert torch.equal(out.cpu(), ref.tile_scales(s))


# ------------------------------------------------------------------------------ layers
class Case:
    """Inputs of a layer whose selection no rounding decides, with MXFP4 and bf16 weights."""

    def __init__(self, T, d, E, k, f, shared=1, skew=False, scale=1.0, bias=True, seed=0):
        gen = torch.Generator().manual_seed(1000 * T + d + E + seed)

        def rnd(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).cuda()

        G = E + shared
        self.k, self.shared, self.scale, self.E, self.d = k, shared, scale, E, d
        self.router = rnd(E, d, std=d ** -0.5)
        if skew:  # most tokens to a few experts: empty groups beside crowded ones
            b = -1.3 * torch.log(torch.randperm(E, generator=gen).float() + 1)
        else:
            b = torch.rand(E, generator=gen) * 0.2 - 0.1
        self.bias = b.cuda() if bias else None
        self.x = self.draw(rnd, T)
        self.bf16 = [rnd(G, f, d, std=d ** -0.5), rnd(G, f, d, std=d ** -0.5),
                     rnd(G, d, f, std=f ** -0.5)]
        self.mx = [mxfp4_quantize(w) for w in self.bf16]

    def draw(self, rnd, T):
        x = rnd(T, self.d)
        for _ in range(200):
            s = x.double() @ self.router.double().T + (0 if self.bias is None
                                                       else self.bias.double())
            top = s.topk(min(self.E, self.k + 1), dim=1).values
            if self.E == 1 or not (near := (top[:, :-1] - top[:, 1:]).amin(dim=1) < 1e-4).any():
                return x
            x[near] = rnd(int(near.sum()), self.d)
        raise AssertionError("ties remain")

    def layer(self, mx, max_tokens=None):
        cls, w = (MoELayerMXFP4, self.mx) if mx else (MoELayer, self.bf16)
        return cls(self.router, self.bias, *w, top_k=self.k,
                   max_tokens=max_tokens or self.x.shape[0], n_shared=self.shared,
                   routed_scale=self.scale)

    def exact(self, mx, x=None):
        w = [(lambda g, p=p: ref.values(p[0][g], p[1][g])) for p in self.mx] if mx else \
            [(lambda g, p=p: p[g].double()) for p in self.bf16]
        return ref.layer(self.x if x is None else x, self.router, self.bias, *w, self.k,
                         self.shared, self.scale, mx)


def _check(out, exact):
    want, bound = exact
    over = (out.double() - want).abs() / bound
    assert not over.isnan().any() and over.max() <= 1, float(over.max())


FEW = [
    dict(T=1, d=256, E=64, k=8, f=128),
    dict(T=1, d=4096, E=16, k=8, f=1280),
    dict(T=2, d=128, E=1, k=1, f=128, shared=0),          # one expert, the smallest sizes
    dict(T=5, d=384, E=40, k=6, f=384, scale=2.5),        # odd numbers of tiles
    dict(T=8, d=640, E=288, k=8, f=256),
    dict(T=9, d=640, E=17, k=3, f=384, shared=0),
    dict(T=16, d=1024, E=64, k=8, f=640, bias=False),
    dict(T=17, d=128, E=16, k=4, f=1152),
    dict(T=33, d=896, E=5, k=5, f=256),                   # every expert, several token tiles
    dict(T=64, d=512, E=288, k=8, f=128, skew=True),
    dict(T=64, d=256, E=8, k=8, f=128),
    dict(T=16, d=256, E=64, k=32, f=128),                 # the most pairs
    dict(T=3, d=8192, E=4, k=2, f=128),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw", FEW, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_few_tokens(cuda_ok, kw, mx):
    c = Case(**kw)
    layer = c.layer(mx)
    out = layer.forward_few(c.x)
    _check(out, c.exact(mx))
    assert layer.device_status() == 0
    assert torch.equal(out, layer.forward_few(c.x))  # deterministic
    if mx:
        assert torch.equal(out, layer.forward(c.x))  # the same call


LAYER = [
    dict(T=65, d=256, E=16, k=2, f=128),
    dict(T=77, d=384, E=40, k=6, f=384),
    dict(T=129, d=640, E=64, k=8, f=256, skew=True),       # empty and crowded experts
    dict(T=300, d=512, E=8, k=4, f=640, scale=0.5),
    dict(T=257, d=128, E=1, k=1, f=128, shared=0),         # one tile, the peer without rows
    dict(T=1000, d=384, E=4, k=2, f=1152, skew=True),
    dict(T=113, d=896, E=2, k=1, f=384, bias=False),
    dict(T=2048, d=256, E=16, k=8, f=256, skew=True),
    dict(T=70, d=256, E=600, k=8, f=128),                  # more experts than the decode router takes
    dict(T=50, d=256, E=1024, k=32, f=128),                # the routing's limits
]


@pytest.mark.parametrize("kw", LAYER, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_mxfp4_layer(cuda_ok, kw):
    c = Case(**kw)
    layer = c.layer(True)
    out = layer.forward(c.x)
    _check(out, c.exact(True))
    assert layer.device_status() == 0
    assert torch.equal(out, layer.forward(c.x))


def test_mxfp4_layer_writes_its_output_rows_only(cuda_ok):
    c = Case(T=300, d=512, E=8, k=4, f=256)
    layer = c.layer(True)
    for T in (1, 17, 64, 65, 130, 300):
        buf = torch.full((T + 2, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        x = c.x[:T].contiguous()
        layer.forward(x, out=buf[1:T + 1])
        assert (buf[0] == 7).all() and (buf[T + 1] == 7).all()
        _check(buf[1:T + 1], c.exact(True, x))


def test_sizes_in_any_order_on_one_layer(cuda_ok):
    """The workspace's counters and the grid barrier are left as the next call needs them."""
    c = Case(T=700, d=256, E=16, k=4, f=384)
    layer = c.layer(True)
    want = {T: layer.forward(c.x[:T].contiguous()).clone() for T in (700, 1, 64, 65, 16, 200)}
    for T in (16, 700, 1, 200, 64, 65, 700, 16, 1):
        assert torch.equal(layer.forward(c.x[:T].contiguous()), want[T]), T
    assert layer.forward(c.x[:0].contiguous()).shape == (0, 256)
    assert layer.device_status() == 0


@pytest.mark.parametrize("mx,T", [(False, 4), (True, 1), (True, 16), (True, 100), (True, 600)])
def test_captured_in_a_graph(cuda_ok, mx, T):
    c = Case(T=T, d=512, E=16, k=4, f=256)
    layer = c.layer(mx)
    call = layer.forward_few if T <= 64 else layer.forward
    x, out = c.x.clone(), torch.empty_like(c.x)
    eager = call(x).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(x, out=out)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    x2 = Case(T=T, d=512, E=16, k=4, f=256, seed=1).x
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call(x2))
    assert layer.device_status() == 0


@pytest.mark.parametrize("T1,T2", [(1, 16), (16, 300), (300, 300), (100, 64)])
def test_two_calls_at_once(cuda_ok, T1, T2):
    """Two layers with workspaces of their own on two streams."""
    a, b = Case(T=T1, d=512, E=16, k=4, f=256), Case(T=T2, d=512, E=16, k=4, f=384, seed=4)
    la, lb = a.layer(True), b.layer(True)
    want_a, want_b = la.forward(a.x).clone(), lb.forward(b.x).clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [torch.empty_like(a.x) for _ in range(20)], [torch.empty_like(b.x) for _ in range(20)]
    for i in range(20):
        la.forward(a.x, out=oa[i], stream=sa)
        lb.forward(b.x, out=ob[i], stream=sb)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want_a) for o in oa) and all(torch.equal(o, want_b) for o in ob)
    assert la.device_status() == 0 and lb.device_status() == 0


@pytest.mark.parametrize("T", [1, 40, 200])
def test_first_call_on_another_stream(cuda_ok, T):
    """The layer's tables and its workspace are ready for whichever stream calls first."""
    c = Case(T=T, d=1024, E=64, k=4, f=512)
    want = c.layer(True).forward(c.x).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(c.x)
    torch.cuda.synchronize()
    for _ in range(5):
        c.layer(True).forward(c.x, out=out, stream=s)
        s.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [6, 90, 400])
def test_not_a_number_stays_with_its_tokens(cuda_ok, T):
    """A block of NaN in one expert, and an infinity in one token: the tokens that meet them become
    NaN, the others keep their bits."""
    c = Case(T=T, d=256, E=8, k=2, f=128, shared=0)
    layer = c.layer(True)
    want = layer.forward(c.x).clone()
    idx = layer.route(x=c.x)["idx"]
    codes, scales = c.mx[0]
    bad = int(idx[0, 0])
    scales = scales.clone()
    codes = codes.clone()
    scales[bad, 3, 1] = 255
    codes[bad, 3, 16:32] = 0
    poisoned = MoELayerMXFP4(c.router, c.bias, (codes, scales), c.mx[1], c.mx[2], top_k=2,
                             max_tokens=T, n_shared=0)
    out = poisoned.forward(c.x)
    hit = (idx == bad).any(dim=1)
    assert hit.any() and not hit.all()
    assert out[hit].isnan().all() and torch.equal(out[~hit], want[~hit])
    x = c.x.clone()
    x[1, 5] = float("nan")
    # its own scores are NaN too, so its experts may change; every other token's result stays
    out = layer.forward(x)
    rest = torch.arange(T, device="cuda") != 1
    assert out[1].isnan().all() and torch.equal(out[rest], want[rest])
    assert layer.device_status() == 0


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("power", [-100, -8, 8, 60])
def test_activations_of_any_scale(cuda_ok, T, power):
    """x times a power of two: tiny values keep their precision (one scale for 32 neighbours), in the
    projections before the nonlinearity.  Weights shrink the other way, so that h stays in range."""
    c = Case(T=T, d=256, E=4, k=2, f=128, bias=False)
    c.x = (c.x.double() * 2.0 ** power).to(torch.bfloat16)
    c.router = (c.router.double() * 2.0 ** -power).to(torch.bfloat16)
    for i in (0, 1):
        codes, scales = c.mx[i]
        c.mx[i] = (codes, (scales.int() - power).clamp(1, 253).to(torch.uint8))
    layer = c.layer(True)
    _check(layer.forward(c.x), c.exact(True))


def test_outliers_in_a_block(cuda_ok):
    """One large activation in a block of 32: its neighbours are held to 2^-21 of it."""
    c = Case(T=70, d=256, E=4, k=2, f=128)
    c.router[:, 7] = 0
    c.x[::3, 7] *= 300
    layer = c.layer(True)
    _check(layer.forward(c.x), c.exact(True))


def test_served_together(cuda_ok):
    """A bf16 layer converted for serving: a prefill through the layer, then decode steps through the
    one-launch layer, each against the same 64-bit form."""
    c = Case(T=200, d=512, E=32, k=4, f=256)
    trained = c.layer(False)
    served = trained.to_mxfp4()
    exact = c.exact(True)
    _check(served.forward(c.x), exact)
    for lo, n in ((0, 1), (5, 1), (40, 4), (100, 16), (136, 64)):
        part = served.forward_few(c.x[lo:lo + n].contiguous())
        _check(part, (exact[0][lo:lo + n], exact[1][lo:lo + n]))
    # codes of the converted weights are the quantiser's
    for mine, theirs in zip(served.tensors[2:], c.mx):
        assert torch.equal(mine[0], theirs[0])
    assert served.device_status() == 0
    with pytest.raises(ValueError):
        served.to_mxfp4()


def test_few_selects_as_the_layer_does(cuda_ok):
    """Equal scores: both paths take the lower expert."""
    c = Case(T=4, d=256, E=16, k=2, f=128)
    c.router[5] = c.router[11] = c.router[2]
    c.bias[:] = -5.0
    c.bias[[2, 5, 11]] = 5.0
    layer = c.layer(False, max_tokens=4)
    idx = layer.route(x=c.x)["idx"].sort(dim=1).values
    assert (idx == torch.tensor([2, 5], device="cuda", dtype=torch.int32)).all()
    few, full = layer.forward_few(c.x), layer.forward(c.x)
    _, bound = c.exact(False)
    assert ((few.double() - full.double()).abs() <= 2 * bound).all()


# one launch; else router, top-k, scatter, split rows, experts, combine
@pytest.mark.parametrize("T,expected", [(1, 1), (64, 1), (65, 6), (300, 6)])
def test_launch_count(cuda_ok, T, expected):
    from cuda.bindings import runtime as rt

    c = Case(T=T, d=256, E=16, k=4, f=128)
    layer = c.layer(True)
    assert moe_forward_launch_count(layer.handle, T) == expected
    x, out = c.x, torch.empty_like(c.x)
    layer.forward(x, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        layer.forward(x, out=out)
    graph = rt.cudaGraph_t(init_value=g.raw_cuda_graph())
    _, _, n = rt.cudaGraphGetNodes(graph, 0)
    _, nodes, n = rt.cudaGraphGetNodes(graph, n)
    kinds = [rt.cudaGraphNodeGetType(node)[1] for node in nodes[:n]]
    assert kinds.count(rt.cudaGraphNodeType.cudaGraphNodeTypeKernel) == expected


def test_refusals(cuda_ok):
    c = Case(T=65, d=256, E=16, k=4, f=128)
    mx, bf = c.layer(True), c.layer(False)
    for layer in (mx, bf):
        with pytest.raises(MoEError):
            layer.forward_few(c.x)                      # more than 64 tokens
        with pytest.raises(ValueError):
            layer.forward_few(c.x[:4].float())
        with pytest.raises(ValueError):
            layer.forward_few(c.x[:4], out=torch.empty_like(c.x[:5]))
        with pytest.raises(ValueError):
            layer.forward_few(c.x[:8, :].t().contiguous().t())
        assert layer.forward_few(c.x[:0].contiguous()).shape == (0, 256)
    with pytest.raises(MoEError):
        mx.backward(c.x, c.x)                           # serving only
    # calls that read bf16 weights, with arguments that a bf16 handle takes
    f32 = torch.empty(65, 256, device="cuda")
    big = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    for call in (
        lambda: binding.moe_forward_partial(mx.handle, c.x, 65, None, None, 0, 16, 0, 65, f32, big),
        lambda: binding.moe_forward_save(mx.handle, c.x, 65, torch.empty_like(c.x),
                                         big.view(torch.float32), big),
        lambda: mx.expert_health(65),
    ):
        with pytest.raises(MoEError) as e:
            call()
        assert e.value.status == binding.MOE_ERR_UNSUPPORTED
    wide = Case(T=17, d=256, E=40, k=32, f=128)         # 544 pairs
    with pytest.raises(MoEError):
        wide.layer(False).forward_few(wide.x)
    single = MoELayer(c.router.float(), c.bias, *(w.float() for w in c.bf16), top_k=4,
                      max_tokens=4)
    with pytest.raises(MoEError):
        single.forward_few(c.x[:4].float())
    lib = binding.load_library()
    x, out = c.x[:4].contiguous(), torch.empty_like(c.x[:4])
    ws = mx.workspace(4)

    def few(h, px, n, po, pw, size):
        return lib.moe_forward_few(h, ctypes.c_void_p(px), n, ctypes.c_void_p(po),
                                   ctypes.c_void_p(pw), size, None)

    args = (x.data_ptr(), 4, out.data_ptr(), ws.data_ptr(), ws.numel())
    assert few(mx.handle, *args) == binding.MOE_OK
    assert few(mx.handle, args[0], -1, *args[2:]) == binding.MOE_ERR_INVALID_ARG
    assert few(mx.handle, args[0], 66, *args[2:]) == binding.MOE_ERR_INVALID_ARG
    assert few(mx.handle, 0, *args[1:]) == binding.MOE_ERR_INVALID_ARG
    assert few(mx.handle, args[0] + 2, *args[1:]) == binding.MOE_ERR_ALIGNMENT
    assert few(mx.handle, *args[:4], 1000) == binding.MOE_ERR_WORKSPACE
    assert few(mx.handle, *args[:3], args[3] + 16, args[4]) == binding.MOE_ERR_ALIGNMENT
    torch.cuda.synchronize()
    assert mx.device_status() == 0


def test_offsets_past_32_bits(cuda_ok):
    """A matrix of more than 2^31 values: the last rows come out as they do by themselves."""
    rows, cols = 131_080, 16_512  # 2.16e9 values, 4.3 GB
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    tail = _matrix(8, cols, torch.bfloat16, 1).cuda()
    w[-8:] = tail
    codes, scales = mxfp4_quantize(w)
    want = mxfp4_quantize(tail)
    assert torch.equal(codes[-8:], want[0]) and torch.equal(scales[-8:], want[1])
    back = mxfp4_dequantize(codes, scales)
    assert torch.equal(back[-8:], mxfp4_dequantize(*want)) and (back[:-8] == 0.5).all()
