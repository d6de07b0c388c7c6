"""The MXFP4 layer at its own size (d 4096, 288 experts and a shared one, top-8, d_ff 1280) and as the
dense FFN (d_ff 11264), against the 64-bit form of a sample of tokens (tests/mxfp4_reference.py)."""
import pytest
import torch

from sparse_moe_layer_warp_b200 import MoELayer, MoELayerMXFP4, mxfp4_dequantize
from tests import mxfp4_reference as ref

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

FULL = dict(d=4096, E=288, k=8, f=1280, shared=1)


class Full:
    """A layer with random codes and scales (values about N(0, 1 / fan-in)) and tokens whose selection
    no rounding decides."""

    def __init__(self, T, d, E, k, f, shared, skew=False, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.k, self.shared = E, k, shared
        G = E + shared

        def mx(rows, cols):
            codes = torch.randint(0, 256, (G, rows, cols // 2), generator=gen, device="cuda",
                                  dtype=torch.uint8)
            # e2m1 codes drawn evenly have a mean square of 8.6
            s = 127 + round(-0.5 * torch.log2(torch.tensor(8.6 * cols)).item())
            scales = torch.randint(s - 1, s + 2, (G, rows, cols // 32), generator=gen,
                                   device="cuda", dtype=torch.uint8)
            return codes, scales

        def rnd(n, std=1.0):
            return (torch.randn(n, d, generator=gen, device="cuda") * std).to(torch.bfloat16)

        self.w = [mx(f, d), mx(f, d), mx(d, f)]
        self.router = rnd(E, d ** -0.5)
        if skew:
            self.bias = -1.1 * torch.log(torch.randperm(E, generator=gen, device="cuda") + 1.0)
        else:
            self.bias = torch.rand(E, generator=gen, device="cuda") * 0.2 - 0.1
        self.x = rnd(T)
        while E > 1:
            s = self.x.double() @ self.router.double().T + self.bias.double()
            top = s.topk(min(E, k + 1), dim=1).values
            near = (top[:, :-1] - top[:, 1:]).amin(dim=1) < 1e-4
            if not near.any():
                break
            self.x[near] = rnd(int(near.sum()))
        self.layer = MoELayerMXFP4(self.router, self.bias, *self.w, top_k=k, max_tokens=T,
                                   n_shared=shared)


@pytest.mark.parametrize("priority", [0, -1])
def test_prefill_beside_another_call(cuda_ok, priority):
    """Two layers past 64 tokens on two streams, one of them of higher priority: their grids compete
    for the SMs, and either may get a part of them only."""
    a, b = Full(8192, **FULL, seed=1), Full(600, **FULL, seed=2)
    want_a, want_b = a.layer.forward(a.x).clone(), b.layer.forward(b.x).clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream(priority=priority)
    n = 4
    oa, ob = [torch.empty_like(a.x) for _ in range(n)], [torch.empty_like(b.x) for _ in range(4 * n)]
    torch.cuda.synchronize()
    for i in range(n):
        a.layer.forward(a.x, out=oa[i], stream=sa)
        for j in range(4):
            b.layer.forward(b.x, out=ob[4 * i + j], stream=sb)
    torch.cuda.synchronize()
    assert a.layer.device_status() == 0 and b.layer.device_status() == 0
    assert all(torch.equal(o, want_a) for o in oa) and all(torch.equal(o, want_b) for o in ob)


def _sample(idx, E):
    """Tokens that between them meet every expert that any token meets: the first and the last of each,
    and the batch's ends."""
    T = idx.shape[0]
    tok = torch.arange(T, device=idx.device).unsqueeze(1).expand_as(idx).reshape(-1)
    flat = idx.reshape(-1).long()
    first = torch.full((E,), T, device=idx.device).scatter_reduce_(0, flat, tok, "amin")
    last = torch.full((E,), -1, device=idx.device).scatter_reduce_(0, flat, tok, "amax")
    met = last >= 0
    ends = torch.tensor([0, T - 1], device=idx.device)
    return torch.unique(torch.cat((first[met], last[met], ends)))


def _check(c, out, layer, weights, mx):
    idx = layer.route(x=c.x)["idx"]
    rows = _sample(idx, c.E)
    assert set(idx[rows].flatten().tolist()) == set(idx.flatten().tolist())
    want, bound = ref.layer(c.x[rows], c.router, c.bias, *weights, c.k, c.shared, 1.0, mx)
    over = (out[rows].double() - want).abs() / bound
    assert not over.isnan().any() and over.max() <= 1, float(over.max())


CASES = [
    dict(T=1, **FULL), dict(T=16, **FULL), dict(T=64, **FULL),  # one launch
    dict(T=65, **FULL), dict(T=256, **FULL),                    # CTA pairs, 32 rows
    dict(T=256, **dict(FULL, shared=0)),
    dict(T=4096, skew=True, **FULL), dict(T=8192, **FULL),      # 112 rows
    dict(T=8192, **dict(FULL, shared=0)),
    dict(T=1000, d=4096, E=1, k=1, f=11264, shared=0),          # the dense FFN
    dict(T=20, d=4096, E=1, k=1, f=11264, shared=0),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_full_size(cuda_ok, kw):
    c = Full(**kw)
    out = c.layer.forward(c.x)
    weights = [(lambda g, p=p: ref.values(p[0][g], p[1][g])) for p in c.w]
    _check(c, out, c.layer, weights, True)
    assert torch.equal(out, c.layer.forward(c.x))
    assert c.layer.device_status() == 0


@pytest.mark.parametrize("kw", CASES[:3], ids=lambda kw: f"T{kw['T']}")
def test_one_launch_full_size_bf16(cuda_ok, kw):
    c = Full(**kw)
    w = [mxfp4_dequantize(*p) for p in c.w]
    layer = MoELayer(c.router, c.bias, *w, top_k=c.k, max_tokens=kw["T"], n_shared=c.shared)
    out = layer.forward_few(c.x)
    _check(c, out, layer, [(lambda g, p=p: p[g].double()) for p in w], False)
    assert torch.equal(out, layer.forward_few(c.x))
    assert layer.device_status() == 0


# CTA pairs with 32 rows a tile (at most 12 rows an expert on average), with no shared expert
SMALL = [dict(T=70, d=256, E=64, k=4, f=128, shared=0), dict(T=129, d=640, E=288, k=8, f=384, shared=0),
         dict(T=200, d=384, E=40, k=2, f=256, shared=0, skew=True)]


@pytest.mark.parametrize("kw", SMALL, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_small_token_tiles_without_a_shared_expert(cuda_ok, kw):
    c = Full(**kw)
    out = c.layer.forward(c.x)
    weights = [(lambda g, p=p: ref.values(p[0][g], p[1][g])) for p in c.w]
    want, bound = ref.layer(c.x, c.router, c.bias, *weights, c.k, c.shared, 1.0, True)
    over = (out.double() - want).abs() / bound
    assert not over.isnan().any() and over.max() <= 1, float(over.max())
    assert torch.equal(out, c.layer.forward(c.x)) and c.layer.device_status() == 0


def test_one_launch_beside_prefill(cuda_ok):
    """A cooperative launch of the whole device on one stream, prefill's persistent grids on another."""
    a, b = Full(8192, **FULL, seed=1), Full(16, **FULL, seed=2)
    want_a, want_b = a.layer.forward(a.x).clone(), b.layer.forward(b.x).clone()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    n = 4
    oa, ob = [torch.empty_like(a.x) for _ in range(n)], [torch.empty_like(b.x) for _ in range(8 * n)]
    torch.cuda.synchronize()
    for i in range(n):
        a.layer.forward(a.x, out=oa[i], stream=sa)
        for j in range(8):
            b.layer.forward(b.x, out=ob[8 * i + j], stream=sb)
    torch.cuda.synchronize()
    assert a.layer.device_status() == 0 and b.layer.device_status() == 0
    assert all(torch.equal(o, want_a) for o in oa) and all(torch.equal(o, want_b) for o in ob)
