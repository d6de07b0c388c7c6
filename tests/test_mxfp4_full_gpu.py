"""The MXFP4 layer at its own size (d 4096, 288 experts and a shared one, top-8, d_ff 1280) and as the
dense FFN (d_ff 11264), against the 64-bit form of a sample of tokens (tests/mxfp4_reference.py)."""
import pytest
import torch

from sparse_moe_layer_warp_b200 import MoELayerMXFP4
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
