"""The MXFP4 layer selects as moe_route does, in scores that only the order of a sum tells apart."""
import pytest
import torch

from sparse_moe_layer_warp_b200 import moe_forward_launch_count
from tests import mxfp4_reference as ref
from tests.test_mxfp4_gpu import Case, _check

pytestmark = pytest.mark.gpu


def _close_scores(c):
    """Router rows that differ in 32 tiny weights each: every token's scores agree but for the last bits
    of fp32."""
    gen = torch.Generator().manual_seed(5)
    row = torch.randn(c.d, generator=gen) * c.d ** -0.5
    rows = row.repeat(c.E, 1)
    rows[:, :32] = torch.randn(c.E, 32, generator=gen) * 2.0 ** -25
    c.router = rows.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("kw,launches", [
    (dict(T=60, d=256, E=64, k=12, f=128), 4),   # more than 512 pairs: routing in one launch
    (dict(T=64, d=256, E=288, k=9, f=128), 4),
    (dict(T=20, d=512, E=40, k=32, f=128), 4),
    (dict(T=60, d=256, E=320, k=12, f=128), 5),  # more experts than that routing takes
    (dict(T=40, d=256, E=64, k=12, f=128), 1),   # the one-launch layer
    (dict(T=70, d=256, E=64, k=12, f=128), 6),
], ids=lambda v: "-".join(f"{k}{x}" for k, x in v.items()) if isinstance(v, dict) else str(v))
def test_selects_as_the_routing_call(cuda_ok, kw, launches):
    c = Case(**kw, bias=False)
    _close_scores(c)
    layer = c.layer(True)
    out = layer.forward(c.x)
    r = layer.route(x=c.x, want_logits=True)
    idx = r["idx"].long()
    if kw["T"] <= 64 and kw["E"] <= 288:
        # another order of the sum selects other experts for some tokens: the case can tell
        by_static = layer.route(logits=layer.router_logits_static(c.x))["idx"].long()
        assert not torch.equal(by_static.sort(dim=1).values, idx.sort(dim=1).values)
    chosen = torch.zeros(c.x.shape[0], c.E, device="cuda").scatter_(1, idx, 1000.0)
    w = [(lambda g, p=p: ref.values(p[0][g], p[1][g])) for p in c.mx]
    _check(out, ref.layer(c.x, c.router, chosen, *w, c.k, c.shared, c.scale, True))
    assert moe_forward_launch_count(layer.handle, c.x.shape[0]) == launches
    assert layer.device_status() == 0
