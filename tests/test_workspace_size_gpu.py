"""A workspace sized for n tokens serves every smaller call: sizes do not fall as tokens grow, across
the changes of kernels and token tiles.  The handles get addresses that nothing reads."""
import ctypes

import pytest

from sparse_moe_layer_warp_b200 import binding

pytestmark = pytest.mark.gpu

CONFIGS = [
    dict(d=4096, E=288, k=8, f=1280, shared=1),
    dict(d=1024, E=100, k=8, f=1024, shared=1),
    dict(d=128, E=288, k=8, f=11264, shared=1),
    dict(d=4096, E=8, k=2, f=14336, shared=0),
    dict(d=256, E=64, k=32, f=128, shared=1),       # 512 pairs at 16 tokens
    dict(d=256, E=40, k=9, f=256, shared=0),
    dict(d=256, E=1024, k=32, f=128, shared=1),     # no one-launch layer
    dict(d=8320, E=16, k=4, f=128, shared=0),       # past the decode router's width
    dict(d=4096, E=1, k=1, f=11264, shared=0),
]
MOST = 1500


def _handle(kind, d, E, k, f, shared):
    lib = binding.load_library()
    dtype = binding.MOE_F32 if kind == "f32" else binding.MOE_BF16
    cfg, h = binding.moe_config(MOST, d, E, k, f, shared, dtype, 1.0), ctypes.c_void_p()
    if kind == "mxfp4":
        w = binding.moe_mxfp4_weights(1 << 20, None, *([1 << 20] * 6))
        s = lib.moe_layer_init_mxfp4(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h))
    else:
        w = binding.moe_weights(1 << 20, None, *([1 << 20] * 3))
        s = lib.moe_layer_init(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h))
    assert s == binding.MOE_OK
    return h


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f32"])
@pytest.mark.parametrize("kw", CONFIGS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_sizes_do_not_fall(cuda_ok, kind, kw):
    h = _handle(kind, **kw)
    calls = [binding.moe_workspace_size]
    if kind != "mxfp4":
        calls += [binding.moe_backward_workspace_size, binding.moe_saved_size]
    for size in calls:
        sizes = [size(h, T) for T in range(1, MOST + 1)]
        falls = [T + 2 for T, (a, b) in enumerate(zip(sizes, sizes[1:])) if b < a]
        assert sizes[0] > 0 and not falls, (size.__name__, falls[:10])
    binding.moe_layer_destroy(h)
