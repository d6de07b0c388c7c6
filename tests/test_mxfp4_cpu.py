"""MXFP4 operators and the one-launch layer: what the host refuses, and the 64-bit definitions that
the GPU tests compare with, checked against hand-computed blocks.  No GPU."""
import ctypes

import pytest
import torch

from sparse_moe_layer_warp_b200 import binding
from sparse_moe_layer_warp_b200.build import build
from tests import mxfp4_reference as ref

OK, INVALID, UNSUPPORTED, ALIGN = (binding.MOE_OK, binding.MOE_ERR_INVALID_ARG,
                                   binding.MOE_ERR_UNSUPPORTED, binding.MOE_ERR_ALIGNMENT)


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


def test_quantise_definition_on_known_blocks():
    w = torch.zeros(3, 32)
    w[0, :8] = torch.tensor([6.0, -6.0, 0.25, 0.75, 2.5, 5.0, -0.25, 0.2501])  # scale 1
    w[1, 0] = 7.99  # scale 1, saturates
    codes, scales = ref.quantize(w)
    assert scales[:, 0].tolist() == [127, 127, 0]
    low = [int(c) & 15 for c in codes[0, :4]]
    high = [int(c) >> 4 for c in codes[0, :4]]
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1.0 (code 2), 2.5 -> 2 (code 4), 5 -> 4 (code 6)
    assert low == [7, 0, 4, 8] and high == [15, 2, 6, 1]
    assert int(codes[1, 0]) & 15 == 7 and int(codes[2].sum()) == 0
    back = ref.values(codes, scales)
    assert back[0, :8].tolist() == [6, -6, 0, 1, 2, 4, 0, 0.5] and back[1, 0] == 6


def test_quantise_definition_of_non_finite_blocks():
    w = torch.ones(1, 64)
    w[0, 3] = float("inf")
    codes, scales = ref.quantize(w)
    assert scales.tolist() == [[255, 125]] and int(codes[0, :16].sum()) == 0
    back = ref.values(codes, scales)
    assert back[0, :32].isnan().all() and (back[0, 32:] == 1).all()


def test_quantise_refusals(lib):
    q, d = lib.moe_mxfp4_quantize, lib.moe_mxfp4_dequantize
    bf16 = binding.MOE_BF16
    assert q(None, bf16, 4, 64, 16, 16, None) == INVALID
    assert q(16, bf16, 4, 64, None, 16, None) == INVALID
    assert q(16, bf16, 4, 64, 16, None, None) == INVALID
    assert q(16, bf16, -1, 64, 16, 16, None) == INVALID
    assert q(16, bf16, 4, 48, 16, 16, None) == INVALID  # not whole blocks
    assert q(16, 7, 4, 64, 16, 16, None) == INVALID     # unknown dtype
    assert q(24, bf16, 4, 64, 16, 16, None) == ALIGN
    assert q(16, bf16, 4, 64, 24, 16, None) == ALIGN
    assert d(None, 16, 4, 64, 16, bf16, None) == INVALID
    assert d(16, None, 4, 64, 16, bf16, None) == INVALID
    assert d(16, 16, 4, 64, None, bf16, None) == INVALID
    assert d(16, 16, 4, -32, 16, bf16, None) == INVALID
    assert d(16, 16, 4, 64, 24, bf16, None) == ALIGN
    # nothing to do: no pointer is looked at
    assert q(None, bf16, 0, 64, None, None, None) == OK
    assert d(None, None, 4, 0, None, bf16, None) == OK


def test_tile_scales_refusals(lib):
    t = lib.moe_mxfp4_tile_scales
    assert t(None, 128, 128, 16, None) == INVALID
    assert t(16, 128, 128, None, None) == INVALID
    assert t(16, -128, 128, 16, None) == INVALID
    assert t(16, 64, 128, 16, None) == INVALID
    assert t(16, 128, 96, 16, None) == INVALID
    assert t(20, 128, 128, 16, None) == ALIGN
    assert t(16, 128, 128, 24, None) == ALIGN
    assert t(None, 0, 128, None, None) == OK and t(None, 128, 0, None, None) == OK


def test_layer_init_refusals(lib):
    init = lib.moe_layer_init_mxfp4
    h = ctypes.c_void_p()

    def cfg(T=16, d=4096, E=288, k=8, f=1280, shared=1, dtype=binding.MOE_BF16):
        return binding.moe_config(T, d, E, k, f, shared, dtype, 1.0)

    def weights(**kw):
        p = dict(w_router=16, router_bias=None, w_gate=32, w_up=64, w_down=96, scale_gate=16,
                 scale_up=32, scale_down=48)
        p.update(kw)
        return binding.moe_mxfp4_weights(*(p[n] for n in (
            "w_router", "router_bias", "w_gate", "w_up", "w_down", "scale_gate", "scale_up",
            "scale_down")))

    def call(c, w):
        return init(ctypes.byref(c), ctypes.byref(w), ctypes.byref(h))

    assert init(None, ctypes.byref(weights()), ctypes.byref(h)) == INVALID
    assert init(ctypes.byref(cfg()), None, ctypes.byref(h)) == INVALID
    assert init(ctypes.byref(cfg()), ctypes.byref(weights()), None) == INVALID
    assert call(cfg(dtype=binding.MOE_F32), weights()) == UNSUPPORTED
    assert call(cfg(f=1344), weights()) == UNSUPPORTED        # d_ff not a multiple of 128
    assert call(cfg(d=4160), weights()) == UNSUPPORTED
    assert call(cfg(T=2**26, f=131072), weights()) == UNSUPPORTED  # counts of pieces of h
    for name in ("w_router", "w_gate", "scale_gate", "scale_up", "scale_down"):
        assert call(cfg(), weights(**{name: None})) == INVALID, name
    for name in ("w_gate", "w_up", "w_down"):  # codes: 32 bytes
        assert call(cfg(), weights(**{name: 48})) == ALIGN, name
    assert call(cfg(), weights(scale_up=24)) == ALIGN


def test_forward_few_refuses_a_null_handle(lib):
    assert lib.moe_forward_few(None, None, 1, None, None, 0, None) == INVALID


def test_python_calls_check_their_tensors(lib):
    w = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        binding.mxfp4_quantize(w.half())
    with pytest.raises(ValueError, match="multiple of 32"):
        binding.mxfp4_quantize(w[:, :40].contiguous())
    with pytest.raises(ValueError, match="CUDA tensors"):
        binding.mxfp4_quantize(w)
    with pytest.raises(ValueError, match="contiguous"):
        binding.mxfp4_quantize(torch.zeros(64, 64, dtype=torch.bfloat16).t())
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        binding.mxfp4_dequantize(codes, scales, dtype=torch.float16)
    with pytest.raises(ValueError, match="scales"):
        binding.mxfp4_dequantize(codes, scales[:, :1])
    with pytest.raises(ValueError, match="codes"):
        binding.mxfp4_dequantize(codes.int(), scales)
    with pytest.raises(ValueError, match="CUDA tensors"):
        binding.mxfp4_dequantize(codes, scales)


def test_layer_class_checks_shapes(lib):
    E, d, f = 4, 256, 128

    def pair(rows, cols, G=E + 1):
        return (torch.zeros(G, rows, cols // 2, dtype=torch.uint8),
                torch.zeros(G, rows, cols // 32, dtype=torch.uint8))

    router = torch.zeros(E, d, dtype=torch.bfloat16)
    good = dict(w_gate=pair(f, d), w_up=pair(f, d), w_down=pair(d, f))
    for change in (dict(w_gate=pair(f, d, E)), dict(w_up=pair(f, 2 * d)),
                   dict(w_down=(pair(d, f)[0], pair(d, 2 * f)[1])),
                   dict(w_down=(pair(d, f)[0].int(), pair(d, f)[1]))):
        kw = dict(good, **change)
        with pytest.raises(ValueError):
            binding.MoELayerMXFP4(router, None, kw["w_gate"], kw["w_up"], kw["w_down"], top_k=2,
                                  max_tokens=8)
    with pytest.raises(ValueError):
        binding.MoELayerMXFP4(router.float(), None, *good.values(), top_k=2, max_tokens=8)
