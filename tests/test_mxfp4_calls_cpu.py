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
