"""Which tile the 8-bit products take where the weights' bytes bound several of
them alike (no GPU needed)."""

import pytest

import rotation_activation_quantization_amd as R

FAKE = 0x100000  # never dereferenced


@pytest.mark.parametrize("t", [33, 48, 64])
@pytest.mark.parametrize("n", [2048, 4096, 8192, 14336])
def test_tokens_that_fill_half_a_tile_take_the_smaller_one(t, n):
    """28672 channels are 224 tiles of 128 channels either way; of 128 tokens half
    would be no tokens at all."""
    assert R.lib().signrot_int8_linear_kernel_name(FAKE, n, t, n, FAKE, n, 28672) == b"w8_tile_64x128"


@pytest.mark.parametrize("t", [33, 64])
def test_a_split_row_that_fills_the_device_goes_before_one_that_does_not(t):
    """8192 channels in two parts: 256 work-groups of 64 x 64, 128 of 64 x 128."""
    L = R.lib()
    assert L.signrot_int8_linear_kernel_name(FAKE, 28672, t, 28672, FAKE, 28672, 8192) == b"w8_tile_64x64"
    assert L.signrot_int4_w8_linear_kernel_name(FAKE, t, 28672, FAKE, 28672, 8192) == b"w8_tile_64x64_deep"
