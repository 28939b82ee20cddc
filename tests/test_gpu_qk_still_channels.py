"""Channels that are neither normed nor rotated come through bit for bit."""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: torch.int16, torch.float32: torch.int32}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(128, 0), (128, 64), (128, 32), (80, 36), (36, 18), (10, 6), (8, 4), (512, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_and_signs_of_zeros(d, rotary, dtype, interleaved):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((6, 5, d), generator=g, device="cuda").to(dtype)
    x[:, :, ::3], x[:, :, 1::3] = -0.0, 0.0
    x[1, 2, 2::3] = torch.finfo(dtype).smallest_normal / 4  # subnormal
    x[3, 1, 2::3] = torch.finfo(dtype).max
    angle = torch.rand((6, rotary // 2), generator=g, device="cuda") * 7
    tables = (angle.cos(), angle.sin()) if rotary else (None, None)
    for out in {dtype, torch.float32}:
        got, _ = R.qk_norm_rope(x, cos=tables[0], sin=tables[1], norm="none", interleaved=interleaved, dtype=out)
        assert torch.equal(got[:, :, rotary:].contiguous().view(BITS[out]),
                           x[:, :, rotary:].to(out).contiguous().view(BITS[out]))
