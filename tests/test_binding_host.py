"""What the binding checks and hands to the library, with stand-ins for GPU
tensors (no GPU needed): operands on the wrong device are refused before any
call of the library."""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402


def test_operands_in_host_memory_are_refused_with_a_value_error():
    codes = torch.zeros((2, 32), dtype=torch.uint8)
    f = torch.ones(2)
    w = torch.zeros((8, 64), dtype=torch.int8)
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: R.dequant(codes, f, f), lambda: R.quant_int8(x),
                 lambda: R.int8_linear(codes.view(torch.int8), f, w[:, :32], torch.ones(8)),
                 lambda: R.int4_w8_linear(codes, f, f, w, torch.ones(8), torch.zeros(8, dtype=torch.int32)),
                 lambda: R.residual_norm(x), lambda: R.rotate_quant_int4_outlier(x, 0, 1)):
        with pytest.raises(ValueError):
            call()
