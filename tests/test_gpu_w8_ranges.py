"""Sizes at the ends of what the 8-bit products and the row kernels accept."""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,rows", [(1, 2 ** 30 - 1), (70, 2 ** 28 + 77)])
def test_more_tiles_than_one_launch_holds(t, rows):
    """2^24 tiles of 64 x 64 results, 256 threads each, are one more thread than a
    launch may have.  One channel, unit scales, a product below 2^8: exact in bf16."""
    codes = torch.randint(-11, 12, (t, 1), device="cuda").to(torch.int8)
    w = torch.randint(-11, 12, (rows, 1), dtype=torch.int8, device="cuda")
    print(f"[gpu] int8_linear {t} x 1 x {rows} [{R.int8_linear_kernel_name(codes, w)}]", flush=True)
    out = R.int8_linear(codes, torch.ones(t, device="cuda"), w, torch.ones(rows, device="cuda"))
    step = 1 << 26
    for at in range(0, rows, step):
        part = w[at:at + step, 0].to(torch.bfloat16)
        for token in {0, t // 2, t - 1}:
            assert torch.equal(out[token, at:at + step], part * codes[token, 0]), (token, at)
    last = w[-5:, 0].to(torch.bfloat16)
    assert torch.equal(out[:, -5:], codes.to(torch.bfloat16) * last)
