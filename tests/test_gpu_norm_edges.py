"""Rows at which the residual norms could go wrong: equal values, values whose
squares leave binary32's range, streams updated in place, and more rows than a
launch has work-groups."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [5, 7, 72, 1000, 1111, 5120, 11008, 28672, 40000])
def test_layer_norm_of_equal_values_is_the_bias(n, stream):
    """The sum of n equal bf16 values is exact in binary32 (8 + 16 bits), its quotient
    by n the value itself: the centred row is zero, and the result the bias,
    whatever the weight."""
    values = torch.tensor([1.0, -3.0, 1000.0, 0.0078125, 255.0, -17.75, 3.140625], device="cuda")
    x = values[:, None].expand(len(values), n).to(torch.bfloat16).contiguous()
    g = torch.Generator(device="cuda").manual_seed(n)
    weight, bias = (torch.randn(n, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    print(f"[gpu] equal values, {n} {stream}", flush=True)
    h, u = R.residual_norm(x.to(stream), norm="layer", weight=weight, bias=bias)
    assert torch.equal(h, x.to(stream)) and torch.equal(u, bias.expand_as(u))
    # the same of the branch: the stream gets the bias
    h, _ = R.residual_norm(torch.zeros_like(x).to(stream), x, norm="layer", post_weight=weight, post_bias=bias)
    assert torch.equal(h, bias.expand_as(x).to(stream))
    _, codes, scale = R.residual_norm_quant_int8(x.to(stream), norm="layer", weight=weight)
    assert (codes == 0).all() and (scale == 1).all()
