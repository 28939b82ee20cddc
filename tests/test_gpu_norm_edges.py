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


@pytest.mark.parametrize("size", [1e19, 3e25, 2e34, 3e38])
@pytest.mark.parametrize("n", [5, 64, 1003, 4096, 8192, 32776])
def test_squares_beyond_binary32(n, size):
    """Finite rows whose squares pass 2^128: RMS of the branch and of the stream.  The
    factor 1 / rms may be a subnormal number, down to 2^-128 in steps of 2^-149: 2^-22
    relative.  With the statistics' roundings (n / 64 + 16 additions at most in a row, as many
    of 2^-24) and the result's to bf16 (2^-8), or to float32."""
    g = np.random.default_rng([3, n])
    x = torch.from_numpy(g.uniform(0.3, 1.0, (3, n)) * g.choice([-1.0, 1.0], (3, n)) * size).to(torch.bfloat16)
    x[1] = torch.from_numpy(g.standard_normal(n)).to(torch.bfloat16)  # an ordinary row between
    want = x.double() / (x.double().pow(2).mean(dim=1, keepdim=True) + 1e-6).sqrt()
    close = 2.0 ** -22 + (n / 64 + 20) * 2.0 ** -24
    x = x.cuda()
    for stream in (torch.bfloat16, torch.float32):
        print(f"[gpu] {size} {n} {stream}", flush=True)
        h, u = R.residual_norm(x.to(stream))
        assert torch.equal(h, x.to(stream))
        assert ((u.double().cpu() - want).abs() <= (2.0 ** -8 + close) * want.abs()).all()
        h, _ = R.residual_norm(torch.zeros_like(x).to(stream), x)
        half = 2.0 ** -8 if stream == torch.bfloat16 else 2.0 ** -24
        assert ((h.double().cpu() - want).abs() <= (half + close) * want.abs()).all()
        _, codes, scale = R.residual_norm_quant_int8(x.to(stream))
        top = want.abs().amax(dim=1)
        assert ((scale.double().cpu() - top / 127).abs() <= 2 * close * top / 127).all()
        assert ((codes.double().cpu() - 127 * want / top[:, None]).abs() <= 0.5 + 127 * 3 * close).all()


@pytest.mark.parametrize("n", [6, 1000, 4096, 40000])
def test_squares_beyond_binary32_layer_norm(n):
    """The centred squares too.  The sum is far below 2^128; its error and the mean's
    are as for ordinary rows: (n / 64 + 16) roundings of the values' mean size."""
    g = np.random.default_rng([4, n])
    x = torch.from_numpy((g.standard_normal((2, n)) + 0.5) * 1e24).to(torch.bfloat16)
    d = x.double() - x.double().mean(dim=1, keepdim=True)
    sd = d.pow(2).mean(dim=1, keepdim=True).sqrt()
    want = d / sd
    depth = (n / 64 + 20) * 2.0 ** -24
    _, u = R.residual_norm(x.cuda(), norm="layer")
    assert ((u.double().cpu() - want).abs() <= (2.0 ** -8 + depth) * want.abs() + 2 * depth * x.double().abs().mean() / sd).all()


@pytest.mark.parametrize("n", [6, 1000, 4096, 40000])
def test_an_infinity_is_no_overflow(n):
    """A row that holds an infinity stays visible, its neighbours as they were."""
    x = torch.randn((3, n), device="cuda").to(torch.bfloat16)
    want = R.residual_norm_quant_int8(x, x)
    for where in ("h", "y"):
        h, y = x.clone(), x.clone()
        (h if where == "h" else y)[1, n // 2] = float("-inf")
        got = R.residual_norm_quant_int8(h, y)
        assert not torch.isfinite(got[2][1])
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
