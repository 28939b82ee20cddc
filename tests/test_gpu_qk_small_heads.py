"""The per-head norms where a head's squares leave binary32's normal range: heads of small values and an eps that
does not hide what their squares lose, against the float64 definition."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import mx_oracle as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24

# (head, rotary): partners in a lane 1 to 32 away, through LDS in chunks and one by one, rows of no whole vectors
FORMS = [(128, 128), (16, 16), (512, 512), (128, 64), (80, 36), (8, 6), (36, 18), (64, 0)]


def host(x):
    return None if x is None else x.double().cpu().numpy()


def make(t, heads, d, rotary, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((t, heads, d), generator=g, device="cuda", dtype=torch.float64)
    angle = torch.rand((t, rotary // 2), generator=g, device="cuda", dtype=torch.float64) * 7
    w = (torch.randn(d, generator=g, device="cuda") + 1).to(BF16)
    b = torch.randn(d, generator=g, device="cuda").to(BF16)
    return x, angle.cos().float(), angle.sin().float(), w, b


def check(got, x, cos, sin, norm, eps, w, b, interleaved):
    """Binary32 roundings: 48 u of both channels of a pair and, for LAYER, of |w| r max|x| (v = x r w + b, r from a
    sum of at most 512 squares, a mean that is off by 16 half-steps of the largest magnitude's sum, three operations
    of the rotation), and the result's own.  Scaling by a power of two adds none."""
    xs, rotary = host(x), 2 * cos.shape[1]
    eps = float(np.float32(eps))
    ref, v = M.qk_norm_rope(xs, host(cos), host(sin), np.arange(len(xs)), norm, eps, host(w), host(b), interleaved)
    size = np.abs(v) + (0 if b is None else np.abs(host(b)))
    if norm == "layer":
        c = xs - xs.mean(axis=2, keepdims=True)
        r = 1 / np.sqrt((c * c).mean(axis=2, keepdims=True) + eps)
        size = size + r * np.abs(xs).max(axis=2, keepdims=True) * np.abs(host(w))
    other, h = size.copy(), rotary // 2
    if interleaved:
        other[:, :, 0:rotary:2], other[:, :, 1:rotary:2] = size[:, :, 1:rotary:2], size[:, :, 0:rotary:2]
    else:
        other[:, :, :h], other[:, :, h:rotary] = size[:, :, h:rotary], size[:, :, :h]
    off = np.abs(host(got) - ref) - 48 * U * (size + other) - U * np.abs(ref)
    assert not np.isnan(off).any()
    worst = np.unravel_index(np.argmax(off), off.shape)
    assert off[worst] <= 0, f"over by {off[worst]} at {worst}: {host(got)[worst]} for {ref[worst]}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rotary", FORMS)
def test_small_heads(d, rotary, dtype, interleaved):
    """Head h of a token has values around 10^-h, down to subnormal ones, beside each other in a wave."""
    x, cos, sin, w, b = make(7, 39, d, rotary, 1)
    x *= 10.0 ** -torch.arange(39, device="cuda", dtype=torch.float64)[:, None]
    # whole steps of the least subnormal number, so that subnormal values are as exact as others in either type
    x = x.float().to(dtype)
    for norm in ("rms", "layer"):
        bias = b if norm == "layer" else None
        got, _ = R.qk_norm_rope(x, cos=cos, sin=sin, norm=norm, eps=0.0, q_weight=w, q_bias=bias,
                                interleaved=interleaved, dtype=F32)
        check(got, x, cos, sin, norm, 0.0, w, bias, interleaved)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("eps", [1e-45, 1e-38, 3e-31, 1e-30, 1e-12])
def test_small_eps(eps, norm):
    """An eps below and above the squares, which are far apart from head to head."""
    x, cos, sin, w, b = make(5, 31, 128, 128, 2)
    x = (x * 10.0 ** -torch.arange(31, device="cuda", dtype=torch.float64)[:, None]).float()
    bias = b if norm == "layer" else None
    got, _ = R.qk_norm_rope(x, cos=cos, sin=sin, norm=norm, eps=eps, q_weight=w, q_bias=bias)
    check(got, x, cos, sin, norm, eps, w, bias, False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zero_and_equal_heads_with_a_small_eps(dtype):
    """Zero heads give the bias; so do heads of equal values, whose deviation alone is small, whatever their size."""
    x = torch.zeros((2, 6, 64), device="cuda")
    x[:, 1], x[:, 2], x[:, 3], x[:, 4] = 1.0, -2.0 ** 60, 2.0 ** -30, 2.0 ** -120
    x = x.to(dtype)
    b = torch.randn(64, device="cuda")
    for eps in (1e-45, 1e-35, 1e-20):
        got, _ = R.qk_norm_rope(x, norm="layer", eps=eps, q_bias=b, dtype=F32)
        assert torch.equal(got, b.expand_as(got)), eps
        got, _ = R.qk_norm_rope(x[:, :1], norm="rms", eps=eps)
        assert not got.any()


def test_small_large_and_ordinary_heads_of_one_wave():
    x, cos, sin, w, _ = make(3, 8, 64, 64, 3)
    scale = torch.tensor([1e-25, 1.0, 1e30, 1e-38, 1e-10, 3e37, 1e-20, 1.0], device="cuda", dtype=torch.float64)
    x = (x * scale[:, None]).float()
    got, _ = R.qk_norm_rope(x, cos=cos, sin=sin, eps=0.0, q_weight=w)
    check(got, x, cos, sin, "rms", 0.0, w, None, False)
    # the others' results do not depend on a neighbour that is normed again
    alone = [R.qk_norm_rope(x[:, h:h + 1].contiguous(), cos=cos, sin=sin, eps=0.0, q_weight=w)[0] for h in range(8)]
    assert torch.equal(got, torch.cat(alone, dim=1))


def test_small_heads_in_place():
    x, cos, sin, w, _ = make(9, 5, 96, 48, 4)
    x = (x * 1e-24).float()
    ref, _ = R.qk_norm_rope(x, cos=cos, sin=sin, eps=0.0, q_weight=w)
    R.qk_norm_rope(x, cos=cos, sin=sin, eps=0.0, q_weight=w, q_out=x)
    assert torch.equal(x, ref) and torch.isfinite(x).all()


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_an_eps_that_takes_the_mean_square_past_the_range(norm):
    """Squares whose sum is finite, beside an eps near binary32's largest: their sum is not."""
    x = torch.tensor([6e18, -6e18] * 4, device="cuda").repeat(2, 3, 1)
    x[:, 1] *= 1e-3
    angle = torch.rand((2, 4), device="cuda", dtype=torch.float64) * 7
    cos, sin, w = angle.cos().float(), angle.sin().float(), torch.ones(8, device="cuda")
    got, _ = R.qk_norm_rope(x, cos=cos, sin=sin, norm=norm, eps=3.35e38, q_weight=w)
    check(got, x, cos, sin, norm, 3.35e38, w, None, False)
