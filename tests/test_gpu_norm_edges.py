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


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 9, 1003, 1024, 4099, 32768, 32776])
def test_in_place_equals_out_of_place(n, stream):
    """h_out is h, in rows whose last chunk is moved back over the one before, in
    kernels that read a row again, and without a reduction (so no barrier) before the
    first store: bit for bit what a separate output gets."""
    t = 37
    g = torch.Generator(device="cuda").manual_seed(n)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    y = normal(t, n).to(torch.bfloat16)
    gate, weight = normal(n).to(torch.bfloat16), normal(n).to(torch.bfloat16)
    for ld, off in ((n, 0), (n + 3, 1), ((n + 7) // 8 * 8 + 8, 8)):
        buf = torch.full((off + t * ld,), 9.0, dtype=stream, device="cuda")
        h = buf[off:].view(t, ld)[:, :n]
        start = normal(t, n).to(stream)
        for branch, post in ((None, "none"), (y, "none"), (y, "rms"), (y, "layer")):
            kw = {"post_norm": post, "weight": weight, "beta": 0.75, "alpha": 1.25}
            if branch is not None:
                kw["gate"] = gate
            for call in (R.residual_norm, R.residual_norm_quant_int8):
                h.copy_(start)
                want = call(h, branch, **kw)
                assert torch.equal(h, start)
                got = call(h, branch, h_out=h, **kw)
                print(f"[gpu] in place {n} {stream} {ld} {post} {call.__name__}", flush=True)
                assert got[0] is h and all(torch.equal(a, b) for a, b in zip(got, want))
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[off:].view(t, ld)[:, :n] = False
        assert (buf[keep] == 9).all()


@pytest.mark.parametrize("n", [5, 9, 1024])
def test_more_rows_than_work_groups(n):
    """A launch has 2^20 work-groups at most; the rows beyond are second ones of some,
    whose reductions go through the same words."""
    t = 2 ** 20 + 3
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((t, n), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((t, n), generator=g, device="cuda").to(torch.bfloat16)
    weight = torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)
    # 700 rows: with up to 512 a thread takes one chunk, whose sums are added in another order
    parts = (slice(0, 700), slice(2 ** 19, 2 ** 19 + 700), slice(t - 700, t))
    print(f"[gpu] {t} rows of {n}", flush=True)
    codes, scale, sums = R.quant_int8(x, sums=True)
    top = x.float().abs().amax(dim=1)
    quotient = top.cpu().numpy() / np.float32(127)  # rounded once; torch multiplies by 1 / 127 on the GPU
    assert np.array_equal(scale.cpu().numpy(), np.where(quotient > 0, quotient, np.float32(1)))
    assert torch.equal(sums, codes.sum(dim=1, dtype=torch.int32))
    assert torch.equal(codes.abs().amax(dim=1), (top > 0).to(torch.int8) * 127)
    for norm in ("rms", "layer"):
        h, u = R.residual_norm(x, y, norm=norm, weight=weight)
        h8, codes8, scale8 = R.residual_norm_quant_int8(x, y, norm=norm, weight=weight)
        assert torch.equal(h, h8)
        for p in parts:
            alone = R.residual_norm(x[p], y[p], norm=norm, weight=weight)
            assert torch.equal(h[p], alone[0]) and torch.equal(u[p], alone[1])
            alone = R.residual_norm_quant_int8(x[p], y[p], norm=norm, weight=weight)
            assert torch.equal(codes8[p], alone[1]) and torch.equal(scale8[p], alone[2])
    for p in parts:
        alone = R.quant_int8(x[p], sums=True)
        assert torch.equal(codes[p], alone[0]) and torch.equal(sums[p], alone[2])


@pytest.mark.parametrize("t,index", [(1, False), (1, True), (6, True)])
@pytest.mark.parametrize("n", [100, 4096])
def test_one_modulation_row_of_any_stride_is_the_shared_one(t, index, n):
    """[1, n] rows, contiguous or cut from a wider projection, give what [n] vectors do."""
    wide = torch.randn((1, 6 * n), device="cuda").to(torch.bfloat16)
    h, y = (torch.randn((t, n), device="cuda").to(torch.bfloat16) for _ in range(2))
    gate, scale, shift = wide[:, :n], wide[:, n:2 * n].clone(), wide[:, 2 * n:3 * n]
    where = torch.zeros(t, dtype=torch.int32, device="cuda") if index else None
    got = R.residual_norm(h, y, gate=gate, mod_scale=scale, mod_shift=shift, mod_index=where)
    want = R.residual_norm(h, y, gate=gate[0], mod_scale=scale[0], mod_shift=shift[0])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
