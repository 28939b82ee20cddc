"""The INT8 quantizer and the products on 8-bit weights against float64.

Codes, scales and sums of the quantizer have to be equal: the codes are the
exact rint of a rational, the scale one rounded quotient.

A product's integer sum is exact in int32, so with u = 2^-24 the only
roundings are those of the epilogue: the sum widened to binary32 (u |acc|),
the zero-point's fused multiply-add (u |acc - shift|), two multiplications
(2u |product|) and the bias (u |out|); 1.01 covers the second-order terms:

    tol = 1.01 (|s v| u (|acc| + 3 |acc - shift|) + u |out|) + 2^-8 |out| for bf16

(2^-8: half a unit in the last of the 8 significant bits of a bf16 number).  With unit scales and sums below
2^24 every step is exact and the float32 results are compared bit for bit.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import block_oracle as B  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GUARD = 93


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def strided(a, ld, offset=0):
    """`a` as a view of a wider, `offset` elements shifted buffer on the GPU."""
    rows, n = a.shape
    flat = np.full(rows * ld + offset, GUARD).astype(a.dtype)
    view = torch.from_numpy(flat).cuda()[offset:].view(rows, ld)[:, :n]
    view.copy_(torch.from_numpy(a))
    return view


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def tolerance(out, acc, shift, s, v, dtype):
    sv = np.abs(np.outer(s, v))
    tol = 1.01 * (sv * U * (np.abs(acc) + 3 * np.abs(acc - shift)) + U * np.abs(out))
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * 1.01 * np.abs(out)
    return tol + 1e-37


def check_product(got, ref, s, v, dtype, label):
    out, acc, shift = ref
    assert got.dtype == dtype
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all(), label
    over = np.abs(g - out) / tolerance(out, acc, shift, s, v, dtype)
    print(f"[gpu] {label}: worst {over.max() if over.size else 0:.3f} of the tolerance", flush=True)
    assert not over.size or over.max() <= 1.0, label


# ---- quantizer ---------------------------------------------------------------

QUANT = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 64), (3, 255), (9, 1000), (2, 1111), (7, 2048), (3, 4096), (2, 5120),
         (2, 8192), (33, 14336), (2, 28672), (2, 32776), (1, 131071)]


@pytest.mark.parametrize("t,n", QUANT)
def test_quant_int8_equals_definition(t, n):
    g = np.random.default_rng([1, t, n])
    x = bf16(g.standard_normal((t, n)) * np.exp(3 * g.standard_normal((t, 1))))
    if n >= 7:
        x[:, n // 2] *= 30
        x[-1, : n // 3] = x[-1, n // 2] / 2  # exact ties at 63.5
    q, s, total = B.quant_int8(x.double().numpy())
    codes, scale, sums = R.quant_int8(x.cuda(), sums=True)
    print(f"[gpu] quant_int8 {t} x {n}", flush=True)
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(sums.cpu().numpy(), total)
    a = x.float().abs().amax(dim=1).numpy()
    assert np.array_equal(scale.cpu().numpy(), np.where(a > 0, a / np.float32(127), np.float32(1)))


@pytest.mark.parametrize("top", [127.0, 254.0, 1.0, 0.75])
def test_quant_int8_ties_and_every_bf16_magnitude(top):
    """Every bf16 number up to `top` in one row: among them, where the top's
    significand holds the factor 127, all the exact ties."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float()) & (bits.float().abs() <= top)][None, :]
    q, _, total = B.quant_int8(x.double().numpy())
    codes, _, sums = R.quant_int8(x.cuda(), sums=True)
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(sums.cpu().numpy(), total)


def test_quant_int8_zero_rows_strides_and_guards():
    g = np.random.default_rng(2)
    for n, ld, off, ldc, offc in [(1000, 1003, 1, 1001, 3), (4096, 4104, 8, 4112, 16), (130, 136, 0, 131, 0)]:
        x = bf16(g.standard_normal((4, n)))
        x[1] = 0.0
        x[2, :] = -0.0
        xs = torch.empty(off + 4 * ld, dtype=torch.bfloat16, device="cuda")[off:].view(4, ld)[:, :n]
        xs.copy_(x)
        buf = torch.full((offc + 4 * ldc,), GUARD, dtype=torch.int8, device="cuda")
        codes = buf[offc:].view(4, ldc)[:, :n]
        scale = torch.empty(4, device="cuda")
        R.quant_int8(xs, out=(codes, scale))
        q, _, _ = B.quant_int8(x.double().numpy())
        assert np.array_equal(codes.cpu().numpy(), q)
        assert scale[1].item() == 1.0 and scale[2].item() == 1.0
        assert (buf[:offc] == GUARD).all() and (buf[offc:].view(4, ldc)[:, n:] == GUARD).all()


def test_quant_int8_non_finite_rows_stay_visible_and_apart():
    x = bf16(np.random.default_rng(4).standard_normal((5, 700)))
    ref, rs = R.quant_int8(x.cuda())
    x[1, 3] = float("inf")
    x[3, 699] = float("nan")
    codes, scale = R.quant_int8(x.cuda())
    assert not torch.isfinite(scale[1]) and not torch.isfinite(scale[3])
    for r in (0, 2, 4):
        assert torch.equal(codes[r], ref[r]) and scale[r] == rs[r]


def test_quant_int8_subnormal_rows():
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    x[0, :3] = torch.tensor([1, 2, 3], dtype=torch.int16).view(torch.bfloat16)  # the smallest magnitudes
    q, _, _ = B.quant_int8(x.double().numpy())
    codes, scale = R.quant_int8(x.cuda())
    assert np.array_equal(codes.cpu().numpy(), q)
    assert scale.item() == np.float32(x.float().abs().max().item()) / np.float32(127)


# ---- products ----------------------------------------------------------------

# tokens, n, rows: single tokens, every edge of 16-, 64-, 128- and 256-wide tiles, ragged k
SHAPES = [(1, 1, 1), (1, 2, 5), (1, 64, 16), (1, 4096, 257), (1, 14336, 64), (2, 48, 33), (3, 1111, 17), (4, 1024, 512),
          (5, 8192, 96), (8, 100, 130), (15, 272, 48), (16, 4096, 1024), (16, 5120, 100), (17, 2048, 64), (31, 128, 16),
          (32, 1024, 300), (33, 192, 257), (48, 11008, 256), (63, 656, 65), (64, 2048, 512), (65, 1040, 192),
          (100, 777, 129), (128, 4096, 256), (129, 96, 385), (200, 5504, 512), (255, 64, 255), (256, 1024, 256),
          (257, 320, 260), (300, 4096, 600), (512, 512, 768), (700, 1111, 333), (1024, 2048, 1024), (1025, 256, 513),
          (2048, 1024, 2048), (2060, 160, 2304)]


def operands(t, n, rows, seed, a4):
    g = np.random.default_rng([7, t, n, rows, seed])
    w = g.integers(-128, 128, (rows, n)).astype(np.int8)
    if a4:
        n2 = n // 2
        codes = g.integers(0, 256, (t, n2)).astype(np.uint8)
    else:
        codes = g.integers(-128, 128, (t, n)).astype(np.int8)
    s = (g.random(t) * 2 + 0.01).astype(np.float32)
    z = (g.standard_normal(t) * 40).astype(np.float32)
    v = (g.random(rows) / np.sqrt(n)).astype(np.float32)
    b = (g.standard_normal(rows) * 50).astype(np.float32)
    return codes, s, z, w, v, b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,rows", SHAPES)
def test_int8_linear_parity(t, n, rows, dtype):
    codes, s, _, w, v, b = operands(t, n, rows, 0, False)
    ref = B.w8_linear(codes.astype(np.float64), s, None, w, v, b)
    dc, dw = dev(codes), dev(w)
    got = R.int8_linear(dc, dev(s), dw, dev(v), bias=dev(b), dtype=dtype)
    check_product(got, ref, s, v, dtype, f"int8_linear {t} x {n} x {rows} {dtype} [{R.int8_linear_kernel_name(dc, dw)}]")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,rows", [(t, n + n % 2, r) for t, n, r in SHAPES])
def test_int4_w8_linear_parity(t, n, rows, dtype):
    codes, s, z, w, v, b = operands(t, n, rows, 1, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, b)
    dc, dw = dev(codes), dev(w)
    got = R.int4_w8_linear(dc, dev(s), dev(z), dw, dev(v), dev(w.sum(axis=1, dtype=np.int32)), bias=dev(b),
                           dtype=dtype)
    check_product(got, ref, s, v, dtype,
                  f"int4_w8_linear {t} x {n} x {rows} {dtype} [{R.int4_w8_linear_kernel_name(dc, dw)}]")


@pytest.mark.parametrize("t,n,rows", [(1, 992, 40), (16, 1008, 72), (40, 1000, 66), (300, 896, 520), (513, 960, 300)])
def test_products_are_exact_whole_numbers(t, n, rows):
    """Unit scales, whole zero-points, sums below 2^24: bit for bit."""
    codes, _, _, w, _, _ = operands(t, n, rows, 2, False)
    one, unit = torch.ones(t, device="cuda"), torch.ones(rows, device="cuda")
    got = R.int8_linear(dev(codes), one, dev(w), unit, dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), codes.astype(np.float64) @ w.T.astype(np.float64))
    packed, _, _, w, _, _ = operands(t, n, rows, 3, True)
    z = np.random.default_rng(6).integers(-40, 40, t).astype(np.float32)
    total = w.sum(axis=1, dtype=np.int32)
    got = R.int4_w8_linear(dev(packed), one, dev(z), dev(w), unit, dev(total), dtype=torch.float32)
    ref = B.unpack_int4(packed) @ w.T.astype(np.float64) - np.outer(z.astype(np.float64), total)
    assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("t,n,rows", [(1, 131071, 3), (20, 131071, 20), (1, 131056, 16), (300, 131056, 40)])
def test_int8_linear_longest_sums_do_not_overflow(t, n, rows):
    """All codes -128: the sum 2^14 n is the largest there is, below 2^31."""
    codes = torch.full((t, n), -128, dtype=torch.int8, device="cuda")
    w = torch.full((rows, n), -128, dtype=torch.int8, device="cuda")
    got = R.int8_linear(codes, torch.ones(t, device="cuda"), w, torch.ones(rows, device="cuda"), dtype=torch.float32)
    assert (got == float(np.float32(16384 * n))).all()


@pytest.mark.parametrize("ld,off,ldw,offw,ldo,offo", [(520, 8, 513, 1, 203, 1), (528, 16, 528, 16, 208, 8),
                                                      (517, 3, 512, 0, 200, 0), (512, 0, 544, 0, 201, 3)])
@pytest.mark.parametrize("t", [1, 16, 70, 300])
def test_int8_linear_strides_offsets_and_guards(t, ld, off, ldw, offw, ldo, offo):
    n, rows = 512, 200
    codes, s, _, w, v, _ = operands(t, n, rows, 4, False)
    ref = B.w8_linear(codes.astype(np.float64), s, None, w, v, None)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((offo + t * ldo,), float(GUARD), dtype=dtype, device="cuda")
        out = buf[offo:].view(t, ldo)[:, :rows]
        got = R.int8_linear(strided(codes, ld, off), dev(s), strided(w, ldw, offw), dev(v), out=out)
        assert got is out
        check_product(out, ref, s, v, dtype, f"int8_linear strided {t} {ld} {ldw} {ldo}")
        assert (buf[:offo] == GUARD).all() and (buf[offo:].view(t, ldo)[:, rows:] == GUARD).all()


@pytest.mark.parametrize("t", [1, 16, 70, 300])
def test_int4_w8_linear_strides_offsets_and_guards(t):
    n, rows = 1024, 144
    codes, s, z, w, v, b = operands(t, n, rows, 5, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, b)
    shifted = torch.empty(t * n // 2 + 5, dtype=torch.uint8, device="cuda")[5:].view(t, n // 2)
    shifted.copy_(dev(codes))
    total = dev(w.sum(axis=1, dtype=np.int32))
    for c, dw in ((shifted, dev(w)), (dev(codes), strided(w, 1031, 3)), (dev(codes), strided(w, 1040, 16))):
        buf = torch.full((t, rows + 7), float(GUARD), device="cuda")
        R.int4_w8_linear(c, dev(s), dev(z), dw, dev(v), total, bias=dev(b), out=buf[:, :rows])
        check_product(buf[:, :rows], ref, s, v, torch.float32, f"int4_w8_linear strided {t}")
        assert (buf[:, rows:] == GUARD).all()


@pytest.mark.parametrize("t,n,rows", [(1030, 4099, 2050), (2100, 2047, 2304), (4100, 1023, 1100)])
def test_large_unaligned_rows_are_laid_out_anew(t, n, rows):
    """Both operands unaligned; codes in aligned rows that end inside a chunk, with
    other bytes after them, unaligned weights; packed INT4 codes."""
    codes, s, z, w, v, b = operands(t, n, rows, 6, False)
    ref = B.w8_linear(codes.astype(np.float64), s, None, w, v, b)
    dw = dev(w)
    for c in (dev(codes), strided(codes, (n + 15) // 16 * 16)):
        name = R.int8_linear_kernel_name(c, dw)
        assert name.startswith("w8_pack_tile"), name
        check_product(R.int8_linear(c, dev(s), dw, dev(v), bias=dev(b), dtype=torch.float32), ref, s, v,
                      torch.float32, f"int8_linear {t} x {n} x {rows} [{name}]")
    n4 = n + 1 + 2 * (n % 4 == 3)  # even, and no multiple of four bytes of codes
    codes, s, z, w, v, b = operands(t, n4, rows, 7, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, b)
    c, dw = dev(codes), dev(w)
    name = R.int4_w8_linear_kernel_name(c, dw)
    assert name.startswith("w8_pack_tile"), name
    got = R.int4_w8_linear(c, dev(s), dev(z), dw, dev(v), dev(w.sum(axis=1, dtype=np.int32)), bias=dev(b),
                           dtype=torch.float32)
    check_product(got, ref, s, v, torch.float32, f"int4_w8_linear {t} x {n4} x {rows} [{name}]")


@pytest.mark.parametrize("t,n,rows,kind", [
    (64, 14336, 512, "tile_64x64"), (70, 4096, 4096, "tile_64x64"), (512, 4096, 4096, "tile_64x128"),
    (1024, 4096, 2048, "tile_64x128"), (2048, 4096, 4096, "tile_128x128"), (4096, 2048, 4096, "tile_256x256"),
    (2048, 14336, 4096, "tile_256x256"), (64, 28672, 2048, "tile_64x64")])
def test_every_tile_and_split_against_the_definition(t, n, rows, kind):
    """Shapes at which the plan takes each of its tiles, some with the row split."""
    codes, s, _, w, v, _ = operands(t, n, rows, 8, False)
    ref = B.w8_linear(codes.astype(np.float64), s, None, w, v, None)
    c, dw = dev(codes), dev(w)
    name = R.int8_linear_kernel_name(c, dw)
    assert kind in name, name
    check_product(R.int8_linear(c, dev(s), dw, dev(v), dtype=torch.float32), ref, s, v, torch.float32,
                  f"int8_linear {t} x {n} x {rows} [{name}]")
    codes, s, z, w, v, _ = operands(t, n, rows, 9, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, None)
    c, dw = dev(codes), dev(w)
    got = R.int4_w8_linear(c, dev(s), dev(z), dw, dev(v), dev(w.sum(axis=1, dtype=np.int32)), dtype=torch.float32)
    check_product(got, ref, s, v, torch.float32,
                  f"int4_w8_linear {t} x {n} x {rows} [{R.int4_w8_linear_kernel_name(c, dw)}]")


def test_products_over_four_gib_offsets():
    """An output whose last rows lie beyond 2^31 and 2^32 bytes."""
    t, n, rows = 140000, 64, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(-128, 128, (t, n), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (rows, n), generator=g, device="cuda").to(torch.int8)
    got = R.int8_linear(codes, torch.ones(t, device="cuda"), w, torch.ones(rows, device="cuda"), dtype=torch.float32)
    for rows_at in (0, 65530, 131068, t - 64):
        part = codes[rows_at:rows_at + 64].double() @ w.double().T.contiguous()
        assert torch.equal(got[rows_at:rows_at + 64].double(), part), rows_at


def test_products_empty_and_non_finite():
    w = torch.ones((8, 32), dtype=torch.int8, device="cuda")
    v = torch.ones(8, device="cuda")
    assert R.int8_linear(torch.empty((0, 32), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), w,
                         v).shape == (0, 8)
    codes = torch.ones((3, 32), dtype=torch.int8, device="cuda")
    out = R.int8_linear(codes, torch.tensor([1.0, float("inf"), float("nan")], device="cuda"), w, v)
    assert (out[0] == 32).all() and not torch.isfinite(out[1:]).any()


@pytest.mark.parametrize("t,n,rows", [(1, 2048, 512), (16, 4096, 256), (70, 4096, 512), (300, 1024, 520)])
def test_products_on_a_side_stream_and_in_a_graph(t, n, rows):
    """Another stream than the tensors' own, and a captured graph replayed with
    new inputs and the program's own work between the replays."""
    codes, s, _, w, v, b = operands(t, n, rows, 9, False)
    dc, ds, dw, dv, db = dev(codes), dev(s), dev(w), dev(v), dev(b)
    eager = R.int8_linear(dc, ds, dw, dv, bias=db)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = R.int8_linear(dc, ds, dw, dv, bias=db)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(eager, other)
    x = torch.randn((t, n), device="cuda").to(torch.bfloat16)

    def path():
        q, sc = R.quant_int8(x)
        return R.int8_linear(q, sc, dw, dv, bias=db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = path()
    for i in range(4):
        x.copy_(torch.randn((t, n), device="cuda").to(torch.bfloat16) * (i + 1))
        want = path()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want), i


def test_quantized_chain_is_near_the_bf16_product():
    """quant_int8 on activations and weight rows, then the product: within the
    quantization steps of x . w^T.  |x_hat - x| <= s/2 and |w_hat - w| <= v/2 give
    |out - x w| <= sum_j (s/2 |w| + v/2 |x| + s v / 4), and the product's own tolerance."""
    g = np.random.default_rng(12)
    x, w = bf16(g.standard_normal((40, 512))), bf16(g.standard_normal((96, 512)) / 20)
    q, s = R.quant_int8(x.cuda())
    qw, v, _ = R.quant_int8(w.cuda(), sums=True)
    out = R.int8_linear(q, s, qw, v, dtype=torch.float32).double().cpu().numpy()
    xd, wd = x.double().numpy(), w.double().numpy()
    sd, vd = s.double().cpu().numpy()[:, None], v.double().cpu().numpy()[None, :]
    bound = (sd / 2 * np.abs(wd).sum(1)[None, :] + vd / 2 * np.abs(xd).sum(1)[:, None] + 512 * sd * vd / 4) * (1 + 1e-5)
    assert (np.abs(out - xd @ wd.T) <= bound).all()


# ---- refusals ----------------------------------------------------------------


def test_bindings_refuse_wrong_operands():
    c = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    s, v = torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    w = torch.zeros((8, 32), dtype=torch.int8, device="cuda")
    bad = [lambda: R.int8_linear(c.cpu(), s, w, v), lambda: R.int8_linear(c.float(), s, w, v),
           lambda: R.int8_linear(c, s[:3], w, v), lambda: R.int8_linear(c, s, w[:, :16], v),
           lambda: R.int8_linear(c, s, w.t(), v), lambda: R.int8_linear(c, s.double(), w, v),
           lambda: R.int8_linear(c, s, w, v[:7]), lambda: R.int8_linear(c, s, w, v, dtype=torch.float16),
           lambda: R.int8_linear(c, s, w, v, bias=torch.ones(7, device="cuda")),
           lambda: R.int8_linear(c, s, w, v, out=torch.empty((4, 9), device="cuda")),
           lambda: R.int8_linear(c, s, w.cpu(), v),
           lambda: R.int4_w8_linear(c, s, s, w, v, v.int()),
           lambda: R.int4_w8_linear(c.view(torch.uint8), s, s, w, v, v.int()),
           lambda: R.quant_int8(torch.zeros((4, 8), device="cuda")),
           lambda: R.quant_int8(torch.zeros((4, 8), dtype=torch.bfloat16)),
           lambda: R.quant_int8(torch.zeros((8, 4), dtype=torch.bfloat16, device="cuda").t())]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted", i)


@pytest.mark.parametrize("n", [16, 22, 30])
def test_many_short_int4_rows(n):
    t, rows = 4100, 4000
    codes, s, z, w, v, b = operands(t, n, rows, 11, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, b)
    c, dw = dev(codes), dev(w)
    assert R.int4_w8_linear_kernel_name(c, dw) == "w8_any"
    got = R.int4_w8_linear(c, dev(s), dev(z), dw, dev(v), dev(w.sum(axis=1, dtype=np.int32)), bias=dev(b),
                           dtype=torch.float32)
    check_product(got, ref, s, v, torch.float32, f"int4_w8_linear {t} x {n} x {rows}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,rows", [(40, 2048, 2046), (200, 4096, 1030), (700, 256, 515), (520, 1024, 2049),
                                      (2500, 128, 1537)])
def test_output_rows_of_any_alignment(t, n, rows, dtype):
    """Output rows that start anywhere and end inside a vector, on the aligned tiles
    (with and without the split row): every element, and nothing around them."""
    codes, s, z, w, v, b = operands(t, n, rows, 12, False)
    ref = B.w8_linear(codes.astype(np.float64), s, None, w, v, b)
    dc, dw = dev(codes), dev(w)
    name = R.int8_linear_kernel_name(dc, dw)
    for ldo, off in ((rows, 1), (rows + 3, 0)):
        buf = torch.full((off + t * ldo,), float(GUARD), dtype=dtype, device="cuda")
        out = buf[off:].view(t, ldo)[:, :rows]
        R.int8_linear(dc, dev(s), dw, dev(v), bias=dev(b), out=out)
        check_product(out, ref, s, v, dtype, f"int8_linear into {ldo} + {off} [{name}]")
        assert (buf[:off] == GUARD).all() and (buf[off:].view(t, ldo)[:, rows:] == GUARD).all()
    codes, s, z, w, v, b = operands(t, n, rows, 13, True)
    ref = B.w8_linear(B.unpack_int4(codes), s, z, w, v, b)
    out = torch.full((t, rows + 1), float(GUARD), dtype=dtype, device="cuda")
    R.int4_w8_linear(dev(codes), dev(s), dev(z), dev(w), dev(v), dev(w.sum(axis=1, dtype=np.int32)), bias=dev(b),
                     out=out[:, :rows])
    check_product(out[:, :rows], ref, s, v, dtype, f"int4_w8_linear into {rows + 1}")
    assert (out[:, rows:] == GUARD).all()
