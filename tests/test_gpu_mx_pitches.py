"""The MXFP4 product on operands and results whose rows lie megabytes apart: pitches up to the greatest that the
kernels read in place, so that a tile's offsets come near 2^31 and its base passes 2^32, and the first that is laid
out anew.  The same results, bit for bit, as on compact operands, and nothing but the rows is read."""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu

MOST = 1 << 23  # bytes: pitches below it are read in place
TOTAL = 6 << 30  # bytes of a spread operand at most


def operand(rows, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (rows, n // 2), dtype=torch.uint8, device="cuda", generator=g)
    pitch = (n // 32 + 3) // 4 * 4
    scale = torch.randint(124, 130, (rows, pitch), dtype=torch.uint8, device="cuda", generator=g)
    return [codes, scale[:, :n // 32]]


def spread(v, pitch):
    """The rows of v at a pitch, NaN scales (255) between them."""
    rows, width = v.shape
    buf = torch.full(((rows - 1) * pitch + width,), 255, dtype=torch.uint8, device="cuda")
    return buf.as_strided((rows, width), (pitch, 1)).copy_(v)


def workspace(x, w):
    return R.lib().signrot_mxfp4_linear_workspace(
        x[0].data_ptr(), x[0].stride(0), x[1].data_ptr(), x[1].stride(0), x[0].shape[0], 2 * x[0].shape[1],
        w[0].data_ptr(), w[0].stride(0), w[1].data_ptr(), w[1].stride(0), w[0].shape[0])


# name, tokens, n, rows
CASES = [("mx_few16", 16, 8224, 700), ("mx_few16_k32", 13, 1056, 4100), ("mx_few32", 32, 4128, 700),
         ("mx_few32_k32", 25, 1056, 5119), ("mx_tile64x64", 600, 544, 700), ("mx_tile64x64", 700, 544, 600),
         ("mx_tile64x128", 129, 4096, 1040), ("mx_tile128x128_s4", 700, 8224, 700),
         ("mx_tile128x128_s2", 700, 1056, 8200), ("mx_tile256x256", 777, 1056, 14340),
         ("mx_tile256x256", 14340, 1056, 777)]


@pytest.mark.parametrize("name,t,n,rows", CASES)
def test_rows_megabytes_apart(name, t, n, rows):
    x, w = operand(t, n, 1), operand(rows, n, 2)
    assert R.mxfp4_linear_kernel_name(*x, *w) == name
    ref, need = R.mxfp4_linear(*x, *w), workspace(x, w)
    for side, op in (("tokens", x), ("weights", w)):
        for k, what in enumerate(("codes", "scales")):
            pitch = min(MOST - 16, TOTAL // op[k].shape[0] // 16 * 16)
            print(f"[gpu] {name} {t} x {n} x {rows}: {what} of the {side} {pitch} bytes apart", flush=True)
            far = list(op)
            far[k] = spread(op[k], pitch)
            a, b = (far, w) if op is x else (x, far)
            assert R.mxfp4_linear_kernel_name(*a, *b) == name and workspace(a, b) == need
            assert torch.equal(R.mxfp4_linear(*a, *b), ref), (what, side)


@pytest.mark.parametrize("t,n,rows", [(16, 1056, 40), (33, 544, 40), (777, 1056, 14340)])
def test_the_first_pitch_that_is_laid_out_anew(t, n, rows):
    """Codes, and scales but for the largest tiles', which order them from any pitch."""
    x, w = operand(t, n, 3), operand(rows, n, 4)
    ref, need = R.mxfp4_linear(*x, *w), workspace(x, w)
    ordered = R.mxfp4_linear_kernel_name(*x, *w) == "mx_tile256x256"
    for k, width in enumerate((n // 2, n // 32)):
        far = list(x)
        far[k] = spread(x[k], MOST)
        more = 0 if ordered and k == 1 else t * ((width + 15) // 16 * 16)
        assert workspace(far, w) >= need + more
        assert torch.equal(R.mxfp4_linear(*far, *w), ref), k


@pytest.mark.parametrize("name,t,n,rows", [c for c in CASES if c[1] < 14340])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_megabytes_apart(name, t, n, rows, dtype):
    x, w = operand(t, n, 5), operand(rows, n, 6)
    ref = R.mxfp4_linear(*x, *w, dtype=dtype)
    pitch = TOTAL // ref.element_size() // t + 1
    out = torch.empty((t - 1) * pitch + rows, dtype=dtype, device="cuda").as_strided((t, rows), (pitch, 1))
    R.mxfp4_linear(*x, *w, out=out)
    assert torch.equal(out, ref)
