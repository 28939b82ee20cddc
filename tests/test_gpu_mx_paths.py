"""Every kernel that the MXFP4 product chooses between, by its exact name, with and
without the row split: ragged tokens, channels and last quads of blocks, bias or none,
both output types, and work-groups that take several tiles in turn.

The reference is the product in 64 bits on the GPU.  Tolerance, u = 2^-24: sums of n
binary32 terms in any order, 4 sqrt(n) u times the sum of their sizes (roundings at
random, beyond four deviations), the bias among them, and half a unit of the result's
digits (bf16 2^-8, binary32 u).
"""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
TILES = {"mx_tile256x256": (256, 256), "mx_tile128x128_s4": (128, 128), "mx_tile128x128_s2": (128, 128),
         "mx_tile64x128": (64, 128), "mx_tile64x64": (64, 64)}
VALUES = [s * m for s in (1.0, -1.0) for m in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)]


def operand(rows, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = n // 32
    pitch = (nb + 15) // 16 * 16
    codes = torch.randint(0, 256, (rows, n // 2), dtype=torch.uint8, device="cuda", generator=g)
    scale = torch.randint(124, 130, (rows, pitch), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scale[:, :nb]


def exact(op):
    codes, scale = op
    table = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    power = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [float("nan")], dtype=torch.float64, device="cuda")
    v = table[torch.stack((codes & 15, codes >> 4), dim=2).long().reshape(codes.shape[0], -1)]
    return v * power[scale.long()].repeat_interleave(32, dim=1)


def splits_of(x, w, name):
    """Parts of a row, from the workspace: partial sums, and the large tiles' ordered scales."""
    t, n, rows = x[0].shape[0], 2 * x[0].shape[1], w[0].shape[0]
    size = R.lib().signrot_mxfp4_linear_workspace(x[0].data_ptr(), n // 2, x[1].data_ptr(), x[1].stride(0), t, n,
                                                  w[0].data_ptr(), n // 2, w[1].data_ptr(), w[1].stride(0), rows)
    if name not in TILES:
        assert size == 0
        return 1
    bm, bn = TILES[name]
    if name == "mx_tile256x256":
        size -= 4096 * ((n + 511) // 512) * ((t + 255) // 256 + (rows + 255) // 256)
    part = 4 * bm * bn * ((t + bm - 1) // bm) * ((rows + bn - 1) // bn)
    assert size % part == 0
    return max(size // part, 1)


CASES = [
    # name, parts, tokens, n, rows
    ("mx_few16", 1, 1, 32, 1), ("mx_few16", 1, 1, 4096, 14336), ("mx_few16", 1, 16, 8224, 40), ("mx_few16", 1, 4, 2080, 8199),
    ("mx_few16_k32", 1, 7, 2080, 8199), ("mx_few16_k32", 1, 16, 14336, 4100), ("mx_few16_k32", 1, 13, 32, 28673),
    ("mx_few32", 1, 17, 32, 3), ("mx_few32", 1, 32, 4128, 1040), ("mx_few32", 1, 29, 14336, 777),
    ("mx_few32_k32", 1, 17, 96, 4097), ("mx_few32_k32", 1, 32, 8224, 16384), ("mx_few32_k32", 1, 25, 4128, 5119),
    ("mx_tile64x64", 1, 33, 544, 40), ("mx_tile64x64", 1, 300, 1024, 2100), ("mx_tile64x64", 3, 4100, 4096, 40),
    ("mx_tile64x64", 8, 33, 4128, 40), ("mx_tile64x64", 16, 33, 8224, 40),
    ("mx_tile64x128", 1, 33, 32, 40), ("mx_tile64x128", 1, 100, 96, 4099), ("mx_tile64x128", 2, 33, 8224, 14340),
    ("mx_tile64x128", 6, 129, 4096, 1040), ("mx_tile64x128", 16, 33, 8224, 77),
    ("mx_tile128x128_s4", 1, 200, 32, 8200), ("mx_tile128x128_s4", 4, 3000, 8224, 130),
    ("mx_tile128x128_s4", 12, 65, 14336, 2100), ("mx_tile128x128_s2", 1, 257, 32, 14340),
    ("mx_tile128x128_s2", 1, 4099, 1056, 2050), ("mx_tile128x128_s2", 3, 200, 14336, 8200),
    ("mx_tile256x256", 1, 777, 1056, 14340), ("mx_tile256x256", 1, 3000, 2080, 14336),
    ("mx_tile256x256", 2, 257, 14336, 14340), ("mx_tile256x256", 3, 1030, 8224, 4096),
]


@pytest.mark.parametrize("name,parts,t,n,rows", CASES)
def test_each_kernel(name, parts, t, n, rows):
    x, w = operand(t, n, t + n), operand(rows, n, rows + n + 1)
    assert R.mxfp4_linear_kernel_name(*x, *w) == name
    assert splits_of(x, w, name) == parts
    a, b = exact(x), exact(w).T.contiguous()
    ref, size = torch.matmul(a, b), torch.matmul(a.abs(), b.abs())
    del a, b
    bias = torch.randn(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows)) * 50
    for dtype in (BF16, F32):
        for add in (None, bias):
            print(f"[gpu] {name} {t} x {n} x {rows} {dtype} bias {add is not None}", flush=True)
            out = R.mxfp4_linear(*x, *w, bias=add, dtype=dtype)
            c = torch.zeros_like(ref[0]) if add is None else add.double()
            want = ref + c
            allowed = 4 * n ** 0.5 * U * (size + c.abs()) + (2.0 ** -8 if dtype is BF16 else U) * want.abs()
            over = ((out.double() - want).abs() - allowed).max().item()
            assert over <= 0, (dtype, add is not None, over)
            again = R.mxfp4_linear(*x, *w, bias=add, dtype=dtype)
            assert torch.equal(out, again)


@pytest.mark.parametrize("name,t,n,rows", [("mx_tile256x256", 8192, 2080, 14336), ("mx_tile128x128_s2", 4099, 1056, 2050),
                                           ("mx_tile64x128", 70, 160, 8200)])
def test_rows_depend_on_their_own_operands_only(name, t, n, rows):
    """Many tiles a work-group: each result equals that of a product of its token alone
    within the roundings, and the place of a token does not matter."""
    x, w = operand(t, n, 5), operand(rows, n, 6)
    assert R.mxfp4_linear_kernel_name(*x, *w) == name
    out = R.mxfp4_linear(*x, *w, dtype=F32)
    order = torch.randperm(t, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    moved = R.mxfp4_linear(x[0][order].contiguous(), x[1][order].contiguous(), *w, dtype=F32)
    assert torch.equal(moved, out[order])


def test_two_graphs_and_eager_calls_between():
    """Captured products of their own workspaces, replayed in turn with eager work between."""
    todo = []
    for t, n, rows in ((300, 1024, 2100), (65, 14336, 2100), (1030, 8224, 4096), (3, 4096, 512)):
        x, w = operand(t, n, t), operand(rows, n, rows)
        todo.append([x, w, R.mxfp4_linear(*x, *w), torch.empty(t, rows, dtype=BF16, device="cuda"), None])
    torch.cuda.synchronize()
    for c in todo:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            R.mxfp4_linear(*c[0], *c[1], out=c[3])
        c[4] = g
    for _ in range(3):
        for x, w, want, out, g in todo:
            out.zero_()
            g.replay()
            assert torch.equal(R.mxfp4_linear(*x, *w), want)
        torch.cuda.synchronize()
        for _, _, want, out, _ in todo:
            assert torch.equal(out, want)
    for x, w, want, out, g in todo:  # new operands in the captured places
        x[0].copy_(x[0].flip(0).contiguous())
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, R.mxfp4_linear(*x, *w))


def test_products_on_two_streams_at_once():
    a, b = operand(300, 8224, 1), operand(2100, 8224, 2)
    want = R.mxfp4_linear(*a, *b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(R.mxfp4_linear(*a, *b))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("t", [1, 3, 16, 29, 33, 70, 300])
@pytest.mark.parametrize("n,rows", [(32, 300), (64, 40), (96, 8200), (160, 77), (1120, 777), (2080, 8200), (4256, 2100)])
def test_scales_at_any_address(t, n, rows):
    """The same bits as from aligned rows, whatever stands beside them (0xff: NaN)."""
    x, w = operand(t, n, t + 3), operand(rows, n, n)
    want = R.mxfp4_linear(*x, *w, dtype=F32)
    assert torch.isfinite(want).all()

    def moved(scale, off, pitch):
        count, nb = scale.shape
        room = torch.full((off + count * pitch + 64,), 255, dtype=torch.uint8, device="cuda")
        view = room[off:off + count * pitch].view(count, pitch)[:, :nb]
        view.copy_(scale)
        return view

    nb = n // 32
    for off_x, off_w, wide in ((0, 0, 0), (1, 2, 0), (3, 1, 1), (2, 0, 2), (0, 3, 3)):
        a, b = moved(x[1], off_x, nb + wide), moved(w[1], off_w, nb + wide)
        assert torch.equal(R.mxfp4_linear(x[0], a, w[0], b, dtype=F32), want), (off_x, off_w, wide)
        assert torch.equal(R.mxfp4_linear(x[0], x[1], w[0], b, dtype=F32), want)
        assert torch.equal(R.mxfp4_linear(x[0], a, *w, dtype=F32), want)
