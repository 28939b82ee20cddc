"""Every kernel that the 8-bit products choose between, by its exact name, with and
without the row split: ragged tokens, channels and last steps, bias or none, both
output types, and work-groups that take a second tile.

The reference is the product in 64 bits on the GPU (whole numbers, so exact),
the tolerance that of the epilogue's roundings, u = 2^-24: the sum widened
(u |acc|), the zero-point's fused multiply-add (u |acc - shift|), two
multiplications (2u |product|), the bias (u |out|), 1.01 for second-order terms, and
half a unit of bf16's 8 significant bits (2^-8).
"""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Product:
    """Operands of one product and its value in 64 bits."""

    def __init__(self, t, n, rows, a4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(1000 * seed + t + n + rows)
        self.t, self.n, self.rows, self.a4 = t, n, rows, a4

        def whole(low, high, *shape):
            return torch.randint(low, high, shape, generator=g, device="cuda")

        def uniform(size):
            return torch.rand(size, generator=g, device="cuda")

        self.w = whole(-128, 128, rows, n).to(torch.int8)
        self.scale, self.w_scale = uniform(t) * 2 + 0.01, uniform(rows) / n ** 0.5
        self.bias = torch.randn(rows, generator=g, device="cuda") * 50
        if a4:
            self.codes = whole(0, 256, t, n // 2).to(torch.uint8)
            q = torch.stack((self.codes & 15, self.codes >> 4), dim=2).reshape(t, n).double()
            self.zero = torch.randn(t, generator=g, device="cuda") * 40
            self.w_sum = self.w.sum(dim=1, dtype=torch.int32)
            shift = self.zero.double()[:, None] * self.w_sum.double()[None, :]
        else:
            self.codes = whole(-128, 128, t, n).to(torch.int8)
            q, shift = self.codes.double(), 0.0
        acc = torch.matmul(q, self.w.double().T.contiguous())
        sv = self.scale.double()[:, None] * self.w_scale.double()[None, :]
        self.plain = sv * (acc - shift)
        self.slack = 1.01 * sv * U * (acc.abs() + 3 * (acc - shift).abs())

    def name(self):
        return (R.int4_w8_linear_kernel_name if self.a4 else R.int8_linear_kernel_name)(self.codes, self.w)

    def workspace(self):
        L, c, w = R.lib(), self.codes, self.w
        if self.a4:
            return L.signrot_int4_w8_linear_workspace(c.data_ptr(), self.t, self.n, w.data_ptr(), w.stride(0), self.rows)
        return L.signrot_int8_linear_workspace(c.data_ptr(), c.stride(0), self.t, self.n, w.data_ptr(), w.stride(0),
                                               self.rows)

    def __call__(self, bias, dtype):
        if self.a4:
            return R.int4_w8_linear(self.codes, self.scale, self.zero, self.w, self.w_scale, self.w_sum, bias=bias,
                                    dtype=dtype)
        return R.int8_linear(self.codes, self.scale, self.w, self.w_scale, bias=bias, dtype=dtype)

    def check(self):
        label = f"{'int4_w8' if self.a4 else 'int8'}_linear {self.t} x {self.n} x {self.rows} [{self.name()}]"
        for bias in (self.bias, None):
            want = self.plain if bias is None else self.plain + bias.double()[None, :]
            for dtype in (torch.float32, torch.bfloat16):
                print(f"[gpu] {label} bias {bias is not None} {dtype}", flush=True)
                got = self(bias, dtype)
                assert got.dtype is dtype and got.shape == want.shape
                tol = self.slack + 1.01 * (U + (2.0 ** -8 if dtype is torch.bfloat16 else 0.0)) * want.abs() + 1e-37
                over = ((got.double() - want).abs() / tol).max().item()
                assert over <= 1.0, (label, over)


# (tokens, n, rows, tile, row split); the second of a pair has more tiles than the
# device holds work-groups
TILES8 = [(405, 80, 16390, "256x256", False), (4101, 80, 4130, "256x256", False), (6007, 1040, 8203, "256x256", False),
          (201, 6000, 16390, "256x256", True), (65, 80, 16390, "128x128", False), (201, 80, 16390, "128x128", False),
          (67, 8208, 8203, "128x128", True), (33, 80, 77, "64x128", False), (129, 80, 16390, "64x128", False),
          (65, 14352, 1555, "64x128", True), (8201, 80, 130, "64x64", False), (33, 14352, 4130, "64x64", True),
          (33, 144, 77, "64x64_deep", False), (301, 4112, 601, "64x64_deep", False), (33, 4112, 77, "64x64_deep", True)]
TILES4 = [(405, 96, 16390, "256x256", False), (4101, 96, 4130, "256x256", False), (6007, 1056, 8203, "256x256", False),
          (201, 6176, 16390, "256x256", True), (65, 96, 16390, "128x128", False), (201, 96, 16390, "128x128", False),
          (65, 8224, 8203, "128x128", True), (33, 96, 77, "128x64", False), (201, 288, 16390, "128x64", False),
          (65, 4128, 77, "128x64", True), (33, 96, 16390, "64x64", False), (129, 96, 16390, "64x64", False),
          (33, 14368, 8203, "64x64", True), (33, 544, 77, "64x64_deep", False), (33, 4128, 77, "64x64_deep", True)]


@pytest.mark.parametrize("t,n,rows,tile,split", TILES8)
def test_int8_tiles(t, n, rows, tile, split):
    p = Product(t, n, rows, False)
    assert (p.name(), p.workspace() > 0) == ("w8_tile_" + tile, split)
    p.check()


@pytest.mark.parametrize("t,n,rows,tile,split", TILES4)
def test_int4_w8_tiles(t, n, rows, tile, split):
    p = Product(t, n, rows, True)
    assert (p.name(), p.workspace() > 0) == ("w8_tile_" + tile, split)
    p.check()


@pytest.mark.parametrize("a4", [False, True])
@pytest.mark.parametrize("t", [1, 16, 17, 32])
@pytest.mark.parametrize("rows", [4200, 8192, 8200, 14336, 16384, 16400])
def test_few_tokens_and_many_rows(t, rows, a4):
    """Groups of sixteen and of thirty-two channels, of two to eight waves, whole and
    cut off; last units of the row that are short, and rows of fewer units than waves."""
    for n in (96, 1056, 4128):
        p = Product(t, n, rows, a4)
        assert p.name() == "w8_few"
        p.check()


@pytest.mark.parametrize("t,n,rows,a4", [(6007, 1042, 8203, False), (6007, 1042, 8203, True),
                                         (5000, 4099, 4200, False), (5000, 4098, 4200, True)])
def test_rows_laid_out_anew_for_the_largest_tile(t, n, rows, a4):
    p = Product(t, n, rows, a4)
    assert p.name() == "w8_pack_tile_256x256"
    p.check()
    if not a4:  # aligned codes, which are read where they are: any bytes after a row's end
        pitch = (n + 15) // 16 * 16
        wide = torch.randint(-128, 128, (t, pitch), device="cuda").to(torch.int8)
        wide[:, :n] = p.codes
        whole = p.workspace()
        p.codes = wide[:, :n]
        assert p.name() == "w8_pack_tile_256x256" and p.workspace() == whole - t * pitch
        p.check()
