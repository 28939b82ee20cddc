"""The rotation straight to MXFP4: the codes and scales of the rotated rows that
the INT4 entry points give with y_out, bit for bit, and near the oracle's
rotation."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import mx_oracle as M  # noqa: E402

pytestmark = pytest.mark.gpu

FAST = (3584, 7168, 14336, 28672, 4096, 8192, 16384)
# an outer order with 1, 2, 4, 8 and 16 column tiles, small and large orders among them
OUTER = (320, 896, 192, 5504, 640, 11008, 1280, 8960, 5120, 13824, 18944, 27648, 24576, 32768, 64)
GENERIC = (2, 8, 16, 32, 96, 224, 7424)


def rows(t, n, c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((t, n), generator=g, device="cuda") * 0.7
    x[::3, c] = 1500.0
    pitch = (n + 7) // 8 * 8  # the entry points' rows start on 16-byte boundaries
    out = torch.zeros((t, pitch), dtype=torch.bfloat16, device="cuda")[:, :n]
    return out.copy_(x)


def equal(got, ref, label):
    for name, a, b in zip(("codes", "scale"), got, ref):
        assert torch.equal(a, b), f"{label}: {(a != b).sum().item()} {name} differ"


@pytest.mark.parametrize("rule", ["floor", "noclip"])
@pytest.mark.parametrize("n", FAST + OUTER + GENERIC)
def test_rotated_codes_equal_the_quantizer_on_the_rotated_rows(n, rule):
    for t, c, sigma in ((1, 0, 1), (7, n - 1, -1), (601, n // 3, 1), (1300 if n <= 14336 else 2, n // 2, -1)):
        x = rows(t, n, c, 5)
        y = R.rotate_quant_int4_outlier(x, c, sigma, y_out=True)[3]
        equal(R.rotate_quant_mxfp4(x, c, sigma, rule=rule), R.quant_mxfp4(y, rule=rule), (n, t, R.kernel_name(n)))


@pytest.mark.parametrize("n", (4096, 14336, 28672, 13824, 5504, 224))
def test_rotated_values_are_near_the_oracle(n):
    t, c, sigma = 5, n // 5, -1
    x = rows(t, n, c, 6)
    y = O.rotate(x.double().cpu().numpy()) * (sigma * O.hadamard_row(n, c))
    codes, scale = R.rotate_quant_mxfp4(x, c, sigma, rule="noclip")
    # a value is off its nearest level by at most half the widest gap, 1 scale, and y by binary32's roundings
    step = np.repeat(np.ldexp(1.0, scale.cpu().numpy().astype(int) - 127), 32, axis=1)[:, :n]
    off = np.abs(R.dequant_mxfp4(codes, scale, n=n).double().cpu().numpy() - y)
    assert (off <= step * (1 + 1e-5) + 1e-5 * np.abs(y).max(axis=1, keepdims=True)).all()


@pytest.mark.parametrize("n", FAST)
def test_swiglu_rotated_codes_equal_the_unfused_path(n):
    for t, c, sigma in ((1, 0, -1), (37, n - 1, 1), (900, n // 7, 1)):
        both = torch.randn((t, 2 * n), device="cuda").to(torch.bfloat16)
        gate, up = both[:, :n], both[:, n:]
        y = R.swiglu_rotate_quant_int4(gate, up, c, sigma, y_out=True)[3]
        for rule in ("floor", "noclip"):
            equal(R.swiglu_rotate_quant_mxfp4(gate, up, c, sigma, rule=rule), R.quant_mxfp4(y, rule=rule), (n, t))


@pytest.mark.parametrize("n", (8192, 14336, 28672, 5120, 5504, 320, 224))
def test_strided_rows_outputs_and_guards(n):
    t, c = 9, 3
    wide = rows(t, n + 24, c, 7)
    x, nb = wide[:, 8:8 + n], (n + 31) // 32
    cbuf = torch.full((t, 16 * nb + 48), 77, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((t, nb + 3), 78, dtype=torch.uint8, device="cuda")
    out = cbuf[:, 16:16 + 16 * nb], sbuf[:, 1:1 + nb]
    assert R.rotate_quant_mxfp4(x, c, 1, out=out)[0] is out[0]
    equal(out, R.rotate_quant_mxfp4(x.contiguous(), c, 1), n)
    assert (cbuf[:, :16] == 77).all() and (cbuf[:, 16 + 16 * nb:] == 77).all()
    assert (sbuf[:, 0] == 78).all() and (sbuf[:, 1 + nb:] == 78).all()


@pytest.mark.parametrize("n", (4096, 28672, 13824))
def test_non_finite_rows_are_visible_and_apart(n):
    x = rows(12, n, 5, 8)
    clean = R.rotate_quant_mxfp4(x, 5, 1)
    x[4, 100], x[9, n - 1] = float("nan"), float("inf")
    codes, scale = R.rotate_quant_mxfp4(x, 5, 1)
    bad = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad[4] = bad[9] = True
    assert (scale[bad] == 255).all() and not codes[bad].any()
    equal((codes[~bad], scale[~bad]), (clean[0][~bad], clean[1][~bad]), n)


@pytest.mark.parametrize("n", (14336, 28672, 13824, 224))
def test_in_a_graph_and_on_a_side_stream(n):
    x, y = rows(40, n, 5, 9), rows(40, n, 5, 10)
    refs = [R.rotate_quant_mxfp4(v, 5, -1) for v in (x, y)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        equal(R.rotate_quant_mxfp4(x, 5, -1), refs[0], "side stream")
    torch.cuda.current_stream().wait_stream(side)
    if n == 224:
        return  # the general kernel allocates
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = R.rotate_quant_mxfp4(held, 5, -1)
    for k, (src, ref) in enumerate(((x, refs[0]), (y, refs[1]), (x, refs[0]))):
        held.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        equal(out, ref, k)


def test_refusals():
    x = rows(4, 4096, 0, 11)
    ok = R.rotate_quant_mxfp4(x, 0, 1)
    for call in (lambda: R.rotate_quant_mxfp4(x, 0, 1, rule="up"), lambda: R.rotate_quant_mxfp4(x.float(), 0, 1),
                 lambda: R.rotate_quant_mxfp4(x, 0, 1, out=(ok[0][:3], ok[1])),
                 lambda: R.swiglu_rotate_quant_mxfp4(x, x[:, :2048], 0, 1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: R.rotate_quant_mxfp4(x, 4096, 1), lambda: R.rotate_quant_mxfp4(x, 0, 2),
                 lambda: R.rotate_quant_mxfp4(x[:, :4090].contiguous(), 0, 1),
                 lambda: R.swiglu_rotate_quant_mxfp4(x[:, :896].contiguous(), x[:, :896].contiguous(), 0, 1)):
        with pytest.raises(R.SignRotError):
            call()
