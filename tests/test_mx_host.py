"""Argument errors of the MXFP4 operators and of the per-head norms: found on
the host before any HIP call (no GPU needed)."""

import ctypes

import pytest

import rotation_activation_quantization_amd as R

FAKE = 0x100000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    return R.lib()


def test_quant_argument_errors(L):
    def q(x=FAKE, kind=1, t=4, n=100, ld=100, rule=0, codes=FAKE, ldc=64, scale=FAKE, lds=4):
        return L.signrot_quant_mxfp4(x, kind, t, n, ld, rule, codes, ldc, scale, lds, None)

    for kw in ({"t": -1}, {"t": 1 << 31}, {"n": 0}, {"n": 131073, "ld": 1 << 20, "ldc": 1 << 20, "lds": 1 << 20},
               {"ld": 99}, {"ldc": 63}, {"lds": 3}, {"kind": 2}, {"kind": -1}, {"rule": 2}, {"rule": -1}, {"x": None},
               {"codes": None}, {"scale": None}, {"x": FAKE + 1}, {"x": FAKE + 2, "kind": 0}):
        assert q(**kw) == R.SIGNROT_EINVAL, kw
        assert L.signrot_last_error()
    assert q(t=0, x=None, codes=None, scale=None) == R.SIGNROT_OK


def test_dequant_argument_errors(L):
    def d(codes=FAKE, ldc=64, scale=FAKE, lds=4, t=4, n=100, y=FAKE, kind=0, ldy=100):
        return L.signrot_dequant_mxfp4(codes, ldc, scale, lds, t, n, y, kind, ldy, None)

    for kw in ({"t": -1}, {"n": 0}, {"ldc": 63}, {"lds": 3}, {"ldy": 99}, {"kind": 5}, {"y": None}, {"codes": None},
               {"scale": None}, {"y": FAKE + 2}, {"y": FAKE + 1, "kind": 1}):
        assert d(**kw) == R.SIGNROT_EINVAL, kw
    assert d(t=0, codes=None, y=None) == R.SIGNROT_OK


def test_linear_argument_errors(L):
    def lin(codes=FAKE, ldc=32, scale=FAKE, lds=2, t=4, n=64, w=FAKE, ldw=32, ws=FAKE, ldws=2, bias=None, rows=8,
            out=FAKE, ldo=8, kind=1, work=FAKE, size=1 << 40):
        return L.signrot_mxfp4_linear(codes, ldc, scale, lds, t, n, w, ldw, ws, ldws, bias, rows, out, ldo, kind, work,
                                      size, None)

    big = {"ldc": 1 << 20, "lds": 1 << 20, "ldw": 1 << 20, "ldws": 1 << 20}
    for kw in ({"t": -1}, {"rows": -1}, {"t": 1 << 30}, {"rows": 1 << 30, "ldo": 1 << 31}, {"n": 0}, {"n": 48},
               {"n": 131104, **big}, {"ldc": 31}, {"lds": 1}, {"ldw": 31}, {"ldws": 1}, {"ldo": 7}, {"kind": 2},
               {"codes": None}, {"scale": None}, {"w": None}, {"ws": None}, {"out": None}, {"out": FAKE + 1},
               {"out": FAKE + 2, "kind": 0}, {"bias": FAKE + 2}):
        assert lin(**kw) == R.SIGNROT_EINVAL, kw
    assert lin(t=0, codes=None, out=None) == R.SIGNROT_OK
    assert lin(rows=0, w=None, out=None) == R.SIGNROT_OK


@pytest.mark.parametrize("t,n,rows", [(1, 4096, 14336), (16, 14336, 4096), (33, 28672, 8192), (613, 1120, 777),
                                      (8192, 4096, 14336)])
@pytest.mark.parametrize("off", [0, 1])
def test_linear_workspace_is_asked_for_and_checked(L, t, n, rows, off):
    nb = n // 32
    sizes = (FAKE, 16 * nb, FAKE + off, nb, t, n, FAKE + 16 * off, 16 * nb, FAKE, nb)
    need = L.signrot_mxfp4_linear_workspace(*sizes, rows)
    assert need >= 0 and L.signrot_mxfp4_linear_kernel_name(*sizes, rows)
    if need > 0:
        for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 4, need)):
            assert L.signrot_mxfp4_linear(*sizes, None, rows, FAKE, rows, 1, ws, size, None) == R.SIGNROT_EINVAL
    assert L.signrot_mxfp4_linear_workspace(*sizes[:5], n + 1, *sizes[6:], rows) == -1
    assert L.signrot_mxfp4_linear_kernel_name(*sizes[:5], n + 1, *sizes[6:], rows) is None


def test_rotate_quant_argument_errors(L):
    def rot(x=FAKE, t=4, n=4096, ld=4096, c=5, sigma=1, rule=0, codes=FAKE, ldc=2048, scale=FAKE, lds=128, work=FAKE,
            size=1 << 40):
        return L.signrot_rotate_quant_mxfp4(x, t, n, ld, c, sigma, rule, codes, ldc, scale, lds, work, size, None)

    for kw in ({"t": -1}, {"t": 1 << 31}, {"ld": 4095}, {"ld": 4097}, {"c": -1}, {"c": 4096}, {"sigma": 0},
               {"rule": 2}, {"ldc": 2047}, {"ldc": 2056}, {"lds": 127}, {"x": None}, {"codes": None}, {"scale": None},
               {"x": FAKE + 2}, {"codes": FAKE + 8}):
        assert rot(**kw) == R.SIGNROT_EINVAL, kw
    assert rot(n=4098, ld=8192) == R.SIGNROT_EUNSUPPORTED_N
    assert rot(t=0, x=None, codes=None, scale=None, work=None, size=0) == R.SIGNROT_OK
    assert L.signrot_rotate_quant_mxfp4_workspace(-1, 4096) == -1
    assert L.signrot_rotate_quant_mxfp4_workspace(4, 4098) == -1
    assert L.signrot_rotate_quant_mxfp4_workspace(4, 4096) == 0  # a fused width
    need = L.signrot_rotate_quant_mxfp4_workspace(4, 224)
    assert need >= 4 * 4 * 224
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 4, need)):
        assert rot(n=224, ld=224, ldc=112, lds=7, work=ws, size=size) == R.SIGNROT_EINVAL


def test_swiglu_rotate_quant_argument_errors(L):
    def rot(gate=FAKE, up=FAKE, t=4, n=4096, ld=4096, c=5, sigma=1, rule=0, codes=FAKE, ldc=2048, scale=FAKE, lds=128):
        return L.signrot_swiglu_rotate_quant_mxfp4(gate, up, t, n, ld, c, sigma, rule, codes, ldc, scale, lds, None)

    for kw in ({"t": -1}, {"ld": 4095}, {"c": 4096}, {"sigma": 2}, {"rule": -1}, {"ldc": 2047}, {"lds": 127},
               {"gate": None}, {"up": None}, {"codes": None}, {"scale": None}, {"up": FAKE + 2}, {"codes": FAKE + 4}):
        assert rot(**kw) == R.SIGNROT_EINVAL, kw
    assert rot(n=192, ld=192, ldc=96, lds=6) == R.SIGNROT_EUNSUPPORTED_N
    assert rot(t=0, gate=None, up=None, codes=None, scale=None) == R.SIGNROT_OK


def _qk_args(**kw):
    f = dict(tokens=4, head=64, rotary=64, q=FAKE, ldq=256, hsq=64, q_out=FAKE + 65536, ldqo=256, hsqo=64, k=FAKE,
             ldk=128, hsk=64, k_out=FAKE + 131072, ldko=128, hsko=64, cos=FAKE, sin=FAKE, ldt=32, places=16,
             positions=FAKE, q_weight=FAKE, k_weight=FAKE, q_bias=None, k_bias=None, q_heads=4, k_heads=2, eps=1e-6,
             norm=1, interleaved=0, positions_64=0, in_type=1, out_type=1, param_type=1)
    f.update(kw)
    return R._QkNormRopeArgs(**f)


def test_qk_norm_rope_argument_errors(L):
    for kw in ({"tokens": -1}, {"tokens": 1 << 31}, {"head": 6}, {"head": 63}, {"head": 514}, {"rotary": 66},
               {"rotary": 3}, {"rotary": -2}, {"q_heads": 0}, {"q_heads": 65537}, {"k_heads": -1}, {"in_type": 2},
               {"out_type": -1}, {"param_type": 7}, {"norm": 3}, {"norm": -1}, {"eps": -1.0}, {"eps": float("nan")},
               {"eps": float("inf")}, {"interleaved": 2}, {"positions_64": -1}, {"ldq": -1}, {"hsk": -1}, {"ldt": 31},
               {"q": None}, {"q_out": None}, {"k": None}, {"k_out": None}, {"cos": None}, {"sin": None}, {"places": 0},
               {"positions": None, "places": 3}, {"q": FAKE + 1}, {"cos": FAKE + 2}, {"positions": FAKE + 2},
               {"positions": FAKE + 4, "positions_64": 1}, {"q_weight": FAKE + 1},
               {"q_weight": FAKE + 2, "param_type": 0}, {"q_out": FAKE, "ldqo": 512},
               {"q_out": FAKE, "in_type": 0, "ldq": 256}):
        assert L.signrot_qk_norm_rope(ctypes.addressof(_qk_args(**kw)), None) == R.SIGNROT_EINVAL, kw
        assert L.signrot_last_error()
    assert L.signrot_qk_norm_rope(None, None) == R.SIGNROT_EINVAL
    assert L.signrot_qk_norm_rope(ctypes.addressof(_qk_args(tokens=0, q=None)), None) == R.SIGNROT_OK


def test_qk_args_pack_as_the_struct():
    size = ctypes.sizeof(R._QkNormRopeArgs)
    fields = [name for name, _ in R._QkNormRopeArgs._fields_]
    packed = R._pack_qk_args(*[0.5 if name == "eps" else i + 1 for i, name in enumerate(fields)])
    assert len(packed) == size
    back = R._QkNormRopeArgs.from_buffer_copy(packed)
    for i, name in enumerate(fields):
        assert getattr(back, name) == (0.5 if name == "eps" else i + 1)


torch = pytest.importorskip("torch")


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    u = torch.zeros((2, 32), dtype=torch.uint8)
    h = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: R.quant_mxfp4(x), lambda: R.dequant_mxfp4(u, u[:, :2]),
                 lambda: R.mxfp4_linear(u, u[:, :2], u, u[:, :2]), lambda: R.rotate_quant_mxfp4(x, 0, 1),
                 lambda: R.swiglu_rotate_quant_mxfp4(x, x, 0, 1), lambda: R.qk_norm_rope(h)):
        with pytest.raises(ValueError):
            call()
