"""Argument errors of the 8-bit products, the INT8 quantizer and the residual
norms: found on the host before any HIP call (no GPU needed)."""

import ctypes

import pytest

import rotation_activation_quantization_amd as R

FAKE = 0x100000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    return R.lib()


def test_quant_int8_argument_errors(L):
    def q(x=FAKE, t=4, n=64, ld=64, codes=FAKE, ldc=64, scale=FAKE, total=None):
        return L.signrot_quant_int8(x, t, n, ld, codes, ldc, scale, total, None)

    for kw in ({"t": -1}, {"t": 1 << 31}, {"n": 0}, {"n": 131072, "ld": 131072, "ldc": 131072}, {"ld": 63},
               {"ldc": 63}, {"x": None}, {"codes": None}, {"scale": None}, {"x": FAKE + 1}, {"scale": FAKE + 2},
               {"total": FAKE + 1}):
        assert q(**kw) == R.SIGNROT_EINVAL, kw
        assert L.signrot_last_error()
    assert q(t=0, x=None, codes=None, scale=None) == R.SIGNROT_OK


def test_int8_linear_argument_errors(L):
    def lin(codes=FAKE, ldc=64, scale=FAKE, t=4, n=64, w=FAKE, ldw=64, ws=FAKE, bias=None, rows=8, out=FAKE, ldo=8,
            kind=1, work=FAKE, size=1 << 40):
        return L.signrot_int8_linear(codes, ldc, scale, t, n, w, ldw, ws, bias, rows, out, ldo, kind, work, size,
                                     None)

    for kw in ({"t": -1}, {"rows": -1}, {"t": 1 << 31}, {"rows": 1 << 31, "ldo": 1 << 31}, {"n": 0},
               {"n": 131072, "ldc": 131072, "ldw": 131072}, {"ldc": 63}, {"ldw": 63}, {"ldo": 7}, {"kind": 2},
               {"kind": -1}, {"codes": None}, {"scale": None}, {"w": None}, {"ws": None}, {"out": None},
               {"out": FAKE + 1}, {"out": FAKE + 2, "kind": 0}, {"scale": FAKE + 1}, {"bias": FAKE + 2}):
        assert lin(**kw) == R.SIGNROT_EINVAL, kw
    assert lin(t=0, codes=None, out=None) == R.SIGNROT_OK
    assert lin(rows=0, w=None, out=None) == R.SIGNROT_OK


def test_int4_w8_linear_argument_errors(L):
    def lin(codes=FAKE, scale=FAKE, zero=FAKE, t=4, n=64, w=FAKE, ldw=64, ws=FAKE, total=FAKE, bias=None, rows=8,
            out=FAKE, ldo=8, kind=0, work=FAKE, size=1 << 40):
        return L.signrot_int4_w8_linear(codes, scale, zero, t, n, w, ldw, ws, total, bias, rows, out, ldo, kind, work,
                                        size, None)

    for kw in ({"t": -1}, {"n": 63}, {"n": 0}, {"n": 131072, "ldw": 131072}, {"ldw": 63}, {"ldo": 7}, {"kind": 3},
               {"codes": None}, {"zero": None}, {"total": None}, {"w": None}, {"out": None}, {"total": FAKE + 2},
               {"zero": FAKE + 1}):
        assert lin(**kw) == R.SIGNROT_EINVAL, kw
    assert lin(t=0, codes=None) == R.SIGNROT_OK
    assert lin(rows=0, w=None) == R.SIGNROT_OK


@pytest.mark.parametrize("t,n,rows", [(1, 14336, 4096), (16, 4096, 14336), (70, 4096, 512), (200, 11008, 4096),
                                      (8192, 4096, 14336), (613, 1111, 777)])
def test_workspace_sizes_are_checked(L, t, n, rows):
    need = L.signrot_int8_linear_workspace(FAKE, n, t, n, FAKE, n, rows)
    assert need >= 0
    if need:
        args = (FAKE, n, FAKE, t, n, FAKE, n, FAKE, None, rows, FAKE, rows, 1)
        assert L.signrot_int8_linear(*args, None, 0, None) == R.SIGNROT_EINVAL
        assert L.signrot_int8_linear(*args, FAKE, need - 1, None) == R.SIGNROT_EINVAL
        assert L.signrot_int8_linear(*args, FAKE + 4, need, None) == R.SIGNROT_EINVAL
    assert L.signrot_int8_linear_workspace(FAKE, n, t, 0, FAKE, n, rows) == -1
    assert L.signrot_int8_linear_workspace(FAKE, n, -1, n, FAKE, n, rows) == -1
    assert L.signrot_int8_linear_workspace(FAKE, n, t, n, FAKE, n - 1, rows) == -1
    assert L.signrot_int4_w8_linear_workspace(FAKE, t, 3, FAKE, 3, rows) == -1
    assert L.signrot_int4_w8_linear_workspace(FAKE, t, 64, FAKE, 64, rows) >= 0


def test_workspace_holds_the_rows_that_are_laid_out_anew(L):
    """Large unaligned weights and, if they are unaligned too, codes are packed into the workspace."""
    t, n, rows = 4096, 4096, 8192
    aligned = L.signrot_int8_linear_workspace(FAKE, n, t, n, FAKE, n, rows)
    assert L.signrot_int8_linear_workspace(FAKE, n, t, n, FAKE + 1, n, rows) == aligned + rows * n
    assert L.signrot_int8_linear_workspace(FAKE + 1, n, t, n, FAKE, n, rows) == aligned + (t + rows) * n
    assert L.signrot_int8_linear_workspace(FAKE, 5001, t, 5001, FAKE, 5001, rows) >= (t + rows) * 5008
    assert L.signrot_int4_w8_linear_workspace(FAKE, t, 5002, FAKE, 5002, rows) >= t * 2512 + rows * 5024
    # small ones and few tokens are not
    assert L.signrot_int8_linear_workspace(FAKE, 1111, 613, 1111, FAKE, 1111, 777) == 0
    assert L.signrot_int8_linear_workspace(FAKE, 5001, 32, 5001, FAKE, 5001, rows) == 0


def test_kernel_names_are_host_only(L):
    assert L.signrot_int8_linear_kernel_name(FAKE, 64, 4, 64, FAKE, 64, 8)
    assert L.signrot_int8_linear_kernel_name(FAKE, 63, 4, 64, FAKE, 64, 8) is None
    assert L.signrot_int4_w8_linear_kernel_name(FAKE, 4, 64, FAKE, 64, 8)
    assert L.signrot_int4_w8_linear_kernel_name(FAKE, 4, 63, FAKE, 64, 8) is None


GOOD = dict(tokens=4, n=64, h=FAKE, ldh=64, y=FAKE, ldy=64, h_out=FAKE, ldho=64, u=FAKE, ldu=64, alpha=1.0, beta=1.0,
            eps_post=1e-6, eps_pre=1e-6, post_norm=1, pre_norm=1, h_type=1, param_type=1)


@pytest.mark.parametrize("kw", [
    {"tokens": -1}, {"tokens": 1 << 31}, {"n": 0}, {"n": 131072}, {"h": None}, {"ldh": 63}, {"ldy": 63}, {"ldho": 63},
    {"ldho": 65}, {"ldu": 63}, {"h_out": None, "u": None}, {"codes": FAKE, "ldc": 64}, {"code_scale": FAKE},
    {"codes": FAKE, "ldc": 63, "code_scale": FAKE}, {"h_type": 2}, {"param_type": -1}, {"post_norm": 3},
    {"pre_norm": -1}, {"alpha": float("nan")}, {"beta": float("inf")}, {"eps_pre": -1.0}, {"eps_post": float("nan")},
    {"gate": FAKE, "ldg": 63}, {"gate": FAKE, "ldg": 64}, {"gate": FAKE, "ldg": 64, "mod_rows": 3},
    {"mod_shift": FAKE, "ldm": 64, "mod_rows": 0, "mod_index": FAKE}, {"mod_scale": FAKE, "ldm": 1},
    {"h": FAKE + 1}, {"pre_weight": FAKE + 1}, {"mod_index": FAKE + 2}, {"u": FAKE + 1}])
def test_residual_norm_argument_errors(L, kw):
    a = R._ResidualNormArgs(**{**GOOD, **kw})
    assert L.signrot_residual_norm(ctypes.addressof(a), None) == R.SIGNROT_EINVAL
    assert L.signrot_last_error()


def test_residual_norm_null_and_empty(L):
    assert L.signrot_residual_norm(None, None) == R.SIGNROT_EINVAL
    a = R._ResidualNormArgs(**{**GOOD, "tokens": 0, "h": None, "y": None})
    assert L.signrot_residual_norm(ctypes.addressof(a), None) == R.SIGNROT_OK


def test_struct_layout_matches_the_header(tmp_path):
    """Field offsets of the ctypes mirror against the C struct."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f[0] for f in R._ResidualNormArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "signrot.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu\\n", offsetof(signrot_residual_norm_args, {n}));\n' for n in names) +
        '  printf("%zu\\n", sizeof(signrot_residual_norm_args));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    want = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    got = [getattr(R._ResidualNormArgs, n).offset for n in names] + [ctypes.sizeof(R._ResidualNormArgs)]
    assert got == want


def test_rows_shorter_than_a_chunk_are_not_laid_out_anew(L):
    """Laying rows out anew reads sixteen bytes at a time: INT4 rows of fewer (n < 32)
    and INT8 rows of fewer (n < 16) take the kernel that reads what there is, however
    many tokens and channels there are."""
    for tokens, rows in ((33, 40), (4000, 4000), (8192, 28672), (100000, 70000)):
        for n in (16, 18, 24, 30):
            assert L.signrot_int4_w8_linear_kernel_name(FAKE, tokens, n, FAKE, n, rows) == b"w8_any", (tokens, n, rows)
            assert L.signrot_int4_w8_linear_workspace(FAKE, tokens, n, FAKE, n, rows) == 0
        for n in (1, 2, 15):
            assert L.signrot_int8_linear_kernel_name(FAKE, n, tokens, n, FAKE, n, rows) == b"w8_any", (tokens, n, rows)
            assert L.signrot_int8_linear_workspace(FAKE, n, tokens, n, FAKE, n, rows) == 0
