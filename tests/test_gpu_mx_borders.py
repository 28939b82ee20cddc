"""The MXFP4 quantizer where a value decides: every exponent of a block's largest value, maxima on both sides of where
"noclip" takes the next scale, and the values halfway between two levels with their neighbours, of both signs, in
blocks of every scale.  Codes and scales have to equal the definition's."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import mx_oracle as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TIES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def grid(x, dtype):
    """float64 -> its nearest numbers of the type, as bits (0 for what is below half the least one)."""
    t = torch.from_numpy(np.asarray(x, np.float64)).to(dtype)
    return t.view(torch.int16 if dtype is BF16 else torch.int32).to(torch.int64)


def values(bits, dtype):
    return bits.to(torch.int16 if dtype is BF16 else torch.int32).view(dtype)


def blocks(dtype):
    """(x [rows, 128] of the type, lead exponent k and mantissa m of each row): four blocks a row, for either rule's
    exponent and either sign, each led by the same magnitude."""
    digits = 7 if dtype is BF16 else 23
    rows, leads = [], []
    for k in range(-126 - digits, 128):
        for m in (1.0, 1.5 - 2.0 ** -digits, 1.5, 1.5 + 2.0 ** -digits, 1.75, 2.0 - 2.0 ** -digits):
            lead = grid([m * 2.0 ** k], dtype)
            row = []
            for e in (max(k - 2, -127), max(k - 1, -127)):
                near = grid([t * 2.0 ** e for t in TIES + (6.0,)], dtype)
                near = torch.cat((near - 1, near, near + 1)).clamp(min=0)  # 24
                more = grid([v * 2.0 ** e for v in (0.0, 0.5, 1.0, 2.0, 3.0)], dtype)
                more = torch.cat((more, torch.tensor([1, 2])))  # the least numbers of the type
                block = torch.cat((lead, torch.minimum(torch.cat((near, more)), lead)))
                sign = 1 << 15 if dtype is BF16 else 1 << 31
                row += [block, block - sign]  # the sign bit, as two's complement
            rows.append(torch.cat(row))
            leads.append((k, m))
    return values(torch.stack(rows), dtype), np.array(leads)


@pytest.mark.parametrize("off", [0, 1])  # rows of whole aligned vectors, and rows at any address
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_scale_border_and_tie(dtype, off):
    x, leads = blocks(dtype)
    t, n = x.shape
    buf = torch.zeros(off + t * (n + off), dtype=dtype, device="cuda")
    dev = buf[off:].as_strided((t, n), (n + off, 1))
    dev.copy_(x)
    exact = x.double().numpy()
    assert n == 128 and np.isfinite(exact).all()
    scales = {}
    for rule in ("floor", "noclip"):
        codes, scale = (v.cpu().numpy() for v in R.quant_mxfp4(dev, rule=rule))
        want = M.quant(exact, rule)
        for name, got, ref in (("codes", codes, want[0]), ("scale", scale, want[1])):
            bad = np.argwhere(got != ref)
            assert bad.size == 0, (rule, name, len(bad), leads[bad[0][0]], bad[0], got[tuple(bad[0])], ref[tuple(bad[0])])
        assert set(np.concatenate((codes.ravel() & 15, codes.ravel() >> 4))) == set(range(16))
        scales[rule] = scale
    # what the inputs are meant to reach: all scales, and the rules apart where a block passes 6 scales, only there
    assert set(scales["floor"].ravel()) == set(range(253)) and set(scales["noclip"].ravel()) == set(range(254))
    k, m = leads.T
    apart = scales["floor"] != scales["noclip"]
    assert np.array_equal(apart, np.repeat(((m > 1.5) & (k >= -125))[:, None], 4, axis=1))
