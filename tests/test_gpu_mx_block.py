"""A block's operators in MXFP4 as they run one after another: the residual norm, its
codes, the product to queries, keys and values, their norms and rotation, and the MLP
whose activation is gated, rotated and quantized in one pass for a product on folded
weights.  Each step is held against the 64-bit definition of what it was given; the whole
gives the same bits eager, on another stream and from a graph."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import mx_oracle as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HEADS, KV, D, N, FFN = 6, 2, 80, 480, 4096


def host(x):
    return x.double().cpu().numpy()


class Block:
    def __init__(self, t):
        g = torch.Generator(device="cuda").manual_seed(t)

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.h = normal(t, N).to(BF16)
        self.y = normal(t, N).to(BF16)
        self.weight = (normal(N, scale=0.1) + 1).to(BF16)
        self.w_qkv = R.quant_mxfp4(normal((HEADS + 2 * KV) * D, N, scale=N ** -0.5))
        self.w_both = R.quant_mxfp4(normal(2 * FFN, N, scale=N ** -0.5))
        self.c, self.sigma = 17, -1
        plain = normal(N, FFN, scale=FFN ** -0.5).to(BF16)
        row = torch.tensor([1 - 2 * (bin(self.c & j).count("1") & 1) for j in range(FFN)], dtype=torch.int8, device="cuda")
        self.plain = plain
        self.w_down = R.quant_mxfp4(R.fold_weights(plain, self.sigma * row))
        angle = torch.rand((1024, D // 2), generator=g, device="cuda") * 6
        self.cos, self.sin = angle.cos(), angle.sin()
        self.positions = torch.randint(0, 1024, (t,), generator=g, device="cuda", dtype=torch.int64)
        self.q_weight, self.k_weight = normal(D) + 1, normal(D) + 1

    def run(self):
        t = self.h.shape[0]
        o = {}
        o["h"], o["u"] = R.residual_norm(self.h, self.y, weight=self.weight)
        o["codes"] = R.quant_mxfp4(o["u"])
        o["qkv"] = R.mxfp4_linear(*o["codes"], *self.w_qkv)
        o["q_in"] = o["qkv"][:, :HEADS * D].unflatten(1, (HEADS, D))
        o["k_in"] = o["qkv"][:, HEADS * D:(HEADS + KV) * D].unflatten(1, (KV, D))
        o["q"], o["k"] = R.qk_norm_rope(o["q_in"], o["k_in"], self.cos, self.sin, positions=self.positions,
                                        q_weight=self.q_weight, k_weight=self.k_weight)
        o["both"] = R.mxfp4_linear(*o["codes"], *self.w_both)
        assert o["both"].shape == (t, 2 * FFN)
        o["act"] = R.swiglu_rotate_quant_mxfp4(o["both"][:, :FFN], o["both"][:, FFN:], self.c, self.sigma)
        o["down"] = R.mxfp4_linear(*o["act"], *self.w_down, dtype=F32)
        return o


def near(got, ref, size, n, dtype):
    """Sums of n binary32 terms, 4 sqrt(n) u of their sizes, and the result's half-step."""
    allowed = 4 * n ** 0.5 * U * size + (2.0 ** -8 if dtype is BF16 else U) * np.abs(ref)
    return (np.abs(host(got) - ref) <= allowed).all()


def values(op):
    return M.dequant(op[0].cpu().numpy(), op[1].cpu().numpy())


@pytest.mark.parametrize("t", [1, 7, 40, 333])
def test_each_step(t):
    b = Block(t)
    o = b.run()
    codes, scale = M.quant(host(o["u"]))
    assert np.array_equal(o["codes"][0].cpu().numpy(), codes) and np.array_equal(o["codes"][1].cpu().numpy(), scale)
    for x, w, out, n, dtype in (("codes", b.w_qkv, "qkv", N, BF16), ("codes", b.w_both, "both", N, BF16),
                                ("act", b.w_down, "down", FFN, F32)):
        ref, size = M.linear(values(o[x]), values(w), None)
        assert near(o[out], ref, size, n, dtype), out
    for x, w, out in (("q_in", b.q_weight, "q"), ("k_in", b.k_weight, "k")):
        ref, v = M.qk_norm_rope(host(o[x]), host(b.cos), host(b.sin), b.positions.cpu().numpy(), "rms", 1e-6, host(w),
                                None, False)
        # under 48 binary32 half-steps of both channels of a pair, and the result's half-step
        pair = np.abs(v) + np.concatenate((np.abs(v)[:, :, D // 2:], np.abs(v)[:, :, :D // 2]), axis=2)
        assert (np.abs(host(o[out]) - ref) <= 48 * U * pair + 2.0 ** -8 * np.abs(ref)).all(), out
    # the fused activation: what the separate steps give (its values rounded to bf16 before the rotation)
    gate, up = o["both"][:, :FFN], o["both"][:, FFN:]
    y = R.swiglu_rotate_quant_int4(gate, up, b.c, b.sigma, y_out=True)[-1]
    for got, ref in zip(o["act"], R.quant_mxfp4(y)):
        assert torch.equal(got, ref)


def test_the_rotation_cancels_through_the_product():
    """Rotated codes times folded weights are the unrotated product, but for the roundings to four bits: at most
    half the widest gap, one scale of the largest level 6, so 1/6 of a block's maximum for each value of either
    operand."""
    b = Block(40)
    o = b.run()
    gate, up = host(o["both"][:, :FFN]), host(o["both"][:, FFN:])
    x = (torch.from_numpy(gate / (1 + np.exp(-gate))) * torch.from_numpy(up)).to(BF16).double().numpy()
    ref = x @ host(b.plain).T
    act, w = values(o["act"]), values(b.w_down)
    # with e the errors of the four-bit values: (y + e_y) . (w + e_w) - y . w = e_y . w_q + y . e_w; each bounded by
    # its Euclidean sizes
    y = R.swiglu_rotate_quant_int4(o["both"][:, :FFN], o["both"][:, FFN:], b.c, b.sigma, y_out=True)[-1]
    row = torch.tensor([1 - 2 * (bin(b.c & j).count("1") & 1) for j in range(FFN)], dtype=torch.int8, device="cuda")
    fold = host(R.fold_weights(b.plain, b.sigma * row))
    bound = (np.linalg.norm(act - host(y), axis=1)[:, None] * np.linalg.norm(w, axis=1)[None, :] +
             np.linalg.norm(host(y), axis=1)[:, None] * np.linalg.norm(w - fold, axis=1)[None, :])
    # and binary32's: the rotation, the fold and the sum, each under 4 sqrt(n) u of the factors' sizes; the
    # activation's SiLU may round to the neighbouring bf16, 2^-8 of each x
    sizes = np.linalg.norm(x, axis=1)[:, None] * np.linalg.norm(host(b.plain), axis=1)[None, :]
    assert (np.abs(host(o["down"]) - ref) <= bound + (12 * FFN ** 0.5 * U + 2.0 ** -7) * sizes).all()


@pytest.mark.parametrize("t", [1, 40, 333])
def test_same_bits_from_a_graph_and_another_stream(t):
    b = Block(t)
    want = b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = b.run()

    def same(o, ref):
        for key in ("h", "u", "qkv", "q", "k", "down"):
            assert torch.equal(o[key], ref[key]), key
        for key in ("codes", "act"):
            assert torch.equal(o[key][0], ref[key][0]) and torch.equal(o[key][1], ref[key][1]), key

    same(other, want)
    for _ in range(3):
        held["down"].zero_()
        held["q"].zero_()
        g.replay()
        same(b.run(), want)
        torch.cuda.synchronize()
        same(held, want)
    b.h.copy_(b.h.flip(1))
    again = b.run()
    g.replay()
    torch.cuda.synchronize()
    same(held, again)
