"""A transformer block's MLP with 8-bit weights, from the attention's output to
the next block's normed input, in five launches (a few more at widths without
the fused SwiGLU):

    h', codes = residual_norm_quant_int8(h, attn)        residual sum, RMS norm, INT8 codes
    gate | up = int8_linear(codes, W_gate|up)            one product for both projections
    codes4    = swiglu_rotate_quant_int4(gate, up)       SiLU(gate) * up, rotation, INT4 codes
    y         = int4_w8_linear(codes4, W_down')          W_down' = W_down . H . D / sqrt(n)
    h'', u    = residual_norm(h', y)                     residual sum, the next block's norm

    python -m examples.quantized_mlp [--tokens T] [--hidden N] [--inner N]

prints the error against the same block in binary32 with unquantized weights,
and the time per pass.  The weights and activations are random, with one
massive channel at the down projection's input.
"""
import argparse
import math

import torch

import rotation_activation_quantization_amd as R


class QuantizedMLP:
    """Built once, offline: w_gate and w_up [inner, hidden] and w_down [hidden,
    inner] are bf16 on the GPU, x_cal bf16 [T, inner] are inputs of the down
    projection that the massive channel is calibrated on."""

    def __init__(self, w_gate, w_up, w_down, x_cal, norm_weight, next_norm_weight, eps=1e-6):
        self.inner = w_gate.shape[0]
        self.norm_weight, self.next_norm_weight, self.eps = norm_weight, next_norm_weight, eps
        self.w_in, self.w_in_scale = R.quant_int8(torch.cat((w_gate, w_up)))
        d, self.channel, _, peak = R.calibrate(x_cal)
        self.sigma = -1 if peak < 0 else 1
        self.fused = R.kernel_name(self.inner).startswith("rq_mfma")  # the widths of the fused SwiGLU
        folded = R.fold_weights(w_down, d).to(torch.bfloat16)
        self.w_out, self.w_out_scale, self.w_out_sum = R.quant_int8(folded, sums=True)

    def __call__(self, h, attn):
        """The residual stream h [T, hidden] (bf16 or float32) and the attention
        block's output attn (bf16) -> (the stream after this block, the next
        block's normed input in bf16)."""
        h, codes, scale = R.residual_norm_quant_int8(h, attn, eps=self.eps, post_norm="none", weight=self.norm_weight)
        both = R.int8_linear(codes, scale, self.w_in, self.w_in_scale)
        gate, up = both[:, :self.inner], both[:, self.inner:]
        if self.fused:
            codes, scale, zero = R.swiglu_rotate_quant_int4(gate, up, self.channel, self.sigma)
        else:
            x = (torch.nn.functional.silu(gate.float()) * up.float()).to(torch.bfloat16)
            codes, scale, zero = R.rotate_quant_int4_outlier(x, self.channel, self.sigma)
        y = R.int4_w8_linear(codes, scale, zero, self.w_out, self.w_out_scale, self.w_out_sum)
        return R.residual_norm(h, y, eps=self.eps, post_norm="none", weight=self.next_norm_weight)


def rms_norm(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + eps) * weight.float()


def plain(weights, norm_weight, next_norm_weight, h, attn, eps=1e-6):
    """The same block in binary32: (stream, normed, the MLP's branch)."""
    w_gate, w_up, w_down = (w.float() for w in weights)
    h = h.float() + attn.float()
    u = rms_norm(h, norm_weight, eps)
    x = torch.nn.functional.silu(u @ w_gate.T) * (u @ w_up.T)
    y = x @ w_down.T
    return h + y, rms_norm(h + y, next_norm_weight, eps), y


def make_block(hidden, inner, seed=0, device="cuda"):
    """Random weights (w_gate, w_up, w_down) and norm weights, calibration rows
    included: the projections keep unit variance; one channel of the inner
    activations is large on every token."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device)

    weights = [normal(inner, hidden) / math.sqrt(hidden), normal(inner, hidden) / math.sqrt(hidden),
               normal(hidden, inner) / math.sqrt(inner)]
    weights[0][inner // 3] *= 6.0
    weights[1][inner // 3] *= 6.0
    weights = [w.to(torch.bfloat16) for w in weights]
    norms = [(1.0 + 0.1 * normal(hidden)).to(torch.bfloat16) for _ in range(2)]
    u = normal(64, hidden)
    x_cal = torch.nn.functional.silu(u @ weights[0].float().T) * (u @ weights[1].float().T)
    return weights, norms, x_cal.to(torch.bfloat16)


def make_tokens(tokens, hidden, seed=1, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    return [torch.randn((tokens, hidden), generator=gen, device=device).to(torch.bfloat16) for _ in range(2)]


def relative(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--passes", type=int, default=20)
    args = ap.parse_args()
    if not R.supported_n(args.inner):
        ap.error(f"no rotation of order {args.inner}")
    weights, norms, x_cal = make_block(args.hidden, args.inner)
    mlp = QuantizedMLP(*weights, x_cal, *norms)
    h, attn = make_tokens(args.tokens, args.hidden)
    stream, normed = mlp(h, attn)
    want_stream, want_normed, _ = plain(weights, *norms, h, attn)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(args.passes):
        mlp(h, attn)
    end.record()
    torch.cuda.synchronize()
    print(f"{args.tokens} tokens, {args.hidden} x {args.inner}: relative error of the stream "
          f"{relative(stream, want_stream):.4f}, of the next block's input {relative(normed, want_normed):.4f}; "
          f"{1000 * start.elapsed_time(end) / args.passes:.1f} us per pass")


if __name__ == "__main__":
    main()
