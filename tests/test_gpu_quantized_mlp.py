"""The quantized MLP example against the unquantized block in binary32.

The branch's error is that of its INT4 activations; 8-bit weights and
activations (about 1 % each) and bf16 intermediates add little.  A rotated row
is close to bell-shaped with deviation s (the massive channel only moves its
mean, which the zero-point takes up), so its n values span about 2 m s, with m
the expected largest of n normal deviates, and sixteen levels leave an error of
2 m s / (15 sqrt 12) a value:

    n = 1024: m = 3.23, 0.125 s        n = 3584: m = 3.55, 0.137 s

and 0.16 s on the rare row with m = 4.2.  The down projection keeps the ratio,
and the massive channel only adds to the branch's own size.  The INT8 codes'
error passes through SiLU(gate) up with a gain of at most two, 4 %: sqrt(0.16^2
+ 0.04^2) < 0.17, taken as 0.2.  The stream's error is that times the branch's
share of it, and half a unit of bf16 (2^-8).
"""
import pytest

torch = pytest.importorskip("torch")

from examples import quantized_mlp as E  # noqa: E402

pytestmark = pytest.mark.gpu

BOUND = 0.2


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 256, 1024), (33, 256, 1024), (150, 512, 3584), (300, 1000, 3584)])
@pytest.mark.parametrize("stream_type", [torch.bfloat16, torch.float32])
def test_block_is_close_to_the_unquantized_one(tokens, hidden, inner, stream_type):
    weights, norms, x_cal = E.make_block(hidden, inner)
    mlp = E.QuantizedMLP(*weights, x_cal, *norms)
    assert mlp.channel == inner // 3
    h, attn = E.make_tokens(tokens, hidden)
    h = h.to(stream_type)
    before = h.clone()
    stream, normed = mlp(h, attn)
    assert torch.equal(h, before)
    assert stream.dtype is stream_type and normed.dtype is torch.bfloat16
    want_stream, want_normed, branch = E.plain(weights, *norms, h, attn)
    share = float(branch.norm() / want_stream.norm())
    assert E.relative(stream, want_stream) <= BOUND * share + 2.0 ** -8
    # the next norm divides by the row's size, which moves by no more than the error itself
    assert E.relative(normed, want_normed) <= 2 * (BOUND * share + 2.0 ** -8)


def test_a_pass_replays_in_a_graph():
    weights, norms, x_cal = E.make_block(256, 1024)
    mlp = E.QuantizedMLP(*weights, x_cal, *norms)
    h, attn = E.make_tokens(5, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mlp(h, attn)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream, normed = mlp(h, attn)
    for seed in range(2, 6):
        new_h, new_attn = E.make_tokens(5, 256, seed)
        h.copy_(new_h)
        attn.copy_(new_attn)
        graph.replay()
        torch.cuda.synchronize()
        want_stream, want_normed = mlp(new_h, new_attn)
        torch.cuda.synchronize()
        assert torch.equal(stream, want_stream) and torch.equal(normed, want_normed)
