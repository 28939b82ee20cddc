"""The MXFP4 operators and the per-head norms allocate no device memory of their own, and
none of them waits for the GPU's work; their results past 64 MiB, which skip the caches,
are those of small calls."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def calls():
    """(name, the library's call on buffers that are there) of every kernel kind."""
    L = R.lib()
    stream = torch.cuda.current_stream().cuda_stream
    keep = []

    def ptr(v):
        keep.append(v)
        return v.data_ptr()

    def some(*shape):
        return torch.randn(shape, device="cuda").to(BF16)

    def codes(*shape):
        return torch.randint(100, 130, shape, dtype=torch.uint8, device="cuda")

    out = []
    for t, n in ((3, 5), (3, 4096), (4, 1111), (2, 70000)):
        nb = (n + 31) // 32
        q, s = ptr(codes(t, 16 * nb)), ptr(codes(t, nb))
        quant = (ptr(some(t, n)), 1, t, n, n, 0, q, 16 * nb, s, nb, stream)
        back = (q, 16 * nb, s, nb, t, n, ptr(some(t, n)), 1, n, stream)
        out.append((f"quant {t} x {n}", lambda a=quant: L.signrot_quant_mxfp4(*a)))
        out.append((f"dequant {t} x {n}", lambda a=back: L.signrot_dequant_mxfp4(*a)))
    # few tokens, each kind of tile, split rows, operands laid out anew
    for t, n, rows, odd in ((1, 4096, 512, 0), (29, 544, 77, 0), (33, 8224, 40, 0), (300, 1024, 2100, 0), (70, 160, 8200, 0),
                            (65, 14336, 2100, 0), (257, 32, 14340, 0), (200, 14336, 8200, 0), (777, 1056, 14340, 0),
                            (1030, 8224, 4096, 0), (5, 96, 40, 1), (70, 160, 200, 1), (777, 1056, 14340, 1)):
        nb = n // 32
        a = (ptr(codes(t, 16 * nb + odd)), 16 * nb + odd, ptr(codes(t, nb + odd)), nb + odd, t, n,
             ptr(codes(rows, 16 * nb + odd)), 16 * nb + odd, ptr(codes(rows, nb + odd)), nb + odd)
        size = L.signrot_mxfp4_linear_workspace(*a, rows)
        space = ptr(torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")) if size else None
        args = (*a, ptr(torch.rand(rows, device="cuda")), rows, ptr(torch.empty(t, rows, device="cuda")), rows, 0, space,
                size, stream)
        out.append((f"linear {t} x {n} x {rows} {odd}", lambda a=args: L.signrot_mxfp4_linear(*a)))
    for t, n in ((9, 4096), (9, 14336), (9, 28672), (9, 13824), (9, 640), (9, 224), (9, 16)):
        nb = (n + 31) // 32
        size = L.signrot_rotate_quant_mxfp4_workspace(t, n)
        space = ptr(torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")) if size else None
        args = (ptr(some(t, n)), t, n, n, n // 3, 1, 0, ptr(codes(t, 16 * nb)), 16 * nb, ptr(codes(t, nb)), nb, space, size,
                stream)
        out.append((f"rotate {t} x {n}", lambda a=args: L.signrot_rotate_quant_mxfp4(*a)))
    for t, n in ((9, 4096), (9, 14336), (9, 28672)):
        args = (ptr(some(t, n)), ptr(some(t, n)), t, n, n, n // 3, 1, 0, ptr(codes(t, n // 2)), n // 2, ptr(codes(t, n // 32)),
                n // 32, stream)
        out.append((f"swiglu {t} x {n}", lambda a=args: L.signrot_swiglu_rotate_quant_mxfp4(*a)))
    for t, heads, d in ((1, 8, 128), (9, 4, 80), (5, 3, 36), (3, 2, 512)):
        a = R._QkNormRopeArgs(tokens=t, head=d, rotary=d, q=ptr(some(t, heads, d)), ldq=heads * d, hsq=d,
                              q_out=ptr(some(t, heads, d)), ldqo=heads * d, hsqo=d, cos=ptr(torch.rand(64, d // 2, device="cuda")),
                              sin=ptr(torch.rand(64, d // 2, device="cuda")), ldt=d // 2, places=64, q_heads=heads, k_heads=0,
                              eps=1e-6, norm=1, in_type=1, out_type=1, param_type=1)
        keep.append(a)
        out.append((f"heads {t} x {heads} x {d}", lambda a=a: L.signrot_qk_norm_rope(ctypes.addressof(a), stream)))
    return out, keep


def test_calls_leave_the_free_memory_as_it_is():
    todo, _keep = calls()
    for name, call in todo:  # loads the kernels' code
        print(f"[gpu] {name}", flush=True)
        assert call() == R.SIGNROT_OK, name
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for name, call in todo:
        for _ in range(20):
            assert call() == R.SIGNROT_OK
        assert torch.cuda.mem_get_info()[0] == free, name
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free


def test_calls_do_not_wait_for_the_gpu():
    """Many calls are queued behind work of some milliseconds before it is done."""
    todo, _keep = calls()
    for _, call in todo:
        assert call() == R.SIGNROT_OK
    torch.cuda.synchronize()
    a = torch.randn(8192, 8192, device="cuda")
    b = torch.empty_like(a)
    torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    for name, call in todo:
        done = torch.cuda.Event()
        torch.mm(a, a, out=b)
        torch.mm(a, a, out=b)
        done.record()
        assert call() == R.SIGNROT_OK
        assert not done.query(), name
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [4224, 4223])
def test_large_dequantized_results(n):
    x = torch.randn(8200, n, device="cuda").to(BF16)
    codes, scale = R.quant_mxfp4(x)
    large = R.dequant_mxfp4(codes, scale, n=n, dtype=BF16)
    assert 2 * large.numel() > 64 << 20
    wide = R.dequant_mxfp4(codes, scale, n=n)
    assert torch.equal(large.float(), wide)  # both are exact
    for a in range(0, 8200, 4100):
        assert torch.equal(R.dequant_mxfp4(codes[a:a + 4100], scale[a:a + 4100], n=n, dtype=BF16), large[a:a + 4100])


@pytest.mark.parametrize("t,hq,hk,d", [(8200, 32, 2, 128), (8200, 40, 13, 80), (9000, 30, 1, 126)])
def test_large_normed_heads(t, hq, hk, d):
    q, k = (torch.randn(t, h, d, device="cuda").to(BF16) for h in (hq, hk))
    angle = torch.rand(t, d // 2, device="cuda") * 6
    cos, sin = angle.cos(), angle.sin()
    large = R.qk_norm_rope(q, k, cos, sin)
    assert 2 * (q.numel() + k.numel()) > 64 << 20
    for a in range(0, t, 3000):
        b = min(a + 3000, t)
        part = R.qk_norm_rope(q[a:b], k[a:b], cos[a:b], sin[a:b])
        assert torch.equal(part[0], large[0][a:b]) and torch.equal(part[1], large[1][a:b])
    R.qk_norm_rope(q, k, cos, sin, q_out=q, k_out=k)
    assert torch.equal(q, large[0]) and torch.equal(k, large[1])
