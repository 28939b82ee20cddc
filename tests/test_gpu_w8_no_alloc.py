"""The 8-bit products, the INT8 quantizer and the residual norms allocate no device
memory of their own, and none of them waits for the GPU's work."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402

pytestmark = pytest.mark.gpu


def bf16(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def whole(dtype, *shape):
    return torch.randint(0, 100, shape, device="cuda").to(dtype)


def calls():
    """(name, the library's call on buffers that are there) of every kernel kind."""
    L = R.lib()
    stream = torch.cuda.current_stream().cuda_stream
    keep = []

    def ptr(v):
        keep.append(v)
        return v.data_ptr()

    out = []
    for t, n in ((3, 5), (3, 4096), (4, 1111), (2, 70000)):
        args = (ptr(bf16(t, n)), t, n, n, ptr(whole(torch.int8, t, n)), n, ptr(torch.empty(t, device="cuda")),
                ptr(torch.empty(t, dtype=torch.int32, device="cuda")), stream)
        out.append((f"quant_int8 {t} x {n}", lambda args=args: L.signrot_quant_int8(*args)))
        a = R._ResidualNormArgs(tokens=t, n=n, h=ptr(bf16(t, n)), ldh=n, y=ptr(bf16(t, n)), ldy=n, h_out=ptr(bf16(t, n)),
                                ldho=n, u=ptr(bf16(t, n)), ldu=n, alpha=1.0, beta=1.0, eps_post=1e-6, eps_pre=1e-6,
                                post_norm=1, pre_norm=2, h_type=1, param_type=1)
        keep.append(a)
        out.append((f"residual_norm {t} x {n}", lambda a=a: L.signrot_residual_norm(ctypes.addressof(a), stream)))
    # few tokens, tiles, a split row, rows laid out anew, short rows
    for t, n, rows in ((1, 4096, 512), (2, 4098, 512), (512, 4096, 4096), (33, 4128, 77), (2100, 2046, 2304), (200, 14, 300)):
        f = [ptr(torch.rand(k, device="cuda")) for k in (t, t, rows, rows)]
        w, o = ptr(whole(torch.int8, rows, n)), ptr(torch.empty(t, rows, device="cuda"))
        c8, c4 = ptr(whole(torch.int8, t, n)), ptr(whole(torch.uint8, t, n // 2))
        total = ptr(whole(torch.int32, rows))
        for name, size in (("int8_linear", L.signrot_int8_linear_workspace(c8, n, t, n, w, n, rows)),
                           ("int4_w8_linear", L.signrot_int4_w8_linear_workspace(c4, t, n, w, n, rows))):
            space = ptr(torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")) if size else None
            if name == "int8_linear":
                args = (c8, n, f[0], t, n, w, n, f[2], f[3], rows, o, rows, 0, space, size, stream)
            else:
                args = (c4, f[0], f[1], t, n, w, n, f[2], total, f[3], rows, o, rows, 0, space, size, stream)
            out.append((f"{name} {t} x {n} x {rows}", lambda f=getattr(L, "signrot_" + name), args=args: f(*args)))
    return out, keep


def test_calls_leave_the_free_memory_as_it_is():
    todo, _keep = calls()
    for _, call in todo:  # loads the kernels' code
        assert call() == R.SIGNROT_OK
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for name, call in todo:
        print(f"[gpu] {name}", flush=True)
        for _ in range(20):
            assert call() == R.SIGNROT_OK
        assert torch.cuda.mem_get_info()[0] == free, name
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free


def test_calls_can_be_captured():
    """A capture refuses allocations, copies to the host and waits."""
    todo, _keep = calls()
    for _, call in todo:
        assert call() == R.SIGNROT_OK
    torch.cuda.synchronize()
    del todo, _keep
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        todo, _keep = calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            results = [call() for _, call in todo]
    assert results == [R.SIGNROT_OK] * len(todo)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
