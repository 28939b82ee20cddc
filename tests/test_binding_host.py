"""What the binding checks and hands to the library, with stand-ins for GPU
tensors (no GPU needed): operands on the wrong device are refused before any
call of the library."""

import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402


def test_operands_in_host_memory_are_refused_with_a_value_error():
    codes = torch.zeros((2, 32), dtype=torch.uint8)
    f = torch.ones(2)
    w = torch.zeros((8, 64), dtype=torch.int8)
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: R.dequant(codes, f, f), lambda: R.quant_int8(x),
                 lambda: R.int8_linear(codes.view(torch.int8), f, w[:, :32], torch.ones(8)),
                 lambda: R.int4_w8_linear(codes, f, f, w, torch.ones(8), torch.zeros(8, dtype=torch.int32)),
                 lambda: R.residual_norm(x), lambda: R.rotate_quant_int4_outlier(x, 0, 1)):
        with pytest.raises(ValueError):
            call()


class GpuTensor:
    """What the binding asks of a tensor in GPU memory; nothing reads its pointer."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, step=None, gpu=0):
        self.shape, self.dtype, self.gpu = torch.Size(shape), dtype, gpu
        self.device = torch.device("cuda", gpu)
        self.step = step

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = (1,) if self.dim() == 1 else (self.shape[1] if self.step is None else self.step, 1)
        return s if i is None else s[i]

    def is_contiguous(self):
        return self.step is None

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return 0x100000


class Recorder:
    """Stands in for the library and the current device: notes the calls, all of
    which succeed, and the device each was made on."""

    def __init__(self):
        self.calls, self.devices, self.current = [], [], 0

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace"):
                return 0
            self.calls.append((name, args))
            self.devices.append(self.current)
            return 0
        return call

    def device(self, index):
        recorder = self

        class Use:
            def __enter__(self):
                self.before, recorder.current = recorder.current, index

            def __exit__(self, *_):
                recorder.current = self.before

        return Use()


@pytest.fixture
def library(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(R, "_lib", recorder)
    monkeypatch.setattr(R, "_raw_stream", lambda index: 0x5000 + index)
    monkeypatch.setattr(R, "_current_device", lambda: recorder.current)
    monkeypatch.setattr(torch.cuda, "device", recorder.device)
    return recorder


def norm_args(call):
    (name, (packed, _)), = call.calls
    assert name == "signrot_residual_norm"
    return R._ResidualNormArgs.from_buffer_copy(packed)


def norm(tokens=4, n=64, **kw):
    h = GpuTensor(tokens, n)
    return R.residual_norm(h, h, h_out=GpuTensor(tokens, n), out=GpuTensor(tokens, n), **kw)


def test_modulations_of_different_row_counts_are_refused(library):
    """An index that is valid for the longer one would be clamped to the shorter."""
    index = GpuTensor(4, dtype=torch.int32)
    for a, b in (("gate", "mod_scale"), ("gate", "mod_shift"), ("mod_scale", "mod_shift")):
        with pytest.raises(ValueError):
            norm(mod_index=index, **{a: GpuTensor(3, 64), b: GpuTensor(2, 64)})
        with pytest.raises(ValueError):
            norm(mod_index=index, **{a: GpuTensor(1, 64), b: GpuTensor(2, 64)})
    assert not library.calls
    norm(mod_index=index, gate=GpuTensor(64), mod_scale=GpuTensor(3, 64), mod_shift=GpuTensor(3, 64))
    a = norm_args(library)
    assert (a.ldg, a.ldm, a.mod_rows) == (0, 64, 3)


def test_without_an_index_more_modulation_rows_than_tokens_are_taken(library):
    norm(gate=GpuTensor(6, 64), mod_scale=GpuTensor(5, 64))
    a = norm_args(library)
    assert (a.ldg, a.ldm, a.mod_rows) == (64, 64, 5)


@pytest.mark.parametrize("tokens,index", [(1, False), (1, True), (4, True)])
def test_the_stride_of_a_single_modulation_row_does_not_matter(library, tokens, index):
    """One row cut from a wider projection beside a contiguous one."""
    kw = {"mod_index": GpuTensor(tokens, dtype=torch.int32)} if index else {}
    norm(tokens, gate=GpuTensor(1, 64, step=384), mod_scale=GpuTensor(1, 64), mod_shift=GpuTensor(1, 64, step=384), **kw)
    a = norm_args(library)
    assert (a.ldg, a.ldm) == (0, 0) and a.gate and a.mod_scale and a.mod_shift


def test_one_token_takes_the_first_row_of_any_modulations(library):
    norm(1, gate=GpuTensor(3, 64), mod_scale=GpuTensor(1, 64), mod_shift=GpuTensor(2, 64, step=128))
    a = norm_args(library)
    assert (a.ldg, a.ldm) == (0, 0) and a.gate and a.mod_scale and a.mod_shift


def on(gpu, *shape, dtype=torch.float32):
    return GpuTensor(*shape, dtype=dtype, gpu=gpu)


CALLS = {
    "signrot_quant_int8": lambda g: R.quant_int8(
        on(g, 4, 64, dtype=torch.bfloat16), out=(on(g, 4, 64, dtype=torch.int8), on(g, 4))),
    "signrot_int8_linear": lambda g: R.int8_linear(
        on(g, 4, 64, dtype=torch.int8), on(g, 4), on(g, 8, 64, dtype=torch.int8), on(g, 8), out=on(g, 4, 8)),
    "signrot_int4_w8_linear": lambda g: R.int4_w8_linear(
        on(g, 4, 32, dtype=torch.uint8), on(g, 4), on(g, 4), on(g, 8, 64, dtype=torch.int8), on(g, 8),
        on(g, 8, dtype=torch.int32), out=on(g, 4, 8)),
    "signrot_residual_norm": lambda g: R.residual_norm(
        on(g, 4, 64), h_out=on(g, 4, 64), out=on(g, 4, 64, dtype=torch.bfloat16)),
    "signrot_rotate_quant_int4": lambda g: R.rotate_quant_int4(
        on(g, 4, 64, dtype=torch.bfloat16), on(g, 64, dtype=torch.int8),
        out=(on(g, 4, 32, dtype=torch.uint8), on(g, 4), on(g, 4))),
    "signrot_rotate_quant_int4_outlier": lambda g: R.rotate_quant_int4_outlier(
        on(g, 4, 64, dtype=torch.bfloat16), 0, 1, out=(on(g, 4, 32, dtype=torch.uint8), on(g, 4), on(g, 4))),
    "signrot_int4_linear": lambda g: R.int4_linear(
        on(g, 4, 32, dtype=torch.uint8), on(g, 4), on(g, 4), on(g, 8, 64, dtype=torch.bfloat16), on(g, 8),
        out=on(g, 4, 8)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_runs_on_the_gpu_of_its_tensors(library, name):
    """Also when another is the current one, which is the same again afterwards."""
    for gpu, current in ((0, 0), (1, 0), (0, 1), (1, 1)):
        library.current = current
        CALLS[name](gpu)
        assert library.calls[-1][0] == name and library.calls[-1][1][-1] == 0x5000 + gpu
        assert library.devices[-1] == gpu and library.current == current
    assert len(library.calls) == 4
