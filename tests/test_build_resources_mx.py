"""The MXFP4 and per-head norm kernels compile without scratch: a spill would put
vmcnt waits, which also wait for loads and stores on their way, into their loops."""

import pytest

from rotation_activation_quantization_amd import build as B

SOURCES = ["linear_mx.hip", "quant_mx.hip", "qk_norm_rope.hip", "rq_mx.hip"]


@pytest.fixture(scope="module")
def report():
    return B.resource_report(SOURCES)


def test_no_scratch(report):
    assert not {name: r for name, r in report.items() if r["scratch"]}


def test_registers_leave_room_for_the_planned_waves(report):
    """512 registers of a SIMD over the waves that a CU is meant to hold."""
    def of(part):
        hits = [r["vgprs"] + r["agprs"] for name, r in report.items() if part in name]
        assert hits, part
        return max(hits)

    for tile, most in (("mx_tile_kernelILi4ELi2ELi4ELi8ELi2E", 256), ("mx_tile_kernelILi2ELi2ELi4ELi4ELi4E", 512),
                       ("mx_tile_kernelILi2ELi2ELi4ELi4ELi2E", 256), ("mx_tile_kernelILi2ELi2ELi4ELi2ELi4E", 512),
                       ("mx_tile_kernelILi1ELi4ELi4ELi1ELi4E", 256), ("mx_few_kernel", 128), ("qk_norm_rope_kernel", 85),
                       ("quant_mx_kernel", 64), ("rq_fast_kernel", 128), ("rq_halves_kernel", 128)):
        assert of(tile) <= most, tile


def test_every_mxfp4_rotation_is_there(report):
    # six widths with and without the producer, and n = 28672 in two halves
    assert sum("rq_fast_kernel" in name for name in report) == 12
    assert sum("rq_halves_kernel" in name for name in report) == 2
