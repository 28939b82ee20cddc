"""Registers of the kernels of the 8-bit products, the INT8 quantizer and the
residual norm, from the compiler's kernel-resource-usage remarks
(build.resource_report): a spill in a loop turns into scratch traffic there,
with waits that also wait for the ring's loads.

Two kinds of instance may keep a few words in scratch, outside of the tile's
main loop: the 256 x 256 tile of the packed codes, and the norm with four
chunks of a row to a thread, whose row fills the registers."""
import pytest

from rotation_activation_quantization_amd import build as B

TILE_256_A4 = "w8_tile_kernelILb1ELi2ELi4ELi8ELi4ELi1ELi4ELb0E"
WIDE_NORM = "residual_norm_rows_kernelILi4E"


@pytest.fixture(scope="module")
def report():
    return B.resource_report(["linear_w8.hip", "quant_int8.hip", "residual_norm.hip"])


@pytest.mark.parametrize("kernel,instances", [
    ("w8_tile_kernel", 20), ("w8_join_kernel", 10), ("w8_few_kernel", 8), ("w8_few_any_kernel", 8),
    ("w8_any_kernel", 4), ("w8_pack_kernel", 1), ("quant_int8_rows_kernel", 8), ("quant_int8_any_kernel", 1),
    ("residual_norm_rows_kernel", 12), ("residual_norm_any_kernel", 1)])
def test_instances_do_not_spill(report, kernel, instances):
    hits = {name: r for name, r in report.items() if kernel in name}
    assert len(hits) == instances, sorted(hits)
    for name, r in hits.items():
        limit = 32 if TILE_256_A4 in name else 96 if WIDE_NORM in name else 0
        assert r["scratch"] <= limit, (name, r)


def test_tiles_and_norms_keep_their_waves(report):
    # 256 registers: two waves on a SIMD, the 256 x 256 tile's eight on a CU; rows
    # in up to 128: a work-group of sixteen waves on a CU
    for name, r in report.items():
        total = r["vgprs"] + r["agprs"]
        assert total <= (128 if "rows_kernel" in name else 256), (name, r)
