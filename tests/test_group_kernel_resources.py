"""Scratch and registers of the built kernels of the group-scaled operators, as
test_kernel_resources.py reads them: none may spill."""
import os

import pytest

import test_kernel_resources as R


@pytest.mark.parametrize("source,kernels", [
    ("w4", ("w4_few_kernel", "w4_tile_kernel", "w4_prepack_kernel")),
    ("wgrad", ("wgrad_kernel", "wgrad_ring_kernel", "wgrad_join_kernel")),
    ("group_quant", ("quantize_groups_kernel", "quantize_rows_kernel", "dequantize_groups_kernel", "act_fwd_groups_kernel",
                     "act_fwd_rows_kernel", "act_bwd_kernel")),
])
def test_no_group_kernel_uses_scratch(monkeypatch, source, kernels):
    monkeypatch.setattr(R, "OBJ", os.path.join(os.path.dirname(R.OBJ), source + ".o"))
    meta = R._kernel_metadata()
    for k in kernels:
        assert any(k in name for name, _, _ in meta), k
    assert not [(name, p) for name, p, _ in meta if p > 0]
    assert all(v <= 512 for _, _, v in meta)
