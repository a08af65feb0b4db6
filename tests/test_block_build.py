"""Build-level check of the operators around the scan (no GPU needed): none of their kernels spills
registers or uses scratch memory. They keep states, decays and windows in registers across their
loops, and a spill there costs more than most changes gain."""

import os

import pytest

from test_build import BUILD, _kernel_descriptors


@pytest.mark.parametrize("source", ["ssd_conv", "ssd_selective", "ssd_selective_backward", "ssd_norm",
                                    "ssd_sums"])
def test_block_kernels_use_no_scratch(source):
    kernels = _kernel_descriptors(os.path.join(BUILD, source + ".o"))
    assert kernels, source
    bad = {k: v for k, v in kernels.items()
           if v.get("private_segment_fixed_size", 0) or v.get("vgpr_spill_count", 0)}
    assert not bad, f"{source} kernels spilling to scratch: {bad}"
