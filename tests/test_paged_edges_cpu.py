"""CPU checks of the paged-cache operators at the edges of their contract."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "mixed_precision_attention_tm_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_tile_kernel_warpgroups_change_registers_together():
    """setmaxnreg has to be the same instruction for all four warps of a warpgroup: one for the control warps (8 to 11),
    under a condition that they agree on, and before their roles part."""
    text = source("tm_attn_shared_tile.cu")
    assert len(re.findall(r"regs_dec<C::CONTROL_REGS>\(\)", text)) == 1
    assert re.search(r"if \(warp >= 8 && warp < 12\) \{\n(\s*//[^\n]*\n)*\s*regs_dec<C::CONTROL_REGS>\(\);\n\s*if \(warp == 8\)", text)
    assert len(re.findall(r"regs_(?:dec|inc)<", text)) == 3
