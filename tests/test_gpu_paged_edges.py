"""Paged-cache serving operators on the GPU at the edges of their contract, against their 64-bit forms."""

import pytest
import torch

import paged_ref as ref
import test_gpu_paged as base

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixed_precision_attention_tm_b200 import ops


@pytest.mark.parametrize("d,int8", [(128, False), (128, True), (64, False), (64, True)])
def test_several_segments_of_a_tile_block(d, int8):
    """More items of own tokens than SMs, whose row blocks fill one query tile or both and end at different keys, and
    pieces of the prefix's line that cross row blocks: each block of the tile kernel goes through several segments."""
    new = [33 + i % 32 for i in range(40)]
    lens = [n + (i * 37) % 400 for i, n in enumerate(new)]
    base.attend(60, lens, new, 0, d, 64, 32, 4, int8)
    base.attend(61, [900, 690, 3], [900, 690, 1], 2700, d, 64, 16, 16, int8, causal=False)
