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


# Chunks of prompts on tiles (results written directly, and joined), the same with a prefix folded in and with a pass
# of its own for it, single tokens on the split-key kernel; rows that see one key or none.
QUERIES = [
    ([100, 90, 3], [100, 90, 5], 0), ([2500, 100], [100, 100], 0), ([200, 64], [70, 64], 300),
    ([20 + i for i in range(70)], [1 + i % 11 for i in range(70)], 2304), ([70, 1, 0], [1, 1, 1], 0), ([70, 1], [1, 1], 700),
]


@pytest.mark.parametrize("d,int8", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("lens,new,prefix", QUERIES)
def test_queries_that_are_not_finite(lens, new, prefix, d, int8):
    """A NaN or an infinity in a query makes that row NaN (or leaves it 0 where it sees nothing), whichever kernel takes
    it; other rows are what they were."""
    hq, hkv, page = 8, 2, 64
    g = base.gen(62)
    table, shared, total = base.make_table(62, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, hkv, d, int8)
    T = sum(new)
    q = base.randn(g, T, hq, d, scale=2.0)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new))
    want, tol = ref.attention(q, base.values(kv), table.cpu(), lens, new, [] if shared is None else shared.cpu().tolist(),
                              prefix)
    seen = torch.cat([prefix + (torch.arange(n) + 1 + lk - n).clamp(min=0) for lk, n in zip(lens, new)])
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = torch.zeros(T, hq, dtype=torch.bool)
        for i, t in enumerate(sorted({0, 1, T // 2, T - 5, T - 1})):
            if 0 <= t < T:
                bad[t, (3 * i) % hq] = True
        broken = q.clone()
        broken[bad.cuda(), torch.arange(int(bad.sum()), device="cuda") * 7 % d] = value
        got = ops.attn_shared_prefix(broken, kv, table, base.i32(lens), **args).cpu()
        base.ok()
        nothing = (seen == 0)[:, None].expand_as(bad)
        assert bool(got[bad & ~nothing].isnan().all())
        assert bool((got[nothing] == 0).all())
        base.within(got[~bad], want[~bad], tol[~bad])
