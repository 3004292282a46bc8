"""Paged-cache serving operators on the GPU at the edges of their contract, against their 64-bit forms."""

import math

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


# As QUERIES: tiles written directly, joined, with the prefix folded in, with a pass for it; split-key kernel, one piece and several.
PATHS = [
    ([100, 90], [100, 90], 0), ([2500, 100], [100, 100], 0), ([200, 64], [70, 64], 300),
    ([20 + i for i in range(70)], [1 + i % 11 for i in range(70)], 2304), ([70, 200], [1, 2], 0), ([70, 2000], [1, 1], 700),
]


def fill_keys(kv, keys):
    """Sets a pool's keys (one fp16 row for each slot, heads alike), quantised where its pages are INT8."""
    k = keys[:, :, None].expand(*keys.shape[:2], kv.H, kv.d)
    if kv.int8:
        codes, scales = ref.quantise(k.cpu().double())
        kv.k.copy_(codes), kv.k_scales.copy_(scales)
    else:
        kv.k.copy_(k)


@pytest.mark.parametrize("d,int8", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("size", [2.0 ** 5, 2.0 ** 12, 2.0 ** 15])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_scores_up_to_the_end_of_fp16(lens, new, prefix, size, d, int8):
    """Queries and keys up to the largest fp16 numbers, scores up to 2^36: of levels 2^-3 apart and more the highest one
    that a row sees takes all, so the result is the mean of its values."""
    hq, hkv, page = 4, 2, 64
    g = base.gen(63)
    table, shared, total = base.make_table(63, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, hkv, d, int8)
    level = torch.randint(-8, 9, (total, page, 1), generator=g, device="cuda").float() / 8
    fill_keys(kv, (level * size).half().expand(total, page, d))
    q = torch.full((sum(new), hq, d), size, dtype=torch.float16, device="cuda")
    q[::3] *= 1.5                                # 49152 at the most
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new))
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args)
    base.ok()
    k, v = base.values(kv)
    # The sums are exact or off by 2^-17 of themselves, the levels 2^-3: only the highest counts (2^5: 2^10 sqrt(d) / 8 powers
    # of two and more between levels).  Its equal weights are rounded once each, INT8's with the V scale, and summed.
    pages = [] if shared is None else shared.cpu().tolist()
    want, _ = ref.attention(q, (k, v), table.cpu(), lens, new, pages, prefix)
    size_of, _ = ref.attention(q, (k, v.abs()), table.cpu(), lens, new, pages, prefix)
    tol = size_of * (2 * ref.HALF + (prefix + max(lens)) * 2.0 ** -24 + 2.0 ** -16) + ref.TINY
    if not int8 or PATHS.index((lens, new, prefix)) < 3:
        base.within(got, want, tol)
        return
    # The split-key kernel rounds t = score + log2(V scale) to fp32 once and divides a weight 2^t by the scale again in
    # the row's sum: equal scores of 2^13 and more get weights that differ by up to 2^(step of t), the same in both
    # sums.  The result is some mean of the same values: between the least and the largest of them.
    got, t0 = got.cpu().double(), 0
    for b, n in enumerate(new):
        kb, vb = (torch.cat((ref.rows_of(x, pages, prefix), ref.rows_of(x, table[b].cpu(), lens[b]))) for x in (k, v))
        for i in range(n):
            end = prefix + lens[b] - n + i + 1
            best = kb[:end, 0, 0] == kb[:end, 0, 0].max()
            top = vb[:end][best].repeat_interleave(hq // hkv, 1)
            slack = tol[t0 + i] + top.abs().amax(0) * 2 * ref.HALF
            assert bool(((got[t0 + i] <= top.amax(0) + slack) & (got[t0 + i] >= top.amin(0) - slack)).all())
        t0 += n


@pytest.mark.parametrize("d,int8", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_near_scores_far_from_zero_stay_weights(lens, new, prefix, d, int8):
    """Scores a few units apart at 2^22 and further on, where a unit is below fp32's step: whatever their rounding, a
    result is a mean of the values that a row sees."""
    hq, hkv, page = 4, 2, 64
    g = base.gen(64)
    table, shared, total = base.make_table(64, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, hkv, d, int8)
    keys = torch.zeros(total, page, d, device="cuda")
    q = torch.zeros(sum(new), hq, d, dtype=torch.float16, device="cuda")
    # a large product that all keys share, and small ones: 2^21 .. 2^33 in all, 16 apart
    keys[..., 0], q[..., 0] = 2.0 ** 12, (2.0 ** torch.arange(9, 16, device="cuda")).half()[torch.arange(sum(new)) % 7, None]
    keys[..., 1], q[..., 1] = torch.randint(0, 64, (total, page), generator=g, device="cuda").float() * 64, 1.0 / 4
    keys[..., 2:6], q[..., 2:6] = 2.0 ** 13, (2.0 ** torch.arange(9, 16, device="cuda")).half()[torch.arange(sum(new)) % 7, None, None]
    fill_keys(kv, keys.half())
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new))
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args).cpu()
    base.ok()
    v = base.values(kv)[1]
    t0 = 0
    for b, n in enumerate(new):
        vb = torch.cat((ref.rows_of(v, [] if shared is None else shared.cpu(), prefix), ref.rows_of(v, table[b].cpu(), lens[b])))
        vb = vb.repeat_interleave(hq // hkv, 1)
        slack = vb.abs().amax(0) * (3 * ref.HALF)      # the weights' roundings against their sum, and the result's
        assert bool(((got[t0:t0 + n] <= vb.amax(0) + slack) & (got[t0:t0 + n] >= vb.amin(0) - slack)).all())
        t0 += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_int8_scales_of_every_size(lens, new, prefix, causal, d):
    """Codes of the whole range -128 .. 127 under scales from 0 and fp16's smallest to its largest, V's values far past
    fp16's among them (each of little weight, some hidden from most rows): results as the values say."""
    hq, hkv, page = 4, 2, 64
    g = base.gen(65)
    table, shared, total = base.make_table(65, lens, page, extra=prefix)

    def codes():
        return torch.randint(-128, 128, (total, page, hkv, d), generator=g, device="cuda", dtype=torch.int8)

    def scales(lo, hi):
        return (2.0 ** (torch.rand(total, page, hkv, generator=g, device="cuda") * (hi - lo) + lo)).half()
    k, ks, v, vs = codes(), scales(-24, -7), codes(), scales(-24, 4)
    large = torch.rand(total, page, hkv, generator=g, device="cuda") < 1 / 16
    large[table[:, 0].long().clamp(min=0)] = False           # where early rows see few keys
    vs[large] = scales(9, 12)[large]
    for b, n in enumerate(lens):                             # the last key: hidden from all rows but the last
        at = int(table[b, (n - 1) // page]), (n - 1) % page
        if n + prefix > 64:
            vs[at], v[at] = 65504.0 / 8, -128
        if n + prefix > 1000:
            vs[at] = 65504.0
    zero = torch.rand(total, page, hkv, generator=g, device="cuda") < 1 / 20
    ks[zero], vs[zero.flip(0)] = 0.0, 0.0
    kv = ops.PagedKV(k, v, ks, vs)
    q = base.randn(g, sum(new), hq, d)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new), causal=causal)
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args)
    base.ok()
    want, tol = ref.attention(q, base.values(kv), table.cpu(), lens, new, [] if shared is None else shared.cpu().tolist(),
                              prefix, causal)
    fits = want.abs() + tol < 65504                          # others may round to an infinity
    assert bool(fits.float().mean() > 0.9)
    base.within(got.cpu()[fits], want[fits], tol[fits])
    over = got.cpu().double()[~fits]
    assert bool((over.sign() == want[~fits].sign()).all()) and bool((over.abs() > 65000 - tol[~fits]).all())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_a_loose_bound_of_the_rows(lens, new, prefix, int8):
    """max_seqlen far over every sequence, and over what 32 bits hold: the result of the batch's own bound."""
    q, kv, table, shared, _ = base.attend(66, lens, new, prefix, 128, 64, 4, 2, int8)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new))
    want = ops.attn_shared_prefix(q, kv, table, base.i32(lens), max_seqlen=sum(new), **args)
    for n in (100000, 2 ** 31 - 1, 2 ** 32 + 1):
        assert torch.equal(ops.attn_shared_prefix(q, kv, table, base.i32(lens), max_seqlen=n, **args), want)
    base.ok()
    ref_out, tol = ref.attention(q, base.values(kv), table.cpu(), lens, new, [] if shared is None else shared.cpu().tolist(),
                                 prefix)
    base.within(want, ref_out, tol)


def reported():
    torch.cuda.synchronize()
    return ops.get_device_error() == ops.TM_ERR_INVALID_ARG


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_lengths_over_the_bound_are_reported_and_cut(lens, new, prefix, int8):
    """kv_lens above max_kv_len: recorded, and the sequence ends at the bound."""
    page, bound = 64, 64
    g = base.gen(67)
    table, shared, total = base.make_table(67, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, 2, 128, int8)
    q = base.randn(g, sum(new), 4, 128)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new), max_kv_len=bound)
    cut = [min(n, bound) for n in lens]
    want = ops.attn_shared_prefix(q, kv, table, base.i32(cut), **args)
    base.ok()
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args)
    assert reported() == (cut != lens)
    assert torch.equal(got, want)
    pages = [] if shared is None else shared.cpu().tolist()
    ref_out, tol = ref.attention(q, base.values(kv), table.cpu(), cut, new, pages, prefix)
    base.within(want, ref_out, tol)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows,prefix", [(1, 0), (1, 100), (90, 0), (90, 100), (90, 3000), (3, 6000)])
def test_bounds_of_zero(rows, prefix, int8):
    """max_kv_len = 0: own tokens there are all the same are recorded, the prefix alone is seen, rows before the first
    sequence and behind the last are left.  max_seqlen = 0 with rows: right results, or an error is recorded."""
    g = base.gen(68)
    table, shared, total = base.make_table(68, [100, 100], 32, extra=prefix)
    kv = base.make_pool(g, total, 32, 2, 128, int8)
    T = 2 * rows
    q = base.randn(g, T + 5, 8, 128)
    cu = base.i32([2, 2 + rows, 2 + T])
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=cu)
    pages = [] if shared is None else shared.cpu().tolist()
    want, tol = ref.attention(q[2:2 + T], base.values(kv), table.cpu(), [0, 0], [rows, rows], pages, prefix)
    for lens in ([0, 0], [0, 3]):
        out = torch.full_like(q, 5.0)
        ops.attn_shared_prefix(q, kv, table, base.i32(lens), max_seqlen=rows, max_kv_len=0, out=out, **args)
        assert reported() == (lens != [0, 0])
        base.within(out[2:2 + T], want, tol)
        assert bool((out[:2] == 5.0).all()) and bool((out[2 + T:] == 5.0).all())
    out = torch.full_like(q, 5.0)
    ops.attn_shared_prefix(q, kv, table, base.i32([100, 100]), max_seqlen=0, out=out, **args)
    if not reported():
        want, tol = ref.attention(q[2:2 + T], base.values(kv), table.cpu(), [100, 100], [rows, rows], pages, prefix)
        base.within(out[2:2 + T], want, tol)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("prefix", [0, 300, 3000])
def test_rows_over_their_bound_are_reported(prefix, int8):
    """A sequence longer than the rows that max_seqlen made room for: recorded; the other sequences are what they were."""
    g = base.gen(69)
    new, lens = [1, 40, 2, 1], [30, 100, 90, 300]
    table, shared, total = base.make_table(69, lens, 32, extra=prefix)
    kv = base.make_pool(g, total, 32, 2, 128, int8)
    q = base.randn(g, sum(new), 8, 128)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new))
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), max_seqlen=2, **args).cpu()
    assert reported()
    pages = [] if shared is None else shared.cpu().tolist()
    want, tol = ref.attention(q, base.values(kv), table.cpu(), lens, new, pages, prefix)
    for rows in (slice(0, 1), slice(41, 44)):
        base.within(got[rows], want[rows], tol[rows])


def test_pieces_of_a_huge_capacity():
    """Very many sequences with room for millions of tokens each (one shared table row serves them here): a piece of the
    own tokens is no longer than the room, and stays within 32 bits."""
    batch, hkv, d, page = 65536, 8, 64, 256
    cols = 13000
    g = base.gen(70)
    kv = base.make_pool(g, 4, page, hkv, d, False)
    row = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    row[0, :2] = base.i32([2, 1])
    table = row.expand(batch, cols)
    lens = torch.randint(1, 400, (batch,), generator=g, device="cuda", dtype=torch.int32)
    q = base.randn(g, batch, hkv, d)
    want = ops.attn_shared_prefix(q, kv, table, lens, max_kv_len=512)
    got = ops.attn_shared_prefix(q, kv, table, lens)
    base.ok()
    pick = [0, 1, 777, batch - 1]
    ref_out, tol = ref.attention(q[pick], base.values(kv), row.cpu().expand(4, cols), lens[pick].tolist(), [1] * 4)
    base.within(want[pick], ref_out, tol)
    base.within(got[pick], ref_out, tol)
    assert float((got - want).abs().max()) <= 2.0 ** -6      # each off by its weights' rounding and its own, |v| below 8


@pytest.mark.parametrize("d,page,hq,hkv,int8,order", base.CACHES)
@pytest.mark.parametrize("lens", [[9, 33, 0, 700, 16], [5] * 70, [40000, 20, 2000]])
def test_gather_of_the_last_sequences_of_a_batch(d, page, hq, hkv, int8, order, lens):
    """Offsets that begin behind row 0 (the rest of a longer batch): rows before them are left as they were, and are no
    error."""
    g = base.gen(71 + sum(lens))
    table, _, total = base.make_table(71, lens, page)
    kv = base.make_pool(g, total, page, hkv, d, int8, order)
    T, cu = sum(lens), base.offsets(lens)
    whole, rest = (tuple(torch.full((T + 3, hkv, d), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)) for _ in range(2))
    ops.kv_gather(kv, table, cu, out=whole)
    base.ok()
    ops.kv_gather(kv, table[1:], cu[1:], out=rest)
    base.ok()
    for a, b in zip(whole, rest):
        assert torch.equal(a[lens[0]:], b[lens[0]:]) and bool((b[:lens[0]] == 5.0).all())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,prefix", PATHS)
def test_infinities_where_nothing_is_read(lens, new, prefix, causal, int8):
    """Infinities and NaN in the slots behind a sequence's end, behind the prefix's, and in pages of no sequence."""
    page = 64
    g = base.gen(72)
    table, shared, total = base.make_table(72, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, 2, 128, int8)
    q = base.randn(g, sum(new), 4, 128)
    args = dict(prefix_pages=shared, prefix_len=prefix, cu_seqlens=base.offsets(new), max_seqlen=max(new), causal=causal)
    want = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args)
    unused = torch.ones(total, page, dtype=torch.bool)
    for pages, n in [([] if shared is None else shared.tolist(), prefix)] + [(table[b].tolist(), n) for b, n in enumerate(lens)]:
        for i, p in enumerate(pages[:-(-n // page)]):
            unused[p, :max(0, min(page, n - i * page))] = False
    at = unused.cuda().nonzero()
    junk = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=torch.float16, device="cuda")
    for x in (kv.k_scales, kv.v_scales) if int8 else (kv.k, kv.v):
        fill = junk[torch.arange(len(at), device="cuda") % 3]
        x[at[:, 0], at[:, 1]] = fill.view(-1, *[1] * (x.dim() - 2)).expand(-1, *x.shape[2:])
    got = ops.attn_shared_prefix(q, kv, table, base.i32(lens), **args)
    base.ok()
    assert torch.equal(got, want) and bool(want.isfinite().all())


@pytest.mark.parametrize("d,int8", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("lens,new,prefix", PATHS + [([300, 5, 1000, 64], [1, 1, 1, 1], 0), ([1] * 9, [1] * 9, 100)])
def test_a_capacity_far_over_the_lengths(lens, new, prefix, d, int8):
    """max_kv_len at a table's capacity of 32768 tokens: the results of the lengths, and none past a short table row."""
    page = 64
    g = base.gen(73)
    table, shared, total = base.make_table(73, lens, page, extra=prefix)
    kv = base.make_pool(g, total, page, 2, d, int8)
    q = base.randn(g, sum(new), 8, d, scale=2.0)
    wide = torch.full((len(lens), 512), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    got = ops.attn_shared_prefix(q, kv, wide, base.i32(lens), prefix_pages=shared, prefix_len=prefix,
                                 cu_seqlens=base.offsets(new), max_seqlen=max(new))
    base.ok()
    want, tol = ref.attention(q, base.values(kv), table.cpu(), lens, new, [] if shared is None else shared.cpu().tolist(),
                              prefix)
    base.within(got, want, tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("around", [2.0 ** 22, -2.0 ** 22, 2.0 ** 21, 2.0 ** 23, 2.0 ** 27])
@pytest.mark.parametrize("rising", [True, False])
def test_near_scores_far_from_zero_on_a_tile(around, rising, d):
    """Scores 2^22 powers of two from zero, where a tile's references change their form, a few units apart and exact in
    fp32: rows of one tile, whose exponents come from exact products, weigh them as 64 bits do."""
    n, hq, hkv, page = 100, 4, 2, 64
    g = base.gen(74)
    table, _, total = base.make_table(74, [n, n], page)
    kv = base.make_pool(g, total, page, hkv, d, False)
    unit = 2.0 ** (round(math.log2(abs(around) * math.sqrt(d) * math.log(2))) - 20)      # of the sums: 16 of fp32's steps
    big = round(around * math.sqrt(d) * math.log(2) / unit) - 10                         # about 2^20 units
    step = torch.randint(0, 8, (total, page), generator=g, device="cuda")
    for b in range(2):                           # later keys higher (or lower) by up to 24 units
        for j in range(n):
            step[int(table[b, j // page]), j % page] += (j if rising else n - j) // 4
    scale = 2.0 ** round(math.log2(unit) / 2)    # sums of products: (hi 2^10 + lo) units, and the step
    hi, lo = divmod(big, 1024)
    keys = torch.zeros(total, page, d, device="cuda")
    keys[..., 0], keys[..., 1], keys[..., 2] = hi * scale, lo * scale, step * scale
    fill_keys(kv, keys.half())
    q = torch.zeros(2 * n, hq, d, dtype=torch.float16, device="cuda")
    other = unit / scale
    q[..., 0], q[..., 1], q[..., 2] = 1024 * other, other, other
    got = ops.attn_shared_prefix(q, kv, table, base.i32([n, n]), max_kv_len=n)
    base.ok()
    values = base.values(kv)
    assert bool((values[0][..., 0] == hi * scale).all()) and bool((q[..., 0] == 1024 * other).all())
    want, _ = ref.attention(q, values, table.cpu(), [n, n], [n, n])
    size, _ = ref.attention(q, (values[0], values[1].abs()), table.cpu(), [n, n], [n, n])
    # weights to 2^-17 of an exact exponent, rounded once, their sum the same; the result's rounding
    base.within(got, want, size * (2 * ref.HALF + 2.0 ** -15) + n * 2.0 ** -24 * 8 + ref.TINY)
