"""Paged-cache serving operators on the GPU against their 64-bit forms."""

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu

torch_cuda = torch.cuda.is_available()
if torch_cuda:
    from mixed_precision_attention_tm_b200 import ops


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).half()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(n):
    return i32([0] + torch.tensor(n).cumsum(0).tolist())


def ok():
    torch.cuda.synchronize()
    assert ops.get_device_error() == ops.TM_OK


def within(got, want, tol):
    err = (got.cpu().double() - want).abs()
    worst = (err - tol).max()
    assert worst <= 0, f"{worst} over the allowed error; largest error {err.max()}"


def make_pool(g, pages, page, h, d, int8, order="page"):
    """A pool of random pages with every slot filled: order is the layout, slots or heads first."""
    if order == "head":
        def make():
            return randn(g, pages, h, page, d).transpose(1, 2)
    else:
        def make():
            return randn(g, pages, page, h, d)
    k, v = make(), make()
    if not int8:
        return ops.PagedKV(k, v)
    (kc, ks), (vc, vs) = ref.quantise(k.cpu().double()), ref.quantise(v.cpu().double())
    if order == "head":
        kc, vc = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (kc, vc))
        ks, vs = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (ks, vs))
    return ops.PagedKV(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda())


def make_table(seed, lens, page, spare=2, extra=0):
    """A block table for sequences of lens tokens; (table, pages of a prefix of `extra` tokens, pages in all)."""
    need = [-(-n // page) for n in lens]
    shared = -(-extra // page)
    total = sum(need) + shared + spare
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32)
    at = shared
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), i32(ids[:shared]) if shared else None, total


def values(kv):
    return tuple(ref.pool_values(x, s) for x, s in ((kv.k, kv.k_scales), (kv.v, kv.v_scales)))


# ------------------------------------------------------------ rotation, norms
TURNS = [
    dict(rot_dim=128, interleaved=False, scaling=None, factor=1.0),
    dict(rot_dim=32, interleaved=True, scaling="linear", factor=4.0),
    dict(rot_dim=48, interleaved=False, scaling="ntk", factor=2.0),
    dict(rot_dim=128, interleaved=True, scaling="yarn", factor=16.0),
    dict(rot_dim=64, interleaved=False, scaling="bands", factor=8.0),
    dict(rot_dim=16, interleaved=False, scaling="yarn", factor=40.0),
]


def rope_pair(turn, d, **kw):
    rot = min(turn["rot_dim"], d)
    r = ops.Rope(d, rot, interleaved=turn["interleaved"], scaling=turn["scaling"], factor=turn["factor"], **kw)
    return r, dict(rot=rot, interleaved=turn["interleaved"], scaling=turn["scaling"], factor=turn["factor"], **kw)


@pytest.mark.parametrize("turn", TURNS)
@pytest.mark.parametrize("T,hq,hkv,d", [(1, 8, 1, 128), (3, 5, 3, 64), (130, 32, 8, 128), (2049, 3, 1, 64)])
def test_rope_and_norm(turn, T, hq, hkv, d):
    g = gen(T + d)
    q, k = randn(g, T, hq, d), randn(g, T, hkv, d, scale=3.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").int()
    qw, kw_ = randn(g, d), randn(g, d)
    r, spec = rope_pair(turn, d)
    q0, k0 = q.cpu().double(), k.cpu().double()
    for normed in (False, True):
        if normed:
            got = ops.qk_norm_rope(q, k, q_weight=qw, k_weight=kw_, eps=1e-5, rope=r, positions=pos)
            a, b = ref.norm(q0, qw.cpu(), 1e-5), ref.norm(k0, kw_.cpu(), 1e-5)
        else:
            got = ops.rope(q, k, rope=r, positions=pos)
            a, b = q0, k0
        ok()
        for x, y in zip(got, (a, b)):
            want, size = ref.turn(y, pos.cpu(), **spec)
            within(x, want, ref.turn_error(want, size))


def test_rope_far_positions_and_offset():
    """Positions near 2^31 with an offset past 32 bits keep their angle."""
    g = gen(5)
    q = randn(g, 4, 2, 128)
    pos = i32([0, 1, (1 << 31) - 1, 12345])
    off = (1 << 33) + 77
    got = ops.rope(q, rope=ops.Rope(128), positions=pos, pos_offset=off)
    ok()
    # 64-bit angles of such positions are off by 2^-53 p; the kernel's by 2^-64 p: the frequencies' own rounding leads
    want, size = ref.turn(q.cpu().double(), pos.cpu().long() + off, 128)
    far = (pos.cpu().long() + off).double()[:, None, None]
    within(got, want, ref.turn_error(want, size) + size * far * 2.0 ** -51)


def test_rope_strides_in_place_and_row_index():
    g = gen(6)
    base = randn(g, 7, 12, 128)
    q, k = base[:, :8], base[:, 8:]          # views of one buffer
    r = ops.Rope(128, 64)
    want_q, want_k = ops.rope(q, k, rope=r, positions=torch.arange(7, dtype=torch.int32, device="cuda") + 9)
    heads_first = randn(g, 12, 7, 128).transpose(0, 1)
    heads_first.copy_(base)
    out = ops.rope(heads_first[:, :8], heads_first[:, 8:], rope=r, pos_offset=9,
                   out=(heads_first[:, :8], heads_first[:, 8:]))
    ok()
    assert torch.equal(out[0], want_q) and torch.equal(out[1], want_k)
    assert torch.equal(heads_first[:, 8:], want_k)


def test_norm_alone_extremes_and_nan_stay_in_their_row():
    g = gen(7)
    q = randn(g, 6, 4, 64)
    q[1, 2] = 0
    q[2, 1, 5] = float("nan")
    q[3, 0] = 60000.0
    w = randn(g, 64)
    got = ops.qk_norm_rope(q, q_weight=w, eps=1e-6)
    ok()
    want = ref.norm(q.cpu().double(), w.cpu(), 1e-6)
    assert got[2, 1].isnan().all() and torch.equal(got[1, 2], torch.zeros_like(got[1, 2]))
    keep = torch.ones(6, 4, dtype=torch.bool)
    keep[2, 1] = False
    within(got.cpu()[keep], want[keep], want[keep].abs() * (ref.HALF + 2.0 ** -19) + ref.TINY)


# ---------------------------------------------------------------------- cache
CACHES = [(128, 16, 8, 2, False, "page"), (128, 64, 4, 4, True, "page"), (64, 32, 7, 1, True, "head"),
          (64, 128, 6, 3, False, "head"), (128, 256, 3, 1, True, "head")]


@pytest.mark.parametrize("d,page,hq,hkv,int8,order", CACHES)
@pytest.mark.parametrize("lens,new", [([1], [1]), ([5, 17, 300, 64], [1, 17, 33, 0]), ([1] * 40, [1] * 40),
                                      ([3, 90], [7, 20])])
def test_append(d, page, hq, hkv, int8, order, lens, new):
    g = gen(sum(lens) + d)
    table, _, total = make_table(3, lens, page)
    kv = make_pool(g, total, page, hkv, d, int8, order)
    before = [x.clone() if x is not None else None for x in (kv.k, kv.v, kv.k_scales, kv.v_scales)]
    T = sum(new)
    q, k, v = randn(g, T + 2, hq, d), randn(g, T + 2, hkv, d), randn(g, T + 2, hkv, d)
    v[0, 0] = 0                                   # a row whose scale is zero
    qw, kw = randn(g, d), randn(g, d)
    r, spec = rope_pair(TURNS[4], d)
    q_out = torch.full_like(q, 7.0)
    got = ops.kv_append(k, v, kv, table, i32(lens), cu_seqlens=offsets(new), rope=r, pos_offset=1000, q=q, q_weight=qw,
                        k_weight=kw, eps=1e-5, q_out=q_out)
    ok()
    assert got is q_out and bool((q_out[T:] == 7.0).all())       # rows behind the last sequence
    b = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    i = torch.cat([torch.arange(n) for n in new])
    j = torch.tensor(lens)[b] - torch.tensor(new)[b] + i
    want_q, size = ref.turn(ref.norm(q[:T].cpu().double(), qw.cpu(), 1e-5), j + 1000, **spec)
    within(q_out[:T], want_q, ref.turn_error(want_q, size))
    want_k, size = ref.turn(ref.norm(k[:T].cpu().double(), kw.cpu(), 1e-5), j + 1000, **spec)
    here = j >= 0
    t = table.cpu().long()
    jj = j.clamp(min=0)
    at = t[b, jj // page] * page + jj % page

    def flat(x):
        return x.cpu().contiguous().flatten(0, 1)
    touched = torch.zeros(total * page, dtype=torch.bool)
    touched[at[here]] = True
    for x, old in zip((kv.k, kv.v, kv.k_scales, kv.v_scales), before):
        if x is not None:
            assert torch.equal(flat(x)[~touched], flat(old)[~touched])
    k_err = ref.turn_error(want_k, size)
    if not int8:
        within(flat(kv.k)[at[here]], want_k[here], k_err[here])
        assert torch.equal(flat(kv.v)[at[here]], v[:T].cpu()[here])
        return
    codes, scales = ref.quantise(v[:T].cpu().double())
    assert torch.equal(flat(kv.v)[at[here]], codes[here]) and torch.equal(flat(kv.v_scales)[at[here]], scales[here])
    ks = flat(kv.k_scales)[at[here]].double()
    amax = want_k.abs().amax(-1)[here]
    slack = (size * 2.0 ** -19).amax(-1)[here]                  # fp32 error of the values
    assert bool(((ks - amax / 127).abs() <= ks * ref.HALF + ref.TINY + slack / 127).all())
    # half a code, the clamp (amax may lie up to 127 half steps of the scale above 127 codes), the values' own error
    err = (flat(kv.k)[at[here]].double() * ks[..., None] - want_k[here]).abs()
    assert bool((err <= (ks * (0.5 + 127.5 * ref.HALF) + 128 * ref.TINY)[..., None] + size[here] * 2.0 ** -18).all())


def test_append_equal_rows_without_offsets_equals_packed():
    g = gen(11)
    lens, page, d, h = [9, 33, 21], 16, 128, 2
    table, _, total = make_table(4, lens, page)
    kv1, kv2 = make_pool(g, total, page, h, d, False), make_pool(gen(11), total, page, h, d, False)
    kv2.k.copy_(kv1.k), kv2.v.copy_(kv1.v)
    k, v = randn(g, 6, h, d), randn(g, 6, h, d)
    assert ops.kv_append(k, v, kv1, table, i32(lens)) is None
    ops.kv_append(k, v, kv2, table, i32(lens), cu_seqlens=i32([0, 2, 4, 6]))
    ok()
    assert torch.equal(kv1.k, kv2.k) and torch.equal(kv1.v, kv2.v)


def test_append_nan_and_inf_rows_of_an_int8_cache():
    g = gen(12)
    table, _, total = make_table(4, [4], 16)
    kv = make_pool(g, total, 16, 2, 64, True)
    k, v = randn(g, 4, 2, 64), randn(g, 4, 2, 64)
    k[1, 0, 3], v[2, 1, 60] = float("nan"), float("inf")
    ops.kv_append(k, v, kv, table, i32([4]))
    ok()
    page = int(table[0, 0])
    assert kv.k_scales[page, 1, 0].isnan() and kv.v_scales[page, 2, 1].isinf()
    assert int(kv.k_scales[page, :4].isfinite().sum()) == 7 and int(kv.v_scales[page, :4].isfinite().sum()) == 7


@pytest.mark.parametrize("d,page,hq,hkv,int8,order", CACHES)
@pytest.mark.parametrize("lens", [[1], [0, 33, 0, 700, 16], [5] * 70])
def test_gather(d, page, hq, hkv, int8, order, lens):
    g = gen(sum(lens))
    table, _, total = make_table(8, lens, page)
    kv = make_pool(g, total, page, hkv, d, int8, order)
    T = sum(lens)
    out = tuple(torch.full((T + 3, hkv, d), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
    ops.kv_gather(kv, table, offsets(lens), out=out)
    ok()
    for got, pool in zip(out, values(kv)):
        want = torch.cat([ref.rows_of(pool, table[b], n) for b, n in enumerate(lens)])
        assert torch.equal(got[:T].cpu(), want.half())       # a code times its scale is exact in fp32: one rounding
        assert bool((got[T:] == 5.0).all())


# ------------------------------------------------------------------ attention
def attend(seed, lens, new, prefix, d, page, hq, hkv, int8, order="page", causal=True, scale=2.0, packed=True,
           tail=0, **kw):
    g = gen(seed)
    table, shared, total = make_table(seed, lens, page, extra=prefix)
    kv = make_pool(g, total, page, hkv, d, int8, order)
    T = sum(new)
    q = randn(g, T + tail, hq, d, scale=scale)
    out = torch.full_like(q, 3.0)
    args = dict(prefix_pages=shared, prefix_len=prefix, causal=causal, out=out, **kw)
    if packed:
        args.update(cu_seqlens=offsets(new), max_seqlen=max(new))
    ops.attn_shared_prefix(q, kv, table, i32(lens), **args)
    ok()
    want, tol = ref.attention(q[:T], values(kv), table.cpu(), lens, new,
                              [] if shared is None else shared.cpu().tolist(), prefix, causal)
    within(out[:T], want, tol)
    assert bool((out[T:] == 3.0).all())
    return q, kv, table, shared, out


SETS = [
    ([1], [1], 0), ([1], [1], 1), ([130], [1], 0), ([17, 1, 129, 64], [1, 1, 1, 1], 1000),
    ([40, 9, 100], [40, 9, 0], 0), ([3, 300, 65], [3, 70, 65], 513), ([0, 5, 0], [0, 2, 0], 31), ([2, 4], [5, 6], 0),
]


@pytest.mark.parametrize("d,page,hq,hkv,int8,order", CACHES)
@pytest.mark.parametrize("lens,new,prefix", SETS)
def test_attention(d, page, hq, hkv, int8, order, lens, new, prefix):
    attend(20, lens, new, prefix, d, page, hq, hkv, int8, order, tail=2)


@pytest.mark.parametrize("d,page,hq,hkv,int8,order", CACHES)
@pytest.mark.parametrize("prefix", [2300, 2304])
def test_attention_on_tiles(d, page, hq, hkv, int8, order, prefix):
    """Enough rows and keys for the tile kernel: chunks of prompts, with the prefix folded in, and short rows of many
    sequences, with a pass of its own for the prefix; rows behind the last sequence."""
    attend(43, [301, 100, 4, 0], [300, 100, 1, 0], prefix, d, page, hq, hkv, int8, order, tail=3)
    attend(47, [20 + i for i in range(70)], [1 + i % 11 for i in range(70)], prefix, d, page, hq, hkv, int8, order, tail=3)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,new", [([0, 3, 200], [90, 3, 70]), ([2500, 40], [100, 40]), ([900], [700])])
@pytest.mark.parametrize("prefix", [1, 128, 200, 777])
def test_attention_with_the_prefix_folded_in(lens, new, prefix, int8):
    """Own tokens behind the prefix's whole tiles: rows that see the prefix only, splits that end in either part."""
    attend(48, lens, new, prefix, 128, 16, 4, 2, int8)
    attend(49, lens, new, prefix, 64, 256, 4, 1, int8, "head", causal=False)


@pytest.mark.parametrize("hq,hkv", [(28, 4), (6, 2), (8, 2)])
@pytest.mark.parametrize("int8", [False, True])
def test_attention_on_tiles_groups(hq, hkv, int8):
    """Query heads per K/V head that do and do not divide a tile's 128 rows."""
    attend(44, [200, 150], [200, 97], 1900, 128, 32, hq, hkv, int8)
    attend(45, [200, 150], [200, 97], 1900, 64, 64, hq, hkv, int8, causal=False)


@pytest.mark.parametrize("d,int8", [(64, False), (128, True)])
def test_attention_in_pieces_of_the_line(d, int8):
    """As many row blocks as SMs, whose key tiles are cut without regard to the blocks."""
    attend(46, [900, 690, 3], [900, 690, 1], 2700, d, 128, 16, 16, int8)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 1), (28, 4), (24, 8), (64, 2), (40, 2)])
@pytest.mark.parametrize("int8", [False, True])
def test_attention_groups(hq, hkv, int8):
    attend(21, [50, 200, 7], [2, 1, 3], 200, 64, 16, hq, hkv, int8)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 3), (7, 1), (16, 2), (9, 1)])
@pytest.mark.parametrize("d,int8,scale", [(64, False, 2.0), (128, True, 2.0), (128, False, 30.0), (64, True, 0.0)])
def test_attention_single_tokens_of_many_sequences(hq, hkv, d, int8, scale):
    """Rows of eight query heads and fewer (and of nine), the shared prefix in blocks as small."""
    lens = [0, 1, 15, 16, 17, 700, 128, 129] + [257 + 31 * i for i in range(16)]
    attend(50, lens, [1] * len(lens), 100, d, 32, hq, hkv, int8, scale=scale, tail=1)
    attend(51, lens, [0, 1, 1, 0] * 6, 0, d, 64, hq, hkv, int8, "head", scale=scale, causal=False)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_rows_and_many(d, int8):
    """Splits of both kinds, rows of several tiles."""
    attend(22, [2100, 900], [150, 1], 3000, d, 64, 4, 1, int8)
    attend(23, [70] * 33, [1] * 33, 5000, d, 32, 8, 2, int8)


@pytest.mark.parametrize("int8", [False, True])
def test_attention_not_causal(int8):
    attend(24, [33, 80, 1], [4, 1, 2], 100, 128, 16, 4, 2, int8, causal=False)


def test_attention_one_shape_without_offsets():
    attend(25, [33, 80, 10], [2, 2, 2], 70, 128, 16, 8, 2, False, packed=False)


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_attention_flat_and_peaked(scale):
    attend(26, [200, 90], [3, 1], 400, 64, 16, 4, 2, False, scale=scale)


@pytest.mark.parametrize("prefix", [150, 2500])        # on the split-key kernel, on the tile kernel
def test_attention_ignores_what_no_row_sees(prefix):
    """NaN and infinities in unused slots, unused pages and (as keys) at causally hidden positions change nothing."""
    lens, new, page = [70, 21, 140] + [9] * 40, [1, 1, 130] + [3] * 40, 64
    g = gen(27)
    table, shared, total = make_table(27, lens, page, extra=prefix)
    q = randn(g, sum(new), 8, 128)
    for int8 in (False, True):
        kv = make_pool(g, total, page, 2, 128, int8)
        args = dict(cu_seqlens=offsets(new), max_seqlen=130, prefix_pages=shared, prefix_len=prefix)
        want = ops.attn_shared_prefix(q, kv, table, i32(lens), **args)
        used = torch.zeros(total, page, dtype=torch.bool, device="cuda")
        for pages, n in [(shared, prefix)] + [(table[b], n) for b, n in enumerate(lens)]:
            for j in range(n):
                used[int(pages[j // page]), j % page] = True
        for x in (kv.k_scales, kv.v_scales) if int8 else (kv.k, kv.v):
            x[~used] = float("nan")
        got = ops.attn_shared_prefix(q, kv, table, i32(lens), **args)
        ok()
        assert torch.equal(got, want)


@pytest.mark.parametrize("bad", ["past the pool", "negative", "in the prefix"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows,prefix", [(1, 64), (100, 64), (100, 3000)])
def test_attention_bad_pages_are_reported_and_not_read(rows, prefix, int8, bad):
    g = gen(28)
    table, shared, total = make_table(28, [100, 140], 16, extra=prefix)
    kv = make_pool(g, total, 16, 2, 64, int8)
    q = randn(g, 2 * rows, 8, 64)
    args = dict(prefix_pages=shared, prefix_len=prefix)
    where = shared[1:2] if bad == "in the prefix" else table[0, 3:4]
    old = where.clone()
    where.fill_(total if bad == "past the pool" else -3)
    out = ops.attn_shared_prefix(q, kv, table, i32([100, 140]), **args)
    torch.cuda.synchronize()
    assert ops.get_device_error() == ops.TM_ERR_INVALID_ARG
    where.copy_(old)
    good = ops.attn_shared_prefix(q, kv, table, i32([100, 140]), **args)
    ok()
    if bad != "in the prefix":
        assert torch.equal(out[rows:], good[rows:])      # the other sequence does not see that page


def test_two_graphs_with_their_workspaces_and_streams():
    """Decoding captured once and replayed while the lengths grow, on two streams side by side."""
    g = gen(29)
    page, hq, hkv, d, prefix, n = 16, 8, 2, 128, 200, 3
    state = []
    for i in range(2):
        table, shared, total = make_table(30 + i, [64] * n, page, extra=prefix)
        kv = make_pool(g, total, page, hkv, d, bool(i))
        k, v, q = randn(g, n, hkv, d), randn(g, n, hkv, d), randn(g, n, hq, d)
        lens = i32([10, 20, 30])
        s = dict(table=table, shared=shared, kv=kv, k=k, v=v, q=q, lens=lens, qr=torch.empty_like(q),
                 out=torch.empty_like(q), rope=ops.Rope(d),
                 ws=torch.empty(ops.shared_prefix_workspace_bytes(kv, n, n, hq, prefix_len=prefix, max_kv_len=64),
                                dtype=torch.uint8, device="cuda"))
        state.append(s)

    def step(s):
        ops.kv_append(s["k"], s["v"], s["kv"], s["table"], s["lens"], rope=s["rope"], pos_offset=prefix, q=s["q"],
                      q_out=s["qr"])
        ops.attn_shared_prefix(s["qr"], s["kv"], s["table"], s["lens"], prefix_pages=s["shared"], prefix_len=prefix,
                               max_kv_len=64, workspace=s["ws"], out=s["out"])
    graphs, streams = [], [torch.cuda.Stream() for _ in state]
    for s in state:
        step(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s)
        graphs.append(graph)
    for _ in range(5):
        for s in state:
            s["k"].copy_(randn(g, n, hkv, d)), s["q"].copy_(randn(g, n, hq, d))
            s["lens"] += 1
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for s in state:
            got = s["out"].clone()
            want, tol = ref.attention(s["qr"], values(s["kv"]), s["table"].cpu(), s["lens"].tolist(), [1] * n,
                                      s["shared"].tolist(), prefix)
            within(got, want, tol)
    ok()
    graphs.clear()


def test_results_repeat_exactly():
    q, kv, table, shared, out = attend(31, [500, 80], [30, 1], 900, 128, 32, 8, 2, True)
    again = [ops.attn_shared_prefix(q, kv, table, i32([500, 80]), cu_seqlens=i32([0, 30, 31]), max_seqlen=30,
                                    prefix_pages=shared, prefix_len=900) for _ in range(3)]
    ok()
    assert all(torch.equal(out, a) for a in again)


def test_prompt_then_steps_agrees_with_prefill_attention():
    """A prompt appended, read back and attended by attn_fwd, equals attention over the pages; then single steps."""
    g = gen(33)
    d, hq, hkv, page = 128, 8, 2, 32
    new = [70, 1, 133]
    table, _, total = make_table(33, [n + 40 for n in new], page)
    kv = make_pool(g, total, page, hkv, d, False)
    r = ops.Rope(d, theta=500000.0)
    T = sum(new)
    q, k, v = randn(g, T, hq, d), randn(g, T, hkv, d), randn(g, T, hkv, d)
    cu, lens = offsets(new), i32(new)
    qr = ops.kv_append(k, v, kv, table, lens, cu_seqlens=cu, rope=r, q=q)
    rows = tuple(torch.empty(T, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    ops.kv_gather(kv, table, cu, out=rows)
    dense = ops.attn_fwd(qr, *rows, causal=True, cu_seqlens=cu, max_seqlen=max(new))
    paged = ops.attn_shared_prefix(qr, kv, table, lens, cu_seqlens=cu, max_seqlen=max(new))
    ok()
    want, tol = ref.attention(qr, values(kv), table.cpu(), new, new)
    within(dense, want, tol + 2.0 ** -10 * want.abs())
    within(paged, want, tol)
    kq = ops.rope(k, rope=r, positions=torch.cat([torch.arange(n) for n in new]).int().cuda())
    assert torch.equal(rows[0], kq) and torch.equal(rows[1], v)
    for step in range(1, 4):
        n = len(new)
        q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
        lens = i32([x + step for x in new])
        qr = ops.kv_append(k, v, kv, table, lens, rope=r, q=q)
        out = ops.attn_shared_prefix(qr, kv, table, lens)
        ok()
        want, tol = ref.attention(qr, values(kv), table.cpu(), lens.tolist(), [1] * n)
        within(out, want, tol)


def test_offsets_past_32_bits():
    """Pages that lie more than 4 GB into the pool."""
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    page, h, d = 256, 8, 128
    pages = (5 << 30) // (page * h * d * 2)
    kv = ops.PagedKV(*(torch.zeros(pages, page, h, d, dtype=torch.float16, device="cuda") for _ in range(2)))
    g = gen(40)
    table = i32([[pages - 1, 0], [1, pages - 2]])
    lens = [300, 270]
    k, v, q = randn(g, sum(lens), h, d), randn(g, sum(lens), h, d), randn(g, 2, h, d)
    ops.kv_append(k, v, kv, table, i32(lens), cu_seqlens=offsets(lens))
    out = ops.attn_shared_prefix(q, kv, table, i32(lens))
    rows = tuple(torch.empty_like(k) for _ in range(2))
    ops.kv_gather(kv, table, offsets(lens), out=rows)
    ok()
    assert torch.equal(rows[0], k) and torch.equal(rows[1], v)
    small = ops.PagedKV(*(torch.zeros(4, page, h, d, dtype=torch.float16, device="cuda") for _ in range(2)))
    near = i32([[3, 0], [1, 2]])
    ops.kv_append(k, v, small, near, i32(lens), cu_seqlens=offsets(lens))
    assert torch.equal(out, ops.attn_shared_prefix(q, small, near, i32(lens)))


@pytest.mark.parametrize("d,int8", [(128, False), (64, True), (128, True), (64, False)])
def test_attention_pieces_of_row_blocks(d, int8):
    """More key tiles of the prefix than SMs."""
    attend(41, [40 + i for i in range(60)], [1 + i % 5 for i in range(60)], 2500, d, 32, 16, 4, int8)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 2, 130]])
@pytest.mark.parametrize("prefix", [0, 100])
def test_in_place_queries(new, prefix):
    """Queries rotated in place by the append, then the result in their place."""
    g = gen(50)
    lens = [150, 40, 140]
    table, shared, total = make_table(50, lens, 32, extra=prefix)
    kv = make_pool(g, total, 32, 2, 128, False)
    T = sum(new)
    q, k, v = randn(g, T, 8, 128), randn(g, T, 2, 128), randn(g, T, 2, 128)
    args = dict(cu_seqlens=offsets(new))
    r = ops.Rope(128)
    want_q = ops.kv_append(k, v, kv, table, i32(lens), rope=r, pos_offset=prefix, q=q, **args)
    assert ops.kv_append(k, v, kv, table, i32(lens), rope=r, pos_offset=prefix, q=q, q_out=q, **args) is q
    args.update(max_seqlen=max(new), prefix_pages=shared, prefix_len=prefix)
    want = ops.attn_shared_prefix(want_q, kv, table, i32(lens), **args)
    ops.attn_shared_prefix(q, kv, table, i32(lens), out=q, **args)
    ok()
    assert torch.equal(q, want)


def test_calls_on_another_stream():
    """A call on a side stream, ordered by events only."""
    g = gen(51)
    table, shared, total = make_table(51, [70, 33], 16, extra=300)
    kv = make_pool(g, total, 16, 2, 64, True)
    q = randn(g, 2, 8, 64)
    args = dict(prefix_pages=shared, prefix_len=300)
    lens = i32([70, 33])
    want = ops.attn_shared_prefix(q, kv, table, lens, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [ops.attn_shared_prefix(q, kv, table, lens, **args) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(side)
    ok()
    assert all(torch.equal(x, want) for x in got)
