"""CPU checks of the paged-cache operators: rotation frequencies, block-table
checks, plans, and refusals before any launch."""

import ctypes
import math
import random

import pytest
import torch

import paged_ref as ref
from mixed_precision_attention_tm_b200 import build as tmbuild

tmbuild.build()
from mixed_precision_attention_tm_b200 import ops  # noqa: E402

BUF = ctypes.create_string_buffer(1 << 16)
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256


def thd(T, H, d, st=None, sh=None, ptr=PTR):
    return ops.TmTensor(ptr, T, H, d, H * d if st is None else st, d if sh is None else sh)


def cache(page=16, H=2, d=128, pages=4, int8=False, **kw):
    args = dict(k=PTR, v=PTR, k_scales=PTR if int8 else None, v_scales=PTR if int8 else None, num_pages=pages,
                page_size=page, H=H, d=d, stride_page=page * H * d, stride_t=H * d, stride_h=d,
                scale_stride_page=page * H, scale_stride_t=H, scale_stride_h=1)
    args.update(kw)
    return ops.TmPagedKv(**args)


# ------------------------------------------------------------------- rotation
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 48), (64, 16), (64, 64)])
@pytest.mark.parametrize("theta,factor,first", [(10000.0, 8.0, 4096), (500000.0, 1.0, 8192), (1000.0, 40.0, 64)])
def test_frequencies(scaling, d, rot, theta, factor, first):
    r = ops.Rope(d, rot, theta=theta, scaling=scaling, factor=factor, original_max=first)
    f, m = ref.frequencies(rot, theta=theta, scaling=scaling, factor=factor, original_max=first)
    assert r.struct.mscale == pytest.approx(m, rel=2 ** -24)
    for i in range(64):
        want = float(f[i]) / (2 * math.pi) if i < rot // 2 else 0.0
        # two 64-bit evaluations of a power: a few of their roundings times the exponent's logarithm
        assert abs(r.struct.turns[i] / 2.0 ** 64 - want) <= want * 2.0 ** -47 + 2.0 ** -64


@pytest.mark.parametrize("kw", [dict(d=96), dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=144), dict(theta=1.0),
                                dict(theta=float("nan")), dict(scaling="linear", factor=0.5),
                                dict(scaling="yarn", factor=2.0, original_max=0),
                                dict(scaling="bands", factor=2.0, fast=1.0, slow=1.0),
                                dict(scaling="ntk", factor=float("inf")),
                                dict(scaling="yarn", factor=2.0, slow=-1.0)])
def test_rope_refusals(kw):
    args = dict(d=128)
    args.update(kw)
    with pytest.raises(ops.TmError):
        ops.Rope(args.pop("d"), **args)


def test_rope_unknown_scaling():
    with pytest.raises(ValueError):
        ops.Rope(128, scaling="other")


def rope_status(q, k, qo, ko, rope, pos=None, norm=False, w=PTR, eps=1e-6):
    refs = [None if x is None else ctypes.byref(x) for x in (q, k, qo, ko)]
    r = None if rope is None else ctypes.byref(rope)
    if norm:
        return ops._lib().tm_qk_norm_rope(*refs, w, w, eps, r, pos, 0, None)
    return ops._lib().tm_rope(*refs, r, pos, 0, None)


def test_rope_call_refusals():
    r = ops.Rope(128).struct
    bad = ops.TM_ERR_INVALID_ARG
    x = thd(4, 2, 128)
    assert rope_status(x, None, x, None, None) == bad
    assert rope_status(None, None, x, None, r) == bad
    assert rope_status(x, x, x, None, r) == bad                            # k without its output
    assert rope_status(x, None, thd(4, 3, 128), None, r) == bad            # shapes differ
    assert rope_status(x, thd(5, 2, 128), x, thd(5, 2, 128), r) == bad     # rows differ
    assert rope_status(thd(4, 2, 64), None, thd(4, 2, 64), None, r) == bad  # heads of another size than the rope's
    assert rope_status(thd(4, 2, 128, ptr=PTR + 2), None, x, None, r) == bad
    assert rope_status(thd(4, 2, 128, st=257), None, x, None, r) == bad
    assert rope_status(x, None, thd(4, 2, 128, sh=0), None, r) == bad      # output heads on top of each other
    assert rope_status(x, None, thd(4, 2, 128, st=128), None, r) == bad
    assert rope_status(x, None, x, None, r, pos=PTR + 1) == bad
    assert rope_status(x, None, x, None, r, norm=True, w=None) == bad
    assert rope_status(x, None, x, None, r, norm=True, w=PTR + 2) == bad
    assert rope_status(x, None, x, None, r, norm=True, eps=-1.0) == bad
    assert rope_status(x, None, x, None, r, norm=True, eps=float("nan")) == bad
    assert rope_status(thd(4, 2, 96), None, thd(4, 2, 96), None, None, norm=True) == ops.TM_ERR_UNSUPPORTED
    e = thd(0, 2, 128, ptr=None)
    assert rope_status(e, None, e, None, r) == ops.TM_OK                   # no rows: nothing to do


def test_unaligned_stride_of_a_lone_row_is_not_refused():
    r = ops.Rope(128).struct
    x = thd(0, 1, 128, sh=3)
    assert rope_status(x, None, x, None, r) == ops.TM_OK


# ---------------------------------------------------------------- block tables
def test_block_table_check():
    table = torch.tensor([[3, 1, -1], [0, 9, 9]], dtype=torch.int32)
    ops.block_table_check(table, [32, 16], 4, 16)
    ops.block_table_check(table, [0, 0], 4, 16)
    for lens, where in (([33, 1], "sequence 0, column 2"), ([1, 17], "sequence 1, column 1"),
                        ([1, 16 * 5], "sequence 1, column 1")):
        with pytest.raises(ValueError, match=where):
            ops.block_table_check(table, lens, 4, 16)
    with pytest.raises(ValueError, match="sequence 0, column 3"):
        ops.block_table_check(torch.zeros(1, 3, dtype=torch.int32), [49], 4, 16)     # longer than the table
    with pytest.raises(ops.TmError):
        ops.block_table_check(table, [1], 4, 24)
    with pytest.raises(ValueError):
        ops.block_table_check(table, [1, 1, 1], 4, 16)


# ------------------------------------------------------------------- refusals
def append_status(k=None, v=None, c=None, table=PTR, cols=4, stride=4, lens=PTR, cu=PTR, batch=2, rope=None, q=None,
                  q_out=None, qw=None, kw=None, eps=1e-6):
    k = thd(4, 2, 128) if k is None else k
    v = thd(4, 2, 128) if v is None else v
    c = cache() if c is None else c
    ref_ = [None if x is None else ctypes.byref(x) for x in (rope, q, q_out)]
    return ops._lib().tm_kv_append(ctypes.byref(k), ctypes.byref(v), ctypes.byref(c), table, stride, cols, lens, cu,
                                   batch, ref_[0], 0, ref_[1], ref_[2], qw, kw, eps, None)


BAD_CACHES = [dict(k=None), dict(v=PTR + 4), dict(num_pages=0), dict(H=0), dict(stride_t=0), dict(stride_page=-4096),
              dict(stride_h=4), dict(k_scales=PTR), dict(int8=True, scale_stride_t=0), dict(int8=True, v_scales=PTR + 1),
              dict(int8=True, stride_h=8)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused(kw):
    assert append_status(c=cache(**kw)) == ops.TM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(page=8), dict(page=48), dict(page=512), dict(d=96)])
def test_caches_of_other_sizes_are_unsupported(kw):
    assert append_status(c=cache(**kw)) == ops.TM_ERR_UNSUPPORTED


def test_append_refusals():
    bad = ops.TM_ERR_INVALID_ARG
    assert append_status(table=None) == bad
    assert append_status(table=PTR + 2) == bad
    assert append_status(cols=0) == bad
    assert append_status(stride=-1) == bad
    assert append_status(lens=None) == bad
    assert append_status(batch=0) == bad
    assert append_status(k=thd(4, 3, 128)) == bad
    assert append_status(v=thd(5, 2, 128)) == bad
    assert append_status(k=thd(5, 2, 128), v=thd(5, 2, 128), cu=None) == bad       # 5 rows for 2 sequences
    assert append_status(q=thd(4, 8, 128)) == bad
    assert append_status(q=thd(4, 8, 128), q_out=thd(4, 8, 128, sh=0)) == bad
    assert append_status(rope=ops.Rope(64).struct) == bad
    assert append_status(kw=PTR + 8) == bad
    assert append_status(kw=PTR, eps=-1.0) == bad
    assert append_status(k=thd(0, 2, 128), v=thd(0, 2, 128)) == ops.TM_OK


def attn_status(T=4, hq=4, c=None, out=None, batch=2, max_seqlen=2, pages=PTR, prefix=16, max_kv=64, ws=PTR, nbytes=1 << 40,
                lens=PTR, cu=PTR):
    c = cache() if c is None else c
    q = thd(T, hq, 128)
    out = thd(T, hq, 128) if out is None else out
    return ops._lib().tm_attn_shared_prefix(ctypes.byref(q), ctypes.byref(c), ctypes.byref(out), PTR, 4, 4, lens, cu, batch,
                                            max_seqlen, pages, prefix, max_kv, 1, ws, nbytes, None)


def test_attention_refusals():
    bad = ops.TM_ERR_INVALID_ARG
    assert attn_status(hq=3) == bad
    assert attn_status(out=thd(4, 2, 128)) == bad
    assert attn_status(out=thd(4, 4, 128, st=0)) == bad
    assert attn_status(batch=0) == bad
    assert attn_status(lens=None) == bad
    assert attn_status(cu=None, T=5) == bad
    assert attn_status(pages=None) == bad
    assert attn_status(prefix=-1) == bad
    assert attn_status(max_kv=65) == bad                       # the table holds 64
    assert attn_status(max_seqlen=-1) == bad
    assert attn_status(ws=None) == bad
    assert attn_status(ws=PTR + 16) == bad
    need = ops._lib().tm_attn_shared_prefix_workspace(4, 4, 2, 128, 2, 2, 16, 64)
    assert need > 256 and attn_status(nbytes=need - 1) == bad
    assert attn_status(T=0) == ops.TM_OK
    assert ops._lib().tm_attn_shared_prefix_workspace(4, 3, 2, 128, 2, 2, 16, 64) == -1
    assert ops._lib().tm_attn_shared_prefix_workspace(4, 4, 2, 96, 2, 2, 16, 64) == -1


def test_gather_refusals():
    def status(cu=PTR, batch=2, k=None, v=None):
        k, v = thd(4, 2, 128) if k is None else k, thd(4, 2, 128) if v is None else v
        return ops._lib().tm_kv_gather(ctypes.byref(cache()), PTR, 4, 4, cu, batch, ctypes.byref(k), ctypes.byref(v), None)
    bad = ops.TM_ERR_INVALID_ARG
    assert status(cu=None) == bad
    assert status(batch=0) == bad
    assert status(k=thd(4, 1, 128)) == bad
    assert status(v=thd(3, 2, 128)) == bad
    assert status(v=thd(4, 2, 128, sh=64)) == bad
    assert status(k=thd(0, 2, 128), v=thd(0, 2, 128)) == ops.TM_OK


def test_python_checks_before_the_library():
    with pytest.raises(ValueError, match="CUDA"):
        ops.PagedKV(torch.zeros(2, 16, 2, 128, dtype=torch.float16), torch.zeros(2, 16, 2, 128, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        ops.rope(torch.zeros(2, 2, 128, dtype=torch.float16), rope=ops.Rope(128))
    with pytest.raises(ValueError, match="rope is for heads of 64"):
        ops.rope(torch.zeros(2, 2, 128, dtype=torch.float16), rope=ops.Rope(64))
    with pytest.raises(ValueError, match="weight"):
        ops.qk_norm_rope(torch.zeros(2, 2, 128, dtype=torch.float16), q_weight=None)
    k = torch.zeros(2, 16, 2, 128)
    with pytest.raises(ValueError, match="fp16 or int8"):
        ops.PagedKV(k, k)
    k = torch.zeros(2, 16, 2, 128, dtype=torch.int8)
    with pytest.raises(ValueError, match="scales"):
        ops.PagedKV(k, k)


def test_workspace_grows_with_the_rows_only():
    """The splits are bounded: the partial results stay within 64 slots of each row whatever the lengths."""
    rng = random.Random(1)
    for _ in range(200):
        hkv = rng.choice((1, 2, 8))
        hq = hkv * rng.randint(1, 16)
        batch, n = rng.randint(1, 300), rng.randint(1, 200)
        prefix, longest = rng.randint(0, 1 << 20), rng.randint(0, 1 << 20)
        d = rng.choice((64, 128))
        got = ops._lib().tm_attn_shared_prefix_workspace(batch * n, hq, hkv, d, batch, n, prefix, longest)
        assert 256 <= got <= 64 * batch * n * hq * (4 * d + 8) + 512
