"""Serving operators over a paged K/V cache: the cases that are measured.

Five operators around one cache: rotary positions (``rope``), norms of
queries and keys with the rotation (``norm``), appending rotated keys and
values to pages (``append``), pages read back as contiguous rows (``gather``)
and attention for a batch that shares a long prefix (``attend``).

Sequence lengths follow from the case alone (``_lens``); a seed draws the
values, the positions and which pages a sequence owns.
"""

import math

import torch

own = False

GROUPS = ((32, 8), (32, 4), (16, 16), (16, 2), (24, 8), (28, 4), (8, 1))   # (query heads, K/V heads)


def listed():
    return [
        # one decoding step of a small batch: latency
        dict(name="rope_step", op="rope", tokens=16, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             scaling="none", factor=1.0, far=8192),
        # a long prompt, half of the head rotated in the interleaved layout, positions far past the first training length
        dict(name="rope_prompt", op="rope", tokens=16384, hq=32, hkv=8, d=128, rot=64, interleaved=True,
             scaling="yarn", factor=32.0, far=131072),
        # one decoding step of a full batch with normed queries and keys
        dict(name="norm_step", op="norm", tokens=64, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             scaling="bands", factor=8.0, far=65536),
        # a prompt of an odd length, heads of 64
        dict(name="norm_prompt", op="norm", tokens=8191, hq=32, hkv=8, d=64, rot=64, interleaved=False,
             scaling="ntk", factor=4.0, far=32768),
        # one new token for each of 64 sequences
        dict(name="append_step", op="append", batch=64, new_lo=1, new_hi=1, old_lo=100, old_hi=1000, hq=32, hkv=8,
             d=128, rot=128, interleaved=False, scaling="none", factor=1.0, page=16, int8=False, norm=True, prefix=4096),
        # ragged chunks of prompts into an INT8 cache, then the whole context read back for the prefill attention
        dict(name="append_prompt_int8", op="append", batch=7, new_lo=700, new_hi=2048, old_lo=0, old_hi=4000, hq=32,
             hkv=4, d=128, rot=128, interleaved=True, scaling="linear", factor=2.0, page=64, int8=True, norm=False,
             prefix=0),
        # short contexts, small heads
        dict(name="gather_short", op="gather", batch=5, len_lo=33, len_hi=700, hkv=8, d=64, page=16, int8=False),
        # ragged long contexts of a prefill over cached tokens
        dict(name="gather_long", op="gather", batch=8, len_lo=1024, len_hi=16001, hkv=8, d=128, page=32, int8=False),
        # a few users behind one system prompt: latency
        dict(name="attend_small", op="attend", batch=4, lq_lo=1, lq_hi=1, prefix=1000, len_lo=17, len_hi=130, hq=32,
             hkv=8, d=128, page=16, int8=False),
        # a full batch behind one long document
        dict(name="attend_batch", op="attend", batch=64, lq_lo=1, lq_hi=1, prefix=32768, len_lo=64, len_hi=1024, hq=32,
             hkv=8, d=128, page=64, int8=False),
        # the same kind of batch over an INT8 cache, with answers as long as the prompts
        dict(name="attend_int8", op="attend", batch=32, lq_lo=1, lq_hi=1, prefix=16383, len_lo=200, len_hi=4096, hq=32,
             hkv=4, d=128, page=32, int8=True),
        # many questions' prompts of odd lengths on top of the shared document
        dict(name="attend_chunk", op="attend", batch=16, lq_lo=65, lq_hi=160, prefix=16384, len_lo=65, len_hi=600,
             hq=32, hkv=8, d=128, page=64, int8=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "norm", "append", "gather", "attend", "attend", "attend"))
    hq, hkv = rng.choice(GROUPS)
    d = rng.choice((64, 128))
    turn = dict(rot=16 * rng.randint(1, d // 16) if rng.random() < 0.4 else d, interleaved=rng.random() < 0.5,
                scaling=rng.choice(("none", "linear", "ntk", "yarn", "bands")), factor=float(rng.choice((2, 4, 8, 32))))
    if op in ("rope", "norm"):
        return dict(op=op, tokens=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, far=_log(rng, 20000, 1000000), **turn)
    page, int8 = rng.choice((16, 32, 64, 128)), rng.random() < 0.4
    if op == "append":
        new = _log(rng, 1, 2000)
        old = _log(rng, 1, 4000)
        batch = min(_log(rng, 1, 64), max(1, 20000 // (new + old)))
        return dict(op=op, batch=batch, new_lo=(new + 1) // 2, new_hi=new, old_lo=old // 3, old_hi=old, hq=hq, hkv=hkv,
                    d=d, page=page, int8=int8, norm=rng.random() < 0.5, prefix=_log(rng, 1, 30000), **turn)
    if op == "gather":
        n = _log(rng, 1, 16000)
        return dict(op=op, batch=min(_log(rng, 1, 64), max(1, 64000 // n)), len_lo=n // 5, len_hi=n, hkv=hkv, d=d,
                    page=page, int8=int8)
    batch = _log(rng, 1, 64)
    lq = 1 if rng.random() < 0.6 else min(_log(rng, 2, 128), max(1, 2000 // batch))
    n = lq + _log(rng, 1, 2000)
    return dict(op=op, batch=batch, lq_lo=(lq + 1) // 2, lq_hi=lq, prefix=_log(rng, 40, 30000), len_lo=lq + (n - lq) // 8,
                len_hi=n, hq=hq, hkv=hkv, d=d, page=page, int8=int8)


# ------------------------------------------------------------------ inputs
def _lens(n, lo, hi):
    """n lengths spread over lo..hi, both ends among them where n allows."""
    if n == 1:
        return [hi]
    order = [(i * 0.6180339887498949) % 1.0 for i in range(n)]
    rank = {i: r for r, i in enumerate(sorted(range(n), key=order.__getitem__))}
    return [lo + (hi - lo) * rank[i] // (n - 1) for i in range(n)]


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _turn_args(case):
    """Arguments of the rotation as a user gives them."""
    return dict(rot_dim=case["rot"], theta=10000.0, interleaved=case["interleaved"],
                scaling=None if case["scaling"] == "none" else case["scaling"], factor=case["factor"],
                original_max=4096)


def _frequencies(case):
    """(angle per position of each pair, multiplier of the rotated part), 64 bits."""
    rot, theta, factor, first = case["rot"], 10000.0, case["factor"], 4096.0
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    kind = case["scaling"]
    if kind == "ntk" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "yarn":
        def dim(turns):
            return rot * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if kind == "bands":
        smooth = ((first * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f / factor * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


def _rows(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32).to(torch.float16)


def _quantised(x):
    """INT8 codes and fp16 scales of each row: scale = fp16(amax / 127)."""
    x = x.float()
    scale = (x.abs().amax(-1) / 127.0).half()
    s = scale.float()[..., None]
    codes = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0).round().clamp(-127, 127).to(torch.int8)
    return codes, scale


def _pool(case, g, lens, shared):
    """A page pool that holds sequences of `lens` tokens and one of `shared`: (state, table, shared pages)."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [-(-n // page) for n in lens]
    first = -(-shared // page)
    total = first + sum(need) + 3
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(lens), max(max(need), 1), dtype=torch.int32, device="cuda")
    at = first
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    k, v = (_rows(g, total, page, hkv, d) for _ in range(2))
    if case["int8"]:
        kc, ks = _quantised(k)
        vc, vs = _quantised(v)
        pool = dict(k=kc, v=vc, ks=ks, vs=vs)
    else:
        pool = dict(k=k, v=v, ks=None, vs=None)
    return pool, table, ids[:first].clone()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    op, d = case["op"], case["d"]
    if own:
        from mixed_precision_attention_tm_b200 import ops
        s["ops"] = ops
    if op in ("rope", "norm"):
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        s["q"], s["k"] = _rows(g, t, hq, d), _rows(g, t, hkv, d)
        if t > 256:      # a prompt: one run of positions that ends at `far`
            s["pos"] = torch.arange(t, device="cuda", dtype=torch.int32) + (max(case["far"] - t, 0))
        else:            # a step: every row is another sequence's newest token
            s["pos"] = torch.randint(0, case["far"], (t,), device="cuda", generator=g).to(torch.int32)
        s["out"] = (torch.empty_like(s["q"]), torch.empty_like(s["k"]))
        if op == "norm":
            s["qw"], s["kw"] = (1.0 + 0.2 * _rows(g, d) for _ in range(2))
        if own:
            s["rope"] = ops.Rope(d, **_turn_args(case))
    elif op == "append":
        n, hq, hkv = case["batch"], case["hq"], case["hkv"]
        new, old = _lens(n, case["new_lo"], case["new_hi"]), _lens(n, case["old_lo"], case["old_hi"])
        s["lens"] = [a + b for a, b in zip(new, old)]
        s["new"] = new
        s["pool"], s["table"], _ = _pool(case, g, s["lens"], 0)
        t = sum(new)
        s["q"], s["k"], s["v"] = _rows(g, t, hq, d), _rows(g, t, hkv, d), _rows(g, t, hkv, d)
        s["kv_lens"] = _ints(s["lens"])
        s["cu"] = _ints(_offsets(new))
        s["cu_all"] = _ints(_offsets(s["lens"]))
        s["qw"], s["kw"] = ((1.0 + 0.2 * _rows(g, d) for _ in range(2)) if case["norm"] else (None, None))
        s["q_out"] = torch.empty_like(s["q"])
        if case["int8"]:
            s["rows"] = tuple(torch.empty(sum(s["lens"]), hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
        if own:
            p = s["pool"]
            s["rope"] = ops.Rope(d, **_turn_args(case))
            s["kv"] = ops.PagedKV(p["k"], p["v"], p["ks"], p["vs"])
    elif op == "gather":
        s["lens"] = _lens(case["batch"], case["len_lo"], case["len_hi"])
        s["pool"], s["table"], _ = _pool(case, g, s["lens"], 0)
        s["cu_all"] = _ints(_offsets(s["lens"]))
        s["rows"] = tuple(torch.empty(sum(s["lens"]), case["hkv"], d, dtype=torch.float16, device="cuda") for _ in range(2))
        if own:
            p = s["pool"]
            s["kv"] = ops.PagedKV(p["k"], p["v"], p["ks"], p["vs"])
    else:
        n, hq = case["batch"], case["hq"]
        s["lq"] = _lens(n, case["lq_lo"], case["lq_hi"])
        s["lens"] = [max(a, b) for a, b in zip(_lens(n, case["len_lo"], case["len_hi"]), s["lq"])]
        s["pool"], s["table"], s["prefix_pages"] = _pool(case, g, s["lens"], case["prefix"])
        s["q"] = (2.0 * _rows(g, sum(s["lq"]), hq, d).float()).half()
        s["kv_lens"], s["cu"] = _ints(s["lens"]), _ints(_offsets(s["lq"]))
        s["out"] = torch.empty_like(s["q"])
        if own:
            p = s["pool"]
            s["kv"] = ops.PagedKV(p["k"], p["v"], p["ks"], p["vs"])
            s["max_q"], s["max_len"] = max(s["lq"]), max(s["lens"])
            s["workspace"] = torch.empty(
                ops.shared_prefix_workspace_bytes(s["kv"], n, sum(s["lq"]), hq, max_seqlen=s["max_q"],
                                                  prefix_len=case["prefix"], max_kv_len=s["max_len"]),
                dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _turned(x, pos, case):
    """The rotation of x [T, H, d] (32 bits) at pos [T]."""
    f, mul = _frequencies(case)
    ang = pos.double()[:, None] * f.to(pos.device)
    c, sn = (ang.cos() * mul).float()[:, None], (ang.sin() * mul).float()[:, None]
    rot = case["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((y, rest), -1)


def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _places(s, lens, width):
    """Pool slot of position j of each sequence, [B, width]; positions past the table's end repeat its last."""
    page = s["case"]["page"]
    j = torch.arange(width, device="cuda")
    col = (j // page).clamp(max=s["table"].shape[1] - 1)
    return s["table"].long()[:, col] * page + j % page


def _values(pool, which, slots):
    """The pool's rows at `slots` in 32 bits."""
    x = pool[which].flatten(0, 1)[slots].float()
    if pool["ks"] is not None:
        x = x * pool[which + "s"].flatten(0, 1)[slots].float()[..., None]
    return x


def _sequence_of(cu, t):
    """(sequence, place in it) of rows 0..t of a packed batch."""
    row = torch.arange(t, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, row, right=True) - 1
    return b, (row - cu[b]).long()


def _plain_gather(s):
    b, j = _sequence_of(s["cu_all"], s["rows"][0].shape[0])
    page = s["case"]["page"]
    slots = s["table"].long()[b, j // page] * page + j % page
    return tuple(_values(s["pool"], w, slots).half() for w in ("k", "v"))


def _plain_append(s):
    case, pool = s["case"], s["pool"]
    b, i = _sequence_of(s["cu"], s["q"].shape[0])
    lens, new = s["kv_lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    j = lens[b] - new[b] + i
    slots = s["table"].long()[b, j // case["page"]] * case["page"] + j % case["page"]
    q, k = s["q"].float(), s["k"].float()
    if case["norm"]:
        q, k = _normed(q, s["qw"]), _normed(k, s["kw"])
    pos = j + case["prefix"]
    q, k, v = _turned(q, pos, case), _turned(k, pos, case), s["v"].float()
    if not case["int8"]:
        pool["k"].flatten(0, 1)[slots] = k.half()
        pool["v"].flatten(0, 1)[slots] = v.half()
        return q.half(), pool["k"], pool["v"]
    for name, x in (("k", k), ("v", v)):
        codes, scale = _quantised(x)
        pool[name].flatten(0, 1)[slots] = codes
        pool[name + "s"].flatten(0, 1)[slots] = scale
    return (q.half(), *_plain_gather(s))


def _plain_attend(s):
    case, pool = s["case"], s["pool"]
    hq, hkv, d, page, p = case["hq"], case["hkv"], case["d"], case["page"], case["prefix"]
    g, n, t = hq // hkv, case["batch"], s["q"].shape[0]
    q = s["q"].float() / math.sqrt(d)
    # the shared prefix: every row of the batch against it in one product
    at = torch.arange(p, device="cuda")
    slots = s["prefix_pages"].long()[at // page] * page + at % page
    kp, vp = (_values(pool, w, slots).transpose(0, 1) for w in ("k", "v"))               # [hkv, p, d]
    rows = q.view(t, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, t * g, d)
    sp = rows @ kp.transpose(1, 2)
    mp = sp.amax(-1, keepdim=True)
    ep = torch.exp(sp.sub_(mp))
    lp, op = ep.sum(-1, keepdim=True), ep @ vp
    del sp, ep
    mp, lp, op = (x.view(hkv, t, g, -1).permute(1, 0, 2, 3) for x in (mp, lp, op))      # [t, hkv, g, .]
    # own tokens, padded to the longest sequence
    lq, width = max(s["lq"]), max(s["lens"])
    b, i = _sequence_of(s["cu"], t)
    padded = torch.zeros(n, lq, hkv, g, d, device="cuda")
    padded[b, i] = q.view(t, hkv, g, d)
    slots = _places(s, s["lens"], width)
    ko, vo = (_values(pool, w, slots).transpose(1, 2) for w in ("k", "v"))              # [n, hkv, width, d]
    padded = padded.permute(0, 2, 1, 3, 4).reshape(n, hkv, lq * g, d)
    so = (padded @ ko.transpose(2, 3)).view(n, hkv, lq, g, width)
    lens, new = s["kv_lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    j = torch.arange(width, device="cuda")
    last = (lens - new)[:, None] + torch.arange(lq, device="cuda")                       # [n, lq]
    seen = (j <= last[..., None]) & (j < lens[:, None, None])
    so = so.masked_fill_(~seen[:, None, :, None], -torch.inf)
    mo = so.amax(-1, keepdim=True).clamp(min=-1e30)
    eo = torch.exp(so.sub_(mo))
    lo = eo.sum(-1, keepdim=True)
    oo = (eo.view(n, hkv, lq * g, width) @ vo).view(n, hkv, lq, g, d)
    mo, lo, oo = (x.permute(0, 2, 1, 3, 4)[b, i] for x in (mo, lo, oo))                  # [t, hkv, g, .]
    m = torch.maximum(mp, mo)
    wp, wo = torch.exp(mp - m), torch.exp(mo - m)
    return ((op * wp + oo * wo) / (lp * wp + lo * wo)).reshape(t, hq, d).half()


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        ops = s["ops"]
        if op == "rope":
            return ops.rope(s["q"], s["k"], rope=s["rope"], positions=s["pos"], out=s["out"])
        if op == "norm":
            return ops.qk_norm_rope(s["q"], s["k"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, rope=s["rope"],
                                    positions=s["pos"], out=s["out"])
        if op == "append":
            q = ops.kv_append(s["k"], s["v"], s["kv"], s["table"], s["kv_lens"], cu_seqlens=s["cu"], rope=s["rope"],
                              pos_offset=case["prefix"], q=s["q"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                              q_out=s["q_out"])
            if not case["int8"]:
                return q, s["pool"]["k"], s["pool"]["v"]
            return (q, *ops.kv_gather(s["kv"], s["table"], s["cu_all"], out=s["rows"]))
        if op == "gather":
            return ops.kv_gather(s["kv"], s["table"], s["cu_all"], out=s["rows"])
        return ops.attn_shared_prefix(s["q"], s["kv"], s["table"], s["kv_lens"], prefix_pages=s["prefix_pages"],
                                      prefix_len=case["prefix"], cu_seqlens=s["cu"], max_seqlen=s["max_q"],
                                      max_kv_len=s["max_len"], workspace=s["workspace"], out=s["out"])
    if op in ("rope", "norm"):
        q, k = s["q"].float(), s["k"].float()
        if op == "norm":
            q, k = _normed(q, s["qw"]), _normed(k, s["kw"])
        return _turned(q, s["pos"], case).half(), _turned(k, s["pos"], case).half()
    if op == "append":
        return _plain_append(s)
    if op == "gather":
        return _plain_gather(s)
    return _plain_attend(s)


# ------------------------------------------------------------------- work
def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    held = hkv * (d + 2 if case.get("int8") else 2 * d)      # one token's K or V in the cache
    if op in ("rope", "norm"):
        t, heads = case["tokens"], case["hq"] + hkv
        return dict(bytes=t * heads * d * 4 + 4 * t, flops=t * heads * d * (3 if op == "rope" else 7))
    if op == "append":
        new = sum(_lens(case["batch"], case["new_lo"], case["new_hi"]))
        n = new * (case["hq"] * d * 4 + 2 * hkv * d * 2 + 2 * held)
        if case["int8"]:
            n += (new + sum(_lens(case["batch"], case["old_lo"], case["old_hi"]))) * 2 * (held + hkv * d * 2)
        return dict(bytes=n, flops=new * (case["hq"] + hkv) * d * 3)
    if op == "gather":
        n = sum(_lens(case["batch"], case["len_lo"], case["len_hi"]))
        return dict(bytes=n * 2 * (held + hkv * d * 2), flops=0)
    lq = _lens(case["batch"], case["lq_lo"], case["lq_hi"])
    lens = [max(a, b) for a, b in zip(_lens(case["batch"], case["len_lo"], case["len_hi"]), lq)]
    pairs = sum(a * (case["prefix"] + n - a) + a * (a + 1) // 2 for a, n in zip(lq, lens))
    return dict(bytes=(case["prefix"] + sum(lens)) * 2 * held + sum(lq) * case["hq"] * d * 4,
                flops=4 * d * case["hq"] * pairs)


# ------------------------------------------------------- 64-bit definitions
def _exact_phase(case, pos):
    """mul * e^(i angle) of each pair at each position, complex 128 bits: angles one pair at a time."""
    rot, factor, kind = case["rot"], case["factor"], case["scaling"]
    mul, freq = 1.0, []
    for pair in range(rot // 2):
        base = 10000.0 * (factor ** (rot / (rot - 2)) if kind == "ntk" and rot > 2 else 1.0)
        w = math.exp(-2.0 * pair / rot * math.log(base))
        if kind == "linear":
            w /= factor
        elif kind == "yarn":
            mul = 1.0 + math.log(factor) / 10.0
            ends = [rot * math.log(4096.0 / (n * 2.0 * math.pi)) / (2.0 * math.log(10000.0)) for n in (32.0, 1.0)]
            lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
            share = min(max((pair - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = w * (1.0 - share) + w * share / factor
        elif kind == "bands":
            turns = 4096.0 * w / (2.0 * math.pi)         # turns over the first training length
            w = w if turns > 4.0 else w / factor if turns < 1.0 else (
                w / factor + (turns - 1.0) / 3.0 * (w - w / factor))
        freq.append(w)
    ang = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device=pos.device))
    return torch.polar(torch.full_like(ang, mul), ang)


def _exact_turn(x, z, case):
    rot = case["rot"]
    y = x.clone()
    if case["interleaved"]:
        pairs = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * z[:, None]
        y[..., :rot] = torch.view_as_real(pairs).flatten(-2)
    else:
        pairs = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z[:, None]
        y[..., :rot // 2], y[..., rot // 2:rot] = pairs.real, pairs.imag
    return y


def _exact_norm(x, w):
    return x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + 1e-6).sqrt() * w.double()


def _exact_rows(s, b, n, which):
    """Positions 0..n of sequence b (None: of the shared prefix) as 64-bit values."""
    page, pool = s["case"]["page"], s["pool"]
    pages = (s["prefix_pages"] if b is None else s["table"][b])[:-(-n // page)].long()
    x = pool[which][pages].double()
    if pool["ks"] is not None:
        x = x * pool[which + "s"][pages].double()[..., None]
    return x.flatten(0, 1)[:n]


def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    op = case["op"]
    if op in ("rope", "norm"):
        z = _exact_phase(case, s["pos"])
        q, k = s["q"].double(), s["k"].double()
        if op == "norm":
            q, k = _exact_norm(q, s["qw"]), _exact_norm(k, s["kw"])
        return _exact_turn(q, z, case), _exact_turn(k, z, case)
    if op == "gather":
        return tuple(torch.cat([_exact_rows(s, b, n, w) for b, n in enumerate(s["lens"])]) for w in ("k", "v"))
    if op == "append":
        old = [n - a for n, a in zip(s["lens"], s["new"])]
        at = torch.cat([torch.arange(o, n, device="cuda") for o, n in zip(old, s["lens"])])
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        if case["norm"]:
            q, k = _exact_norm(q, s["qw"]), _exact_norm(k, s["kw"])
        z = _exact_phase(case, at + case["prefix"])
        q, k = _exact_turn(q, z, case), _exact_turn(k, z, case)
        if case["int8"]:
            def held(x):      # what the codes and the fp16 scale of each row stand for
                scale = (x.abs().amax(-1, keepdim=True) / 127).half().double()
                return torch.where(scale > 0, (x / scale).round().clamp(-127, 127) * scale, 0.0)
            k, v, got, first = held(k), held(v), [], 0
            for w, x in (("k", k), ("v", v)):
                parts, first = [], 0
                for b, (o, a) in enumerate(zip(old, s["new"])):
                    parts += [_exact_rows(s, b, o, w), x[first:first + a]]
                    first += a
                got.append(torch.cat(parts))
            return (q, *got)
        pools = [s["pool"][w].double() for w in ("k", "v")]
        first = 0
        for b, (o, a) in enumerate(zip(old, s["new"])):
            for place in range(o // case["page"], -(-(o + a) // case["page"])):   # page by page
                lo, hi = max(o, place * case["page"]), min(o + a, (place + 1) * case["page"])
                for pool, x in zip(pools, (k, v)):
                    page = int(s["table"][b, place])
                    pool[page, lo - place * case["page"]:hi - place * case["page"]] = x[first + lo - o:first + hi - o]
            first += a
        return (q, *pools)
    hkv, g, d, p = case["hkv"], case["hq"] // case["hkv"], case["d"], case["prefix"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    shared = [_exact_rows(s, None, p, w) for w in ("k", "v")]
    first = 0
    for b, (a, n) in enumerate(zip(s["lq"], s["lens"])):
        mine = [_exact_rows(s, b, n, w) for w in ("k", "v")]
        hidden = torch.arange(n, device="cuda") > (n - a) + torch.arange(a, device="cuda")[:, None]
        hidden = torch.cat((torch.zeros(a, p, dtype=torch.bool, device="cuda"), hidden), 1)
        for h in range(hkv):
            k, v = (torch.cat((x[:, h], y[:, h])) for x, y in zip(shared, mine))
            q = s["q"][first:first + a, h * g:(h + 1) * g].double()
            score = torch.einsum("agd,kd->agk", q, k) * d ** -0.5
            w = score.masked_fill(hidden[:, None], -torch.inf).softmax(-1)
            out[first:first + a, h * g:(h + 1) * g] = torch.einsum("agk,kd->agd", w, v)
        first += a
    return out
