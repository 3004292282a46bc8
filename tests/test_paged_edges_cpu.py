"""CPU checks of the paged-cache operators at the edges of their contract."""

import os
import re

import pytest
import torch

from mixed_precision_attention_tm_b200 import build as tmbuild

tmbuild.build()
from mixed_precision_attention_tm_b200 import ops  # noqa: E402

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


def turn_program(t, segments, sync, arrive, last):
    """What softmax warpgroup t does at the turn barriers, over segments of so many turns each."""
    steps, owed = [], False
    for turns in segments:
        for c in range(turns):
            at = dict(c=c, t=t, turns=turns, owed=owed)
            if eval(sync, {}, at):
                steps.append(("sync", t))
            if eval(arrive, {}, at):
                steps.append(("arrive", 1 - t))
        if turns:
            owed = t == 0
        steps.append(("results", t))
    if last and owed:
        steps.append(("sync", t))
    return steps


def turn_faults(programs):
    """Every order of the two warpgroups' steps over barriers that complete with two arrivals, whoever's."""
    faults, seen, todo = set(), set(), [((0, 0), ((), ()), (False, False))]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, bars, waits = state
        moved = False
        for w in (0, 1):
            if waits[w] or at[w] == len(programs[w]):
                continue
            moved = True
            kind, b = programs[w][at[w]]
            at2, bars2, waits2 = list(at), [list(x) for x in bars], list(waits)
            if kind != "results":
                bars2[b].append((w, kind))
            if kind == "sync":
                waits2[w] = True
            else:
                at2[w] += 1
            if kind != "results" and len(bars2[b]) == 2:
                if {x for x, _ in bars2[b]} != {0, 1}:
                    faults.add("one warpgroup's arrivals complete a barrier")
                for x, k in bars2[b]:
                    if k == "sync":
                        waits2[x] = False
                        at2[x] += 1
                bars2[b] = []
            todo.append((tuple(at2), tuple(tuple(x) for x in bars2), tuple(waits2)))
        if not moved and (any(waits) or any(at[w] < len(programs[w]) for w in (0, 1))):
            faults.add("stuck")
        elif not moved and any(bars):
            faults.add("an arrival is left over")
    return faults


def test_tile_kernel_turns_over_several_segments():
    """The conditions of the kernel's turn barriers, in every order in which the two warpgroups may come to them."""
    text = source("tm_attn_shared_tile.cu")

    def conditions(call):
        return [c.replace("&&", "and").replace("||", "or")
                for c in re.findall(r"if \((.+)\) named_bar_" + call + r", 256\);", text)]
    syncs, arrives = conditions(r"sync\(NB_TURN \+ t"), conditions(r"arrive\(NB_TURN \+ 1 - t")
    assert len(arrives) == 1 and syncs[1:] in ([], ["owed"])
    for segments in ([2], [2, 2], [4, 2, 0, 2], [0, 2, 0, 4], [2, 0, 0, 2, 2]):
        programs = [turn_program(t, segments, syncs[0], arrives[0], len(syncs) == 2) for t in (0, 1)]
        assert turn_faults(programs) == set(), segments


class Pages:
    """What the workspace query reads of a PagedKV."""
    H, d = 8, 128


def test_workspace_with_a_loose_bound_of_the_rows():
    """No sequence has more rows than the batch: a larger max_seqlen is the same call, past 32 bits too."""
    def size(n, batch=64, T=64, Hq=32):
        return ops.shared_prefix_workspace_bytes(Pages, batch, T, Hq, max_seqlen=n, prefix_len=1000, max_kv_len=4096)
    for n in (65, 8192, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 40):
        assert size(n) == size(64)
    wide = Pages()
    wide.H = 1
    for n in (3, 2 ** 31 - 1):
        a = ops.shared_prefix_workspace_bytes(wide, 1, 2, 4096, max_seqlen=n, max_kv_len=1 << 20)
        assert a == ops.shared_prefix_workspace_bytes(wide, 1, 2, 4096, max_seqlen=2, max_kv_len=1 << 20)


def test_launches_whose_items_pass_32_bits_are_refused():
    """A block of the tile kernel goes from item to item in steps of the grid: the last step stays below 2^31 too."""
    few = Pages()
    few.H = 63
    for batch, fits in ((34087042, False), (34087040, False), (34000000, True)):       # 63 items each: 2^31 - 2, 2^31 - 128
        def size():
            return ops.shared_prefix_workspace_bytes(few, batch, 100, 63, max_seqlen=100, max_kv_len=64)
        if fits:
            assert size() > 0
        else:
            with pytest.raises(ValueError):
                size()


def test_block_table_check_of_64_bit_tables():
    """Page numbers and lengths past 32 bits are what they are, not what is left of them."""
    ops.block_table_check(torch.tensor([[3, 1]]), torch.tensor([32]), 4, 16)
    for page in (2 ** 32 + 1, 2 ** 32, -2 ** 32 + 3, 2 ** 31, -1, 2 ** 63 - 1):
        with pytest.raises(ValueError, match="sequence 0, column 1"):
            ops.block_table_check(torch.tensor([[3, page]]), torch.tensor([32]), 4, 16)
        with pytest.raises(ValueError, match="sequence 0, column 1"):
            ops.block_table_check([[3, page]], [32], 4, 16)
        ops.block_table_check(torch.tensor([[3, page]]), torch.tensor([16]), 4, 16)
    for n in (33, 2 ** 31, 2 ** 32, 2 ** 32 + 16, 2 ** 63 - 1):
        with pytest.raises(ValueError, match="sequence 0, column 2"):
            ops.block_table_check(torch.tensor([[3, 1]]), torch.tensor([n]), 4, 16)
    ops.block_table_check(torch.tensor([[3, 1]]), torch.tensor([-2 ** 32 + 33]), 4, 16)      # empty


def test_workspace_of_no_sequences_is_refused():
    for batch in (0, -1):
        for n in (None, 4):
            with pytest.raises(ValueError):
                ops.shared_prefix_workspace_bytes(Pages, batch, 8, 32, max_seqlen=n, max_kv_len=64)
