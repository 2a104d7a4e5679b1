"""What pkv_attn_prefix would like as workspace goes by where its key rows lie, as its plan does: the query takes k_start."""
import ctypes

import pytest

import paged_kv_gqa_nx_gb300 as pkv

# (prefix, queries, own keys, rows a slot) of sequences in slots, heads: the same rows behind one another need less
SLOTS = [(753, [1] * 28, [1] * 28, 8, (64, 8, 128)), (994, [7, 30] * 10, [8, 30] * 10, 67, (16, 2, 128)),
         (3293, [1] * 66, [1 + i % 30 for i in range(66)], 31, (64, 8, 128)), (719, [4, 1, 2] * 22, [4, 1, 2] * 22, 20, (6, 2, 160)),
         (5016, [30, 11, 2, 7, 25], [300, 20, 2, 8, 25], 327, (32, 8, 128))]


def starts(n, room):
    return [i * room for i in range(n)]


def test_slots_are_another_plan():
    more = 0
    for prefix, ql, kl, room, heads in SLOTS:
        packed = pkv.pkv_attn_prefix_workspace(prefix, ql, kl, *heads)
        slots = pkv.pkv_attn_prefix_workspace(prefix, ql, kl, *heads, k_start=starts(len(ql), room))
        assert packed >= 0 and slots >= 0
        more += slots > packed
    assert more >= 2
    # 28 tokens behind 753 rows: none as rows behind one another, four records a query in slots of 8
    assert pkv.pkv_attn_prefix_workspace(*SLOTS[0][:3], *SLOTS[0][4]) == 0
    assert pkv.pkv_attn_prefix_workspace(*SLOTS[0][:3], *SLOTS[0][4], k_start=starts(28, 8)) >= 4 * 28 * 64 * 4 * (128 + 2)


@pytest.mark.parametrize("prefix,ql,kl,room,heads", SLOTS)
def test_rows_behind_one_another_are_the_default(prefix, ql, kl, room, heads):
    behind = [sum(kl[:i]) for i in range(len(kl))]
    plain = pkv.pkv_attn_prefix_workspace(prefix, ql, kl, *heads)
    assert pkv.pkv_attn_prefix_workspace(prefix, ql, kl, *heads, k_start=behind) == plain
    assert pkv.pkv_attn_prefix_workspace_at(prefix, ql, kl, None, *heads) == plain
    arr = lambda v: (ctypes.c_int32 * len(v))(*v)
    assert pkv._lib.pkv_attn_prefix_workspace(prefix, arr(ql), arr(kl), len(ql), *heads) == plain


def test_refusals():
    assert pkv.pkv_attn_prefix_workspace(100, [1, 1], [1, 1], 4, 2, 16, k_start=[0, -1]) == -1 and pkv.pkv_last_error()
    assert pkv.pkv_attn_prefix_workspace(100, [1, 1], [1, 1], 4, 2, 16, k_start=[0, 2 ** 31 - 1]) == -1
    with pytest.raises(TypeError, match="entry for each"):
        pkv.pkv_attn_prefix_workspace(100, [1, 1], [1, 1], 4, 2, 16, k_start=[0])


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,ql,kl,room,heads", SLOTS)
def test_a_call_in_slots_wants_no_more_than_it_asked_for(prefix, ql, kl, room, heads):
    """With the advised bytes a call is planned as with any number more: the same launches and the same bits."""
    import torch
    from ragged_helpers import Case
    c = Case(ql, kl, *heads, torch.bfloat16, prefix=prefix, k_start=starts(len(ql), room))
    advised = pkv.pkv_attn_prefix_workspace(prefix, ql, kl, *heads, k_start=c.k_start)
    outs, launches = [], []
    for size in (max(advised, 16), advised + (64 << 20)):
        n = pkv.pkv_launch_count()
        outs.append(c.call(workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda")))
        launches.append(pkv.pkv_launch_count() - n)
    c.check(got=outs[0])
    assert torch.equal(*outs) and launches[0] == launches[1]
