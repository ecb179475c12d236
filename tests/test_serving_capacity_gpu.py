"""The serving operators on arrays of a fixed capacity: more rows than the sequences have, and
a promised N_max that says little about their lengths.

Tolerances: those of test_serving_gpu (their derivation stands there).
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from oracle import serving as ref
from tests.test_serving_gpu import (append_inputs, attend_inputs, check_attend, check_rule, host,
                                    ints, rule_inputs, run_append, run_attend)

pytestmark = pytest.mark.gpu


def padded(x, T):
    """The same call with arrays of T rows; the rows past the sequences' hold NaN."""
    def grow(t):
        if t is None:
            return None
        out = torch.full((T, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")
        out[:t.shape[0]] = t
        return out

    parent = np.full(T, -7, dtype=np.int32)
    parent[:len(x["parent"])] = x["parent"]
    return dict(x, q=grow(x["q"]), k=grow(x["k"]), v=grow(x["v"]), parent=parent)


@pytest.mark.parametrize("nodes,ctx,prefix,own", [
    # 4 query heads a key head: up to 4 rows are few, 5 are many
    ([8, 4], [30, 70], 0, True),
    ([20, 1, 4, 5, 0], [10, 300, 0, 64, 7], 0, True),
    ([20, 1, 4, 5, 0], [10, 300, 1, 64, 7], 33, False),
    ([20, 1, 4] * 4, [40, 3, 0] * 4, 6000, True),     # the prefix by units of its own
    ([60, 1, 4], [5000, 4000, 3], 0, True),           # keys in parts
    ([128, 1, 2, 3, 4, 5], [200, 9, 0, 1, 64, 65], 130, True),
])
@pytest.mark.parametrize("spare", [0, 37])
@pytest.mark.parametrize("tree", ["random", "chain"])
def test_attend_rows_of_a_full_capacity(nodes, ctx, prefix, own, spare, tree):
    """T = B * N_max rows (and more) say nothing of the sequences: short ones among long ones
    are computed all the same, and rows of no sequence are left alone."""
    x = attend_inputs(nodes, ctx, prefix, 8, 2, 128, 64, "bf16", seed=len(nodes) + prefix,
                      tree=tree, own=own)
    T, used = len(nodes) * max(nodes) + spare, sum(nodes)
    y = padded(x, T)
    o = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 8), 7.0, device="cuda")
    status = torch.full((len(nodes),), -7, dtype=torch.int32, device="cuda")
    run_attend(y, chain=tree == "chain", N_max=max(nodes), o=o, lse=lse, dev_status=status)
    assert (status == 0).all()
    check_attend(o[:used], lse[:used], x, chain=tree == "chain")
    assert (o[used:] == 7.0).all() and (lse[used:] == 7.0).all()


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("N", [1 << 20, INT_MAX])
def test_a_promise_past_the_rows_changes_nothing(N):
    """N_max is a bound, however loose: results and workspaces are those of min(N_max, T)."""
    x = rule_inputs([100, 0, 70], 2, 4, 128, 128, "bf16", seed=21)
    dims = lambda n: gt.Dims(3, n, 2, 4, 128, 128, gt.BF16)  # noqa: E731
    assert gt.prefill_workspace(dims(N), 170) == gt.prefill_workspace(dims(170), 170) > 0
    o, pool = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]),
                         x["pool"], state_slot=ints(x["slot"]), N_max=N)
    check_rule(o, pool, x)
    for case in (([1, 40, 3], [10, 130, 0], 77, 8, 2, 64, 16, "bf16"),
                 ([1, 40, 3], [10, 130, 0], 77, 6, 2, 64, 24, "f32"),
                 ([1], [300], 0, 32, 8, 128, 16, "bf16"),
                 ([1, 2], [0, 9], 0, 4, 4, 16, 16, "f32")):
        y = attend_inputs(*case, seed=22, tree="chain")
        status = torch.full((len(case[0]),), -7, dtype=torch.int32, device="cuda")
        o, lse = run_attend(y, chain=True, N_max=N, dev_status=status)
        assert (status == 0).all()
        check_attend(o, lse, y, chain=True)
    for Lmax in (None, 24):
        z = append_inputs([64, 3, 0], [0, 100, 7], 2, 64, 16, "bf16", seed=23, Lmax=Lmax)
        want = ref.cache_append(host(z["k"]), host(z["v"]), z["cu"], host(z["k_cache"]),
                                host(z["v_cache"]), z["table"], z["ctx"], z["path"], z["path_len"])
        new_len = run_append(z, N_max=N)
        assert np.array_equal(host(z["k_cache"]), want[0])
        assert np.array_equal(host(z["v_cache"]), want[1])
        assert new_len.tolist() == want[2].tolist()


def test_a_prompt_past_its_pages_is_reported():
    """More rows than the page table has room for: those that fit are written."""
    z = append_inputs([40, 5], [0, 3], 2, 64, 16, "bf16", seed=24)
    table = z["table"][:, :2].copy()  # room for 32 rows each
    before = z["k_cache"].clone()
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    run_append(dict(z, table=table), dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT, 0]
    for j in range(32):
        assert torch.equal(z["k_cache"][table[0, j // 16], j % 16], z["k"][j])
    third = int(z["table"][0, 2])
    assert torch.equal(z["k_cache"][third], before[third])


def test_row_offsets_that_wrap_are_reported():
    """Offsets whose 32-bit difference wraps to a small number are no sequence's rows."""
    cu = ints([0, INT_MAX, -2 ** 31, 7, 12])
    bad = [gt.STATUS_BAD_LAYOUT] * 3 + [0]
    for case in (([3, 3, 1, 5], [10, 5, 0, 20], 70, 8, 2, 64, 16, "bf16"),
                 ([30, 30, 10, 50], [10, 5, 0, 20], 70, 8, 2, 64, 16, "bf16"),
                 ([3, 3, 1, 5], [10, 5, 0, 20], 70, 8, 2, 64, 16, "f32")):
        x = attend_inputs(*case, seed=25, tree="chain")
        T = sum(case[0])
        offsets = ints([0, INT_MAX, -2 ** 31, T - case[0][-1], T])
        status = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        o = torch.full_like(x["q"], 7.0)
        gt.attend(x["q"], x["k"], x["v"], None, offsets, x["k_cache"], x["v_cache"],
                  ints(x["table"]), ints(x["ctx"]), prefix_pages=ints(x["prefix_pages"]),
                  prefix_len=x["prefix"], N_max=T, o=o, dev_status=status)
        assert status.tolist() == bad
        assert (o[:T - case[0][-1]] == 7.0).all()
        assert (o[T - case[0][-1]:] != 7.0).any()
    z = append_inputs([3, 3, 1, 5], [0, 9, 7, 2], 2, 64, 16, "bf16", seed=26)
    before, status = z["k_cache"].clone(), torch.empty(4, dtype=torch.int32, device="cuda")
    new_len = gt.cache_append(z["k"], z["v"], cu, z["k_cache"], z["v_cache"], ints(z["table"]),
                              ints(z["ctx"]), N_max=12, dev_status=status)
    assert status.tolist() == bad and new_len.tolist() == [0, 9, 7, 7]
    changed = (z["k_cache"] != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(z["table"][3, 0])]
    x = rule_inputs([40, 100, 10], 1, 2, 128, 128, "bf16", seed=27)
    status = torch.empty(3, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints([0, -2 ** 31, 140, 150]),
               x["pool"], state_slot=ints(x["slot"]), N_max=100, o=o, dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT] * 2 + [0]
    assert (o[:140] == 7.0).all() and (o[140:] != 7.0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_status_of_a_batch_without_rows(dtype):
    """The statuses of a call are its own, also where it has nothing to compute; a promise of no
    rows that the offsets break is reported like any other."""
    x = attend_inputs([0, 0], [3, 200], 40, 8, 2, 64, 16, dtype, seed=28)
    status = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    run_attend(x, N_max=1, dev_status=status)
    assert status.tolist() == [0, 0]
    y = attend_inputs([2, 0], [3, 200], 40, 8, 2, 64, 16, dtype, seed=29)
    o = torch.full_like(y["q"], 7.0)
    status.fill_(-7)
    run_attend(y, N_max=0, o=o, dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT, 0]
    assert (o == 7.0).all()
    run_attend(dict(y, cu=np.zeros(3, dtype=np.int32)), N_max=0, o=o, dev_status=status)
    assert status.tolist() == [0, 0]
    assert (o == 7.0).all()


@pytest.mark.parametrize("nodes,ctx,prefix,dtype", [
    ([60], [5000], 0, "bf16"),                        # keys in parts
    ([20, 1] * 6, [40] * 12, 6000, "bf16"),           # the prefix by units of its own
    ([60, 2], [300, 10], 0, "bf16"), ([2], [5000], 0, "bf16"), ([60], [500], 40, "f32")])
def test_rows_whose_query_is_nan(nodes, ctx, prefix, dtype):
    """All scores of such a row are NaN, in every part: so are its o and its lse."""
    x = attend_inputs(nodes, ctx, prefix, 8, 2, 128, 64, dtype, seed=30)
    good = run_attend(x)
    bad = [0, sum(nodes) - 1]
    x["q"][bad] = float("nan")
    o, lse = run_attend(x)
    rest = np.setdiff1d(np.arange(sum(nodes)), bad)
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(o[rest], good[0][rest]) and torch.equal(lse[rest], good[1][rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [[0, 3, 1], [0, 40, 30]])
def test_a_bad_page_of_the_prefix_is_told_to_all(nodes, dtype):
    x = attend_inputs(nodes, [9, 0, 20], 70, 8, 2, 64, 16, dtype, seed=34)
    pages = x["prefix_pages"].copy()
    pages[2] = -1
    status = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    run_attend(dict(x, prefix_pages=pages), dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT] * 3


@pytest.mark.parametrize("B,N,avg,Hv", [(1, 32768, 32768, 32), (16, 2048, 700, 32), (64, 512, 512, 32),
                                        (256, 512, 512, 32), (256, 2048, 2048, 32),
                                        (1024, 2048, 100, 32), (4096, 4096, 4096, 32),
                                        (300, 32768, 600, 32), (4096, 33, 33, 64), (1, 64, 64, 128)])
def test_prefill_workspace_is_bounded(B, N, avg, Hv):
    """512 MB, or what eight chunks of every sequence (fewer, where all have fewer) take."""
    T, head = B * avg, Hv * 50176
    need = gt.prefill_workspace(gt.Dims(B, N, Hv, Hv, 128, 128, gt.BF16), T)
    assert 0 < need <= max(512 << 20, head * min(8 * B, T // 64 + B + 1))
