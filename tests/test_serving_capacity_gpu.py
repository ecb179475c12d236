"""The serving operators on arrays of a fixed capacity: more rows than the sequences have, and
a promised N_max that says little about their lengths.

Tolerances: those of test_serving_gpu (their derivation stands there).
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from tests.test_serving_gpu import attend_inputs, check_attend, run_attend

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
