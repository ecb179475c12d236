"""The operators in front of the attention on many rows: more than their numbers' 32 bits hold, and
more than the SMs take at once, where a warp's passes follow one another.

Tolerances, inputs and definitions are those of test_rope_gpu.
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from oracle import rope as ref
from tests.test_rope_gpu import append_inputs, check, host, ints, run_append, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at_the_end", [False, True])
def test_append_of_arrays_of_very_many_rows(at_the_end):
    """Arrays with room for 2^27 rows (32 threads each: 2^32 of them), of which a few hundred are
    in use: the first ones or the last.  The array's rows are one row that lies there once."""
    B, T, page, D = 300, (1 << 27) + 8, 4, 16
    lens, ctx = [b % 3 for b in range(B)], [b % 7 for b in range(B)]
    x = append_inputs(lens, ctx, 0, 1, D, D, page, "bf16", "same", "rms", seed=41, prefix=5)
    before, n = (x["k_cache"].clone(), x["v_cache"].clone()), sum(lens)
    first = T - n if at_the_end else 0
    kept = torch.full((3 * B,), -7, dtype=torch.int32, device="cuda")
    new_len, status = kept[B:2 * B], torch.full((B,), -7, dtype=torch.int32, device="cuda")
    big = dict(x, cu=x["cu"] + np.int32(first), k=x["k"][:1].expand(T, 1, D),
               v=x["v"][:1].expand(T, 1, D))
    run_append(big, False, new_len=new_len, dev_status=status, N_max=2)
    assert (status == 0).all() and (kept[:B] == -7).all() and (kept[2 * B:] == -7).all()
    assert new_len.tolist() == [c + m for c, m in zip(ctx, lens)]
    at, positions = ref.append_positions(x["cu"], x["ctx"], 5, n)
    k, size = want(x, "k", False, positions)
    kc = ref.place(host(before[0]), k, x["cu"], x["table"], x["ctx"])
    check(x["k_cache"], (kc, ref.place(np.zeros(kc.shape), size, x["cu"], x["table"], x["ctx"])),
          "bf16")
    vc = ref.place(host(before[1]), host(x["v"]), x["cu"], x["table"], x["ctx"])
    assert np.array_equal(host(x["v_cache"]), vc)
