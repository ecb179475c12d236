"""The bounded on-device waits of the serving kernels, made to run out on purpose (no fault, no
trap): a short wait limit and an arrival that is withheld, test-only controls read from the
environment.  The call must report GDN_TREE_STATUS_TIMEOUT for the sequences that it could not
finish, leave the others right, and leave the context usable."""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from tests.test_serving_gpu import (EPS_BF16, TOL_F32, attend_inputs, check_attend, check_rule,
                                    host, ints, max_err, rule_inputs, rule_ref, run_attend)

pytestmark = pytest.mark.gpu


@pytest.fixture
def short_waits(monkeypatch):
    monkeypatch.setenv("GDN_TREE_TEST_WAIT_LIMIT_NS", "1000000")  # 1 ms
    return monkeypatch


ATTEND = [
    # fewer units than SMs: each has a CTA of its own
    ([60, 70, 90], [600, 300, 0], 0, 16, 4, 128, 64, "bf16"),    # two row tiles
    ([20, 30, 17], [600, 300, 0], 100, 8, 4, 64, 16, "bf16"),    # one, its key tiles by turns
    ([60, 70, 30], [600, 300, 0], 0, 4, 2, 96, 24, "bf16"),      # rows without TMA
    ([30, 40, 20], [5000, 300, 0], 0, 8, 4, 128, 128, "bf16"),   # keys in parts
]


@pytest.mark.parametrize("case", ATTEND, ids=["two-tiles", "one-tile", "no-tma", "parts"])
@pytest.mark.parametrize("warp", [0, 13])
def test_attention_wait_runs_out(short_waits, case, warp):
    x = attend_inputs(*case, seed=41)
    hkv, b = case[4], 1
    short_waits.setenv("GDN_TREE_TEST_WITHHOLD_NODE", f"{b * hkv + 1}:{warp}")
    status = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    o, lse = run_attend(x, dev_status=status)
    assert status.tolist() == [0, gt.STATUS_TIMEOUT, 0]
    rows = np.flatnonzero(np.repeat([True, False, True], case[0]))
    check_attend(o, lse, x, rows=rows)
    short_waits.undo()
    o, lse = run_attend(x, dev_status=status)
    assert status.tolist() == [0, 0, 0]
    check_attend(o, lse, x)


def test_shared_prefix_wait_runs_out(short_waits):
    """A unit of the shared prefix holds rows of several sequences: all of them are told."""
    x = attend_inputs([1] * 30, [5] * 30, 4000, 16, 4, 128, 128, "bf16", seed=42)
    short_waits.setenv("GDN_TREE_TEST_WITHHOLD_NODE", "2:3")
    status = torch.full((30,), -7, dtype=torch.int32, device="cuda")
    run_attend(x, dev_status=status)
    assert status.tolist() == [gt.STATUS_TIMEOUT] * 30
    short_waits.undo()
    o, lse = run_attend(x, dev_status=status)
    assert status.tolist() == [0] * 30
    check_attend(o, lse, x)


@pytest.mark.parametrize("what", ["copy", "arrival"])
@pytest.mark.parametrize("lens,Hqk,Hv", [([200, 130, 64], 2, 4), ([200] * 5, 16, 32)],
                         ids=["one-chain", "two-chains"])
def test_prefill_wait_runs_out(short_waits, what, lens, Hqk, Hv):
    x = rule_inputs(lens, Hqk, Hv, 128, 128, "bf16", seed=43)
    B, b = len(lens), 1
    if what == "copy":
        short_waits.setenv("GDN_TREE_TEST_WITHHOLD_COPY", str(b))
    else:
        short_waits.setenv("GDN_TREE_TEST_WITHHOLD_NODE", f"{b * Hv + 3}:5")
    args = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")] + [ints(x["cu"]), x["pool"]]
    status = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    out = x["pool"].clone()
    o, pool = gt.prefill(*args, state_slot=ints(x["slot"]), pool_out=out, dev_status=status)
    assert status.tolist() == [gt.STATUS_TIMEOUT if i == b else 0 for i in range(B)]
    ro, rp = rule_ref(x)
    o, pool = host(o), host(pool)
    for i in range(B):
        if i == b:
            continue
        rows, slot = slice(x["cu"][i], x["cu"][i + 1]), x["slot"][i]
        assert max_err(pool[slot], rp[slot]) <= TOL_F32
        assert (np.abs(o[rows] - ro[rows]) <= EPS_BF16 * np.abs(ro[rows])
                + TOL_F32 * np.abs(ro).max()).all()
    if what == "arrival":  # the state of the head is left unwritten
        assert (pool[x["slot"][b], 3] == host(x["pool"])[x["slot"][b], 3]).all()
    short_waits.undo()
    o, pool = gt.prefill(*args, state_slot=ints(x["slot"]), dev_status=status)
    assert (status == 0).all()
    check_rule(o, pool, x)
