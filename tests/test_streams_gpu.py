"""Calls with `stream=` and nothing else given: the workspace, the copies of the states and the
outputs that the binding makes are safe from what the current stream does next."""

import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from tests.test_serving_gpu import append_inputs, attend_inputs, cu_of, ints, rule_inputs

pytestmark = pytest.mark.gpu


def litter():
    """Allocations of many sizes on the current stream, filled with NaN (all bits set)."""
    for _ in range(3):
        for p in range(9, 28):
            torch.empty(1 << p, dtype=torch.uint8, device="cuda").fill_(255)
            torch.empty((1 << p) + (1 << (p - 1)), dtype=torch.uint8, device="cuda").fill_(255)


def calls():
    x = rule_inputs([2000, 500, 33], 4, 8, 128, 128, "bf16", seed=31)
    rule = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    cu, slot = ints(x["cu"]), ints(x["slot"])
    yield lambda **k: gt.prefill(*rule, cu, x["pool"], state_slot=slot, **k)
    one = [t[:3].contiguous() for t in rule]
    yield lambda **k: gt.decode_step(*one, x["pool"], state_slot=slot, **k)
    y = attend_inputs([60, 30], [6000, 3000], 500, 8, 2, 128, 64, "bf16", seed=32)
    table, ctx, pre = ints(y["table"]), ints(y["ctx"]), ints(y["prefix_pages"])
    par, nodes = ints(y["parent"]), ints(y["cu"])
    dims = gt.AttendDims(2, 90, 60, 8, 2, 128, gt.BF16, 64, y["k_cache"].shape[0],
                         table.shape[1], 500)
    assert gt.attend_workspace(dims) > 0
    yield lambda **k: gt.attend(y["q"], y["k"], y["v"], par, nodes, y["k_cache"], y["v_cache"],
                                table, ctx, prefix_pages=pre, prefix_len=500, **k)
    z = append_inputs([700, 3, 64], [5, 0, 64], 8, 128, 32, "bf16", seed=33)
    zt, zc, zn = ints(z["table"]), ints(z["ctx"]), ints(z["cu"])

    def append(**k):
        new_len = gt.cache_append(z["k"], z["v"], zn, z["k_cache"], z["v_cache"], zt, zc, **k)
        return new_len, z["k_cache"], z["v_cache"]

    yield append
    path = ints([[0, 1, 2], [0, 1, -1], [0, -1, -1]])
    tree = cu_of([40, 20, 33])
    tpar = ints([p for n in (40, 20, 33) for p in range(-1, n - 1)])
    rows = [t[:93].contiguous() for t in rule]

    def iteration(**k):
        o, U = gt.verify_packed(*rows, tpar, ints(tree), x["pool"], state_slot=slot, **k)
        pool = gt.commit_packed(path, ints([3, 2, 1]), U, rows[1], rows[3], ints(tree), x["pool"],
                                state_slot=slot, **k)
        return o, U, pool

    yield iteration


@pytest.mark.parametrize("n", range(5), ids=["prefill", "decode_step", "attend", "cache_append",
                                             "verify-commit"])
def test_a_call_on_a_given_stream_alone(n):
    call = list(calls())[n]
    want = [t.clone() for t in call()]
    other = torch.cuda.Stream()
    for _ in range(5):
        other.wait_stream(torch.cuda.current_stream())
        got = call(stream=other)
        litter()
        other.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
