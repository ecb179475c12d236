"""The serving operators (prefill, decode_step, attend, cache_append) on the GPU against
their fp64 definitions.

Tolerances, from the arithmetic:
  bf16 outputs   a rounding to 8 significant bits is at most 2^-8 of the value; attention
                 weights rounded to bf16 for a product add at most 2^-8 of sum_j p_j |v_j|
  fp32 outputs   dots of up to 128 terms and a few hundred accumulations: 128 * 2^-24 =
                 7.6e-6 of the largest value, rounded up to 1e-5
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from oracle import serving as ref

pytestmark = pytest.mark.gpu

EPS_BF16 = 2.0 ** -8
TOL_F32 = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(x):
    return x.float().cpu().numpy()


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def max_err(x, y):
    return float(np.max(np.abs(x - y)) / max(np.max(np.abs(y)), 1e-30)) if y.size else 0.0


# ---------------------------------------------------------------------------
# the gated delta rule
# ---------------------------------------------------------------------------

def rule_inputs(lens, Hqk, Hv, dk, dv, dtype, seed, gates="mixed"):
    r = np.random.default_rng(seed)
    T, B = int(sum(lens)), len(lens)
    dt = DT[dtype]

    def unit(*shape):
        x = r.standard_normal(shape)
        x /= np.linalg.norm(x, axis=-1, keepdims=True)
        return torch.tensor(x, dtype=dt, device="cuda")

    q, k = unit(T, Hqk, dk), unit(T, Hqk, dk)
    v = torch.tensor(r.standard_normal((T, Hv, dv)), dtype=dt, device="cuda")
    la = -np.exp(r.uniform(np.log(2e-3), np.log(1.0), size=(1, Hv))) * r.uniform(0.5, 1.5, (T, Hv))
    beta = 1 / (1 + np.exp(-r.standard_normal((T, Hv))))
    if gates == "strong":
        la = -r.uniform(0.0, 60.0, (T, Hv))
        beta = r.uniform(0.9, 0.99, (T, Hv))
    elif gates == "reset":  # alpha = 0 now and then, alpha = 1 elsewhere
        la = np.where(r.random((T, Hv)) < 0.05, -np.inf, np.where(r.random((T, Hv)) < 0.3, 0.0, la))
        beta = np.where(r.random((T, Hv)) < 0.2, 0.0, beta)
    elif gates == "same_key":  # every token writes the same key: X is full
        k[:] = k[:1] if T else k
        beta = r.uniform(0.9, 1.0, (T, Hv))
        la = -r.uniform(0.0, 0.01, (T, Hv))
    slots = r.permutation(B + 2)[:B]
    pool = torch.tensor(0.1 * r.standard_normal((B + 2, Hv, dk, dv)), dtype=torch.float32,
                        device="cuda")
    f = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    return dict(q=q, k=k, v=v, log_alpha=f(la), beta=f(beta), cu=cu_of(lens), slot=slots,
                pool=pool)


def rule_ref(x):
    return ref.delta_rule(host(x["q"]), host(x["k"]), host(x["v"]), host(x["log_alpha"]),
                          host(x["beta"]), x["cu"], host(x["pool"]), x["slot"])


def check_rule(o, pool, x):
    ro, rp = rule_ref(x)
    o, pool = host(o), host(pool)
    assert np.isfinite(pool).all()
    assert max_err(pool, rp) <= TOL_F32
    top = np.max(np.abs(ro)) if ro.size else 0.0
    eps = EPS_BF16 if x["q"].dtype == torch.bfloat16 else 0.0
    assert (np.abs(o - ro) <= eps * np.abs(ro) + TOL_F32 * top).all(), max_err(o, ro)


RULE_SHAPES = [
    ([1], 1, 1, 128, 128, "bf16"),
    ([64], 2, 4, 128, 128, "bf16"),
    ([63, 65, 0, 1, 129], 2, 4, 128, 128, "bf16"),
    ([300, 5, 128], 3, 3, 128, 128, "bf16"),
    ([700], 1, 2, 128, 128, "bf16"),
    ([40, 41], 1, 8, 128, 128, "bf16"),
    ([33, 90, 0], 2, 4, 64, 96, "bf16"),
    ([20, 70], 1, 2, 128, 16, "bf16"),
    ([50, 3], 2, 2, 16, 48, "f32"),
    ([129, 0, 64], 2, 4, 128, 128, "f32"),
    ([17, 100], 1, 3, 80, 112, "f32"),
]


@pytest.mark.parametrize("case", RULE_SHAPES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
@pytest.mark.parametrize("gates", ["mixed", "strong", "reset", "same_key"])
def test_prefill(case, gates):
    lens, Hqk, Hv, dk, dv, dtype = case
    x = rule_inputs(lens, Hqk, Hv, dk, dv, dtype, seed=sum(lens) + dk, gates=gates)
    status = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    o, pool = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]),
                         x["pool"], state_slot=ints(x["slot"]), dev_status=status)
    torch.cuda.synchronize()
    assert (status == 0).all()
    check_rule(o, pool, x)


def test_prefill_in_place_and_default_slots():
    x = rule_inputs([100, 70], 2, 4, 128, 128, "bf16", seed=5)
    x["slot"] = np.arange(2)
    want = rule_ref(x)[1]
    pool = x["pool"].clone()
    _, out = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]), pool,
                        pool_out=pool)
    assert out is pool
    assert max_err(host(pool), want) <= TOL_F32
    assert torch.equal(pool[2:], x["pool"][2:])  # no other slot is touched


def test_prefill_continues_where_it_stopped():
    """A prompt in two calls gives the state and outputs of one call."""
    x = rule_inputs([257], 2, 4, 128, 128, "bf16", seed=6)
    ro, rp = rule_ref(x)
    pool, outs, slot = x["pool"].clone(), [], ints(x["slot"])
    for a, b in ((0, 100), (100, 257)):
        part = [x[n][a:b].contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
        o, _ = gt.prefill(*part, ints([0, b - a]), pool, state_slot=slot, pool_out=pool)
        outs.append(host(o))
    assert max_err(host(pool), rp) <= TOL_F32
    assert (np.abs(np.concatenate(outs) - ro) <= EPS_BF16 * np.abs(ro) + TOL_F32).all()


def test_prefill_does_not_mix_sequences():
    """NaN in one sequence's rows stays in that sequence."""
    x = rule_inputs([70, 30, 100], 1, 2, 128, 128, "bf16", seed=7)
    clean = rule_ref(x)
    for n in ("q", "k", "v", "log_alpha", "beta"):
        x[n][70:100] = float("nan")
    o, pool = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]),
                         x["pool"], state_slot=ints(x["slot"]))
    o, pool = host(o), host(pool)
    assert np.isnan(o[70:100]).all() and np.isnan(pool[x["slot"][1]]).all()
    for rows, b in ((slice(0, 70), 0), (slice(100, 200), 2)):
        assert (np.abs(o[rows] - clean[0][rows]) <= EPS_BF16 * np.abs(clean[0][rows]) + TOL_F32).all()
        assert max_err(pool[x["slot"][b]], clean[1][x["slot"][b]]) <= TOL_F32


def test_prefill_is_deterministic():
    x = rule_inputs([300, 200], 2, 4, 128, 128, "bf16", seed=8)
    runs = [gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]), x["pool"],
                       state_slot=ints(x["slot"])) for _ in range(3)]
    for o, pool in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(pool, runs[0][1])


def test_prefill_on_another_stream():
    x = rule_inputs([200], 2, 4, 128, 128, "bf16", seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, pool = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]),
                             x["pool"], state_slot=ints(x["slot"]))
    s.synchronize()
    check_rule(o, pool, x)


def test_prefill_bad_layout_is_reported():
    x = rule_inputs([10, 20, 30], 1, 2, 128, 128, "bf16", seed=10)
    status = torch.empty(3, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    pool = x["pool"].clone()
    gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints([0, 10, 30, 61]), x["pool"],
               state_slot=ints([0, 99, 1]), N_max=64, pool_out=pool, o=o, dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_LAYOUT, gt.STATUS_BAD_LAYOUT]
    assert (o[10:] == 7.0).all() and torch.equal(pool[1:], x["pool"][1:])
    # a sequence longer than the N_max that was promised
    gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints([0, 10, 30, 60]), x["pool"],
               state_slot=ints([0, 1, 2]), N_max=20, dev_status=status)
    assert status.tolist() == [0, 0, gt.STATUS_BAD_LAYOUT]


@pytest.mark.parametrize("B,Hqk,Hv,dk,dv,dtype", [
    (1, 16, 32, 128, 128, "bf16"), (5, 2, 4, 128, 128, "bf16"), (33, 1, 2, 128, 128, "bf16"),
    (40, 4, 8, 128, 128, "bf16"), (160, 1, 2, 96, 128, "f32"), (311, 1, 1, 16, 128, "bf16"),
    (3, 2, 2, 64, 32, "bf16"), (2, 1, 3, 16, 16, "f32"), (4, 2, 4, 128, 128, "f32"),
    (3, 1, 1, 80, 112, "f32")])
@pytest.mark.parametrize("gates", ["mixed", "strong", "reset"])
def test_decode_step(B, Hqk, Hv, dk, dv, dtype, gates):
    x = rule_inputs([1] * B, Hqk, Hv, dk, dv, dtype, seed=B + dk, gates=gates)
    status = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    o, pool = gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["pool"],
                             state_slot=ints(x["slot"]), dev_status=status)
    assert (status == 0).all()
    check_rule(o, pool, x)
    again = x["pool"].clone()
    gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], again,
                   state_slot=ints(x["slot"]), pool_out=again)
    assert torch.equal(again, pool)  # in place


@pytest.mark.parametrize("B,Hqk,Hv,dk,dtype", [
    (1850, 1, 2, 128, "bf16"), (3701, 1, 1, 16, "f32"), (1000, 2, 4, 48, "bf16")])
def test_decode_step_of_thousands_of_states(B, Hqk, Hv, dk, dtype):
    x = rule_inputs([1] * B, Hqk, Hv, dk, 128, dtype, seed=B, gates="reset")
    status = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    slot = ints(x["slot"])
    o, pool = gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["pool"],
                             state_slot=slot, dev_status=status)
    assert (status == 0).all()
    check_rule(o, pool, x)
    again = x["pool"].clone()
    gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], again, state_slot=slot,
                   pool_out=again)
    assert torch.equal(again, pool)  # in place
    slot[5] = B + 2  # no such state: reported, and nothing else changes
    other = torch.full_like(o, 7.0)
    gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["pool"], state_slot=slot,
                   o=other, dev_status=status)
    assert status[5] == gt.STATUS_BAD_LAYOUT and (status != 0).sum() == 1
    assert (other[5] == 7.0).all()
    assert torch.equal(other[:5], o[:5]) and torch.equal(other[6:], o[6:])


@pytest.mark.parametrize("lens,Hqk,Hv", [
    ([20000, 130, 0, 5000, 64], 16, 32),  # all tiles at once would be over 600 MB
    ([16500], 2, 4), ([8200], 4, 4), ([100, 17000, 0, 9000], 2, 4)],
    ids=["batch", "one", "two-halves", "few-heads"])
def test_prefill_in_several_segments(lens, Hqk, Hv):
    """Long batches, whose tiles are made in parts, give what parts of them give."""
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(normal(T, Hqk, 128), dim=-1).bfloat16() for _ in range(2))
    v, la, beta = normal(T, Hv, 128).bfloat16(), -normal(T, Hv).abs(), torch.sigmoid(normal(T, Hv))
    pool = 0.1 * normal(len(lens), Hv, 128, 128)
    cu = cu_of(lens)
    dims = gt.Dims(len(lens), max(lens), Hqk, Hv, 128, 128, gt.BF16)
    assert gt.prefill_workspace(dims, T) <= 512 << 20
    o, out = gt.prefill(q, k, v, la, beta, ints(cu), pool)
    for b, n in enumerate(lens):
        state, a = pool[b:b + 1].clone(), cu[b]
        for lo in range(0, n, 2048):
            hi = min(n, lo + 2048)
            part = [x[a + lo:a + hi].contiguous() for x in (q, k, v, la, beta)]
            got, _ = gt.prefill(*part, ints([0, hi - lo]), state, pool_out=state)
            assert max_err(host(got), host(o[a + lo:a + hi])) <= EPS_BF16
        assert max_err(host(state), host(out[b:b + 1])) <= TOL_F32


def test_decode_step_bad_slot_is_reported():
    x = rule_inputs([1, 1], 1, 2, 128, 128, "bf16", seed=3)
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    gt.decode_step(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["pool"],
                   state_slot=ints([-1, 2]), o=o, dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT, 0]
    assert (o[0] == 7.0).all() and (o[1] != 7.0).any()


def test_prefill_is_the_verification_of_a_chain():
    """The same tokens as a chain tree, verified and committed, end in the same state."""
    x = rule_inputs([96], 2, 4, 128, 128, "bf16", seed=12)
    x["slot"] = np.arange(1)
    o, pool = gt.prefill(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], ints(x["cu"]), x["pool"])
    parent = ints(np.arange(-1, 95)[None])
    args = [x[n][None].contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
    ov, U = gt.verify(*args, parent, x["pool"][:1].contiguous())
    S1 = gt.commit(ints(np.arange(96)[None]), ints([96]), U, args[1], args[3],
                   x["pool"][:1].contiguous())
    assert max_err(host(pool[:1]), host(S1)) <= 1e-4  # the commit's own tolerance
    assert max_err(host(o), host(ov[0])) <= 1e-2


# ---------------------------------------------------------------------------
# attention over a paged cache
# ---------------------------------------------------------------------------

def attend_inputs(nodes, ctx, prefix, Hq, Hkv, D, page, dtype, seed, tree="random", own=True,
                  size=1.0, extra_width=1):
    r = np.random.default_rng(seed)
    dt = DT[dtype]
    T, B = int(sum(nodes)), len(nodes)
    t = lambda *s: torch.tensor(size * r.standard_normal(s), dtype=dt, device="cuda")  # noqa: E731
    n_prefix = -(-prefix // page)
    held = [-(-c // page) for c in ctx]
    n_pages = n_prefix + sum(held) + 3
    order = r.permutation(n_pages).astype(np.int32)
    width = max(held + [0]) + extra_width
    table = np.full((B, width), 1 << 30, dtype=np.int32)  # entries past a context are not read
    at = n_prefix
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    kc, vc = t(n_pages, page, Hkv, D), t(n_pages, page, Hkv, D)
    # what no row may use holds NaN and infinities
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    for pages, length in [(order[:n_prefix], prefix)] + [(table[b], ctx[b]) for b in range(B)]:
        for p in range(length):
            used[pages[p // page], p % page] = True
    kc[~used.cuda()] = float("nan")
    vc[~used.cuda()] = float("nan")
    vc[(~used.cuda()).nonzero()[::2, 0], (~used.cuda()).nonzero()[::2, 1]] = float("inf")
    parent = []
    for n in nodes:
        if tree == "chain":
            parent += list(range(-1, n - 1))
        elif tree == "star":
            parent += [-1] * n
        else:
            parent += [int(r.integers(-1, i)) for i in range(n)]
    return dict(q=t(T, Hq, D), k=t(T, Hkv, D) if own else None, v=t(T, Hkv, D) if own else None,
                parent=np.array(parent, dtype=np.int32), cu=cu_of(nodes), k_cache=kc, v_cache=vc,
                table=table, ctx=np.array(ctx, dtype=np.int32), prefix_pages=order[:n_prefix],
                prefix=prefix)


def run_attend(x, chain=False, **kw):
    return gt.attend(x["q"], x["k"], x["v"], None if chain else ints(x["parent"]), ints(x["cu"]),
                     x["k_cache"], x["v_cache"], ints(x["table"]), ints(x["ctx"]),
                     prefix_pages=ints(x["prefix_pages"]) if x["prefix"] else None,
                     prefix_len=x["prefix"], **kw)


def check_attend(o, lse, x, chain=False, scale=None, rows=slice(None)):
    opt = lambda t: None if t is None else host(t)  # noqa: E731
    ro, rl, ra = ref.attend(host(x["q"]), opt(x["k"]), opt(x["v"]), None if chain else x["parent"],
                            x["cu"], host(x["k_cache"]), host(x["v_cache"]), x["table"], x["ctx"],
                            x["prefix_pages"], x["prefix"],
                            x["q"].shape[2] ** -0.5 if scale is None else scale)
    o, lse, ro, rl, ra = (t[rows] for t in (host(o), host(lse), ro, rl, ra))
    bf16 = x["q"].dtype == torch.bfloat16
    top = np.max(np.abs(ra)) if ra.size else 0.0
    bound = (EPS_BF16 * (np.abs(ro) + ra) if bf16 else 0.0) + TOL_F32 * top
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= bound).all(), float(np.max(np.abs(o - ro) - bound))
    empty = np.isinf(rl)
    assert (np.isneginf(lse) == empty).all()
    assert (np.abs(lse - rl)[~empty] <= TOL_F32 * (1 + np.abs(rl[~empty]))).all()


ATTEND = [
    # nodes, context lengths, prefix, Hq, Hkv, D, page, dtype
    ([1], [300], 0, 32, 8, 128, 16, "bf16"),
    ([1], [0], 0, 4, 2, 128, 16, "bf16"),
    ([1, 1, 1], [0, 1, 129], 0, 8, 1, 128, 16, "bf16"),
    ([1] * 9, [5, 0, 64, 65, 200, 1, 17, 128, 300], 333, 8, 2, 128, 64, "bf16"),
    ([1] * 40, list(range(40)), 700, 16, 2, 128, 16, "bf16"),
    ([128], [200], 0, 4, 1, 128, 64, "bf16"),
    ([128, 128], [0, 257], 130, 8, 4, 128, 64, "bf16"),
    ([1, 40, 0, 130, 7], [10, 0, 50, 128, 300], 77, 6, 2, 128, 24, "bf16"),
    ([256], [100], 64, 2, 2, 128, 128, "bf16"),
    ([300], [20], 5, 3, 1, 128, 1, "bf16"),
    ([33, 64], [130, 127], 128, 4, 4, 64, 32, "bf16"),
    ([5, 100], [33, 257], 40, 8, 2, 64, 48, "bf16"),
    ([9, 2], [70, 5], 40, 4, 2, 96, 16, "bf16"),
    ([3, 20], [70, 5], 33, 4, 2, 16, 7, "bf16"),
    ([1, 40, 3], [10, 130, 0], 77, 6, 2, 64, 24, "f32"),
    ([30], [65], 0, 2, 1, 128, 16, "f32"),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
@pytest.mark.parametrize("tree", ["random", "chain", "star"])
def test_attend(case, tree):
    x = attend_inputs(*case, seed=len(case[0]) + case[2], tree=tree)
    status = torch.full((len(case[0]),), -7, dtype=torch.int32, device="cuda")
    o, lse = run_attend(x, chain=tree == "chain", dev_status=status)
    assert (status == 0).all()
    check_attend(o, lse, x, chain=tree == "chain")


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_attend_cache_alone(case):
    """Without own rows; a sequence without context then sees nothing where there is no
    prefix: zeros and lse = -inf."""
    x = attend_inputs(*case, seed=3 + case[2], own=False)
    o, lse = run_attend(x)
    check_attend(o, lse, x)


LONG = [
    # long chains; long contexts, which are split over CTAs and into parts; full prefix units
    ([1500, 3], [10, 700], 200, 4, 2, 128, 64, "bf16"),
    ([2100], [0], 0, 2, 1, 64, 16, "bf16"),
    ([1100, 40], [30, 0], 50, 2, 1, 64, 16, "f32"),
    ([1, 3], [9000, 30], 0, 8, 2, 128, 16, "bf16"),
    ([1] * 16, [300 * (i + 1) for i in range(16)], 0, 8, 4, 64, 64, "bf16"),
    ([60], [5000], 0, 4, 1, 128, 64, "bf16"),
    ([20] * 12, [40] * 12, 6000, 8, 2, 128, 64, "bf16"),
    ([1] * 30, [5] * 30, 4000, 16, 4, 128, 128, "bf16"),
    ([1, 2], [2500, 100], 300, 4, 2, 128, 24, "f32"),
]


MANY = [
    # more units than SMs, and a last round of few: the shortest contexts in smaller units
    ([70] * 20, [37 * (i * 7 % 20) for i in range(20)], 40, 16, 4, 128, 64, "bf16"),
    ([70, 3, 1, 40] * 5 + [66], [11 * (i * 5 % 21) for i in range(21)], 0, 16, 4, 64, 16, "bf16"),
    ([150] * 10, [0] * 9 + [200], 0, 8, 8, 128, 32, "bf16"),
]


@pytest.mark.parametrize("case", MANY, ids=["equal", "ragged", "one-head"])
@pytest.mark.parametrize("tree", ["random", "chain"])
def test_attend_many_units(case, tree):
    x = attend_inputs(*case, seed=len(case[0]) + case[2], tree=tree)
    status = torch.full((len(case[0]),), -7, dtype=torch.int32, device="cuda")
    o, lse = run_attend(x, chain=tree == "chain", dev_status=status)
    assert (status == 0).all()
    check_attend(o, lse, x, chain=tree == "chain")
    # sequences with a length that cannot be are reported, and no other's rows change
    bad = np.arange(len(x["ctx"])) % 6 == 5
    o, lse = run_attend(dict(x, ctx=np.where(bad, -1, x["ctx"])), chain=tree == "chain",
                        dev_status=status)
    assert (status.cpu().numpy() == np.where(bad, gt.STATUS_BAD_LAYOUT, 0)).all()
    check_attend(o, lse, dict(x, ctx=np.where(bad, 0, x["ctx"])), chain=tree == "chain",
                 rows=np.flatnonzero(np.repeat(~bad, np.diff(x["cu"]))))


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)).replace(" ", "")[:60])
def test_attend_long(case):
    x = attend_inputs(*case, seed=len(case[0]) + case[2], tree="chain")
    status = torch.full((len(case[0]),), -7, dtype=torch.int32, device="cuda")
    o, lse = run_attend(x, chain=True, dev_status=status)
    assert (status == 0).all()
    check_attend(o, lse, x, chain=True)


@pytest.mark.parametrize("size,scale", [(6.0, 1.0), (1.0, 0.0), (1.0, -0.3), (30.0, None)])
def test_attend_scales_and_sharp_rows(size, scale):
    """Scores of thousands (one key takes the whole weight), a scale of zero (a mean) and a
    negative one."""
    x = attend_inputs([1, 60], [200, 300], 150, 8, 2, 128, 64, "bf16", seed=4, size=size)
    kw = {} if scale is None else dict(scale=scale)
    o, lse = run_attend(x, **kw)
    check_attend(o, lse, x, scale=scale)


@pytest.mark.parametrize("dtype,D,nodes", [("bf16", 128, [60, 150]), ("bf16", 64, [1, 40]),
                                           ("f32", 64, [30, 40])])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_attend_unseen_nodes_may_hold_anything(dtype, D, nodes, what):
    """Infinities and NaN in the keys and values of nodes that a row does not see leave the
    row alone; the rows that see them get them."""
    x = attend_inputs(nodes, [70, 0], 40, 8, 2, D, 32, dtype, seed=11)
    good = run_attend(x)
    bad = [int(x["cu"][b] + n - 1) for b, n in enumerate(nodes)]  # the last node is a leaf
    x["k"][bad], x["v"][bad] = what, what
    x["v"][bad, :, 1::2] = 1.0  # beside finite values
    o, lse = run_attend(x)
    rest = np.setdiff1d(np.arange(sum(nodes)), bad)
    assert torch.equal(o[rest], good[0][rest]) and torch.equal(lse[rest], good[1][rest])
    assert not np.isfinite(host(o[bad])[:, :, ::2]).any()
    # a value alone that is not finite: the columns that it sits in, no others
    x = attend_inputs(nodes, [70, 0], 40, 8, 2, D, 32, dtype, seed=11)
    x["v"][bad, :, 3] = what
    o, lse = run_attend(x)
    assert torch.equal(o[rest], good[0][rest]) and torch.equal(lse, good[1])
    keep = np.setdiff1d(np.arange(D), [3])
    assert torch.equal(o[:, :, keep], good[0][:, :, keep])
    assert not np.isfinite(host(o[bad])[:, :, 3]).any()


def test_attend_is_deterministic():
    x = attend_inputs([1] * 20, [50 * i for i in range(20)], 2000, 8, 2, 128, 64, "bf16", seed=5)
    first = run_attend(x)
    for _ in range(3):
        o, lse = run_attend(x)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_attend_shared_prefix_is_the_prefix_of_each():
    """The shared prefix gives what the same rows at the head of each context give."""
    x = attend_inputs([1, 30, 3], [40, 0, 100], 192, 8, 2, 128, 64, "bf16", seed=6)
    o, lse = run_attend(x)
    y = dict(x, prefix=0, ctx=x["ctx"] + 192,
             table=np.concatenate([np.tile(x["prefix_pages"], (3, 1)), x["table"]], axis=1))
    o2, lse2 = run_attend(y)
    assert max_err(host(lse), host(lse2)) <= TOL_F32
    check_attend(o2, lse2, x)
    check_attend(o, lse, x)


def test_attend_cache_past_32_bit_offsets():
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements of the cache."""
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 31) // (page * Hkv * D) + 64
    x = attend_inputs([1, 40], [200, 130], 70, 16, Hkv, D, page, "bf16", seed=7)
    small = x["k_cache"].shape[0]
    far = np.arange(n_pages - small, n_pages, dtype=np.int32)
    kc = torch.empty(n_pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[n_pages - small:], vc[n_pages - small:] = x["k_cache"], x["v_cache"]
    y = dict(x, k_cache=kc, v_cache=vc, prefix_pages=far[x["prefix_pages"]],
             table=np.where(x["table"] < small, far[np.minimum(x["table"], small - 1)], 1 << 30))
    o, lse = run_attend(y)
    check_attend(o, lse, x)


def test_attend_bad_device_data_is_reported():
    x = attend_inputs([1, 20, 5], [40, 70, 100], 64, 8, 2, 128, 32, "bf16", seed=8)
    good = run_attend(x)
    status = torch.empty(3, dtype=torch.int32, device="cuda")
    run_attend(dict(x, ctx=np.array([40, 100000, -1])), dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_LAYOUT, gt.STATUS_BAD_LAYOUT]
    par = x["parent"].copy()
    par[1 + 7] = 7
    o, _ = run_attend(dict(x, parent=par), dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_TREE, 0]
    assert torch.equal(o[:1], good[0][:1]) and torch.equal(o[21:], good[0][21:])
    tab = x["table"].copy()
    tab[2, 1] = 10 ** 6
    run_attend(dict(x, table=tab), dev_status=status)
    assert status.tolist() == [0, 0, gt.STATUS_BAD_LAYOUT]
    run_attend(dict(x, prefix_pages=np.array([0, -5], dtype=np.int32)), dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT] * 3
    run_attend(dict(x, cu=np.array([0, 1, 27, 26])), N_max=26, dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_LAYOUT, gt.STATUS_BAD_LAYOUT]


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

def append_inputs(nodes, ctx, Hkv, D, page, dtype, seed, Lmax=None):
    r = np.random.default_rng(seed)
    dt = DT[dtype]
    T, B = int(sum(nodes)), len(nodes)
    t = lambda *s: torch.tensor(r.standard_normal(s), dtype=dt, device="cuda")  # noqa: E731
    path = plen = None
    if Lmax is not None:
        plen = np.array([min(n, int(r.integers(0, Lmax + 1))) for n in nodes], dtype=np.int32)
        path = np.full((B, Lmax), -1, dtype=np.int32)
        for b, n in enumerate(nodes):
            path[b, :plen[b]] = np.sort(r.permutation(n)[:plen[b]])
    held = [-(-(c + n) // page) for c, n in zip(ctx, nodes)]
    order = r.permutation(sum(held) + 2).astype(np.int32)
    table = np.full((B, max(held + [1])), 1 << 30, dtype=np.int32)
    for b, h in enumerate(held):
        table[b, :h] = order[sum(held[:b]):sum(held[:b]) + h]
    return dict(k=t(T, Hkv, D), v=t(T, Hkv, D), cu=cu_of(nodes),
                k_cache=t(sum(held) + 2, page, Hkv, D), v_cache=t(sum(held) + 2, page, Hkv, D),
                table=table, ctx=np.array(ctx, dtype=np.int32), path=path, path_len=plen)


def run_append(x, **kw):
    opt = lambda a: None if a is None else ints(a)  # noqa: E731
    return gt.cache_append(x["k"], x["v"], ints(x["cu"]), x["k_cache"], x["v_cache"],
                           ints(x["table"]), ints(x["ctx"]), path=opt(x["path"]),
                           path_len=opt(x["path_len"]), **kw)


@pytest.mark.parametrize("nodes,ctx,Hkv,D,page,dtype,Lmax", [
    ([128] * 4, [0, 1, 63, 1000], 8, 128, 64, "bf16", 24),
    ([1], [15], 1, 16, 16, "bf16", None),
    ([1, 0, 700, 64], [5, 7, 0, 64], 2, 128, 32, "bf16", None),
    ([40, 3, 9], [0, 100, 31], 3, 48, 7, "f32", 5),
    ([2000], [3], 1, 64, 1, "f32", None),
    ([5, 6], [1, 2], 2, 80, 24, "bf16", 0),
])
def test_cache_append(nodes, ctx, Hkv, D, page, dtype, Lmax):
    x = append_inputs(nodes, ctx, Hkv, D, page, dtype, seed=sum(nodes), Lmax=Lmax)
    want = ref.cache_append(host(x["k"]), host(x["v"]), x["cu"], host(x["k_cache"]),
                            host(x["v_cache"]), x["table"], x["ctx"], x["path"], x["path_len"])
    status = torch.full((len(nodes),), -7, dtype=torch.int32, device="cuda")
    new_len = run_append(x, dev_status=status)
    assert (status == 0).all()
    assert np.array_equal(host(x["k_cache"]), want[0])
    assert np.array_equal(host(x["v_cache"]), want[1])
    assert new_len.tolist() == want[2].tolist()


def test_cache_append_bad_device_data_is_reported():
    x = append_inputs([20] * 5, [10] * 5, 2, 64, 16, "bf16", seed=1, Lmax=4)
    x["path_len"][:] = 3
    x["path"][:, :3] = [0, 1, 2]
    x["path"][1, 1] = 20           # no such node
    x["path_len"][2] = 5           # past Lmax
    x["table"][3, 0] = -1          # no page for its rows
    x["ctx"][4] = 10 ** 6          # past the table
    before = x["k_cache"].clone()
    status = torch.empty(5, dtype=torch.int32, device="cuda")
    new_len = run_append(x, dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_PATH, gt.STATUS_BAD_PATH, gt.STATUS_BAD_LAYOUT,
                               gt.STATUS_BAD_LAYOUT]
    assert new_len.tolist()[0] == 13 and new_len.tolist()[2] == 10 and new_len.tolist()[4] == 10 ** 6
    changed = (x["k_cache"] != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {int(x["table"][0, 0]), int(x["table"][1, 0])}
