"""The operators in front of the attention on many rows: more than their numbers' 32 bits hold, and
more than the SMs take at once, where a warp's passes follow one another.

Tolerances, inputs and definitions are those of test_rope_gpu.
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from oracle import rope as ref
from tests.test_rope_gpu import (append_inputs, check, check_append, host, inputs, ints, laid,
                                 run, run_append, want)

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


# Heads enough for 5 to 7 passes of a warp that takes a whole row: more than the copies that it has
# on their way at once, and a change from queries to keys between them.
MANY = [
    # Hq, Hkv, D, R, dtype
    (16, 5, 128, 128, "bf16"),
    (16, 5, 128, 32, "bf16"),
    (14, 6, 128, 40, "bf16"),    # pairs across vectors: two at a time
    (13, 7, 128, 126, "bf16"),   # and one by one (R / 2 odd)
    (20, 10, 80, 80, "bf16"),
    (21, 9, 80, 40, "bf16"),
    (16, 8, 96, 24, "bf16"),
    (40, 10, 64, 64, "bf16"),
    (100, 70, 16, 16, "bf16"),
    (99, 37, 16, 14, "bf16"),
    (33, 11, 48, 48, "bf16"),
    (15, 5, 112, 0, "bf16"),
    (8, 3, 128, 128, "f32"),
    (7, 4, 128, 20, "f32"),
    (14, 5, 80, 20, "f32"),
    (24, 8, 48, 32, "f32"),
    (9, 3, 112, 10, "f32"),
    (64, 40, 16, 16, "f32"),
]


def few(x, rows):
    """The same call's rows `rows` alone, for the definition."""
    return dict(x, q=x["q"][rows], k=x["k"][rows], positions=x["positions"][rows.numpy()])


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_of_many_rows(shape, interleaved):
    """From rows that are divided over several warps, so that one takes the last queries and the
    first keys, to a warp a row (from 14 rows an SM on)."""
    Hq, Hkv, D, R, dtype = shape
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for i, T in enumerate((2 * sms + 1, 5 * sms, 9 * sms - 5, 14 * sms + 372)):
        at = D + R // 2 + i + interleaved
        x = inputs(T, Hq, Hkv, D, R, dtype, ("dense", "fused", "gated", "heads", "same")[at % 5],
                   seed=T + D + R, norm=("rms", "rms", "unit", None)[at % 4])
        q, k = run(x, interleaved)
        some = np.random.default_rng(T).choice(np.arange(40, T - 40), 120, replace=False)
        rows = torch.tensor(np.concatenate([np.arange(40), np.sort(some), np.arange(T - 40, T)]))
        y = few(x, rows)
        check(q[rows], want(y, "q", interleaved), dtype)
        check(k[rows], want(y, "k", interleaved), dtype)


@pytest.mark.parametrize("shape", [MANY[i] for i in (0, 2, 3, 5, 8, 10, 12, 14)],
                         ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows", ["fused", "gated"])
def test_many_rows_in_place_and_into_views(shape, interleaved, rows):
    """Every row of every kind of output is the same, and nothing beside the heads changes."""
    Hq, Hkv, D, R, dtype = shape
    T = 14 * torch.cuda.get_device_properties(0).multi_processor_count + 372
    x = inputs(T, Hq, Hkv, D, R, dtype, rows, seed=D + R, norm="rms")
    q, k = run(x, interleaved)
    part = torch.arange(0, T, 17)
    y = few(x, part)
    check(q[part], want(y, "q", interleaved), dtype)
    check(k[part], want(y, "k", interleaved), dtype)
    r = np.random.default_rng(5)
    a, b = laid(r, T, Hq, D, dtype, "gated"), laid(r, T, Hkv, D, dtype, "fused")
    for out, fresh, n in ((a, q, "q_out"), (b, k, "k_out")):
        kept, own = out._base.clone(), out.clone()
        run(x, interleaved, **{n: out})
        assert torch.equal(out, fresh)
        out.copy_(own)
        assert torch.equal(out._base, kept)
    was = {n: (x[n]._base.clone(), x[n].clone()) for n in "qk"}
    run(x, interleaved, q_out=x["q"], k_out=x["k"])
    assert torch.equal(x["q"], q) and torch.equal(x["k"], k)
    for n, (base, own) in was.items():
        x[n].copy_(own)
        assert torch.equal(x[n]._base, base)


@pytest.mark.parametrize("missing", ["wq", "wk"])
@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("bf16", 80, 40), ("f32", 80, 20)])
def test_many_rows_with_weights_of_one_of_the_two(missing, dtype, D, R):
    """A warp goes from queries with weights to keys without, or the other way round."""
    T = 14 * torch.cuda.get_device_properties(0).multi_processor_count + 40
    x = inputs(T, 10, 7, D, R, dtype, "fused", seed=23, norm="rms")
    x[missing] = None
    q, k = run(x, False)
    rows = torch.arange(0, T, 11)
    check(q[rows], want(few(x, rows), "q", False), dtype)
    check(k[rows], want(few(x, rows), "k", False), dtype)


@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("bf16", 80, 40), ("f32", 48, 10)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows_infinities_and_nan_stay_in_their_heads(dtype, D, R, interleaved):
    T = 14 * torch.cuda.get_device_properties(0).multi_processor_count + 40
    x = inputs(T, 16, 8, D, R, dtype, "dense", seed=8, norm="rms")
    q, k = run(x, interleaved)
    r = np.random.default_rng(3)
    bad = [(int(r.integers(T)), int(r.integers(16)), int(r.integers(D))) for _ in range(50)]
    for n, (t, h, e) in enumerate(bad):
        x["q"][t, h, e] = (float("inf"), float("nan"), float("-inf"))[n % 3]
    got, got_k = run(x, interleaved)
    for t, h, _ in bad:
        assert not torch.isfinite(got[t, h]).all()
        got[t, h] = q[t, h]
    assert torch.equal(got, q) and torch.equal(got_k, k)


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens", [[700, 1, 0, 1300, 33, 400], [90, 0, 250, 1, 7], [1] * 900])
def test_append_of_many_rows(shape, interleaved, lens):
    """A batch of prompts that has a warp a row (from 12 rows an SM on), and batches whose rows are
    divided over several, one with the last queries and the first keys, or keys and values; beside
    the cache, and in place."""
    Hq, Hkv, D, R, dtype = shape
    Hq, Hkv = (Hq + 1) // 2, (Hkv + 1) // 2
    at = D + R // 2 + len(lens) + interleaved
    rows = ("dense", "fused", "gated", "heads")[at % 4]
    x = append_inputs(lens, [(37 * b + 5) % 90 for b in range(len(lens))], Hq, Hkv, D, R,
                      (16, 24, 64)[at % 3], dtype, rows, ("rms", "rms", "unit", None)[at % 4],
                      seed=sum(lens) + D, prefix=1000, extra=at % 3)
    x["q"] = None if at % 5 == 0 else x["q"]
    x["wq"] = None if x["q"] is None else x["wq"]
    before = x["k_cache"].clone(), x["v_cache"].clone()
    status = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    k_out, v_out = (torch.empty(x["T"], Hkv, D, dtype=x["k"].dtype, device="cuda") for _ in "kv")
    q, new_len = run_append(x, interleaved, k_out=k_out, v_out=v_out, dev_status=status)
    assert (status == 0).all()
    check_append(x, interleaved, before, q, new_len, k_out, v_out)
    y = dict(x, k_cache=before[0], v_cache=before[1])
    y.update({n: x[n] if x[n] is None else x[n].clone() for n in "qkv"})
    run_append(y, interleaved, q_out=y["q"], k_out=y["k"], v_out=y["v"])
    assert torch.equal(y["k_cache"], x["k_cache"]) and torch.equal(y["v_cache"], x["v_cache"])
    n = sum(lens)
    assert torch.equal(y["k"][:n], k_out[:n]) and torch.equal(y["v"], x["v"])
    assert torch.equal(y["k"][n:], x["k"][n:])
    if q is not None:
        assert torch.equal(y["q"][:n], q[:n]) and torch.equal(y["q"][n:], x["q"][n:])


@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("bf16", 80, 40), ("f32", 48, 32)])
@pytest.mark.parametrize("lens", [[3, 1], [1500, 0, 800]])
def test_values_are_copied_whatever_they_are(dtype, D, R, lens):
    """The norm is the keys': values pass bit for bit, infinities and NaN (with their own bits), and
    nothing of them reaches another head."""
    x = append_inputs(lens, [7] * len(lens), 4, 6, D, R, 16, dtype, "dense", "rms", seed=12)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    clean = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
    q, _ = run_append(clean, False)
    r = np.random.default_rng(13)
    odd = np.array([0x7f80, 0xff80, 0x7fff, 0x7f81, 0xffc1, 1], dtype=np.uint16)  # (of bf16)
    odd = odd.view(np.int16) if dtype == "bf16" else (odd.astype(np.uint32) << 16).view(np.int32)
    flat = x["v"].view(bits).view(-1)
    for n in range(60):
        flat[int(r.integers(flat.numel()))] = int(odd[n % len(odd)])
    out = torch.empty_like(x["v"])
    got, _ = run_append(x, False, v_out=out)
    assert torch.equal(got, q) and torch.equal(x["k_cache"], clean["k_cache"])
    assert torch.equal(out.view(bits), x["v"].view(bits))
    at, _ = ref.append_positions(x["cu"], x["ctx"], 0, x["T"])
    b = np.repeat(np.arange(len(lens)), lens)
    pages = torch.tensor(x["table"][b, at // 16].astype(np.int64)), torch.tensor(at % 16)
    assert torch.equal(x["v_cache"].view(bits)[pages], x["v"].view(bits))


def test_norm_rope_and_positions_of_very_many_rows():
    """2^27 rows, that one row lies for, at positions of their own; a chain of as many rows."""
    T, D, R = (1 << 27) + 5, 16, 16
    x = inputs(1, 1, 1, D, R, "bf16", "dense", seed=51, norm="rms")
    x["q"], x["wq"] = None, None
    x["freq"], x["scale"] = gt.rope_frequencies(R, 1e4)
    starts, ctx = [0, T - 40, T - 7], [3, 2 ** 31 - 100, 0]
    cu, ends = ints(starts + [T]), np.array(starts[1:] + [T])
    status = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    pos = gt.tree_positions(None, cu, context_len=ints(ctx), T=T, dev_status=status)
    rows = np.array([0, 1, 77, 1 << 25, (1 << 26) - 1, 1 << 26, (1 << 26) + 1] +
                    list(range(T - 45, T)))
    b = np.searchsorted(ends, rows, side="right")
    want_pos = np.array(ctx)[b] + rows - np.array(starts)[b]
    assert (status == 0).all() and pos[torch.tensor(rows)].tolist() == want_pos.tolist()
    _, k = gt.norm_rope(None, x["k"].expand(T, 1, D), pos, x["freq"], rope_scale=x["scale"],
                        norm="rms", k_weight=x["wk"])
    y = dict(x, k=x["k"].expand(len(rows), 1, D))
    check(k[torch.tensor(rows)], want(y, "k", False, want_pos), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1 << 19, 1 << 18), (3, 70001, 33), (2500, 300, 1)])
def test_very_many_heads(dtype, T, Hq, Hkv):
    x = inputs(T, Hq, Hkv, 16, 16, dtype, "fused", seed=52, norm="rms")
    q, k = run(x, False)
    rows = torch.arange(0, T, 40)
    check(q[rows], want(few(x, rows), "q", False), dtype)
    check(k[rows], want(few(x, rows), "k", False), dtype)


@pytest.mark.parametrize("T", [5, 2500])
@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 128), ("bf16", 80, 40), ("f32", 64, 64)])
def test_one_head_for_all(T, dtype, D, R):
    """An input's heads may be one head that lies there once, its rows overlapping windows."""
    x = inputs(T, 8, 4, D, R, dtype, "dense", seed=53, norm="unit")
    x["k"] = x["k"][:, :1].expand(T, 4, D)
    flat = x["q"].reshape(-1)
    step = 16 // flat.element_size()
    x["q"] = torch.as_strided(flat, (T, 8, D), (step, 2 * step, 1))
    q, k = run(x, False)
    rows = torch.arange(0, T, 9)
    check(q[rows], want(few(x, rows), "q", False), dtype)
    check(k[rows], want(few(x, rows), "k", False), dtype)


@pytest.mark.parametrize("norm", ["rms", "unit"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_no_eps_and_any_frequency(norm, interleaved):
    """An eps of 0, and frequencies over the whole of 64 bits (backwards, and past a half turn)."""
    x = inputs(40, 3, 2, 64, 12, "f32", "dense", seed=54, norm=norm, far=2 ** 31)
    x["freq"] = torch.tensor([-1, -(1 << 63), (1 << 63) - 1, 1 << 62, -12345678901234567, 0],
                             device="cuda")
    q, k = run(x, interleaved, eps=0.0)
    check(q, want(x, "q", interleaved, eps=0.0), "f32")
    check(k, want(x, "k", interleaved, eps=0.0), "f32")
