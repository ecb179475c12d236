"""The operators in front of the attention (tree_positions, norm_rope, cache_append_rope) on the
GPU against their fp64 definitions.

Tolerances, from the arithmetic, in units of u = 2^-24 (half a step of fp32, relative):
  norm      the squares of a head's 128 elements and their sum: each term passes at most 9
            products and additions in a lane and 4 additions between lanes, 13 u of the sum; its
            factor and eps 2 u; a root halves that, 7.5 u; the root's reciprocal is within 2 steps,
            4 u; its products with the weight and with the element 1 u each: under 16 u of a
            normalised element
  rotation  the fraction of a turn is rounded to 24 bits, at most pi u as an angle; sine and
            cosine are within 2 steps, 4 u; their product with the scale 1 u; the two products and
            the sum 3 u: 12 u of scale (|x| + |y|), x and y being the pair
so 28 u of scale (|x| + |y|) (where nothing is rotated, of |x|), and the rounding to the output's
type, u of the value in fp32 and 2^-8 in bf16.  Positions and statuses are exact.
"""

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from oracle import rope as ref
from oracle import serving

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(x):
    return x.float().cpu().numpy()


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def check(got, want, dtype):
    y, size = want
    assert got.shape == y.shape
    err = np.abs(host(got).astype(np.float64) - y)
    assert (err <= STEP[dtype] * np.abs(y) + 28 * U * size).all(), float((err / (size + 1e-30)).max())


def laid(r, T, H, D, dtype, rows):
    """Heads [T, H, D] as views of a larger array."""
    t = lambda *s: torch.tensor(r.standard_normal(s), dtype=DT[dtype], device="cuda")  # noqa: E731
    pad = 8 if dtype == "bf16" else 4
    if rows == "dense":
        return t(T, H, D)
    if rows == "fused":   # columns of a wider array
        return t(T, 3 * pad + H * D + 16)[:, pad:pad + H * D].unflatten(1, (H, D))
    if rows == "gated":   # every head followed by its gate
        return t(T, H, 2 * D)[..., :D]
    if rows == "heads":   # head by head
        return t(H, T, D).transpose(0, 1)
    assert rows == "same"  # one row for all (an input only)
    return t(1, H, D).expand(T, H, D)


def inputs(T, Hq, Hkv, D, R, dtype, rows, seed, norm, far=5000):
    r = np.random.default_rng(seed)
    x = dict(q=laid(r, T, Hq, D, dtype, rows) if Hq else None, k=laid(r, T, Hkv, D, dtype, rows),
             v=laid(r, T, Hkv, D, dtype, rows), D=D, R=R, dtype=dtype, norm=norm,
             positions=r.integers(0, far, T).astype(np.int64), freq=None, scale=1.0, wq=None, wk=None)
    if R:
        x["freq"], x["scale"] = gt.rope_frequencies(R, 1e4, stretch="yarn", factor=4.0,
                                                    trained_len=far / 4)
    if norm == "rms":
        x["wq"], x["wk"] = (torch.tensor(1 + 0.3 * r.standard_normal(D), dtype=torch.float32,
                                         device="cuda") for _ in range(2))
        x["wq"] = x["wq"] if Hq else None
    return x


def want(x, name, interleaved, positions=None, eps=1e-6):
    w = {"q": x["wq"], "k": x["wk"]}[name]
    f = None if x["freq"] is None else [int(v) for v in x["freq"].tolist()]
    return ref.head_rows(host(x[name]), None if w is None else host(w),
                         x["positions"] if positions is None else positions, f, interleaved,
                         x["scale"], x["norm"], eps)


def run(x, interleaved, **kw):
    args = dict(interleaved=interleaved, rope_scale=x["scale"], norm=x["norm"], q_weight=x["wq"],
                k_weight=x["wk"])
    args.update(kw)
    pos = ints(x["positions"]) if x["R"] else None
    return gt.norm_rope(x["q"], x["k"], pos, x["freq"], **args)


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------

SHAPES = [
    # T, Hq, Hkv, D, R, dtype
    (1, 32, 8, 128, 128, "bf16"),
    (1, 1, 1, 16, 16, "bf16"),
    (37, 6, 2, 128, 64, "bf16"),
    (19, 5, 3, 128, 16, "bf16"),
    (130, 16, 16, 64, 64, "bf16"),
    (9, 7, 1, 80, 80, "bf16"),
    (9, 8, 4, 80, 20, "bf16"),
    (11, 3, 3, 48, 6, "bf16"),
    (12, 9, 3, 112, 112, "bf16"),
    (13, 9, 1, 112, 2, "bf16"),
    (5, 40, 8, 96, 48, "bf16"),
    (300, 33, 1, 32, 32, "bf16"),
    (17, 2, 2, 16, 14, "bf16"),
    (33, 4, 2, 128, 126, "bf16"),
    (21, 4, 1, 128, 0, "bf16"),
    (1, 32, 8, 128, 128, "f32"),
    (29, 6, 2, 80, 20, "f32"),
    (14, 4, 4, 48, 32, "f32"),
    (31, 5, 5, 112, 108, "f32"),
    (23, 2, 1, 16, 10, "f32"),
    (15, 3, 1, 96, 8, "f32"),
    (16, 12, 4, 64, 0, "f32"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("norm", [None, "rms", "unit"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(shape, norm, interleaved):
    T, Hq, Hkv, D, R, dtype = shape
    rows = ("dense", "fused", "gated", "heads", "same")[(T + D + R // 2) % 5]
    x = inputs(T, Hq, Hkv, D, R, dtype, rows, seed=T + D + R, norm=norm)
    q, k = run(x, interleaved)
    check(q, want(x, "q", interleaved), dtype)
    check(k, want(x, "k", interleaved), dtype)


@pytest.mark.parametrize("rows", ["dense", "fused", "gated", "heads"])
@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("bf16", 80, 20), ("f32", 48, 48)])
def test_in_place_and_into_views(rows, dtype, D, R):
    """In place gives what a new array gets, bit for bit, and nothing beside the heads changes;
    so does an output with strides."""
    r = np.random.default_rng(3)
    x = inputs(50, 6, 2, D, R, dtype, rows, seed=2, norm="rms")
    q, k = run(x, False)
    for out in rows, "fused":
        a, b = laid(r, 50, 6, D, dtype, out), laid(r, 50, 2, D, dtype, out)
        kept = (a._base if a._base is not None else a).clone(), a.clone()
        run(x, False, q_out=a, k_out=b)
        assert torch.equal(a, q) and torch.equal(b, k)
        a.copy_(kept[1])
        assert torch.equal(a._base if a._base is not None else a, kept[0])
    whole = x["q"]._base if x["q"]._base is not None else x["q"]
    before, own = whole.clone(), x["q"].clone()
    q2, k2 = run(x, False, q_out=x["q"], k_out=x["k"])
    assert q2 is x["q"] and torch.equal(q2, q) and torch.equal(k2, k)
    x["q"].copy_(own)
    assert torch.equal(whole, before)


def test_columns_of_one_projection_in_place():
    """q, k and v are columns of the same rows; q and k are rotated where they lie."""
    r = np.random.default_rng(4)
    wide = torch.tensor(r.standard_normal((77, 12 * 64)), dtype=torch.bfloat16, device="cuda")
    was = wide.clone()
    q, k, v = (p.unflatten(1, (-1, 64)) for p in wide.split([8 * 64, 2 * 64, 2 * 64], dim=1))
    x = inputs(77, 8, 2, 64, 64, "bf16", "dense", seed=5, norm="unit")
    x["q"], x["k"] = q.clone(), k.clone()
    a, b = run(x, True)
    run(dict(x, q=q, k=k), True, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(wide[:, 10 * 64:], was[:, 10 * 64:])
    # queries into the places of the gates beside them
    gated = laid(r, 77, 8, 128, "bf16", "dense")
    x["q"] = gated[..., :64]
    first = x["q"].clone()
    run(x, True, q_out=gated[..., 64:])
    check(gated[..., 64:], want(dict(x, q=first), "q", True), "bf16")
    assert torch.equal(gated[..., :64], first)


def test_one_of_the_two_and_no_rows():
    x = inputs(21, 4, 2, 128, 128, "bf16", "dense", seed=6, norm="rms")
    q, k = run(x, False)
    a, none = run(dict(x, k=None), False)  # (a weight without its heads does not count)
    assert none is None and torch.equal(a, q)
    none, b = run(dict(x, q=None), False)
    assert none is None and torch.equal(b, k)
    with pytest.raises(ValueError, match="with q"):
        run(dict(x, q=None), False, q_out=q)
    empty = dict(x, q=x["q"][:0], k=x["k"][:0], positions=x["positions"][:0])
    a, b = run(empty, False)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
    # nothing to do: a copy
    same, _ = gt.norm_rope(x["q"])
    assert torch.equal(same, x["q"])


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    """The angle is as exact at the ends of 32 bits as near 0."""
    x = inputs(12, 2, 1, 64, 64, "f32", "dense", seed=7, norm=None)
    x["freq"], x["scale"] = gt.rope_frequencies(64, 1e6)
    x["positions"] = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 10 ** 6 + 3, 131071, 2 ** 24 + 1,
                               -77777, 2 ** 31 - 64, 5])
    q, k = run(x, interleaved)
    check(q, want(x, "q", interleaved), "f32")
    check(k, want(x, "k", interleaved), "f32")
    assert torch.equal(q[0], x["q"][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [128, 64, 40])
@pytest.mark.parametrize("interleaved", [False, True])
def test_zero_rows_infinities_and_nan(dtype, R, interleaved):
    """A head of zeros stays zeros; what is not finite stays in its own head, and in its own pair
    where there is no norm."""
    x = inputs(9, 4, 2, 128, R, dtype, "dense", seed=8, norm="rms")
    x["q"][4] = 0
    q, _ = run(x, interleaved)
    assert (q[4] == 0).all()
    x["q"][2, 1, 5] = float("inf")
    x["q"][3, 3, 127] = float("nan")
    bad, _ = run(x, interleaved)
    bad[2, 1], bad[3, 3] = q[2, 1], q[3, 3]
    assert torch.equal(bad, q)
    x["norm"], x["wq"], x["wk"] = None, None, None
    x["q"][2, 1, 5], x["q"][3, 3, 127] = 1.0, 1.0
    q, _ = run(x, interleaved)
    x["q"][2, 1, 5], x["q"][3, 3, 127] = float("inf"), float("nan")
    bad, _ = run(x, interleaved)
    touched = (bad != q) | bad.isnan()
    pair = {5, 4 if interleaved else 5 + R // 2}
    last = {127} if R < 128 else {127, 126 if interleaved else 63}
    spots = {(2, 1, e) for e in pair} | {(3, 3, e) for e in last}
    assert {tuple(s) for s in touched.nonzero().tolist()} == spots


def test_large_and_tiny_elements():
    """Squares within fp32's range, and rows so small that eps decides."""
    for norm in ("rms", "unit"):
        x = inputs(4, 2, 1, 64, 64, "f32", "dense", seed=9, norm=norm)
        for row, size in enumerate((1e17, 1e-3, 1e-12, 1e-30)):
            x["q"][row] *= size
        q, _ = run(x, False)
        check(q, want(x, "q", False), "f32")
    q, _ = run(x, False, eps=0.25)
    check(q, want(x, "q", False, eps=0.25), "f32")


@pytest.mark.parametrize("norm", ["rms", "unit"])
@pytest.mark.parametrize("dtype,D,R", [("bf16", 128, 64), ("bf16", 96, 10), ("f32", 32, 0)])
def test_weights_of_one_of_the_two(norm, dtype, D, R):
    """Weights scale either norm, and may be given for queries or keys alone."""
    for missing in ("wq", "wk", None):
        x = inputs(40, 5, 3, D, R, dtype, "fused", seed=23, norm="rms")
        x["norm"] = norm
        if missing:
            x[missing] = None
        q, k = run(x, False)
        check(q, want(x, "q", False), dtype)
        check(k, want(x, "k", False), dtype)


def test_values_of_a_call_are_read_when_it_is_made():
    """Sizes and scales given as tensors count with the value that they have at the call."""
    x = append_inputs([3, 5], [2, 0], 2, 1, 64, 64, 16, "f32", "dense", "rms", seed=24)
    scale, most = torch.tensor(1.0), torch.tensor(5)
    first, _ = run_append(x, False, rope_scale=scale, N_max=most)
    scale.fill_(2.0)
    second, _ = run_append(x, False, rope_scale=scale, N_max=most)
    assert torch.allclose(second, 2 * first)
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    most.fill_(4)
    run_append(x, False, N_max=most, dev_status=status)
    assert status.tolist() == [0, gt.STATUS_BAD_LAYOUT]


def test_refused_on_the_gpu():
    x = inputs(6, 4, 2, 64, 64, "bf16", "dense", seed=10, norm="rms")
    with pytest.raises(ValueError, match="contiguous"):
        run(dict(x, q=x["q"].transpose(1, 2).contiguous().transpose(1, 2)), False)
    with pytest.raises(ValueError, match="shape"):
        run(x, False, q_out=x["q"][:5])
    with pytest.raises(TypeError, match="float32"):
        run(x, False, q_weight=x["wq"].bfloat16())
    with pytest.raises(ValueError, match="shape"):
        run(x, False, q_weight=x["wq"][:32].contiguous())
    with pytest.raises(TypeError, match="bfloat16"):
        run(dict(x, k=x["k"].float()), False)
    with pytest.raises(ValueError, match="norm"):
        run(x, False, norm="l1")
    for kw in (dict(q_out=x["q"].flatten(1)), dict(q_out=x["q"][..., None]),
               dict(k_out=x["k"].flatten(1)), dict(q_weight=x["wq"][None])):
        with pytest.raises(ValueError, match="shape"):
            run(x, False, **kw)
    for kw in (dict(q_out=5), dict(k_weight=[1.0] * 64), dict(q_weight=np.ones(64))):
        with pytest.raises(TypeError, match="torch.Tensor"):
            run(x, False, **kw)
    pos = ints(x["positions"])
    for p, f, what in ((pos[:5], x["freq"], ValueError), (pos.long(), x["freq"], TypeError),
                       (pos, x["freq"].int(), TypeError), (pos, x["freq"][None], ValueError),
                       (pos, x["freq"][0], ValueError), (pos.cpu(), x["freq"], ValueError),
                       (x["positions"], x["freq"], TypeError), (pos, [1, 2], TypeError),
                       (torch.stack([pos, pos], 1)[:, 0], x["freq"], ValueError)):
        with pytest.raises(what):
            gt.norm_rope(x["q"], x["k"], p, f)
    for k in (x["k"][:5], x["k"][..., :32], x["k"][..., None], x["k"].cpu()):
        with pytest.raises(ValueError):
            gt.norm_rope(x["q"], k, pos, x["freq"])
    one_row = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(6, 4, 64)
    for kw in (dict(q_out=one_row), dict(norm=None), dict(k_out=x["q"][:, 1:3])):
        with pytest.raises(gt.GdnTreeError) as e:
            run(x, False, **kw)
        assert e.value.code == gt.EINVAL
    flat = torch.zeros(6 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    shifted = flat[4:4 + 6 * 4 * 64].view(6, 4, 64)
    with pytest.raises(gt.GdnTreeError):
        run(dict(x, q=shifted), False)
    with pytest.raises(gt.GdnTreeError):
        gt.norm_rope(x["q"], None, ints(x["positions"]), torch.zeros(40, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------------------
# rows into the cache
# ---------------------------------------------------------------------------

def append_inputs(lens, ctx, Hq, Hkv, D, R, page, dtype, rows, norm, seed, prefix=0, extra=0):
    """extra: rows of the arrays behind the last sequence."""
    r = np.random.default_rng(seed)
    T = int(sum(lens)) + extra
    x = inputs(T, Hq, Hkv, D, R, dtype, rows, seed, norm, far=20000)
    held = [-(-(c + n) // page) for c, n in zip(ctx, lens)]
    order = r.permutation(sum(held) + 2).astype(np.int32)
    table = np.full((len(lens), max(held + [1])), 1 << 30, dtype=np.int32)
    start = np.concatenate([[0], np.cumsum(held)])
    for b, h in enumerate(held):
        table[b, :h] = order[start[b]:start[b] + h]
    t = lambda *s: torch.tensor(r.standard_normal(s), dtype=DT[dtype], device="cuda")  # noqa: E731
    x.update(cu=cu_of(lens), ctx=np.array(ctx, dtype=np.int32), table=table, prefix=prefix, T=T,
             k_cache=t(sum(held) + 2, page, Hkv, D), v_cache=t(sum(held) + 2, page, Hkv, D))
    return x


def run_append(x, interleaved, **kw):
    args = dict(prefix_len=x["prefix"], interleaved=interleaved, rope_scale=x["scale"],
                norm=x["norm"], q_weight=x["wq"], k_weight=x["wk"])
    args.update(kw)
    return gt.cache_append_rope(x["q"], x["k"], x["v"], ints(x["cu"]), x["k_cache"], x["v_cache"],
                                ints(x["table"]), ints(x["ctx"]), x["freq"], **args)


def check_append(x, interleaved, before, q, new_len, k_out=None, v_out=None):
    at, positions = ref.append_positions(x["cu"], x["ctx"], x["prefix"], x["T"])
    mine = at >= 0
    k, size = want(x, "k", interleaved, positions)
    if q is not None:
        wq, sq = want(x, "q", interleaved, positions)
        check(q[torch.tensor(mine)], (wq[mine], sq[mine]), x["dtype"])
    kc = ref.place(host(before[0]), k, x["cu"], x["table"], x["ctx"])
    sc = ref.place(np.zeros(kc.shape), size, x["cu"], x["table"], x["ctx"])
    placed = ref.place(np.zeros(kc.shape), np.ones(size.shape), x["cu"], x["table"], x["ctx"]) > 0
    check(x["k_cache"], (kc, sc), x["dtype"])
    assert np.array_equal(host(x["k_cache"])[~placed], host(before[0])[~placed])
    vc = ref.place(host(before[1]), host(x["v"]), x["cu"], x["table"], x["ctx"])
    assert np.array_equal(host(x["v_cache"]), vc)
    assert new_len.tolist() == (x["ctx"] + np.diff(x["cu"])).tolist()
    if k_out is not None:
        check(k_out[torch.tensor(mine)], (k[mine], size[mine]), x["dtype"])
        assert torch.equal(v_out[torch.tensor(mine)], x["v"][torch.tensor(mine)])


@pytest.mark.parametrize("lens,ctx,Hq,Hkv,D,R,page,dtype,rows,norm,prefix", [
    ([1], [300], 32, 8, 128, 128, 64, "bf16", "fused", "rms", 0),
    ([1], [0], 1, 1, 16, 16, 1, "bf16", "dense", None, 7),
    ([1, 0, 77, 64, 3], [5, 7, 0, 64, 31], 8, 2, 128, 64, 32, "bf16", "gated", "rms", 1000),
    ([40, 3, 9], [0, 100, 31], 0, 3, 48, 6, 7, "f32", "dense", "unit", 77),
    ([200], [3], 5, 2, 80, 20, 24, "bf16", "fused", "rms", 0),
    ([5, 6], [1, 2], 2, 2, 96, 96, 16, "f32", "heads", None, 1 << 20),
    ([0, 0], [4, 0], 2, 1, 64, 64, 16, "bf16", "dense", "rms", 0),
    ([1] * 70, [3 * b for b in range(70)], 4, 2, 64, 64, 16, "bf16", "fused", "rms", 500),
    ([b % 3 for b in range(1100)], [b % 17 for b in range(1100)], 2, 1, 32, 32, 8, "bf16", "dense",
     "unit", 0),
    ([30, 20], [10, 0], 4, 4, 112, 0, 16, "bf16", "same", "rms", 0),
], ids=lambda v: None)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(lens, ctx, Hq, Hkv, D, R, page, dtype, rows, norm, prefix, interleaved):
    x = append_inputs(lens, ctx, Hq, Hkv, D, R, page, dtype, rows, norm, seed=sum(lens) + D,
                      prefix=prefix, extra=sum(lens) % 4)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    status = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    q, new_len = run_append(x, interleaved, dev_status=status)
    assert (status == 0).all()
    check_append(x, interleaved, before, q, new_len)


def test_append_beside_the_rows_and_behind_the_last():
    """k_out and v_out get the rows too, rows behind the last sequence and states of the outputs
    there are left as they were; outputs may be the inputs."""
    x = append_inputs([33, 0, 5], [7, 3, 0], 6, 2, 64, 32, 16, "bf16", "fused", "rms", seed=3, extra=9)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    out = [torch.full((x["T"], h, 64), 5.0, dtype=torch.bfloat16, device="cuda") for h in (6, 2, 2)]
    q, new_len = run_append(x, False, q_out=out[0], k_out=out[1], v_out=out[2])
    check_append(x, False, before, q, new_len, out[1], out[2])
    assert all((o[38:] == 5.0).all() for o in out)
    y = dict(x, k_cache=before[0].clone(), v_cache=before[1].clone())
    y.update({n: x[n].clone() for n in "qkv"})
    run_append(y, False, q_out=y["q"], k_out=y["k"], v_out=y["v"])
    assert torch.equal(y["k_cache"], x["k_cache"]) and torch.equal(y["v_cache"], x["v_cache"])
    for n, o in zip("qkv", out):
        assert torch.equal(y[n][:38], o[:38]) and torch.equal(y[n][38:], x[n][38:])


def test_append_at_the_farthest_positions():
    """Positions past 2^31: a prefix of the largest length, and the rows behind it."""
    x = append_inputs([40, 3], [5000, 100], 2, 1, 64, 64, 16, "f32", "dense", None, seed=25,
                      prefix=2 ** 31 - 4097)
    x["freq"], x["scale"] = gt.rope_frequencies(64, 1e6)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    q, new_len = run_append(x, True)
    check_append(x, True, before, q, new_len)


def test_append_with_one_of_the_outputs():
    x = append_inputs([9, 4], [3, 20], 2, 2, 64, 64, 8, "bf16", "fused", "rms", seed=26)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    k_out, v_out = (torch.empty(13, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, n = run_append(x, False, k_out=k_out)
    run_append(x, False, v_out=v_out)
    check_append(x, False, before, q, n, k_out, v_out)


@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [30, 0, 7]])
@pytest.mark.parametrize("gated", [False, True])
def test_append_in_place_on_a_projection(lens, gated):
    """q, k and v are columns of the same rows (each query head followed by its gate, or not) and
    are normalised and rotated where they lie; nothing beside them changes."""
    ctx = [5 * b for b in range(len(lens))]
    x = append_inputs(lens, ctx, 6, 2, 64, 32, 16, "bf16", "dense", "rms", seed=28, prefix=9)
    r = np.random.default_rng(29)
    wide = torch.tensor(r.standard_normal((x["T"], (6 * (1 + gated) + 2 * 2) * 64 + 16)),
                        dtype=torch.bfloat16, device="cuda")
    q, k, v, rest = wide.split([6 * (1 + gated) * 64, 128, 128, 16], dim=1)
    q = q.unflatten(1, (6, -1))[..., :64]
    k, v = k.unflatten(1, (2, 64)), v.unflatten(1, (2, 64))
    x.update(q=q.clone(), k=k.clone(), v=v.clone())
    was, before = wide.clone(), (x["k_cache"].clone(), x["v_cache"].clone())
    a, n = run_append(dict(x, q=q, k=k, v=v), False, q_out=q, k_out=k, v_out=v)
    assert a is q
    check_append(x, False, before, q, n, k, v)
    for t, old in ((q, x["q"]), (k, x["k"])):
        t.copy_(old)
    assert torch.equal(wide, was)


def test_append_is_norm_rope_and_cache_append():
    x = append_inputs([50, 1, 0, 200], [10, 63, 5, 0], 8, 2, 128, 128, 64, "bf16", "dense", "rms",
                      seed=4, prefix=3000)
    y = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
    q, new_len = run_append(x, False)
    pos = gt.tree_positions(None, ints(x["cu"]), context_len=ints(x["ctx"]), prefix_len=3000, T=251)
    q2, k2 = gt.norm_rope(x["q"], x["k"], pos, x["freq"], rope_scale=x["scale"], norm="rms",
                          q_weight=x["wq"], k_weight=x["wk"])
    n2 = gt.cache_append(k2, x["v"], ints(x["cu"]), y["k_cache"], y["v_cache"], ints(x["table"]),
                         ints(x["ctx"]))
    assert torch.equal(q, q2) and torch.equal(new_len, n2)
    assert torch.equal(x["k_cache"], y["k_cache"]) and torch.equal(x["v_cache"], y["v_cache"])


def test_append_bad_device_data_is_reported():
    x = append_inputs([20] * 6, [10] * 6, 4, 2, 64, 64, 16, "bf16", "dense", "rms", seed=1)
    good = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
    q_good, _ = run_append(good, False)
    x["table"][1, 0] = -1               # no page for its first rows
    x["table"][2, 1] = len(x["k_cache"])
    x["ctx"][3] = 10 ** 6               # past the table
    x["ctx"][4] = -1
    before = x["k_cache"].clone(), x["v_cache"].clone()
    out = [torch.full((120, h, 64), 5.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    status = torch.empty(6, dtype=torch.int32, device="cuda")
    q, new_len = run_append(x, False, dev_status=status, q_out=out[0], k_out=out[1], v_out=out[2])
    L = gt.STATUS_BAD_LAYOUT
    assert status.tolist() == [0, L, L, L, L, 0]
    assert new_len.tolist() == [30, 30, 30, 10 ** 6, -1, 30]
    rows = [r for b in (0, 1, 2, 5) for r in range(20 * b, 20 * b + 20)]
    assert torch.equal(q[rows], q_good[rows])
    assert all((o[60:100] == 5.0).all() for o in out)
    for cache, was, ok in ((x["k_cache"], before[0], good["k_cache"]),
                           (x["v_cache"], before[1], good["v_cache"])):
        for b in range(6):
            pages = [int(p) for p in good["table"][b]]
            if b in (0, 5):
                assert torch.equal(cache[pages], ok[pages])
        touched = (cache != was).flatten(1).any(1).nonzero().flatten().tolist()
        allowed = {int(p) for b in (0, 1, 2, 5) for p in x["table"][b] if 0 <= p < len(cache)}
        assert set(touched) <= allowed
    # offsets that decrease, or run past the rows: reported, and nothing outside is touched
    for cu in ([0, 20, 60, 40, 80, 100, 120], [0, 20, 40, 60, 80, 100, 10 ** 9],
               [-5, 20, 40, 60, 80, 100, 120], [0, 20, 40, 60, -2 ** 31, 100, 2 ** 31 - 1]):
        y = append_inputs([20] * 6, [10] * 6, 4, 2, 64, 64, 16, "bf16", "dense", "rms", seed=1)
        y["cu"] = np.array(cu, dtype=np.int32)
        _, n = run_append(y, False, dev_status=status, N_max=30)
        bad = [not (0 <= a <= b <= 120 and b - a <= 30) for a, b in zip(cu, cu[1:])]
        assert [s == L for s in status.tolist()] == bad
        assert [int(v) for v in n] == [10 if w else 10 + b - a for a, b, w in zip(cu, cu[1:], bad)]


def test_append_refused_on_the_gpu():
    """Each argument of a wrong type, shape, layout or place is named; nothing is written."""
    x = append_inputs([6, 3], [10, 0], 4, 2, 64, 64, 16, "bf16", "dense", "rms", seed=27)
    good = dict(q=x["q"], k=x["k"], v=x["v"], cu_nodes=ints(x["cu"]), k_cache=x["k_cache"],
                v_cache=x["v_cache"], page_table=ints(x["table"]), context_len=ints(x["ctx"]),
                freq=x["freq"], norm="rms", q_weight=x["wq"], k_weight=x["wk"],
                q_out=torch.empty_like(x["q"]), k_out=torch.empty_like(x["k"]),
                v_out=torch.empty_like(x["v"]), new_len=ints([0, 0]), dev_status=ints([0, 0]), N_max=6)
    gt.cache_append_rope(**good)
    before = {n: t.clone() for n, t in good.items() if isinstance(t, torch.Tensor)}
    for name, t in before.items():
        names = [name]
        bad = [t.cpu(), t[..., None] if name != "k" else t[:, :1], t.double(), "text"]
        if t.dim() > 1 and name not in ("k", "v", "q", "k_out", "v_out", "q_out"):
            bad.append(torch.stack([t, t], -1)[..., 0])
        for b in bad:
            if name == "k" and isinstance(b, str):
                continue
            with pytest.raises((TypeError, ValueError, AttributeError)) as e:
                gt.cache_append_rope(**dict(good, **{name: b}))
            if name not in ("k", "cu_nodes", "k_cache", "page_table") or not isinstance(b, str):
                assert any(n in str(e.value) for n in names + (["v"] if name == "k" else [])), (name, b)
    assert all(torch.equal(t, before[n]) for n, t in good.items() if n in before)


def test_append_past_the_table():
    """Rows that the table has no entry for are reported; those before them are written."""
    x = append_inputs([40], [0], 2, 1, 64, 64, 16, "bf16", "dense", None, seed=5)
    full = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone())
    q, _ = run_append(full, False)
    x["table"] = x["table"][:, :2].copy()
    status = torch.empty(1, dtype=torch.int32, device="cuda")
    q2, n = run_append(x, False, dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT] and torch.equal(q, q2) and n.tolist() == [40]
    pages = [int(p) for p in x["table"][0]]
    assert torch.equal(x["k_cache"][pages], full["k_cache"][pages])
    # a table without entries
    x["table"] = x["table"][:, :0].copy()
    q3, _ = run_append(x, False, dev_status=status)
    assert status.tolist() == [gt.STATUS_BAD_LAYOUT] and torch.equal(q, q3)


def test_very_many_sequences():
    """The most sequences there may be, most of them empty: every row finds its own."""
    r = np.random.default_rng(13)
    B = 65535
    lens = (r.random(B) < 0.03).astype(int) * r.integers(1, 4, B)
    lens[[0, 31, 32, 1023, 1024, B - 1]] = 2
    ctx = r.integers(0, 9, B)
    x = append_inputs(list(lens), list(ctx), 2, 1, 16, 16, 4, "f32", "dense", None, seed=14, extra=5)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    status = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    q, new_len = run_append(x, False, dev_status=status)
    assert (status == 0).all()
    check_append(x, False, before, q, new_len)
    out = torch.full((x["T"],), -7, dtype=torch.int32, device="cuda")
    gt.tree_positions(None, ints(x["cu"]), context_len=ints(ctx), prefix_len=3, positions=out,
                      dev_status=status)
    assert (status == 0).all()
    assert out.tolist() == ref.tree_positions(None, x["cu"], ctx, 3, x["T"], fill=-7).tolist()


def test_arrays_of_a_fixed_capacity():
    """Arrays with room for more rows than there are, and a promise far above them: the rows of no
    sequence and their outputs stay as they were."""
    x = append_inputs([1, 3, 0, 2], [9, 0, 5, 31], 4, 2, 64, 32, 16, "bf16", "fused", "rms", seed=15,
                      extra=250)
    before = x["k_cache"].clone(), x["v_cache"].clone()
    out = torch.full((256, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    q, new_len = run_append(x, False, N_max=2 ** 31 - 1, q_out=out)
    check_append(x, False, before, q, new_len)
    assert (out[6:] == 5.0).all()
    par = ints([-1, -1, 0, 1, -1, 0] + [77] * 250)
    pos = torch.full((256,), -7, dtype=torch.int32, device="cuda")
    gt.tree_positions(par, ints(x["cu"]), context_len=ints(x["ctx"]), positions=pos, N_max=1024)
    assert pos.tolist() == [9, 0, 1, 2, 31, 32] + [-7] * 250
    # no rows at all, in arrays with room
    none = dict(x, cu=np.zeros(5, dtype=np.int32))
    keep = x["k_cache"].clone()
    _, new_len = run_append(none, False)
    assert new_len.tolist() == list(x["ctx"]) and torch.equal(x["k_cache"], keep)


def test_append_cache_past_32_bit_offsets():
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements of the cache."""
    page, Hkv, D = 64, 8, 128
    x = append_inputs([1, 90], [200, 130], 16, Hkv, D, 128, page, "bf16", "fused", "rms", seed=7)
    small = x["k_cache"].shape[0]
    n_pages = (1 << 31) // (page * Hkv * D) + 64
    kc = torch.empty(n_pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-small:], vc[-small:] = x["k_cache"], x["v_cache"]
    before = x["k_cache"].clone(), x["v_cache"].clone()
    y = dict(x, k_cache=kc, v_cache=vc,
             table=np.where(x["table"] < small, x["table"] + n_pages - small, 1 << 30))
    q, n = run_append(y, False)
    x["k_cache"], x["v_cache"] = kc[-small:].clone(), vc[-small:].clone()
    check_append(x, False, before, q, n)


def test_rows_past_32_bit_offsets():
    """Rows further apart than 2^31 elements in all."""
    stride = (1 << 31) // 3 // 8 * 8
    far = torch.empty(4 * stride + 256, dtype=torch.bfloat16, device="cuda")
    x = inputs(5, 2, 1, 128, 128, "bf16", "dense", seed=8, norm="rms")
    q = torch.as_strided(far, (5, 2, 128), (stride, 128, 1))
    q.copy_(x["q"])
    a, b = run(x, False)
    c, d = run(dict(x, q=q), False, q_out=q)
    assert torch.equal(a, c) and torch.equal(b, d)


# ---------------------------------------------------------------------------
# positions
# ---------------------------------------------------------------------------

def parents(lens, kind, r):
    out = []
    for n in lens:
        if kind == "chain":
            out += list(range(-1, n - 1))
        elif kind == "roots":
            out += [-1] * n
        elif kind == "star":
            out += [-1] + [0] * (n - 1) if n else []
        else:
            out += [-1 if i == 0 or r.random() < 0.02 else int(r.integers(max(0, i - 9), i))
                    for i in range(n)]
    return np.array(out, dtype=np.int32)


@pytest.mark.parametrize("lens", [[1], [128] * 3, [1024], [0, 1, 33, 31, 32, 0, 1000, 2], [5] * 700])
@pytest.mark.parametrize("kind", ["random", "chain", "star", "roots", None])
def test_positions(lens, kind):
    r = np.random.default_rng(len(lens))
    par = None if kind is None else parents(lens, kind, r)
    if kind is None:
        lens = lens + [5000]
    T = sum(lens) + 3
    ctx = r.integers(0, 10 ** 6, len(lens)).astype(np.int32)
    full = None if par is None else np.concatenate([par, [-9, -9, -9]])
    out = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    status = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    got = gt.tree_positions(None if par is None else ints(full), ints(cu_of(lens)),
                            context_len=ints(ctx), prefix_len=77, positions=out,
                            dev_status=status)
    assert got is out and (status == 0).all()
    assert out.tolist() == ref.tree_positions(par, cu_of(lens), ctx, 77, T, fill=-7).tolist()


def test_positions_defaults():
    cu = ints([0, 4, 9])
    assert gt.tree_positions(None, cu, T=9).tolist() == [0, 1, 2, 3, 0, 1, 2, 3, 4]
    with pytest.raises(ValueError, match="how many rows"):
        gt.tree_positions(None, cu)
    with pytest.raises(ValueError, match="rows"):
        gt.tree_positions(ints([-1] * 9), cu, T=8)
    assert gt.tree_positions(ints([]), ints([0, 0])).shape == (0,)


def test_positions_bad_device_data_is_reported():
    lens = [20] * 6
    par = parents(lens, "random", np.random.default_rng(0))
    par[20 + 7], par[40] = 7, -2
    ctx = np.array([0, 0, 0, -1, 2 ** 31 - 3, 5], dtype=np.int32)
    par[80:100] = np.arange(-1, 19)
    status = torch.empty(6, dtype=torch.int32, device="cuda")
    out = torch.full((120,), -7, dtype=torch.int32, device="cuda")
    gt.tree_positions(ints(par), ints(cu_of(lens)), context_len=ints(ctx), positions=out,
                      dev_status=status)
    T, L = gt.STATUS_BAD_TREE, gt.STATUS_BAD_LAYOUT
    assert status.tolist() == [0, T, T, L, L, 0]
    assert (out[20:100] == -7).all()
    clean = ref.tree_positions(par, [0, 20], ctx, 0, 20)
    assert out[:20].tolist() == clean.tolist()
    # chains: a position too far; offsets out of range or in the wrong order
    gt.tree_positions(None, ints(cu_of(lens)), context_len=ints(ctx), positions=out, dev_status=status)
    assert status.tolist() == [0, 0, 0, L, L, 0]
    for cu in ([0, 20, 10, 60, 80, 100, 121], [-1, 20, 40, 60, 80, 100, 120]):
        for p in (ints(par), None):
            gt.tree_positions(p, ints(cu), positions=out, dev_status=status, N_max=50)
            bad = [not (0 <= a <= b <= 120 and b - a <= 50) for a, b in zip(cu, cu[1:])]
            assert [s == L for s in status.tolist()] == bad
    # more rows than promised
    gt.tree_positions(ints(par), ints(cu_of(lens)), positions=out, dev_status=status, N_max=19)
    assert status.tolist() == [L] * 6


# ---------------------------------------------------------------------------
# together, captured, on other streams
# ---------------------------------------------------------------------------

def test_a_layers_attention_from_its_projection():
    """A prompt, a drafted tree, its accepted path and a single token of two sequences behind a
    shared prefix: each call's rows go straight from a projection through the operators, and
    attend's outputs are those of the definition on rotated rows of the whole sequences.

    Tolerance: o is a weighted mean of v; the weights' scores differ by what q and k are off,
    2^-8 of each, so |d score| <= 2 * 2^-8 |q| |k| / sqrt(D) <= 2^-7 sqrt(D) = 0.0625 for unit
    root-mean-square heads; a weight is then off by a factor of at most e^(2 * 0.0625) (its own
    score and the sum's), 0.134 of sum p |v|; rounding of the weights and of o 2 * 2^-8 more."""
    r = np.random.default_rng(11)
    Hq, Hkv, D, page, prefix = 8, 2, 64, 16, 40
    G, B = Hq // Hkv, 2
    freq, scale = gt.rope_frequencies(D, 1e4)
    fl = [int(v) for v in freq.tolist()]
    w = [torch.tensor(1 + 0.1 * r.standard_normal(D), dtype=torch.float32, device="cuda") for _ in "qk"]
    kw = dict(norm="rms", q_weight=w[0], k_weight=w[1], rope_scale=scale)
    cache = [torch.zeros(64, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    order = r.permutation(64).astype(np.int32)
    pre, table = ints(order[:3]), ints(order[3:23].reshape(2, 10))
    seen = [[], []]  # the definition's rotated keys and values of each sequence

    def project(n):
        wide = torch.tensor(r.standard_normal((n, (Hq + 2 * Hkv) * D)), dtype=torch.bfloat16, device="cuda")
        return [p.unflatten(1, (-1, D)) for p in wide.split([Hq * D, Hkv * D, Hkv * D], dim=1)]

    def exact(x, weight, positions):
        return ref.head_rows(host(x), host(weight), positions, fl, False, 1.0, "rms", 1e-6)[0]

    def attended(o, q, own, b_rows, see):
        """o against the definition: row i sees seen[b] and `see(i)` of its own rows."""
        for b, rows in enumerate(b_rows):
            for n, i in enumerate(rows):
                K = np.concatenate([s[0] for s in seen[b]] + [own[0][[rows[m] for m in see(b, n)]]])
                V = np.concatenate([s[1] for s in seen[b]] + [own[1][[rows[m] for m in see(b, n)]]])
                for h in range(Hq):
                    s = K[:, h // G] @ q[i, h] / np.sqrt(D)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    tol = (np.expm1(0.125) + 2.0 ** -7) * (p @ np.abs(V[:, h // G]))
                    assert (np.abs(host(o[i, h]) - p @ V[:, h // G]) <= tol).all()

    # the shared prefix, as the only sequence of its table
    q, k, v = project(prefix)
    gt.cache_append_rope(q, k, v, ints([0, prefix]), *cache, pre[None], ints([0]), freq, **kw)
    for s in seen:
        s.append((exact(k, w[1], range(prefix)), host(v)))
    # prompts of 30 and 5 rows: into the cache, and beside it for their own causal attention
    ctx, cu = ints([0, 0]), ints([0, 30, 35])
    q, k, v = project(35)
    ko, vo = (torch.empty(35, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo, new = gt.cache_append_rope(q, k, v, cu, *cache, table, ctx, freq, prefix_len=prefix, k_out=ko,
                                   v_out=vo, **kw)
    o, _ = gt.attend(qo, ko, vo, None, cu, *cache, table, ctx, prefix_pages=pre, prefix_len=prefix)
    at = [prefix + i for i in range(30)] + [prefix + i for i in range(5)]
    own = exact(k, w[1], at), host(v)
    rows = [list(range(30)), list(range(30, 35))]
    attended(o, exact(q, w[0], at), own, rows, lambda b, n: range(n + 1))
    for b in range(B):
        seen[b].append((own[0][rows[b]], own[1][rows[b]]))
    ctx = new
    # trees of 7 and 3 nodes: positions by depth, nothing joins the cache but the accepted path
    par = [-1, 0, 0, 1, 1, 2, 5, -1, 0, 1]
    depth = [0, 1, 1, 2, 2, 2, 3, 0, 1, 2]
    cu = ints([0, 7, 10])
    pos = gt.tree_positions(ints(par), cu, context_len=ctx, prefix_len=prefix)
    at = [prefix + (30 if i < 7 else 5) + d for i, d in enumerate(depth)]
    assert pos.tolist() == at
    q, k, v = project(10)
    qo, ko = gt.norm_rope(q, k, pos, freq, **kw)
    v = v.contiguous()
    o, _ = gt.attend(qo, ko, v, ints(par), cu, *cache, table, ctx, prefix_pages=pre, prefix_len=prefix)
    own = exact(k, w[1], at), host(v)
    rows = [list(range(7)), list(range(7, 10))]

    def path_to(b, n):
        first, up = (0, 7)[b], []
        while n >= 0:
            up.append(n)
            n = par[first + n]
        return up

    attended(o, exact(q, w[0], at), own, rows, path_to)
    path = [[0, 2, 5, 6], [0, 1, -1, -1]]
    ctx = gt.cache_append(ko, v, cu, *cache, table, ctx, path=ints(path), path_len=ints([4, 2]))
    for b in range(B):
        took = [rows[b][n] for n in path[b] if n >= 0]
        seen[b].append((own[0][took], own[1][took]))
    # a token each: into the cache, then attention to the cache alone
    q, k, v = project(2)
    cu = ints([0, 1, 2])
    qo, new = gt.cache_append_rope(q, k, v, cu, *cache, table, ctx, freq, prefix_len=prefix, **kw)
    o, _ = gt.attend(qo, None, None, None, cu, *cache, table, new, prefix_pages=pre, prefix_len=prefix)
    at = [prefix + 34, prefix + 7]
    own = exact(k, w[1], at), host(v)
    attended(o, exact(q, w[0], at), own, [[0], [1]], lambda b, n: [0])
    assert new.tolist() == [35, 8]


def calls():
    x = append_inputs([70, 3, 64], [5, 0, 64], 8, 2, 128, 128, 32, "bf16", "fused", "rms", seed=33)
    cu, ctx, table = ints(x["cu"]), ints(x["ctx"]), ints(x["table"])
    par = ints(parents([70, 3, 64], "random", np.random.default_rng(1)))
    pos = ints(x["positions"])
    kw = dict(norm="rms", q_weight=x["wq"], k_weight=x["wk"], rope_scale=x["scale"])

    def append(**k):
        q, n = gt.cache_append_rope(x["q"], x["k"], x["v"], cu, x["k_cache"], x["v_cache"], table, ctx,
                                    x["freq"], **kw, **k)
        return q, n, x["k_cache"], x["v_cache"]

    return {"tree_positions": lambda **k: (gt.tree_positions(par, cu, context_len=ctx, **k),),
            "norm_rope": lambda **k: gt.norm_rope(x["q"], x["k"], pos, x["freq"], **kw, **k),
            "cache_append_rope": append}


@pytest.mark.parametrize("name", ["tree_positions", "norm_rope", "cache_append_rope"])
def test_a_call_on_a_given_stream_and_in_a_graph(name):
    from tests.test_streams_gpu import litter
    call = calls()[name]
    first = [t.clone() for t in call()]
    other = torch.cuda.Stream()
    for _ in range(3):
        other.wait_stream(torch.cuda.current_stream())
        got = call(stream=other)
        litter()
        other.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    kw = {} if name == "norm_rope" else dict(N_max=70)
    with torch.cuda.graph(graph):
        got = call(**kw)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, first):
        if a.dim() == 4:  # (a cache: the rows that the call writes)
            touched = (a != 0).any(-1)
            assert torch.equal(a[touched], b[touched]) and touched.sum() == 137 * 2
        else:
            assert torch.equal(a, b)


def test_two_graphs_in_turn():
    """Two captured calls of different shapes, replayed in turn on changing inputs."""
    x = [append_inputs([40, 7], [3, 60], 8, 2, 128, 128, 32, "bf16", "fused", "rms", seed=21),
         append_inputs([5] * 9, [b for b in range(9)], 4, 4, 64, 20, 16, "f32", "dense", "unit", seed=22)]
    held = [[ints(y[n]) for n in ("cu", "table", "ctx")] for y in x]
    status = [torch.empty(len(y["ctx"]), dtype=torch.int32, device="cuda") for y in x]

    def call(i, inter, **kw):
        y, (cu, table, ctx) = x[i], held[i]
        return gt.cache_append_rope(y["q"], y["k"], y["v"], cu, y["k_cache"], y["v_cache"], table, ctx,
                                    y["freq"], prefix_len=11, norm=y["norm"], q_weight=y["wq"],
                                    k_weight=y["wk"], rope_scale=y["scale"], interleaved=inter,
                                    N_max=40, dev_status=status[i], **kw)

    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i, bool(i)))
        graphs.append(g)
    for turn in range(3):
        for y in x:
            for n in "qkv":
                y[n].copy_(torch.randn(y[n].shape, device="cuda"))
        before = [(y["k_cache"].clone(), y["v_cache"].clone()) for y in x]
        for i in (0, 1) if turn % 2 else (1, 0):
            status[i].fill_(-7)
            graphs[i].replay()
        for i, y in enumerate(x):
            assert (status[i] == 0).all()
            check_append(dict(y, prefix=11), bool(i), before[i], *outs[i])


def test_two_calls_at_once():
    """Two calls on two streams share nothing."""
    x = [inputs(3000, 16, 4, 128, 128, "bf16", "dense", seed=s, norm="rms") for s in (1, 2)]
    pos = [ints(y["positions"]) for y in x]  # (held: a freed one could be handed out again)

    def call(y, p, **kw):
        return gt.norm_rope(y["q"], y["k"], p, y["freq"], norm="rms", q_weight=y["wq"],
                            k_weight=y["wk"], rope_scale=y["scale"], **kw)

    first = [call(y, p) for y, p in zip(x, pos)]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(y, p, stream=s) for y, p, s in zip(x, pos, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, first):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_accepted_rows_agree_with_serving_definition():
    """The values' rows and lengths are those of the append without rotation."""
    x = append_inputs([9, 4], [3, 20], 0, 2, 64, 0, 8, "f32", "dense", None, seed=12)
    before = host(x["k_cache"]), host(x["v_cache"])
    _, n = run_append(x, False)
    k, v, m = serving.cache_append(host(x["k"]), host(x["v"]), x["cu"], *before, x["table"], x["ctx"])
    assert np.array_equal(host(x["k_cache"]), k) and np.array_equal(host(x["v_cache"]), v)
    assert n.tolist() == m.tolist()
