"""The operators in front of the attention without a GPU: refusals that are answered before any
CUDA call, the frequencies, and the fp64 definitions against closed forms."""

import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from gated_deltanet_tree_gdn_gb300 import _binding, build
from oracle import rope as ref
from tests.test_streams_cpu import Library


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _binding.load()


def P(i=0, off=0):
    """Distinct, aligned placeholder addresses (no call here gets past the host checks)."""
    return (1 << 40) + (i << 34) + off


T, HQ, HKV, D = 20, 8, 2, 64
S = _binding.HeadStrides


def shape(**kw):
    d = dict(B=2, T=T, N=16, Hq=HQ, Hkv=HKV, D=D, dtype=gt.BF16, page_size=16, n_pages=64,
             table_width=8, prefix_len=40)
    d.update(kw)
    return gt.AttendDims(**d)


def turn(**kw):
    d = dict(rotary_dim=32, interleaved=0, norm=1, scale=1.0, eps=1e-6)
    d.update(kw)
    return _binding.Rope(**d)


def norm_rope(lib, dims=None, rope=None, q=P(0), qs=(HQ * D, D), k=P(1), ks=(HKV * D, D), pos=P(2),
              freq=P(3), qw=P(4), kw=P(5), qo=P(6), qos=(HQ * D, D), ko=P(7), kos=(HKV * D, D)):
    return lib.gdn_tree_norm_rope(q, k, pos, freq, qw, kw, qo, ko,
                                  S(q=qs, k=ks, q_out=qos, k_out=kos), dims or shape(),
                                  rope or turn(), None)


def append(lib, dims=None, rope=None, freq=P(3), cu=P(8), cache=P(9), v_cache=P(10), table=P(11),
           ctx=P(12), new=P(13), status=None, **kw):
    x = dict(q=P(0), k=P(1), v=P(2), q_out=P(6), k_out=None, v_out=None)
    strides = dict(q=(HQ * D, D), k=(HKV * D, D), v=(HKV * D, D))
    strides.update({n + "_out": s for n, s in list(strides.items())})
    for n, v in kw.items():
        if n.endswith("_strides"):
            strides[n[:-8]] = v
        else:
            x[n] = v
    return lib.gdn_tree_cache_append_rope(
        x["q"], x["k"], x["v"], freq, P(4), P(5), cu, x["q_out"], x["k_out"], x["v_out"], cache,
        v_cache, table, ctx, new, S(**strides), dims or shape(), rope or turn(), status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=24), gt.EUNSUPPORTED), (dict(D=144), gt.EUNSUPPORTED), (dict(dtype=2), gt.EUNSUPPORTED),
    (dict(T=-1), gt.EINVAL), (dict(Hq=0), gt.EINVAL), (dict(Hkv=-1), gt.EINVAL),
    (dict(Hq=1 << 21), gt.EUNSUPPORTED)])
def test_dims(lib, kw, code):
    assert norm_rope(lib, shape(**kw)) == code
    assert append(lib, shape(**kw)) == code


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=31), dict(rotary_dim=66), dict(rotary_dim=-2), dict(interleaved=2),
    dict(norm=3), dict(norm=-1), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
    dict(norm=0)])  # (weights without a norm)
def test_rope(lib, kw):
    assert norm_rope(lib, rope=turn(**kw)) == gt.EINVAL
    assert append(lib, rope=turn(**kw)) == gt.EINVAL


def test_pointers(lib):
    for call in (norm_rope, append):
        assert call(lib, q=P(0, 8)) == gt.EINVAL               # 8-byte aligned only
        assert call(lib, k=P(1, 2)) == gt.EINVAL
        assert call(lib, freq=None) == gt.EINVAL               # a rotation without frequencies
        assert call(lib, freq=P(3, 4)) == gt.EINVAL
    assert norm_rope(lib, qo=None) == gt.EINVAL
    assert norm_rope(lib, ko=None) == gt.EINVAL
    assert norm_rope(lib, pos=None) == gt.EINVAL
    assert norm_rope(lib, pos=P(2, 2)) == gt.EINVAL
    assert norm_rope(lib, qw=P(4, 4)) == gt.EINVAL
    assert norm_rope(lib, q=None, k=None) == gt.EINVAL
    assert norm_rope(lib, shape(T=0), q=None, k=None) == gt.OK  # nothing to do
    assert norm_rope(lib, shape(T=0)) == gt.OK
    assert append(lib, k=None) == gt.EINVAL
    assert append(lib, v=None) == gt.EINVAL
    assert append(lib, q_out=None) == gt.EINVAL
    assert append(lib, cu=None) == gt.EINVAL
    assert append(lib, ctx=None) == gt.EINVAL
    assert append(lib, table=None) == gt.EINVAL
    assert append(lib, cache=None) == gt.EINVAL
    assert append(lib, v_cache=P(10, 8)) == gt.EINVAL
    assert append(lib, new=P(13, 2)) == gt.EINVAL
    assert append(lib, shape(page_size=0)) == gt.EINVAL
    assert append(lib, shape(prefix_len=-1)) == gt.EINVAL
    assert append(lib, shape(B=70000)) == gt.EUNSUPPORTED
    assert append(lib, shape(B=0), k=None, cu=None) == gt.OK


def test_strides(lib):
    """Rows and heads lie on 16 bytes; an output's do not overlap.  Those of a single row or head
    do not count."""
    for bad in ((HQ * D + 4, D), (HQ * D, D + 4), (-HQ * D, D), (HQ * D, -D)):
        assert norm_rope(lib, qs=bad) == gt.EINVAL
        assert norm_rope(lib, qos=bad) == gt.EINVAL
        assert append(lib, q_strides=bad) == gt.EINVAL
        assert append(lib, q_out_strides=bad) == gt.EINVAL
    assert append(lib, v_strides=(HKV * D + 4, D)) == gt.EINVAL
    for over in ((0, D), (HQ * D - 8, D), (HQ * D, 0), (HQ * D, D - 8), (D, D), (D, T * D - 8)):
        assert norm_rope(lib, qos=over) == gt.EINVAL
    assert norm_rope(lib, qs=(1 << 60, D)) == gt.EUNSUPPORTED
    assert norm_rope(lib, q=None, qs=(3, -5), ks=(1 << 60, D)) == gt.EUNSUPPORTED  # (k's, not q's)
    assert norm_rope(lib, q=None, qs=(3, -5), qos=(3, -5), ko=P(2)) == gt.EINVAL    # ko over positions
    # (a null freq is the last thing wrong: the strides before it were taken)
    assert norm_rope(lib, shape(Hq=1), qos=(D, 3), freq=None) == gt.EINVAL
    h = (1 << 60) * 8
    assert norm_rope(lib, shape(T=1), qs=(3, D), qos=(h, D), ko=P(0)) == gt.EINVAL  # ko over q


def test_overlaps(lib):
    """An output may be its own input; beside other columns of the same rows it is apart."""
    fused = (HQ + 2 * HKV) * D
    row = (fused, D)
    inplace = dict(q=P(0), qs=row, qo=P(0), qos=row, k=P(0, 2 * HQ * D), ks=row)
    assert norm_rope(lib, **inplace, ko=P(0, 2 * HQ * D), kos=row, pos=P(0, 64)) == gt.EINVAL
    # outputs in the other's place, shifted, or with other strides
    assert norm_rope(lib, qo=P(0), qos=(2 * HQ * D, D)) == gt.EINVAL
    assert norm_rope(lib, qo=P(0, 16)) == gt.EINVAL
    assert norm_rope(lib, qo=P(1)) == gt.EINVAL
    assert norm_rope(lib, ko=P(6)) == gt.EINVAL
    assert norm_rope(lib, **inplace, ko=P(0, 2 * (HQ - 1) * D), kos=row) == gt.EINVAL
    for small in (dict(pos=P(6)), dict(freq=P(6, 256)), dict(qw=P(7)), dict(kw=P(6, 16))):
        assert norm_rope(lib, **small) == gt.EINVAL
    assert append(lib, q_out=P(9)) == gt.EINVAL
    assert append(lib, k_out=P(6)) == gt.EINVAL
    assert append(lib, v_out=P(1)) == gt.EINVAL
    assert append(lib, k=P(9, 4096)) == gt.EINVAL
    assert append(lib, v_cache=P(9, 64)) == gt.EINVAL
    assert append(lib, new=P(12)) == gt.EINVAL
    assert append(lib, new=P(12, 4)) == gt.EINVAL
    assert append(lib, new=P(8, 8)) == gt.EINVAL
    assert append(lib, status=P(13, 4)) == gt.EINVAL
    assert append(lib, status=P(9, 64)) == gt.EINVAL


def positions(lib, parent=P(0), cu=P(1), ctx=P(2), prefix=0, out=P(3), B=2, T=20, N=16, status=None):
    return lib.gdn_tree_positions(parent, cu, ctx, prefix, out, B, T, N, status, None)


def test_positions_arguments(lib):
    assert positions(lib, cu=None) == gt.EINVAL
    assert positions(lib, out=None) == gt.EINVAL
    assert positions(lib, out=P(3, 2)) == gt.EINVAL
    assert positions(lib, out=P(0, 4)) == gt.EINVAL      # overlaps parent
    assert positions(lib, out=P(2)) == gt.EINVAL
    assert positions(lib, status=P(3, 4)) == gt.EINVAL
    assert positions(lib, status=P(2)) == gt.EINVAL
    assert positions(lib, N=1025) == gt.EUNSUPPORTED     # (a chain may be longer)
    for kw in (dict(B=-1), dict(T=-1), dict(N=-1), dict(prefix=-1)):
        assert positions(lib, **kw) == gt.EINVAL
    assert positions(lib, B=70000) == gt.EUNSUPPORTED
    assert positions(lib, B=0, cu=None) == gt.OK


@pytest.mark.parametrize("args", [
    dict(), dict(base=1e6), dict(base=5e5, stretch="linear", factor=7.5),
    dict(stretch="ntk", factor=4.0), dict(base=1e6, stretch="yarn", factor=32.0, trained_len=32768),
    dict(stretch="yarn", factor=4.0, trained_len=100.0, fast=8.0, slow=2.0),
    dict(base=5e5, stretch="bands", factor=8.0, trained_len=8192, fast=4.0, slow=1.0)], ids=str)
@pytest.mark.parametrize("R", [2, 20, 64, 128])
def test_frequencies(lib, R, args):
    """freq 2^-64 turns a position: within the few roundings of its evaluation in 64 bits (power,
    blend, division by 2 pi: 16 half steps of 2^-53) of the formula."""
    if R == 2 and args.get("stretch") == "ntk":
        with pytest.raises(gt.GdnTreeError):
            gt.rope_frequencies(R, device="cpu", **args)
        return
    freq, scale = gt.rope_frequencies(R, device="cpu", **args)
    f, s = ref.frequencies(R, args.get("base", 10000.0), **{k: v for k, v in args.items()
                                                            if k != "base"})
    want = (f / (2 * np.pi)).astype(np.float64)
    assert freq.dtype == torch.int64 and freq.shape == (R // 2,)
    got = freq.double().numpy() * 2.0 ** -64
    # (the power's exponent, up to ln(base) = 14 in size, is rounded before it)
    assert (np.abs(got - want) <= (16 + 16) * 2.0 ** -53 * want + 2.0 ** -64).all()
    assert abs(scale - s) <= 2.0 ** -23 * s


def test_frequencies_refused(lib):
    ok = dict(base=1e4, stretch="yarn", factor=4.0, trained_len=100.0)
    for R, kw in ((3, {}), (0, {}), (-2, {}), (64, dict(base=1.0)), (64, dict(base=math.nan)),
                  (64, dict(stretch="linear", factor=0.5)), (64, dict(ok, trained_len=0.0)),
                  (64, dict(ok, slow=0.0)), (64, dict(ok, fast=1.0)),
                  (64, dict(ok, factor=math.inf))):
        with pytest.raises(gt.GdnTreeError) as e:
            gt.rope_frequencies(R, device="cpu", **kw)
        assert e.value.code == gt.EINVAL
    with pytest.raises(gt.GdnTreeError) as e:
        gt.rope_frequencies(130, device="cpu")
    assert e.value.code == gt.EUNSUPPORTED
    with pytest.raises(ValueError, match="stretch"):
        gt.rope_frequencies(64, stretch="longer", device="cpu")
    bad = _binding.RopeStretch(9, 1.0, 1.0, 2.0, 1.0)
    out, s = (ctypes.c_uint64 * 32)(), ctypes.c_float()
    assert lib.gdn_tree_rope_frequencies(64, 1e4, bad, out, ctypes.byref(s)) == gt.EUNSUPPORTED
    bad.kind = 0
    assert lib.gdn_tree_rope_frequencies(64, 1e4, bad, None, ctypes.byref(s)) == gt.EINVAL


def test_host_tensors_and_mixed_types_are_refused():
    t = torch.zeros
    q, k = t(4, 2, 16), t(4, 1, 16)
    cu, one = t(2, dtype=torch.int32), t(1, dtype=torch.int32)
    cache = t(2, 4, 1, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.norm_rope(q, k)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.cache_append_rope(q, k, k, cu, cache, cache, one[None], one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.tree_positions(one, cu)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gt.norm_rope(q.half())
    with pytest.raises(ValueError, match="q or k"):
        gt.norm_rope(None)
    with pytest.raises(ValueError, match="together"):
        gt.norm_rope(q, positions=one)
    with pytest.raises(ValueError, match="together"):
        gt.norm_rope(q, freq=one.long())


def test_definitions_closed_forms():
    """Positions of 0 change nothing, a quarter turn swaps the pair, two rotations are one by the
    sum, and scores depend on the distance alone."""
    r = np.random.default_rng(0)
    x = r.standard_normal((3, 2, 16))
    quarter = np.full(4, 1 << 62, dtype=object)
    for inter in (False, True):
        assert np.allclose(ref.head_rows(x, None, [0] * 3, quarter, inter, 1.0, None, 0)[0], x)
        y = ref.head_rows(x, None, [1] * 3, quarter, inter, 2.0, None, 0)[0]
        i = np.arange(4)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
        assert np.allclose(y[..., a], -2 * x[..., b]) and np.allclose(y[..., b], 2 * x[..., a])
        assert np.array_equal(y[..., 8:], x[..., 8:])
    f = np.array([round(2.0 ** 64 * v) for v in (0.1, 0.01)], dtype=object)
    rot = lambda z, p: ref.head_rows(z, None, p, f, False, 1.0, None, 0)[0]  # noqa: E731
    assert np.allclose(rot(rot(x, [5, 6, 7]), [10 ** 6, -6, 2]), rot(x, [10 ** 6 + 5, 0, 9]))
    q, k = r.standard_normal((2, 1, 1, 16))
    at = lambda a, b: float((rot(q, [a]) * rot(k, [b])).sum())  # noqa: E731
    assert np.isclose(at(7, 3), at(10 ** 9 + 7, 10 ** 9 + 3))
    unit = ref.head_rows(x, None, None, None, False, 1.0, "unit", 0.0)[0]
    assert np.allclose((unit ** 2).sum(-1), 1)
    rms = ref.head_rows(x, np.full(16, 3.0), None, None, False, 1.0, "rms", 0.0)[0]
    assert np.allclose((rms ** 2).mean(-1), 9)
    p = ref.tree_positions([-1, 0, 0, 2, -1, -1, 0], [0, 5, 5, 7], [3, 0, 1], 10, 8, fill=-1)
    assert p.tolist() == [13, 14, 14, 15, 13, 11, 12, -1]


f32 = lambda *s: torch.zeros(*s)  # noqa: E731
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
CALLS = {
    "tree_positions": lambda s: gt.tree_positions(i32(6), torch.tensor([0, 3, 6]).int(), stream=s),
    "norm_rope": lambda s: gt.norm_rope(f32(6, 2, 16), f32(6, 1, 16), i32(6), i32(8).long(),
                                        norm="rms", q_weight=f32(16), stream=s),
    "cache_append_rope": lambda s: gt.cache_append_rope(
        f32(6, 2, 16), f32(6, 1, 16), f32(6, 1, 16), torch.tensor([0, 3, 6]).int(),
        f32(8, 4, 1, 16), f32(8, 4, 1, 16), i32(2, 2), i32(2), i32(4).long(), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [True, False])
def test_everything_of_a_call_is_on_its_stream(monkeypatch, name, given):
    """What the binding allocates or reads on the caller's behalf belongs to the call's stream.
    (The library and the stream context are stand-ins.)"""
    current, done, launched = ["current"], [], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    def noted(what, fn):
        def wrapped(*a, **k):
            done.append((what, current[-1]))
            return fn(*a, **k)
        return wrapped

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(_binding, "_check", lambda *a: None)
    monkeypatch.setattr(_binding, "_check_device", lambda *a: None)
    monkeypatch.setattr(_binding, "_refuse_device", lambda *a: None)
    monkeypatch.setattr(_binding, "_check_heads", lambda *a: None)
    monkeypatch.setattr(_binding, "load", lambda: Library(launched))
    monkeypatch.setattr(_binding, "_raw_stream", lambda device: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for owner, what in ((torch, "empty"), (torch.Tensor, "item")):
        monkeypatch.setattr(owner, what, noted(what, getattr(owner, what)))
    stream = type("Stream", (), {"cuda_stream": "other"})()
    CALLS[name](stream if given else None)
    want = stream if given else "current"
    assert done and {where for _, where in done} == {want}
    assert launched == [want] or launched == [stream.cuda_stream]


@pytest.fixture
def taken(monkeypatch):
    """Calls on host tensors that a stand-in of the library takes: what it was called with."""
    args = []

    class Takes:
        def __getattr__(self, name):
            return lambda *a: args.append(a) or gt.OK

    for name in ("_check", "_check_device", "_refuse_device", "_check_heads"):
        monkeypatch.setattr(_binding, name, lambda *a: None)
    monkeypatch.setattr(_binding, "load", Takes)
    monkeypatch.setattr(_binding, "_raw_stream", lambda device: 0)
    return args


def far_call(name, **kw):
    cu = torch.tensor([0, 3, 6]).int()
    if name == "tree_positions":
        return gt.tree_positions(i32(6), cu, **kw)
    return gt.cache_append_rope(None, f32(6, 1, 16), f32(6, 1, 16), cu, f32(8, 4, 1, 16),
                                f32(8, 4, 1, 16), i32(2, 2), i32(2), **kw)


@pytest.mark.parametrize("name", ["tree_positions", "cache_append_rope"])
@pytest.mark.parametrize("arg", ["prefix_len", "N_max"])
def test_values_that_32_bits_do_not_hold_are_refused(taken, name, arg):
    for far in (2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5, -2 ** 31 - 1, torch.tensor(2 ** 32 + 5)):
        with pytest.raises(ValueError, match=arg):
            far_call(name, **{arg: far})
    assert not taken
    far_call(name, **{arg: 2 ** 31 - 1})
    far_call(name, **{arg: -2 ** 31})  # (the library's own check refuses it)
    assert len(taken) == 2


def test_arrays_that_32_bits_do_not_count_are_refused(taken):
    """More rows than that: one that lies there once (and 5 are not what is left of them)."""
    rows = f32(1, 1, 16).expand(2 ** 32 + 5, 1, 16)
    one = i32(1).expand(2 ** 32 + 5)
    cu = torch.tensor([0, 3]).int()
    with pytest.raises(ValueError, match="T is 4294967301"):
        gt.cache_append_rope(None, rows, rows, cu, f32(8, 4, 1, 16), f32(8, 4, 1, 16), i32(1, 2),
                             i32(1), N_max=3)
    with pytest.raises(ValueError, match="T is 4294967301"):
        gt.norm_rope(None, rows, k_out=rows)
    with pytest.raises(ValueError, match="T is 4294967301"):
        gt.tree_positions(None, cu, positions=one, N_max=3)
    with pytest.raises(ValueError, match="B is 4294967300"):
        gt.tree_positions(None, one, T=3, N_max=3)
    with pytest.raises(ValueError, match="rotary_dim"):
        gt.norm_rope(None, f32(6, 1, 16), i32(6), i32(1).long().expand(2 ** 31 + 8))
    assert not taken
    for far in (2 ** 32 + 64, 2 ** 31, -2 ** 32 + 64):
        with pytest.raises(ValueError, match="rotary_dim"):
            gt.rope_frequencies(far, device="cpu")
    assert not taken


def test_very_many_frequencies_are_refused(lib):
    for R in (2 ** 31 - 2, 1 << 20):
        with pytest.raises(gt.GdnTreeError) as e:
            gt.rope_frequencies(R, device="cpu")
        assert e.value.code == gt.EUNSUPPORTED


@pytest.mark.parametrize("name", ["tree_positions", "cache_append_rope"])
@pytest.mark.parametrize("arg", ["prefix_len", "N_max"])
def test_lengths_that_are_no_whole_numbers_are_refused(taken, name, arg):
    """As by the calls that read the cache: 5.7 is not 5."""
    for part in (5.7, "5", torch.tensor(5.7), math.inf):
        with pytest.raises(TypeError):
            far_call(name, **{arg: part})
    assert not taken
    for whole in (5, np.int64(5), torch.tensor(5)):
        far_call(name, **{arg: whole})
    assert len(taken) == 3


@pytest.mark.parametrize("stretch", ["yarn", "bands"])
@pytest.mark.parametrize("trained_len", [2.0, 5.0, 2 * math.pi, 6.5, 40.0, 300.0, 4096.0, 1e30])
def test_which_pairs_are_slower(lib, stretch, trained_len):
    """Pairs that turn `slow` times or less in the trained length are slower by the factor, those
    that turn `fast` times or more are not, and the ones between are between: where all pairs are
    of one kind too."""
    R, factor, fast, slow = 64, 8.0, 4.0, 1.0
    freq, _ = gt.rope_frequencies(R, stretch=stretch, factor=factor, trained_len=trained_len,
                                  fast=fast, slow=slow, device="cpu")
    plain, _ = gt.rope_frequencies(R, device="cpu")
    for got, f in zip(freq.tolist(), plain.tolist()):
        turns = trained_len * f * 2.0 ** -64
        if turns <= slow * (1 - 1e-12):
            want = f / factor, f / factor
        elif turns >= fast * (1 + 1e-12):
            want = f, f
        else:
            want = f / factor, f
        # (4 roundings of 64 bits, and that to a whole number)
        assert want[0] * (1 - 2.0 ** -51) - 1 <= got <= want[1] * (1 + 2.0 ** -51) + 1
