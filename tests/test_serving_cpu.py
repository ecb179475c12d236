"""Refusals of the serving operators that are answered before any CUDA call (no GPU needed),
and their fp64 definitions against closed forms."""

import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from gated_deltanet_tree_gdn_gb300 import _binding, build
from oracle import serving as ref


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return _binding.load()


def P(i=0, off=0):
    """Distinct, aligned placeholder pointers (no call here gets past the host checks)."""
    return ctypes.c_void_p((1 << 40) + (i << 34) + off)


def rule_dims(**kw):
    d = dict(B=2, N=16, Hqk=2, Hv=4, dk=64, dv=64, dtype=gt.BF16)
    d.update(kw)
    return gt.Dims(**d)


def prefill(lib, dims=None, T=32, n_slots=4, pool_out=None, q=P(0), cu=P(6), slot=P(9), ws=P(12),
            ws_bytes=1 << 60):
    return lib.gdn_tree_prefill(q, P(1), P(2), P(3), P(4), cu, T, P(7),
                                P(8) if pool_out is None else pool_out, slot, n_slots, P(10),
                                dims or rule_dims(), None, ws, ws_bytes, None)


def step(lib, dims=None, n_slots=4, pool_out=None, q=P(0), slot=P(9)):
    return lib.gdn_tree_decode_step(q, P(1), P(2), P(3), P(4), P(7),
                                    P(8) if pool_out is None else pool_out, slot, n_slots, P(10),
                                    dims or rule_dims(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=24), gt.EUNSUPPORTED), (dict(dv=144), gt.EUNSUPPORTED), (dict(dtype=2), gt.EUNSUPPORTED),
    (dict(Hv=3), gt.EINVAL), (dict(Hqk=0), gt.EINVAL), (dict(B=-1), gt.EINVAL),
    (dict(B=70000), gt.EUNSUPPORTED)])
def test_rule_dims(lib, kw, code):
    assert prefill(lib, rule_dims(**kw)) == code
    assert step(lib, rule_dims(**kw)) == code


def test_rule_arguments(lib):
    for call in (prefill, step):
        assert call(lib, q=None) == gt.EINVAL
        assert call(lib, q=P(0, 8)) == gt.EINVAL               # 8-byte aligned only
        assert call(lib, slot=None, n_slots=1) == gt.EINVAL    # fewer states than sequences
        assert call(lib, n_slots=-1) == gt.EINVAL
        assert call(lib, pool_out=P(7, 256)) == gt.EINVAL      # overlaps pool_in in part
        assert call(lib, rule_dims(B=0), q=None) == gt.OK      # nothing to do
    assert prefill(lib, cu=None) == gt.EINVAL
    assert prefill(lib, T=-1) == gt.EINVAL
    assert prefill(lib, rule_dims(N=-1)) == gt.EINVAL


def test_prefill_workspace(lib):
    """The workspace grows with the rows up to a bound, and one that is too small is refused.
    (Without a GPU no tensor map can be made: the chunked kernels are then not chosen.)"""
    d = rule_dims(N=5000, dk=128, dv=128)
    need = lib.gdn_tree_prefill_workspace(d, 10000)
    if need:
        assert prefill(lib, d, T=10000, ws_bytes=need - 1) == gt.EINVAL
        assert prefill(lib, d, T=10000, ws=None) == gt.EINVAL
        assert need <= lib.gdn_tree_prefill_workspace(d, 20000)
    assert lib.gdn_tree_prefill_workspace(rule_dims(N=5000, dk=64), 10000) == 0
    assert lib.gdn_tree_prefill_workspace(rule_dims(Hv=3), 10000) == 0
    assert lib.gdn_tree_prefill_workspace(d, 0) == 0


def attend_dims(**kw):
    d = dict(B=2, T=20, N=16, Hq=8, Hkv=2, D=128, dtype=gt.BF16, page_size=16, n_pages=64,
             table_width=8, prefix_len=40)
    d.update(kw)
    return gt.AttendDims(**d)


def attend(lib, dims=None, k=P(1), v=P(2), q=P(0), table=P(6), prefix=P(8), cache=P(5), ctx=P(7),
           ws=P(12), ws_bytes=1 << 60, parent=None):
    return lib.gdn_tree_attend(q, k, v, parent, P(4), cache, cache, table, ctx, prefix, 1.0, P(10),
                               P(11), dims or attend_dims(), None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=24), gt.EUNSUPPORTED), (dict(D=256), gt.EUNSUPPORTED), (dict(dtype=2), gt.EUNSUPPORTED),
    (dict(Hq=7), gt.EINVAL), (dict(Hkv=0), gt.EINVAL),
    (dict(page_size=0), gt.EINVAL), (dict(prefix_len=-1), gt.EINVAL), (dict(T=-1), gt.EINVAL),
    (dict(table_width=1 << 28), gt.EUNSUPPORTED), (dict(B=70000), gt.EUNSUPPORTED),
    (dict(n_pages=-1), gt.EINVAL), (dict(table_width=-1), gt.EINVAL)])
def test_attend_dims(lib, kw, code):
    assert attend(lib, attend_dims(**kw)) == code


def test_attend_arguments(lib):
    assert attend(lib, q=None) == gt.EINVAL
    assert attend(lib, q=P(0, 8)) == gt.EINVAL
    assert attend(lib, v=None) == gt.EINVAL          # k without v
    assert attend(lib, k=P(1, 4)) == gt.EINVAL
    assert attend(lib, table=None) == gt.EINVAL
    assert attend(lib, prefix=None) == gt.EINVAL     # a prefix without its pages
    assert attend(lib, cache=None) == gt.EINVAL
    assert attend(lib, ctx=None) == gt.EINVAL
    assert attend(lib, attend_dims(N=1025), parent=P(3)) == gt.EUNSUPPORTED  # (a chain may be longer)
    assert attend(lib, attend_dims(B=0), q=None) == gt.OK
    assert attend(lib, attend_dims(T=0), q=None) == gt.OK
    d = attend_dims()
    need = lib.gdn_tree_attend_workspace(d)
    if need:
        assert attend(lib, d, ws_bytes=need - 1) == gt.EINVAL
        assert attend(lib, d, ws=None) == gt.EINVAL
    assert lib.gdn_tree_attend_workspace(attend_dims(Hq=7)) == 0


def append(lib, dims=None, k=P(1), path=P(3), plen=P(4), Lmax=4, table=P(6), ctx=P(7), new=P(8)):
    return lib.gdn_tree_cache_append(k, P(2), path, plen, Lmax, P(5), P(9), P(10), table, ctx, new,
                                     dims or attend_dims(), None, None)


def test_append_arguments(lib):
    assert append(lib, k=None) == gt.EINVAL
    assert append(lib, k=P(1, 8)) == gt.EINVAL
    assert append(lib, path=None) == gt.EINVAL           # a length without a path
    assert append(lib, plen=None) == gt.EINVAL
    assert append(lib, Lmax=-1) == gt.EINVAL
    assert append(lib, table=None) == gt.EINVAL
    assert append(lib, ctx=None) == gt.EINVAL
    assert append(lib, new=P(7, 4)) == gt.EINVAL         # overlaps context_len
    assert append(lib, attend_dims(D=24)) == gt.EUNSUPPORTED
    assert append(lib, attend_dims(B=0), k=None) == gt.OK


def test_host_tensors_and_mixed_types_are_refused():
    t = torch.zeros
    rule = (t(4, 1, 16), t(4, 1, 16), t(4, 2, 16), t(4, 2), t(4, 2))
    cu, pool = t(2, dtype=torch.int32), t(1, 2, 16, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.prefill(*rule, cu, pool)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.decode_step(*rule, pool)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gt.decode_step(rule[0].half(), *rule[1:], pool)
    cache, one = t(2, 4, 1, 16), t(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.attend(t(4, 2, 16), t(4, 1, 16), t(4, 1, 16), None, cu, cache, cache, one[None], one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gt.cache_append(t(4, 1, 16), t(4, 1, 16), cu, cache, cache, one[None], one)


def test_delta_rule_definition_closed_forms():
    """beta = 0 leaves a decayed state; alpha = 1, beta = 1 and orthonormal keys store the
    values exactly (o_t of q = k_s is v_s)."""
    r = np.random.default_rng(0)
    T, d = 8, 16
    k = np.eye(d)[:T, None]
    v = r.standard_normal((T, 1, d))
    zero, one = np.zeros((T, 1)), np.ones((T, 1))
    pool = r.standard_normal((1, 1, d, d))
    _, out = ref.delta_rule(k, k, v, -one, zero, [0, T], pool, [0])
    assert np.allclose(out, pool * np.exp(-T))
    o, out = ref.delta_rule(k, k, v, zero, one, [0, T], 0 * pool, [0])
    assert np.allclose(o, v) and np.allclose(out[0, 0, :T], v[:, 0])


def test_attend_definition_closed_forms():
    """Equal scores average the values seen; the cache in pages is the cache in order."""
    r = np.random.default_rng(1)
    kc = r.standard_normal((3, 4, 1, 16))
    vc = r.standard_normal((3, 4, 1, 16))
    q, k, v = (r.standard_normal((2, 1, 16)) for _ in range(3))
    args = (q, k, v, [-1, -1], [0, 2], kc, vc, [[2, 0]], [5], [1], 3)
    o, lse, _ = ref.attend(*args, 0.0)
    rows = np.concatenate([vc[1, :3, 0], vc[2, :, 0], vc[0, :1, 0]])
    for i in range(2):
        assert np.allclose(o[i, 0], np.concatenate([rows, v[i]]).mean(0))
    assert np.allclose(lse, np.log(9))


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("kw", [
    dict(), dict(prefix_len=0), dict(B=32, T=4096, Hq=32, Hkv=8, table_width=256),
    dict(B=1, T=1, table_width=600), dict(B=40, T=40, prefix_len=4000), dict(B=3, T=700, Hkv=8)])
def test_attend_plan_knows_the_rows(lib, kw):
    """A promised N past the rows there are promises no more than those rows: the parts (whose
    place is the workspace) are planned for min(N, T)."""
    T = kw.get("T", 20)
    need = lib.gdn_tree_attend_workspace(attend_dims(**kw, N=T))
    for N in (T + 1, 1 << 20, INT_MAX):
        assert lib.gdn_tree_attend_workspace(attend_dims(**kw, N=N)) == need
