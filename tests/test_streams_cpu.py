"""A call's `stream=` without a GPU: whatever the binding allocates, copies or reads on the
caller's behalf belongs to that stream, as the kernels do.  (A workspace of the current stream
could be handed out again while the kernels on the other one still use it, and a copy of the
states be made after them.)  The library and the stream context are stand-ins."""

import contextlib

import pytest
import torch

import gated_deltanet_tree_gdn_gb300 as gt
from gated_deltanet_tree_gdn_gb300 import _binding

B, N, T, HQK, HV, D, PAGE, WIDTH = 2, 3, 6, 1, 2, 16, 4, 2
f = lambda *s: torch.zeros(*s)  # noqa: E731
i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
CU = torch.tensor([0, 3, 6], dtype=torch.int32)
TREE = (f(B, N, HQK, D), f(B, N, HQK, D), f(B, N, HV, D), f(B, N, HV), f(B, N, HV))
ROWS = (f(T, HQK, D), f(T, HQK, D), f(T, HV, D), f(T, HV), f(T, HV))
STATES, POOL = f(B, HV, D, D), f(4, HV, D, D)
PATH, LEN = i(B, 2), i(B)
CACHE = (f(8, PAGE, HQK, D), f(8, PAGE, HQK, D), i(B, WIDTH), i(B))

CALLS = {
    "verify": lambda s: gt.verify(*TREE, i(B, N), STATES, stream=s),
    "verify_recurrent": lambda s: gt.verify_recurrent(*TREE, i(B, N), STATES, stream=s),
    "commit": lambda s: gt.commit(PATH, LEN, f(B, HV, N, D), TREE[1], TREE[3], STATES, stream=s),
    "commit_verify": lambda s: gt.commit_verify(PATH, LEN, f(B, HV, N, D), TREE[1], TREE[3], STATES,
                                                *TREE, i(B, N), stream=s),
    "verify_packed": lambda s: gt.verify_packed(*ROWS, i(T), CU, POOL, stream=s),
    "commit_packed": lambda s: gt.commit_packed(PATH, LEN, f(HV, T, D), ROWS[1], ROWS[3], CU, POOL,
                                                stream=s),
    "commit_verify_packed": lambda s: gt.commit_verify_packed(
        PATH, LEN, f(HV, T, D), ROWS[1], ROWS[3], CU, POOL, *ROWS, i(T), CU, stream=s),
    "build_topw": lambda s: gt.build_topw(f(B, N, 2), 2, 3, stream=s),
    "prefill": lambda s: gt.prefill(*ROWS, CU, POOL, stream=s),
    "decode_step": lambda s: gt.decode_step(*(x[:B] for x in ROWS), POOL, stream=s),
    "attend": lambda s: gt.attend(f(T, HV, D), *ROWS[:2], i(T), CU, *CACHE, stream=s),
    "cache_append": lambda s: gt.cache_append(*ROWS[:2], CU, *CACHE, stream=s),
}


class Library:
    """Every entry point succeeds; workspaces have 64 bytes."""

    def __init__(self, launched):
        self.launched = launched

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace"):
                return 64
            self.launched.append(args[-1])
            return gt.OK
        return call


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [True, False])
def test_everything_of_a_call_is_on_its_stream(monkeypatch, name, given):
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
    monkeypatch.setattr(_binding, "load", lambda: Library(launched))
    monkeypatch.setattr(_binding, "_prefill_cache", {})
    monkeypatch.setattr(_binding, "_attend_cache", {})
    monkeypatch.setattr(_binding, "_raw_stream", lambda device: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for owner, what in ((torch, "empty"), (torch, "empty_like"), (torch.Tensor, "clone"),
                        (torch.Tensor, "item")):
        monkeypatch.setattr(owner, what, noted(what, getattr(owner, what)))
    stream = type("Stream", (), {"cuda_stream": "other"})()
    CALLS[name](stream if given else None)
    want = stream if given else "current"
    assert done and {where for _, where in done} == {want}
    assert launched == [want] or launched == [stream.cuda_stream]
