"""CPU tests of the 4-bit calls' Python binding."""
import sys

import pytest


@pytest.fixture(scope="module")
def lk():
    import __graft_entry__
    __graft_entry__.build()
    import position_agnostic_kv_gb300 as m
    return m


def test_first_calls_of_two_threads(lk, monkeypatch):
    """A thread that finds torch bound skips the binding: by then every other name has to be there.  Looked
    at after each attribute of torch that the binding takes, which is where another thread can come in."""
    import torch
    names = ("_BF16", "_I32", "_I64", "_F32", "_U8", "_raw_stream", "_device_index")
    for n in names:
        monkeypatch.setattr(lk, n, None, raising=False)
        monkeypatch.delattr(lk, n)
    monkeypatch.setattr(lk, "_torch", None)
    seen = []

    class Watched:
        def __getattr__(self, name):
            seen.append(lk._torch is None or all(hasattr(lk, n) for n in names))
            return getattr(torch, name)

    with monkeypatch.context() as c:
        c.setitem(sys.modules, "torch", Watched())
        lk._bind_torch()
    assert seen and all(seen)
    assert lk._torch is not None and all(hasattr(lk, n) for n in names)
    lk._bind_torch()
    assert lk._torch is torch
