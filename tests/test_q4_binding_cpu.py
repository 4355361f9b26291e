"""CPU tests of the 4-bit calls: the Python binding, and refusals of positional tables."""
import sys

import pytest

from tests.test_q4_cpu import _Args


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


@pytest.mark.parametrize("what", ["write", "decode", "prefill"])
def test_a_table_of_a_negative_number_of_rows_is_refused(lk, what):
    a = _Args(lk)
    a.cfg.cos_sin, a.cfg.max_pos = a.p, -1
    assert a.call(what) == -1
    assert "max_pos" in lk.lib.lazy_last_error().decode()
    a.cfg.max_pos = 0  # no rows: angles on the fly
    a.call(what, D=96)
    assert "head_dim" in lk.lib.lazy_last_error().decode()
    a.cfg.cos_sin, a.cfg.max_pos = None, -1  # without a table it says nothing
    import torch
    if not torch.cuda.is_available():
        assert a.call(what) in (-3, -4)
