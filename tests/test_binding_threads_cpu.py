"""The paged calls' first use of torch, which any thread may make: whoever sees
that it has been made finds everything that it brings."""
import sys

import pytest

import latent_attention_b200 as P

NAMES = ("_I32", "_F32", "_FP8", "_U8", "_DTYPES", "_raw_stream", "_current_device")


@pytest.fixture
def unused(monkeypatch):
    monkeypatch.setattr(P, "_T", None)
    for n in NAMES:
        monkeypatch.setattr(P, n, None, raising=False)
        monkeypatch.delattr(P, n)


def test_the_mark_of_the_first_call_is_set_last(unused):
    seen = []

    def trace(frame, event, arg):                 # between any two lines of _torch
        if frame.f_code is P._torch.__code__:
            if P._T is not None:
                seen.append([n for n in NAMES if not hasattr(P, n)])
            return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        P._torch()
    finally:
        sys.settrace(old)
    assert P._T is not None and all(hasattr(P, n) for n in NAMES)
    assert seen and not any(seen), seen
