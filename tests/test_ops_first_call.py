"""The binding's first call: what it takes from torch is there whole, or
not at all, whatever another thread does meanwhile."""
import sys

from bit_exact_matrix_amd import ops


def test_the_first_call_sets_everything_before_it_shows(monkeypatch):
    """_Call starts the binding where _torch is not set.  At every bytecode of
    the start, a thread that finds _torch finds the rest."""
    for name in ("_torch", "_dt", "_raw_stream"):
        monkeypatch.setattr(ops, name, None)
    half = []

    def look(frame, event, arg):
        if frame.f_code.co_filename != ops.__file__:
            return None
        frame.f_trace_opcodes = True
        if ops._torch is not None and (ops._dt is None or ops._raw_stream is None):
            half.append(frame.f_lineno)
        return look

    sys.settrace(look)
    try:
        ops._start()
    finally:
        sys.settrace(None)
    assert ops._torch is not None and ops._dt and ops._raw_stream
    assert not half


def test_the_functions_are_loaded_whole(monkeypatch):
    monkeypatch.setattr(ops, "_fns", None)
    seen = []

    def look(frame, event, arg):
        if frame.f_code.co_filename != ops.__file__:
            return None
        frame.f_trace_opcodes = True
        if ops._fns is not None:
            seen.append(len(ops._fns))
        return look

    sys.settrace(look)
    try:
        ops._load()
    finally:
        sys.settrace(None)
    assert set(seen) <= {len(ops.EXPORTED)}
