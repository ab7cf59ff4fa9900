"""Two threads' first calls at the same time: whoever sees that the host functions
have been looked up finds both of them."""
import sys

import pytest

import segmented_reduction_csr_gb300 as sr


@pytest.mark.skipif(not hasattr(sys, "monitoring"), reason="looks on between single instructions")
def test_both_functions_are_there_once_the_lookup_seems_done(monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(sr, "_raw_stream", None)
    monkeypatch.setattr(sr, "_current_device", None)
    steps, half = [], []

    def look(code, offset):
        # (another thread may run between any two of them)
        steps.append(offset)
        if sr._raw_stream is not None and sr._current_device is None:
            half.append(offset)
    mon, code = sys.monitoring, sr._find_host_functions.__code__
    mon.use_tool_id(mon.DEBUGGER_ID, "looking on")
    try:
        mon.register_callback(mon.DEBUGGER_ID, mon.events.INSTRUCTION, look)
        mon.set_local_events(mon.DEBUGGER_ID, code, mon.events.INSTRUCTION)
        sr._find_host_functions()
    finally:
        mon.set_local_events(mon.DEBUGGER_ID, code, mon.events.NO_EVENTS)
        mon.register_callback(mon.DEBUGGER_ID, mon.events.INSTRUCTION, None)
        mon.free_tool_id(mon.DEBUGGER_ID)
    assert sr._raw_stream is not None and sr._current_device is not None
    assert len(steps) > 5 and not half
