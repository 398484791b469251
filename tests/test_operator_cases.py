"""The calls of perf/operators.py."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _operators():
    path = os.path.join(os.path.dirname(__file__), "..", "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators_under_test", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


def test_streams_have_attention_workspaces_of_their_own():
    """Calls of two streams may overlap: what one leaves in its workspace is not the other's to read."""
    ops = _operators()
    case = next(c for c in ops.listed() if c["name"] == "attn_tiny_8")
    state = ops.prepare(case, 1)
    torch.cuda.synchronize()
    outs = []
    for stream in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        with torch.cuda.stream(stream):
            outs.append(ops.run(state)["out"].clone())
        torch.cuda.synchronize()
    held = list(ops._workspaces.values())
    assert len({t.data_ptr() for t in held}) == 3
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert int(state["status"]) == 0
