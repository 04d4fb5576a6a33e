"""The workspace of the single-launch NVFP4 cast while a graph is captured (CPU: the choice of memory alone)."""
import torch

import nvfp4_block_scaled_amax_gb300 as nv


def test_a_captured_call_has_its_own(monkeypatch):
    """Two graphs captured on one stream may be replayed on two at once, and an eager call on that stream may run before
    either: neither may share the barrier's counters with another, nor rely on zeros that only a replay writes."""
    dev, stream = torch.device("cpu"), 0x7F00DEAD
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(nv, "_workspaces", {})
    eager = nv.single_pass_workspace(dev, stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    a, b = nv.single_pass_workspace(dev, stream), nv.single_pass_workspace(dev, stream)
    assert len({t.data_ptr() for t in (eager, a, b)}) == 3 and not a.any() and a.numel() == eager.numel()
    other = nv.single_pass_workspace(dev, stream + 1)              # first seen in a capture: nothing of it is kept
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert nv.single_pass_workspace(dev, stream) is eager
    assert nv.single_pass_workspace(dev, stream + 1) is not other
    assert nv.single_pass_workspace(dev, stream + 1) is nv.single_pass_workspace(dev, stream + 1)
