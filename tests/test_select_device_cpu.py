"""The allocating windowed and tree decodes ask for the workspace of the device
that their tensors are on: the size depends on that device's clusters, and the
call plans its splits there."""
import pytest
import torch

import mla_decode_context_gb300 as dcp


class _On(torch.Tensor):
    """A host tensor that says it is on cuda:1."""
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("now", [0, 1])
def test_workspace_is_that_of_the_tensors_device(monkeypatch, tree, now):
    current = [now]
    asked, called = [], []

    class Guard:
        def __init__(self, device):
            self.to = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.back, current[0] = current[0], self.to

        def __exit__(self, *exc):
            current[0] = self.back

    monkeypatch.setattr(dcp, "_device_now", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(dcp, "dcp_decode_select_workspace_size", lambda *a: asked.append(current[0]) or 0)
    monkeypatch.setattr(dcp, "_decode_select", lambda *a: called.append(a))
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    q = torch.zeros((2, 1, 576), dtype=torch.bfloat16).as_subclass(_On)
    args = [q, torch.zeros((1, 16, 576), dtype=torch.bfloat16), torch.zeros((1, 1), dtype=torch.int32),
            torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)]
    kw = dict(D=1, interleave=1, scale=1.0, max_seq_len=16, max_q_len=2)
    if tree:
        dcp.decode_partial_tree(*args, torch.zeros((2, 1), dtype=torch.int64), **kw)
    else:
        dcp.decode_partial_window(*args, window=4, **kw)
    assert asked == [1] and len(called) == 1 and current == [now]
