"""CPU: which workspaces a BitStackLinear keeps: captured graphs go on using those that it has outgrown, and one that is made
during a capture is zeroed by the graph alone."""
import torch

import residual_block_decomp_b200 as R


def linear():
    lin = R.BitStackLinear.__new__(R.BitStackLinear)
    lin.m, lin.d, lin.k, lin.plain, lin.handle = 512, 4096, 16, False, None
    lin.device, lin._ws, lin._outgrown = "cpu", None, []
    return lin


def test_workspaces_are_kept_for_captured_graphs():
    lin = linear()
    sizes = sorted({b: R.bs_workspace_bytes(512, 4096, 16, 3, b) for b in (1, 4, 16, 64)}.items(), key=lambda x: x[1])
    (small, a), (large, b) = sizes[0], sizes[-1]
    assert 0 < a < b
    first = lin.workspace(3, small)
    second = lin.workspace(3, large)
    assert second.numel() == b and lin._outgrown[0] is first and lin.workspace(3, small) is second


def test_a_workspace_of_a_capture_is_not_kept(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    capturing = True
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    lin = linear()
    during = lin.workspace(3, 16)
    capturing = False
    eager = lin.workspace(3, 16)
    assert eager is not during and lin.workspace(3, 16) is eager and not eager.any()
    capturing = True
    assert lin.workspace(3, 16) is eager              # large enough: zero between calls
