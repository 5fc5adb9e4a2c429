"""CPU: the attention takes its own kind of workspace and no other.  A linear's workspace is as
large, but holds partial results where the attention's joins count: no piece would be the last
one, and the output would keep what its memory held."""
import pytest
import torch

import w4a8_gemm_amd as w4

X = torch.zeros(3, 4, 128, dtype=torch.bfloat16)


class Other:
    def __init__(self):
        self.buf = torch.zeros(1 << 20, dtype=torch.uint8)


def _call(workspace):
    cache = w4.KVCacheMXFP4.empty(3, 2, 128, 16, device="cpu")
    return w4.attention_mxfp4(X, cache, torch.zeros(3, 4, dtype=torch.int32), torch.ones(3, dtype=torch.int32),
                              workspace=workspace)


@pytest.mark.parametrize("make", [Other, lambda: torch.zeros(1 << 20, dtype=torch.uint8), lambda: 1 << 20,
                                  lambda: w4.Workspace.__new__(w4.Workspace), lambda: False])
def test_other_workspaces_are_refused(make):
    workspace = make()
    if isinstance(workspace, w4.Workspace):
        workspace.nbytes, workspace.buf = 1 << 20, torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(TypeError, match="AttentionWorkspace"):
        _call(workspace)


def test_its_own_and_none_pass():
    for workspace in (None, w4.AttentionWorkspace(3, 1, 4, 2, 128, device="cpu")):
        with pytest.raises(ValueError, match="GPU"):              # the last check: the tensors are on the CPU
            _call(workspace)
