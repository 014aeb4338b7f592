"""Workspaces of the training-step operators: every call has its own.  CPU only."""

import pytest
import torch

import block_scaled_precision_02_gb300 as mxq


def test_policy_loss_calls_share_no_workspace(monkeypatch):
    """A second call that starts before the first one's kernels have all been
    launched (another host thread on the same stream) has a workspace of its
    own, and no tensor outlives the calls in the module: a recorded graph is
    the only holder of the memory that it writes."""
    spaces = []

    def launch(name, device, *args):
        assert name == "mxq_policy_loss" and args[-1] >= 256 + 4 * 3
        spaces.append((args[-2], args[-1]))
        if len(spaces) == 1:
            call()

    def call():
        v = torch.zeros(3)
        return mxq.policy_loss(torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), v, v, v)

    monkeypatch.setattr(mxq, "_launch", launch)
    monkeypatch.setattr(mxq, "_same_device", lambda names, *ts: torch.device("cpu"))
    monkeypatch.setattr(mxq, "_size", lambda name, device, tokens: 256 + 4 * tokens)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    call()
    assert len(spaces) == 2 and spaces[0][0] != spaces[1][0]
    kept = [v for d in vars(mxq).values() if isinstance(d, dict) for v in d.values() if isinstance(v, torch.Tensor)]
    assert not kept
