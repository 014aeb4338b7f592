"""clip_grad_norm's outputs are written by many CTAs at once: two that share
memory, or an output that is another tensor's input, would race.  CPU only."""

import pytest
import torch

import block_scaled_precision_02_gb300 as mxq


def test_outputs_that_share_memory_are_refused():
    a, b, c = torch.zeros(8), torch.zeros(8), torch.zeros(0)
    with pytest.raises(ValueError, match=r"grads\[2\] and grads\[0\] share memory"):
        mxq.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError, match=r"grads\[1\] and grads\[0\] share memory"):
        mxq.clip_grad_norm([a, a.view(2, 4)], 1.0)
    with pytest.raises(ValueError, match=r"out\[1\] and out\[0\] share memory"):
        mxq.clip_grad_norm([a, b], 1.0, out=[torch.zeros(8)] * 2)
    with pytest.raises(ValueError, match=r"out\[0\] and grads\[1\] share memory"):
        mxq.clip_grad_norm([a, b], 1.0, out=[b, a])


def test_lists_that_may_share_memory_pass_the_check():
    """Reading a tensor twice, writing each in place by name, and empty tensors: on to the device check."""
    a, b, c = torch.zeros(8), torch.zeros(8), torch.zeros(0)
    for call in (lambda: mxq.grad_norm([a, a]),
                 lambda: mxq.clip_grad_norm([a, a], 1.0, out=[torch.zeros(8), torch.zeros(8)]),
                 lambda: mxq.clip_grad_norm([a, b], 1.0, out=[a, b]),
                 lambda: mxq.clip_grad_norm([a, b], 1.0, out=[torch.zeros(8), b]),
                 lambda: mxq.clip_grad_norm([c, torch.zeros(0), a, c], 1.0),
                 lambda: mxq.clip_grad_norm([c, a], 1.0, out=[c, torch.zeros(8)])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
