"""Policy training of an output layer in MX precision, with every operator that
runs around the products:

    residual x (float32) -> layer norm straight to MX (row and column copies)
    -> logits = h W^T (MXFP8 product) -> clipped policy loss and its gradient
    -> gradient to MX E5M2 -> dW = dz^T h and dh = dz W (MXFP8 products)
    -> layer norm backward -> gradient norm, clipping into float32 buffers -> SGD

    python examples/policy_step.py [steps]

The task: every state has one good token and one bad one, and the policy is
trained on both with advantages +1 and -1.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_precision_02_gb300 as mxq  # noqa: E402


class OutputLayer:
    """Layer norm and projection to the vocabulary: float32 master parameters
    and the float32 buffers that clipped gradients go to."""

    def __init__(self, hidden: int, vocab: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.params = [torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda"),
                       torch.randn(vocab, hidden, device="cuda", generator=g) * hidden ** -0.5]
        self.grads = [torch.zeros_like(p) for p in self.params]

    def step(self, x, targets, old_logp, ref_logp, advantages, weights, lr=0.5, max_norm=1.0, beta=0.02):
        """One training step; returns (loss, logp, gradient norm, gradient of x)."""
        gamma, bias, w = self.params
        # forward: the norm writes both operands that the products read
        h, hs, hT, hTs, mean, rstd = mxq.mx_layer_norm(x, gamma, bias, fmt="e4m3", orientation="dual", sf_layout="mma")
        q, qs, qT, qTs = mxq.mx_quantize(w.bfloat16(), "e4m3", "dual", sf_layout="mma")
        logits = mxq.mx_gemm(h, hs, q, qs, "e4m3")
        old = mxq.policy_loss(logits, targets, torch.zeros_like(advantages), advantages, weights, grad=False)[1] \
            if old_logp is None else old_logp
        ref = old if ref_logp is None else ref_logp
        loss, logp, dz = mxq.policy_loss(logits, targets, old, advantages, weights, ref_logp=ref, beta=beta)
        # backward: E5M2 gradient beside E4M3 operands
        z, zs, zT, zTs = mxq.mx_quantize(dz, "e5m2", "dual", sf_layout="mma")
        dw = mxq.mx_gemm(zT, zTs, hT, hTs, "e5m2", b_fmt="e4m3")
        dh = mxq.mx_gemm(z, zs, qT, qTs, "e5m2", b_fmt="e4m3")
        dx, dgamma, dbias = mxq.layer_norm_backward(dh, x, mean, rstd, gamma)
        norm = mxq.clip_grad_norm([dgamma, dbias, dw], max_norm, out=self.grads)
        for p, g in zip(self.params, self.grads):
            p.add_(g, alpha=-lr)
        return loss, logp, norm, dx


def train(steps: int = 20, tokens: int = 512, hidden: int = 256, vocab: int = 1024, seed: int = 0):
    """Runs the task; returns the mean log-probability of the good and of the
    bad tokens per step, and the gradient norms."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    states = torch.randn(tokens // 2, hidden, device="cuda", generator=g)
    x = torch.cat([states, states])
    targets = torch.randint(vocab, (tokens,), device="cuda", generator=g)
    good = torch.arange(tokens, device="cuda") < tokens // 2
    advantages = torch.where(good, 1.0, -1.0)
    weights = torch.full((tokens,), 1.0 / tokens, device="cuda")
    layer = OutputLayer(hidden, vocab, seed + 1)
    history = []
    ref = None
    for _ in range(steps):
        loss, logp, norm, _ = layer.step(x, targets, None, ref, advantages, weights)
        ref = logp.clone() if ref is None else ref
        history.append(torch.stack([logp[good].mean(), logp[~good].mean(), norm[0], loss[0]]))
    return torch.stack(history).cpu()


if __name__ == "__main__":
    table = train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    print("step  logp(good)  logp(bad)  |gradient|    loss")
    for i, (a, b, n, l) in enumerate(table.tolist()):
        print(f"{i:4d}  {a:10.4f}  {b:9.4f}  {n:10.4f}  {l:8.4f}")
    assert mxq.last_device_status() == 0
