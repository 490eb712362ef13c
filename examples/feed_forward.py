"""A gated feed-forward layer trained and then served with 4-bit weights.

The layer is Y = H Wd with H = silu(X Wg) * (X Wu).  Training in FP32 fits it
to another layer's outputs: the block and its gradients (feedforward), the
products around them (gemm.matmul), the gradients clipped by their global norm
and a step of gradient descent.  The trained weights are then rounded to 4 bits
with group scales, and single tokens go through the quantised block and
projection.  Run ``python examples/feed_forward.py`` on a GB300.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from roofline_gb300 import build, feedforward as ff, gemm  # noqa: E402

WIDTH, HIDDEN, TOKENS, GROUP = 256, 768, 1024, 64


def make(seed, width=WIDTH, hidden=HIDDEN):
    """Wg and Wu (width x hidden) and Wd (hidden x width)."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * s[0] ** -0.5).cuda()
            for s in ((width, hidden), (width, hidden), (hidden, width))]


def train_step(X, target, W, lr, max_norm):
    """One step on the mean square error; returns the loss and the gradients' norm."""
    Wg, Wu, Wd = W
    H, G, U = ff.gated_ff(X, Wg, Wu, act="silu", save=True)
    diff = gemm.matmul(H, Wd) - target
    loss = diff.square().mean()
    dY = diff * (2.0 / diff.numel())
    dWd = gemm.matmul(H.t(), dY)
    dH = gemm.matmul(dY, Wd.t())
    _, dWg, dWu = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, act="silu", need_dx=False)
    norm = ff.clip_grad_norm([dWg, dWu, dWd], max_norm)
    for w, d in zip(W, (dWg, dWu, dWd)):
        w.sub_(d, alpha=lr)
    return loss, norm


def quantise(W, group=GROUP):
    """4-bit codes, scales and zero points of an N x K matrix (K a multiple of
    the group), each group over its own range."""
    w = W.view(W.shape[0], -1, group)
    lo, hi = w.amin(2), w.amax(2)
    scale = (hi - lo).clamp_min(1e-12) / 15
    zero = (-lo / scale).round().clamp(0, 15)
    code = ((w / scale[..., None]).round() + zero[..., None]).clamp(0, 15)
    code = code.to(torch.uint8).view(W.shape)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scale, zero


def serve(x, packed):
    """Y for a few tokens through the quantised layer: two launches."""
    (qg, sg, zg), (qu, su, zu), (qd, sd, zd) = packed
    H = ff.q4_gated(x, qg, sg, qu, su, zeros_g=zg, zeros_u=zu, group=GROUP, act="silu")
    return ff.q4_matmul(H, qd, sd, zeros=zd, group=GROUP)


def main(steps=300, lr=300.0, max_norm=0.01):
    build.build()
    teacher, W = make(1), make(2)
    g = torch.Generator().manual_seed(3)
    X = torch.randn(TOKENS, WIDTH, generator=g).cuda()
    target = gemm.matmul(ff.gated_ff(X, teacher[0], teacher[1]), teacher[2])
    losses = []
    for step in range(steps):
        loss, norm = train_step(X, target, W, lr, max_norm)
        if step % (steps // 6) == 0 or step == steps - 1:
            losses.append(float(loss))
            print(f"step {step:4d}  loss {float(loss):.5f}  gradient norm {float(norm):.5f}")
    # the codes are stored out x in: rows along the outputs
    packed = [quantise(w.t().contiguous()) for w in W]
    full = gemm.matmul(ff.gated_ff(X, W[0], W[1]), W[2])
    one = torch.cat([serve(X[i:i + 1], packed) for i in range(16)])
    error = float((one - full[:16]).norm() / full[:16].norm())
    print(f"16 tokens one at a time with 4-bit weights: {100 * error:.1f} % off the FP32 layer")
    assert gemm.check_status() == gemm.OK
    return losses, error


if __name__ == "__main__":
    main()
