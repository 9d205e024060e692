"""Gradients against differences of a loss in 64 bits, along random directions,
with a tolerance that a wrong gradient fails."""
import torch

BF16 = 2.0 ** -8      # half a bf16 step, relative
DIRECTIONS = 16


def slopes_agree(got, loss, args, which, g, off, step=1e-5):
    """Whether got, the gradient of loss(*args) for args[which] (64-bit tensors), has the slopes of central differences
    along random directions d.  off bounds the norm of got's error.  got . d is then off by a normal variable of at
    most that deviation: 6 of them, and the difference's own error, some step^2 of the slope, beside it.  (Bounded by
    off times the norm of d, any gradient of about the right size would pass.)"""
    base = args[which]
    for _ in range(DIRECTIONS):
        d = torch.randn(base.shape, generator=g, device=base.device, dtype=torch.float64)
        lo, hi = list(args), list(args)
        lo[which], hi[which] = base - step * d, base + step * d
        slope = float(loss(*hi) - loss(*lo)) / (2 * step)
        along = float((got.double() * d).sum())
        if not abs(along - slope) <= 6 * off + 1e-6 * float(got.double().norm()):
            return False
    return True


def norm_loss(dy, eps):
    def loss(h, w):
        return (h * w / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + eps) * dy).sum()
    return loss


def experts_loss(dy, seg, I):
    """Of a13 [E, 2 I, H], a2 [E, H, I] and rows a [R, H] in segments: the local experts' SwiGLU layer, times dy."""
    def loss(a13, a2, a):
        total = 0
        for e in range(a13.shape[0]):
            s = slice(seg[e], seg[e + 1])
            gu = a[s] @ a13[e].t()
            total = total + ((gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]) @ a2[e].t() * dy[s]).sum()
        return total
    return loss
