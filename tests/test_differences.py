"""The comparison of gradients with differences (differences.py) passes right
gradients, rounded as the kernels round theirs, and fails wrong ones."""
import pytest
import torch

import differences as D


def rounded(t):
    return t.to(torch.bfloat16).double()


def norm_case():
    g = torch.Generator().manual_seed(2)
    h, dy = rounded(torch.randn(6, 200, generator=g)), rounded(torch.randn(6, 200, generator=g))
    w = rounded(1 + 0.3 * torch.randn(200, generator=g))
    r = 1 / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6)
    d = dy * w
    return g, h, w, dy, r, d, h * r


@pytest.mark.parametrize("mistake,passes", [(None, True), ("sign", False), ("twice", False), ("half", False), ("no projection", False),
                                            ("projection twice", False), ("projection over T", False), ("5% more", False)])
def test_norm_rows(mistake, passes):
    g, h, w, dy, r, d, n = norm_case()
    term = n * (d * n).mean(-1, keepdim=True)
    dx = {"sign": -r * (d - term), "twice": 2 * r * (d - term), "half": r * (d - term) / 2, "no projection": r * d,
          "projection twice": r * (d - 2 * term), "projection over T": r * (d - term * 200 / 6),
          "5% more": 1.05 * r * (d - term)}.get(mistake, r * (d - term))
    dx = rounded(dx)
    assert D.slopes_agree(dx, D.norm_loss(dy, 1e-6), [h, w], 0, g, D.BF16 * float(dx.norm())) == passes


@pytest.mark.parametrize("mistake,passes", [(None, True), ("sign", False), ("twice", False), ("bf16", False), ("row left out", False),
                                            ("unscaled rows", False)])
def test_norm_weight(mistake, passes):
    g, h, w, dy, r, d, n = norm_case()
    dw = {"sign": -(dy * n).sum(0), "twice": 2 * (dy * n).sum(0), "bf16": rounded((dy * n).sum(0)), "row left out": (dy * n)[1:].sum(0),
          "unscaled rows": (dy * h).sum(0)}.get(mistake, (dy * n).sum(0)).float()
    assert D.slopes_agree(dw, D.norm_loss(dy, 1e-6), [h, w], 1, g, 2.0 ** -20 * float(dw.norm())) == passes


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("mistake,passes", [(None, True), ("sign", False), ("half", False), ("gate and up swapped", False),
                                            ("no second part of silu'", False)])
def test_experts(which, mistake, passes):
    g = torch.Generator().manual_seed(5)
    E, H, I, seg = 3, 32, 24, [0, 20, 21, 50]
    w13, w2 = rounded(torch.randn(E, 2 * I, H, generator=g) * H ** -0.5), rounded(torch.randn(E, H, I, generator=g) * I ** -0.5)
    x, dy = rounded(torch.randn(50, H, generator=g)), rounded(torch.randn(50, H, generator=g))
    grads = [torch.zeros_like(w13), torch.zeros_like(w2), torch.zeros_like(x)]
    for e in range(E):
        s = slice(seg[e], seg[e + 1])
        gate, up = (x[s] @ w13[e].t()).chunk(2, -1)
        sg = torch.sigmoid(gate)
        dh = dy[s] @ w2[e]
        dgu = [dh * up * sg * (1 + (0 if mistake == "no second part of silu'" else gate * (1 - sg))), dh * gate * sg]
        dgu = torch.cat(dgu[::-1] if mistake == "gate and up swapped" else dgu, -1)
        grads[0][e], grads[1][e], grads[2][s] = dgu.t() @ x[s], dy[s].t() @ (gate * sg * up), dgu @ w13[e]
    got = rounded(grads[which]) * {"sign": -1, "half": 0.5}.get(mistake, 1)
    if which == 1 and mistake in ("gate and up swapped", "no second part of silu'"):
        passes = True                                        # (w2's gradient does not have that part)
    ok = D.slopes_agree(got, D.experts_loss(dy, seg, I), [w13, w2, x], which, g, 3 * D.BF16 * float(got.norm()))
    assert ok == passes
