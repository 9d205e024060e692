"""The comparisons of experts_check.py take right outputs and refuse NaN and
wrong ones (CPU)."""
import pytest
import torch

import experts_check as C
import experts_ref as R


def mx(g, *shape):
    q = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8)
    return q, torch.randint(122, 127, (*shape[:-1], shape[-1] // 32), generator=g).to(torch.uint8)


def refused(check, *args):
    with pytest.raises(AssertionError):
        check(*args)


def test_grouped_comparison():
    g = torch.Generator().manual_seed(1)
    a, sa = mx(g, 9, 64)
    w, sw = mx(g, 2, 24, 64)
    counts, begins = [3, 4], [0, 4]
    canary = torch.full((1,), -7.5, dtype=torch.bfloat16)
    out = canary.expand(9, 24).contiguous()
    for e in range(2):
        at = slice(begins[e], begins[e] + counts[e])
        out[at] = (R.values(a[at], sa[at]) @ R.values(w[e], sw[e]).t()).to(torch.bfloat16)
    args = (a, sa, w, sw, counts, begins)
    C.check_grouped(*args, out, canary)
    for row, value in ((1, torch.nan), (7, torch.nan), (2, 1e4), (3, 0.0), (8, torch.nan)):
        bad = out.clone()
        bad[row, 5] = value
        refused(C.check_grouped, *args, bad, canary)
    refused(C.check_grouped, *args, torch.full_like(out, torch.nan), canary)


def test_swiglu_comparison():
    g = torch.Generator().manual_seed(2)
    a, sa = mx(g, 5, 64)
    w, sw = mx(g, 64, 64)
    gu = R.values(a, sa) @ R.values(w, sw).t()
    h = gu[:, :32] * torch.sigmoid(gu[:, :32]) * gu[:, 32:]
    codes, scales = R.quantise((h.float().view(torch.int32) >> 16).to(torch.int16).numpy().view("uint16"))
    # the definition at the 64-bit values: scales as of h cut to bf16, codes by the nearest grid point
    s = torch.from_numpy(scales)
    p = torch.exp2(s.double() - 127)
    up = h.unflatten(-1, (-1, 32)).abs().amax(-1) > 6 * p
    s = s + up.to(torch.uint8)
    p = torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    grid = torch.tensor(R.GRID, dtype=torch.float64)
    code = (h.abs() / p).unsqueeze(-1).sub(grid).abs().argmin(-1).to(torch.uint8) | ((h < 0).to(torch.uint8) << 3)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    C.check_swiglu(a, sa, w, sw, q, s, 32)
    bad = s.clone()
    bad[3] = 255
    refused(C.check_swiglu, a, sa, w, sw, q, bad, 32)
    bad = s.clone()
    bad[3] += 1
    refused(C.check_swiglu, a, sa, w, sw, q, bad, 32)


def test_layer_comparison():
    g = torch.Generator().manual_seed(3)
    T, H, I, L, k = 4, 32, 32, 3, 2
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    v13, v2 = torch.randn(L, 2 * I, H, generator=g).double(), torch.randn(L, H, I, generator=g).double()
    ids = torch.rand(T, L, generator=g).topk(k, -1).indices.to(torch.int32)
    wts = torch.softmax(torch.randn(T, k, generator=g), -1)
    out = R.layer(x.double(), ids, wts, v13, v2, 0)[0].to(torch.bfloat16)
    C.check_layer_output(out, x, ids, wts, v13, v2, 0)
    bad = out.clone()
    bad[2, 7] = torch.nan
    refused(C.check_layer_output, bad, x, ids, wts, v13, v2, 0)
    refused(C.check_layer_output, out * 1.1, x, ids, wts, v13, v2, 0)
