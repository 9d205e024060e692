"""Plain 64-bit forms of the MXFP4 rows, the grouped product and the MoE layer
of a few tokens, with bounds on what fp32 accumulation and bf16 rounding may
change (no code shared with the kernels)."""
import numpy as np
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
U32 = 2.0 ** -23      # one fp32 operation, rounded or truncated
BF16 = 2.0 ** -8      # half a bf16 step, relative
TINY = 1e-30          # results that underflow bf16's or fp32's normal range


def quantise(bits):
    """(codes [rows, H] 0..15, scale bytes [rows, H / 32]) of bf16 bit
    patterns [rows, H] (numpy uint16), element by element from the definition."""
    rows, H = bits.shape
    with np.errstate(invalid="ignore"):                 # signalling NaNs among the patterns
        x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(rows, H // 32, 32)
    nan = np.isnan(x).any(-1)
    mag = np.abs(np.where(np.isnan(x), 0.0, x))
    amax = mag.max(-1)
    e = np.full(amax.shape, -127)
    for cand in range(-126, 128):                       # the smallest with 6 * 2^e >= amax
        e = np.where(6 * 2.0 ** (cand - 1) < amax, cand, e)
    with np.errstate(invalid="ignore", over="ignore"):
        t = mag / np.exp2(e.astype(np.float64))[..., None]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    code = (t[..., None] > mids).sum(-1)                # ties stay low ...
    for i, m in enumerate(mids):                        # ... unless the upper code is the even one
        if (i + 1) % 2 == 0:
            code = np.where(t == m, i + 1, code)
    sign = (bits >> 15).reshape(rows, H // 32, 32)
    code = np.where(nan[..., None], 0, code | (sign.astype(np.int64) << 3))
    return code.reshape(rows, H).astype(np.uint8), np.where(nan, 255, e + 127).astype(np.uint8)


def unpack(q):
    """Codes [..., H] of packed bytes [..., H / 2] (torch)."""
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def values(q, s):
    """float64 values of MXFP4 rows (torch, any device)."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=q.device)
    p = torch.exp2(s.to(torch.float64) - 127)
    p = torch.where(s == 255, torch.nan, p)
    return (grid[unpack(q).long()].unflatten(-1, (-1, 32)) * p.unsqueeze(-1)).flatten(-2)


def product(a, w):
    """(a @ w^T, bound on its fp32 error) in 64 bits: each of the K products is
    exact in fp32 up to one rounding, each of the K sums off by U32 of a
    partial sum, which the sum of magnitudes bounds."""
    y = a @ w.t()
    return y, (a.shape[1] + 2) * U32 * (a.abs() @ w.abs().t())


def swiglu(g, dg, u, du):
    """h = g / (1 + exp(-g)) * u and a bound on its error: |silu'| < 1.1; the
    exponential, its argument's product with log2(e), the sum, the division
    and the product are off by at most (8 + |g|) fp32 steps together."""
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * dg * (u.abs() + du) + s.abs() * du + (8 + g.abs()) * 2 * U32 * h.abs()


def bf16_step(v):
    """Distance between bf16 neighbours at v."""
    _, e = torch.frexp(v.abs())
    return torch.ldexp(torch.ones_like(v), e - 8)


def layer(x, ids, wts, w13, w2, expert_begin):
    """(out [T, H], bound) of the MoE layer in 64 bits; x, w13 [L, 2 I, H], w2
    [L, H, I] float64 values.  h is rounded to bf16 as the operator defines
    (up to two tokens keep the remainder); where the fp32 error could carry h over a rounding border the bound grows
    by that step."""
    T, k = ids.shape
    L, I = w13.shape[0], w13.shape[1] // 2
    H = x.shape[1]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    slots = 0
    for e in range(L):
        t, j = torch.nonzero(ids == e + expert_begin, as_tuple=True)
        if not len(t):
            continue
        gu, d = product(x[t], w13[e])
        h, dh = swiglu(gu[:, :I], d[:, :I], gu[:, I:], d[:, I:])
        if T <= 2:
            # h = hi + lo: the remainder is at most BF16 |h|, its rounding
            # loses at most BF16 of it (lo is exact in fp32: hi is h's nearest)
            hr, flip = h, dh + BF16 * BF16 * h.abs()
        else:
            hr = h.to(torch.bfloat16).double()
            step = bf16_step(hr)
            flip = torch.where((h - hr).abs() + dh > step / 2 * (1 - 2.0 ** -10), step + dh, 0.0)
        y, dy = product(hr, w2[e])
        dy = dy + flip @ w2[e].abs().t()
        w = wts[t, j].double().unsqueeze(1)
        out.index_add_(0, t, y * w)
        err.index_add_(0, t, dy * w.abs())
        mag.index_add_(0, t, hr.abs() @ w2[e].abs().t() * w.abs())
    n = k * (I // 32 + 4)                                # partial sums joined per output
    return out, err + n * U32 * mag + BF16 * (out.abs() + err) + TINY
