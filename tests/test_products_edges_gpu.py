"""The products grouped by expert where ordinary values and sizes do not tell
a mistake: sums that a matrix instruction's own alignment would lose."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import products_ref as R
from gpu_util import DEV, announce
from test_products_gpu import BF, check_fp8_values, fp8_rows, fp8_weights, gen, rand, Rows

pytestmark = pytest.mark.gpu


def one_expert(n):
    return torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int64, device=DEV)


def fp32_product(q, p, wq, ws):
    """(sum, bound) of fp8 rows times weights whose 128 products of a group are exact and whose sums are fp32's."""
    a = (R.e4m3(q).unflatten(-1, (-1, 128)) * p.unsqueeze(-1)).flatten(-2)
    w = R.block_weights(wq, ws)
    return a @ w.t(), (a.shape[1] + 6 + a.shape[1] // 128) * R.U32 * (a.abs() @ w.abs().t())


@pytest.mark.parametrize("flags", [0, 7])
@pytest.mark.parametrize("n", [3, 100, 200, 300])
def test_quantised_swiglu_keeps_small_products_beside_large_ones(n, flags):
    """In every 8 neighbours two products of 2^16 cancel, and six of 2^2 are left: 2^-14 of the largest, 64 times
    what fp32 sums of such a group may be off by."""
    announce("fp8 swiglu, cancelling products, n=%d flags=%d" % (n, flags))
    g, K, I = gen(n), 256, 128
    code = lambda v: torch.tensor([v], device=DEV).to(torch.float8_e4m3fn).view(torch.uint8).item()   # noqa: E731
    q = torch.full((n, K), code(2.0), dtype=torch.uint8, device=DEV)
    q[:, 0::8], q[:, 1::8] = code(256.0), code(-256.0)
    flip = torch.rand(n, 1, generator=g, device=DEV) < 0.5                      # some rows the other way round
    q = torch.where(flip, q ^ 0x80, q)
    wq = torch.full((1, 2 * I, K), code(2.0), dtype=torch.uint8, device=DEV)
    wq[:, :, 0::8] = wq[:, :, 1::8] = code(256.0)
    wq[:, :, 2::8] = torch.randint(code(1.0), code(4.0), (1, 2 * I, K // 8), generator=g, device=DEV).to(torch.uint8)
    ws = torch.full((1, 2 * I // 128, K // 128), 2.0 ** -9, device=DEV)
    ids = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    # scales of the format, then the codes put in
    _, s = cdl.dispatch_fp8(torch.full((n, K), 448.0, dtype=BF, device=DEV), cdl.dispatch_layout(ids, 0, 1), rows=n,
                            scale_flags=flags)
    p = R.scales(s, flags, n, K // 128, n)
    assert bool((p == 1).all())
    y, err = fp32_product(q, p, wq[0], ws[0])
    assert float((err / y.abs()).max()) < 0.2
    h, dh = R.swiglu(y[:, :I], err[:, :I], y[:, I:], err[:, I:])
    hq, hs = cdl.grouped_swiglu_fp8(q, s, wq, ws, *one_expert(n), scale_flags=flags)
    check_fp8_values(h, dh, hq, R.scales(hs, flags, n, 1, n), flags & 1)


@pytest.mark.parametrize("counts,K,I", [([700], 1024, 512), ([100, 0, 180, 33], 640, 256)], ids=str)
def test_quantised_swiglu_lands_on_the_codes_of_exact_sums(counts, K, I):
    """The share of codes that differ from those of 64-bit sums is that of fp32 ones.  h is off by about
    2^-24 sqrt(K) of the sums' size, |h| by a few times that; a code changes where a border lies between, of which
    there are 8 to an octave: some 2^-24 sqrt(K) 4 8 of the values, less than one in 10^4 here."""
    announce("fp8 swiglu, share of other codes, %s K=%d" % (counts, K))
    r, g = Rows(counts, False), gen(K)
    q, s, p = fp8_rows(g, r, K, 0)
    wq, ws = fp8_weights(g, len(counts), 2 * I, K)
    hq, _ = cdl.grouped_swiglu_fp8(q, s, wq, ws, r.c, r.seg)
    other = total = 0
    for e, at in r.each():
        y, _ = fp32_product(q[at], p[at], wq[e], ws[e])
        h = (torch.sigmoid(y[:, :I]) * y[:, :I] * y[:, I:]).unflatten(-1, (-1, 128))
        scale = (h.abs().amax(-1, keepdim=True) / 448).float().double()
        want = (h / scale).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
        other += int((hq[at] != want).sum())
        total += want.numel()
    assert other < 1e-4 * total, (other, total)
