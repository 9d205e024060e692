"""The root-mean-square norm where ordinary rows do not tell a mistake: squares
of very unlike size, and weights whose products leave fp32's range."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import differences as D
import products_ref as R
from gpu_util import DEV, announce
from test_products_gpu import BF, gen, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [512, 1024, 2048, 4096, 7168, 8320])
def test_sums_of_unlike_squares_keep_the_small_ones(H):
    """Of every 8 elements one is 2^12 to 2^13 and seven are near 1: an fp32 sum loses most of the squares of the seven
    beside 2^24 and more, some 2e-7 of the whole, and with it the codes of the values that lie that near to a border
    between two.  The codes have to be those of the fp32 values nearest to 64-bit ones."""
    announce("norm of unlike squares H=%d" % H)
    g, T = gen(H), (1 << 23) // H
    x = 1 + 0.25 * torch.randn(T, H, generator=g, device=DEV)
    x[:, ::8] = 4096 * (1 + torch.rand(T, 1, generator=g, device=DEV))             # (a scale of every row's own)
    x, w = x.to(BF), (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(BF)
    q, s = cdl.rms_norm_fp8(x, w, scale_flags=cdl.FP8_SCALE_UE8M0)
    h = x.double()
    y = h * w.double() / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6)
    want = (y.unflatten(-1, (-1, 128)) / s.double().unsqueeze(-1)).flatten(-2).float().to(torch.float8_e4m3fn)
    assert int((q != want.view(torch.uint8)).sum()) == 0


@pytest.mark.parametrize("power", [-100, 100])
@pytest.mark.parametrize("H", [100, 512, 2592, 9000, 9001])
def test_rows_far_from_one(H, power):
    """Rows of about 2^power, whose squares 32 bits do not hold, give what rows of about 1 give, and their gradient
    that of those times 2^-power."""
    announce("norm of rows of 2^%d H=%d" % (power, H))
    g, T = gen(H), 6
    x, w, dy = rand(g, T, H), rand(g, H, scale=0.3) + 1, rand(g, T, H)
    far = x * 2.0 ** power
    assert torch.equal(cdl.rms_norm(far, w, eps=0.0), cdl.rms_norm(x, w, eps=0.0))
    dx, dw = cdl.rms_norm_grad(dy, x, w, 0.0)
    fx, fw = cdl.rms_norm_grad(dy, far, w, 0.0)
    assert torch.equal(fw, dw) and torch.equal(fx.float() * 2.0 ** power, dx.float())


@pytest.mark.parametrize("H", [100, 512, 2048, 9000, 9001])
def test_infinite_weights_and_products_beyond_fp32(H):
    announce("norm with infinite weights and large products H=%d" % H)
    g, T = gen(H), 5
    x, w = rand(g, T, H), rand(g, H, scale=0.3) + 1
    w[3], w[H - 1] = float("inf"), float("-inf")
    x[1, 3] = 0
    y = cdl.rms_norm(x, w)
    want = x.double() / torch.sqrt(x.double().pow(2).mean(-1, keepdim=True) + 1e-6) * w.double()
    keep = torch.arange(H, device=DEV)
    keep = (keep != 3) & (keep != H - 1)
    a, b = y[:, ~keep].double(), want[:, ~keep]              # (infinite, or NaN where the element is zero)
    assert bool(((a == b) | (a.isnan() & b.isnan())).all()) and bool(torch.isnan(y[1, 3])) and bool(torch.isinf(y[0, 3]))
    ref, err = R.norm(x.double(), torch.where(keep, w, 0).double(), 1e-6)
    R.assert_within(y[:, keep], ref[:, keep], R.to_bf16_bound(ref, err)[:, keep])
    # h w = 2^140, h w r = 2^80
    x, w = rand(g, T, H) * 2.0 ** 60, rand(g, H) * 2.0 ** 80
    ref, err = R.norm(x.double(), w.double(), 1e-6)
    assert bool(torch.isinf((x.float() * w.float())).any())
    R.assert_within(cdl.rms_norm(x, w), ref, R.to_bf16_bound(ref, err))


@pytest.mark.parametrize("flags", [0, 1])
def test_quantised_infinite_values_are_the_dispatchs(flags):
    """A value that an infinite weight makes infinite is quantised as the dispatch quantises an infinite element."""
    announce("fp8 norm with infinite weights, flags %d" % flags)
    g, T, H = gen(flags), 4, 384
    x, w = rand(g, T, H), rand(g, H)
    w[200] = float("inf")
    y = torch.empty(T, H, dtype=BF, device=DEV)
    q, s = cdl.rms_norm_fp8(x, w, scale_flags=flags, out=y)
    assert bool(torch.isinf(y[:, 200]).all())
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    dq, ds = cdl.dispatch_fp8(y, cdl.dispatch_layout(ids, 0, 1), rows=T, scale_flags=flags)
    assert torch.equal(s[:, 1], ds[:, 1]) and torch.equal(q[:, 128:256], dq[:, 128:256])


@pytest.mark.parametrize("T,H", [(6, 200), (40, 2049), (3, 8320), (600, 64)])
def test_gradient_has_the_slopes_of_differences(T, H):
    announce("norm gradient, differences, T=%d H=%d" % (T, H))
    g = gen(T)
    h, dy, w = rand(g, T, H), rand(g, T, H), rand(g, H, scale=0.3) + 1
    args, loss = [h.double(), w.double()], D.norm_loss(dy.double(), 1e-6)
    dx, dw = cdl.rms_norm_grad(dy, h, w)
    _, _, _, err_w = R.norm_grad(dy.double(), h.double(), w.double(), 1e-6, None)
    assert D.slopes_agree(dx, loss, args, 0, g, R.BF16 * float(dx.double().norm()))
    assert D.slopes_agree(dw, loss, args, 1, g, float(err_w.norm()))


def test_residual_out_without_residual_is_ignored():
    """Whatever it is: it neither refuses the call nor takes it off the vector path, nor is written."""
    announce("norm, C entry points, residual_out without residual")
    g, T, H = gen(9), 5, 256
    x, w = rand(g, T, H), rand(g, H)
    want, (wq, ws) = cdl.rms_norm(x, w), cdl.rms_norm_fp8(x, w)
    rest = torch.full((T * H + 8,), 0x55, dtype=torch.uint8, device=DEV)
    y, q, s = torch.empty_like(want), torch.empty_like(wq), torch.empty_like(ws)
    stream = torch.cuda.current_stream().cuda_stream
    for off in (0, 1, 2):
        ro = rest.data_ptr() + off
        assert cdl.library().cdl_rms_norm(x.data_ptr(), None, w.data_ptr(), 1e-6, T, H, y.data_ptr(), ro, stream) == 0
        assert cdl.library().cdl_rms_norm_fp8(x.data_ptr(), None, w.data_ptr(), 1e-6, T, H, q.data_ptr(), s.data_ptr(), 0, None,
                                              ro, stream) == 0
        assert torch.equal(y, want) and torch.equal(q, wq) and torch.equal(s, ws) and bool((rest == 0x55).all())
