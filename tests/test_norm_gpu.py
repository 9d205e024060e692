"""The root-mean-square norm, its 8-bit form and gradient, and the fp8
conversions outside a scatter, against 64-bit forms (products_ref.py)."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import products_ref as R
from gpu_util import DEV, announce
from test_products_gpu import BF, FORMATS, check_fp8_values, gen, rand

pytestmark = pytest.mark.gpu

# both sides of every form: one wave (512, 1024 columns), the workgroup's 2048, 4096, 8192, rows read twice; odd widths
WIDTHS = [1, 2, 7, 8, 64, 127, 512, 513, 520, 1024, 1025, 1032, 2048, 2049, 2056, 4096, 4097, 4104, 7168, 8192, 8193, 8200, 20001]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm(H, residual):
    for T in (1, 3, 6, 130):
        announce("norm T=%d H=%d residual=%d" % (T, H, residual))
        g = gen(H + T)
        x, w = rand(g, T, H), rand(g, H, scale=0.3) + 1
        res = rand(g, T, H, scale=3.0) if residual else None
        got = cdl.rms_norm(x, w, res, 1e-5)
        h = x
        if residual:
            got, h = got
            assert torch.equal(h, (x.float() + res.float()).to(BF))
        y, err = R.norm(h.double(), w.double(), 1e-5)
        R.assert_within(got, y, R.to_bf16_bound(y, err))


@pytest.mark.parametrize("flags", FORMATS)
@pytest.mark.parametrize("H", [128, 256, 640, 1024, 1152, 2048, 2176, 4224, 7168, 8192, 8320, 16512])
def test_norm_fp8(H, flags):
    for T, residual in ((1, True), (5, False), (131, True)):
        announce("fp8 norm T=%d H=%d flags=%d" % (T, H, flags))
        g = gen(H + T + flags)
        x, w = rand(g, T, H), rand(g, H, scale=0.3) + 1
        x[:, :128] *= 100
        res = rand(g, T, H) if residual else None
        if T > 3:
            x[2] = 0
            if residual:
                res[2] = 0
        y = torch.empty(T, H, dtype=BF, device=DEV)
        got = cdl.rms_norm_fp8(x, w, res, scale_flags=flags, out=y)
        plain = cdl.rms_norm(x, w, res)
        h = x
        if residual:
            h = got[2]
            assert torch.equal(h, plain[1])
            plain = plain[0]
        assert torch.equal(y, plain)
        q, s = got[:2]
        ref, err = R.norm(h.double(), w.double(), 1e-6)
        p = R.scales(s, flags, T, H // 128, T)
        live = torch.ones(T, dtype=torch.bool, device=DEV)
        if T > 3:
            live[2] = False
            assert bool((q[2] & 127 == 0).all()) and bool((p[2] == (2.0 ** -127 if flags & 1 else 0)).all())
        check_fp8_values(ref[live], err[live], q[live], p[live], flags & 1)
        if flags & R.PACKED and (H // 128) % 4 and not flags & R.COLMAJOR:
            assert bool((s[:, -1] >> (8 * (H // 128 % 4)) == 0).all())
        # read back: the exact product of code and scale, rounded
        v = R.e4m3(q) * p.repeat_interleave(128, 1)
        R.assert_within(cdl.dequant_fp8(q, s, scale_flags=flags), v, v.abs() * (R.BF16 + R.U32) + R.TINY)
        # without the bf16 rows: the same 8-bit ones
        assert torch.equal(cdl.rms_norm_fp8(x, w, res, scale_flags=flags)[0], q)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_gradient(H, residual):
    for T in (1, 3, 130, 513, 1100 if H < 3000 else 520):
        announce("norm gradient T=%d H=%d residual=%d" % (T, H, residual))
        g = gen(H + T + 1)
        h, dy, w = rand(g, T, H, scale=2.0), rand(g, T, H), rand(g, H, scale=0.3) + 1
        dres = rand(g, T, H) if residual else None
        dx, dw = cdl.rms_norm_grad(dy, h, w, 1e-5, dres)
        want, err, want_w, err_w = R.norm_grad(dy.double(), h.double(), w.double(), 1e-5, dres.double() if residual else None)
        R.assert_within(dx, want, R.to_bf16_bound(want, err))
        assert dw.dtype == torch.float32
        R.assert_within(dw, want_w, err_w)


def test_norm_gradient_against_differences():
    announce("norm gradient, differences")
    g, T, H = gen(2), 6, 200
    h, dy, w = rand(g, T, H), rand(g, T, H), rand(g, H, scale=0.3) + 1

    def loss(a, b):
        return (a * b / torch.sqrt(a.pow(2).mean(-1, keepdim=True) + 1e-6) * dy.double()).sum()

    dx, dw = cdl.rms_norm_grad(dy, h, w)
    for got, at in ((dx, 0), (dw, 1)):
        args = [h.double(), w.double()]
        d = torch.randn(args[at].shape, generator=g, device=DEV, dtype=torch.float64)
        lo, hi = list(args), list(args)
        lo[at], hi[at] = args[at] - 1e-5 * d, args[at] + 1e-5 * d
        slope = float((loss(*hi) - loss(*lo)) / 2e-5)
        assert abs(float((got.double() * d).sum()) - slope) < R.BF16 * float(got.double().norm() * d.norm())


def test_empty_batches():
    announce("norm of no rows")
    w = torch.ones(128, dtype=BF, device=DEV)
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    assert cdl.rms_norm(x, w).shape == (0, 128)
    assert cdl.rms_norm_fp8(x, w)[0].shape == (0, 128)
    dw = torch.full((128,), 7.0, device=DEV)
    dx, _ = cdl.rms_norm_grad(x, x, w, dweight=dw)
    assert dx.shape == (0, 128) and bool((dw == 0).all())
    assert cdl.quant_fp8_blocks(torch.empty(0, 5, 128, dtype=BF, device=DEV))[0].shape == (0, 5, 128)
    assert cdl.dequant_fp8(torch.empty(0, 128, dtype=torch.uint8, device=DEV), torch.empty(0, 1, device=DEV)).shape == (0, 128)


@pytest.mark.parametrize("H", [520, 1111, 7168, 8200, 9001])
def test_outputs_in_place(H):
    """out and residual_out may be x or residual; the gradient's out may be any of its rows."""
    announce("norm in place H=%d" % H)
    g, T = gen(H), 40
    x, res, w, dy, dres = rand(g, T, H), rand(g, T, H), rand(g, H), rand(g, T, H), rand(g, T, H)
    y, h = cdl.rms_norm(x, w, res)
    for order in (0, 1):
        a, b = x.clone(), res.clone()
        cdl.rms_norm(a, w, b, out=a if order else b, residual_out=b if order else a)
        assert torch.equal(a if order else b, y) and torch.equal(b if order else a, h)
    a = x.clone()
    cdl.rms_norm(a, w, out=a)
    assert torch.equal(a, cdl.rms_norm(x, w))
    dx, dw = cdl.rms_norm_grad(dy, h, w, 1e-6, dres)
    for i in range(3):
        t = [dy.clone(), h.clone(), dres.clone()]
        got, gw = cdl.rms_norm_grad(t[0], t[1], w, 1e-6, t[2], out=t[i])
        assert torch.equal(got, dx) and torch.equal(gw, dw), i


def test_rows_at_odd_addresses():
    announce("norm of rows at 2-byte alignment")
    g, T, H = gen(4), 33, 1032
    x, res, w = rand(g, T, H), rand(g, T, H), rand(g, H)

    def odd(t):
        o = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return o.copy_(t)

    y, h = cdl.rms_norm(x, w, res)
    y2, h2 = cdl.rms_norm(odd(x), odd(w), odd(res), out=odd(x), residual_out=odd(x))
    assert torch.equal(h, h2)
    want, err = R.norm(h.double(), w.double(), 1e-6)
    R.assert_within(y2, want, R.to_bf16_bound(want, err))
    dx, dw = cdl.rms_norm_grad(odd(x), odd(h), odd(w), 1e-6, odd(res), out=odd(x))
    want, err, want_w, err_w = R.norm_grad(x.double(), h.double(), w.double(), 1e-6, res.double())
    R.assert_within(dx, want, R.to_bf16_bound(want, err))
    R.assert_within(dw, want_w, err_w)
    with pytest.raises(cdl.CdlError):
        cdl.rms_norm_fp8(odd(x)[:, :1024].contiguous().view(-1)[8:8 + 32 * 1024 - 1024 + 1][1:].view(31, 1024), w[:1024].contiguous())


def test_nonfinite_rows_stay_in_their_row():
    announce("norm of non-finite rows")
    g, T, H = gen(5), 9, 512
    x, w = rand(g, T, H), rand(g, H)
    want, want_q = cdl.rms_norm(x, w), cdl.rms_norm_fp8(x, w)
    bad = x.clone()
    bad[2, 5], bad[4, 6] = float("nan"), float("inf")
    fine = [0, 1, 3, 5, 6, 7, 8]
    y, (q, s) = cdl.rms_norm(bad, w), cdl.rms_norm_fp8(bad, w)
    assert torch.equal(y[fine], want[fine]) and torch.equal(q[fine], want_q[0][fine]) and torch.equal(s[fine], want_q[1][fine])
    assert bool(torch.isnan(y[2]).all()) and bool((q[2] & 127 == 127).all())
    # an infinite element: 1 / inf scales every finite one to zero, itself to NaN
    other = torch.arange(H, device=DEV) != 6
    assert bool((y[4][other] == 0).all()) and bool(torch.isnan(y[4, 6]))
    assert int(q[4, 6] & 127) == 127 and bool((q[4][other] & 127 == 0).all())


def test_norm_on_streams_and_in_graphs():
    announce("norm captured and replayed")
    g, T, H = gen(6), 700, 2592
    x, res, w, dy = rand(g, T, H), rand(g, T, H), rand(g, H), rand(g, T, H)
    x8, w8 = rand(g, 300, 1024), rand(g, 1024)
    bufs = [torch.zeros(T, H, dtype=BF, device=DEV) for _ in range(3)]
    bufs += [torch.zeros(H, device=DEV), torch.zeros(300, 1024, dtype=torch.uint8, device=DEV),
             cdl.new_scale_tensor(300, 1024, 7, DEV).zero_(), torch.zeros(300, 1024, dtype=BF, device=DEV)]
    ws = torch.empty(cdl.rms_norm_grad_workspace_size(T, H), dtype=torch.uint8, device=DEV)

    def run():
        cdl.rms_norm(x, w, res, out=bufs[0], residual_out=bufs[1])
        cdl.rms_norm_grad(dy, bufs[1], w, out=bufs[2], dweight=bufs[3], workspace=ws)
        cdl.rms_norm_fp8(x8, w8, scale_flags=7, out_q=bufs[4], out_scales=bufs[5])
        cdl.dequant_fp8(bufs[4], bufs[5], scale_flags=7, out=bufs[6])

    run()
    want = [b.clone() for b in bufs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want)), i
        x.copy_(x.flip(0))
        graph.replay()
        got = [b.clone() for b in bufs]
        run()
        assert all(torch.equal(a, b) for a, b in zip(bufs, got)), i
        x.copy_(x.flip(0))


@pytest.mark.parametrize("mats,N,K", [(1, 128, 128), (2, 1, 128), (3, 200, 384), (1, 129, 1024), (5, 640, 256)])
def test_weights_in_blocks(mats, N, K):
    announce("fp8 blocks %d x %d x %d" % (mats, N, K))
    g = gen(N + K)
    w = rand(g, mats, N, K)
    w[:, :, ::7] *= 1e3
    w[0, :, :128] = 0
    q, s = cdl.quant_fp8_blocks(w)
    assert s.shape == (mats, -(-N // 128), K // 128)
    v = w.double()
    for b in range(s.shape[1]):
        for c in range(K // 128):
            blk = v[:, 128 * b:128 * b + 128, 128 * c:128 * c + 128]
            assert torch.equal(s[:, b, c], (blk.abs().amax((1, 2)) / 448).float())
            p = s[:, b, c].double()[:, None, None]
            t = torch.where(p > 0, blk / torch.where(p > 0, p, 1.0), 0.0)
            got = R.e4m3(q[:, 128 * b:128 * b + 128, 128 * c:128 * c + 128])
            R.assert_within(got, t, torch.maximum(t.abs() * R.E4M3, torch.full_like(t, 2.0 ** -10)) * (1 + 2 * R.U32))
    assert bool((q[0, :, :128] & 127 == 0).all())


@pytest.mark.parametrize("flags", FORMATS)
def test_read_back_of_dispatched_rows(flags):
    """dequant_fp8 on what the dispatches write, padded buffers included."""
    announce("fp8 read-back flags=%d" % flags)
    g, T, H, E, k = gen(flags), 90, 640, 6, 2
    x = rand(g, T, H)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    lay, q, s = cdl.permute_fp8(x, ids, 0, E, scale_flags=flags)
    n = lay.num_rows()
    y = cdl.dequant_fp8(q, s, scale_flags=flags)
    v = R.e4m3(q[:n]) * R.scales(s, flags, q.shape[0], H // 128, q.shape[0])[:n].repeat_interleave(128, 1)
    R.assert_within(y[:n], v, v.abs() * (R.BF16 + R.U32) + R.TINY)
    _, q, s, mm, _ = cdl.permute_ll_fp8(x, ids, 0, E, 70, scale_flags=flags)
    y = cdl.dequant_fp8(q, s, scale_flags=flags)
    p = R.scales(s, flags, E * 70, H // 128, 70).view(E, 70, -1)
    for e in range(E):
        c = int(mm[e])
        v = R.e4m3(q[e, :c]) * p[e, :c].repeat_interleave(128, 1)
        R.assert_within(y[e, :c], v, v.abs() * (R.BF16 + R.U32) + R.TINY)
