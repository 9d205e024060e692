"""The products grouped by expert in bf16 and fp8, their SwiGLU forms and
gradients against 64-bit forms (products_ref.py), at the sizes, masks and
values where they can go wrong."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import products_ref as R
from gpu_util import DEV, announce, status_word

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CANARY = -1.0e30
FORMATS = [0, 1, 2, 3, 5, 7]
# rows per expert: none, one, both sides of a wave's block, of a fragment set and of every tile size, several tiles
COUNTS = [[0, 1, 5, 0], [16, 17, 64, 65], [128, 129, 192, 193], [256, 257, 300, 0], [700, 3, 0, 0, 90], [1], [0], [513]]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


class Rows:
    """Places of the experts' rows: segments with gaps, or a padded buffer."""

    def __init__(self, counts, padded, gap=3):
        self.counts, self.padded = counts, padded
        self.cap = max(counts) + 2
        self.first, at = [], 0
        for e, c in enumerate(counts):
            self.first.append(e * self.cap if padded else at)
            at += c + (gap if e % 2 else 0)
        self.n = len(counts) * self.cap if padded else at + 4
        self.c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        self.seg = None if padded else torch.tensor(self.first + [at], dtype=torch.int64, device=DEV)
        self.live = torch.zeros(self.n, dtype=torch.bool, device=DEV)
        for e, c in enumerate(counts):
            self.live[self.first[e]:self.first[e] + c] = True

    def lead(self):
        return (len(self.counts), self.cap) if self.padded else (self.n,)

    def shape(self, t):
        return t.view(*self.lead(), *t.shape[1:])

    def poisoned(self, t):
        """The rows of no expert hold NaNs: no call may read them."""
        t = t.clone()
        t[~self.live] = 0x7F if t.dtype == torch.uint8 else float("nan")
        return t

    def each(self):
        for e, c in enumerate(self.counts):
            if c:
                yield e, slice(self.first[e], self.first[e] + c)

    def check_rest(self, out, canary):
        out = out.reshape(self.n, -1)
        assert torch.equal(out[~self.live], canary.expand_as(out[~self.live]))


def canaries(r, width):
    return torch.full((*r.lead(), width), CANARY, dtype=BF, device=DEV)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(64, 256), (200, 331), (8, 8), (584, 515), (1096, 72)])
def test_bf16_product(counts, K, N, padded):
    announce("bf16 %s K=%d N=%d padded=%d" % (counts, K, N, padded))
    r, g = Rows(counts, padded), gen(K + N)
    x, w = rand(g, r.n, K), rand(g, len(counts), N, K)
    st, out = status_word(), canaries(r, N)
    got = cdl.grouped_bf16(r.shape(r.poisoned(x)), w, r.c, r.seg, out=out, status=st)
    assert got is out and int(st.item()) == 0
    flat = out.view(r.n, N)
    for e, at in r.each():
        y, err = R.product(x[at].double(), w[e].double())
        R.assert_within(flat[at], y, R.to_bf16_bound(y, err), e)
    r.check_rest(out, torch.tensor(CANARY, dtype=BF, device=DEV))


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,I", [(64, 128), (200, 165), (8, 4), (584, 257), (72, 264)])
def test_bf16_swiglu_and_its_gradient(counts, K, I, padded):
    announce("bf16 swiglu %s K=%d I=%d padded=%d" % (counts, K, I, padded))
    r, g = Rows(counts, padded), gen(K + I)
    x, w, dh = rand(g, r.n, K), rand(g, len(counts), 2 * I, K, scale=K ** -0.5), rand(g, r.n, I)
    out, dgu = canaries(r, I), canaries(r, 2 * I)
    cdl.grouped_swiglu_bf16(r.shape(r.poisoned(x)), w, r.c, r.seg, out=out)
    cdl.grouped_swiglu_bf16_grad(r.shape(r.poisoned(x)), w, r.shape(r.poisoned(dh)), r.c, r.seg, out=dgu)
    for e, at in r.each():
        gu, d = R.product(x[at].double(), w[e].double())
        gate, up, eg, eu = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        h, err = R.swiglu(gate, eg, up, eu)
        R.assert_within(out.view(r.n, I)[at], h, R.to_bf16_bound(h, err), e)
        dg, bg, du, bu = R.swiglu_grad(gate, eg, up, eu, dh[at].double())
        R.assert_within(dgu.view(r.n, 2 * I)[at], torch.cat([dg, du], 1),
                        torch.cat([R.to_bf16_bound(dg, bg), R.to_bf16_bound(du, bu)], 1), e)
    for t in (out, dgu):
        r.check_rest(t, torch.tensor(CANARY, dtype=BF, device=DEV))


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(64, 256), (200, 328), (8, 8), (584, 520), (264, 1096)])
def test_bf16_gradients(counts, K, N, padded):
    announce("bf16 gradients %s K=%d N=%d padded=%d" % (counts, K, N, padded))
    r, g = Rows(counts, padded), gen(K + N + 1)
    L = len(counts)
    x, w, dy = rand(g, r.n, K), rand(g, L, N, K), rand(g, r.n, N)
    st, dx = status_word(), canaries(r, K)
    dw = torch.full((L, N, K), CANARY, dtype=BF, device=DEV)
    cdl.grouped_bf16_dx(r.shape(r.poisoned(dy)), w, r.c, r.seg, out=dx, status=st)
    cdl.grouped_bf16_dw(r.shape(r.poisoned(dy)), r.shape(r.poisoned(x)), r.c, r.seg, out=dw, status=st)
    assert int(st.item()) == 0
    for e, at in r.each():
        y, err = R.product(dy[at].double(), w[e].double().t())
        R.assert_within(dx.view(r.n, K)[at], y, R.to_bf16_bound(y, err), ("dx", e))
        y, err = R.product(dy[at].double().t(), x[at].double().t())
        R.assert_within(dw[e], y, R.to_bf16_bound(y, err), ("dw", e))
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e], torch.zeros_like(dw[e]))
    r.check_rest(dx, torch.tensor(CANARY, dtype=BF, device=DEV))


def fp8_rows(g, r, K, flags):
    """Quantised random rows in the format, by the framework's own dispatch: (q, scales, [rows, G] values)."""
    x = rand(g, r.n, K)
    ids = torch.zeros(r.n, 1, dtype=torch.int32, device=DEV)
    lay = cdl.dispatch_layout(ids, 0, 1)
    if r.padded and flags & R.COLMAJOR:
        L, cap = len(r.counts), r.cap
        parts = [cdl.dispatch_fp8(x[e * cap:(e + 1) * cap], cdl.dispatch_layout(ids[:cap], 0, 1), rows=cap,
                                  scale_flags=flags) for e in range(L)]
        q, s = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    else:
        q, s = cdl.dispatch_fp8(x, lay, rows=r.n, scale_flags=flags)
        if r.padded:
            s = r.shape(s)
    return q, s, R.scales(s, flags, r.n, K // 128, r.cap if r.padded else r.n)


def fp8_weights(g, L, N, K):
    w = rand(g, L, N, K, scale=K ** -0.5)
    w[:, ::3] *= 8
    return cdl.quant_fp8_blocks(w)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("flags", FORMATS)
@pytest.mark.parametrize("counts,K,N", [([0, 1, 5, 0], 128, 128), ([16, 17, 64, 65], 640, 331), ([128, 129, 192, 193], 256, 136),
                                        ([300, 0, 257], 384, 257), ([700, 3], 1152, 72), ([1], 512, 8)], ids=str)
def test_fp8_product(counts, K, N, flags, padded):
    announce("fp8 %s K=%d N=%d flags=%d padded=%d" % (counts, K, N, flags, padded))
    r, g = Rows(counts, padded), gen(K + N + flags)
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, len(counts), N, K)
    out = canaries(r, N)
    cdl.grouped_fp8(r.shape(r.poisoned(q)), s, wq, ws, r.c, r.seg, scale_flags=flags, out=out)
    for e, at in r.each():
        y, err = R.fp8_product(q[at], p[at], wq[e], ws[e])
        R.assert_within(out.view(r.n, N)[at], y, R.to_bf16_bound(y, err), e)
    r.check_rest(out, torch.tensor(CANARY, dtype=BF, device=DEV))


def check_fp8_values(h, dh, q, p, ue8m0):
    """Rows (q, scales p) against values h known to within dh."""
    hb, db = h.unflatten(-1, (-1, 128)), dh.unflatten(-1, (-1, 128))
    lo, hi = (hb.abs() - db).amax(-1), (hb.abs() + db).amax(-1)
    if ue8m0:
        assert bool((448 * p >= lo).all()) and bool(((p <= 2.0 ** -127) | (224 * p < hi)).all())
    else:
        assert bool((p >= lo / 448 * (1 - R.U32)).all()) and bool((p <= hi / 448 * (1 + R.U32)).all())
    v = R.e4m3(q).unflatten(-1, (-1, 128)) * p.unsqueeze(-1)
    t = (hb.abs() + db) / p.unsqueeze(-1)
    half = torch.maximum(t * R.E4M3, torch.full_like(t, 2.0 ** -10)) * p.unsqueeze(-1)
    R.assert_within(v, hb, half * (1 + 4 * R.U32) + db + 448 * p.unsqueeze(-1) * R.U32)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("flags", FORMATS)
@pytest.mark.parametrize("counts,K,I", [([0, 1, 5, 0], 128, 128), ([16, 17, 64, 65], 640, 384), ([128, 129, 192, 193], 256, 640),
                                        ([300, 0, 257], 384, 256)], ids=str)
def test_fp8_swiglu(counts, K, I, flags, padded):
    announce("fp8 swiglu %s K=%d I=%d flags=%d padded=%d" % (counts, K, I, flags, padded))
    r, g = Rows(counts, padded), gen(K + I + flags)
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, len(counts), 2 * I, K)
    oq = torch.full((*r.lead(), I), 0xA5, dtype=torch.uint8, device=DEV)
    gq, gs = cdl.grouped_swiglu_fp8(r.shape(r.poisoned(q)), s, wq, ws, r.c, r.seg, scale_flags=flags, out_q=oq)
    assert gq is oq
    hp = R.scales(gs, flags, r.n, I // 128, r.cap if padded else r.n)
    for e, at in r.each():
        gu, d = R.fp8_product(q[at], p[at], wq[e], ws[e])
        h, dh = R.swiglu(gu[:, :I], d[:, :I], gu[:, I:], d[:, I:])
        check_fp8_values(h, dh, gq.view(r.n, I)[at], hp[at], flags & 1)
        if flags & R.PACKED and (I // 128) % 4:        # the last word's unused bytes are zero
            w = gs.reshape(-1, gs.shape[-1]) if not flags & R.COLMAJOR else None
            if w is not None:
                assert bool((w[at][:, -1] >> (8 * (I // 128 % 4)) == 0).all())
    r.check_rest(gq.view(r.n, I), torch.tensor(0xA5, dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------------------
# strides, alignment, limits of the arrays
# ---------------------------------------------------------------------------

def test_outputs_that_are_only_element_aligned():
    announce("bf16 and fp8 products into odd addresses")
    g, K, N, n = gen(3), 256, 264, 200
    x, w = rand(g, n, K), rand(g, 1, N, K)
    c, seg = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int64, device=DEV)
    buf = torch.full((n * N + 64,), CANARY, dtype=BF, device=DEV)
    want = cdl.grouped_bf16(x, w, c, seg)
    for off in (1, 4, 7):
        buf.fill_(CANARY)
        cdl.grouped_bf16(x, w, c, seg, out=buf[off:off + n * N].view(n, N))
        assert torch.equal(buf[off:off + n * N].view(n, N), want)
        assert bool((buf[:off] == buf[-1]).all()) and bool((buf[off + n * N:] == buf[-1]).all())
    sw = cdl.grouped_swiglu_bf16(x, w, c, seg)
    cdl.grouped_swiglu_bf16(x, w, c, seg, out=buf[1:1 + n * N // 2].view(n, N // 2))
    assert torch.equal(buf[1:1 + n * N // 2].view(n, N // 2), sw)
    dh = rand(g, n, N // 2)
    odd = torch.empty(dh.numel() + 1, dtype=BF, device=DEV)[1:].view_as(dh)
    odd.copy_(dh)
    assert torch.equal(cdl.grouped_swiglu_bf16_grad(x, w, odd, c, seg), cdl.grouped_swiglu_bf16_grad(x, w, dh, c, seg))


def test_counts_that_do_not_fit_are_cut_and_reported():
    announce("products with counts beyond the buffer")
    g, K, N, n = gen(4), 64, 136, 40
    x, w, dy = rand(g, n, K), rand(g, 3, N, K), rand(g, n, N)
    seg = torch.tensor([0, 30, 38, 45], dtype=torch.int64, device=DEV)
    c = torch.tensor([30, 8, 7], dtype=torch.int32, device=DEV)        # the last: 2 rows fit
    cut = torch.tensor([30, 8, 2], dtype=torch.int32, device=DEV)
    for f in (lambda c, st: cdl.grouped_bf16(x, w, c, seg, out=torch.zeros(n, N, dtype=BF, device=DEV), status=st),
              lambda c, st: cdl.grouped_bf16_dx(dy, w, c, seg, out=torch.zeros(n, K, dtype=BF, device=DEV), status=st),
              lambda c, st: cdl.grouped_bf16_dw(dy, x, c, seg, status=st)):
        st, st0 = status_word(), status_word()
        assert torch.equal(f(c, st), f(cut, st0))
        assert int(st.item()) == cdl.CDL_STATUS_ROWS_OVERFLOW and int(st0.item()) == 0
    bad = torch.tensor([-5, 1 << 30, 8], dtype=torch.int32, device=DEV)
    wild = torch.tensor([0, -7, 1 << 40, 3], dtype=torch.int64, device=DEV)
    st = status_word()
    out = cdl.grouped_bf16(x, w, bad, wild, out=torch.full((n, N), CANARY, dtype=BF, device=DEV), status=st)
    assert int(st.item()) == cdl.CDL_STATUS_ROWS_OVERFLOW and bool((out == out[0, 0]).all())
    # padded: cap rows at most
    xp, dyp = x.view(2, 20, K), dy.view(2, 20, N)
    st = status_word()
    over = torch.tensor([21, 20], dtype=torch.int32, device=DEV)
    full = torch.tensor([20, 20], dtype=torch.int32, device=DEV)
    assert torch.equal(cdl.grouped_bf16(xp, w[:2], over, status=st), cdl.grouped_bf16(xp, w[:2], full))
    assert int(st.item()) == cdl.CDL_STATUS_LL_OVERFLOW
    st = status_word()
    assert torch.equal(cdl.grouped_bf16_dw(dyp, xp, over, status=st), cdl.grouped_bf16_dw(dyp, xp, full))
    assert int(st.item()) == cdl.CDL_STATUS_LL_OVERFLOW


@pytest.mark.parametrize("L", [65, 700, 2048])
def test_many_experts(L):
    announce("products of %d experts" % L)
    g, K, N = gen(L), 128, 128
    counts = [(7 * e) % 5 for e in range(L)]
    r = Rows(counts, False, gap=0)
    x, w, dy = rand(g, r.n, K), rand(g, L, N, K), rand(g, r.n, N)
    y, dx = cdl.grouped_bf16(x, w, r.c, r.seg), cdl.grouped_bf16_dx(dy, w, r.c, r.seg)
    dw = cdl.grouped_bf16_dw(dy, x, r.c, r.seg)
    q, s, p = fp8_rows(g, r, K, 0)
    wq, ws = fp8_weights(g, L, N, K)
    y8 = cdl.grouped_fp8(q, s, wq, ws, r.c, r.seg)
    for e, at in list(r.each())[:20] + list(r.each())[-20:]:
        for out, (v, err) in ((y[at], R.product(x[at].double(), w[e].double())),
                              (dx[at], R.product(dy[at].double(), w[e].double().t())),
                              (dw[e], R.product(dy[at].double().t(), x[at].double().t())),
                              (y8[at], R.fp8_product(q[at], p[at], wq[e], ws[e]))):
            R.assert_within(out, v, R.to_bf16_bound(v, err), e)
    assert bool((dw[r.c == 0] == 0).all()) and int((r.c == 0).sum()) > L // 8


def test_rows_and_weights_beyond_32_bit_offsets():
    announce("products over operands of more than 4 GiB")
    g = gen(9)
    # rows: the last expert's lie beyond 2^32 bytes of x, dy and out
    K, N, n = 4096, 4096, 540000
    x = torch.zeros(n, K, dtype=BF, device=DEV)
    tail = n - 70
    x[tail:] = rand(g, 70, K)
    w = rand(g, 2, N, K, scale=K ** -0.5)
    c = torch.tensor([3, 70], dtype=torch.int32, device=DEV)
    seg = torch.tensor([0, tail, n], dtype=torch.int64, device=DEV)
    out = torch.full((n, N), CANARY, dtype=BF, device=DEV)
    cdl.grouped_bf16(x, w, c, seg, out=out)
    y, err = R.product(x[tail:].double(), w[1].double())
    R.assert_within(out[tail:], y, R.to_bf16_bound(y, err))
    assert bool((out[:3] == 0).all()) and bool((out[3:3000] == out[3, 0]).all()) and bool((out[tail - 3000:tail] == out[3, 0]).all())
    cdl.grouped_bf16_dx(x, w, c, seg, out=out)
    y, err = R.product(x[tail:].double(), w[1].double().t())
    R.assert_within(out[tail:], y, R.to_bf16_bound(y, err))
    dw = cdl.grouped_bf16_dw(x, x, c, seg)
    y, err = R.product(x[tail:].double().t(), x[tail:].double().t())
    R.assert_within(dw[1], y, R.to_bf16_bound(y, err))
    del x, out, dw, y, err
    # weights: the last expert's lie beyond 2^32 bytes
    L, K, N = 3, 32768, 32768 + 8
    w = torch.zeros(L, N, K, dtype=BF, device=DEV)
    w[2, -40:] = rand(g, 40, K, scale=K ** -0.5)
    x, c = rand(g, 5, K), torch.tensor([0, 0, 5], dtype=torch.int32, device=DEV)
    seg = torch.tensor([0, 0, 0, 5], dtype=torch.int64, device=DEV)
    y, err = R.product(x.double(), w[2, -40:].double())
    out = cdl.grouped_bf16(x, w, c, seg)
    R.assert_within(out[:, -40:], y, R.to_bf16_bound(y, err))
    assert bool((out[:, :-40] == 0).all())
    dy = torch.zeros(5, N, dtype=BF, device=DEV)
    dy[:, -40:] = rand(g, 5, 40)
    y, err = R.product(dy[:, -40:].double(), w[2, -40:].double().t())
    R.assert_within(cdl.grouped_bf16_dx(dy, w, c, seg), y, R.to_bf16_bound(y, err))


# ---------------------------------------------------------------------------
# values
# ---------------------------------------------------------------------------

def test_infinite_and_nan_operands_reach_their_own_results_only():
    announce("non-finite operands of the products")
    g, K, N, n = gen(5), 200, 136, 150
    x, w, dy = rand(g, n, K), rand(g, 1, N, K), rand(g, n, N)
    c, seg = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int64, device=DEV)
    base = cdl.grouped_bf16(x, w, c, seg)
    xn, wn, dyn = x.clone(), w.clone(), dy.clone()
    xn[77, K - 1] = float("nan")
    xn[12, 3] = float("inf")
    wn[0, 100, 0] = float("nan")
    out = cdl.grouped_bf16(xn, wn, c, seg)
    bad = torch.zeros(n, N, dtype=torch.bool, device=DEV)
    bad[[12, 77]] = True
    bad[:, 100] = True
    assert torch.equal(out[~bad], base[~bad]) and bool(torch.isnan(out[77]).all()) and bool(torch.isnan(out[:, 100]).all())
    keep = torch.arange(N, device=DEV) != 100
    assert bool(torch.isinf(out[12][keep]).all()) and torch.equal(torch.signbit(out[12][keep]), torch.signbit(w[0, keep, 3]))
    dyn[140, N - 1] = float("nan")
    dx, dx0 = cdl.grouped_bf16_dx(dyn, w, c, seg), cdl.grouped_bf16_dx(dy, w, c, seg)
    assert bool(torch.isnan(dx[140]).all()) and torch.equal(dx[:140], dx0[:140]) and torch.equal(dx[141:], dx0[141:])
    dw, dw0 = cdl.grouped_bf16_dw(dyn, x, c, seg), cdl.grouped_bf16_dw(dy, x, c, seg)
    assert bool(torch.isnan(dw[0, N - 1]).all()) and torch.equal(dw[0, :N - 1], dw0[0, :N - 1])


def test_large_gates():
    """exp overflows at gates below -88: the product is then zero, not NaN; large positive gates pass."""
    announce("swiglu at large gates")
    K, I = 8, 16
    x = torch.zeros(4, K, dtype=BF, device=DEV)
    x[:, 0] = torch.tensor([1.0, -1.0, 1e4, -1e4])
    w = torch.zeros(1, 2 * I, K, dtype=BF, device=DEV)
    w[0, :I, 0], w[0, I:, 0] = 200.0, 0.5
    c, seg = torch.tensor([4], dtype=torch.int32, device=DEV), torch.tensor([0, 4], dtype=torch.int64, device=DEV)
    out = cdl.grouped_swiglu_bf16(x, w, c, seg)
    want = torch.tensor([100.0, 0.0, 1e10, 0.0], dtype=torch.float64, device=DEV)
    R.assert_within(out, want[:, None].expand(4, I), want[:, None] * 2 * R.BF16 + 1e-30)
    d = cdl.grouped_swiglu_bf16_grad(x, w, torch.ones(4, I, dtype=BF, device=DEV), c, seg)
    assert bool(torch.isfinite(d).all())
    R.assert_within(d[0], torch.tensor([0.5] * I + [200.0] * I, dtype=torch.float64, device=DEV),
                    torch.full((2 * I,), 200 * 2 * R.BF16, dtype=torch.float64, device=DEV))
    assert bool((d[1] == 0).all()) and bool((d[3] == 0).all())


@pytest.mark.parametrize("flags", [0, 1, 7])
def test_fp8_nonfinite_and_zero_rows(flags):
    announce("fp8 product of non-finite and zero rows, flags=%d" % flags)
    g, K, N, n = gen(6), 256, 256, 20
    x = rand(g, n, K)
    x[3] = 0
    x[5, 7] = float("nan")
    x[6, 200] = float("inf")
    ids = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    q, s = cdl.dispatch_fp8(x, cdl.dispatch_layout(ids, 0, 1), rows=n, scale_flags=flags)
    wq, ws = fp8_weights(g, 1, N, K)
    c, seg = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int64, device=DEV)
    y = cdl.grouped_fp8(q, s, wq, ws, c, seg, scale_flags=flags)
    h, hs = cdl.grouped_swiglu_fp8(q, s, wq, ws, c, seg, scale_flags=flags)
    fine = torch.ones(n, dtype=torch.bool, device=DEV)
    fine[[5, 6]] = False
    assert bool((y[3] == 0).all()) and bool(torch.isfinite(y[fine]).all())
    assert bool(torch.isnan(y[5]).all()) and not bool(torch.isfinite(y[6]).any())
    assert bool((h[3] & 127 == 0).all()) and bool((h[5] & 127 == 127).all())
    x2 = x[fine]
    q2, s2 = cdl.dispatch_fp8(x2, cdl.dispatch_layout(ids[:len(x2)], 0, 1), rows=len(x2), scale_flags=flags)
    c2, seg2 = torch.tensor([len(x2)], dtype=torch.int32, device=DEV), torch.tensor([0, len(x2)], dtype=torch.int64, device=DEV)
    assert torch.equal(y[fine], cdl.grouped_fp8(q2, s2, wq, ws, c2, seg2, scale_flags=flags))
    assert torch.equal(h[fine], cdl.grouped_swiglu_fp8(q2, s2, wq, ws, c2, seg2, scale_flags=flags)[0])


# ---------------------------------------------------------------------------
# streams, graphs, overlap, repeated calls
# ---------------------------------------------------------------------------

def all_forms(seed, counts=(300, 0, 65, 1)):
    """Every product as a call on fixed inputs."""
    r, g = Rows(list(counts), False), gen(seed)
    L, K, N = len(counts), 384, 512
    x, w, dy, dh = rand(g, r.n, K), rand(g, L, N, K, scale=K ** -0.5), rand(g, r.n, N), rand(g, r.n, N // 2)
    q, s, _ = fp8_rows(g, r, K, 7)
    wq, ws = fp8_weights(g, L, N, K)
    z = lambda *shape: torch.zeros(*shape, dtype=BF, device=DEV)      # noqa: E731
    bufs = [z(r.n, N), z(r.n, N // 2), z(r.n, N), z(r.n, K), z(L, N, K), z(r.n, N),
            torch.zeros(r.n, N // 2, dtype=torch.uint8, device=DEV), cdl.new_scale_tensor(r.n, N // 2, 7, DEV).zero_()]
    at = (r.c, r.seg)

    def run():
        cdl.grouped_bf16(x, w, *at, out=bufs[0])
        cdl.grouped_swiglu_bf16(x, w, *at, out=bufs[1])
        cdl.grouped_swiglu_bf16_grad(x, w, dh, *at, out=bufs[2])
        cdl.grouped_bf16_dx(dy, w, *at, out=bufs[3])
        cdl.grouped_bf16_dw(dy, x, *at, out=bufs[4])
        cdl.grouped_fp8(q, s, wq, ws, *at, scale_flags=7, out=bufs[5])
        cdl.grouped_swiglu_fp8(q, s, wq, ws, *at, scale_flags=7, out_q=bufs[6], out_scales=bufs[7])

    return run, bufs, (x, dy, dh, q)


def snapshot(bufs):
    return [b.clone() for b in bufs]


def test_products_are_deterministic_and_captured_graphs_replay():
    announce("products: repeated, on another stream, captured and replayed")
    run, bufs, inputs = all_forms(1)
    run()
    want = snapshot(bufs)
    for b in bufs:
        b.zero_()
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
        # other inputs in the same buffers
        for t in inputs:
            t.copy_(t.flip(0))
        graph.replay()
        got = snapshot(bufs)
        run()
        assert all(torch.equal(a, b) for a, b in zip(bufs, got)), i
        for t in inputs:
            t.copy_(t.flip(0))


def test_products_on_two_streams_at_once():
    announce("products on two streams at once")
    (run1, b1, _), (run2, b2, _) = all_forms(1), all_forms(2, (130, 700, 2))
    run1()
    run2()
    want1, want2 = snapshot(b1), snapshot(b2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s1):
            run1()
        with torch.cuda.stream(s2):
            run2()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(b1, want1)) and all(torch.equal(a, b) for a, b in zip(b2, want2))


def test_a_row_does_not_depend_on_its_batch():
    """The same rows among others, in another expert position and in either buffer kind give the same bits."""
    announce("products: a row's bits in any batch")
    g, K, N = gen(8), 384, 264
    w, x = rand(g, 1, N, K), rand(g, 900, K)
    one = lambda n: (torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int64, device=DEV))  # noqa: E731
    full = cdl.grouped_bf16(x, w, *one(900))
    for n in (1, 15, 64, 65, 130, 200, 300, 513):
        assert torch.equal(cdl.grouped_bf16(x[:n].contiguous(), w, *one(n)), full[:n]), n
        assert torch.equal(cdl.grouped_bf16(x[None, :n].contiguous(), w, one(n)[0])[0], full[:n]), n


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------

def test_fp8_layer_from_the_norm_to_the_combine():
    """Norm, dispatch in 8 bits, gate/up with SwiGLU, down, combine, and a shared expert on the norm's own 8-bit
    rows, against the chain of 64-bit forms of every step on the same 8-bit intermediates."""
    announce("fp8 layer")
    g, T, H, I, E, k = gen(10), 300, 512, 384, 8, 3
    x, res, nw = rand(g, T, H), rand(g, T, H), rand(g, H, scale=0.1) + 1
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    wts = torch.softmax(torch.randn(T, k, generator=g, device=DEV), -1)
    w13, w2 = fp8_weights(g, E, 2 * I, H), fp8_weights(g, E, H, I)
    s13, s2 = fp8_weights(g, 1, 2 * I, H), fp8_weights(g, 1, H, I)
    y = torch.empty(T, H, dtype=BF, device=DEV)
    nq, ns, h = cdl.rms_norm_fp8(x, nw, res, out=y)
    lay, q, s = cdl.permute_fp8(y, ids, 0, E, alignment=16)
    hq, hs = cdl.grouped_swiglu_fp8(q, s, *w13, lay.counts, lay.seg_indptr)
    o = cdl.grouped_fp8(hq, hs, *w2, lay.counts, lay.seg_indptr)
    routed = cdl.combine(o, lay.src2dst, wts)
    one = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int64, device=DEV)
    sq, ss = cdl.grouped_swiglu_fp8(nq, ns, *s13, *one)
    shared = cdl.grouped_fp8(sq, ss, *s2, *one)
    # every step on what the one before gave
    want_h = (x.float() + res.float()).to(BF)
    assert torch.equal(h, want_h)
    ref, err = R.norm(h.double(), nw.double(), 1e-6)
    R.assert_within(y, ref, R.to_bf16_bound(ref, err))
    check_fp8_values(ref, err, nq, ns.double(), 0)
    seg, counts = lay.seg_indptr.tolist(), lay.counts.tolist()
    rows = torch.zeros(q.shape[0], H, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(rows)
    for e in range(E):
        at = slice(seg[e], seg[e] + counts[e])
        gu, d = R.fp8_product(q[at], s[at].double(), w13[0][e], w13[1][e])
        v, dv = R.swiglu(gu[:, :I], d[:, :I], gu[:, I:], d[:, I:])
        check_fp8_values(v, dv, hq[at], hs[at].double(), 0)
        rows[at], err = R.fp8_product(hq[at], hs[at].double(), w2[0][e], w2[1][e])
        bound[at] = R.to_bf16_bound(rows[at], err)
    dst = lay.src2dst.long()
    want = (rows[dst].view(T, k, H) * wts.double().unsqueeze(-1)).sum(1)
    far = ((bound[dst] + R.U32 * rows[dst].abs()).view(T, k, H) * wts.double().unsqueeze(-1)).sum(1)
    R.assert_within(routed, want, R.to_bf16_bound(want, far * (1 + k * R.U32)))
    v, err = R.fp8_product(sq, ss.double(), s2[0][0], s2[1][0])
    R.assert_within(shared, v, R.to_bf16_bound(v, err))


def test_training_pass_of_the_experts():
    """Forward and backward of the local experts, each gradient against the formula's and against differences of
    the forward pass in 64 bits."""
    announce("bf16 training pass")
    g, T, H, I, E, k = gen(11), 120, 64, 72, 4, 2
    x = rand(g, T, H)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    w13, w2 = rand(g, E, 2 * I, H, scale=H ** -0.5), rand(g, E, H, I, scale=I ** -0.5)
    lay, rows = cdl.permute(x, ids, 0, E)
    at = (lay.counts, lay.seg_indptr)
    h = cdl.grouped_swiglu_bf16(rows, w13, *at)
    y = cdl.grouped_bf16(h, w2, *at)
    dy = rand(g, *y.shape)
    dh = cdl.grouped_bf16_dx(dy, w2, *at)
    dw2 = cdl.grouped_bf16_dw(dy, h, *at)
    dgu = cdl.grouped_swiglu_bf16_grad(rows, w13, dh, *at)
    drows = cdl.grouped_bf16_dx(dgu, w13, *at)
    dw13 = cdl.grouped_bf16_dw(dgu, rows, *at)
    dx = cdl.combine(drows, lay.src2dst, torch.ones(T, k, device=DEV))

    seg = lay.seg_indptr.tolist()

    def loss(a13, a2, a):
        total = 0
        for e in range(E):
            s = slice(seg[e], seg[e + 1])
            gu = a[s] @ a13[e].t()
            total = total + ((gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]) @ a2[e].t() * dy[s].double()).sum()
        return total

    a13, a2, a = (t.double().requires_grad_() for t in (w13, w2, rows))
    loss(a13, a2, a).backward()
    # bf16 intermediates (h, dh, dgu) move a gradient by their roundings: at most two in a row, and its own
    for got, want in ((dw13, a13.grad), (dw2, a2.grad), (drows, a.grad)):
        off = float((got.double() - want).norm() / want.norm())
        assert off < 3 * R.BF16, off
    dst = lay.src2dst.view(T, k).long()
    want = a.grad[dst].sum(1)
    assert float((dx.double() - want).norm() / want.norm()) < 4 * R.BF16
    # differences along a direction: the loss is smooth, a central difference is off by about step^2
    for got, base, which in ((dw13, w13, 0), (dw2, w2, 1), (drows, rows, 2)):
        d = torch.randn(base.shape, generator=g, device=DEV, dtype=torch.float64)
        args = [w13.double(), w2.double(), rows.double()]
        step = 1e-4
        lo, hi = list(args), list(args)
        lo[which], hi[which] = args[which] - step * d, args[which] + step * d
        slope = float((loss(*hi) - loss(*lo)) / (2 * step))
        along = float((got.double() * d).sum())
        assert abs(along - slope) < 3 * R.BF16 * float(got.double().norm() * d.norm()) ** 1.0, (which, along, slope)


@pytest.mark.parametrize("flags,packed", [(0, False), (7, True)])
def test_fp8_padded_buffers_of_many_experts(flags, packed):
    """2000 experts, whose tile table leaves no room for the smaller tiles' third stage."""
    announce("padded fp8 products of 2000 experts, flags %d" % flags)
    L, K, N, g = 2000, 256, 256, gen(flags)
    counts = [(5 * e) % 4 for e in range(L)]
    r = Rows(counts, True)
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, L, N, K)
    y = cdl.grouped_fp8(r.shape(q), s, wq, ws, r.c, scale_flags=flags).view(r.n, N)
    hq, hs = cdl.grouped_swiglu_fp8(r.shape(q), s, wq, ws, r.c, scale_flags=flags)
    hq, hp = hq.view(r.n, N // 2), R.scales(hs, flags, r.n, 1, r.cap)
    for e, at in list(r.each())[:20] + list(r.each())[-20:]:
        v, err = R.fp8_product(q[at], p[at], wq[e], ws[e])
        R.assert_within(y[at], v, R.to_bf16_bound(v, err), e)
        h, dh = R.swiglu(v[:, :N // 2], err[:, :N // 2], v[:, N // 2:], err[:, N // 2:])
        check_fp8_values(h, dh, hq[at], hp[at], bool(flags & 1))


def test_outputs_over_operands_are_refused():
    announce("overlapping outputs")
    g, T, K = gen(3), 12, 128
    x, w = rand(g, T, K), rand(g, 1, K, K)
    c, seg = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], device=DEV)
    q = torch.zeros(T, K, dtype=torch.uint8, device=DEV)
    s = torch.ones(T, 1, device=DEV)
    wq, ws = cdl.quant_fp8_blocks(rand(g, 1, 2 * K, K))
    both = torch.zeros(T + 1, K, dtype=BF, device=DEV)
    rows = torch.zeros(T, K, dtype=BF, device=DEV)
    ws32 = torch.zeros(cdl.rms_norm_grad_workspace_size(T, K) // 4, device=DEV)
    for call in (lambda: cdl.grouped_bf16(x, w, c, seg, out=x),
                 lambda: cdl.grouped_bf16(both[:T], w, c, seg, out=both[1:]),
                 lambda: cdl.grouped_swiglu_bf16(x, rand(g, 1, 2 * K, K), c, seg, out=x),
                 lambda: cdl.grouped_swiglu_bf16_grad(x, w, rows[:, :K // 2].contiguous(), c, seg, out=x),
                 lambda: cdl.grouped_bf16_dx(x, w, c, seg, out=x),
                 lambda: cdl.grouped_bf16_dw(big := rand(g, K, K), big, torch.tensor([K], dtype=torch.int32, device=DEV),
                                             torch.tensor([0, K], device=DEV), out=big.view(1, K, K)),
                 lambda: cdl.grouped_fp8(both[:T // 2].view(torch.uint8).view(T, K), s, wq, ws, c, seg,
                                         out=both[:T]),
                 lambda: cdl.grouped_swiglu_fp8(q, s, wq, ws, c, seg, out_q=q),
                 lambda: cdl.grouped_swiglu_fp8(q, s, wq, ws, c, seg, out_scales=s),
                 lambda: cdl.rms_norm(x, w[0, 0], rows, out=both[:T], residual_out=both[:T]),
                 lambda: cdl.rms_norm(both[:T], w[0, 0], out=both[1:]),
                 lambda: cdl.rms_norm_fp8(x, w[0, 0], out_q=x.view(torch.uint8).view(2 * T, K)[:T]),
                 lambda: cdl.rms_norm_grad(both[:T], x, w[0, 0], out=both[1:]),
                 lambda: cdl.rms_norm_grad(rows, x, w[0, 0], dweight=ws32[:K], workspace=ws32),
                 lambda: cdl.dequant_fp8(both[:T // 2].view(torch.uint8).view(T, K), s, out=both[:T])):
        with pytest.raises(ValueError, match="overlaps"):
            call()
