"""GPU tests of the MXFP4 rows, the grouped MXFP4 product and the MoE layer of
a few tokens against their plain 64-bit forms.

Quantised rows and read-back values are compared bit for bit.  Products are
held to a bound computed with them: fp32 accumulation (one step per product
and sum, relative to the sum of magnitudes) and half a bf16 step for each
rounding to bf16 (experts_ref.py).
"""
import numpy as np
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import experts_ref as R
import oracle
from combine_dispatch_layout_amd import workloads as W
from gpu_util import DEV, announce, npy, status_word

pytestmark = pytest.mark.gpu

CANARY = 0xA5


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def mx_random(g, *shape, lo=120, hi=130):
    """Random MXFP4 rows [..., H]: any code, scales 2^(lo-127) to 2^(hi-127)."""
    q = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(lo, hi + 1, (*shape[:-1], shape[-1] // 32), generator=g, device=DEV, dtype=torch.int32)
    return q, s.to(torch.uint8)


def bits_of(x):
    return x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def assert_mx(q, s, bits):
    codes, scales = R.quantise(bits)
    assert np.array_equal(npy(s), scales)
    assert np.array_equal(npy(R.unpack(q)), codes)


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------

def test_quant_every_bf16_pattern():
    """Every bf16 pattern in groups whose largest magnitude it is (alone, with
    smaller neighbours), and every exponent's border to the next scale."""
    announce("quantise all bf16 patterns")
    p = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    alone = np.zeros((65536, 32), np.uint16)
    alone[:, 5] = p
    rng = np.random.default_rng(3)
    mixed = rng.integers(0, 65536, (65536, 32)).astype(np.uint16)
    # neighbours a few binary steps below the pattern, so that every code occurs
    drop = rng.integers(0, 4 * 128, (65536, 32))
    near = np.maximum((p[:, None] & 0x7FFF).astype(np.int64) - drop, 0).astype(np.uint16)
    near |= (rng.integers(0, 2, near.shape) << 15).astype(np.uint16)
    for bits in (alone, mixed, near):
        q, s = cdl.quant_mxfp4(W.bits_to_bf16(bits).to(DEV))
        assert_mx(q, s, bits)


@pytest.mark.parametrize("rows,H", [(1, 32), (3, 64), (5, 1024), (2, 1056), (7, 7168), (4, 7200), (2, 14336 + 32),
                                    (1000, 96), (1, 50000 * 32)])
def test_quant_dequant_sizes(rows, H):
    announce("quantise rows=%d H=%d" % (rows, H))
    x = randn(gen(rows * 7 + H), rows, H, scale=3.0)
    x[0, :32] = 0
    q = torch.full((rows + 1, H // 2), CANARY, dtype=torch.uint8, device=DEV)
    s = torch.full((rows + 1, H // 32), CANARY, dtype=torch.uint8, device=DEV)
    cdl.quant_mxfp4(x, out_q=q[:rows], out_scales=s[:rows])
    assert_mx(q[:rows], s[:rows], bits_of(x))
    assert bool((q[rows:] == CANARY).all()) and bool((s[rows:] == CANARY).all())
    out = cdl.dequant_mxfp4(q[:rows], s[:rows])
    assert torch.equal(out.double(), R.values(q[:rows], s[:rows]))


def test_dequant_every_code_and_scale():
    q = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)[:, :, None].expand(256, 256, 16).contiguous()
    s = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None, None].expand(256, 256, 1).contiguous()
    out = cdl.dequant_mxfp4(q, s).double()
    want = R.values(q, s)
    want = torch.where(want.abs() >= 2.0 ** 128, torch.sign(want) * torch.inf, want)
    assert bool((torch.isnan(out) == torch.isnan(want)).all())
    assert torch.equal(torch.nan_to_num(out, nan=0.0, posinf=1e300, neginf=-1e300),
                       torch.nan_to_num(want, nan=0.0, posinf=1e300, neginf=-1e300))


SCATTER = [  # T, H, E, L, k, begin, alignment, dist
    (64, 256, 8, 8, 2, 0, 1, "uniform"), (1, 32, 4, 4, 1, 0, 1, "uniform"), (3, 96, 16, 4, 3, 5, 16, "uniform"),
    (700, 2592, 32, 8, 8, 8, 1, "zipf"), (513, 7168, 64, 16, 6, 0, 128, "uniform"), (33, 7200, 8, 8, 4, 0, 1, "zipf"),
    (5000, 64, 128, 128, 8, 0, 1, "zipf"), (40, 128, 64, 2, 64, 3, 1, "uniform"),
    (512, 64, 16, 16, 8, 0, 1, "uniform"), (513, 96, 16, 5, 7, 2, 32, "uniform"), (2048, 64, 4, 4, 2, 0, 1, "uniform"),
    (4097, 32, 4, 3, 1, 0, 1, "zipf"), (64, 64, 2048, 2048, 64, 0, 1, "uniform"), (65, 64, 2048, 2048, 64, 0, 4, "uniform"),
    # both sides of the borders where the layout leaves the rows' launch
    (4095, 64, 32, 8, 2, 1, 16, "zipf"), (4096, 64, 32, 8, 2, 1, 16, "zipf"), (4096, 4096, 16, 4, 2, 3, 1, "uniform"),
    (4096, 4128, 16, 4, 2, 3, 1, "uniform"), (5120, 4128, 16, 4, 2, 0, 8, "zipf"), (5121, 4128, 16, 4, 2, 0, 8, "zipf"),
    (16385, 32, 256, 256, 8, 0, 128, "zipf"),
]


def scatter_inputs(T, H, E, L, k, b, dist):
    w = W.Workload("t", T=T, H=H, E=E, L=L, k=k, dist=dist, expert_begin=b, seed_base=T + H + k)
    return W.make_inputs(w)


@pytest.mark.parametrize("T,H,E,L,k,b,A,dist", SCATTER)
def test_permute_and_dispatch(T, H, E, L, k, b, A, dist):
    announce("mxfp4 permute T=%d H=%d L=%d k=%d A=%d" % (T, H, L, k, A))
    x, ids, _ = scatter_inputs(T, H, E, L, k, b, dist)
    codes, scales = R.quantise(W.bf16_bits(x))
    xd, idd = x.to(DEV), ids.to(DEV)
    want = cdl.dispatch_layout(idd, b, L, alignment=A)
    n = want.num_rows() + 2
    q = torch.full((n, H // 2), CANARY, dtype=torch.uint8, device=DEV)
    s = torch.full((n, H // 32), CANARY, dtype=torch.uint8, device=DEV)
    st = status_word()
    lay, _, _ = cdl.permute_mxfp4(xd, idd, b, L, out_q=q, out_scales=s, status=st, alignment=A)
    for f in ("counts", "seg_indptr", "src2dst"):
        assert torch.equal(getattr(lay, f), getattr(want, f)), f
    assert torch.equal(lay.reorder_topk_ids, want.reorder_topk_ids)
    assert int(st.item()) == 0
    wq = np.full((n, H // 2), CANARY, np.uint8)
    ws = np.full((n, H // 32), CANARY, np.uint8)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    dst = npy(want.src2dst)
    for i in np.nonzero(dst >= 0)[0]:
        wq[dst[i]], ws[dst[i]] = packed[i // k], scales[i // k]
    assert np.array_equal(npy(q), wq) and np.array_equal(npy(s), ws)
    q2, s2 = torch.full_like(q, CANARY), torch.full_like(s, CANARY)
    cdl.dispatch_mxfp4(xd, want, out_q=q2, out_scales=s2)
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_scatter_into_too_few_rows():
    x, ids, _ = scatter_inputs(200, 256, 8, 8, 2, 0, "uniform")
    lay = cdl.dispatch_layout(ids.to(DEV), 0, 8)
    full, fs = cdl.dispatch_mxfp4(x.to(DEV), lay)
    st = status_word()
    q = torch.full((100, 128), CANARY, dtype=torch.uint8, device=DEV)
    s = torch.full((100, 8), CANARY, dtype=torch.uint8, device=DEV)
    cdl.permute_mxfp4(x.to(DEV), ids.to(DEV), 0, 8, out_q=q[:90], out_scales=s[:90], status=st)
    assert int(st.item()) == cdl.CDL_STATUS_ROWS_OVERFLOW
    assert torch.equal(q[:90], full[:90]) and torch.equal(s[:90], fs[:90])
    assert bool((q[90:] == CANARY).all()) and bool((s[90:] == CANARY).all())


def test_long_permute_into_too_few_rows():
    x, ids, _ = scatter_inputs(4500, 64, 16, 4, 4, 2, "uniform")
    lay = cdl.dispatch_layout(ids.to(DEV), 2, 4)
    full, fs = cdl.dispatch_mxfp4(x.to(DEV), lay)
    n = full.shape[0] - 37
    st = status_word()
    q = torch.full((n + 5, 32), CANARY, dtype=torch.uint8, device=DEV)
    s = torch.full((n + 5, 2), CANARY, dtype=torch.uint8, device=DEV)
    cdl.permute_mxfp4(x.to(DEV), ids.to(DEV), 2, 4, out_q=q[:n], out_scales=s[:n], status=st)
    assert int(st.item()) == cdl.CDL_STATUS_ROWS_OVERFLOW
    assert torch.equal(q[:n], full[:n]) and torch.equal(s[:n], fs[:n])
    assert bool((q[n:] == CANARY).all()) and bool((s[n:] == CANARY).all())


@pytest.mark.parametrize("T,H,E,L,k,b,cap", [(128, 7168, 256, 32, 8, 0, 128), (64, 256, 8, 8, 2, 0, 9),
                                             (600, 96, 16, 4, 3, 5, 700), (30, 64, 4, 4, 2, 0, 0),
                                             (1500, 64, 16, 4, 3, 5, 1200), (1024, 7200, 8, 8, 4, 0, 300)])
def test_permute_ll(T, H, E, L, k, b, cap):
    announce("mxfp4 low-latency T=%d H=%d L=%d cap=%d" % (T, H, L, cap))
    x, ids, _ = scatter_inputs(T, H, E, L, k, b, "uniform")
    codes, scales = R.quantise(W.bf16_bits(x))
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    st, st0 = status_word(), status_word()
    _, _, mm0, map0 = cdl.permute_ll(x.to(DEV), ids.to(DEV), b, L, cap, status=st0)
    q = torch.full((L, cap, H // 2), CANARY, dtype=torch.uint8, device=DEV)
    s = torch.full((L, cap, H // 32), CANARY, dtype=torch.uint8, device=DEV)
    _, _, _, mm, ll = cdl.permute_ll_mxfp4(x.to(DEV), ids.to(DEV), b, L, cap, out_q=q, out_scales=s, status=st)
    assert torch.equal(mm, mm0) and torch.equal(ll, map0) and torch.equal(st, st0)
    wq, ws = np.full((L * cap, H // 2), CANARY, np.uint8), np.full((L * cap, H // 32), CANARY, np.uint8)
    for i, d in enumerate(npy(ll)):
        if d >= 0:
            wq[d], ws[d] = packed[i // k], scales[i // k]
    assert np.array_equal(npy(q).reshape(wq.shape), wq) and np.array_equal(npy(s).reshape(ws.shape), ws)


def test_empty_batch_rows():
    x, ids = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    lay, q, s = cdl.permute_mxfp4(x, ids, 0, 4)
    assert npy(lay.counts).tolist() == [0] * 4 and npy(lay.seg_indptr).tolist() == [0] * 5
    _, q, s, mm, ll = cdl.permute_ll_mxfp4(x, ids, 0, 4, 3)
    assert npy(mm).tolist() == [0] * 4 and ll.numel() == 0
    assert cdl.quant_mxfp4(x)[0].shape == (0, 32)


# ---------------------------------------------------------------------------
# grouped product
# ---------------------------------------------------------------------------

def segments(counts, align=1, gap=0):
    """seg_indptr with every segment padded to `align` and `gap` rows between."""
    seg = [0]
    for c in counts:
        seg.append(seg[-1] + (c + align - 1) // align * align + gap)
    return seg


def check_grouped(a, sa, w, sw, counts, begins, out, canary_rows):
    """out (2-D rows) against the 64-bit product of every expert's rows; all
    other rows hold the canary."""
    live = torch.zeros(out.shape[0], dtype=torch.bool, device=DEV)
    for e, c in enumerate(counts):
        at = slice(begins[e], begins[e] + c)
        live[at] = True
        if c:
            y, err = R.product(R.values(a[at], sa[at]), R.values(w[e], sw[e]))
            bad = (out[at].double() - y).abs() > err + R.BF16 * (y.abs() + err) + R.TINY
            assert not bool(bad.any()), (e, int(bad.sum()))
    rest = out[~live]
    assert torch.equal(rest.view(torch.int16), canary_rows.expand_as(rest).view(torch.int16))


COUNTS = [
    ([1], 32, 1), ([5], 64, 3), ([33, 0, 31], 96, 40), ([0, 0, 0], 64, 32), ([64, 1, 0, 130], 256, 256),
    ([128] * 4, 512, 512), ([7, 200, 65, 0, 1, 300], 1440, 500), ([100, 28], 7168, 136), ([1] * 70, 160, 33),
    ([257, 255, 256], 2048, 264), ([3, 0, 9, 16, 2], 7168, 1032), ([600], 288, 1000), ([17] * 33, 544, 72),
    ([48, 96], 15 * 32, 2000),
    # more than 256 tiles of 64 rows, 64 rows an expert or more: the large tile
    ([64, 1, 0, 330], 96, 8200), ([257, 255, 256], 2048, 5000), ([7, 200, 65, 0, 1, 300], 1440, 7000),
    ([600], 288, 7400), ([100, 428], 7168, 8000), ([4136, 17], 64, 1000),
]


@pytest.mark.parametrize("counts,K,N", COUNTS)
@pytest.mark.parametrize("form", ["segments", "padded segments", "masked"])
def test_grouped(counts, K, N, form):
    announce("grouped %s counts=%s K=%d N=%d" % (form, counts[:6], K, N))
    g = gen(K + N + len(counts))
    L = len(counts)
    w, sw = mx_random(g, L, N, K)
    st = status_word()
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    canary = torch.full((1,), -7.5, dtype=torch.bfloat16, device=DEV)
    if form == "masked":
        cap = max(counts) + 3
        a, sa = mx_random(g, L, cap, K)
        out = canary.expand(L, cap, N).contiguous()
        cdl.grouped_mxfp4(a, sa, w, sw, c, out=out, status=st)
        begins = [e * cap for e in range(L)]
        a, sa, out = a.view(L * cap, -1), sa.view(L * cap, -1), out.view(L * cap, N)
    else:
        seg = segments(counts) if form == "segments" else segments(counts, 16, 5)
        a, sa = mx_random(g, seg[-1] + 4, K)
        out = canary.expand(seg[-1] + 4, N).contiguous()
        cdl.grouped_mxfp4(a, sa, w, sw, c, torch.tensor(seg, device=DEV), out=out, status=st)
        begins = seg
    assert int(st.item()) == 0
    check_grouped(a, sa, w, sw, counts, begins, out, canary)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("counts,K,N", [([70, 3], 1056, 260), ([300, 212], 736, 40), ([20, 90, 1], 2048, 513),
                                        ([300, 212], 736, 8256), ([300, 213], 1056, 8191)])
def test_grouped_scales_at_any_byte(counts, K, N, shift):
    """Scale tensors that start at any byte, rows of an odd number of scales,
    output rows at 2-byte alignment; the scales' neighbours are NaN codes."""
    announce("grouped, scales at byte %d, counts=%s K=%d N=%d" % (shift, counts, K, N))
    g = gen(shift + K)
    L, rows = len(counts), sum(counts)

    def moved(s):
        flat = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device=DEV)
        flat[shift:shift + s.numel()] = s.flatten()
        return flat[shift:shift + s.numel()].view(s.shape)

    w, sw = mx_random(g, L, N, K)
    a, sa = mx_random(g, rows, K)
    canary = torch.full((1,), -7.5, dtype=torch.bfloat16, device=DEV)
    whole = canary.expand(rows * N + 16).contiguous()
    out = whole[shift:shift + rows * N].view(rows, N)
    seg = segments(counts)
    cdl.grouped_mxfp4(a, moved(sa), w, moved(sw), torch.tensor(counts, dtype=torch.int32, device=DEV),
                      torch.tensor(seg, device=DEV), out=out)
    check_grouped(a, sa, w, sw, counts, seg, out, canary)
    assert bool((whole[:shift] == -7.5).all()) and bool((whole[shift + rows * N:] == -7.5).all())
    if N % 64 == 0 or N == 260:
        I = N // 64 * 32
        w2, sw2 = w[:, :2 * I].contiguous(), sw[:, :2 * I].contiguous()
        q, s = cdl.grouped_swiglu_mxfp4(a, moved(sa), w2, moved(sw2),
                                        torch.tensor(counts, dtype=torch.int32, device=DEV),
                                        torch.tensor(seg, device=DEV))
        for e, n in enumerate(counts):
            at = slice(seg[e], seg[e] + n)
            check_swiglu(a[at], sa[at], w2[e], sw2[e], q[at], s[at], I)


@pytest.mark.parametrize("L,cap,n", [(128, 40, 7), (300, 3, 2), (2048, 2, 1)])
def test_grouped_many_experts(L, cap, n):
    """More experts than one scan of a wave takes; every third is empty."""
    g = gen(L)
    w, sw = mx_random(g, L, 24, 64)
    a, sa = mx_random(g, L, cap, 64)
    counts = [0 if e % 3 == 1 else n for e in range(L)]
    canary = torch.full((1,), -7.5, dtype=torch.bfloat16, device=DEV)
    out = canary.expand(L, cap, 24).contiguous()
    cdl.grouped_mxfp4(a, sa, w, sw, torch.tensor(counts, dtype=torch.int32, device=DEV), out=out)
    check_grouped(a.view(L * cap, -1), sa.view(L * cap, -1), w, sw, counts, [e * cap for e in range(L)],
                  out.view(L * cap, 24), canary)


def test_grouped_same_result_for_every_form_and_call():
    """A row's result does not depend on the form or on the call."""
    g = gen(11)
    counts = [40, 0, 3, 150]
    L, K, N, cap = 4, 1056, 200, 160
    w, sw = mx_random(g, L, N, K)
    a, sa = mx_random(g, L, cap, K)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    ref = cdl.grouped_mxfp4(a, sa, w, sw, c)
    for _ in range(3):
        again = cdl.grouped_mxfp4(a, sa, w, sw, c)
        for e, n in enumerate(counts):
            assert torch.equal(again[e, :n], ref[e, :n])


def test_grouped_counts_beyond_the_buffer_are_cut():
    """Counts and offsets that do not fit the buffer are cut to what does and
    flagged; nothing outside is written."""
    g = gen(5)
    w, sw = mx_random(g, 2, 40, 64)
    a, sa = mx_random(g, 20, 64)
    whole = torch.full((24, 40), 3.0, dtype=torch.bfloat16, device=DEV)
    canary = torch.full((1,), 3.0, dtype=torch.bfloat16, device=DEV)
    for counts, seg, eff in (([8, 50], [0, 8, 58], [8, 12]), ([-4, 5], [0, 3, 8], [0, 5]),
                             ([4, 3], [-9, 30, 33], [0, 0]), ([2 ** 31 - 1, 0], [0, 20, 20], [20, 0])):
        whole.fill_(3.0)
        st = status_word()
        cdl.grouped_mxfp4(a, sa, w, sw, torch.tensor(counts, dtype=torch.int32, device=DEV),
                          torch.tensor(seg, device=DEV), out=whole[:20], status=st)
        assert int(st.item()) == cdl.CDL_STATUS_ROWS_OVERFLOW
        check_grouped(a, sa, w, sw, eff, [max(0, min(s, 20)) for s in seg], whole[:20], canary)
        assert bool((whole[20:] == 3.0).all())
    am, sm = a.view(2, 10, -1), sa.view(2, 10, -1)
    st = status_word()
    whole.fill_(3.0)
    cdl.grouped_mxfp4(am, sm, w, sw, torch.tensor([11, 4], dtype=torch.int32, device=DEV),
                      out=whole[:20].view(2, 10, 40), status=st)
    assert int(st.item()) == cdl.CDL_STATUS_LL_OVERFLOW
    check_grouped(a, sa, w, sw, [10, 4], [0, 10], whole[:20], canary)


def test_grouped_extreme_scales_and_nan():
    """NaN scales reach their own row or column only; scales at both ends of
    the range give the exact products (single terms), infinity on overflow."""
    g = gen(8)
    a, sa = mx_random(g, 40, 96)
    w, sw = mx_random(g, 1, 50, 96)
    sa[3, 1] = 255
    sw[0, 7, 0] = 255
    c, seg = torch.tensor([40], dtype=torch.int32, device=DEV), torch.tensor([0, 40], device=DEV)
    out = cdl.grouped_mxfp4(a, sa, w, sw, c, seg)
    nan = torch.zeros(40, 50, dtype=torch.bool, device=DEV)
    nan[3] = True
    nan[:, 7] = True
    assert torch.equal(torch.isnan(out), nan)
    for ea, ew in ((1, 127), (127, 1), (10, 120), (253, 2), (60, 194), (250, 250)):
        a = torch.zeros(1, 16, dtype=torch.uint8, device=DEV)
        a[0, 0] = 0x02                                   # 1.0 in element 0
        w = torch.zeros(1, 1, 16, dtype=torch.uint8, device=DEV)
        w[0, 0, 0] = 0x05                                # 3.0
        sa = torch.full((1, 1), ea, dtype=torch.uint8, device=DEV)
        sw = torch.full((1, 1, 1), ew, dtype=torch.uint8, device=DEV)
        out = cdl.grouped_mxfp4(a, sa, w, sw, torch.ones(1, dtype=torch.int32, device=DEV),
                                torch.tensor([0, 1], device=DEV))
        want = 3.0 * 2.0 ** (ea + ew - 254)
        assert float(out.item()) == (want if want < 2.0 ** 128 else float("inf")), (ea, ew)


def check_swiglu(a, sa, w, sw, q, s, I):
    gu, d = R.product(R.values(a, sa), R.values(w, sw))
    h, dh = R.swiglu(gu[:, :I], d[:, :I], gu[:, I:], d[:, I:])
    hb, db = h.unflatten(-1, (-1, 32)), dh.unflatten(-1, (-1, 32))
    # the scale is the definition's for some h within the bound
    lo, hi = (hb.abs() - db).amax(-1), (hb.abs() + db).amax(-1)
    p = torch.exp2(s.double() - 127)
    assert bool((6 * p >= lo).all())
    assert bool(((s == 0) | (3 * p < hi)).all())
    # each value is a nearest grid point of some h within the bound
    v = R.values(q, s).unflatten(-1, (-1, 32))
    t = (hb.abs() + db) / p.unsqueeze(-1)
    half = torch.where(t < 2, 0.25, torch.where(t < 4, 0.5, 1.0)) * p.unsqueeze(-1)
    bad = (v - hb).abs() > half + db
    assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("counts,K,I", [([1], 32, 32), ([5, 0, 70], 96, 64), ([64, 130], 256, 256),
                                        ([7, 200, 65, 0, 1], 1440, 544), ([100, 28], 7168, 160),
                                        ([257, 255], 2048, 288), ([3, 9, 16], 7168, 1056),
                                        ([257, 255], 2048, 4128), ([70, 200, 65, 0, 61], 1440, 4160),
                                        ([300, 212], 96, 4128)])
@pytest.mark.parametrize("form", ["segments", "masked"])
def test_grouped_swiglu(counts, K, I, form):
    announce("grouped swiglu %s counts=%s K=%d I=%d" % (form, counts, K, I))
    g = gen(K + I)
    L = len(counts)
    w, sw = mx_random(g, L, 2 * I, K, lo=118, hi=121)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    if form == "masked":
        cap = max(counts) + 2
        a, sa = mx_random(g, L, cap, K, lo=122, hi=126)
        q = torch.full((L, cap, I // 2), CANARY, dtype=torch.uint8, device=DEV)
        s = torch.full((L, cap, I // 32), CANARY, dtype=torch.uint8, device=DEV)
        cdl.grouped_swiglu_mxfp4(a, sa, w, sw, c, out_q=q, out_scales=s)
        begins = [e * cap for e in range(L)]
        a, sa, q, s = (t.view(L * cap, -1) for t in (a, sa, q, s))
    else:
        begins = segments(counts, 8)
        a, sa = mx_random(g, begins[-1] + 3, K, lo=122, hi=126)
        q = torch.full((begins[-1] + 3, I // 2), CANARY, dtype=torch.uint8, device=DEV)
        s = torch.full((begins[-1] + 3, I // 32), CANARY, dtype=torch.uint8, device=DEV)
        cdl.grouped_swiglu_mxfp4(a, sa, w, sw, c, torch.tensor(begins, device=DEV), out_q=q, out_scales=s)
    live = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for e, n in enumerate(counts):
        at = slice(begins[e], begins[e] + n)
        live[at] = True
        if n:
            check_swiglu(a[at], sa[at], w[e], sw[e], q[at], s[at], I)
    assert bool((q[~live] == CANARY).all()) and bool((s[~live] == CANARY).all())


def test_swiglu_saturated_gates():
    """Gates far out on both sides: silu(g) -> g and -> 0, never NaN."""
    K, I = 32, 32
    a, sa = torch.zeros(4, 16, dtype=torch.uint8, device=DEV), torch.full((4, 1), 127, dtype=torch.uint8, device=DEV)
    a[:, 0] = torch.tensor([2, 10, 2, 10], dtype=torch.uint8)        # +-1
    w = torch.zeros(1, 64, 16, dtype=torch.uint8, device=DEV)
    w[0, :, 0] = 2
    sw = torch.full((1, 64, 1), 127, dtype=torch.uint8, device=DEV)
    sw[0, :32] = 140                                                  # gates of +-8192
    q, s = cdl.grouped_swiglu_mxfp4(a, sa, w, sw, torch.tensor([4], dtype=torch.int32, device=DEV),
                                    torch.tensor([0, 4], device=DEV))
    v = R.values(q, s)
    want = torch.tensor([8192.0, 0.0, 8192.0, 0.0], dtype=torch.float64, device=DEV)
    assert torch.equal(v.abs(), want[:, None].expand(4, 32))


def test_grouped_offsets_past_32_bits():
    """Weights and output rows beyond 4 GiB from the tensors' start."""
    announce("grouped, far offsets")
    L, N, K = 5, 4096, 1 << 19                                        # 1 GiB of codes an expert
    g = gen(2)
    w = torch.randint(0, 256, (L, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    sw = torch.full((L, N, K // 32), 118, dtype=torch.uint8, device=DEV)
    counts, seg = [1, 0, 0, 0, 3], [0, 1, 1, 1, 1, 4]
    a, sa = mx_random(g, 4, K, lo=120, hi=122)
    canary = torch.full((1,), -7.5, dtype=torch.bfloat16, device=DEV)
    out = canary.expand(4, N).contiguous()
    cdl.grouped_mxfp4(a, sa, w, sw, torch.tensor(counts, dtype=torch.int32, device=DEV),
                      torch.tensor(seg, device=DEV), out=out)
    for e, at in ((0, slice(0, 1)), (4, slice(1, 4))):
        for n0 in (0, 2000, N - 8):
            y, err = R.product(R.values(a[at], sa[at]), R.values(w[e, n0:n0 + 8], sw[e, n0:n0 + 8]))
            assert bool(((out[at, n0:n0 + 8].double() - y).abs() <= err + R.BF16 * (y.abs() + err) + R.TINY).all())


# ---------------------------------------------------------------------------
# the layer of a few tokens
# ---------------------------------------------------------------------------

LAYERS = [  # T, H, I, E, L, k, begin
    (1, 64, 32, 4, 4, 1, 0), (1, 7168, 96, 32, 32, 8, 0), (3, 96, 64, 8, 8, 2, 0), (5, 2592, 1056, 12, 6, 4, 3),
    (16, 256, 128, 8, 8, 2, 0), (17, 512, 160, 4, 2, 2, 1), (64, 256, 128, 8, 8, 2, 0), (128, 416, 224, 64, 8, 8, 8),
    (2, 160, 96, 32, 32, 32, 0), (13, 64, 64, 128, 128, 5, 0), (13, 64, 64, 128, 100, 4, 20), (3, 16416, 32, 4, 4, 2, 0),
    (9, 64, 8224, 3, 3, 1, 0), (40, 4128, 64, 16, 16, 3, 0), (128, 32, 32, 2048, 2048, 32, 0),
    (128, 64, 32, 1, 1, 1, 0), (128, 128, 64, 40, 40, 32, 0), (37, 2080, 544, 40, 40, 6, 0), (8, 64, 2080, 64, 4, 3, 60),
]


def layer_inputs(T, H, I, E, L, k, seed=0):
    g = gen(T * 31 + H + I + seed)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    wts = torch.softmax(torch.randn(T, k, generator=g, device=DEV), -1)
    x = randn(g, T, H)
    w13, w2 = randn(g, L, 2 * I, H, scale=H ** -0.5), randn(g, L, H, I, scale=I ** -0.5)
    return x, ids, wts, w13, w2


def run_layer(kind, x, ids, wts, w13, w2, b, **kw):
    """(output, weights' float64 values) of either weight type."""
    if kind == "bf16":
        return cdl.moe_layer(x, ids, wts, w13, w2, b, **kw), w13.double(), w2.double()
    (q13, s13), (q2, s2) = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
    return (cdl.moe_layer_mxfp4(x, ids, wts, q13, s13, q2, s2, b, **kw), R.values(q13, s13), R.values(q2, s2))


def check_layer(kind, x, ids, wts, w13, w2, b, **kw):
    out, v13, v2 = run_layer(kind, x, ids, wts, w13, w2, b, **kw)
    want, bound = R.layer(x.double(), ids, wts, v13, v2, b)
    bad = (out.double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), float(((out.double() - want).abs() / bound).max()))
    return out


@pytest.mark.parametrize("T,H,I,E,L,k,b", LAYERS)
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer(T, H, I, E, L, k, b, kind):
    announce("layer %s T=%d H=%d I=%d E=%d L=%d k=%d" % (kind, T, H, I, E, L, k))
    check_layer(kind, *layer_inputs(T, H, I, E, L, k), b)


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (4, 40, 24), (20, 1000, 200), (9, 264, 1048)])
def test_layer_bf16_rows_of_eight(T, H, I):
    announce("layer bf16 T=%d H=%d I=%d" % (T, H, I))
    check_layer("bf16", *layer_inputs(T, H, I, 6, 6, 3), 0)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_routing_edges(kind):
    """No local slot at all, ids of other ranks and negative ids, an expert
    named twice by one token (both slots count), every token on one expert."""
    x, ids, wts, w13, w2 = layer_inputs(40, 128, 64, 8, 4, 4)
    none = torch.full_like(ids, 99)
    out, _, _ = run_layer(kind, x, none, wts, w13, w2, 0, out=torch.full_like(x, 5.0))
    assert bool((out.view(torch.int16) == 0).all())
    mixed = ids.clone()
    mixed[::3] = -1
    mixed[1, :] = 2 ** 31 - 1
    mixed[2, 0] = -2 ** 31
    check_layer(kind, x, mixed, wts, w13, w2, 2)
    one = torch.full((1, 4), 1, dtype=torch.int32, device=DEV)      # one token, four slots of one expert
    check_layer(kind, x[:1].contiguous(), one, wts[:1].contiguous(), w13, w2, 0)
    twice = ids.clone()
    twice[:, 1] = twice[:, 0]
    twice[5, :] = 3
    check_layer(kind, x, twice, wts, w13, w2, 0)
    check_layer(kind, x, torch.full_like(ids, 1), wts, w13, w2, 0)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_nonfinite_rows_stay_apart(kind):
    x, ids, wts, w13, w2 = layer_inputs(24, 256, 96, 4, 4, 2)
    clean, _, _ = run_layer(kind, x, ids, wts, w13, w2, 0)
    x2 = x.clone()
    x2[7, 5] = float("nan")
    x2[11, 9] = float("inf")
    out, _, _ = run_layer(kind, x2, ids, wts, w13, w2, 0)
    keep = [t for t in range(24) if t not in (7, 11)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[7]).all())
    assert not bool(torch.isfinite(out[11]).all())


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3])
def test_layer_infinite_activations_stay_infinite(kind, T):
    """g = u = 2^66 overflows h in fp32: its remainder is none, not inf - inf.
    Sums of +inf times positive weights are +inf; other tokens are exact."""
    announce("layer %s infinite h T=%d" % (kind, T))
    H, I = 64, 32
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[0, 0] = 1.0
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    wts = torch.full((T, 1), 0.5, device=DEV)
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device=DEV)
    w13[:, :, 0] = 2.0 ** 66
    w2 = torch.ones(1, H, I, dtype=torch.bfloat16, device=DEV)
    if kind == "bf16":
        out = cdl.moe_layer(x, ids, wts, w13, w2)
    else:
        out = cdl.moe_layer_mxfp4(x, ids, wts, *cdl.quant_mxfp4(w13), *cdl.quant_mxfp4(w2))
    assert bool((out[0] == float("inf")).all())
    assert bool((out[1:] == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_is_deterministic_on_a_side_stream(kind):
    a = layer_inputs(50, 512, 256, 16, 16, 4)
    ref, _, _ = run_layer(kind, *a, 0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s):
            out, _, _ = run_layer(kind, *a, 0)
        s.synchronize()
        assert torch.equal(out, ref)


def test_layer_int64_ids_and_reused_workspace():
    x, ids, wts, w13, w2 = layer_inputs(12, 128, 64, 8, 8, 2)
    big = layer_inputs(100, 128, 64, 8, 8, 2, seed=1)
    ws = torch.full((cdl.moe_layer_workspace_size(100, 2, 64, 8),), 0xFF, dtype=torch.uint8, device=DEV)
    check_layer("bf16", *big, 0, workspace=ws)
    check_layer("bf16", x, ids.long(), wts, w13, w2, 0, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        cdl.moe_layer(x, ids, wts, w13, w2, workspace=ws[:100])


def test_layer_empty_batch():
    _, _, _, w13, w2 = layer_inputs(1, 64, 32, 4, 4, 2)
    x, ids = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    out = cdl.moe_layer(x, ids, torch.empty(0, 2, device=DEV), w13, w2)
    assert out.shape == (0, 64)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def step(x, ids, wts, w13, w2, b, alignment):
    L = w13[0].shape[0]
    lay, q, s = cdl.permute_mxfp4(x, ids, b, L, alignment=alignment)
    h, hs = cdl.grouped_swiglu_mxfp4(q, s, *w13, lay.counts, lay.seg_indptr)
    y = cdl.grouped_mxfp4(h, hs, *w2, lay.counts, lay.seg_indptr)
    return lay, (q, s), (h, hs), y, cdl.combine(y, lay.src2dst, wts)


@pytest.mark.parametrize("T,H,I,E,L,k,b,A", [(200, 512, 288, 16, 8, 4, 4, 1), (90, 7168, 128, 8, 8, 2, 0, 16)])
def test_expert_step(T, H, I, E, L, k, b, A):
    """permute -> gate/up with SwiGLU -> down -> combine: every stage against
    the 64-bit form of its own inputs, and the low-latency form of the step
    gives the same rows."""
    announce("expert step T=%d H=%d I=%d" % (T, H, I))
    x, ids, wts, w13, w2 = layer_inputs(T, H, I, E, L, k)
    w13, w2 = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
    lay, (q, s), (h, hs), y, out = step(x, ids, wts, w13, w2, b, A)
    counts, seg = npy(lay.counts), npy(lay.seg_indptr)
    for e in range(L):
        at = slice(int(seg[e]), int(seg[e]) + int(counts[e]))
        if counts[e]:
            check_swiglu(q[at], s[at], w13[0][e], w13[1][e], h[at], hs[at], I)
            v, err = R.product(R.values(h[at], hs[at]), R.values(w2[0][e], w2[1][e]))
            assert bool(((y[at].double() - v).abs() <= err + R.BF16 * (v.abs() + err) + R.TINY).all())
    P = bits_of(y)
    want = oracle.combine(P, npy(lay.src2dst), wts.cpu().numpy(), T, k)
    assert np.array_equal(bits_of(out), want)
    cap = int(counts.max())
    _, ql, sl, mm, ll = cdl.permute_ll_mxfp4(x, ids, b, L, cap)
    hl, hsl = cdl.grouped_swiglu_mxfp4(ql, sl, *w13, mm)
    yl = cdl.grouped_mxfp4(hl, hsl, *w2, mm)
    assert torch.equal(cdl.combine(yl, ll, wts), out)


def test_graph_replays_match_eager():
    """The expert step and the layer captured into two graphs, replayed in
    turn with eager work between, on changed inputs."""
    announce("graphs")
    x, ids, wts, w13, w2 = layer_inputs(64, 256, 128, 8, 8, 2)
    m13, m2 = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
    ws = [torch.empty(cdl.moe_layer_workspace_size(64, 2, 128, 8), dtype=torch.uint8, device=DEV) for _ in range(2)]

    def first():
        return step(x, ids, wts, m13, m2, 0, 1)[4], cdl.moe_layer(x, ids, wts, w13, w2, workspace=ws[0])

    def second():
        return cdl.moe_layer_mxfp4(x, ids, wts, *m13, *m2, workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first(), second()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1, o2 = first()
    with torch.cuda.graph(g2):
        o3 = second()
    g = gen(77)
    for i in range(4):
        x.copy_(randn(g, 64, 256))
        ids.copy_(torch.rand(64, 8, generator=g, device=DEV).topk(2, -1).indices)
        e1, e2 = first()
        e3 = second()
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, e1) and torch.equal(o2, e2) and torch.equal(o3, e3), i


def test_binding_checks_operands():
    g = gen(1)
    a, sa = mx_random(g, 8, 64)
    w, sw = mx_random(g, 2, 16, 64)
    c, seg = torch.tensor([4, 4], dtype=torch.int32, device=DEV), torch.tensor([0, 4, 8], device=DEV)
    with pytest.raises(ValueError, match="scales"):
        cdl.grouped_mxfp4(a, sa[:, :1], w, sw, c, seg)
    with pytest.raises(ValueError, match="contiguous"):
        cdl.grouped_mxfp4(a, sa, w.transpose(0, 1), sw, c, seg)
    with pytest.raises(ValueError, match="w_q"):
        cdl.grouped_mxfp4(a, sa, *mx_random(g, 2, 16, 96), c, seg)
    with pytest.raises(TypeError, match="counts"):
        cdl.grouped_mxfp4(a, sa, w, sw, c.long(), seg)
    with pytest.raises(ValueError, match="counts"):
        cdl.grouped_mxfp4(a, sa, w, sw, c[:1], seg)
    with pytest.raises(ValueError, match="without seg_indptr"):
        cdl.grouped_mxfp4(a, sa, w, sw, c)
    with pytest.raises(ValueError, match="out"):
        cdl.grouped_mxfp4(a, sa, w, sw, c, seg, out=torch.empty(8, 8, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(cdl.CdlError):
        cdl.grouped_swiglu_mxfp4(a, sa, w, sw, c, seg)                # I = 8
    with pytest.raises(TypeError, match="bfloat16"):
        cdl.quant_mxfp4(torch.zeros(2, 64, device=DEV))
    with pytest.raises(cdl.CdlError):
        cdl.quant_mxfp4(randn(g, 2, 48))
    x, ids, wts, w13, w2 = layer_inputs(4, 64, 32, 4, 4, 2)
    with pytest.raises(cdl.CdlError):
        cdl.moe_layer(torch.zeros(129, 64, dtype=torch.bfloat16, device=DEV), ids.repeat(33, 1)[:129],
                      torch.ones(129, 2, device=DEV), w13, w2)
    with pytest.raises(ValueError, match="w2"):
        cdl.moe_layer(x, ids, wts, w13, w2[:, :, :16].contiguous())
    with pytest.raises(ValueError, match="topk_weights"):
        cdl.moe_layer(x, ids, wts[:, :1].contiguous(), w13, w2)
    with pytest.raises(TypeError, match="topk_weights"):
        cdl.moe_layer(x, ids, wts.double(), w13, w2)
