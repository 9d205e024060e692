"""GPU tests of the expert operators at values and sizes that their random
cases do not reach."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import experts_check as C
import experts_ref as R
from gpu_util import DEV, announce, status_word
from test_experts_gpu import COUNTS, LAYERS, gen, layer_inputs, mx_random, run_layer, step

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# permutes
# ---------------------------------------------------------------------------

# both sides of the borders up to which a batch counts itself in the row launch
BORDERS = [  # T, E, L, k
    (512, 8, 8, 6), (512, 8, 8, 7), (511, 63, 63, 7), (511, 64, 64, 7), (512, 512, 512, 8), (400, 513, 513, 10),
    (512, 1024, 1024, 6), (512, 1024, 1024, 7), (512, 1025, 1025, 1), (171, 1025, 1025, 3), (128, 1500, 1500, 4),
    (129, 1500, 1500, 4), (100, 1100, 1100, 16), (100, 1100, 1100, 17), (513, 8, 8, 5), (513, 8, 8, 6), (2560, 256, 32, 1),
    (2752, 256, 32, 1), (2753, 256, 32, 1), (1152, 256, 256, 2), (1153, 256, 256, 2), (2048, 32, 4, 2), (4096, 16, 4, 1),
]

# and those from which the layout has kernels of its own: T, H, E, L, k
APART = [
    (3068, 2048, 33, 33, 2), (3080, 2048, 33, 33, 2), (3080, 2048, 32, 32, 2), (3080, 2080, 129, 129, 2),
    (3080, 2080, 128, 128, 2), (3080, 4128, 513, 513, 2), (3080, 4128, 512, 512, 2), (4097, 32, 3, 3, 1),
]


@pytest.mark.parametrize("T,H,E,L,k", [(T, 96, E, L, k) for T, E, L, k in BORDERS] + APART)
def test_permutes_at_the_borders_of_their_forms(T, H, E, L, k):
    """The one-call permutes give the layout's own results and the rows that
    the scatter from a given layout stores, tokens without a local slot among
    them."""
    announce("mxfp4 permutes T=%d H=%d E=%d L=%d k=%d" % (T, H, E, L, k))
    b, A = (E - L) // 2, 4
    g = gen(T + E + k)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    ids[::5] = -1
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    want = cdl.dispatch_layout(ids, b, L, alignment=A)
    n, st = want.num_rows(), status_word()
    q = torch.full((n + 3, H // 2), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((n + 3, H // 32), 0xA5, dtype=torch.uint8, device=DEV)
    q2, s2 = q.clone(), s.clone()
    lay = cdl.permute_mxfp4(x, ids, b, L, out_q=q, out_scales=s, status=st, alignment=A)[0]
    for f in ("counts", "seg_indptr", "src2dst", "reorder_topk_ids"):
        assert torch.equal(getattr(lay, f), getattr(want, f)), f
    cdl.dispatch_mxfp4(x, want, out_q=q2, out_scales=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2) and int(st.item()) == 0
    # padded, with room for all but the fullest experts' last rows
    cap = max(1, int(want.counts.max()) - 1)
    st0 = status_word()
    _, _, mm0, map0 = cdl.permute_ll(x, ids, b, L, cap, status=st0)
    _, ql, sl, mm, ll = cdl.permute_ll_mxfp4(x, ids, b, L, cap, status=st)
    assert torch.equal(mm, mm0) and torch.equal(ll, map0) and torch.equal(st, st0)
    kept = ll >= 0
    rows, at = cdl.quant_mxfp4(x), torch.arange(T, device=DEV).repeat_interleave(k)[kept]
    assert torch.equal(ql.view(L * cap, -1)[ll[kept].long()], rows[0][at])
    assert torch.equal(sl.view(L * cap, -1)[ll[kept].long()], rows[1][at])


# ---------------------------------------------------------------------------
# grouped product
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("L", [2, 70])
@pytest.mark.parametrize("counts,flag", [(0, 0), (3, 1), (-1, 1)])
def test_grouped_counts_of_an_empty_buffer(L, counts, flag):
    """A buffer of no rows: counts that are not zero do not fit it and are
    flagged, as in any other buffer."""
    announce("grouped, no rows, L=%d counts=%d" % (L, counts))
    g = gen(L)
    w, sw = mx_random(g, L, 64, 64)
    c = torch.zeros(L, dtype=torch.int32, device=DEV)
    c[L - 1] = counts
    none = torch.empty(0, 32, dtype=torch.uint8, device=DEV), torch.empty(0, 2, dtype=torch.uint8, device=DEV)
    padded = [t.new_empty(L, 0, t.shape[1]) for t in none]
    seg = torch.zeros(L + 1, dtype=torch.int64, device=DEV)
    for call in (cdl.grouped_mxfp4, cdl.grouped_swiglu_mxfp4):
        st = status_word()
        call(*none, w, sw, c, seg, status=st)
        assert int(st.item()) == flag * cdl.CDL_STATUS_ROWS_OVERFLOW
        st = status_word()
        call(*padded, w, sw, c, status=st)
        assert int(st.item()) == flag * cdl.CDL_STATUS_LL_OVERFLOW


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K,N", [(1056, 5056), (64, 6400), (7168, 4992)])
def test_grouped_forms_give_the_same_bits(K, N, swiglu):
    """A row's result is the same in plain and padded segments and in padded
    buffers, with tiles of 64 rows (up to 256 rows an expert in a padded
    buffer) and of 256."""
    announce("grouped forms K=%d N=%d swiglu=%d" % (K, N, swiglu))
    g = gen(K + N)
    counts = [150, 40, 0, 256, 256, 8]                # segments: 280 tiles of 64 rows and more, so the large tile
    L, rows = len(counts), sum(counts)
    w, sw = mx_random(g, L, N, K, lo=118, hi=121)
    a, sa = mx_random(g, rows, K, lo=122, hi=126)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)

    def run(begins, total, shape, seg):
        """The live rows of a buffer of `total` rows, expert e's from begins[e] on."""
        q = torch.zeros(total, K // 2, dtype=torch.uint8, device=DEV)
        s = torch.zeros(total, K // 32, dtype=torch.uint8, device=DEV)
        live, first = [], 0
        for e, n in enumerate(counts):
            q[begins[e]:begins[e] + n], s[begins[e]:begins[e] + n] = a[first:first + n], sa[first:first + n]
            live += range(begins[e], begins[e] + n)
            first += n
        call = cdl.grouped_swiglu_mxfp4 if swiglu else cdl.grouped_mxfp4
        out = call(q.view(*shape, -1), s.view(*shape, -1), w, sw, c, seg)
        return [o.reshape(total, -1)[live] for o in (out if swiglu else (out,))]

    def segments(align, gap):
        seg = [0]
        for n in counts:
            seg.append(seg[-1] + (n + align - 1) // align * align + gap)
        return run(seg[:-1], seg[-1], (seg[-1],), torch.tensor(seg, device=DEV))

    def padded(cap):
        return run([e * cap for e in range(L)], L * cap, (L, cap), None)

    first = padded(256)
    for other in (padded(257), padded(700), segments(1, 0), segments(16, 3), segments(128, 500)):
        assert all(torch.equal(x, y) for x, y in zip(first, other))


def test_grouped_infinite_and_nan_activations():
    """MXFP4 has no infinity: a quantised one is the number 6 * 2^127, which the
    products multiply as such (it is infinite where the product is, and read
    back as bf16); the finite elements of its group are nothing beside it.  A
    NaN stays NaN."""
    announce("grouped, infinite activations")
    K, N = 96, 64
    x = torch.zeros(5, K, dtype=torch.bfloat16, device=DEV)
    x[0, 5], x[1, 40], x[2, 70], x[3, 5] = torch.inf, -torch.inf, torch.nan, 2.0
    x[0, 6] = 3.0                                      # of the infinity's group
    q, s = cdl.quant_mxfp4(x)
    assert torch.equal(cdl.dequant_mxfp4(q, s)[:2, [5, 40]], x[:2, [5, 40]])
    wide = torch.zeros(1, N, K, dtype=torch.float64, device=DEV)
    n = torch.arange(N, device=DEV)
    wide[0, n, 5] = wide[0, n, 40] = torch.exp2(-(n // 2).double()) * torch.where(n % 2 == 1, -1.5, 1.0)
    wide[0, :, 6] = 1.0 * wide[0, :, 5]
    w = cdl.quant_mxfp4(wide.to(torch.bfloat16))
    assert torch.equal(R.values(*w), wide)
    out = cdl.grouped_mxfp4(q, s, *w, torch.tensor([5], dtype=torch.int32, device=DEV),
                            torch.tensor([0, 5], device=DEV))
    big = 6 * 2.0 ** 127 * wide[0, :, 5]
    big = torch.where(big.abs() >= 2.0 ** 128, torch.sign(big) * torch.inf, big).to(torch.bfloat16)
    assert int(torch.isfinite(big).sum()) > 50 and bool(torch.isinf(big).any())
    assert torch.equal(out[0], big) and torch.equal(out[1], -big)
    assert bool(torch.isnan(out[2]).all())
    assert torch.equal(out[3], (2 * wide[0, :, 5]).to(torch.bfloat16)) and not bool(out[4].any())


def test_swiglu_infinite_and_nan_values():
    """h beyond fp32 is stored as +-6 * 2^127, as a quantised infinity is, h
    with a NaN as NaN; the groups beside them are as without."""
    announce("swiglu, infinite values")
    K, I = 32, 96
    x = torch.zeros(3, K, dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0], x[2, 1] = 1.0, 1.0, 1.0, torch.nan
    wide = torch.zeros(1, 2 * I, K, dtype=torch.bfloat16, device=DEV)
    wide[0, :, 0] = 1.0
    wide[0, [40, I + 40], 0] = 2.0 ** 66               # h = 2^132 in the second group
    wide[0, [50, I + 50], 0] = torch.tensor([2.0 ** 66, -2.0 ** 66], dtype=torch.bfloat16, device=DEV)
    q, s = cdl.grouped_swiglu_mxfp4(*cdl.quant_mxfp4(x), *cdl.quant_mxfp4(wide),
                                    torch.tensor([3], dtype=torch.int32, device=DEV), torch.tensor([0, 3], device=DEV))
    v = R.values(q, s)
    one = 0.75                                         # of silu(1) = 0.731 at the scale 2^-3
    want = torch.full((I,), one, dtype=torch.float64, device=DEV)
    want[32:64] = 0.0
    want[40], want[50] = 6 * 2.0 ** 127, -6 * 2.0 ** 127
    assert torch.equal(v[0], want) and torch.equal(v[1], want)
    assert bool(torch.isnan(v[2]).all())
    back = cdl.dequant_mxfp4(q, s)
    assert float(back[0, 40]) == torch.inf and float(back[0, 50]) == -torch.inf


def test_expert_step_nonfinite_tokens_stay_apart():
    """A token with a NaN gives NaN; one with an infinity, and one whose
    activations overflow, leave every other token's row as it is."""
    announce("expert step, non-finite tokens")
    x, ids, wts, w13, w2 = layer_inputs(24, 256, 96, 4, 4, 2)
    w13, w2 = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
    clean = step(x, ids, wts, w13, w2, 0, 1)[4]
    x2 = x.clone()
    x2[7, 5], x2[11, 9] = torch.nan, torch.inf
    x2[13] = x2[13] * 2.0 ** 70
    out = step(x2, ids, wts, w13, w2, 0, 1)[4]
    keep = [t for t in range(24) if t not in (7, 11, 13)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[7]).all())
    # sums of +-6 * 2^127 w: huge, infinite, or NaN where both signs overflow
    assert not torch.equal(out[11], clean[11]) and not float(out[13].abs().max()) <= 2.0 ** 100


@pytest.mark.parametrize("counts,K,N", COUNTS)
@pytest.mark.parametrize("form", ["segments", "padded"])
def test_grouped_exact_sums(counts, K, N, form):
    """Random codes at scales of 1 and 2: products are multiples of 2^-2 up to
    144, sums of K < 29000 of them exact in fp32 in any order, results one
    rounding to bf16 away."""
    announce("grouped exact %s counts=%s K=%d N=%d" % (form, counts[:6], K, N))
    assert K * 144 * 4 < 2 ** 24
    g = gen(K + N + len(counts))
    L = len(counts)
    w, sw = mx_random(g, L, N, K, lo=127, hi=128)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    if form == "padded":
        cap, seg = max(counts) + 1, None
        begins, shape = [e * cap for e in range(L)], (L, cap)
    else:
        begins = [sum(counts[:e]) + 3 * e for e in range(L)]
        shape = (sum(counts) + 3 * L,)
        seg = torch.tensor(begins + [shape[0]], device=DEV)
    a, sa = mx_random(g, *shape, K, lo=127, hi=128)
    out = torch.full((*shape, N), -7.5, dtype=torch.bfloat16, device=DEV)
    cdl.grouped_mxfp4(a, sa, w, sw, c, seg, out=out)
    a, sa, out = a.view(-1, K // 2), sa.view(-1, K // 32), out.view(-1, N)
    want = torch.full_like(out, -7.5)
    for e, n in enumerate(counts):
        at = slice(begins[e], begins[e] + n)
        want[at] = (R.values(a[at], sa[at]) @ R.values(w[e], sw[e]).t()).to(torch.bfloat16)
    assert torch.equal(out, want)


FAR = (0, 31, 127, 128, 255, 256, 511, 4096, 131071, 131072, 200000, 262143)      # bytes of a row of 2^19 elements


def far_rows(g, q, s):
    """Random codes at the FAR bytes of rows q (zero elsewhere), random scales
    at their groups: dense rows of those elements alone, and their scales.
    Products of two such rows are multiples of 2^-2 below 2^20, so their
    fp32 sums are exact in any order."""
    at = torch.tensor(FAR, device=DEV)
    q[..., at] = torch.randint(0, 256, (*q.shape[:-1], len(FAR)), generator=g, device=DEV, dtype=torch.uint8)
    s[..., at // 16] = torch.randint(127, 132, (*s.shape[:-1], len(FAR)), generator=g, device=DEV,
                                     dtype=torch.int32).to(torch.uint8)
    grid = torch.tensor(R.GRID + tuple(-v for v in R.GRID), dtype=torch.float64, device=DEV)
    codes = q[..., at]
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1)
    return (v * torch.exp2(s[..., at // 16].double() - 127).unsqueeze(-1)).flatten(-2)


def test_grouped_far_weights_and_rows():
    """Weights of an expert and rows of a segment more than 4 GiB from their
    tensors' start, exact sums: another expert's or row's operands, or another
    row's scales, give other numbers."""
    announce("grouped, far weights and rows")
    L, N, K = 5, 4096, 1 << 19                                        # 1 GiB of codes an expert
    g = gen(2)
    w = torch.zeros(L, N, K // 2, dtype=torch.uint8, device=DEV)
    sw = torch.full((L, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    counts, seg = [3, 0, 2, 0, 5], [0, 3, 9000, 9002, 18000, 18005]   # row 18000 is 4.4 GiB in
    a = torch.zeros(18005, K // 2, dtype=torch.uint8, device=DEV)
    sa = torch.full((18005, K // 32), 127, dtype=torch.uint8, device=DEV)
    vw, va = [far_rows(g, w[e], sw[e]) for e in range(L)], far_rows(g, a, sa)
    out = torch.full((18005, N), -7.5, dtype=torch.bfloat16, device=DEV)
    cdl.grouped_mxfp4(a, sa, w, sw, torch.tensor(counts, dtype=torch.int32, device=DEV),
                      torch.tensor(seg, device=DEV), out=out)
    want = torch.full_like(out, -7.5)
    for e, c in enumerate(counts):
        at = slice(seg[e], seg[e] + c)
        want[at] = (va[at] @ vw[e].t()).to(torch.bfloat16)
        assert c == 0 or not torch.equal(want[at], (va[at] @ vw[(e + 1) % L].t()).to(torch.bfloat16))
    assert torch.equal(out, want)


def test_grouped_far_outputs():
    """Output rows (bf16, and MXFP4 behind SwiGLU) more than 4 GiB from the
    tensors' start; products of 32 elements at equal scales are exact."""
    announce("grouped, far outputs")
    g = gen(3)
    R1, L, N, K = 300001, 2, 8192, 32                                 # 4.6 GiB of output
    a, sa = mx_random(g, R1, K, lo=127, hi=127)
    w, sw = mx_random(g, L, N, K, lo=127, hi=127)
    counts, seg = [149000, R1 - 149003], [0, 149003, R1]
    dev = torch.tensor(counts, dtype=torch.int32, device=DEV), torch.tensor(seg, device=DEV)
    out = torch.full((R1, N), -7.5, dtype=torch.bfloat16, device=DEV)
    cdl.grouped_mxfp4(a, sa, w, sw, *dev, out=out)
    for e in range(L):
        v = R.values(w[e], sw[e])
        for r in range(seg[e], seg[e] + counts[e], 20000):
            at = slice(r, min(r + 20000, seg[e] + counts[e]))
            assert torch.equal(out[at], (R.values(a[at], sa[at]) @ v.t()).to(torch.bfloat16)), (e, r)
    assert bool((out[149000:149003] == -7.5).all())
    del out
    I = 32768                                                         # 4.6 GiB of codes
    w, sw = mx_random(g, L, 2 * I, K, lo=124, hi=124)
    q, s = cdl.grouped_swiglu_mxfp4(a, sa, w, sw, *dev)
    for e, r in ((0, 0), (0, 148950), (1, 149003), (1, R1 - 50)):
        at = slice(r, r + 50)
        C.check_swiglu(a[at], sa[at], w[e], sw[e], q[at], s[at], I)


def test_far_quantised_rows():
    """Rows and read-back values more than 4 GiB from the tensors' start."""
    announce("quantise, far rows")
    rows, H = 20000, 131072                                           # 4.9 GiB of bf16
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    at = [0, 1, 16383, 16384, 16385, rows - 1]
    x[at] = torch.randn(len(at), H, generator=gen(4), device=DEV).to(torch.bfloat16)
    q, s = cdl.quant_mxfp4(x)
    near = cdl.quant_mxfp4(x[at].contiguous())
    assert torch.equal(q[at], near[0]) and torch.equal(s[at], near[1])
    out = cdl.dequant_mxfp4(q, s)
    assert torch.equal(out[at].double(), R.values(*near))
    out[at] = 0
    assert not bool(out.any())


# ---------------------------------------------------------------------------
# the layer of a few tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3])
def test_layer_infinite_and_nan_weights(kind, T):
    """Row n of the down weights has one infinity, against h[n % I] alone, or
    one NaN: the output is that infinity times h's sign and the token's weight,
    or NaN, whatever the rounding of h left over."""
    announce("layer %s non-finite down weights T=%d" % (kind, T))
    H, I = 256, 96
    x, ids, wts, w13, w2 = layer_inputs(T, H, I, 1, 1, 1)
    n = torch.arange(H, device=DEV)
    i = n % I
    w2[0, n, i] = torch.where(n % 3 == 1, -torch.inf, torch.inf).to(torch.bfloat16)
    w2[0, 2::3, 5] = torch.nan
    if kind == "bf16":
        v13 = w13.double()
        out = cdl.moe_layer(x, ids, wts, w13, w2)
    else:
        q13, q2 = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
        v13 = cdl.dequant_mxfp4(*q13).double()
        out = cdl.moe_layer_mxfp4(x, ids, wts, *q13, *q2)
    gu = x.double() @ v13[0].t()
    h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    assert bool((h.abs() > 1e-20).all())               # signs that no rounding changes
    want = torch.sign(h[:, i]) * torch.where(n % 3 == 1, -torch.inf, torch.inf) * wts.double()
    want[:, 2::3] = torch.nan
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out.double(), nan=0.0, posinf=1.0, neginf=-1.0),
                       torch.nan_to_num(want, nan=0.0, posinf=1.0, neginf=-1.0))


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_smaller_batches_in_one_workspace(kind):
    """The workspace of three tokens serves two and one; nothing behind its
    size is written."""
    H, I, L, k = 128, 96, 8, 4
    size = cdl.moe_layer_workspace_size(3, k, I, L)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    for T in (3, 2, 1):
        announce("layer %s T=%d in the workspace of 3" % (kind, T))
        a = layer_inputs(T, H, I, L, L, k)
        out, v13, v2 = run_layer(kind, *a, 0, workspace=ws[:size])
        C.check_layer_output(out, *a[:3], v13, v2, 0)
        assert bool((ws[size:] == 0xA5).all())


@pytest.mark.parametrize("T,H,I,E,L,k", [(1, 96, 64, 64, 64, 64), (2, 96, 64, 64, 64, 64), (2, 64, 544, 2048, 2048, 64),
                                         (3, 4128, 32, 80, 70, 64), (64, 64, 96, 70, 64, 64), (128, 4128, 32, 40, 30, 32),
                                         (2, 64, 32, 128, 1, 64), (128, 64, 288, 2, 2, 2)])
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_many_slots(T, H, I, E, L, k, kind):
    """The most slots a token and a batch, and many of one expert, at both
    ends of the batch."""
    announce("layer %s T=%d H=%d I=%d E=%d L=%d k=%d" % (kind, T, H, I, E, L, k))
    a = layer_inputs(T, H, I, E, L, k)
    out, v13, v2 = run_layer(kind, *a, 0)
    C.check_layer_output(out, *a[:3], v13, v2, 0)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("T,H,I", [(1, 96, 160), (2, 1056, 32), (5, 2592, 96), (40, 288, 544), (6, 16416, 32)])
def test_layer_scales_at_any_byte(T, H, I, shift):
    """Scale tensors that start at any byte between NaN codes."""
    announce("layer, scales at byte %d, T=%d H=%d I=%d" % (shift, T, H, I))
    x, ids, wts, w13, w2 = layer_inputs(T, H, I, 5, 4, 3)

    def moved(s):
        flat = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device=DEV)
        flat[shift:shift + s.numel()] = s.flatten()
        return flat[shift:shift + s.numel()].view(s.shape)

    (q13, s13), (q2, s2) = cdl.quant_mxfp4(w13), cdl.quant_mxfp4(w2)
    out = cdl.moe_layer_mxfp4(x, ids, wts, q13, moved(s13), q2, moved(s2))
    C.check_layer_output(out, x, ids, wts, R.values(q13, s13), R.values(q2, s2), 0)


def exact_layer_inputs(T, H, I, E, L, k, b):
    """Inputs of the layer whose every intermediate is exact, and its output in
    64 bits.  x: n = 2^j ones at odd places, for the gates, and up to 16 of +-1
    and +-2 at even ones; gate rows 32 / n or 64 / n at every odd place, so g is
    32 or 64 and 1 + exp(-g) is 1 in fp32: silu(g) = g; up rows of -2 to 2 at
    even places, so |u| <= 64 and h = g u is a bf16 number; down rows of -1 to
    1, token weights 1, 1/2 and 1/4: sums are multiples of 8."""
    g = gen(T * 7 + H + I + k)

    def places(first, count):
        """[T, count] distinct indices of the same parity."""
        return torch.rand(T, H // 2, generator=g, device=DEV).topk(count, -1).indices * 2 + first

    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    wts = torch.exp2(-torch.randint(0, 3, (T, k), generator=g, device=DEV).float())
    n = 1 << (min(32, H // 2).bit_length() - 1)
    x = torch.zeros(T, H, device=DEV)
    x.scatter_(1, places(1, n), torch.ones(T, n, device=DEV))
    m = min(16, H // 2)
    x.scatter_(1, places(0, m), torch.tensor([-2.0, -1.0, 1.0, 2.0], device=DEV)[
        torch.randint(0, 4, (T, m), generator=g, device=DEV)])
    w13 = torch.zeros(L, 2 * I, H, device=DEV)
    w13[:, :I, 1::2] = torch.randint(1, 3, (L, I, 1), generator=g, device=DEV).float() * (32 / n)
    w13[:, I:, 0::2] = torch.randint(-2, 3, (L, I, H // 2), generator=g, device=DEV).float()
    w2 = torch.randint(-1, 2, (L, H, I), generator=g, device=DEV).float()
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    most = torch.zeros_like(out)
    for e in range(L):
        t, j = torch.nonzero(ids == e + b, as_tuple=True)
        gu = x[t].double() @ w13[e].double().t()
        assert bool(((gu[:, :I] == 32) | (gu[:, :I] == 64)).all())
        h = gu[:, :I] * gu[:, I:]
        assert torch.equal(h.to(torch.bfloat16).double(), h)
        w = wts[t, j].double().unsqueeze(1)
        out.index_add_(0, t, (h @ w2[e].double().t()) * w)
        most.index_add_(0, t, (h.abs() @ w2[e].double().abs().t()) * w)
    assert float(most.max()) < 8 * 2 ** 24                 # 24 bits of multiples of 8
    return x.to(torch.bfloat16), ids, wts, w13.to(torch.bfloat16), w2.to(torch.bfloat16), out


@pytest.mark.parametrize("T,H,I,E,L,k,b", LAYERS + [(1, 16416, 64, 4, 4, 2, 0), (2, 7168, 96, 32, 32, 8, 0),
                                                   (128, 4128, 96, 40, 40, 4, 0), (64, 2048, 320, 16, 16, 8, 0)])
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_layer_exact_sums(T, H, I, E, L, k, b, kind):
    """Bounds of random sums grow with their depth; these sums are exact, so
    that the output is one rounding to bf16 away, whatever the sizes."""
    announce("layer exact %s T=%d H=%d I=%d E=%d L=%d k=%d" % (kind, T, H, I, E, L, k))
    x, ids, wts, w13, w2, want = exact_layer_inputs(T, H, I, E, L, k, b)
    out, v13, v2 = run_layer(kind, x, ids, wts, w13, w2, b)
    assert torch.equal(v13, w13.double()) and torch.equal(v2, w2.double())
    # (+ 0: a token without a slot gets +0)
    assert torch.equal(out, want.to(torch.bfloat16) + 0)
