"""The products grouped by expert where ordinary values and sizes do not tell
a mistake: sums that a matrix instruction's own alignment would lose, tiles of
every size with up to all of their rows live, and workgroups that walk several."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import differences as D
import products_ref as R
import products_tiles as tiles
from gpu_util import DEV, announce
from test_products_gpu import BF, CANARY, canaries, check_fp8_values, fp8_rows, fp8_weights, gen, rand, Rows

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


# ---------------------------------------------------------------------------
# tiles of 128, 192 and 256 rows
# ---------------------------------------------------------------------------

# up to 1, 2, 3 and 4 blocks of 64 rows live in a tile of 256, and all but one of its rows
COUNTS = [193, 255, 0, 256, 257, 600]
# column tiles, the rows of a tile that the rule takes for them, and whether a workgroup has several tiles
SIZES = [(8, 128, False), (20, 192, False), (24, 256, False), (52, 192, True), (64, 256, True)]


def expect(r, width, rows, several, **form):
    L = len(r.counts)
    assert tiles.tile_rows(r.n, L, width, **form) == rows
    assert (tiles.tiles(r.counts, rows, width, form.get("swiglu", False)) > 256) == several


def same_outside(r, out):
    r.check_rest(out, torch.tensor(CANARY, dtype=BF, device=DEV))


@pytest.mark.parametrize("columns,rows,several", SIZES)
def test_bf16_product_in_every_tile(columns, rows, several):
    announce("bf16 product, %d column tiles, %d rows a tile" % (columns, rows))
    r, g, K, N = Rows(COUNTS, False), gen(columns), 328, 256 * columns - 77
    expect(r, N, rows, several)
    x, w, out = rand(g, r.n, K), rand(g, len(COUNTS), N, K), canaries(r, N)
    cdl.grouped_bf16(r.poisoned(x), w, r.c, r.seg, out=out)
    for e, at in r.each():
        y, err = R.product(x[at].double(), w[e].double())
        R.assert_within(out[at], y, R.to_bf16_bound(y, err), e)
    same_outside(r, out)


@pytest.mark.parametrize("columns,rows,several", SIZES)
def test_bf16_swiglu_and_its_gradient_in_every_tile(columns, rows, several):
    announce("bf16 swiglu, %d column tiles, %d rows a tile" % (columns, rows))
    r, g, K, I = Rows(COUNTS, False), gen(columns + 1), 328, 128 * columns - 53
    expect(r, I, rows, several, swiglu=True)
    x, w, dh = rand(g, r.n, K), rand(g, len(COUNTS), 2 * I, K, scale=K ** -0.5), rand(g, r.n, I)
    out, dgu = canaries(r, I), canaries(r, 2 * I)
    cdl.grouped_swiglu_bf16(r.poisoned(x), w, r.c, r.seg, out=out)
    cdl.grouped_swiglu_bf16_grad(r.poisoned(x), w, r.poisoned(dh), r.c, r.seg, out=dgu)
    for e, at in r.each():
        gu, d = R.product(x[at].double(), w[e].double())
        gate, up, eg, eu = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        h, err = R.swiglu(gate, eg, up, eu)
        R.assert_within(out[at], h, R.to_bf16_bound(h, err), e)
        dg, bg, du, bu = R.swiglu_grad(gate, eg, up, eu, dh[at].double())
        R.assert_within(dgu[at, :I], dg, R.to_bf16_bound(dg, bg), e)
        R.assert_within(dgu[at, I:], du, R.to_bf16_bound(du, bu), e)
    same_outside(r, out)
    same_outside(r, dgu)


@pytest.mark.parametrize("columns,rows,several", SIZES)
def test_bf16_row_gradient_in_every_tile(columns, rows, several):
    announce("bf16 dx, %d column tiles, %d rows a tile" % (columns, rows))
    r, g, K, N = Rows(COUNTS, False), gen(columns + 2), 256 * columns - 72, 328
    expect(r, K, rows, several)
    dy, w, dx = rand(g, r.n, N), rand(g, len(COUNTS), N, K), canaries(r, K)
    cdl.grouped_bf16_dx(r.poisoned(dy), w, r.c, r.seg, out=dx)
    for e, at in r.each():
        y, err = R.product(dy[at].double(), w[e].double().t())
        R.assert_within(dx[at], y, R.to_bf16_bound(y, err), e)
    same_outside(r, dx)


@pytest.mark.parametrize("flags,K", [(0, 1152), (7, 1152), (2, 640)])
@pytest.mark.parametrize("columns,rows,several", SIZES)
def test_fp8_product_in_every_tile(columns, rows, several, flags, K):
    """Scale groups past a word of four, whose number is no multiple of it."""
    announce("fp8 product, %d column tiles, %d rows a tile, flags %d" % (columns, rows, flags))
    r, g, N = Rows(COUNTS, False), gen(columns + flags), 256 * columns - 77
    expect(r, N, rows, several, fp8=True)
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, len(COUNTS), N, K)
    out = canaries(r, N)
    cdl.grouped_fp8(r.poisoned(q), s, wq, ws, r.c, r.seg, scale_flags=flags, out=out)
    for e, at in r.each():
        for c in range(0, N, 4096):                          # (the reference's working memory)
            y, err = R.fp8_product(q[at], p[at], *part(wq[e], ws[e], c, min(c + 4096, N)))
            R.assert_within(out[at, c:c + 4096], y, R.to_bf16_bound(y, err), e)
    same_outside(r, out)


def part(wq, ws, a, b):
    """Weight rows a to b (a a multiple of 128)."""
    return wq[a:b], ws[a // 128:-(-b // 128)]


@pytest.mark.parametrize("flags,K", [(0, 1152), (7, 1152), (2, 640)])
@pytest.mark.parametrize("columns,rows,several", [(8, 128, False), (20, 192, False), (52, 192, True), (70, 192, True)])
def test_fp8_swiglu_in_every_tile(columns, rows, several, flags, K):
    announce("fp8 swiglu, %d column tiles, %d rows a tile, flags %d" % (columns, rows, flags))
    r, g, I = Rows(COUNTS, False), gen(columns + flags), 128 * columns
    expect(r, I, rows, several, fp8=True, swiglu=True, quantised=True)
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, len(COUNTS), 2 * I, K)
    oq = torch.full((r.n, I), 0xA5, dtype=torch.uint8, device=DEV)
    hq, hs = cdl.grouped_swiglu_fp8(r.poisoned(q), s, wq, ws, r.c, r.seg, scale_flags=flags, out_q=oq)
    hp = R.scales(hs, flags, r.n, I // 128, r.n)
    for e, at in r.each():
        y, err = fp32_product(q[at], p[at], wq[e], ws[e])
        h, dh = R.swiglu(y[:, :I], err[:, :I], y[:, I:], err[:, I:])
        check_fp8_values(h, dh, hq[at], hp[at], flags & 1)
    r.check_rest(hq, torch.tensor(0xA5, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("flags", [0, 7])
def test_fp8_full_tiles_of_256_rows_beside_many_experts(flags):
    """1300 experts, whose tile table leaves the quantised SwiGLU 256 rows a tile alone, with one to four blocks of
    64 of them live; several experts of a workgroup in a row."""
    announce("fp8 products of 1300 experts, up to 257 rows, flags %d" % flags)
    L, K, N, g = 1300, 640, 256, gen(flags)
    counts = [0] * L
    for e, c in ((3, 257), (4, 64), (5, 65), (200, 129), (201, 128), (202, 193), (600, 256), (1298, 255), (1299, 200)):
        counts[e] = c
    r = Rows(counts, True)
    assert tiles.tile_rows(r.n, L, N, fp8=True, padded=True) == 256
    q, s, p = fp8_rows(g, r, K, flags)
    wq, ws = fp8_weights(g, L, N, K)
    y = cdl.grouped_fp8(r.shape(q), s, wq, ws, r.c, scale_flags=flags).view(r.n, N)
    hq, hs = cdl.grouped_swiglu_fp8(r.shape(q), s, wq, ws, r.c, scale_flags=flags)
    hq, hp = hq.view(r.n, N // 2), R.scales(hs, flags, r.n, 1, r.cap)
    for e, at in r.each():
        v, err = R.fp8_product(q[at], p[at], wq[e], ws[e])
        R.assert_within(y[at], v, R.to_bf16_bound(v, err), e)
        v, err = fp32_product(q[at], p[at], wq[e], ws[e])
        h, dh = R.swiglu(v[:, :N // 2], err[:, :N // 2], v[:, N // 2:], err[:, N // 2:])
        check_fp8_values(h, dh, hq[at], hp[at], flags & 1)


def test_a_row_has_the_same_bits_in_every_tile():
    """1024, 1500 and 2048 rows of one expert take 128, 192 and 256 rows a tile, a padded buffer 192: the rows that
    they share have the same bits in all forms."""
    announce("products: a row's bits in tiles of 128, 192 and 256 rows")
    g, most, K, W = gen(21), 2048, 384, 8192
    sizes = [(1024, 128), (1500, 192), (2048, 256)]
    x, dy, dh = rand(g, most, K), rand(g, most, K), rand(g, most, W // 2)
    w, wt, wg = rand(g, 1, W, K, scale=K ** -0.5), rand(g, 1, K, W, scale=K ** -0.5), rand(g, 1, W, K, scale=K ** -0.5)
    for n, rows in sizes:
        assert tiles.tile_rows(n, 1, W) == tiles.tile_rows(n, 1, W, fp8=True) == rows
        assert tiles.tile_rows(n, 1, W // 2, swiglu=True) == rows
    assert [tiles.tile_rows(n, 1, W // 2, fp8=True, swiglu=True, quantised=True) for n, _ in sizes] == [128, 192, 128]
    lay = cdl.dispatch_layout(torch.zeros(most, 1, dtype=torch.int32, device=DEV), 0, 1)
    q, s = cdl.dispatch_fp8(x, lay, rows=most)
    w8, w8s = cdl.quant_fp8_blocks(w)
    forms = {
        "product": lambda n, c, g, v: cdl.grouped_bf16(v(x[:n]), w, c, g),
        "swiglu": lambda n, c, g, v: cdl.grouped_swiglu_bf16(v(x[:n]), wg, c, g),
        "swiglu gradient": lambda n, c, g, v: cdl.grouped_swiglu_bf16_grad(v(x[:n]), wg, v(dh[:n]), c, g),
        "dx": lambda n, c, g, v: cdl.grouped_bf16_dx(v(dy[:n]), wt, c, g),
        "fp8": lambda n, c, g, v: cdl.grouped_fp8(v(q[:n]), v(s[:n]), w8, w8s, c, g),
        "fp8 swiglu": lambda n, c, g, v: cdl.grouped_swiglu_fp8(v(q[:n]), v(s[:n]), w8, w8s, c, g),
    }
    for name, call in forms.items():
        got = []
        for n, _ in sizes:
            c, seg = one_expert(n)
            got.append((n, call(n, c, seg, lambda t: t)))
            got.append((n, call(n, c, None, lambda t: t[None])))
        flat = lambda o, k: [t.reshape(-1, t.shape[-1])[:k] for t in (o if isinstance(o, tuple) else (o,))]   # noqa: E731
        n0, first = got[0]
        for n, o in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(flat(o, n0), flat(first, n0))), (name, n)
        assert all(torch.equal(a, b) for a, b in zip(flat(got[4][1], 1500), flat(got[2][1], 1500))), name


def test_training_pass_has_the_slopes_of_differences():
    """The experts' layer as a torch.autograd.Function: its gradients against differences of the layer in 64 bits."""
    announce("bf16 training pass, differences")
    g, T, H, I, E, k = gen(31), 120, 64, 72, 4, 2
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.to(torch.int32)
    lay, rows = cdl.permute(rand(g, T, H), ids, 0, E)
    at = (lay.counts, lay.seg_indptr)

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w13, w2):
            h = cdl.grouped_swiglu_bf16(x, w13, *at)
            ctx.save_for_backward(x, w13, w2, h)
            return cdl.grouped_bf16(h, w2, *at)

        @staticmethod
        def backward(ctx, dy):
            x, w13, w2, h = ctx.saved_tensors
            dgu = cdl.grouped_swiglu_bf16_grad(x, w13, cdl.grouped_bf16_dx(dy, w2, *at), *at)
            return cdl.grouped_bf16_dx(dgu, w13, *at), cdl.grouped_bf16_dw(dgu, x, *at), cdl.grouped_bf16_dw(dy, h, *at)

    w13, w2 = rand(g, E, 2 * I, H, scale=H ** -0.5), rand(g, E, H, I, scale=I ** -0.5)
    dy = rand(g, rows.shape[0], H)
    leaves = [t.clone().requires_grad_() for t in (rows, w13, w2)]
    Experts.apply(*leaves).backward(dy)
    args, loss = [w13.double(), w2.double(), rows.double()], D.experts_loss(dy.double(), lay.seg_indptr.tolist(), I)
    # h, dh and dgu are rounded to bf16 on the way, at most two of them in a row before the result itself
    for got, which in ((leaves[1].grad, 0), (leaves[2].grad, 1), (leaves[0].grad, 2)):
        assert D.slopes_agree(got, loss, args, which, g, 3 * R.BF16 * float(got.double().norm())), which
