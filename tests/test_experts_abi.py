"""Refusals of the MXFP4 and MoE-layer entry points: every bad argument is
answered on the host before any HIP call (CPU only; pointers are never
dereferenced)."""
import ctypes

import pytest
import torch

import combine_dispatch_layout_amd as cdl

OK, ENULL, ESIZE, EUNSUP, EWS, EBIG = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10001)
BIG = (1 << 24) + 32


def call(name, base, **over):
    args = dict(base)
    args.update(over)
    return getattr(cdl.library(), name)(*args.values())


QUANT = dict(x=FAKE, rows=4, H=64, q=FAKE, s=FAKE, stream=None)
DEQUANT = dict(q=FAKE, s=FAKE, rows=4, H=64, out=FAKE, stream=None)
DISPATCH = dict(x=FAKE, T=4, H=64, k=2, map=FAKE, q=FAKE, s=FAKE, cap=8, status=None, stream=None)
PERMUTE = dict(x=FAKE, T=4, H=64, k=2, ids=FAKE, b=0, L=4, A=1, counts=FAKE, seg=FAKE, s2d=FAKE, reo=FAKE, rc=8,
               q=FAKE, s=FAKE, cap=8, status=None, ws=FAKE, wsb=1 << 20, stream=None)
PERMUTE_LL = dict(x=FAKE, T=4, H=64, k=2, ids=FAKE, b=0, L=4, counts=FAKE, seg=FAKE, s2d=FAKE, reo=FAKE, rc=8,
                  cap=8, q=FAKE, s=FAKE, mm=FAKE, ll=FAKE, status=None, ws=FAKE, wsb=1 << 20, stream=None)
GROUPED = dict(q=FAKE, s=FAKE, rows=8, K=64, wq=FAKE, ws=FAKE, L=4, N=16, counts=FAKE, seg=FAKE, cap=0, out=FAKE,
               status=None, stream=None)
SWIGLU = dict(q=FAKE, s=FAKE, rows=8, K=64, wq=FAKE, ws=FAKE, L=4, I=32, counts=FAKE, seg=FAKE, cap=0, oq=FAKE,
              os=FAKE, status=None, stream=None)
LAYER = dict(x=FAKE, T=4, H=64, k=2, ids=FAKE, wts=FAKE, b=0, L=4, I=32, w13=FAKE, w2=FAKE, out=FAKE, ws=FAKE,
             wsb=1 << 20, stream=None)
LAYER4 = dict(x=FAKE, T=4, H=64, k=2, ids=FAKE, wts=FAKE, b=0, L=4, I=32, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE,
              out=FAKE, ws=FAKE, wsb=1 << 20, stream=None)


def cases():
    def add(name, base, *items):
        for over, code in items:
            yield pytest.param(name, base, over, code, id="%s-%s" % (name, "-".join(over)))

    row = [(dict(H=0), ESIZE), (dict(H=48), EUNSUP), (dict(H=BIG), EBIG)]
    yield from add("cdl_quant_mxfp4", QUANT, *row, (dict(rows=-1), ESIZE), (dict(x=None), ENULL),
                   (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(x=ODD), EUNSUP), (dict(q=ODD), EUNSUP),
                   (dict(rows=0, x=None), OK))
    yield from add("cdl_dequant_mxfp4", DEQUANT, *row, (dict(rows=-1), ESIZE), (dict(out=None), ENULL),
                   (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(out=ODD), EUNSUP), (dict(q=ODD), EUNSUP),
                   (dict(rows=1 << 60), EBIG), (dict(rows=0, q=None), OK))
    yield from add("cdl_dispatch_mxfp4", DISPATCH, *row, (dict(T=-1), ESIZE), (dict(k=0), ESIZE),
                   (dict(k=65), ESIZE), (dict(T=1 << 31), EBIG), (dict(cap=-1), ESIZE), (dict(cap=1 << 31), EBIG),
                   (dict(x=None), ENULL), (dict(map=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL),
                   (dict(x=ODD), EUNSUP), (dict(q=ODD), EUNSUP), (dict(T=0, x=None, map=None), OK))
    yield from add("cdl_permute_mxfp4", PERMUTE, *row, (dict(L=0), ESIZE), (dict(L=2049), ESIZE), (dict(A=0), ESIZE),
                   (dict(cap=-1), ESIZE), (dict(cap=1 << 31), EBIG), (dict(x=None), ENULL), (dict(ids=None), ENULL),
                   (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(ws=None), ENULL), (dict(wsb=8), EWS),
                   (dict(x=ODD), EUNSUP), (dict(q=ODD), EUNSUP))
    yield from add("cdl_permute_ll_mxfp4", PERMUTE_LL, *row, (dict(cap=-1), ESIZE), (dict(cap=1 << 30), EBIG),
                   (dict(mm=None), ENULL), (dict(ll=None), ENULL), (dict(x=None), ENULL), (dict(q=None), ENULL),
                   (dict(s=None), ENULL), (dict(wsb=8), EWS), (dict(x=ODD), EUNSUP), (dict(q=ODD), EUNSUP))
    common = [(dict(rows=-1), ESIZE), (dict(K=0), ESIZE), (dict(K=48), EUNSUP), (dict(K=BIG), EBIG),
              (dict(L=0), ESIZE), (dict(L=2049), ESIZE), (dict(rows=1 << 31), EBIG), (dict(counts=None), ENULL),
              (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(wq=None), ENULL), (dict(ws=None), ENULL),
              (dict(q=ODD), EUNSUP), (dict(wq=ODD), EUNSUP), (dict(seg=None, cap=3), ESIZE),
              (dict(seg=None, cap=-2), ESIZE), (dict(rows=0, q=None, s=None), OK)]
    yield from add("cdl_grouped_mxfp4", GROUPED, *common, (dict(N=0), ESIZE), (dict(N=BIG), EBIG),
                   (dict(out=None), ENULL), (dict(rows=(1 << 31) - 1, N=1 << 24), EBIG))
    yield from add("cdl_grouped_swiglu_mxfp4", SWIGLU, *common, (dict(I=0), ESIZE), (dict(I=BIG), EBIG),
                   (dict(I=48), EUNSUP), (dict(oq=None), ENULL), (dict(os=None), ENULL), (dict(oq=ODD), EUNSUP))
    layer = [(dict(T=-1), ESIZE), (dict(k=0), ESIZE), (dict(H=0), ESIZE), (dict(I=0), ESIZE), (dict(L=0), ESIZE),
             (dict(L=2049), ESIZE), (dict(H=BIG), EBIG), (dict(I=BIG), EBIG), (dict(T=129), EUNSUP),
             (dict(T=128, k=33), EUNSUP), (dict(x=None), ENULL), (dict(ids=None), ENULL), (dict(wts=None), ENULL),
             (dict(w13=None), ENULL), (dict(w2=None), ENULL), (dict(out=None), ENULL), (dict(ws=None), ENULL),
             (dict(wsb=64), EWS), (dict(x=ODD), EUNSUP), (dict(w13=ODD), EUNSUP), (dict(w2=ODD), EUNSUP),
             (dict(out=ODD), EUNSUP), (dict(ws=ODD), EUNSUP), (dict(T=0, x=None), OK)]
    yield from add("cdl_moe_layer", LAYER, *layer, (dict(H=36), EUNSUP), (dict(I=36), EUNSUP))
    yield from add("cdl_moe_layer_mxfp4", LAYER4, *layer, (dict(H=40), EUNSUP), (dict(I=40), EUNSUP),
                   (dict(s13=None), ENULL), (dict(s2=None), ENULL))


@pytest.mark.parametrize("name,base,over,code", cases())
def test_refusals(name, base, over, code):
    assert call(name, base, **over) == code


def test_layer_workspace_size():
    f = cdl.library().cdl_moe_layer_workspace_size
    assert f(1, 8, 2048, 32) >= 8 * 2048 * 2
    assert f(128, 8, 2048, 32) >= 1024 * 2048 * 2
    assert f(0, 8, 2048, 32) > 0
    for bad in ((-1, 8, 64, 4), (129, 8, 64, 4), (128, 33, 64, 4), (4, 0, 64, 4), (4, 2, 0, 4), (4, 2, 64, 0)):
        assert f(*bad) == 0
    with pytest.raises(cdl.CdlError):
        cdl.moe_layer_workspace_size(129, 8, 64, 4)


def test_binding_refuses_cpu_tensors():
    u8, bf = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, 2, dtype=torch.uint8)
    ids, wts = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    counts = torch.zeros(1, dtype=torch.int32)
    for call_ in (lambda: cdl.quant_mxfp4(bf), lambda: cdl.dequant_mxfp4(u8, s),
                  lambda: cdl.permute_mxfp4(bf, ids, 0, 1), lambda: cdl.permute_ll_mxfp4(bf, ids, 0, 1, 2),
                  lambda: cdl.grouped_mxfp4(u8[None], s[None], u8[None], s[None], counts),
                  lambda: cdl.grouped_swiglu_mxfp4(u8[None], s[None], u8[None], s[None], counts),
                  lambda: cdl.moe_layer(bf, ids, wts, bf[None], bf[None]),
                  lambda: cdl.moe_layer_mxfp4(bf, ids, wts, u8[None], s[None], u8[None], s[None])):
        with pytest.raises(ValueError, match="GPU"):
            call_()


def test_grouped_tile_numbers_leave_room_for_a_step():
    """Device counts may claim the whole buffer for every expert.  1302 experts
    of 49981 x 33 tiles are 2^31 - 2 tiles: a workgroup's step past the last
    tile would not fit 32 bits."""
    over = dict(rows=49981 * 256, N=33 * 256, L=1302)
    assert 1302 * 49981 * 33 == 2 ** 31 - 2
    assert call("cdl_grouped_mxfp4", GROUPED, **over) == EBIG
    assert call("cdl_grouped_swiglu_mxfp4", SWIGLU, rows=49981 * 256, I=33 * 128, L=1302) == EBIG


@pytest.mark.parametrize("k,I,L", [(1, 32, 1), (8, 2048, 32), (6, 1056, 40), (32, 64, 2048), (64, 96, 300), (2, 1 << 22, 4)])
def test_layer_workspace_grows_with_the_batch(k, I, L):
    """A workspace of the largest batch serves every smaller one."""
    f = cdl.library().cdl_moe_layer_workspace_size
    most = min(128, 4096 // k)
    sizes = [f(T, k, I, L) for T in range(most + 1)]
    assert all(0 < a <= b for a, b in zip(sizes, sizes[1:])), sizes[:5]


def test_layer_sizes_at_the_32_bit_limit():
    """Byte offsets into the token rows and the activations stay below 2^32: T
    * H, and the activations' elements of T tokens (4 tokens' from 2 to 4, 2
    tokens' for one), reach 2^31 - 9 at most.  The workspace's size is asked for only
    of sizes that are taken."""
    H = 1 << 24
    for name, base in (("cdl_moe_layer", LAYER), ("cdl_moe_layer_mxfp4", LAYER4)):
        assert call(name, base, T=127, H=H, wsb=64) == EWS
        assert call(name, base, T=128, H=H, wsb=64) == EBIG
        for k, T, most in ((64, 2, 4), (64, 3, 4), (64, 4, 4), (64, 1, 2), (64, 5, 5)):
            I = (2 ** 31 - 9) // (most * k) // 32 * 32
            assert call(name, base, T=T, k=k, I=I, wsb=64) == EWS, (T, I)
            assert call(name, base, T=T, k=k, I=I + 32, wsb=64) == EBIG, (T, I)
