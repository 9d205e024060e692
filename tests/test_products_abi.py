"""Refusals of the bf16 and fp8 products and of the norm: every bad argument is
answered on the host before any HIP call (CPU only; pointers are never
dereferenced)."""
import ctypes

import pytest
import torch

import combine_dispatch_layout_amd as cdl

OK, ENULL, ESIZE, EUNSUP, EWS, EBIG = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
FAKE, ODD, BY4 = P(0x10000), P(0x10001), P(0x10004)
WIDE = (1 << 21) + 128

AT = dict(counts=FAKE, seg=FAKE, cap=0)
END = dict(out=FAKE, status=None, stream=None)
BF16 = dict(x=FAKE, rows=8, K=64, w=FAKE, L=4, N=16, **AT, **END)
GRAD = dict(x=FAKE, rows=8, K=64, w=FAKE, L=4, N=16, dh=FAKE, **AT, **END)
DX = dict(x=FAKE, rows=8, N=16, w=FAKE, L=4, K=64, **AT, **END)
DW = dict(dy=FAKE, x=FAKE, rows=8, N=16, K=64, L=4, **AT, **END)
FP8 = dict(x=FAKE, s=FAKE, flags=0, rows=8, K=256, w=FAKE, ws=FAKE, L=4, N=16, **AT, **END)
SWIGLU8 = dict(x=FAKE, s=FAKE, flags=0, rows=8, K=256, w=FAKE, ws=FAKE, L=4, N=128, **AT, out=FAKE, os=FAKE, status=None,
               stream=None)
QUANT = dict(w=FAKE, mats=2, N=16, K=256, q=FAKE, s=FAKE, stream=None)
DEQUANT = dict(q=FAKE, s=FAKE, flags=0, rows=8, H=256, rpm=8, out=FAKE, stream=None)
NORM = dict(x=FAKE, res=FAKE, w=FAKE, eps=ctypes.c_float(1e-6), T=4, H=64, out=FAKE, ro=FAKE, stream=None)
NORM8 = dict(x=FAKE, res=FAKE, w=FAKE, eps=ctypes.c_float(1e-6), T=4, H=256, q=FAKE, s=FAKE, flags=0, out=FAKE, ro=FAKE,
             stream=None)
NGRAD = dict(dy=FAKE, h=FAKE, w=FAKE, dres=FAKE, eps=ctypes.c_float(1e-6), T=4, H=64, dx=FAKE, dw=FAKE, ws=FAKE,
             wsb=1 << 20, stream=None)


def cases():
    def add(name, base, *items):
        for over, code in items:
            yield pytest.param(name, base, over, code, id="%s-%s" % (name, "-".join("%s=%s" % (k, getattr(v, "value", v))
                                                                                    for k, v in over.items())))

    sizes = [(dict(rows=-1), ESIZE), (dict(K=0), ESIZE), (dict(N=0), ESIZE), (dict(L=0), ESIZE), (dict(L=2049), ESIZE),
             (dict(K=WIDE), EBIG), (dict(N=WIDE), EBIG), (dict(rows=1 << 31), EBIG), (dict(counts=None), ENULL),
             (dict(seg=None, cap=3), ESIZE), (dict(seg=None, cap=-2), ESIZE),
             # L * row tiles * column tiles beyond the tile numbers
             (dict(rows=(1 << 31) - 1, N=1 << 20, L=2048), EBIG)]
    bf16 = [(dict(x=None), ENULL), (dict(w=None), ENULL), (dict(out=None), ENULL), (dict(K=60), EUNSUP),
            (dict(x=BY4), EUNSUP), (dict(w=BY4), EUNSUP), (dict(out=ODD), EUNSUP), (dict(rows=0, x=None, out=None), OK),
            (dict(seg=None, rows=0, x=None, out=None), OK)]
    yield from add("cdl_grouped_bf16", BF16, *sizes, *bf16)
    yield from add("cdl_grouped_swiglu_bf16", BF16, *sizes[:-1], *bf16, (dict(N=1 << 20, rows=0, x=None, out=None), OK),
                   (dict(N=(1 << 20) + 1), EBIG), (dict(N=1 << 62), EBIG))
    yield from add("cdl_grouped_swiglu_bf16_grad", GRAD, *sizes[:-1], *bf16[:-2], (dict(dh=None), ENULL), (dict(dh=ODD), EUNSUP),
                   (dict(rows=0, x=None, out=None, dh=None), OK))
    yield from add("cdl_grouped_bf16_dx", DX, *sizes[:-1], (dict(rows=(1 << 31) - 1, K=1 << 20, L=2048), EBIG),
                   *bf16, (dict(N=12), EUNSUP), (dict(out=P(0x10002)), EUNSUP))
    yield from add("cdl_grouped_bf16_dw", DW, *sizes[:-1], (dict(N=1 << 20, K=1 << 20, L=2048), EBIG), (dict(dy=None), ENULL),
                   (dict(x=None), ENULL), (dict(out=None), ENULL), (dict(out=None, rows=0), ENULL), (dict(K=60), EUNSUP),
                   (dict(N=12), EUNSUP), (dict(dy=BY4), EUNSUP), (dict(x=BY4), EUNSUP), (dict(out=BY4), EUNSUP))
    fp8 = [(dict(x=None), ENULL), (dict(s=None), ENULL), (dict(w=None), ENULL), (dict(ws=None), ENULL), (dict(out=None), ENULL),
           (dict(K=192), EUNSUP), (dict(flags=4), EUNSUP), (dict(flags=8), EUNSUP), (dict(flags=-1), EUNSUP),
           (dict(x=BY4), EUNSUP), (dict(w=BY4), EUNSUP), (dict(s=P(0x10002)), EUNSUP), (dict(ws=P(0x10002)), EUNSUP)]
    yield from add("cdl_grouped_fp8", FP8, *sizes, *fp8, (dict(out=ODD), EUNSUP),
                   (dict(rows=0, x=None, s=None, out=None), OK))
    yield from add("cdl_grouped_swiglu_fp8", SWIGLU8, *sizes[:-1], *fp8, (dict(os=None), ENULL), (dict(N=64), EUNSUP),
                   (dict(out=BY4), EUNSUP), (dict(os=P(0x10002)), EUNSUP),
                   (dict(rows=0, x=None, s=None, out=None, os=None), OK))
    yield from add("cdl_quant_fp8_blocks", QUANT, (dict(mats=-1), ESIZE), (dict(N=0), ESIZE), (dict(K=0), ESIZE),
                   (dict(K=192), EUNSUP), (dict(K=(1 << 24) + 128), EBIG), (dict(N=(1 << 24) + 1), EBIG),
                   (dict(mats=1 << 40), EBIG), (dict(w=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL),
                   (dict(w=BY4), EUNSUP), (dict(q=BY4), EUNSUP), (dict(s=P(0x10002)), EUNSUP), (dict(mats=0, w=None), OK))
    yield from add("cdl_dequant_fp8", DEQUANT, (dict(rows=-1), ESIZE), (dict(H=0), ESIZE), (dict(rpm=0), ESIZE),
                   (dict(rpm=-1), ESIZE), (dict(H=192), EUNSUP), (dict(flags=4), EUNSUP), (dict(H=(1 << 24) + 128), EBIG),
                   (dict(rows=1 << 31), EBIG), (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(out=None), ENULL),
                   (dict(q=BY4), EUNSUP), (dict(out=BY4), EUNSUP), (dict(s=P(0x10002)), EUNSUP), (dict(rows=0, q=None), OK))
    eps = [(dict(eps=ctypes.c_float(-1e-6)), ESIZE), (dict(eps=ctypes.c_float(float("nan"))), ESIZE)]
    rows = [(dict(T=-1), ESIZE), (dict(H=0), ESIZE), (dict(H=(1 << 24) + 128), EBIG), (dict(T=1 << 31), EBIG), *eps]
    yield from add("cdl_rms_norm", NORM, *rows, (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(out=None), ENULL),
                   (dict(ro=None), ENULL), (dict(x=ODD), EUNSUP), (dict(res=ODD), EUNSUP), (dict(w=ODD), EUNSUP),
                   (dict(out=ODD), EUNSUP), (dict(ro=ODD), EUNSUP), (dict(T=0, x=None), OK))
    yield from add("cdl_rms_norm_fp8", NORM8, *rows, (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(q=None), ENULL),
                   (dict(s=None), ENULL), (dict(ro=None), ENULL), (dict(H=192), EUNSUP), (dict(flags=6), EUNSUP),
                   (dict(x=BY4), EUNSUP), (dict(res=BY4), EUNSUP), (dict(w=BY4), EUNSUP), (dict(out=BY4), EUNSUP),
                   (dict(ro=BY4), EUNSUP), (dict(q=BY4), EUNSUP), (dict(s=P(0x10002)), EUNSUP), (dict(T=0, x=None), OK))
    yield from add("cdl_rms_norm_grad", NGRAD, *rows, (dict(dy=None), ENULL), (dict(h=None), ENULL), (dict(w=None), ENULL),
                   (dict(dx=None), ENULL), (dict(dw=None), ENULL), (dict(ws=None), ENULL), (dict(wsb=255), EWS),
                   (dict(dw=P(0x10002)), EUNSUP), (dict(ws=BY4), EUNSUP), (dict(dy=ODD), EUNSUP), (dict(dres=ODD), EUNSUP),
                   (dict(dw=None, T=0), ENULL))


@pytest.mark.parametrize("name,base,over,code", cases())
def test_refusals(name, base, over, code):
    args = dict(base)
    assert not set(over) - set(args)
    args.update(over)
    assert getattr(cdl.library(), name)(*args.values()) == code


def test_workspace_of_the_norm_gradient():
    size = cdl.library().cdl_rms_norm_grad_workspace_size
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, (1 << 24) + 1) == 0 and size(1 << 31, 64) == 0
    assert size(0, 64) > 0
    for H in (1, 64, 7168, 8192, 8193, 1 << 20):
        n = [size(T, H) for T in (0, 1, 100, 511, 512, 513, 100000)]
        assert n == sorted(n)


@pytest.mark.parametrize("call", [
    lambda t: cdl.rms_norm(t, t[0]), lambda t: cdl.rms_norm_fp8(t, t[0]), lambda t: cdl.rms_norm_grad(t, t, t[0]),
    lambda t: cdl.grouped_bf16(t, t[None], t), lambda t: cdl.grouped_bf16_dx(t, t[None], t),
    lambda t: cdl.grouped_bf16_dw(t, t, t), lambda t: cdl.grouped_fp8(t, t, t[None], t, t),
    lambda t: cdl.quant_fp8_blocks(t), lambda t: cdl.dequant_fp8(t, t)])
def test_host_tensors_are_refused(call):
    with pytest.raises((ValueError, TypeError)):
        call(torch.zeros(4, 128, dtype=torch.bfloat16))
