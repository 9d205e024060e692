"""What the binding of the bf16 and fp8 products and of the norm refuses before any call of the
library (CPU only: the check for GPU tensors is left out, and a call that gets
through is a failure)."""
import math

import pytest
import torch

import combine_dispatch_layout_amd as cdl
from combine_dispatch_layout_amd import api

BF = torch.bfloat16
L, T, K, N = 2, 16, 128, 256


class Launched(Exception):
    pass


@pytest.fixture
def host(monkeypatch):
    def launch(what, *a):
        raise Launched(what)
    monkeypatch.setattr(api, "_need_gpu", lambda t, name: None)
    monkeypatch.setattr(api, "_launch", launch)


class Arena:
    """One allocation, from which overlapping arrays are cut."""

    def __init__(self):
        self.b = torch.zeros(1 << 20, dtype=torch.uint8)

    def cut(self, at, dtype, *shape):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        return self.b[at:at + n].view(dtype).view(shape)


def forms():
    """name, call(counts, seg_indptr, status, **outputs), {output: (dtype, shape)}"""
    x, w = torch.zeros(T, K, dtype=BF), torch.zeros(L, N, K, dtype=BF)
    dy, dh = torch.zeros(T, N, dtype=BF), torch.zeros(T, N // 2, dtype=BF)
    q, s = torch.zeros(T, K, dtype=torch.uint8), torch.ones(T, 1)
    wq, ws = torch.zeros(L, N, K, dtype=torch.uint8), torch.ones(L, 2, 1)
    u8 = torch.uint8
    return [
        ("bf16", lambda c, g, st, **o: cdl.grouped_bf16(x, w, c, g, status=st, **o), dict(out=(BF, (T, N)))),
        ("swiglu", lambda c, g, st, **o: cdl.grouped_swiglu_bf16(x, w, c, g, status=st, **o), dict(out=(BF, (T, N // 2)))),
        ("swiglu_grad", lambda c, g, st, **o: cdl.grouped_swiglu_bf16_grad(x, w, dh, c, g, status=st, **o),
         dict(out=(BF, (T, N)))),
        ("dx", lambda c, g, st, **o: cdl.grouped_bf16_dx(dy, w, c, g, status=st, **o), dict(out=(BF, (T, K)))),
        ("dw", lambda c, g, st, **o: cdl.grouped_bf16_dw(dy, x, c, g, status=st, **o), dict(out=(BF, (L, N, K)))),
        ("fp8", lambda c, g, st, **o: cdl.grouped_fp8(q, s, wq, ws, c, g, status=st, **o), dict(out=(BF, (T, N)))),
        ("swiglu_fp8", lambda c, g, st, **o: cdl.grouped_swiglu_fp8(q, s, wq, ws, c, g, status=st, **o),
         dict(out_q=(u8, (T, N // 2)), out_scales=(torch.float32, (T, 1)))),
    ]


NAMES = [f[0] for f in forms()]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_over_counts_segments_or_status(host, name):
    """The kernels read counts and seg_indptr again while others already store results."""
    _, call, outs = forms()[NAMES.index(name)]
    arena = Arena()
    counts, seg, status = torch.zeros(L, dtype=torch.int32), torch.zeros(L + 1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(Launched):
        call(counts, seg, status, **{k: arena.cut(1 << 19 if k == "out_scales" else 0, v[0], *v[1]) for k, v in outs.items()})
    for k, (dtype, shape) in outs.items():
        out = arena.cut(0, dtype, *shape)
        last = out.numel() * out.element_size()
        for at in (0, (last - 8) // 8 * 8):
            with pytest.raises(ValueError, match="%s overlaps counts" % k):
                call(arena.cut(at, torch.int32, L), seg, None, **{k: out})
            with pytest.raises(ValueError, match="%s overlaps seg_indptr" % k):
                call(counts, arena.cut(at, torch.int64, L + 1), None, **{k: out})
            with pytest.raises(ValueError, match="%s overlaps status" % k):
                call(counts, seg, arena.cut(at, torch.int32, 1), **{k: out})
        with pytest.raises(Launched):                        # right behind it is no overlap
            call(arena.cut((last + 7) // 8 * 8, torch.int32, L), seg, None, **{k: out})
    both = arena.cut(0, torch.int32, L)
    with pytest.raises(ValueError, match="status overlaps counts"):
        call(both, seg, both[1:])


def differentiable():
    """name, call(*operands), shapes of the operands"""
    c, g = torch.zeros(L, dtype=torch.int32), torch.zeros(L + 1, dtype=torch.int64)
    x, w, dy, dh, row = (T, K), (L, N, K), (T, N), (T, N // 2), (K,)
    return [
        ("grouped_bf16", lambda x, w: cdl.grouped_bf16(x, w, c, g), (x, w)),
        ("grouped_swiglu_bf16", lambda x, w: cdl.grouped_swiglu_bf16(x, w, c, g), (x, w)),
        ("grouped_swiglu_bf16_grad", lambda x, w, dh: cdl.grouped_swiglu_bf16_grad(x, w, dh, c, g), (x, w, dh)),
        ("grouped_bf16_dx", lambda dy, w: cdl.grouped_bf16_dx(dy, w, c, g), (dy, w)),
        ("grouped_bf16_dw", lambda dy, x: cdl.grouped_bf16_dw(dy, x, c, g), (dy, x)),
        ("rms_norm", cdl.rms_norm, (x, row, x)),
        ("rms_norm_fp8", cdl.rms_norm_fp8, (x, row, x)),
        ("rms_norm_grad", lambda dy, h, w, d: cdl.rms_norm_grad(dy, h, w, 1e-6, d), (x, x, row, x)),
    ]


@pytest.mark.parametrize("name,call,shapes", differentiable())
def test_tensors_that_require_a_gradient(host, name, call, shapes):
    """They would get a result without one, silently."""
    for which in range(len(shapes)):
        args = [torch.zeros(s, dtype=BF) for s in shapes]
        with pytest.raises(Launched, match=name):
            call(*args)
        args[which].requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call(*args)
        with torch.no_grad(), pytest.raises(Launched, match=name):
            call(*args)

        class Inside(torch.autograd.Function):               # no gradient is recorded within
            @staticmethod
            def forward(ctx, *a):
                return call(*a)

        with pytest.raises(Launched, match=name):
            Inside.apply(*args)


def test_weights_that_require_a_gradient_can_be_quantised(host):
    with pytest.raises(Launched):
        cdl.quant_fp8_blocks(torch.zeros(L, N, K, dtype=BF, requires_grad=True))
