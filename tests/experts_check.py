"""Comparisons of the expert operators' outputs with their 64-bit forms
(experts_ref.py) that hold only for numbers: a NaN is outside every bound."""
import torch

import experts_ref as R


def assert_within(out, want, bound, what=""):
    """|out - want| <= bound, element by element."""
    ok = (out.double() - want).abs() <= bound
    assert bool(ok.all()), (what, int((~ok).sum()), "of", ok.numel())


def check_grouped(a, sa, w, sw, counts, begins, out, canary_rows):
    """out (2-D rows) against the product of every expert's rows; all other
    rows hold the canary."""
    live = torch.zeros(out.shape[0], dtype=torch.bool, device=out.device)
    for e, c in enumerate(counts):
        at = slice(begins[e], begins[e] + c)
        live[at] = True
        if c:
            y, err = R.product(R.values(a[at], sa[at]), R.values(w[e], sw[e]))
            assert_within(out[at], y, err + R.BF16 * (y.abs() + err) + R.TINY, e)
    rest = out[~live]
    assert torch.equal(rest.view(torch.int16), canary_rows.expand_as(rest).view(torch.int16))


def check_swiglu(a, sa, w, sw, q, s, I):
    """Rows (q, s) against the SwiGLU of the gate/up product: the scale is the
    definition's and every value a nearest grid point for some h in the bound."""
    gu, d = R.product(R.values(a, sa), R.values(w, sw))
    h, dh = R.swiglu(gu[:, :I], d[:, :I], gu[:, I:], d[:, I:])
    hb, db = h.unflatten(-1, (-1, 32)), dh.unflatten(-1, (-1, 32))
    lo, hi = (hb.abs() - db).amax(-1), (hb.abs() + db).amax(-1)
    assert bool((s != 255).all())
    p = torch.exp2(s.double() - 127)
    assert bool((6 * p >= lo).all())
    assert bool(((s == 0) | (3 * p < hi)).all())
    v = R.values(q, s).unflatten(-1, (-1, 32))
    t = (hb.abs() + db) / p.unsqueeze(-1)
    half = torch.where(t < 2, 0.25, torch.where(t < 4, 0.5, 1.0)) * p.unsqueeze(-1)
    assert_within(v, hb, half + db)


def check_layer_output(out, x, ids, wts, v13, v2, b):
    want, bound = R.layer(x.double(), ids, wts, v13, v2, b)
    assert_within(out, want, bound)
