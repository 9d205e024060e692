"""GPU tests of the expert operators at values and sizes that their random
cases do not reach."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
import experts_check as C
from gpu_util import DEV, announce, status_word
from test_experts_gpu import gen, layer_inputs, mx_random, run_layer

pytestmark = pytest.mark.gpu


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
