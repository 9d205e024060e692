"""GPU tests of the expert operators at values and sizes that their random
cases do not reach."""
import pytest
import torch

import combine_dispatch_layout_amd as cdl
from gpu_util import DEV, announce
from test_experts_gpu import layer_inputs

pytestmark = pytest.mark.gpu


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
