"""The random cases of test_experts_gpu.py with the comparisons of
experts_check.py, which a NaN in an output fails."""
import pytest

import experts_check as C
import test_experts_gpu as cases

pytestmark = pytest.mark.gpu


def check_layer(kind, x, ids, wts, w13, w2, b, **kw):
    out, v13, v2 = cases.run_layer(kind, x, ids, wts, w13, w2, b, **kw)
    C.check_layer_output(out, x, ids, wts, v13, v2, b)
    return out


@pytest.fixture(autouse=True)
def only_numbers(monkeypatch):
    monkeypatch.setattr(cases, "check_grouped", C.check_grouped)
    monkeypatch.setattr(cases, "check_swiglu", C.check_swiglu)
    monkeypatch.setattr(cases, "check_layer", check_layer)


test_grouped = cases.test_grouped
test_grouped_scales_at_any_byte = cases.test_grouped_scales_at_any_byte
test_grouped_many_experts = cases.test_grouped_many_experts
test_grouped_counts_beyond_the_buffer_are_cut = cases.test_grouped_counts_beyond_the_buffer_are_cut
test_grouped_swiglu = cases.test_grouped_swiglu
test_layer = cases.test_layer
test_layer_bf16_rows_of_eight = cases.test_layer_bf16_rows_of_eight
test_layer_routing_edges = cases.test_layer_routing_edges
test_layer_int64_ids_and_reused_workspace = cases.test_layer_int64_ids_and_reused_workspace
test_expert_step = cases.test_expert_step
