"""The bounded waits of the weight gradient's kernel give up on barriers that nothing completes, at their limit,
and the plan, the context and the weight gradient stay usable."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import gradient_quantization_communication_b200.gq as G


@pytest.mark.parametrize("limit_ms", [1, 20])
def test_waits_run_out_at_their_limit(limit_ms):
    x = torch.randn(300, 520, device="cuda").bfloat16()
    ck = torch.zeros(G.gq_act_layout(300, 520)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x, ck)
    before, after = torch.empty(520, 520, device="cuda"), torch.empty(520, 520, device="cuda")
    G.gq_act_weight_grad(ck, x, before)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with G.Plan(G.gq_config("orq", 5, 512, 1, False, 0.0, 1, 1024)) as plan:
        torch.cuda.synchronize()
        a.record()
        G.gq_selftest_bounded_wait(plan.handle, limit_ms * 1_000_000)
        b.record()
        assert G.gq_plan_status(plan.handle) == G.GQ_ERR_TIMEOUT   # raised only if every kind of wait gave up
        # twice the limit in cycles: at least the limit at 2 GHz, and not ten times it
        assert 0.9 * limit_ms <= a.elapsed_time(b) <= 10 * limit_ms + 5
        assert G.gq_plan_status(plan.handle) == G.GQ_OK
    G.gq_act_weight_grad(ck, x, after)
    assert torch.equal(before, after)
