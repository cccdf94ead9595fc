"""What the Python binding of the operators around the finalize refuses on a GPU: arguments that are missing."""
import dataclasses

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    return m


@pytest.mark.parametrize("field", ["expert_ids", "expert_scale", "perm_idx", "row_route", "expert_counts"])
@pytest.mark.parametrize("value", [None, [1, 2], "numpy"])
def test_route_refuses_outputs_that_are_missing_or_no_tensors(mfr, field, value):
    x = torch.randn(8, 32).cuda()
    good = mfr.moe_route(x, 2)
    want = good.perm_idx.clone()
    bad = dataclasses.replace(good, **{field: good.perm_idx.cpu().numpy() if value == "numpy" else value})
    with pytest.raises(ValueError):
        mfr.moe_route(-x, 2, out=bad)
    assert torch.equal(good.perm_idx, want)


def test_route_takes_outputs_without_an_order(mfr):
    x = torch.randn(8, 32).cuda()
    good = mfr.moe_route(x, 2)
    out = mfr.Routing(torch.empty_like(good.expert_ids), torch.empty_like(good.expert_scale))
    assert mfr.moe_route(x, 2, out=out) is out and torch.equal(out.expert_ids, good.expert_ids)


def test_calls_refuse_a_routing_without_an_order(mfr):
    x = torch.randn(8, 32).bfloat16().cuda()
    r = mfr.moe_route(x, 2, order=False)
    with pytest.raises(ValueError):
        mfr.moe_dispatch(x, r.perm_idx, 16)
    with pytest.raises(ValueError):
        mfr.moe_finalize_routed_backward(x, mfr.Partial(x, r.perm_idx, r.expert_scale))
    with pytest.raises(ValueError):
        mfr.moe_route_backward(None, x, r.expert_ids)


@pytest.mark.parametrize("dtype", [torch.float64, torch.int32])
def test_calls_refuse_scales_of_another_type(mfr, dtype):
    x = torch.randn(8, 32).bfloat16().cuda()
    r = mfr.moe_route(x, 2)
    with pytest.raises(ValueError):
        mfr.moe_route(x, 2, out=dataclasses.replace(r, expert_scale=r.expert_scale.to(dtype)))
    with pytest.raises(ValueError):
        mfr.moe_route_backward(r.expert_scale.to(dtype), x, r.expert_ids)
    with pytest.raises(ValueError):
        mfr.moe_finalize_routed_backward(x, mfr.Partial(x, torch.zeros_like(r.perm_idx), r.expert_scale.to(dtype)))
