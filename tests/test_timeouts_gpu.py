"""The finalize's count of waits that ran out, of calls on other streams."""
import pytest
import torch

import synth
from helpers import partials_of

pytestmark = pytest.mark.gpu


def test_a_wait_that_runs_out_on_another_stream_is_counted():
    """The count waits for every stream of the device: the call may still be running."""
    import moe_finalize_residual_gb300 as mfr
    g = synth.make_case("timeout-stream", T=4, H=1024, K=8, R=2, E=64, rsf=2.5, shared=True).to("cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert mfr.moe_finalize_read_timeouts() == 0
    out = mfr.moe_finalize_fused(partials_of(g), g.residual, g.gamma, kernel="stream", stream=side, extra_flags=mfr.MFR_FLAG_TEST_STREAM_TIMEOUT)
    first = mfr.moe_finalize_read_timeouts()
    torch.cuda.synchronize()
    again = mfr.moe_finalize_read_timeouts()
    assert first > 0 and again == 0 and out is not None
