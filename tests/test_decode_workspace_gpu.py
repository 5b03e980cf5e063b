"""Decodes of changing batch sizes share the binding's workspace.

The counters at its front have to be zero for every call, whatever an earlier
call with fewer sequences left behind them as partials.
"""

import pytest
import torch

from parallax_local_linear_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_larger_batch_after_a_smaller_one(px, dtype):
    def inputs(batch, length):
        x = W.small_decode_inputs(batch, 4, 2, 64, length, dtype=dtype, seed=batch)
        return {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in x.items()}

    small, large = inputs(1, 8192), inputs(400, 200)

    def run(x):
        return px.decode(x["q"], x["rho"], x["k_cache"], x["v_cache"], x["scale"], out_dtype=torch.float32,
                         out=torch.full(x["q"].shape, float("nan"), device="cuda"), num_ctas=97)

    plan_out = torch.empty(large["q"].shape, device="cuda")
    want = px.DecodePlan(large["q"], large["rho"], large["k_cache"], large["v_cache"], large["scale"], out=plan_out,
                         num_ctas=97).run().clone()     # (a plan has a workspace of its own)
    for _ in range(3):
        run(small)
        assert torch.equal(run(large), want)
    assert px.last_device_error() == 0
