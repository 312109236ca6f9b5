"""GPU tests of the companion operators' results where a gate or a sum could get lost,
against the fp64 references in ops_oracle.py.  Tolerances are those of test_ops_gpu.py."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc
from test_ops_gpu import TOL, ssm_args, ssm_case, ssm_ref_args

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- gates of NaN
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 70, 700])
def test_nan_gate_reaches_the_start_states_gradient(T, dt):
    """The first token's decay multiplies the start state: its NaN is in dS0, in one piece and in
    segments, and in no other head."""
    c = ssm_case(1, 2, 2, T, 64, 64, dt, seed=31)
    c["log_alpha"][0, 1, 0] = float("nan")
    args, t = ssm_args(c, True, True, False)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    assert torch.isnan(got["dS0"][0, 1]).all()
    ref = orc.ssm_backward(*ssm_ref_args({n: x[:, :1] if n != "D" else x[:1] for n, x in c.items()}, True, True),
                           c["dO"][:, :1], c["dS_T"][:, :1])
    for n in ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0"):
        assert orc.rel(got[n][:, :1], ref[n]) <= (1e-5 if n == "dS0" else TOL[dt]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("at", [63, 64, 128, 200])
def test_nan_gate_reaches_the_gradients_before_it(at, dt):
    """Every token before a NaN decay gets a NaN gradient, across the cuts of the sequence too."""
    c = ssm_case(1, 1, 1, 330, 64, 64, dt, seed=32)
    c["log_alpha"][0, 0, at] = float("nan")
    args, t = ssm_args(c, True, True, False)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    assert torch.isnan(got["dlog_alpha"][0, 0, :at + 1]).all()
    assert torch.isnan(got["dv"][0, 0, :at]).all() and torch.isnan(got["dbeta"][0, 0, :at]).all()
