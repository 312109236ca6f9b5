"""GPU tests of the companion operators' accuracy where sums cancel or digits can get
lost, against the fp64 references in ops_oracle.py.

Tolerances.  fp32: 2^-19 of a head's norm.  A result passes through at most about a
thousand roundings of 2^-24 (a score's 64 or 128, a chunk's 64 tokens, the state's 64
of every chunk that its decay still reaches), which are independent: 2^-24 sqrt(1000) =
2^-19.  bf16: 8e-3 as in test_ops_gpu.py.
"""
import math

import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc
from test_ops_gpu import TOL, gen, ssm_args, ssm_case, ssm_ref_args

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -19


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


# ------------------------------------------- slow decays behind strong ones
def behind_strong(H, T, per_block, strong, seed):
    """fp32 inputs with slow decays and per_block strong ones in every 16 tokens, at a random place in
    each of the 16 / per_block parts; and which tokens lie behind one in their 16 tokens."""
    c = ssm_case(1, H, 1, T, 64, 64, "f32", seed=seed, slow=0.1)
    part = 16 // per_block
    at = torch.arange(0, T, part) + torch.randint(0, part, (H, -(-T // part)), generator=gen(seed))
    behind = torch.zeros(H, T, dtype=torch.bool)
    for h in range(H):
        a = at[h][at[h] < T]
        c["log_alpha"][0, h, a] = strong
        mark = torch.zeros(T, dtype=torch.long)
        mark[a] = 1
        blocks = torch.nn.functional.pad(mark, (0, -T % 16)).view(-1, 16).cumsum(1).flatten()[:T]
        behind[h] = blocks > 0
    return c, behind


def rel_at(x, ref, on):
    """Relative distance of [1, H, T, ...] over the tokens on [H, T]."""
    x, ref = x.double().cpu()[0][on], ref.double()[0][on]
    return float((x - ref).norm() / ref.norm())


@pytest.mark.parametrize("strong", [-math.inf, -100.0, -40.0, -9.0])
@pytest.mark.parametrize("per_block", [1, 4, 8])
def test_slow_decays_behind_strong_ones(per_block, strong):
    """Short documents packed into one sequence: the tokens behind a reset keep all digits."""
    H, T = 3, 700
    c, on = behind_strong(H, T, per_block, strong, seed=40 + per_block)
    args, t = ssm_args(c, False, True, False)
    ro, rS = orc.ssm(*ssm_ref_args(c, False, True))
    for ws in ("auto", None):
        o, S = kda.ssm_prefill(*args, workspace=ws)
        torch.cuda.synchronize()
        e = rel_at(o, ro, on)
        print(f"    o {e:.2e} S {orc.rel(S, rS):.2e}", flush=True)
        assert e <= F32 and orc.rel(S, rS) <= F32
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(c, False, True), c["dO"], c["dS_T"])
    for n in ("dv", "dbeta"):
        e = rel_at(got[n], ref[n], on)
        print(f"    {n} {e:.2e}", flush=True)
        assert e <= F32, n
    for n in ("dq", "dk", "dS0"):
        assert orc.rel(got[n], ref[n]) <= F32, n
