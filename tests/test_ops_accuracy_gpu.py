"""GPU tests of the companion operators' accuracy where sums cancel or digits can get
lost, against the fp64 references in ops_oracle.py.

Tolerances.  fp32: 2^-19 of a head's norm.  A result passes through at most about a
thousand roundings of 2^-24 (a score's 64 or 128, a chunk's 64 tokens, the state's 64
of every chunk that its decay still reaches), which are independent: 2^-24 sqrt(1000) =
2^-19.  dlog_alpha adds to each chunk's state terms the rounding of those behind it, one
chunk's 2^-19 each, up to 16 of them between two cuts of a sequence: 2^-19 sqrt(16) = 8e-6,
so 1e-5 as in test_ops_gpu.py.  bf16: 8e-3 as there.
"""
import math

import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc
from test_ops_gpu import DT, TOL, gen, ssm_args, ssm_case, ssm_ref_args, up

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


# ---------------------------------------------------------- dlog_alpha
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,T,dk,dv", [(1, 2, 1, 330, 64, 64), (1, 3, 3, 200, 128, 64), (2, 5, 1, 130, 64, 128),
                                         (1, 9, 1, 150, 128, 128)])
def test_a_resets_gradient_is_zero(B, H, G, T, dk, dv, dt):
    """A decay of exactly zero stays so under any small change of log_alpha.  Resets at the edges of
    16-token blocks, chunks and segments, two in a row, at the first and last token."""
    c = ssm_case(B, H, G, T, dk, dv, dt, seed=50 + T)
    at = [0, 5, 15, 16, 63, 64, 65, 100, 127, 128, T - 1]
    c["log_alpha"][:, 0, at] = -math.inf
    c["log_alpha"][:, H - 1, at[::2]] = -math.inf
    args, t = ssm_args(c, True, True, True)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"])
    la = got["dlog_alpha"].float().cpu()
    assert (la[c["log_alpha"] == -math.inf] == 0).all()
    for n in ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0", "dD"):
        assert orc.rel(got[n], ref[n]) <= (1e-5 if n == "dS0" else TOL[dt]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [10.0, 25.0, 40.0])
def test_gradient_of_decays_that_leave_little(rate, dt):
    """dlog_alpha is as small as the decay itself, and right to its own digits."""
    H, T = 3, 330
    c = ssm_case(1, H, 1, T, 64, 64, dt, seed=60)
    g = torch.rand(1, H, T, generator=gen(61)) * 0.2 + 0.9
    c["log_alpha"] = (-rate * g).to(DT[dt])
    args, t = ssm_args(c, True, True, True)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"])
    for h in range(H):
        e = orc.rel(got["dlog_alpha"][:, h], ref["dlog_alpha"][:, h])
        end = orc.rel(got["dlog_alpha"][:, h, 320:], ref["dlog_alpha"][:, h, 320:])  # in front of a large dS_T
        print(f"    head {h} {e:.2e} {end:.2e}", flush=True)
        assert max(e, end) <= TOL[dt]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 40, 64])
@pytest.mark.parametrize("rate", [0.1, 5.0, 9.0, 14.0])
def test_gradient_of_decays_in_one_chunk(rate, T, dt):
    """Between a start state and a gradient of the end state that are both larger than what the
    decays leave of them."""
    H = 8
    c = ssm_case(1, H, H, T, 64, 64, dt, seed=65)
    c["log_alpha"] = (-rate * (0.9 + 0.2 * torch.rand(1, H, T, generator=gen(66)))).to(DT[dt])
    args, t = ssm_args(c, True, True, True)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"])
    e = orc.rel(got["dlog_alpha"], ref["dlog_alpha"])
    print(f"    {e:.2e}", flush=True)
    assert e <= TOL[dt]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_of_decays_over_a_long_sequence(dt):
    """Enough heads to fill the device, so that few cuts or none help: the gradient of the decays stays
    exact over all of the sequence, for heads that keep much and little."""
    H, T = 512, 8192
    assert kda.ssm_prefill_workspace_bytes(1, H, H, T, 64, 64, DT[dt]) == 0
    rates = (3.2, 1.0, 0.3, 0.05, 0.001)
    n = len(rates)
    heads = [0, 101, 202, 303, 511]
    few = ssm_case(1, n, n, T, 64, 64, dt, seed=71)
    g = gen(70)
    for i, r in enumerate(rates):
        few["log_alpha"][0, i] = (-r * (0.8 + 0.4 * torch.rand(T, generator=g))).to(DT[dt])
    t = {}
    for name, x in few.items():
        d = 0 if name == "D" else 1
        t[name] = up(x).index_select(d, torch.arange(H, device="cuda") % n)
        t[name].index_copy_(d, torch.tensor(heads, device="cuda"), up(x))
    got = kda.ssm_backward(t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], t["D"], t["S0"], t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(few, True, True), few["dO"], few["dS_T"])
    for i, h in enumerate(heads):
        for name in ("dlog_alpha", "dbeta", "dv", "dq", "dk"):
            e = orc.rel(got[name][:, h], ref[name][:, i])
            first = orc.rel(got[name][:, h, :T // 8], ref[name][:, i, :T // 8])
            print(f"    rate {rates[i]} {name} {e:.2e} {first:.2e}", flush=True)
            assert max(e, first) <= TOL[dt], (name, rates[i])


# ------------------------------------------------------------------- SiLU
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_silu_far_from_zero(dt):
    """SiLU and its derivative, element by element, where the exponential is large or small.  fp32: one
    rounding each of the exponential (2^-23, the hardware's), its correction, the sum, the
    reciprocal (2^-23) and the product, under 2^-21 together, and in the derivative of each
    term.  bf16: the output's 2^-8, and the exponent's own rounding, 87 * 2^-24 of the value."""
    T = 4096
    x = torch.linspace(-87, 87, T * 8, dtype=torch.float64).reshape(1, 1, T, 8).to(DT[dt])
    w = torch.tensor([0.0, 1.0]).expand(1, 8, 2).contiguous().to(DT[dt])
    dO = torch.ones(1, 1, T, 8, dtype=DT[dt])
    o, _ = kda.conv_prefill(up(x), up(w))
    s = kda.conv_step(up(x[:, 0].transpose(0, 1).contiguous()), torch.zeros(T, 1, 1, 8, dtype=DT[dt], device="cuda"), up(w))
    g = kda.conv_backward(up(x), up(w), None, None, up(dO))["dx"]
    torch.cuda.synchronize()
    xd = x.double()
    sig = 1 / (1 + torch.exp(-xd))
    tol = 2.0 ** -21 if dt == "f32" else 2.0 ** -8 + 2.0 ** -16
    assert ((o.cpu().double() - xd * sig).abs() <= tol * (xd * sig).abs()).all()
    assert torch.equal(s[:, 0], o[0, 0])
    assert ((g.cpu().double() - (sig + xd * sig * (1 - sig))).abs() <= tol * sig * (1 + xd.abs())).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", [None, "silu"])
def test_not_finite_rows_stay_in_their_window(act, dt):
    """An infinity or NaN in a valid row is in the outputs of its K tokens and channel, as from the
    formula, and in no other."""
    K, T = 4, 150
    x = torch.randn(1, 2, T, 8, generator=gen(80)).to(DT[dt])
    w = torch.rand(2, 8, K, generator=gen(81)).add(0.5).to(DT[dt])
    clean, _ = kda.conv_prefill(up(x), up(w), activation=act)
    bad = x.clone()
    for c, v in enumerate((math.inf, -math.inf, math.nan)):
        bad[0, 1, 70, c] = v
    o, st = kda.conv_prefill(up(bad), up(w), activation=act)
    torch.cuda.synchronize()
    o, clean = o.cpu().float(), clean.cpu().float()
    hit = torch.zeros(1, 2, T, 8, dtype=torch.bool)
    hit[0, 1, 70:70 + K, :3] = True
    assert torch.equal(o[~hit], clean[~hit])
    low = -math.inf if act is None else math.nan  # -inf * 0
    for c, v in enumerate((math.inf, low, math.nan)):
        y = o[0, 1, 70:70 + K, c]
        assert torch.isnan(y).all() if math.isnan(v) else (y == v).all()


# ------------------------------------------------------------- state cache
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_state_cache_loses_no_more_than_stated(fmt):
    """Values from a block's largest down to 2^-30 of it: off by 2^(p-1) (int8) or the larger of 2^-4 of
    themselves and 2^(p-10) (e4m3, whose subnormals share one step of 2^-9); the smallest are zero."""
    g = gen(90)
    S = torch.randn(2, 3, 64, 64, generator=g) * torch.exp2(-30 * torch.rand(2, 3, 64, 64, generator=g))
    S = S * torch.exp2(torch.randint(-60, 60, (2, 3, 64, 1), generator=g).float())
    cache, scales = kda.state_cache(2, 3, 64, 64, fmt, "cuda")
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    kda.state_store(up(S), slots, cache, scales)
    back = kda.state_load(cache, scales, slots)
    torch.cuda.synchronize()
    p, _ = orc.quantise(S, 127.0 if fmt == "int8" else 448.0)
    unit = torch.exp2(p).repeat_interleave(32, -1)
    x, off = S.double(), (back.cpu().double() - S.double()).abs()
    bound = unit / 2 if fmt == "int8" else torch.maximum(x.abs() / 16, unit / 1024)
    assert (off <= bound).all()
    least = unit / 2 if fmt == "int8" else unit / 1024
    assert (back.cpu()[x.abs() < least] == 0).all() and (off > x.abs() / 16).any()


# ------------------------------------------------------- one head, many segments
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_head_in_many_segments(dt):
    """A single head of 16384 tokens is cut into as many segments as the device has room for (64 or
    128 tokens each): decays that reach over many of them, results and gradients."""
    T = 16384
    assert kda.ssm_prefill_workspace_bytes(1, 1, 1, T, 64, 64, DT[dt]) >= 100 * 64 * 64 * 4
    c = ssm_case(1, 1, 1, T, 64, 64, dt, seed=95, slow=0.02)
    args, t = ssm_args(c, True, True, True)
    o, S = kda.ssm_prefill(*args)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    assert orc.rel(o, ro) <= TOL[dt] and orc.rel(S, rS) <= 1e-5
    ref = orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"])
    for n, x in got.items():
        if n == "dD":
            continue
        e = orc.rel(x, ref[n])
        print(f"    {n} {e:.2e}", flush=True)
        assert e <= (1e-5 if n == "dS0" else TOL[dt]), n
    # dD is one sum of 2^20 products of both signs, which may leave any part of them.  Each is in its
    # own rounding and in those of at most 127 sums on its way (8 in a lane, 3 of lanes, 2 tokens of a
    # thread, 8 of a block, 64 segments of a wave, 2 at the end); the sums of one level are of
    # disjoint products, so their roundings are at most 2^-24 of the products' root sum of
    # squares a level where the signs are independent: 2^-17 of it together.
    norm = float((c["dO"].double() * c["v"].double()).norm())
    off = abs(float(got["dD"]) - float(ref["dD"]))
    print(f"    dD off {off:.2e} of {float(ref['dD']):.2e}, products {norm:.2e}", flush=True)
    assert off <= 2.0 ** -17 * norm + (2.0 ** -8 * abs(float(ref["dD"])) if dt == "bf16" else 0)
