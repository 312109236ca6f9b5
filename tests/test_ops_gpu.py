"""GPU tests of the short convolution, the selective scan and the quantised state
cache against the fp64 references in ops_oracle.py.

Tolerances.  bf16 results carry their own rounding (half a step, 2^-8 of the
value) and, in the scan, one rounding of a score or state (2^-8) in front of an
fp32 sum: at most 2 * 2^-8 = 7.9e-3 of the result where terms do not cancel; the
bound is on norms, where rounding errors of many terms average.  Convolutions
round once, element by element.  fp32 results accumulate a few hundred roundings
of 2^-24, 1e-5 with room for cancellation; fp32 states of bf16 inputs take
operands to 24 bits and get the same bound.  A scalar gradient that sums tokens
with cancellation (dlog_alpha) has the bf16 rounding and the same 2^-8.
"""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 8e-3, "f32": 1e-5}


def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def tm(x):
    """The same values in token-major memory order."""
    return x.transpose(1, 2).contiguous().transpose(1, 2)


def up(t):
    return None if t is None else t.to(dev())


# ------------------------------------------------------------- convolution
def conv_case(B, H, T, d, K, dt, bias, state, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    return dict(x=r(B, H, T, d), weight=r(H, d, K), bias=r(H, d) if bias else None,
                state=r(B, H, K - 1, d) if state else None, dO=r(B, H, T, d), dstate_out=r(B, H, K - 1, d))


CONV = [  # B, H, T, d, K, dtype, activation, bias, state, token-major
    (2, 3, 37, 16, 4, "bf16", True, True, True, True),
    (1, 1, 1, 8, 4, "bf16", True, False, True, False),
    (3, 2, 2, 8, 4, "bf16", False, True, False, True),
    (1, 5, 130, 32, 3, "f32", True, True, False, True),
    (2, 2, 64, 4, 2, "f32", False, False, True, False),
    (2, 1, 701, 72, 2, "bf16", True, True, True, True),
    (1, 4, 9, 128, 3, "f32", False, True, True, True),
]


def conv_tol(dt, ref, scale):
    """Elementwise: the output's rounding, and fp32 roundings of the terms' absolute sum."""
    return (2.0 ** -8 if dt == "bf16" else 0.0) * ref.abs() + 2.0 ** -20 * scale + 1e-30


@pytest.mark.parametrize("B,H,T,d,K,dt,act,bias,state,major", CONV)
def test_conv_prefill(B, H, T, d, K, dt, act, bias, state, major):
    print(f"[case] conv_prefill {B} {H} {T} {d} K={K} {dt}", flush=True)
    c = conv_case(B, H, T, d, K, dt, bias, state, seed=T + K)
    ref, st = orc.conv(c["x"], c["weight"], c["bias"], c["state"], act)
    scale, _ = orc.conv(c["x"].abs(), c["weight"].abs(), None if not bias else c["bias"].abs(),
                        None if not state else c["state"].abs(), False)
    x = up(c["x"])
    o, so = kda.conv_prefill(tm(x) if major else x, up(c["weight"]), up(c["bias"]), up(c["state"]),
                             activation="silu" if act else None)
    torch.cuda.synchronize()
    assert o.is_contiguous()
    assert ((o.cpu().double() - ref).abs() <= conv_tol(dt, ref, scale)).all()
    assert torch.equal(so.cpu().double(), st)


@pytest.mark.parametrize("lens", [[0, 5, 40], [40, 1, 2], [-3, 400, 39]])
def test_conv_prefill_lens(lens):
    """Rows behind a sequence's length stay as they were, and its state is the one there."""
    c = conv_case(3, 2, 40, 16, 4, "bf16", True, True, seed=5)
    ref, st = orc.conv(c["x"], c["weight"], c["bias"], c["state"], True, lens)
    x = tm(up(c["x"]))
    o = tm(torch.full((3, 2, 40, 16), 7.0, dtype=torch.bfloat16, device=dev()))
    _, so = kda.conv_prefill(x, up(c["weight"]), up(c["bias"]), up(c["state"]), o=o,
                             lens=torch.tensor(lens, dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    o = o.cpu().double()
    behind = torch.isnan(ref)
    assert (o[behind] == 7.0).all()
    assert orc.rel(o, ref) <= 2.0 ** -8
    assert torch.equal(so.cpu().double(), st)


@pytest.mark.parametrize("N,H,d,K,dt,act,bias", [(1, 1, 8, 2, "bf16", True, False), (7, 3, 40, 4, "bf16", True, True),
                                               (33, 2, 4, 3, "f32", False, True)])
def test_conv_step_follows_prefill(N, H, d, K, dt, act, bias):
    """Token by token from the state a prompt left gives the outputs of the longer prompt."""
    T0, T1 = 5, 4
    c = conv_case(N, H, T0 + T1, d, K, dt, bias, True, seed=9)
    a = "silu" if act else None
    x, w, b, st = up(c["x"]), up(c["weight"]), up(c["bias"]), up(c["state"])
    full, end = kda.conv_prefill(x, w, b, st, activation=a)
    _, s = kda.conv_prefill(x[:, :, :T0], w, b, st, activation=a)
    for t in range(T1):
        o = kda.conv_step(x[:, :, T0 + t], s, w, b, activation=a)
        torch.cuda.synchronize()
        ref = full[:, :, T0 + t].double()
        assert ((o.double() - ref).abs() <= 2 * conv_tol(dt, ref, 1 + ref.abs())).all()
    assert torch.equal(s, end)


@pytest.mark.parametrize("B,H,T,d,K,dt,act,bias,state,major", CONV)
def test_conv_backward(B, H, T, d, K, dt, act, bias, state, major):
    print(f"[case] conv_backward {B} {H} {T} {d} K={K} {dt}", flush=True)
    c = conv_case(B, H, T, d, K, dt, bias, state, seed=T + 2 * K)
    ref = orc.conv_backward(c["x"], c["weight"], c["bias"], c["state"], c["dO"], c["dstate_out"], act)
    x, dO = up(c["x"]), up(c["dO"])
    if major:
        x, dO = tm(x), tm(dO)
    got = kda.conv_backward(x, up(c["weight"]), up(c["bias"]), up(c["state"]), dO, up(c["dstate_out"]),
                            activation="silu" if act else None)
    torch.cuda.synchronize()
    assert set(got) == {"dx", "dweight"} | ({"dbias"} if bias else set()) | ({"dstate"} if state else set())
    for n, t in got.items():
        assert t.dtype == DT[dt]
        assert orc.rel(t, ref[n]) <= (2.0 ** -8 if dt == "bf16" else 2e-6), n


# --------------------------------------------------------------------- scan
def ssm_case(B, H, G, T, dk, dv, dt, seed, slow=1.0):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    step = torch.exp(r(B, H, T) * 0.7 - 2.5) * slow
    rate = 1 + 7 * torch.rand(1, H, 1, generator=g)
    f = lambda t: t.to(DT[dt])  # noqa: E731
    return dict(q=f(r(B, G, T, dk) * dk ** -0.25), k=f(r(B, G, T, dk) * dk ** -0.25), v=f(r(B, H, T, dv)),
                log_alpha=f(-step * rate), beta=f(step), D=f(1 + 0.1 * r(H)), S0=0.3 * r(B, H, dk, dv),
                dO=f(r(B, H, T, dv)), dS_T=0.3 * r(B, H, dk, dv))


SSM = [  # B, H, G, T, dk, dv, dtype, skip, state, token-major
    (1, 1, 1, 1, 64, 64, "bf16", True, True, False),
    (2, 4, 2, 63, 128, 64, "bf16", True, True, True),
    (1, 3, 1, 65, 64, 64, "bf16", False, True, True),
    (1, 2, 1, 200, 128, 128, "bf16", True, False, True),
    (2, 5, 5, 130, 64, 128, "bf16", False, False, False),
    (1, 6, 2, 128, 128, 64, "f32", True, True, True),
    (2, 2, 2, 77, 64, 128, "f32", False, True, False),
    (1, 3, 3, 300, 128, 128, "f32", True, False, True),
    (1, 5, 1, 129, 64, 64, "f32", True, True, True),
]


def ssm_args(c, skip, state, major):
    t = {n: up(x) for n, x in c.items()}
    if major:
        for n in ("q", "k", "v", "dO", "log_alpha", "beta"):
            t[n] = tm(t[n])
    return (t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], t["D"] if skip else None, t["S0"] if state else None), t


def ssm_ref_args(c, skip, state):
    return (c["q"], c["k"], c["v"], c["log_alpha"], c["beta"], c["D"] if skip else None, c["S0"] if state else None)


@pytest.mark.parametrize("B,H,G,T,dk,dv,dt,skip,state,major", SSM)
def test_ssm_prefill(B, H, G, T, dk, dv, dt, skip, state, major):
    print(f"[case] ssm_prefill {B} {H}/{G} {T} {dk}x{dv} {dt}", flush=True)
    c = ssm_case(B, H, G, T, dk, dv, dt, seed=T)
    args, _ = ssm_args(c, skip, state, major)
    ro, rS = orc.ssm(*ssm_ref_args(c, skip, state))
    for ws in ("auto", None):  # cut into segments where that pays, and in one piece
        o, S = kda.ssm_prefill(*args, workspace=ws)
        torch.cuda.synchronize()
        assert orc.rel(o, ro) <= TOL[dt]
        assert orc.rel(S, rS) <= 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,T,dk,dv,slow", [(1, 2, 1, 1500, 128, 64, 1.0), (1, 1, 1, 2049, 64, 128, 0.02),
                                              (2, 3, 3, 1000, 64, 64, 0.02)])
def test_ssm_prefill_segments(B, H, G, T, dk, dv, slow, dt):
    """Few heads: the sequence is cut; with slow decay the states carry across the cuts.  The
    one-piece walk gives the same up to rounding, and S_T may be S0."""
    print(f"[case] ssm_prefill segments {B} {H}/{G} {T} {dk}x{dv} {dt}", flush=True)
    assert kda.ssm_prefill_workspace_bytes(B, H, G, T, dk, dv, DT[dt]) > 0
    c = ssm_case(B, H, G, T, dk, dv, dt, seed=T, slow=slow)
    args, t = ssm_args(c, True, True, True)
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    for ws in ("auto", None):
        o, S = kda.ssm_prefill(*args, workspace=ws)
        torch.cuda.synchronize()
        assert orc.rel(o, ro) <= TOL[dt]
        assert orc.rel(S, rS) <= 1e-5
    o1, S1 = kda.ssm_prefill(*args)
    o2, S2 = kda.ssm_prefill(*args[:6], t["S0"], S_T=t["S0"])
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(S1, S2)


@pytest.mark.parametrize("lens", [[0, 64, 300], [1, 65, 299], [-1, 1000, 128]])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ssm_prefill_lens(lens, dt):
    c = ssm_case(3, 2, 1, 300, 64, 64, dt, seed=8)
    args, _ = ssm_args(c, True, True, True)
    o = torch.full((3, 2, 300, 64), 7.0, dtype=DT[dt], device=dev())
    ln = torch.tensor(lens, dtype=torch.int32)
    _, S = kda.ssm_prefill(*args, lens=up(ln), o=o)
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True), lens=ln)
    assert (o.cpu()[torch.isnan(ro)] == 7.0).all()
    assert orc.rel(o, ro) <= TOL[dt]
    assert orc.rel(S, rS) <= 1e-5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ssm_resets_and_no_decay(dt):
    """log_alpha = -inf clears the state (no NaN from differences of infinite sums), also several
    times in a chunk; log_alpha = 0 keeps it; a token with beta = 0 adds nothing."""
    c = ssm_case(1, 2, 1, 260, 64, 64, dt, seed=4)
    for t in (0, 5, 6, 15, 16, 63, 64, 100, 255):
        c["log_alpha"][0, 0, t] = -float("inf")
    c["log_alpha"][0, 1] = 0.0
    c["beta"][0, 1, 30:90] = 0.0
    args, _ = ssm_args(c, True, True, False)
    o, S = kda.ssm_prefill(*args)
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    for h in range(2):
        assert orc.rel(o[:, h], ro[:, h]) <= TOL[dt]
        assert orc.rel(S[:, h], rS[:, h]) <= 1e-5


def test_ssm_nan_gate_is_not_hidden():
    c = ssm_case(1, 1, 1, 70, 64, 64, "bf16", seed=4)
    c["log_alpha"][0, 0, 3] = float("nan")
    args, _ = ssm_args(c, False, True, False)
    o, S = kda.ssm_prefill(*args)
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 3:].float()).all() and torch.isnan(S).all()


@pytest.mark.parametrize("N,H,G,dk,dv,dt,skip", [(1, 1, 1, 64, 64, "bf16", False), (5, 4, 2, 128, 64, "bf16", True),
                                               (3, 6, 1, 64, 128, "f32", True), (2, 3, 3, 128, 128, "bf16", True),
                                               (4, 2, 2, 128, 128, "f32", False)])
def test_ssm_step_follows_prefill(N, H, G, dk, dv, dt, skip):
    """Steps from a prompt's end state, against the reference over the longer sequence."""
    T0, T1 = 66, 3
    c = ssm_case(N, H, G, T0 + T1, dk, dv, dt, seed=N)
    ro, rS = orc.ssm(*ssm_ref_args(c, skip, True))
    args, t = ssm_args(c, skip, True, False)
    cut = [x[:, :, :T0] for x in args[:5]]
    _, S = kda.ssm_prefill(*cut, *args[5:])
    for i in range(T0, T0 + T1):
        q, k, v, la, b = (x[:, :, i].contiguous() for x in args[:5])
        o = kda.ssm_step(q, k, v, la, b, S, args[5])
        torch.cuda.synchronize()
        assert orc.rel(o, ro[:, :, i]) <= (2.0 ** -8 if dt == "bf16" else 1e-5)
    assert orc.rel(S, rS) <= 1e-5


def check_grads(got, ref, dt):
    for n, t in got.items():
        assert t.dtype == (torch.float32 if n == "dS0" else DT[dt]), n
        e = orc.rel(t, ref[n])
        print(f"    {n} {e:.2e}", flush=True)
        assert e <= (1e-5 if n == "dS0" else TOL[dt]), (n, e)


@pytest.mark.parametrize("B,H,G,T,dk,dv,dt,skip,state,major", SSM)
def test_ssm_backward(B, H, G, T, dk, dv, dt, skip, state, major):
    print(f"[case] ssm_backward {B} {H}/{G} {T} {dk}x{dv} {dt}", flush=True)
    c = ssm_case(B, H, G, T, dk, dv, dt, seed=T + 1)
    args, t = ssm_args(c, skip, state, major)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"] if state else None)
    torch.cuda.synchronize()
    ref = orc.ssm_backward(*ssm_ref_args(c, skip, state), c["dO"], c["dS_T"] if state else None)
    assert set(got) == {"dq", "dk", "dv", "dlog_alpha", "dbeta"} | ({"dD"} if skip else set()) | ({"dS0"} if state else set())
    check_grads(got, ref, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,T,dk,dv,slow", [(1, 2, 1, 600, 64, 64, 0.05), (1, 3, 1, 520, 128, 64, 1.0),
                                              (1, 2, 2, 513, 64, 128, 0.05)])
def test_ssm_backward_segments(B, H, G, T, dk, dv, slow, dt):
    print(f"[case] ssm_backward segments {B} {H}/{G} {T} {dk}x{dv} {dt}", flush=True)
    c = ssm_case(B, H, G, T, dk, dv, dt, seed=T + 1, slow=slow)
    args, t = ssm_args(c, True, True, True)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"]), dt)


def test_ssm_backward_against_differences():
    """fp32 gradients against central differences of the fp64 forward along random directions."""
    c = ssm_case(1, 2, 1, 70, 64, 64, "f32", seed=3)
    args, t = ssm_args(c, True, True, False)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    names = ("q", "k", "v", "log_alpha", "beta", "D", "S0")
    base = {n: c[n].double() for n in names}

    def loss(x):
        o, S = orc.ssm(*(x[n] for n in names))
        return float((o * c["dO"].double()).sum() + (S * c["dS_T"].double()).sum())

    g = gen(1)
    for n in names:
        u = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        h = 1e-6
        d = (loss({**base, n: base[n] + h * u}) - loss({**base, n: base[n] - h * u})) / (2 * h)
        m = float((got["d" + n].double().cpu() * u).sum())
        assert abs(m - d) <= 1e-4 * max(1.0, abs(d)), (n, m, d)


# -------------------------------------------------------------- state cache
def cache_values(cache):
    return cache.cpu().float().double()


def special_states(n, H, dk, dv, seed):
    g = gen(seed)
    S = torch.randn(n, H, dk, dv, generator=g) * torch.exp(3 * torch.randn(n, H, dk, 1, generator=g))
    S[0, 0, 0] = 0.0
    S[0, 0, 1, :32] = torch.tensor([127.0, 63.5, 0.5, 1.5, -127.0, -0.5] + [0.0] * 26)  # ties, exact ends
    S[0, 0, 2, :32] = torch.tensor([448.0, 17.0, 19.0, -448.0, 2.0 ** -10] + [0.0] * 27)
    S[0, 0, 3, :32] = 1e-42  # subnormal
    S[0, 0, 4, :32] = 3e38
    S[0, 0, 5, :32] = 127.00001
    return S


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,nslots,H,dk,dv", [(1, 1, 1, 8, 32), (5, 9, 3, 64, 64), (3, 4, 2, 128, 128), (4, 7, 1, 7, 96)])
def test_state_store_and_load(fmt, n, nslots, H, dk, dv):
    print(f"[case] state cache {n}/{nslots} {H} {dk}x{dv} {fmt}", flush=True)
    S = special_states(n, H, dk, dv, seed=n)
    cache, scales = kda.state_cache(nslots, H, dk, dv, fmt, dev())
    before = cache.view(torch.uint8).clone()
    slots = torch.randperm(nslots, generator=gen(2))[:n].to(torch.int32)
    kda.state_store(up(S), up(slots), cache, scales)
    torch.cuda.synchronize()
    p, y = orc.quantise(S, 127.0 if fmt == "int8" else 448.0)
    at = slots.long()
    assert torch.equal(scales.cpu()[at].double(), p + 127)
    ref = y.round() if fmt == "int8" else y.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(cache_values(cache)[at], ref)
    # entries that were not named are as they were
    other = [s for s in range(nslots) if s not in set(slots.tolist())]
    assert torch.equal(cache.view(torch.uint8)[other], before[other])
    back = kda.state_load(cache, scales, up(slots))
    torch.cuda.synchronize()
    exact = (ref.unflatten(-1, (-1, 32)) * torch.exp2(p)[..., None]).flatten(-2)
    assert torch.equal(back.cpu().double(), exact)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_state_slots_outside_and_repeated(fmt):
    """Outside slots are skipped and read as zero; the last of repeated slots is stored."""
    S = torch.randn(6, 2, 64, 64, generator=gen(3))
    cache, scales = kda.state_cache(4, 2, 64, 64, fmt, dev())
    slots = torch.tensor([2, -1, 4, 2, 0, 2], dtype=torch.int32)
    kda.state_store(up(S), up(slots), cache, scales)
    one, ones = kda.state_cache(4, 2, 64, 64, fmt, dev())
    kda.state_store(up(S[4:].contiguous()), up(slots[4:].contiguous()), one, ones)
    torch.cuda.synchronize()
    assert torch.equal(cache.view(torch.uint8), one.view(torch.uint8)) and torch.equal(scales, ones)
    back = kda.state_load(cache, scales, up(torch.tensor([0, -5, 2, 2, 4, 1 << 30], dtype=torch.int32)))
    torch.cuda.synchronize()
    assert (back[[1, 4, 5]] == 0).all()
    assert torch.equal(back[2], back[3]) and (back[2].abs().sum() > 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_state_not_finite_reads_nan(fmt):
    S = torch.ones(1, 1, 2, 64)
    S[0, 0, 0, 3], S[0, 0, 1, 40] = float("inf"), float("nan")
    cache, scales = kda.state_cache(1, 1, 2, 64, fmt, dev())
    z = torch.zeros(1, dtype=torch.int32, device=dev())
    kda.state_store(up(S), z, cache, scales)
    back = kda.state_load(cache, scales, z)
    torch.cuda.synchronize()
    b = back.cpu()[0, 0]
    assert torch.isnan(b[0, :32]).all() and (b[0, 32:] == 1).all()
    assert torch.isnan(b[1, 32:]).all() and (b[1, :32] == 1).all()


# ------------------------------------------------------------ used together
def test_layer_of_both_kinds():
    """A projection's token-major output through the convolution into a KDA prefill with
    snapshots and into the scan; the snapshots and the scan's state parked in the cache; and the
    rest of the prompt resumed from them token by token, against one uninterrupted run."""
    B, H, T, d, K, cut = 2, 2, 576, 64, 4, 512
    g = gen(21)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    proj = up(r(B, T, 3 * H * d).to(torch.bfloat16))
    w = up((r(3 * H, d, K) * 0.5).to(torch.bfloat16))
    la = up((-torch.sigmoid(r(B, H, T, d))).to(torch.bfloat16))
    beta = up(torch.sigmoid(r(B, H, T)).to(torch.bfloat16))
    step = up((0.05 * torch.rand(B, H, T, generator=g)).to(torch.bfloat16))
    decay = -step
    x = proj.view(B, T, 3 * H, d).transpose(1, 2)
    qkv, conv_state = kda.conv_prefill(x, w)
    q, k, v = (t.contiguous() for t in qkv.split(H, 1))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(torch.bfloat16) for t in (q, k))
    o, _, snaps = kda.prefill_snap(q, k, v, la, beta, cut)
    y, _ = kda.ssm_prefill(q, k, v, decay, step)
    cache, scales = kda.state_cache(8, H, d, d, "int8", dev())
    slots = torch.tensor([5, 1], dtype=torch.int32, device=dev())
    kda.state_store(snaps, slots, cache, scales)
    _, S_cut = kda.ssm_prefill(*(t[:, :, :cut] for t in (q, k, v, decay, step)))
    kda.state_store(S_cut, slots + 1, cache, scales)
    S1, S2 = kda.state_load(cache, scales, slots), kda.state_load(cache, scales, slots + 1)
    # int8 in blocks of 32: at most half a step of 2 / 127 of the block's largest value
    for got, ref in ((S1, snaps[:, 0]), (S2, S_cut)):
        m = ref.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True)
        assert ((got - ref).unflatten(-1, (-1, 32)).abs() <= m / 127).all()
    _, cs = kda.conv_prefill(x[:, :, :cut], w)
    n = 0.0
    for t in range(cut, T):
        qkv1 = kda.conv_step(x[:, :, t], cs, w)
        assert ((qkv1.float() - qkv[:, :, t].float()).abs() <= 2.0 ** -7 * qkv[:, :, t].float().abs() + 1e-6).all()
        a = [z[:, :, t].contiguous() for z in (q, k, v)]
        o1 = kda.decode_step(*a, la[:, :, t].contiguous(), beta[:, :, t].contiguous(), S1)
        y1 = kda.ssm_step(*a, decay[:, :, t].contiguous(), step[:, :, t].contiguous(), S2)
        n = max(n, float((o1.float() - o[:, :, t].float()).norm() / o[:, :, t].float().norm()),
                float((y1.float() - y[:, :, t].float()).norm() / y[:, :, t].float().norm()))
    torch.cuda.synchronize()
    assert torch.equal(cs, conv_state)
    # the states' rounding (under 1/127 of a block's largest value, 2.5 deviations or so) and bf16's
    assert n <= 2.5 / 127 + 8e-3
