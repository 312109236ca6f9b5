"""GPU tests of the companion operators away from the ordinary call: captured and
replayed, on two streams at once, with broadcast and far-apart inputs, gaps between
output rows, non-finite padding, empty sizes, too small a workspace, and the input check.

Tolerances are those of test_ops_gpu.py (its docstring derives them); comparisons of one
kernel with itself are exact, since every sum has a fixed order."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc
from test_ops_gpu import DT, TOL, check_grads, conv_case, dev, gen, ssm_args, ssm_case, ssm_ref_args, tm, up

pytestmark = pytest.mark.gpu

ERR_PRECONDITION = 6


def flat(r):
    """All tensors of a call's result."""
    if isinstance(r, torch.Tensor):
        return [r]
    if isinstance(r, dict):
        return list(r.values())
    return [t for t in r if t is not None]


def calls(dt):
    """name -> (static inputs, function of them that returns what it wrote)."""
    c = conv_case(2, 3, 70, 16, 4, dt, True, True, seed=1)
    conv = {n: up(t) for n, t in c.items()}
    s = {n: up(t) for n, t in ssm_case(1, 4, 2, 700, 64, 64, dt, seed=2).items()}
    one = {n: (t[:, :, 0].contiguous() if t.dim() > 2 and n not in ("S0", "dS_T") else t) for n, t in s.items()}
    cache = dict(zip(("cache", "scales"), kda.state_cache(5, 4, 64, 64, "int8", dev())))
    slots = torch.tensor([3], dtype=torch.int32, device=dev())

    def step(t):
        S, cs = t["S0"].clone(), t["state"].clone()
        return (kda.ssm_step(t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], S, t["D"]), S,
                kda.conv_step(t["x"], cs, t["weight"], t["bias"]), cs)

    def park(t):
        kda.state_store(t["S0"], slots, t["cache"], t["scales"])
        return t["cache"].view(torch.uint8), t["scales"], kda.state_load(t["cache"], t["scales"], slots)

    fwd = lambda t: (t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], t["D"], t["S0"])  # noqa: E731
    return {
        "conv": (conv, lambda t: kda.conv_prefill(t["x"], t["weight"], t["bias"], t["state"])),
        "conv_backward": (conv, lambda t: kda.conv_backward(t["x"], t["weight"], t["bias"], t["state"], t["dO"],
                                                            t["dstate_out"])),
        "ssm": (s, lambda t: kda.ssm_prefill(*fwd(t))),
        "ssm_backward": (s, lambda t: kda.ssm_backward(*fwd(t), t["dO"], t["dS_T"])),
        "steps": ({**one, "x": conv["x"][:, :, 0].contiguous(), "state": conv["state"], "weight": conv["weight"],
                   "bias": conv["bias"]}, step),
        "cache": ({"S0": s["S0"], **cache}, park),
    }


NAMES = ["conv", "conv_backward", "ssm", "ssm_backward", "steps", "cache"]


def redraw(inputs, g):
    """New values of the same kind: every tensor's entries permuted (signs of gates stay)."""
    for t in inputs.values():
        if t.dtype in (torch.float32, torch.bfloat16) and t.numel():
            t.copy_(t.flatten()[torch.randperm(t.numel(), generator=g).to(t.device)].view(t.shape))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_capture_and_replay(name, dt):
    """A captured call replayed on changed inputs, with eager calls between, gives the eager result."""
    print(f"[case] capture {name} {dt}", flush=True)
    inputs, f = calls(dt)[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(inputs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f(inputs)
    g = gen(3)
    for rep in range(4):
        redraw(inputs, g)
        ref = [t.clone() for t in flat(f(inputs))]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(flat(got), ref):
            assert torch.equal(a, b), (name, rep)


def test_two_captured_scans_with_their_own_workspaces():
    """Two captured backward passes replayed on two streams at once."""
    runs = []
    for seed in (5, 6):
        t = {n: up(x) for n, x in ssm_case(1, 4, 2, 700, 64, 64, "bf16", seed=seed).items()}
        a = (t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], t["D"], t["S0"], t["dO"], t["dS_T"])
        need = int(kda.load().kda_ssm_backward_workspace_bytes(1, 4, 2, 700, 64, 64, 1))
        ws = torch.empty(need, dtype=torch.uint8, device=dev())
        ref = {n: x.clone() for n, x in kda.ssm_backward(*a, workspace=ws).items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = kda.ssm_backward(*a, workspace=ws)
        runs.append((graph, got, ref, torch.cuda.Stream(), (a, ws)))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, got, _, stream, _ in runs:
            with torch.cuda.stream(stream):
                for x in got.values():
                    x.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, got, ref, _, _ in runs:
            for n in ref:
                assert torch.equal(got[n], ref[n]), n


def test_two_streams_at_once():
    every = [(n, *calls("bf16")[n]) for n in NAMES if n != "cache"]
    refs = [[t.clone() for t in flat(f(i))] for _, i, f in every]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                order = every if k == 0 else every[::-1]
                got[k].append({n: flat(f(i)) for n, i, f in order})
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            for (n, _, _), ref in zip(every, refs):
                for a, b in zip(r[n], ref):
                    assert torch.equal(a, b), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_broadcast_inputs(dt):
    """Inputs of stride 0: q and k of one sequence for all, one decay for all tokens, one dO row.  The
    gradients come back whole, one value per element of the broadcast input."""
    B, H, G, T = 3, 4, 2, 130
    c = ssm_case(B, H, G, T, 64, 64, dt, seed=7)
    c["q"], c["k"] = c["q"][:1].expand(B, G, T, 64), c["k"][:1].expand(B, G, T, 64)
    c["log_alpha"] = c["log_alpha"][:, :, :1].expand(B, H, T)
    c["beta"] = c["beta"][:1, :1].expand(B, H, T)
    c["dO"] = c["dO"][:, :, :1].expand(B, H, T, 64)

    def b(n, first):
        return up(first.contiguous()).expand(c[n].shape)
    t = {n: up(c[n]) for n in ("v", "D", "S0", "dS_T")}
    t.update(q=b("q", c["q"][:1]), k=b("k", c["k"][:1]), log_alpha=b("log_alpha", c["log_alpha"][:, :, :1]),
             beta=b("beta", c["beta"][:1, :1]), dO=b("dO", c["dO"][:, :, :1]))
    args = (t["q"], t["k"], t["v"], t["log_alpha"], t["beta"], t["D"], t["S0"])
    o, S = kda.ssm_prefill(*args)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    assert orc.rel(o, ro) <= TOL[dt] and orc.rel(S, rS) <= 1e-5
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"]), dt)

    cc = conv_case(B, H, T, 16, 4, dt, True, True, seed=8)
    x = up(cc["x"][:1]).expand(B, H, T, 16)
    o, s = kda.conv_prefill(x, up(cc["weight"]), up(cc["bias"]), up(cc["state"]))
    o1, s1 = kda.conv_prefill(x.contiguous(), up(cc["weight"]), up(cc["bias"]), up(cc["state"]))
    gr = kda.conv_backward(x, up(cc["weight"]), up(cc["bias"]), up(cc["state"]), up(cc["dO"]))
    g1 = kda.conv_backward(x.contiguous(), up(cc["weight"]), up(cc["bias"]), up(cc["state"]), up(cc["dO"]))
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(s, s1)
    for n in gr:
        assert torch.equal(gr[n], g1[n]), n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_padding_is_not_read_into_results(dt):
    """NaN and infinities behind the lengths, in every input; also a sequence of no tokens."""
    lens = torch.tensor([0, 1, 63, 64, 65, 200, 130], dtype=torch.int32)
    B, H, G, T = len(lens), 2, 1, 200
    c = ssm_case(B, H, G, T, 64, 128, dt, seed=9)
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True), lens=lens)
    cc = conv_case(B, H, T, 16, 4, dt, True, True, seed=10)
    rc, rs = orc.conv(cc["x"], cc["weight"], cc["bias"], cc["state"], True, lens.tolist())
    for b, n in enumerate(lens.tolist()):
        for name, bad in (("q", "nan"), ("k", "inf"), ("v", "nan"), ("log_alpha", "nan"), ("beta", "inf")):
            c[name][b, :, n:] = float(bad)
        cc["x"][b, :, n:] = float("nan")
    args, _ = ssm_args(c, True, True, True)
    for ws in ("auto", None):
        o = torch.full((B, H, T, 128), 7.0, dtype=DT[dt], device=dev())
        _, S = kda.ssm_prefill(*args, lens=up(lens), o=o, workspace=ws)
        torch.cuda.synchronize()
        assert (o.cpu()[torch.isnan(ro)] == 7.0).all()
        assert orc.rel(o, ro) <= TOL[dt] and orc.rel(S, rS) <= 1e-5
    o = torch.full((B, H, T, 16), 7.0, dtype=DT[dt], device=dev())
    _, s = kda.conv_prefill(tm(up(cc["x"])), up(cc["weight"]), up(cc["bias"]), up(cc["state"]), lens=up(lens), o=o)
    torch.cuda.synchronize()
    assert (o.cpu()[torch.isnan(rc)] == 7.0).all()
    assert orc.rel(o, rc) <= (2.0 ** -8 if dt == "bf16" else 2e-6)
    assert torch.equal(s.cpu().double(), rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gaps_and_odd_addresses(dt):
    """Output rows with gaps between them, whose contents stay; gates, weights and skips that start at
    odd elements."""
    B, H, G, T, d = 2, 3, 1, 75, 64
    c = ssm_case(B, H, G, T, d, d, dt, seed=11)

    def odd(t):
        buf = torch.empty(t.numel() + 3, dtype=t.dtype, device=dev())
        v = buf[3:].view(t.shape)
        v.copy_(up(t))
        return v
    buf = torch.full((B, T, H, d + 8), 7.0, dtype=DT[dt], device=dev())
    o = buf[..., :d].transpose(1, 2)
    gates = torch.full((B, T, H, 3), float("nan"), dtype=DT[dt], device=dev())
    gates[..., 1], gates[..., 2] = up(c["log_alpha"]).transpose(1, 2), up(c["beta"]).transpose(1, 2)
    la, beta = gates[..., 1].transpose(1, 2), gates[..., 2].transpose(1, 2)
    q, k, v = (tm(up(c[n])) for n in ("q", "k", "v"))
    _, S = kda.ssm_prefill(q, k, v, la, beta, odd(c["D"]), up(c["S0"]), o=o)
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    assert orc.rel(o, ro) <= TOL[dt] and orc.rel(S, rS) <= 1e-5
    assert (buf[..., d:] == 7.0).all()
    got = kda.ssm_backward(q, k, v, la, beta, odd(c["D"]), up(c["S0"]), up(c["dO"]), up(c["dS_T"]))
    torch.cuda.synchronize()
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"]), dt)
    one = kda.ssm_step(*(x[:, :, 0].contiguous() for x in (q, k, v)), odd(c["log_alpha"][:, :, 0]),
                       odd(c["beta"][:, :, 0]), up(c["S0"]), odd(c["D"]))
    torch.cuda.synchronize()
    assert orc.rel(one, ro[:, :, 0]) <= (2.0 ** -8 if dt == "bf16" else 1e-5)

    cc = conv_case(B, H, T, 24, 4, dt, True, True, seed=12)
    buf = torch.full((B, T, H, 32), 7.0, dtype=DT[dt], device=dev())
    o = buf[..., :24].transpose(1, 2)
    kda.conv_prefill(up(cc["x"]), odd(cc["weight"]), odd(cc["bias"]), up(cc["state"]), o=o)
    ref, _ = kda.conv_prefill(up(cc["x"]), up(cc["weight"]), up(cc["bias"]), up(cc["state"]))
    torch.cuda.synchronize()
    assert torch.equal(o, ref) and (buf[..., 24:] == 7.0).all()
    a = kda.conv_backward(up(cc["x"]), odd(cc["weight"]), odd(cc["bias"]), up(cc["state"]), up(cc["dO"]))
    b = kda.conv_backward(up(cc["x"]), up(cc["weight"]), up(cc["bias"]), up(cc["state"]), up(cc["dO"]))
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


def far(t, gap):
    """t's values with `gap` elements between the starts of consecutive t[0], t[1], ..."""
    n = t[0].numel()
    buf = torch.empty((t.shape[0] - 1) * gap + n, dtype=t.dtype, device=dev())
    v = buf.as_strided(t.shape, (gap, *t[0].contiguous().stride()))
    v.copy_(up(t))
    return v


def test_distances_past_32_bits():
    """Sequences 2^31 + 64 elements apart, tokens 2^23 apart, and cache entries behind 2^32 values."""
    gap = 2 ** 31 + 64
    c = ssm_case(2, 2, 1, 70, 64, 64, "bf16", seed=13)
    t = {n: far(c[n], gap) for n in ("q", "k", "v", "dO")}
    args = (t["q"], t["k"], t["v"], up(c["log_alpha"]), up(c["beta"]), up(c["D"]), up(c["S0"]))
    near = [up(c[n]) for n in ("q", "k", "v", "log_alpha", "beta", "D", "S0")]
    o = far(torch.zeros(2, 2, 70, 64, dtype=torch.bfloat16), gap)
    _, S = kda.ssm_prefill(*args, o=o)
    o1, S1 = kda.ssm_prefill(*near)
    g = kda.ssm_backward(*args, t["dO"], up(c["dS_T"]))
    g1 = kda.ssm_backward(*near, up(c["dO"]), up(c["dS_T"]))
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(S, S1)
    for n in g:
        assert torch.equal(g[n], g1[n]), n
    cc = conv_case(2, 2, 70, 16, 4, "bf16", True, True, seed=14)
    rest = (up(cc["weight"]), up(cc["bias"]), up(cc["state"]))
    x, dO = far(cc["x"], gap), far(cc["dO"], gap)
    oc = far(torch.zeros(2, 2, 70, 16, dtype=torch.bfloat16), gap)
    _, s = kda.conv_prefill(x, *rest, o=oc)
    o1, s1 = kda.conv_prefill(up(cc["x"]), *rest)
    g = kda.conv_backward(x, *rest, dO)
    g1 = kda.conv_backward(up(cc["x"]), *rest, up(cc["dO"]))
    torch.cuda.synchronize()
    assert torch.equal(oc, o1) and torch.equal(s, s1)
    for n in g:
        assert torch.equal(g[n], g1[n]), n
    del t, args, o, x, dO, oc, g

    wide = 2 ** 23  # the largest distance of tokens
    base = torch.empty(70 * wide, dtype=torch.float32, device=dev())
    c = ssm_case(1, 2, 1, 70, 64, 64, "f32", seed=15)
    at = 0
    v = {}
    for n in ("q", "k", "v", "o", "x"):
        rows = 1 if n in "qk" else 2
        v[n] = base.as_strided((1, rows, 70, 64), (0, 64, wide, 1), at)
        at += rows * 64
    for n in ("q", "k", "v"):
        v[n].copy_(up(c[n]))
    rest = [up(c[n]) for n in ("log_alpha", "beta", "D", "S0")]
    _, S = kda.ssm_prefill(v["q"], v["k"], v["v"], *rest, o=v["o"])
    o1, S1 = kda.ssm_prefill(up(c["q"]), up(c["k"]), up(c["v"]), *rest)
    torch.cuda.synchronize()
    assert torch.equal(v["o"], o1) and torch.equal(S, S1)
    w = torch.randn(2, 64, 4, generator=gen(1)).to(dev())
    v["x"].copy_(up(c["v"]))
    kda.conv_prefill(v["x"], w, o=v["o"])
    o1, _ = kda.conv_prefill(up(c["v"]), w)
    torch.cuda.synchronize()
    assert torch.equal(v["o"], o1)
    del base, v

    nslots = 2 ** 32 // (128 * 128) + 3
    cache, scales = kda.state_cache(nslots, 1, 128, 128, "int8", dev())
    small, ss = kda.state_cache(2, 1, 128, 128, "int8", dev())
    S = torch.randn(2, 1, 128, 128, generator=gen(2)).to(dev())
    slots = torch.tensor([nslots - 1, 1], dtype=torch.int32, device=dev())
    kda.state_store(S, slots, cache, scales)
    kda.state_store(S, torch.tensor([0, 1], dtype=torch.int32, device=dev()), small, ss)
    back = kda.state_load(cache, scales, slots)
    torch.cuda.synchronize()
    assert torch.equal(cache[[nslots - 1, 1]], small) and torch.equal(scales[[nslots - 1, 1]], ss)
    assert torch.equal(back, kda.state_load(small, ss, torch.tensor([0, 1], dtype=torch.int32, device=dev())))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [(40.0, 40.0, 40.0), (40.0, 0.001, 3.0), (0.2, 40.0, 0.001)])
def test_strong_decay(rate, dt):
    """Segments whose states vanish before their ends, alone and next to heads that keep theirs."""
    B, H, T = 1, 3, 1500
    c = ssm_case(B, H, 1, T, 64, 64, dt, seed=16)
    c["log_alpha"] = (-torch.tensor(rate)[None, :, None] * torch.ones(B, H, T)).to(DT[dt])
    args, t = ssm_args(c, True, True, True)
    o, S = kda.ssm_prefill(*args)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    ref = orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"])
    for h in range(H):
        assert orc.rel(o[:, h], ro[:, h]) <= TOL[dt] and orc.rel(S[:, h], rS[:, h]) <= 1e-5
        # (dlog_alpha of a head that keeps nothing is zero but for what underflows)
        for n in ("dv", "dbeta") + (("dlog_alpha",) if rate[h] < 10 else ()):
            assert orc.rel(got[n][:, h], ref[n][:, h]) <= TOL[dt], (n, h)
    assert orc.rel(got["dq"], ref["dq"]) <= TOL[dt] and orc.rel(got["dk"], ref["dk"]) <= TOL[dt]


def test_many_heads_in_one_piece():
    """Enough sequences and heads to fill the device: not cut."""
    B, H, G, T = 8, 128, 8, 65
    assert kda.ssm_prefill_workspace_bytes(B, H, G, T, 64, 64, torch.bfloat16) == 0
    c = ssm_case(B, H, G, T, 64, 64, "bf16", seed=17)
    args, t = ssm_args(c, True, True, True)
    o, S = kda.ssm_prefill(*args)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True))
    assert orc.rel(o, ro) <= TOL["bf16"] and orc.rel(S, rS) <= 1e-5
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"]), "bf16")


@pytest.mark.parametrize("B,H,G,T,dk,dv", [(1, 7, 1, 130, 64, 128), (2, 10, 2, 150, 64, 64), (1, 9, 1, 100, 128, 128),
                                         (1, 18, 2, 65, 128, 64), (3, 2, 1, 64, 64, 128), (1, 4, 1, 1, 128, 64)])
def test_groups_of_many_heads(B, H, G, T, dk, dv):
    """bf16 gradients summed over more heads than one workgroup's two, odd counts among them."""
    print(f"[case] ssm_backward {B} {H}/{G} {T} {dk}x{dv}", flush=True)
    c = ssm_case(B, H, G, T, dk, dv, "bf16", seed=H)
    args, t = ssm_args(c, True, True, True)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, True), c["dO"], c["dS_T"]), "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 130])
def test_first_decay_without_a_start_state(T, dt):
    """The first token's decay multiplies nothing: its gradient is zero, not what rounding leaves."""
    c = ssm_case(2, 4, 2, T, 64, 128, dt, seed=T)
    args, t = ssm_args(c, True, False, False)
    got = kda.ssm_backward(*args, t["dO"], t["dS_T"])
    torch.cuda.synchronize()
    assert (got["dlog_alpha"][:, :, 0] == 0).all()
    check_grads(got, orc.ssm_backward(*ssm_ref_args(c, True, False), c["dO"], c["dS_T"]), dt)


def test_small_workspace_walks_in_one_piece():
    c = ssm_case(1, 2, 1, 700, 64, 64, "bf16", seed=18)
    args, _ = ssm_args(c, True, True, True)
    need = kda.ssm_prefill_workspace_bytes(1, 2, 1, 700, 64, 64, torch.bfloat16)
    o, S = kda.ssm_prefill(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev()))
    o1, S1 = kda.ssm_prefill(*args, workspace=None)
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(S, S1)


def test_empty_sizes():
    bf = torch.bfloat16
    z = lambda *s: torch.zeros(*s, dtype=bf, device=dev())  # noqa: E731
    st = torch.randn(2, 3, 3, 8, generator=gen(1)).to(bf).to(dev())
    o, s = kda.conv_prefill(z(2, 3, 0, 8), z(3, 8, 4), None, st)
    assert o.shape == (2, 3, 0, 8) and torch.equal(s, st)
    _, s = kda.conv_prefill(z(2, 3, 0, 8), z(3, 8, 4))
    assert (s == 0).all()
    assert kda.conv_prefill(z(0, 3, 5, 8), z(3, 8, 4))[0].shape == (0, 3, 5, 8)
    assert kda.conv_step(z(0, 3, 8), z(0, 3, 3, 8), z(3, 8, 4)).shape == (0, 3, 8)
    S0 = torch.randn(2, 4, 64, 64, generator=gen(2)).to(dev())
    o, S = kda.ssm_prefill(z(2, 2, 0, 64), z(2, 2, 0, 64), z(2, 4, 0, 64), z(2, 4, 0), z(2, 4, 0), None, S0)
    torch.cuda.synchronize()
    assert o.shape == (2, 4, 0, 64) and torch.equal(S, S0)
    _, S = kda.ssm_prefill(z(2, 2, 0, 64), z(2, 2, 0, 64), z(2, 4, 0, 64), z(2, 4, 0), z(2, 4, 0))
    assert (S == 0).all()
    assert kda.ssm_prefill(z(0, 2, 9, 64), z(0, 2, 9, 64), z(0, 4, 9, 64), z(0, 4, 9), z(0, 4, 9))[1].shape[0] == 0
    e = torch.zeros(0, 4, 64, 64, device=dev())
    assert kda.ssm_step(z(0, 2, 64), z(0, 2, 64), z(0, 4, 64), z(0, 4), z(0, 4), e).shape == (0, 4, 64)
    cache, scales = kda.state_cache(2, 4, 64, 64, "int8", dev())
    none = torch.zeros(0, dtype=torch.int32, device=dev())
    kda.state_store(e, none, cache, scales)
    assert kda.state_load(cache, scales, none).shape == (0, 4, 64, 64)
    with pytest.raises(kda.KdaError):
        kda.conv_backward(z(2, 3, 0, 8), z(3, 8, 4), None, None, z(2, 3, 0, 8))
    with pytest.raises(kda.KdaError):
        kda.ssm_backward(z(2, 2, 0, 64), z(2, 2, 0, 64), z(2, 4, 0, 64), z(2, 4, 0), z(2, 4, 0), dO=z(2, 4, 0, 64))


def test_input_check():
    """Option check: positive or NaN log_alpha and non-finite beta are refused before anything is written."""
    c = ssm_case(1, 2, 1, 70, 64, 64, "bf16", seed=19)
    for name, bad in (("log_alpha", 0.5), ("log_alpha", float("nan")), ("beta", float("inf"))):
        x = {n: t.clone() for n, t in c.items()}
        x[name][0, 1, 69] = bad
        args, t = ssm_args(x, True, True, True)
        o = torch.full_like(t["v"], 7.0)
        with kda.options(check=1):
            with pytest.raises(kda.KdaError) as e:
                kda.ssm_prefill(*args, o=o)
            assert e.value.status == ERR_PRECONDITION
            with pytest.raises(kda.KdaError) as e:
                kda.ssm_backward(*args, t["dO"])
            assert e.value.status == ERR_PRECONDITION
            with pytest.raises(kda.KdaError) as e:
                kda.ssm_step(*(t[n][:, :, 69].contiguous() for n in ("q", "k", "v", "log_alpha", "beta")), t["S0"])
            assert e.value.status == ERR_PRECONDITION
        torch.cuda.synchronize()
        assert (o == 7.0).all() and torch.equal(t["S0"].cpu(), c["S0"])
    c["log_alpha"][0, 0, 5] = -float("inf")
    args, _ = ssm_args(c, True, True, True)
    with kda.options(check=1):
        o, S = kda.ssm_prefill(*args)
    o1, S1 = kda.ssm_prefill(*args)
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(S, S1)


def test_input_check_leaves_padding_alone():
    c = ssm_case(2, 2, 1, 70, 64, 64, "bf16", seed=21)
    c["log_alpha"][0, :, 30:], c["beta"][0, :, 30:] = float("nan"), float("inf")
    args, _ = ssm_args(c, True, True, True)
    lens = torch.tensor([30, 70], dtype=torch.int32)
    with kda.options(check=1):
        o, S = kda.ssm_prefill(*args, lens=up(lens))
    torch.cuda.synchronize()
    ro, rS = orc.ssm(*ssm_ref_args(c, True, True), lens=lens)
    assert orc.rel(S, rS) <= 1e-5 and orc.rel(o, ro) <= TOL["bf16"]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_far_apart_tokens(dt):
    """Inputs and incoming gradients with tokens 2^22 elements apart, heads between them."""
    wide, H = 2 ** 22, 2
    c = ssm_case(1, H, 1, 70, 64, 64, dt, seed=22)
    base = torch.empty(69 * wide + 4 * H * 64 + 128, dtype=DT[dt], device=dev())
    at, v = 0, {}
    for n in ("q", "k", "v", "dO"):
        rows = c[n].shape[1]
        v[n] = base.as_strided((1, rows, 70, 64), (0, 64, wide, 1), at)
        v[n].copy_(up(c[n]))
        at += rows * 64
    rest = [up(c[n]) for n in ("log_alpha", "beta", "D", "S0")]
    near = [up(c[n]) for n in ("q", "k", "v")]
    g = kda.ssm_backward(v["q"], v["k"], v["v"], *rest, v["dO"], up(c["dS_T"]))
    g1 = kda.ssm_backward(*near, *rest, up(c["dO"]), up(c["dS_T"]))
    torch.cuda.synchronize()
    for n in g:
        assert torch.equal(g[n], g1[n]), n


def test_refusals_of_the_bindings():
    c = {n: up(t) for n, t in ssm_case(1, 2, 1, 10, 64, 64, "bf16", seed=20).items()}
    a = [c["q"], c["k"], c["v"], c["log_alpha"], c["beta"]]
    for i, bad in ((0, c["q"].float()), (1, c["k"][:, :, :9]), (3, c["log_alpha"][:, :1]),
                   (2, c["v"].transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(kda.KdaError):
            kda.ssm_prefill(*a[:i], bad, *a[i + 1:])
    with pytest.raises(kda.KdaError):
        kda.ssm_prefill(*a, S0=c["S0"].bfloat16())
    with pytest.raises(kda.KdaError):
        kda.ssm_prefill(*a, lens=torch.zeros(1, dtype=torch.int64, device=dev()))
    with pytest.raises(kda.KdaError):
        kda.ssm_backward(*a)
    x, w = c["v"], torch.zeros(2, 64, 4, dtype=torch.bfloat16, device=dev())
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(x, w[:1])
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(x, w, activation="gelu")
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(x, w, o=x)
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(x, w, state=torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16, device=dev()))
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(torch.zeros(1, 2, 10, 12, dtype=torch.bfloat16, device=dev()), w[:, :12].contiguous())
    cache, scales = kda.state_cache(2, 2, 64, 64, "int8", dev())
    with pytest.raises(kda.KdaError):
        kda.state_store(c["S0"], torch.zeros(2, dtype=torch.int32, device=dev()), cache, scales)
    with pytest.raises(kda.KdaError):
        kda.state_store(c["S0"], torch.zeros(1, dtype=torch.int64, device=dev()), cache, scales)
