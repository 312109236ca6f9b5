"""GPU tests of the gated linear recurrence, the norm and the drafts away from the ordinary call: sequence
lengths around every tile, captured and replayed, on two streams at once, with broadcast and far-apart
inputs, gaps between output rows, slow and strong decays, empty sizes and the input check.

Tolerances are those of test_layer_ops_gpu.py (its docstring derives them); comparisons of one kernel with
itself are exact, since every sum has a fixed order."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import layer_oracle as orc
from test_layer_ops_gpu import (DT, HALF, check_glr, check_glr_grads, check_norm_grads, dev, gen, glr_case, norm_case,
                                slack, summed, tm, up, verify_case, within)

pytestmark = pytest.mark.gpu

ERR_PRECONDITION = 6


def flat(r):
    if isinstance(r, torch.Tensor):
        return [r]
    return [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]


# ------------------------------------------------------- around the tiles
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("C", [64, 640, 4160])  # 1, 10 and 65 chains of 64 channels: another tile length each
def test_glr_lengths_around_tiles(C, beta, dt):
    """Every length next to a tile's end (runs of 32 to 256 tokens), forwards and backwards, from one reference
    of the longest: shorter prompts are its prefixes."""
    longest = {64: 521, 640: 400, 4160: 270}[C]
    c = glr_case(1, 1, longest, C, dt, C, beta, True, rate=0.02)
    c["x"], c["la"], c["dO"] = (c[n].reshape(1, 1, longest, C) for n in ("x", "la", "dO"))
    ref, _ = orc.glr(c["x"], c["la"], c["beta"], c["h0"], True)
    a = lambda t: None if t is None else t.abs()  # noqa: E731
    size, _ = orc.glr(a(c["x"]), c["la"], a(c["beta"]), a(c["h0"]), True)
    x, la, be, h0 = (up(c[n]) for n in ("x", "la", "beta", "h0"))
    for T in sorted({n for k in (32, 48, 64, 96, 128, 192, 256, 384, 512) for n in (k - 1, k, k + 1) if n <= longest} | {2, longest}):
        cut = lambda t: None if t is None else t[:, :, :T]  # noqa: E731
        o, h = kda.glr_prefill(cut(x), cut(la), cut(be), h0, normalise=True)
        torch.cuda.synchronize()
        within(o, ref[:, :, :T], HALF[dt] * ref[:, :, :T].abs() + slack(dt, T) * size[:, :, :T], T)
        within(h, ref[:, :, T - 1], 2.0 ** -24 * ref[:, :, T - 1].abs() + slack(dt, T) * size[:, :, T - 1], T)
    for T in (33, 65, 97, 129, 257):
        cc = {n: (t[:, :, :T] if t is not None and t.dim() == 4 else t) for n, t in c.items()}
        o, _ = kda.glr_prefill(*(up(cc[n]) for n in ("x", "la", "beta", "h0")), normalise=True)
        got = kda.glr_backward(*(up(cc[n]) for n in ("x", "la", "beta", "h0")), o, up(cc["dO"]), up(cc["dh_T"]), normalise=True)
        torch.cuda.synchronize()
        check_glr_grads(got, cc, o.cpu(), True, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_many_tiles_with_lengths(dt):
    """Sequences of many tiles and of none, next to each other."""
    lens = [0, 1500, 1, 256, 257, 1023]
    c = glr_case(6, 3, 1500, 24, dt, 4, rate=0.01)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev())
    o = torch.full((6, 3, 1500, 24), 7.0, dtype=DT[dt], device=dev())
    _, h = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")), normalise=True, lens=ln, o=o)
    torch.cuda.synchronize()
    ref = check_glr(c, True, dt, o, h, lens)
    assert (o.cpu().double()[torch.isnan(ref)] == 7.0).all()
    got = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), o, up(c["dO"]), up(c["dh_T"]), normalise=True, lens=ln)
    torch.cuda.synchronize()
    check_glr_grads(got, c, torch.where(torch.isnan(ref), 0.0, o.cpu().double()), True, dt, lens)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_without_the_tiles_before(dt, kda_opts):
    """A run of tokens that gets no answer from the run before it walks the sequence itself (option glr_polls 0:
    every run does)."""
    c = glr_case(2, 2, 700, 40, dt, 8, rate=0.02)
    kda_opts("glr_polls", 0)
    lens = [700, 333]
    ln = torch.tensor(lens, dtype=torch.int32, device=dev())
    o = torch.zeros(2, 2, 700, 40, dtype=DT[dt], device=dev())
    _, h = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")), normalise=True, lens=ln, o=o)
    got = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), o, up(c["dO"]), up(c["dh_T"]), normalise=True, lens=ln)
    torch.cuda.synchronize()
    check_glr(c, True, dt, o, h, lens)
    check_glr_grads(got, c, o.cpu(), True, dt, lens)


def test_glr_same_bits_every_time():
    """However far a tile has to look back, the state in front of it is the same."""
    c = glr_case(1, 5, 20000, 128, "bf16", 3, rate=0.01)
    args = [up(c[n]) for n in ("x", "la", "beta", "h0")]
    first = kda.glr_prefill(*args, normalise=True)
    grads = kda.glr_backward(*args, first[0], up(c["dO"]), up(c["dh_T"]), normalise=True)
    for _ in range(5):
        again = kda.glr_prefill(*args, normalise=True)
        g = kda.glr_backward(*args, again[0], up(c["dO"]), up(c["dh_T"]), normalise=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(grads[n], g[n]) for n in grads)


@pytest.mark.parametrize("polls", [None, 0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_states_in_place(dt, polls, kda_opts):
    """h_T in h0's place, with more runs of tokens than the device holds at a time and unequal lengths: whichever run
    ends first, all of them start from the state that was given."""
    if polls is not None:
        kda_opts("glr_polls", polls)
    c = glr_case(6, 16, 2500, 64, dt, 21)
    lens = torch.tensor([2500, 0, 1, 2499, 128, 1300], dtype=torch.int32, device=dev())
    args = [up(c[n]) for n in ("x", "la", "beta")]
    h = up(c["h0"])
    o0, h0 = kda.glr_prefill(*args, h.clone(), lens=lens, o=torch.zeros_like(args[0]))
    for _ in range(3):
        at = h.clone()
        o, got = kda.glr_prefill(*args, at, lens=lens, o=torch.zeros_like(args[0]), h_T=at)
        torch.cuda.synchronize()
        assert got is at and torch.equal(at, h0) and torch.equal(o, o0)


# ------------------------------------------------- captured, concurrent
def calls(dt):
    """name -> (static inputs, function of them that returns what it wrote)."""
    c = {n: up(t) for n, t in glr_case(2, 3, 700, 24, dt, 1).items()}
    c["o"], _ = kda.glr_prefill(c["x"], c["la"], c["beta"], c["h0"], normalise=True)
    n = {k: up(t) for k, t in norm_case(2, 3, 50, 64, dt, 2, True, True, True).items()}
    p, q, tok, u = (up(t) for t in verify_case(7, 3, 9001, dt, 3))
    long = dict(zip(("p", "q", "tok", "u"), (up(t) for t in verify_case(3, 3, 40001, dt, 6))))
    S_pos, S = torch.randn(7, 4, 2, 16, 16, generator=gen(4)).to(dev()), torch.randn(7, 2, 16, 16, generator=gen(5)).to(dev())
    fwd = lambda t: (t["x"], t["la"], t["beta"], t["h0"])  # noqa: E731

    def step(t):
        h = t["h0"].clone()
        return kda.glr_step(t["x"][:, :, 0], t["la"][:, :, 0], h, t["beta"][:, :, 0]), h

    def drafts(t):
        a, out = kda.draft_verify(t["p"], t["q"], tok, t["u"])
        kept = t["S"].clone()
        kda.state_commit(t["S_pos"], a, kept)
        return a, out, kept

    return {
        "glr": (c, lambda t: kda.glr_prefill(*fwd(t), normalise=True)),
        "glr_backward": (c, lambda t: kda.glr_backward(*fwd(t), t["o"], t["dO"], t["dh_T"], normalise=True)),
        "glr_step": (c, step),
        "norm": (n, lambda t: kda.rms_norm(t["x"], t["w"], t["residual"], t["gate"])),
        "norm_quant": (n, lambda t: [x.view(torch.uint8) if x.element_size() == 1 else x
                                     for x in kda.rms_norm_quant(t["x"], t["w"], t["residual"], t["gate"])]),
        "norm_backward": (n, lambda t: kda.rms_norm_backward(t["x"], t["w"], t["dy"], t["ds"], t["gate"])),
        "drafts": (dict(p=p, q=q, u=u, S_pos=S_pos, S=S), drafts),
        "drafts_of_long_rows": (long, lambda t: kda.draft_verify(t["p"], t["q"], t["tok"], t["u"])),
    }


NAMES = ["glr", "glr_backward", "glr_step", "norm", "norm_quant", "norm_backward", "drafts", "drafts_of_long_rows"]


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


def test_two_captured_recurrences_with_their_own_workspaces():
    """Two captured backward passes of many tiles replayed on two streams at once."""
    runs = []
    for seed in (5, 6):
        t = {n: up(x) for n, x in glr_case(2, 4, 3000, 64, "bf16", seed).items()}
        a = (t["x"], t["la"], t["beta"], t["h0"])
        o, _ = kda.glr_prefill(*a, normalise=True)
        need = int(kda.load().kda_glr_backward_workspace_bytes(2, 4, 3000, 64, 1))
        ws = torch.empty(need, dtype=torch.uint8, device=dev())
        ref = {n: x.clone() for n, x in kda.glr_backward(*a, o, t["dO"], t["dh_T"], normalise=True, workspace=ws).items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = kda.glr_backward(*a, o, t["dO"], t["dh_T"], normalise=True, workspace=ws)
        runs.append((graph, got, ref, torch.cuda.Stream(), (a, o, t, ws)))
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
    every = [(n, *calls("bf16")[n]) for n in NAMES]
    refs = [[t.clone() for t in flat(f(i))] for _, i, f in every]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for rep in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append({n: flat(f(i)) for n, i, f in (every if k == 0 else every[::-1])})
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            for (n, _, _), ref in zip(every, refs):
                for a, b in zip(r[n], ref):
                    assert torch.equal(a, b), n


# ------------------------------------------------------ memory layouts
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_broadcast_inputs(dt):
    """Inputs of stride 0: one decay row for all tokens, one x for all sequences, one dO row.  The gradients come
    back whole, one value per element of the broadcast input."""
    B, H, T, d = 3, 2, 300, 16
    c = glr_case(B, H, T, d, dt, 7)
    c["x"] = c["x"][:1].expand(B, H, T, d)
    c["la"] = c["la"][:, :, :1].expand(B, H, T, d)
    c["beta"] = c["beta"][:1, :1].expand(B, H, T, d)
    c["dO"] = c["dO"][:, :, :1].expand(B, H, T, d)
    x = up(c["x"][:1].contiguous()).expand(B, H, T, d)
    la = up(c["la"][:, :, :1].contiguous()).expand(B, H, T, d)
    beta = up(c["beta"][:1, :1].contiguous()).expand(B, H, T, d)
    dO = up(c["dO"][:, :, :1].contiguous()).expand(B, H, T, d)
    o, h = kda.glr_prefill(x, la, beta, up(c["h0"]), normalise=True, o=torch.empty(B, H, T, d, dtype=DT[dt], device=dev()))
    got = kda.glr_backward(x, la, beta, up(c["h0"]), o, dO, up(c["dh_T"]), normalise=True)
    torch.cuda.synchronize()
    check_glr(c, True, dt, o, h)
    check_glr_grads(got, c, o.cpu(), True, dt)

    n = norm_case(B, H, 20, 64, dt, 8, True, True)
    n["gate"] = n["gate"][:1].expand(B, H, 20, 64)
    n["residual"] = n["residual"][:, :, :1].expand(B, H, 20, 64)
    gate = up(n["gate"][:1].contiguous()).expand(B, H, 20, 64)
    res = up(n["residual"][:, :, :1].contiguous()).expand(B, H, 20, 64)
    y, s = kda.rms_norm(up(n["x"]), up(n["w"]), res, gate, residual_out=torch.empty(B, H, 20, 64, dtype=DT[dt], device=dev()))
    g = kda.rms_norm_backward(s, up(n["w"]), up(n["dy"]), res, gate)
    torch.cuda.synchronize()
    ref = orc.rms_norm(summed(n), n["w"], n["gate"])
    within(y, ref, (HALF[dt] + 2.0 ** -18) * ref.abs() + 1e-30)
    check_norm_grads(g, summed(n), n, n["residual"], "sigmoid", dt, 1e-6)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gaps_between_output_rows(dt):
    """Output rows inside larger ones, whose other contents stay."""
    B, H, T, d = 2, 3, 150, 64
    c = glr_case(B, H, T, d, dt, 9)

    def room():
        buf = torch.full((B, T, H, d + 8), 7.0, dtype=DT[dt], device=dev())
        return buf, buf[..., :d].transpose(1, 2)
    buf, o = room()
    _, h = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")), o=o)
    torch.cuda.synchronize()
    check_glr(c, False, dt, o, h)
    assert (buf[..., d:] == 7.0).all()
    n = norm_case(B, H, T, d, dt, 10, True, True, True)
    (b1, y), (b2, s) = room(), room()
    kda.rms_norm(up(n["x"]), up(n["w"]), up(n["residual"]), up(n["gate"]), y=y, residual_out=s)
    y1, s1 = kda.rms_norm(up(n["x"]), up(n["w"]), up(n["residual"]), up(n["gate"]))
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(s, s1) and (b1[..., d:] == 7.0).all() and (b2[..., d:] == 7.0).all()
    # in place, in such a buffer
    s.copy_(up(n["residual"]))
    y2, s2 = kda.rms_norm(up(n["x"]), up(n["w"]), s, up(n["gate"]), residual_out=s)
    torch.cuda.synchronize()
    assert torch.equal(y2, y1) and torch.equal(s, s1) and (b2[..., d:] == 7.0).all()


def far(t, gap):
    """t's values with `gap` elements between the starts of consecutive t[0], t[1], ..."""
    n = t[0].numel()
    buf = torch.empty((t.shape[0] - 1) * gap + n, dtype=t.dtype, device=dev())
    v = buf.as_strided(t.shape, (gap, *t[0].contiguous().stride()))
    v.copy_(up(t))
    return v


def test_distances_past_32_bits():
    """Sequences 2^31 + 64 elements apart, tokens 2^23 apart, rows of probabilities and states behind 2^32 bytes."""
    gap = 2 ** 31 + 64
    c = glr_case(2, 2, 300, 64, "bf16", 13)
    near = [up(c[n]) for n in ("x", "la", "beta", "h0")]
    t = {n: far(c[n], gap) for n in ("x", "la", "beta", "dO")}
    o = far(torch.zeros(2, 2, 300, 64, dtype=torch.bfloat16), gap)
    _, h = kda.glr_prefill(t["x"], t["la"], t["beta"], near[3], normalise=True, o=o)
    o1, h1 = kda.glr_prefill(*near, normalise=True)
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(h, h1)
    g1 = kda.glr_backward(*near, o1, up(c["dO"]), up(c["dh_T"]), normalise=True)
    lib = kda.load()
    outs = {n: far(torch.zeros(2, 2, 300, 64, dtype=torch.bfloat16), gap) for n in ("dx", "dlog_alpha", "dbeta")}
    dh0, ws = torch.empty_like(near[3]), torch.empty(1 << 22, dtype=torch.uint8, device=dev())
    st = kda._GlrStrides(*(kda._Strides(*x.stride()[:3]) for x in (t["x"], t["la"], t["beta"], o)))
    gst = kda._GlrGradStrides(*(kda._Strides(*x.stride()[:3]) for x in (t["dO"], outs["dx"], outs["dlog_alpha"], outs["dbeta"])))
    dh = up(c["dh_T"])
    rc = lib.kda_glr_backward(t["x"].data_ptr(), t["la"].data_ptr(), t["beta"].data_ptr(), near[3].data_ptr(), o.data_ptr(),
                              t["dO"].data_ptr(), dh.data_ptr(), None, *(x.data_ptr() for x in outs.values()), dh0.data_ptr(), st,
                              gst, 2, 2, 300, 64, 1, 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(dh0, g1["dh0"]) and all(torch.equal(outs[n], g1[n]) for n in outs)
    n = norm_case(2, 2, 9, 64, "bf16", 14, True, False)
    r = far(n["residual"], gap)
    y, s = kda.rms_norm(far(n["x"], gap), up(n["w"]), r, residual_out=r)
    y1, s1 = kda.rms_norm(up(n["x"]), up(n["w"]), up(n["residual"]))
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(s, s1)
    del t, o, outs, r, y, s

    wide = 2 ** 23  # the largest distance of tokens
    base = torch.empty(300 * wide, dtype=torch.bfloat16, device=dev())
    v = {k: base.as_strided((1, 2, 300, 64), (0, 64, wide, 1), i * 128) for i, k in enumerate(("x", "la", "beta", "o"))}
    for k in ("x", "la", "beta"):
        v[k].copy_(up(c[k][:1]))
    kda.glr_prefill(v["x"], v["la"], v["beta"], normalise=True, o=v["o"])
    o1, _ = kda.glr_prefill(*(up(c[k][:1]) for k in ("x", "la", "beta")), normalise=True)
    torch.cuda.synchronize()
    assert torch.equal(v["o"], o1)
    del base, v

    p, q, tok, u = verify_case(2, 2, 5000, "bf16", 15)
    a, out = kda.draft_verify(far(p, gap), far(q, gap), up(tok), up(u))
    torch.cuda.synchronize()
    ra, ro = orc.verify(p, q, tok, u)
    assert torch.equal(a.cpu(), ra) and torch.equal(out.cpu(), ro)

    N, ntok, H = 5, 4, 7000  # 2.3e9 floats
    S_pos = torch.empty(N, ntok, H, 128, 128, device=dev())
    for i in range(N):
        for j in range(ntok):
            S_pos[i, j] = 10 * i + j
    S = torch.full((N, H, 128, 128), -1.0, device=dev())
    idx = [3, 0, -1, 2, 3]
    kda.state_commit(S_pos, torch.tensor(idx, dtype=torch.int32, device=dev()), S)
    torch.cuda.synchronize()
    for i, j in enumerate(idx):
        assert (S[i] == (10 * i + j if j >= 0 else -1)).all()


# --------------------------------------------------------------- numbers
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rate", [1e-7, 1e-5, 1e-3, 0.06, 0.07, 0.24, 0.26])
def test_glr_constant_decays_keep_their_digits(rate, norm):
    """One decay for all tokens, whose rounding would add up over 1 / rate of them: states in fp32 from bf16 inputs."""
    B, H, T, d = 1, 1, 4000, 64
    c = glr_case(B, H, T, d, "bf16", 5)
    c["x"] = c["x"].abs()
    c["la"] = torch.full((B, H, T, d), -rate).to(torch.bfloat16)
    ref, end = orc.glr(c["x"], c["la"], c["beta"], c["h0"], norm)
    f32 = {n: (t.float() if t is not None and t.dtype == torch.bfloat16 else t) for n, t in c.items()}
    for src, dt in ((c, "bf16"), (f32, "f32")):
        o, h = kda.glr_prefill(*(up(src[n]) for n in ("x", "la", "beta", "h0")), normalise=norm)
        torch.cuda.synchronize()
        # positive inputs: errors relative to the state; bf16 carries it over 16 tiles of 256 tokens (4 roundings of 2^-24
        # each, and of the 32 lanes' sums in them), fp32 a rounding of 2^-24 a tile
        rel = float(((h.cpu().double() - end).abs() / end.abs().clamp(min=1)).max())
        assert rel <= (2.0 ** -17 if dt == "bf16" else 2.0 ** -19), (dt, rel)
        within(o, ref, HALF[dt] * ref.abs() + 2.0 ** -17 * ref.abs().clamp(min=1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_gates_at_their_ends(dt):
    """log_alpha of zero (with and without the normaliser), tiny, strong and -inf: outputs and gradients."""
    c = glr_case(1, 2, 300, 16, dt, 6)
    for t, v in ((10, 0.0), (11, -0.0), (70, -1e-30), (90, -30.0), (129, -103.0), (130, -float("inf")), (200, -300.0)):
        c["la"][:, :, t] = v
    for norm in (False, True):
        o, h = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")), normalise=norm)
        got = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), o, up(c["dO"]), up(c["dh_T"]), normalise=norm)
        torch.cuda.synchronize()
        check_glr(c, norm, dt, o, h)
        assert not got["dlog_alpha"][:, :, (130, 200)].any()
        if norm:  # 1/n of a gate of -1e-30 is 7e14
            keep = torch.ones(300, dtype=torch.bool)
            keep[70] = False
            assert torch.isfinite(got["dlog_alpha"]).all()
            got = dict(got, dlog_alpha=torch.where(keep[None, None, :, None].to(dev()), got["dlog_alpha"], 0))
            ref = orc.glr_backward(c["x"], c["la"], c["beta"], c["h0"], o.cpu(), c["dO"], c["dh_T"], True)
            rel = (got["dlog_alpha"].cpu().double() - ref["dlog_alpha"] * keep[None, None, :, None]).norm() / (ref["dlog_alpha"] * keep[None, None, :, None]).norm()
            assert rel <= (2.0 ** -8 if dt == "bf16" else 1e-6)
        else:
            check_glr_grads(got, c, o.cpu(), norm, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_what_is_not_finite_stays_in_its_channel(dt):
    """A NaN gate, an infinite input, and infinite gradients: in their channel, up to the next reset."""
    c = glr_case(1, 1, 400, 16, dt, 7)
    c["la"][0, 0, 300] = -float("inf")
    x, la, dO = c["x"].clone(), c["la"].clone(), c["dO"].clone()
    la[0, 0, 150, 2], x[0, 0, 170, 5], dO[0, 0, 350, 9] = float("nan"), float("inf"), float("inf")
    o, h = kda.glr_prefill(up(x), up(la), up(c["beta"]), up(c["h0"]))
    ref, end = orc.glr(c["x"], c["la"], c["beta"], c["h0"])
    clean = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")))[0]
    got = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), clean, up(dO), up(c["dh_T"]))
    fine = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), clean, up(c["dO"]), up(c["dh_T"]))
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 150:300, 2]).all() and not torch.isfinite(o[0, 0, 170:300, 5]).any()
    hit = torch.zeros(400, 16, dtype=torch.bool)
    hit[150:300, 2], hit[170:300, 5] = True, True
    assert torch.isfinite(o[0, 0].cpu()[~hit]).all() and torch.isfinite(h).all()
    # (a run of tokens with such a value in it is walked again: the same numbers up to that walk's zero sums)
    assert torch.equal(o[0, 0].cpu()[~hit], clean[0, 0].cpu()[~hit])
    # its gradient reaches back to the reset and no further
    assert not torch.isfinite(got["dx"][0, 0, 300:351, 9]).any()
    hit = torch.zeros(400, 16, dtype=torch.bool)
    hit[300:351, 9] = True
    for n in ("dx", "dlog_alpha", "dbeta"):
        assert torch.equal(got[n][0, 0].cpu()[~hit], fine[n][0, 0].cpu()[~hit]), n
    assert not got["dlog_alpha"][0, 0, 300].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,beta", [(100, True), (400, False), (1500, True), (17000, True), (17000, False)])
def test_glr_reset_behind_what_is_not_finite(T, beta, dt):
    """A reset any distance behind a NaN gate or input, in the same lane's tokens, the same wave's or another
    tile's: the state behind it, and the gradients in front of it, are what they are without the NaN."""
    gaps = [1, 2, 3, 5, 9, 17, 33, 60]
    d = 2 * len(gaps)
    c = glr_case(1, 1, T, d, dt, 9, beta=beta)
    start = T // 3
    for j, gap in enumerate(gaps):
        for k in (0, 1):
            c["la"][0, 0, start + gap, 2 * j + k] = -float("inf") if j % 2 else -150.0
    x, la, dO = c["x"].clone(), c["la"].clone(), c["dO"].clone()
    la[0, 0, start, 0::2], x[0, 0, start, 1::2] = float("nan"), float("nan")
    args = [up(c[n]) for n in ("x", "la", "beta", "h0")]
    clean, h0 = kda.glr_prefill(*args, normalise=True)
    o, h = kda.glr_prefill(up(x), up(la), args[2], up(c["h0"]), normalise=True)
    for j, gap in enumerate(gaps):  # a NaN that comes to the reset from behind, and a reset's own gate
        dO[0, 0, start + gap, 2 * j:2 * j + 2] = float("nan")
    fine = kda.glr_backward(*args, clean, up(c["dO"]), up(c["dh_T"]), normalise=True)
    got = kda.glr_backward(*args, clean, up(dO), up(c["dh_T"]), normalise=True)
    worse = kda.glr_backward(*args, o, up(c["dO"]), up(c["dh_T"]), normalise=True)
    torch.cuda.synchronize()
    assert torch.equal(h, h0)
    for j, gap in enumerate(gaps):
        at = slice(2 * j, 2 * j + 2)
        assert torch.isnan(o[0, 0, start:start + gap, at]).all(), gap
        assert torch.equal(o[0, 0, start + gap:, at], clean[0, 0, start + gap:, at]), gap
        for n in ("dx", "dlog_alpha", "dbeta")[:3 if beta else 2]:
            assert torch.equal(got[n][0, 0, :start + gap, at], fine[n][0, 0, :start + gap, at]), (n, gap)
        assert torch.equal(got["dh0"][0, 0, at], fine["dh0"][0, 0, at])
        assert not worse["dlog_alpha"][0, 0, start + gap, at].any()  # whatever the state in front of a reset


@pytest.mark.parametrize("scales", ["row", "block"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rms_norm_quant_extremes(fmt, scales):
    """Weights that push results to the ends of fp32: scales that would be below 2^-126, and far above 1."""
    c = norm_case(1, 1, 4, 64, "f32", 3, False, False)
    for f in (1e-37, 1e-44, 1e36):
        w = c["w"] * f
        v, sc = kda.rms_norm_quant(up(c["x"]), up(w), fmt=fmt, scales=scales)
        torch.cuda.synchronize()
        ref = orc.rms_norm(c["x"], w)
        s = sc.cpu().double() if scales == "block" else sc.cpu().double()[..., None]
        assert torch.isfinite(s).all() and (s >= 2.0 ** -126).all()
        got = (v.cpu().double().unflatten(-1, (-1, 32 if scales == "block" else 64)) * s[..., None]).flatten(-2)
        step = s.repeat_interleave(32 if scales == "block" else 64, -1) * (0.5 if fmt == "int8" else 2.0 ** -10)
        tol = step if fmt == "int8" else torch.maximum(step, 2.0 ** -4 * ref.abs())
        # (fp32 results below 2^-126 may be flushed)
        assert ((got - ref).abs() <= 1.001 * tol + 2.0 ** -17 * ref.abs() + 2.0 ** -126).all()


def test_rms_norm_rows_do_not_touch():
    """A row of zeros with eps = 0 is NaN, one with infinities too; the others are what they are alone."""
    for d, H in ((64, 5), (4096, 1), (16384, 1)):
        c = norm_case(2, H, 6, d, "bf16", d, False, False)
        x = c["x"].clone()
        x[0, 0, 1], x[1, 0, 3, 7] = 0, float("inf")
        y, ok = kda.rms_norm(up(x), up(c["w"]), eps=0.0), kda.rms_norm(up(c["x"]), up(c["w"]), eps=0.0)
        g = kda.rms_norm_backward(up(x), up(c["w"]), up(c["dy"]), eps=0.0)
        g1 = kda.rms_norm_backward(up(c["x"]), up(c["w"]), up(c["dy"]), eps=0.0)
        torch.cuda.synchronize()
        hit = torch.zeros(2, H, 6, dtype=torch.bool)
        hit[0, 0, 1], hit[1, 0, 3] = True, True
        assert torch.isnan(y[0, 0, 1]).all() and torch.isnan(y[1, 0, 3, 7])
        for a, b in ((y, ok), (g["dx"], g1["dx"])):
            assert torch.equal(a.cpu()[~hit], b.cpu()[~hit])


def test_gates_far_from_zero():
    """Gates up to 80 from zero, infinite ones, and their gradients' digits on both sides."""
    z = torch.tensor([-80.0, -20.0, -1e-3, 0.0, 1e-3, 20.0, 80.0, 200.0])
    for dt in ("bf16", "f32"):
        for act in ("sigmoid", "silu"):
            c = norm_case(1, 1, 3, 64, dt, 4, False, True)
            c["gate"] = z.repeat(24).reshape(1, 1, 3, 64).to(DT[dt])
            y = kda.rms_norm(up(c["x"]), up(c["w"]), gate=up(c["gate"]), gate_activation=act)
            g = kda.rms_norm_backward(up(c["x"]), up(c["w"]), up(c["dy"]), gate=up(c["gate"]), gate_activation=act)
            torch.cuda.synchronize()
            ref = orc.rms_norm(c["x"], c["w"], c["gate"], act)
            within(y, ref, (HALF[dt] + 2.0 ** -16) * ref.abs() + 1e-37)
            rg = orc.rms_norm_backward(c["x"], c["w"], c["dy"], None, c["gate"], act)["dgate"]
            if act == "sigmoid":  # the exponential's |z| 2^-24 in bf16: 2^-17 at 80
                within(g["dgate"], rg, (HALF[dt] + 2.0 ** -14) * rg.abs() + 1e-36, (dt, act))
    c = norm_case(1, 1, 1, 64, "f32", 5, False, True)
    c["gate"][..., 0], c["gate"][..., 1], c["gate"][..., 2] = float("inf"), -float("inf"), float("nan")
    y = kda.rms_norm(up(c["x"]), up(c["w"]), gate=up(c["gate"]))
    torch.cuda.synchronize()
    plain = orc.rms_norm(c["x"], c["w"])
    assert abs(float(y[0, 0, 0, 0]) - float(plain[0, 0, 0, 0])) <= 1e-5 and abs(float(y[0, 0, 0, 1])) <= 1e-30
    assert torch.isnan(y[0, 0, 0, 2]) and torch.isfinite(y[0, 0, 0, 3:]).all()


# ----------------------------------------------------------- empty, refused
def test_nothing_to_do():
    z = lambda *s, **k: torch.zeros(*s, device=dev(), **k)  # noqa: E731
    o, h = kda.glr_prefill(z(0, 3, 5, 8), z(0, 3, 5, 8))
    assert o.shape == (0, 3, 5, 8) and h.shape == (0, 3, 8)
    assert kda.glr_step(z(0, 3, 8), z(0, 3, 8), z(0, 3, 8)).shape == (0, 3, 8)
    assert kda.rms_norm(z(2, 3, 0, 8), z(8)).shape == (2, 3, 0, 8)
    i32 = dict(dtype=torch.int32)
    a, out = kda.draft_verify(z(0, 3, 10), z(0, 2, 10), z(0, 2, **i32), z(0, 3))
    assert a.shape == (0,) and out.shape == (0, 3)
    kda.state_commit(z(0, 3, 1, 4, 4), z(0, **i32), z(0, 1, 4, 4))
    torch.cuda.synchronize()


def test_refused_on_the_device():
    x = torch.zeros(1, 2, 3000, 8, device=dev())
    with pytest.raises(kda.KdaError, match="workspace"):
        kda.glr_prefill(x, x, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(kda.KdaError, match="contiguous rows"):
        kda.glr_prefill(x.transpose(2, 3), x.transpose(2, 3))
    with pytest.raises(kda.KdaError, match="must not be an input"):
        kda.glr_prefill(x, x.clone(), o=x)
    with pytest.raises(kda.KdaError, match="log_alpha has shape"):
        kda.glr_prefill(x, x[:, :1])
    with pytest.raises(kda.KdaError, match="gate has dtype"):
        kda.rms_norm(x, None, gate=x.bfloat16())
    with pytest.raises(kda.KdaError, match="without a residual"):
        kda.rms_norm(x, None, residual_out=x)
    with pytest.raises(kda.KdaError, match="16 bytes"):
        kda.rms_norm(torch.zeros(1, 1, 2, 9, device=dev())[..., 1:], None)
    with pytest.raises(kda.KdaError, match="tokens has dtype"):
        kda.draft_verify(torch.zeros(1, 2, 5, device=dev()), None, torch.zeros(1, 1, device=dev()), torch.zeros(1, 2, device=dev()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_check_mode(dt, kda_opts):
    """With option "check" a gate above 0 or NaN and a beta that is not finite are refused before anything is
    written; padding is not looked at."""
    c = glr_case(2, 2, 90, 16, dt, 12)
    lens = torch.tensor([90, 40], dtype=torch.int32, device=dev())
    kda_opts("check", 1)
    args = lambda t: [tm(up(t[n])) for n in ("x", "la", "beta")] + [up(t["h0"])]  # noqa: E731
    kda.glr_prefill(*args(c), lens=lens)
    for name, bad in (("la", 0.5), ("la", float("nan")), ("beta", float("inf")), ("beta", float("nan"))):
        for at, refused in (((1, 1, 39, 15), True), ((1, 0, 40, 0), False)):
            t = dict(c)
            t[name] = c[name].clone()
            t[name][at] = bad
            o = torch.full((2, 2, 90, 16), 7.0, dtype=DT[dt], device=dev())
            dO, first = up(c["dO"]), up(c["x"])
            if refused:
                for f in (lambda: kda.glr_prefill(*args(t), lens=lens, o=o),
                          lambda: kda.glr_backward(*args(t), first, dO, lens=lens)):
                    with pytest.raises(kda.KdaError) as e:
                        f()
                    assert e.value.status == ERR_PRECONDITION
                assert (o == 7.0).all()
            else:
                kda.glr_prefill(*args(t), lens=lens, o=o)
    one = [up(c[n][:, :, 0].contiguous()) for n in ("x", "la", "beta")]
    one[1][1, 1, 3] = 1.0
    h = up(c["h0"])
    with pytest.raises(kda.KdaError) as e:
        kda.glr_step(one[0], one[1], h, one[2])
    assert e.value.status == ERR_PRECONDITION and torch.equal(h.cpu(), c["h0"])
