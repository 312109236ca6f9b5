"""GPU tests of values that lie on borders or far outside the ordinary."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import layer_oracle as orc
from test_layer_ops_gpu import DT, HALF, gen, glr_case, norm_case, summed, up, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- 8-bit rows
def nearest(q, fmt):
    """fp64 values to the nearest of the format's, ties to even (all inside its range)."""
    if fmt == "int8":
        return q.round()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (q / step).round() * step


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,T,d,weight", [(1, 1, 64, 4096, True), (3, 2, 50, 64, False), (2, 1, 9, 1000, True), (1, 1, 5, 32768, True)])
def test_quantised_rows_round_to_nearest_even(B, H, T, d, weight, fmt):
    """bf16 rows without a gate: value = p L / m with p = s w of 16 bits, m the row's largest and L = 448 or 127, whatever
    the row's factor is.  A border k between two 8-bit values has at most 8 bits (e4m3: 5), and p L = k m or the two, as
    whole numbers, differ by 1 at least: 1 / (k m) > 2^-24 of k, with k below 2^8 and m below 2^16.  A quotient of fp32 is
    then on the same side of it as the exact one, or equal to it: every value can be rounded exactly, ties to even."""
    top = 448 if fmt == "e4m3" else 127
    c = norm_case(B, H, T, d, "bf16", d, True, False)
    s = summed(c)
    # half of the rows: a largest value of L and others on borders, times a power of two
    g = gen(d + 1)
    ties = nearest(torch.rand(B, H, T, d, generator=g, dtype=torch.float64) * (top - 20), fmt)
    half = 0.5 if fmt == "int8" else torch.exp2(torch.floor(torch.log2(ties.clamp(min=2.0 ** -6))) - 4)
    ties = (ties + half) * torch.where(torch.rand(B, H, T, d, generator=g) < 0.5, -1.0, 1.0)
    ties[..., 3] = top
    odd = torch.arange(T) % 2 == 1
    s[:, :, odd] = (ties * 0.125).to(torch.bfloat16)[:, :, odd]
    w = c["w"] if weight else None
    if weight:  # (powers of two keep the borders, and none above 1 the largest value)
        w = w.clamp(max=1)
        w[: d // 2] = torch.tensor([1.0, 0.5, 0.25, 1.0]).to(torch.bfloat16).repeat(d // 8)
    p = s.double() * (w.double() if weight else 1.0)
    ref = nearest(p * top / p.abs().amax(-1, keepdim=True), fmt)
    v, sc = kda.rms_norm_quant(up(s), up(w), fmt=fmt, scales="row")
    torch.cuda.synchronize()
    wrong = (v.cpu().double() != ref)
    assert not wrong.any(), (int(wrong.sum()), wrong.numel())
    want = orc.rms_norm(s, w).abs().amax(-1) / top
    assert ((sc.cpu().double() - want).abs() <= 2.0 ** -18 * want).all()


def test_quantised_rows_at_the_ends_of_fp32():
    """Rows whose products, or whose factor, are near the ends of fp32's range; the smallest scale; zeros."""
    d = 64
    x = torch.rand(1, 1, 9, d, generator=gen(1)) + 0.5
    scale = torch.tensor([1e18, 1e-18, 1e-30, 3e-39, 1.0, 1.0, 1.0, 0.0, 1e18])
    x = x * scale[:, None]
    for f, eps in ((1.0, 1e-6), (1.0, 0.0), (1e19, 1e-6), (1e-30, 1e-6), (1e-44, 1e-6)):
        w = torch.full((d,), f)
        for fmt, top in (("e4m3", 448), ("int8", 127)):
            v, sc = kda.rms_norm_quant(up(x), up(w), fmt=fmt, scales="row", eps=eps)
            torch.cuda.synchronize()
            sums = x.square().sum(-1)
            ok = (sums > 1e-30) if eps == 0.0 else torch.ones_like(sums, dtype=torch.bool)  # (squares below fp32's range are lost)
            p = x.double() * w.double()
            ok &= p.abs().amax(-1) < 3e38
            ref = orc.rms_norm(x, w, eps=eps)
            s = sc.cpu().double()[..., None]
            assert torch.isfinite(s[ok]).all() and (s[ok] >= 2.0 ** -126).all()
            got = v.cpu().double() * s
            tol = s * (0.5 if fmt == "int8" else 2.0 ** -10)
            tol = tol.expand_as(ref) if fmt == "int8" else torch.maximum(tol, 2.0 ** -4 * ref.abs())
            # (products of fp32 below 2^-126 may be flushed; the factor takes them up by at most its own size)
            r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)
            off = (got - ref).abs() - (1.001 * tol + 2.0 ** -17 * ref.abs() + 2.0 ** -126 * (1 + r))
            assert (off[ok] <= 0).all(), (f, eps, fmt)


def test_quantised_rows_of_large_products():
    """Rows whose values times weight and gate pass fp32's range, but not their norm's."""
    d = 64
    x = (torch.rand(1, 1, 3, d, generator=gen(2)) + 0.5) * torch.tensor([1e18, 1e10, 1.0])[:, None]
    gate = torch.full((1, 1, 3, d), 1e25)
    for fmt, top in (("e4m3", 448), ("int8", 127)):
        v, sc = kda.rms_norm_quant(up(x), None, gate=up(gate), gate_activation="silu", fmt=fmt, scales="row")
        torch.cuda.synchronize()
        ref, s = orc.rms_norm(x) * 1e25, sc.cpu().double()[..., None]
        assert (s / (ref.abs().amax(-1, keepdim=True) / top) - 1).abs().max() <= 2.0 ** -18
        step = s * 0.5 if fmt == "int8" else 2.0 ** -4 * ref.abs()
        assert ((v.cpu().double() * s - ref).abs() <= 1.001 * step + 2.0 ** -17 * ref.abs()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantised_rows_of_subnormal_values(dt):
    """Rows below fp32's normal numbers that their factor brings back among them."""
    d = 64
    x = ((torch.rand(1, 1, 5, d, generator=gen(3)) - 0.5) * 1e-38).to(DT[dt])
    x[..., 0] = 9e-39
    for fmt, top in (("e4m3", 448), ("int8", 127)):
        v, sc = kda.rms_norm_quant(up(x), None, fmt=fmt, scales="row", eps=1e-20)
        torch.cuda.synchronize()
        ref, s = orc.rms_norm(x, eps=1e-20), sc.cpu().double()[..., None]
        assert (s / (ref.abs().amax(-1, keepdim=True) / top) - 1).abs().max() <= 2.0 ** -18
        step = s * 0.5 if fmt == "int8" else torch.maximum(s * 2.0 ** -10, 2.0 ** -4 * ref.abs())
        assert ((v.cpu().double() * s - ref).abs() <= 1.001 * step + 2.0 ** -17 * ref.abs()).all()


# ------------------------------------------------------------------ gates
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_silu_far_from_zero(dt):
    """SiLU and its slope where the sigmoid has reached 0 or 1: z s(z) is 0 or z, the slope 0 or 1."""
    inf = float("inf")
    low, high = [-100.0, -200.0, -1e30, -1e37, -3e38, -inf], [100.0, 200.0, 1e30, 1e37, 3e38, inf]
    z = torch.tensor((low + high) * 2 + [0.0, 1.0, -1.0, 5.0, -5.0, 2.0, -2.0, 0.5]).to(DT[dt])
    d = z.numel()
    c = norm_case(1, 1, 7, d, dt, 4, False, True)
    c["gate"] = z.expand(1, 1, 7, d).contiguous()
    y = kda.rms_norm(up(c["x"]), up(c["w"]), gate=up(c["gate"]), gate_activation="silu")
    g = kda.rms_norm_backward(up(c["x"]), up(c["w"]), up(c["dy"]), gate=up(c["gate"]), gate_activation="silu")
    torch.cuda.synchronize()
    n = orc.rms_norm(c["x"], c["w"])
    zz, small = z.double(), z.double().abs() < 50
    sig = torch.sigmoid(zz)
    value = torch.where(small, zz * sig, torch.where(zz < 0, 0.0, zz))
    slope = torch.where(small, sig * (1 + zz * (1 - sig)), (zz > 0).double())
    most = torch.finfo(DT[dt]).max
    ref = n * value
    ref[(ref.abs() > 0.999 * most) | ~torch.isfinite(ref)] = float("nan")  # (an infinity, or next to one)
    # e^-87 times the bounds that the kernels take: 128 e^-87 < 2^-118 of n
    within(y, ref, (HALF[dt] + 2.0 ** -17) * ref.abs() + 2.0 ** -118 * n.abs(), "y")
    assert (y.cpu().double()[..., (zz == inf)].abs() == inf).all()
    ref = c["dy"].double() * n * slope
    within(g["dgate"], ref, HALF[dt] * ref.abs() + 2.0 ** -15 * (c["dy"].double() * n).abs() * (small | (zz > 0)) + 2.0 ** -110, "dgate")


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gates_of_nan(dt, act):
    """A gate of NaN makes its own result and gradient NaN, and its row's dx, and nothing else."""
    c = norm_case(1, 1, 5, 64, dt, 6, False, True)
    z = c["gate"].clone()
    z[0, 0, 2, 9] = float("nan")
    f = lambda gate: (kda.rms_norm(up(c["x"]), up(c["w"]), gate=up(gate), gate_activation=act),  # noqa: E731
                      kda.rms_norm_backward(up(c["x"]), up(c["w"]), up(c["dy"]), gate=up(gate), gate_activation=act))
    (y, g), (y1, g1) = f(z), f(c["gate"])
    torch.cuda.synchronize()
    hit = torch.zeros(1, 1, 5, 64, dtype=torch.bool)
    hit[0, 0, 2, 9] = True
    for a, b in ((y, y1), (g["dgate"], g1["dgate"])):
        assert torch.equal(torch.isnan(a.cpu()), hit) and torch.equal(a.cpu()[~hit], b.cpu()[~hit])
    hit[0, 0, 2] = True
    assert torch.equal(torch.isnan(g["dx"].cpu()), hit) and torch.equal(g["dx"].cpu()[~hit], g1["dx"].cpu()[~hit])
    col = torch.arange(64) == 9
    assert torch.equal(torch.isnan(g["dweight"].cpu()), col)


# ------------------------------------------------------ decays that clear
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,beta", [(1, True), (40, True), (300, False), (1500, True)])
def test_single_gates_that_clear(T, beta, dt):
    """Any log_alpha below -88 does what -inf does, bit by bit, to states that are not finite too: in a prompt, in one
    token, and in the gradients."""
    values = [-88.5, -90.0, -95.0, -103.0, -104.0, -105.0, -1e4, -3e38]
    d = 2 * len(values)
    c = glr_case(1, 2, T, d, dt, T, beta=beta)
    at = T // 2
    la, end = c["la"].clone(), c["la"].clone()
    la[:, :, at], end[:, :, at] = torch.tensor(values * 2).to(DT[dt]), -float("inf")
    x, h0 = c["x"].clone(), c["h0"].clone()
    h0[0, 0], h0[0, 1, : d // 2] = float("nan"), float("inf")
    if at:
        x[0, 1, at - 1, d // 2:] = float("nan")
    be = up(c["beta"])
    for norm in (False, True):
        got = kda.glr_prefill(up(x), up(la), be, up(h0), normalise=norm)
        ref = kda.glr_prefill(up(x), up(end), be, up(h0), normalise=norm)
        one = [t[:, :, at] if t is not None else None for t in (up(x), up(la), be)]
        h = up(h0)
        o = kda.glr_step(one[0], one[1], h, one[2], normalise=norm)
        g = kda.glr_backward(up(x), up(la), be, up(h0), ref[0], up(c["dO"]), up(c["dh_T"]), normalise=norm)
        r = kda.glr_backward(up(x), up(end), be, up(h0), ref[0], up(c["dO"]), up(c["dh_T"]), normalise=norm)
        torch.cuda.synchronize()
        assert torch.isfinite(ref[0][:, :, at:]).all() and torch.isfinite(ref[1]).all()
        assert torch.equal(got[0][:, :, at:], ref[0][:, :, at:]) and torch.equal(got[1], ref[1])
        assert torch.isfinite(h).all() and torch.isfinite(o).all()
        start = torch.zeros_like(h)
        assert torch.equal(o, kda.glr_step(one[0], one[1], start, one[2], normalise=norm)) and torch.equal(h, start)
        for n in g:
            assert torch.equal(torch.nan_to_num(g[n]), torch.nan_to_num(r[n])) and torch.equal(torch.isnan(g[n]), torch.isnan(r[n])), n
        assert not g["dlog_alpha"][:, :, at].any() and torch.isfinite(g["dh0"]).all()


# ----------------------------------------------------------------- drafts
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 40000])
def test_draft_probabilities_that_are_none(V, dt):
    """What is accepted goes by the same numbers as what is drawn: negative probabilities count as 0 and infinite ones as
    the largest number, the draft's like the target's; a NaN of either at a drafted token refuses it."""
    inf, nan = float("inf"), float("nan")
    rows = [  # target's, draft's, random number, whether it stands
        (0.0, -0.5, 0.5, False), (-0.1, -1.0, 0.5, False), (-0.5, -0.25, 0.9, False), (0.25, -0.25, 0.9, True),
        (inf, inf, 0.5, True), (inf, inf, 0.0, True), (inf, 0.5, 0.5, True), (0.25, inf, 0.5, False), (0.25, inf, 0.0, True),
        (0.25, nan, 0.0, False), (nan, 0.25, 0.5, False), (nan, -0.25, 0.5, False), (0.25, 0.25, 0.5, True), (-inf, -inf, 0.5, False),
    ]
    N = len(rows)
    p, q = torch.full((N, 2, V), 0.5 / V), torch.full((N, 1, V), 0.5 / V)
    tok, u = torch.full((N, 1), 7, dtype=torch.int32), torch.full((N, 2), 0.5)
    for i, (a, b, r, _) in enumerate(rows):
        p[i, 0, 7], q[i, 0, 7], u[i, 0] = a, b, r
    acc, out = kda.draft_verify(up(p.to(DT[dt])), up(q.to(DT[dt])), up(tok), up(u))
    torch.cuda.synchronize()
    assert acc.tolist() == [int(r[3]) for r in rows]
    for (a, b, _, stands), row in zip(rows, out.tolist()):
        assert (row[0] == 7 and 0 <= row[1] < V) if stands else (0 <= row[0] < V and row[1] == -1)
        if not stands and not a > 0:
            assert row[0] != 7  # a token of no mass
