"""GPU tests of the gated linear recurrence, the root-mean-square norm and the verification of drafted
tokens against the fp64 references in layer_oracle.py.

Tolerances, element by element.  A result in bf16 is off by half a step, 2^-8 of itself, one in fp32 by
2^-24; HALF below.
  Recurrence: a token adds at most four roundings of 2^-24 of the state's absolute recurrence H (the decay's, the
  input's product, the two of the update), so that after T tokens a state carried in fp32 is off by at
  most T 2^-22 H, H being the same recurrence over absolute values.  fp32 inputs carry the state in 64 bits:
  what is left are the decay's distance from 1 (a polynomial, 2^-22 of it, and it acts for as many tokens as it
  is small) and the input's products, 2^-22 H each, 2^-21 H together; they leave their 64 bits a few times
  where a sequence is cut.
  normalise adds n's own error, once.  fp32: 1 - a is off by 1.5 2^-24 (the exponential) of at least 0.22, 2^-21.3
  of itself (below 1/4 the polynomial's 2^-22), half of that in the root, 2^-22.3, whose own rounding is 2^-23,
  and three products: less than 2^-21 together.  bf16: from 1/16 on a is off by 1.2 2^-24, so 1 - a^2 by 2.4 2^-24
  of at least 0.117, 2^-19.6 of itself, half of that in the root, 2^-20.6, the root's rounding 2^-23 and two
  products: less than 2^-20.
  Norm: a sum of squares of positive terms takes at most 86 roundings in a row (64 in a lane, 6 over lanes, 16 over
  waves), half of that in its root, and six more products: 49 2^-24 < 2^-18 of the result.  The gradients'
  second sum adds 86 roundings of its terms' absolute sum: 2^-16 of the absolute terms.  dweight adds rows,
  at most 200 of them in a row here: 2^-16 of the absolute sum.
  Gates: the hardware's exponential and reciprocal, 2^-21 of the value for |z| < 20.
"""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import layer_oracle as orc

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


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


def within(got, ref, tol, name=""):
    got, ref = got.cpu().double(), ref.double()
    on = ~torch.isnan(ref)
    bad = (got - ref).abs()[on] > tol.expand_as(ref)[on]
    worst = ((got - ref).abs()[on] / tol.expand_as(ref)[on]).max() if on.any() else 0
    assert not bad.any() and not torch.isnan(got[on]).any(), (name, int(bad.sum()), float(worst))


# ------------------------------------------------ gated linear recurrence
def glr_case(B, H, T, d, dt, seed, beta=True, h0=True, rate=0.05):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    la = -rate * torch.exp(r(1, H, 1, d)) * torch.sigmoid(r(B, H, T, d))
    return dict(x=r(B, H, T, d).to(DT[dt]), la=la.to(DT[dt]),
                beta=torch.sigmoid(r(B, H, T, d)).to(DT[dt]) if beta else None,
                h0=r(B, H, d) if h0 else None, dO=r(B, H, T, d).to(DT[dt]), dh_T=r(B, H, d))


def glr_scale(c, norm, lens=None):
    """The recurrence over absolute values."""
    a = lambda t: None if t is None else t.abs()  # noqa: E731
    return orc.glr(a(c["x"]), c["la"], a(c["beta"]), a(c["h0"]), norm, lens)


def slack(dt, T):
    return T * 2.0 ** -22 + 2.0 ** -20 if dt == "bf16" else 2.0 ** -21 + 2.0 ** -21


def check_glr(c, norm, dt, o, h, lens=None):
    ref, end = orc.glr(c["x"], c["la"], c["beta"], c["h0"], norm, lens)
    so, sh = glr_scale(c, norm, lens)
    T = max(1, c["x"].shape[2])
    within(o, ref, HALF[dt] * ref.abs() + slack(dt, T) * so, "o")
    within(h, end, 2.0 ** -24 * end.abs() + slack(dt, T) * sh, "h_T")
    return ref


GLR = [  # B, H, T, d, dtype, beta, h0, normalise, token-major, rate
    (2, 3, 37, 16, "bf16", True, True, True, True, 0.05),
    (1, 1, 1, 8, "bf16", False, False, False, False, 0.05),
    (1, 2, 700, 64, "bf16", True, False, True, True, 0.02),
    (3, 2, 65, 32, "f32", True, True, False, False, 0.05),
    (1, 1, 1030, 128, "f32", True, True, True, True, 0.001),
    (2, 1, 129, 4, "f32", False, True, True, False, 3.0),
    (1, 5, 517, 72, "bf16", False, True, False, True, 1.0),
    (5, 1, 16, 256, "bf16", True, True, True, False, 0.3),
    (1, 1, 300, 24, "f32", False, False, False, True, 30.0),
    (2, 3, 256, 40, "bf16", True, True, True, True, 0.1),
    (2, 3, 129, 40, "bf16", True, True, False, True, 0.1),
    (2, 3, 384, 40, "bf16", False, True, False, True, 0.1),
    (2, 3, 385, 40, "bf16", False, True, False, True, 0.1),
    (9, 3, 128, 40, "bf16", True, True, True, False, 0.1),
]


@pytest.mark.parametrize("B,H,T,d,dt,beta,h0,norm,major,rate", GLR)
def test_glr_prefill(B, H, T, d, dt, beta, h0, norm, major, rate):
    print(f"[case] glr_prefill {B} {H} {T} {d} {dt}", flush=True)
    c = glr_case(B, H, T, d, dt, T + d, beta, h0, rate)
    f = (lambda t: None if t is None else tm(up(t))) if major else up
    o, h = kda.glr_prefill(f(c["x"]), f(c["la"]), f(c["beta"]), up(c["h0"]), normalise=norm)
    torch.cuda.synchronize()
    assert o.dtype == DT[dt] and h.dtype == torch.float32
    check_glr(c, norm, dt, o, h)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[0, 5, 140], [140, 1, 129], [-3, 400, 128]])
def test_glr_lens(lens, dt):
    """Rows behind a sequence's length stay as they were, whatever the inputs hold there."""
    c = glr_case(3, 2, 140, 16, dt, 5)
    bad = {n: c[n].clone() for n in ("x", "la", "beta")}
    for b, n in enumerate(orc.lengths(lens, 3, 140)):
        bad["x"][b, :, n:], bad["la"][b, :, n:], bad["beta"][b, :, n:] = float("nan"), float("inf"), float("nan")
    o = tm(torch.full((3, 2, 140, 16), 7.0, dtype=DT[dt], device=dev()))
    _, h = kda.glr_prefill(tm(up(bad["x"])), up(bad["la"]), tm(up(bad["beta"])), up(c["h0"]), normalise=True, o=o,
                           lens=torch.tensor(lens, dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    ref = check_glr(c, True, dt, o, h, lens)
    assert (o.cpu().double()[torch.isnan(ref)] == 7.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_glr_long(norm, beta, dt):
    """More than 16384 tokens, where the runs of tokens are longer; channels that end inside a slab, a ragged batch."""
    T = 16384 + 777
    lens = [T, 9001, 16384]
    c = glr_case(3, 3, T, 24, dt, 77, beta=beta)
    c["la"][:, :, 5000:5003] = -float("inf")
    ln = torch.tensor(lens, dtype=torch.int32, device=dev())
    args = [up(c[n]) for n in ("x", "la", "beta", "h0")]
    o = torch.zeros(3, 3, T, 24, dtype=DT[dt], device=dev())
    _, h = kda.glr_prefill(*args, normalise=norm, o=o, lens=ln)
    got = kda.glr_backward(*args, o, up(c["dO"]), up(c["dh_T"]), normalise=norm, lens=ln)
    torch.cuda.synchronize()
    check_glr(c, norm, dt, o, h, lens)
    check_glr_grads(got, c, o.cpu(), norm, dt, lens)


def test_glr_no_tokens():
    h0 = torch.randn(2, 3, 8, generator=gen(1)).to(dev())
    x = torch.empty(2, 3, 0, 8, device=dev())
    assert torch.equal(kda.glr_prefill(x, x, x, h0)[1], h0)
    assert not kda.glr_prefill(x, x)[1].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_resets_clear_everything(dt):
    """A decay of zero starts anew, also behind states of infinity and NaN."""
    c = glr_case(1, 2, 300, 16, dt, 3)
    for t, v in ((0, -float("inf")), (64, -200.0), (128, -float("inf")), (257, -float("inf"))):
        c["la"][:, :, t] = v
    x = c["x"].clone()
    x[0, 0, 100], x[0, 1, 200, 3] = float("inf"), float("nan")
    h0 = torch.full_like(c["h0"], float("nan"))
    o, h = kda.glr_prefill(up(x), up(c["la"]), up(c["beta"]), up(h0))
    torch.cuda.synchronize()
    c["h0"] = None
    ref, end = orc.glr(c["x"], c["la"], c["beta"])
    so, sh = glr_scale(c, False)
    hit = torch.zeros_like(ref, dtype=torch.bool)
    hit[0, 0, 100:128], hit[0, 1, 200:257, 3] = True, True
    assert not torch.isfinite(o.cpu()[hit]).any()
    ref[hit] = float("nan")
    within(o, ref, HALF[dt] * ref.abs() + slack(dt, 300) * so)
    within(h, end, 2.0 ** -24 * end.abs() + slack(dt, 300) * sh)


@pytest.mark.parametrize("N,H,d,dt,beta,norm", [(1, 1, 8, "bf16", False, False), (7, 3, 40, "bf16", True, True),
                                               (33, 2, 4, "f32", True, True), (260, 4, 128, "bf16", True, False)])
def test_glr_step(N, H, d, dt, beta, norm):
    c = glr_case(N, H, 1, d, dt, 9, beta)
    h = up(c["h0"])
    one = lambda t: None if t is None else up(t)[:, :, 0]  # noqa: E731
    o = kda.glr_step(one(c["x"]), one(c["la"]), h, one(c["beta"]), normalise=norm)
    torch.cuda.synchronize()
    check_glr(c, norm, dt, o[:, :, None], h)


def test_glr_steps_follow_the_prompt():
    c = glr_case(4, 2, 9, 16, "f32", 2)
    x, la, beta = (up(c[n]) for n in ("x", "la", "beta"))
    full, end = kda.glr_prefill(x, la, beta, up(c["h0"]), normalise=True)
    _, h = kda.glr_prefill(x[:, :, :5], la[:, :, :5], beta[:, :, :5], up(c["h0"]), normalise=True)
    for t in range(5, 9):
        o = kda.glr_step(x[:, :, t], la[:, :, t], h, beta[:, :, t], normalise=True)
        torch.cuda.synchronize()
        within(o, full[:, :, t].cpu(), 2.0 ** -20 * (1 + full[:, :, t].cpu().double().abs()))
    within(h, end.cpu(), 2.0 ** -20 * (1 + end.cpu().double().abs()))


def check_glr_grads(got, c, o, norm, dt, lens=None, dh_T=True):
    args = (c["x"], c["la"], c["beta"], c["h0"], o, c["dO"], c["dh_T"] if dh_T else None, norm, lens)
    ref = orc.glr_backward(*args)
    names = {"dx", "dlog_alpha"} | ({"dbeta"} if c["beta"] is not None else set()) | ({"dh0"} if c["h0"] is not None else set())
    assert set(got) == names
    # absolute terms: with every factor positive but the normaliser's part of dlog_alpha, which is added
    a = lambda t: None if t is None else t.abs()  # noqa: E731
    top = orc.glr_backward(a(c["x"]), c["la"], a(c["beta"]), a(c["h0"]), a(o), a(c["dO"]), a(c["dh_T"]) if dh_T else None,
                           False, lens)
    T = c["x"].shape[2]
    la = c["la"].double()
    n = torch.sqrt(-torch.expm1(2 * la)) if norm else torch.ones_like(la)
    if norm:
        top["dx"], top["dbeta"] = top["dx"] * n, top["dbeta"] * n
        al = torch.exp(la)
        part = torch.where(n > 0, al * al / n, 0.0) * top["dx"] / torch.where(n > 0, n, 1.0) * c["x"].double().abs()
        top["dlog_alpha"] = top["dlog_alpha"] + part
    for k in names:
        half = 2.0 ** -24 if k == "dh0" else HALF[dt]
        within(got[k], ref[k], half * ref[k].abs() + (slack(dt, T) + 2.0 ** -20) * top[k] + 1e-37, k)


@pytest.mark.parametrize("B,H,T,d,dt,beta,h0,norm,major,rate", GLR)
def test_glr_backward(B, H, T, d, dt, beta, h0, norm, major, rate):
    print(f"[case] glr_backward {B} {H} {T} {d} {dt}", flush=True)
    c = glr_case(B, H, T, d, dt, 2 * T + d, beta, h0, rate)
    f = (lambda t: None if t is None else tm(up(t))) if major else up
    o, _ = kda.glr_prefill(f(c["x"]), f(c["la"]), f(c["beta"]), up(c["h0"]), normalise=norm)
    got = kda.glr_backward(f(c["x"]), f(c["la"]), f(c["beta"]), up(c["h0"]), o, f(c["dO"]), up(c["dh_T"]),
                           normalise=norm)
    torch.cuda.synchronize()
    check_glr_grads(got, c, o.cpu(), norm, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[0, 5, 140], [140, 1, 129], [-3, 400, 128]])
def test_glr_backward_lens(lens, dt):
    """Padding gets zero gradients and passes dh_T on, whatever the inputs hold there."""
    c = glr_case(3, 2, 140, 16, dt, 6)
    o, _ = orc.glr(c["x"], c["la"], c["beta"], c["h0"], True, lens)
    bad = {n: c[n].clone() for n in ("x", "la", "beta", "dO")}
    for b, n in enumerate(orc.lengths(lens, 3, 140)):
        for k in bad:
            bad[k][b, :, n:] = float("nan")
    got = kda.glr_backward(up(bad["x"]), tm(up(bad["la"])), up(bad["beta"]), up(c["h0"]), up(o.to(DT[dt])),
                           tm(up(bad["dO"])), up(c["dh_T"]), normalise=True,
                           lens=torch.tensor(lens, dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    check_glr_grads(got, c, torch.nan_to_num(o.to(DT[dt])), True, dt, lens)


def test_glr_gradients_by_differences():
    """d loss / d input along random directions, fp32, against central differences of the kernel's own outputs
    held in fp64 by the reference."""
    c = glr_case(1, 2, 40, 8, "f32", 4, rate=0.3)
    o, _ = kda.glr_prefill(*(up(c[n]) for n in ("x", "la", "beta", "h0")), normalise=True)
    got = kda.glr_backward(*(up(c[n]) for n in ("x", "la", "beta", "h0")), o, up(c["dO"]), up(c["dh_T"]), normalise=True)
    torch.cuda.synchronize()

    def loss(**k):
        v = {**{n: c[n].double() for n in ("x", "la", "beta", "h0")}, **k}
        y, h = orc.glr(v["x"], v["la"], v["beta"], v["h0"], True)
        return float((y * c["dO"].double()).sum() + (h * c["dh_T"].double()).sum())
    for n, g in (("x", "dx"), ("la", "dlog_alpha"), ("beta", "dbeta"), ("h0", "dh0")):
        u = torch.randn(c[n].shape, generator=gen(8), dtype=torch.float64)
        step = 1e-6
        diff = (loss(**{n: c[n].double() + step * u}) - loss(**{n: c[n].double() - step * u})) / (2 * step)
        size = float((got[g].cpu().double() * u).abs().sum())
        # differences: 1e-16 / 1e-6 of the loss's terms; gradients: 2^-19 of their terms
        assert abs(float((got[g].cpu().double() * u).sum()) - diff) <= 2.0 ** -18 * size + 1e-6, n


# ------------------------------------------------------------------- norm
def norm_case(B, H, T, d, dt, seed, residual, gate, per_head=False):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(B, H, T, d).to(DT[dt]), w=(1 + 0.3 * (r(H, d) if per_head else r(d))).to(DT[dt]),
                residual=(2 * r(B, H, T, d)).to(DT[dt]) if residual else None,
                gate=(2 * r(B, H, T, d)).to(DT[dt]) if gate else None, dy=r(B, H, T, d).to(DT[dt]),
                ds=r(B, H, T, d).to(DT[dt]))


def summed(c):
    return c["x"] if c["residual"] is None else (c["x"].float() + c["residual"].float()).to(c["x"].dtype)


NORM = [  # B, H, T, d, dtype, residual, gate, activation, weight per head, token-major
    (2, 3, 5, 8, "bf16", True, True, "sigmoid", True, True),
    (1, 1, 1, 16, "bf16", False, False, "sigmoid", False, False),
    (3, 4, 7, 64, "bf16", False, True, "silu", False, True),
    (2, 5, 33, 128, "bf16", True, True, "sigmoid", False, True),
    (2, 2, 9, 200, "f32", True, False, "sigmoid", True, False),
    (5, 3, 1, 264, "bf16", True, True, "silu", False, False),
    (1, 2, 11, 520, "f32", False, True, "sigmoid", False, True),
    (1, 1, 37, 1000, "bf16", True, False, "sigmoid", False, False),
    (2, 1, 3, 2048, "f32", True, True, "silu", False, False),
    (1, 1, 5, 4096, "bf16", True, False, "sigmoid", False, False),
    (1, 1, 3, 8200, "bf16", True, True, "sigmoid", False, False),
    (1, 2, 2, 16384, "f32", False, False, "sigmoid", True, False),
    (1, 1, 2, 32768, "bf16", True, False, "sigmoid", False, False),
    (1, 1, 1, 32768, "f32", True, True, "silu", False, False),
]


@pytest.mark.parametrize("B,H,T,d,dt,residual,gate,act,per_head,major", NORM)
def test_rms_norm(B, H, T, d, dt, residual, gate, act, per_head, major):
    print(f"[case] rms_norm {B} {H} {T} {d} {dt}", flush=True)
    c = norm_case(B, H, T, d, dt, d, residual, gate, per_head)
    f = (lambda t: None if t is None else tm(up(t))) if major else up
    got = kda.rms_norm(f(c["x"]), up(c["w"]), f(c["residual"]), up(c["gate"]), gate_activation=act, eps=1e-5)
    torch.cuda.synchronize()
    y, s = got if residual else (got, None)
    if residual:
        assert torch.equal(s.cpu(), summed(c))
    ref = orc.rms_norm(summed(c), c["w"], c["gate"], act, 1e-5)
    within(y, ref, (HALF[dt] + 2.0 ** -18) * ref.abs() + 1e-30)


def test_rms_norm_residual_in_place_and_no_weight():
    c = norm_case(2, 1, 9, 256, "bf16", 3, True, False)
    r = up(c["residual"])
    y, s = kda.rms_norm(up(c["x"]), None, r, residual_out=r)
    torch.cuda.synchronize()
    assert s.data_ptr() == r.data_ptr() and torch.equal(r.cpu(), summed(c))
    ref = orc.rms_norm(summed(c))
    within(y, ref, (HALF["bf16"] + 2.0 ** -18) * ref.abs())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("scales", ["row", "block"])
@pytest.mark.parametrize("B,H,T,d,dt,gate,major", [(2, 3, 5, 32, "bf16", True, True), (1, 1, 9, 256, "f32", False, False),
                                                   (2, 2, 3, 608, "bf16", True, True), (1, 1, 3, 4096, "bf16", False, False),
                                                   (1, 1, 2, 8224, "f32", True, False)])
def test_rms_norm_quant(B, H, T, d, dt, gate, major, scales, fmt):
    """The values times their scale lie within half a step of the exact ones, and the scales are the smallest
    that hold them."""
    print(f"[case] rms_norm_quant {B} {H} {T} {d} {dt} {scales} {fmt}", flush=True)
    c = norm_case(B, H, T, d, dt, d + 1, True, gate)
    c["x"][0, 0, 0, :32] *= 100.0
    if T > 1:  # a row of zeros
        c["x"][0, 0, 1] = 0
        c["residual"][0, 0, 1] = 0
    f = (lambda t: None if t is None else tm(up(t))) if major else up
    v, sc, s = kda.rms_norm_quant(f(c["x"]), up(c["w"]), f(c["residual"]), up(c["gate"]), fmt=fmt, scales=scales)
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), summed(c)) and v.stride() == f(c["x"]).stride()
    ref = orc.rms_norm(summed(c), c["w"], c["gate"])
    top = 448.0 if fmt == "e4m3" else 127.0
    n = 32 if scales == "block" else d
    scale = sc.cpu().double() if scales == "block" else sc.cpu().double()[..., None]
    got, m = v.cpu().double().unflatten(-1, (-1, n)), ref.unflatten(-1, (-1, n))
    most, off = m.abs().amax(-1), 2.0 ** -18
    if scales == "row":
        want = (most / top).clamp(min=2.0 ** -126)
        assert ((scale - want).abs() <= off * want).all()
    else:
        assert (most * (1 - off) <= top * scale).all()
        assert ((most * (1 + off) > top * scale / 2) | (scale == 2.0 ** -126)).all()
    step = scale[..., None] * (0.5 if fmt == "int8" else 2.0 ** -10)
    tol = step if fmt == "int8" else torch.maximum(step, 2.0 ** -4 * m.abs())
    assert ((got * scale[..., None] - m).abs() <= tol * (1 + 2.0 ** -15) + 2 * off * m.abs()).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("scales", ["row", "block"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rms_norm_marks_what_is_not_finite(bad, scales, fmt):
    """A row with an infinity or NaN in it is marked; its neighbours are not touched."""
    c = norm_case(1, 1, 7, 64, "bf16", 1, False, True)
    x, g = c["x"].clone(), c["gate"].clone()
    x[0, 0, 2, 5] = bad
    g[0, 0, 4, 40] = float("nan")
    v, sc = kda.rms_norm_quant(up(x), up(c["w"]), gate=up(g), fmt=fmt, scales=scales)
    ok, osc = kda.rms_norm_quant(up(c["x"]), up(c["w"]), gate=up(c["gate"]), fmt=fmt, scales=scales)
    torch.cuda.synchronize()
    whole = [0, 1, 3, 5, 6]
    as_bytes = lambda t: t.cpu().view(torch.uint8)[0, 0]  # noqa: E731
    assert torch.equal(as_bytes(v)[whole], as_bytes(ok)[whole])
    marked = torch.isnan(sc.cpu().float())[0, 0]
    if scales == "row":
        assert marked.tolist() == [i in (2, 4) for i in range(7)]
    else:
        # (an infinity makes its row's factor zero: the block that holds it is marked, the other may be zero)
        assert marked[4].tolist() == [False, True] and marked[2, 0] and not marked[whole].any()
    assert not as_bytes(v)[2][:32].any()


@pytest.mark.parametrize("B,H,T,d,dt,residual,gate,act,per_head,major", NORM)
def test_rms_norm_backward(B, H, T, d, dt, residual, gate, act, per_head, major):
    print(f"[case] rms_norm_backward {B} {H} {T} {d} {dt}", flush=True)
    c = norm_case(B, H, T, d, dt, d + 2, residual, gate, per_head)
    f = (lambda t: None if t is None else tm(up(t))) if major else up
    s, ds = summed(c), c["ds"] if residual else None
    got = kda.rms_norm_backward(f(s), up(c["w"]), up(c["dy"]), f(ds), f(c["gate"]), gate_activation=act, eps=1e-5)
    torch.cuda.synchronize()
    check_norm_grads(got, s, c, ds, act, dt, 1e-5)


def check_norm_grads(got, s, c, ds, act, dt, eps):
    ref = orc.rms_norm_backward(s, c["w"], c["dy"], ds, c["gate"], act, eps)
    assert set(got) == {"dx", "dweight"} | ({"dgate"} if c["gate"] is not None else set())
    sd, dy, w = s.double(), c["dy"].double(), orc._rows(c["w"], s)
    r = 1 / torch.sqrt(sd.square().mean(-1, keepdim=True) + eps)
    g = torch.ones_like(sd) if c["gate"] is None else orc.gate_factor(c["gate"].double(), act)
    dn = (dy * w * g).abs()
    top = r * (dn + (sd * r).abs() * (dn * (sd * r).abs()).mean(-1, keepdim=True))
    within(got["dx"], ref["dx"], HALF[dt] * ref["dx"].abs() + 2.0 ** -16 * top + (2.0 ** -24 * ds.double().abs() if ds is not None else 0), "dx")
    per = (dy * sd * r * g).abs()
    per = per.sum((0, 2)) if c["w"].dim() == 2 else per.sum((0, 1, 2))
    within(got["dweight"], ref["dweight"], HALF[dt] * ref["dweight"].abs() + 2.0 ** -16 * per, "dweight")
    if c["gate"] is not None:
        sig = 1 / (1 + torch.exp(-c["gate"].double()))
        z = c["gate"].double()
        slope = sig * (1 - sig) if act == "sigmoid" else sig * (1 + (z * (1 - sig)).abs())
        within(got["dgate"], ref["dgate"], HALF[dt] * ref["dgate"].abs() + 2.0 ** -16 * (dy * sd * r * w).abs() * slope + 1e-30, "dgate")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rms_norm_backward_many_rows(dt):
    """More rows than blocks take at once, dealt unevenly, and a weight per head."""
    for shape, per_head in (((3, 5, 701, 64), True), ((2, 1, 2500, 136), False), ((1, 3, 3100, 512), True)):
        c = norm_case(*shape, dt, 5, False, False, per_head)
        got = kda.rms_norm_backward(up(c["x"]), up(c["w"]), up(c["dy"]))
        torch.cuda.synchronize()
        check_norm_grads(got, c["x"], c, None, "sigmoid", dt, 1e-6)


# ----------------------------------------------------------------- drafts
def verify_case(N, K, V, dt, seed, sharp=3.0):
    g = gen(seed)
    t = torch.randn(N, K + 1, V, generator=g) * sharp
    q = t[:, :K] + torch.randn(N, K, V, generator=g)
    p, q = torch.softmax(t, -1).to(DT[dt]), torch.softmax(q, -1).to(DT[dt])
    tok = torch.multinomial(q.reshape(-1, V).float(), 1, generator=g).reshape(N, K).to(torch.int32) if K else torch.zeros(N, 0, dtype=torch.int32)
    return p, q, tok, torch.rand(N, K + 1, generator=g)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (3, 4, 7), (40, 3, 257), (9, 0, 1000), (5, 70, 33), (17, 5, 8192), (6, 2, 50257),
                                   (2, 1, 150001), (256, 2, 40), (257, 2, 40), (2, 3, 32768), (2, 3, 32769)])
def test_draft_verify(N, K, V, dt):
    print(f"[case] draft_verify {N} {K} {V} {dt}", flush=True)
    p, q, tok, u = verify_case(N, K, V, dt, N + V)
    for draft in (q, None):
        if draft is None and K:
            tok = p[:, :K].argmax(-1).to(torch.int32)
        a, out = kda.draft_verify(up(p), up(draft), up(tok), up(u))
        torch.cuda.synchronize()
        ra, ro = orc.verify(p, draft, tok, u)
        assert torch.equal(a.cpu(), ra) and torch.equal(out.cpu(), ro)


def test_draft_verify_counts_and_strides():
    """Unequal numbers of drafts; rows inside larger arrays, at odd addresses."""
    p, q, tok, u = verify_case(8, 4, 301, "bf16", 3)
    counts = torch.tensor([0, 1, 2, 3, 4, 9, -2, 4], dtype=torch.int32)
    P = torch.full((8, 7, 310), 0.5, dtype=torch.bfloat16, device=dev())
    Q = torch.full((9, 8, 305), 0.5, dtype=torch.bfloat16, device=dev())
    P[:, 1:6, 3:304], Q[1:, 2:6, 1:302] = up(p), up(q)
    a, out = kda.draft_verify(P[:, 1:6, 3:304], Q[1:, 2:6, 1:302], up(tok), up(u), counts=up(counts))
    torch.cuda.synchronize()
    ra, ro = orc.verify(p, q, tok, u, counts)
    assert torch.equal(a.cpu(), ra) and torch.equal(out.cpu(), ro)
    # one row of probabilities for every sequence and draft
    a, out = kda.draft_verify(up(p[:1, :1]).expand(8, 5, 301), up(q[:1, :1]).expand(8, 4, 301), up(tok), up(u))
    torch.cuda.synchronize()
    ra, ro = orc.verify(p[:1, :1].expand(8, 5, 301), q[:1, :1].expand(8, 4, 301), tok, u)
    assert torch.equal(a.cpu(), ra) and torch.equal(out.cpu(), ro)


@pytest.mark.parametrize("V", [20000, 40000])
def test_draft_verify_borders(V):
    """Uniforms of 0 and just below 1, masses only at the ends, equal distributions, none at all, tokens outside
    the vocabulary, NaN."""
    K = 2
    z = torch.zeros(10, K + 1, V)
    q = torch.zeros(10, K, V)
    tok = torch.zeros(10, K, dtype=torch.int32)
    u = torch.full((10, K + 1), 0.5)
    z[0, :, 0], z[1, :, V - 1], z[2, :, [0, V - 1]] = 1, 1, 0.5
    u[2, K] = 1 - 2.0 ** -24
    z[3, :, [5, 9000]] = 0.5
    u[3, K] = 0.0
    z[4], q[4] = 1.0 / 32768, 1.0 / 32768  # equal: a refusal (u q < p fails for u = 1) draws from p
    u[4, 0] = 1.0
    tok[5] = torch.tensor([-1, V])  # no such token
    z[5, :, 77] = 1
    z[6, 0, 3], q[6, 0, 3], tok[6, 0] = float("nan"), 0.5, 3
    z[6, 0, 11] = 0.25
    z[7, 0, 4], q[7, 0, 4], tok[7, 0] = 0.0, 0.0, 4  # 0 < 0 fails; nothing is left of row 0
    z[8, :, 1000:3000] = 1.0 / 2000
    u[8, K] = 0.75
    tok[9], z[9, :, V - 2] = V - 2, 1
    q[9, :, V - 2] = 1
    for dt in ("f32", "bf16"):
        args = (z.to(DT[dt]), q.to(DT[dt]), tok, u)
        a, out = kda.draft_verify(*map(up, args))
        torch.cuda.synchronize()
        ra, ro = orc.verify(*args)
        assert torch.equal(a.cpu(), ra) and torch.equal(out.cpu(), ro), dt
    assert out[7].tolist() == [-1, -1, -1] and out[2].tolist() == [0, 0, V - 1] and int(a[9]) == 2


@pytest.mark.parametrize("V", [300, 40000])
def test_draft_verify_infinities(V):
    """An infinite probability counts as the largest number: the next token is that one, unless the draft's is too."""
    p, q = torch.full((3, 2, V), 1.0 / V), torch.zeros(3, 1, V)
    p[:, 0, 7] = float("inf")
    p[:, 0, 0] = 0.0
    q[1, 0, 7], q[2, 0, 7] = 0.5, float("inf")
    tok = torch.zeros(3, 1, dtype=torch.int32)  # refused: its probability is 0
    u = torch.full((3, 2), 0.5)
    a, out = kda.draft_verify(*map(up, (p, q, tok, u)))
    torch.cuda.synchronize()
    assert not a.any() and out[:2, 0].tolist() == [7, 7] and (out[:, 1] == -1).all()
    # (behind token 7 the others' V - 2 equal masses: half of them)
    assert abs(out[2, 0].item() - V // 2) <= 1 and out[2, 0] != 7


@pytest.mark.parametrize("N,ntok,H,dk,dv", [(1, 1, 1, 2, 2), (5, 3, 2, 64, 64), (7, 4, 3, 128, 64), (3, 2, 1, 6, 10)])
def test_state_commit(N, ntok, H, dk, dv):
    g = gen(N)
    pos, S = torch.randn(N, ntok, H, dk, dv, generator=g), torch.randn(N, H, dk, dv, generator=g)
    idx = torch.randint(-1, ntok + 1, (N,), generator=g).to(torch.int32)
    got = up(S)
    kda.state_commit(up(pos), up(idx), got)
    torch.cuda.synchronize()
    ref = torch.stack([pos[n, t] if 0 <= t < ntok else S[n] for n, t in enumerate(idx.tolist())])
    assert torch.equal(got.cpu(), ref)


def test_drafts_through_a_layer():
    """A serving step with drafts: norm, convolution and both recurrences over the last token and the drafts,
    verification, and every state moved to the accepted ones; then the next token gives what it gives
    after those tokens alone."""
    N, H, d, K, V = 6, 2, 64, 3, 500
    T, g = K + 1, gen(11)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = lambda t: up(t.to(torch.bfloat16))  # noqa: E731
    stream, w = bf(r(N, 1, T + 1, H * d)), bf(1 + 0.1 * r(H * d))
    taps, cs = bf(r(H, d, 4) * 0.5), bf(r(N, H, 3, d))
    la, beta = bf(-torch.sigmoid(r(N, H, T + 1, d))), bf(torch.sigmoid(r(N, H, T + 1, d)))
    sb, q = bf(torch.sigmoid(r(N, H, T + 1))), bf(torch.nn.functional.normalize(r(N, H, T + 1, d), dim=-1))
    h, S = up(r(N, H, d)), up(0.1 * r(N, H, d, d))
    hw = bf(1 + 0.1 * r(d))

    def layer(t0, t1, state, h_in, S_in, lens=None, positions=False):
        """Tokens t0 .. t1 from the given states."""
        n = t1 - t0
        cut = lambda t: t[:, :, t0:t1].contiguous()  # noqa: E731
        y = kda.rms_norm(cut(stream), w)
        x = y.view(N, n, H, d).transpose(1, 2)
        c, c_out = kda.conv_prefill(x, taps, state=state, lens=lens)
        o1, h_out = kda.glr_prefill(c, cut(la), cut(beta), h_in, normalise=True, lens=lens)
        o2, pos = kda.decode_tokens(cut(q), cut(q), c, cut(la), cut(sb), S_in, positions=positions)
        return kda.rms_norm(o2, hw, gate=o1), c_out, h_out, pos

    p, dq, tok, u = verify_case(N, K, V, "f32", 5)
    S_run = S.clone()
    _, _, _, pos = layer(0, T, cs, h, S_run, positions=True)
    acc, out = kda.draft_verify(up(p), up(dq), up(tok), up(u))
    kda.state_commit(pos, acc, S_run)
    keep = acc + 1  # the last verified token and the accepted drafts
    _, c_new, h_new, _ = layer(0, T, cs, h, S.clone(), lens=keep)
    y, *_ = layer(T, T + 1, c_new, h_new, S_run)
    torch.cuda.synchronize()
    assert len(set(acc.tolist())) > 1
    for n, k in enumerate(keep.tolist()):
        S1 = S.clone()
        _, c1, h1, _ = layer(0, k, cs, h, S1)
        y1, *_ = layer(T, T + 1, c1, h1, S1)
        torch.cuda.synchronize()
        assert torch.equal(c1[n], c_new[n]) and torch.equal(S1[n], S_run[n])
        assert (h1[n] - h_new[n]).abs().max() <= 2.0 ** -20 * (1 + h1[n].abs().max())
        assert (y1[n].float() - y[n].float()).abs().max() <= 2.0 ** -7 * y1[n].float().abs().max()


def test_training_step_through_a_layer():
    """norm, convolution, recurrence and gated head norm forwards and backwards, against autograd in fp64 on the
    same formulas."""
    B, H, T, d, K = 2, 2, 90, 16, 3
    g = gen(21)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=r(B, 1, T, H * d), res=r(B, 1, T, H * d), w=1 + 0.1 * r(H * d), taps=r(H, d, K) * 0.5,
             la=-0.2 * torch.sigmoid(r(B, H, T, d)), beta=torch.sigmoid(r(B, H, T, d)), hw=1 + 0.1 * r(H, d), z=r(B, H, T, d))
    dy, ds = r(B, H, T, d), r(B, 1, T, H * d)
    v = {k: up(t) for k, t in c.items()}
    y, s = kda.rms_norm(v["x"], v["w"], v["res"])
    heads = y.view(B, T, H, d).transpose(1, 2)
    u, _ = kda.conv_prefill(heads, v["taps"])
    o, _ = kda.glr_prefill(u, v["la"], v["beta"], normalise=True)
    out = kda.rms_norm(o, v["hw"], gate=v["z"])
    g3 = kda.rms_norm_backward(o, v["hw"], up(dy), gate=v["z"])
    g2 = kda.glr_backward(u, v["la"], v["beta"], None, o, g3["dx"], normalise=True)
    g1 = kda.conv_backward(heads, v["taps"], None, None, g2["dx"])
    g0 = kda.rms_norm_backward(s, v["w"], g1["dx"].transpose(1, 2).reshape(B, 1, T, H * d), up(ds))
    torch.cuda.synchronize()
    got = dict(x=g0["dx"], res=g0["dx"], w=g0["dweight"], taps=g1["dweight"], la=g2["dlog_alpha"], beta=g2["dbeta"],
               hw=g3["dweight"], z=g3["dgate"])
    p = {k: t.double().requires_grad_() for k, t in c.items()}
    rn = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    s64 = p["x"] + p["res"]
    hd = (rn(s64) * p["w"]).view(B, T, H, d).transpose(1, 2)
    e = torch.nn.functional.pad(hd, (0, 0, K - 1, 0))
    u64 = torch.nn.functional.silu(sum(p["taps"][:, None, :, k] * e[:, :, k:k + T] for k in range(K)))
    h, hs = torch.zeros(B, H, d, dtype=torch.float64), []
    for t in range(T):
        la = p["la"][:, :, t]
        h = torch.exp(la) * h + torch.sqrt(-torch.expm1(2 * la)) * p["beta"][:, :, t] * u64[:, :, t]
        hs.append(h)
    out64 = rn(torch.stack(hs, 2)) * p["hw"][:, None] * torch.sigmoid(p["z"])
    ref = torch.autograd.grad((out64 * dy.double()).sum() + (s64 * ds.double()).sum(), list(p.values()))
    # fp32 throughout: a few hundred roundings of 2^-24 on norms
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, out64.detach()) <= 1e-5
    for k, b in zip(p, ref):
        assert rel(got[k], b) <= 1e-5, k
