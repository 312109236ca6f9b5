"""GPU tests of outputs that are written past the caches (at least 32 MiB of rows of whole 128-byte lines): bit by bit
what the same call writes into rows with gaps, which take ordinary stores, and a share of it against the fp64 references;
with values that are not finite, whose runs of tokens the recurrence walks twice."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import layer_oracle as orc
from test_layer_ops_gpu import DT, HALF, check_glr_grads, check_norm_grads, dev, slack, within

pytestmark = pytest.mark.gpu


def draw(seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device=dev())


def gapped(B, H, T, d, dt, gap=8):
    """Rows with gaps whose distance is no whole number of lines, and whether the gaps still hold what they held."""
    buf = torch.full((B, H, T, d + gap), 7.0, dtype=dt, device=dev())
    return buf[..., :d], lambda: bool((buf[..., d:] == 7.0).all())


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def streamed(t):
    """The rule by which outputs are written past the caches."""
    e = t.element_size()
    return t.numel() * e >= 32 << 20 and all(n * e % 128 == 0 for n in (t.data_ptr() // e, t.shape[-1], *t.stride()[:3]))


GLR = [  # B, H, T, dtype, beta, normalise: the tokens a lane differ
    (2, 120, 1100, "bf16", True, True), (2, 120, 1100, "bf16", False, True), (2, 120, 1100, "bf16", False, False),
    (1, 16, 16500, "bf16", True, True), (1, 16, 16500, "bf16", False, True), (2, 60, 1100, "f32", True, True),
    (2, 60, 1100, "f32", False, False),
]


@pytest.mark.parametrize("B,H,T,dt,beta,norm", GLR)
def test_recurrence(B, H, T, dt, beta, norm):
    print(f"[case] streaming recurrence {B} {H} {T} {dt}", flush=True)
    d, r = 64, draw(T + H)
    x, dO = (r(B, H, T, d).to(DT[dt]) for _ in range(2))
    la = (-0.05 * torch.exp(r(1, H, 1, d)) * torch.sigmoid(r(B, H, T, d))).to(DT[dt])
    be = torch.sigmoid(r(B, H, T, d)).to(DT[dt]) if beta else None
    h0, dh = r(B, H, d), r(B, H, d)
    lens = torch.tensor([T, T - 37][:B], dtype=torch.int32, device=dev())
    # head 3: an input of infinity, a gate of NaN, an infinite gradient, and resets behind and in front of them
    x[0, 3, 200, 5], la[0, 3, 210, 6], dO[0, 3, 700, 7] = float("inf"), float("nan"), float("inf")
    la[0, 3, [260, 600]] = -float("inf")

    o = torch.zeros(B, H, T, d, dtype=DT[dt], device=dev())
    o2, kept = gapped(B, H, T, d, DT[dt])
    o2.zero_()
    assert streamed(o) and not streamed(o2)
    _, h = kda.glr_prefill(x, la, be, h0, normalise=norm, lens=lens, o=o)
    _, h2 = kda.glr_prefill(x, la, be, h0, normalise=norm, lens=lens, o=o2)
    torch.cuda.synchronize()
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(h), bits(h2)) and kept()
    wrong = ~torch.isfinite(o)
    hit = torch.zeros_like(wrong)
    hit[0, 3, 200:260, 5], hit[0, 3, 210:260, 6] = True, True
    assert torch.equal(wrong, hit)

    got = kda.glr_backward(x, la, be, h0, o, dO, dh, normalise=norm, lens=lens)
    rooms = {n: gapped(B, H, T, d, DT[dt]) for n in ("dx", "dlog_alpha", "dbeta")}
    lib, dh0, code = kda.load(), torch.empty_like(h0), 1 if dt == "bf16" else 0
    ws = torch.empty(int(lib.kda_glr_backward_workspace_bytes(B, H, T, d, code)), dtype=torch.uint8, device=dev())
    st = kda._GlrStrides(*(kda._Strides(*t.stride()[:3]) for t in (x, la, x, o)))
    gst = kda._GlrGradStrides(*(kda._Strides(*t.stride()[:3]) for t in (dO, *(v for v, _ in rooms.values()))))
    rc = lib.kda_glr_backward(x.data_ptr(), la.data_ptr(), be.data_ptr() if beta else None, h0.data_ptr(), o.data_ptr(), dO.data_ptr(),
                              dh.data_ptr(), lens.data_ptr(), *(v.data_ptr() for v, _ in rooms.values()), dh0.data_ptr(), st, gst, B,
                              H, T, d, int(norm), code, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(bits(dh0), bits(got["dh0"]))  # (a gate of NaN is in them)
    for n, (v, kept) in rooms.items():
        if n in got:
            assert streamed(got[n]) and torch.equal(bits(got[n]), bits(v)) and kept(), n

    # two heads of finite values against the reference
    for b, head in ((0, 1), (B - 1, H - 1)):
        cut = lambda t: None if t is None else t[b:b + 1, head:head + 1].cpu()  # noqa: E731
        c = dict(x=cut(x), la=cut(la), beta=cut(be), h0=cut(h0), dO=cut(dO), dh_T=cut(dh))
        ln = [int(lens[b])]
        a = lambda t: None if t is None else t.abs()  # noqa: E731
        ref, end = orc.glr(c["x"], c["la"], c["beta"], c["h0"], norm, ln)
        so, sh = orc.glr(a(c["x"]), c["la"], a(c["beta"]), a(c["h0"]), norm, ln)
        within(cut(o), ref, HALF[dt] * ref.abs() + slack(dt, T) * so, "o")
        within(cut(h), end, 2.0 ** -24 * end.abs() + slack(dt, T) * sh, "h_T")
        check_glr_grads({n: cut(t) for n, t in got.items()}, c, cut(o), norm, dt, ln)


@pytest.mark.parametrize("dt,d,rows", [("bf16", 128, 132000), ("f32", 64, 132000), ("bf16", 4096, 4200)])
def test_norm(dt, d, rows):
    print(f"[case] streaming norm {dt} {d}", flush=True)
    B, H, T = 2, 1, rows // 2
    r = draw(d)
    x, res, gate, dy, ds = (r(B, H, T, d).to(DT[dt]) for _ in range(5))
    w = (1 + 0.3 * r(d)).to(DT[dt])
    x[0, 0, 9, 3], gate[1, 0, 11, 4] = float("inf"), float("nan")
    y, s = kda.rms_norm(x, w, res, gate)
    (y2, yk), (s2, sk) = gapped(B, H, T, d, DT[dt]), gapped(B, H, T, d, DT[dt])
    kda.rms_norm(x, w, res, gate, y=y2, residual_out=s2)
    torch.cuda.synchronize()
    assert streamed(y) and streamed(s) and not streamed(y2)
    assert torch.equal(bits(y), bits(y2)) and torch.equal(bits(s), bits(s2)) and yk() and sk()
    # 8 bits: the sum alone is streamed
    s3, k3 = gapped(B, H, T, d, DT[dt])
    for scales in ("row", "block"):
        a = kda.rms_norm_quant(x, w, res, gate, scales=scales)
        b = kda.rms_norm_quant(x, w, res, gate, scales=scales, residual_out=s3)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(m), bits(n)) for m, n in zip(a, b)) and torch.equal(bits(a[2]), bits(s)) and k3()

    got = kda.rms_norm_backward(s, w, dy, ds, gate)
    rooms = {n: gapped(B, H, T, d, DT[dt]) for n in ("dx", "dgate")}
    lib, dw, code = kda.load(), torch.empty_like(w), 1 if dt == "bf16" else 0
    ws = torch.empty(int(lib.kda_rms_norm_backward_workspace_bytes(B, H, T, d, 0, code)), dtype=torch.uint8, device=dev())
    st = kda._NormGradStrides(*(kda._Strides(*t.stride()[:3]) for t in (s, gate, dy, ds, rooms["dx"][0], rooms["dgate"][0])))
    rc = lib.kda_rms_norm_backward(s.data_ptr(), gate.data_ptr(), w.data_ptr(), dy.data_ptr(), ds.data_ptr(), rooms["dx"][0].data_ptr(),
                                   rooms["dgate"][0].data_ptr(), dw.data_ptr(), st, B, H, T, d, 0, 1e-6, 0, code, ws.data_ptr(),
                                   ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for n, (v, kept) in rooms.items():
        assert streamed(got[n]) and torch.equal(bits(got[n]), bits(v)) and kept(), n
    # (a NaN of one row is in every sum of dweight, whose payload no one holds)
    assert torch.equal(torch.isnan(dw), torch.isnan(got["dweight"])) and torch.equal(torch.nan_to_num(dw), torch.nan_to_num(got["dweight"]))

    # rows of both ends against the reference
    for b, t0 in ((0, 20), (1, T - 40)):
        cut = lambda t: t[b:b + 1, :, t0:t0 + 40].cpu()  # noqa: E731
        c = dict(w=w.cpu(), gate=cut(gate), dy=cut(dy))
        assert torch.equal(cut(s), (cut(x).float() + cut(res).float()).to(DT[dt]))
        ref = orc.rms_norm(cut(s), c["w"], c["gate"])
        within(cut(y), ref, (HALF[dt] + 2.0 ** -18) * ref.abs() + 1e-30, "y")
        one = kda.rms_norm_backward(*(t[b:b + 1, :, t0:t0 + 40].contiguous() if t.dim() == 4 else t for t in (s, w, dy, ds, gate)))
        torch.cuda.synchronize()
        # (the same rows alone: their dweight has no other rows in it)
        assert torch.equal(one["dx"], got["dx"][b:b + 1, :, t0:t0 + 40]) and torch.equal(one["dgate"], got["dgate"][b:b + 1, :, t0:t0 + 40])
        check_norm_grads(one, cut(s), c, cut(ds), "sigmoid", dt, 1e-6)
