"""CPU tests of the gated linear recurrence, the norm and the drafts: the C-ABI's refusals (on the host,
before anything would be launched), the bindings' refusals, and the fp64 references that the GPU tests
use against autograd and plain definitions."""
import pytest
import torch

import gated_delta_rule_104_amd as kda
import layer_oracle as orc

OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_PRECONDITION, ERR_HIP = range(8)
F32, BF16 = 0, 1
A = 0x100000  # 16-byte aligned, never dereferenced: these calls are refused or have nothing to do


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def st(b, h, t):
    return kda._Strides(b, h, t)


# ------------------------------------------------ gated linear recurrence
def glr(lib, B=2, H=3, T=500, d=16, dt=BF16, strides=None, ws=A, nws=1 << 40, norm=1, **p):
    a = dict(x=A, la=A + 64, beta=A + 128, h0=None, lens=None, o=A + 192, h_T=A + 256)
    a.update(p)
    return lib.kda_glr_prefill(*a.values(), strides, B, H, T, d, norm, dt, ws, nws, None)


def test_glr_prefill_refusals(lib):
    assert glr(lib, dt=2) == ERR_UNSUPPORTED
    assert glr(lib, d=12) == ERR_UNSUPPORTED and glr(lib, d=6, dt=F32) == ERR_UNSUPPORTED
    assert glr(lib, B=-1) == ERR_SHAPE and glr(lib, T=-1) == ERR_SHAPE and glr(lib, H=-1) == ERR_SHAPE and glr(lib, d=-8) == ERR_SHAPE
    assert glr(lib, T=(1 << 30) + 1) == ERR_SHAPE and glr(lib, H=1 << 20, d=1 << 12) == ERR_SHAPE
    assert glr(lib, B=1 << 20, H=1, d=64, T=1 << 20) == ERR_SHAPE
    for n in ("x", "la", "o", "h_T"):
        assert glr(lib, **{n: None}) == ERR_NULL, n
    for n in ("x", "la", "beta", "h0", "o", "h_T"):
        assert glr(lib, **{n: A + 8}) == ERR_ALIGN, n
    for n in ("x", "la", "beta"):
        assert glr(lib, **{n: A + 192}) == ERR_UNSUPPORTED, n
    need = lib.kda_glr_prefill_workspace_bytes(2, 3, 500, 16, BF16)
    assert need > 0
    assert glr(lib, ws=None) == ERR_WORKSPACE and glr(lib, nws=need - 1) == ERR_WORKSPACE and glr(lib, ws=A + 8) == ERR_ALIGN
    bad = kda._GlrStrides(*(st(24000, 8000, 16) for _ in range(4)))
    bad.o = st(24000, 8000, 0)
    assert glr(lib, strides=bad) == ERR_SHAPE
    bad.o = st(24000, 8000, 20)
    assert glr(lib, strides=bad) == ERR_ALIGN
    bad.o = st(24000, 8000, 16)
    bad.log_alpha = st(-24000, 8000, 16)
    assert glr(lib, strides=bad) == ERR_SHAPE
    assert glr(lib, B=0) == OK and glr(lib, H=0) == OK


def test_glr_workspaces(lib):
    ws, bw = lib.kda_glr_prefill_workspace_bytes, lib.kda_glr_backward_workspace_bytes
    # one tile of tokens needs none; each tile of 64 channels else takes a word of 64 bits a channel
    assert ws(4, 32, 100, 128, BF16) == 0 and ws(4, 32, 8192, 128, BF16) == 4 * 64 * (8192 // 128) * 64 * 8
    assert bw(4, 32, 8192, 128, BF16) == 4 * 64 * (8192 // 64) * 64 * 8
    for f in (ws, bw):
        assert f(0, 1, 100, 64, BF16) == 0 and f(1, 1, 0, 64, BF16) == 0 and f(1, 1, 1000, 12, BF16) == 0 and f(1, 1, 100, 64, 7) == 0
        assert f(1, 1, 1000, 8, F32) > 0


def test_glr_step_refusals(lib):
    def f(N=2, H=3, d=16, dt=BF16, strides=None, **p):
        a = dict(x=A, la=A + 64, beta=A + 128, h=A + 192, o=A + 256)
        a.update(p)
        return lib.kda_glr_step(*a.values(), strides, N, H, d, 0, dt, None)
    assert f(N=-1) == ERR_SHAPE and f(d=4) == ERR_UNSUPPORTED and f(dt=9) == ERR_UNSUPPORTED
    for n in ("x", "la", "h", "o"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("x", "la", "beta", "h", "o"):
        assert f(**{n: A + 4}) == ERR_ALIGN, n
    for n in ("x", "la", "beta", "h"):
        assert f(**{n: A + 256}) == ERR_UNSUPPORTED, n
    for n in ("x", "la", "beta"):
        assert f(**{n: A + 192}) == ERR_UNSUPPORTED, n
    assert f(N=0) == OK


def test_glr_backward_refusals(lib):
    need = lib.kda_glr_backward_workspace_bytes(2, 3, 500, 16, BF16)

    def f(B=2, H=3, T=500, d=16, dt=BF16, ws=A, nws=need, gst=None, **p):
        a = dict(x=A, la=A + 64, beta=A + 128, h0=A + 192, o=A + 256, dO=A + 320, dh_T=None, lens=None, dx=A + 384,
                 dla=A + 448, dbeta=A + 512, dh0=A + 576)
        a.update(p)
        return lib.kda_glr_backward(*a.values(), None, gst, B, H, T, d, 1, dt, ws, nws, None)
    assert f(B=0) == ERR_SHAPE and f(T=0) == ERR_SHAPE and f(H=0) == OK and f(d=12) == ERR_UNSUPPORTED
    for n in ("x", "la", "o", "dO", "dx", "dla", "dbeta"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("x", "la", "beta", "h0", "o", "dO", "dh_T", "dx", "dla", "dbeta", "dh0"):
        assert f(**{n: A + 8}) == ERR_ALIGN, n
    for g in ("dx", "dla", "dbeta"):
        for at in (A, A + 64, A + 128, A + 256, A + 320):
            assert f(**{g: at}) == ERR_UNSUPPORTED, g
    assert f(dx=A + 448) == ERR_UNSUPPORTED and f(dh0=A + 192) == ERR_UNSUPPORTED and f(dh_T=A + 576) == ERR_UNSUPPORTED
    assert f(ws=None) == ERR_WORKSPACE and f(nws=need - 1) == ERR_WORKSPACE
    g = kda._GlrGradStrides(*(st(24000, 8000, 16) for _ in range(4)))
    g.dx = st(24000, 0, 16)
    assert f(gst=g) == ERR_SHAPE


def test_glr_polls_option(lib):
    for good in (0, 5, 1 << 20):
        assert lib.kda_set_option(b"glr_polls", good) == OK and kda.get_option("glr_polls") == good
    assert lib.kda_set_option(b"glr_polls", (1 << 20) + 1) == ERR_SHAPE and lib.kda_set_option(b"glr_polls", -2) == ERR_SHAPE
    assert lib.kda_set_option(b"glr_polls", -1) == OK and kda.get_option("glr_polls") is None


# ------------------------------------------------------------------- norm
def norm(lib, B=2, H=3, T=5, d=64, per_head=0, eps=1e-6, act=0, out=0, dt=BF16, strides=None, **p):
    a = dict(x=A, residual=A + 64, gate=A + 128, w=A + 192, y=A + 256, scales=None, s=A + 320)
    a.update(p)
    return lib.kda_rms_norm(*a.values(), strides, B, H, T, d, per_head, eps, act, out, dt, None)


def test_norm_refusals(lib):
    assert norm(lib, dt=3) == ERR_UNSUPPORTED and norm(lib, d=20) == ERR_UNSUPPORTED and norm(lib, d=32776) == ERR_UNSUPPORTED
    assert norm(lib, act=2) == ERR_UNSUPPORTED and norm(lib, out=5) == ERR_UNSUPPORTED and norm(lib, out=-1) == ERR_UNSUPPORTED
    assert norm(lib, eps=-1.0) == ERR_UNSUPPORTED and norm(lib, eps=float("nan")) == ERR_UNSUPPORTED and norm(lib, eps=float("inf")) == ERR_UNSUPPORTED
    assert norm(lib, B=-1) == ERR_SHAPE and norm(lib, B=1 << 16, H=1 << 10, T=1 << 10) == ERR_SHAPE
    assert norm(lib, out=4, scales=A + 1, d=72) == ERR_UNSUPPORTED
    for n in ("x", "y"):
        assert norm(lib, **{n: None}) == ERR_NULL, n
    for out in (1, 2, 3, 4):
        assert norm(lib, out=out) == ERR_NULL
    for n in ("x", "residual", "gate", "w", "y", "s"):
        assert norm(lib, **{n: A + 8}) == ERR_ALIGN, n
    assert norm(lib, out=1, scales=A + 2) == ERR_ALIGN
    for n in ("x", "residual", "gate", "w"):
        assert norm(lib, **{n: A + 256}) == ERR_UNSUPPORTED, n
    for n in ("x", "gate", "w"):
        assert norm(lib, **{n: A + 320}) == ERR_UNSUPPORTED, n
    assert norm(lib, residual=None) == ERR_UNSUPPORTED and norm(lib, s=A + 256) == ERR_UNSUPPORTED
    q = kda._NormStrides(*(st(960, 320, 64) for _ in range(6)))
    q.residual_out = st(1920, 640, 128)
    assert norm(lib, residual=A + 320, strides=q) == ERR_UNSUPPORTED  # in place, but elsewhere
    q.y = st(960, 320, 0)
    assert norm(lib, strides=q) == ERR_SHAPE
    assert norm(lib, B=0) == OK and norm(lib, T=0) == OK


def test_norm_backward_refusals(lib):
    ws = lib.kda_rms_norm_backward_workspace_bytes
    need = ws(2, 3, 5, 64, 0, BF16)
    assert need > 0 and ws(2, 3, 5, 64, 1, BF16) >= 3 * 64 * 4 and ws(0, 3, 5, 64, 0, BF16) == 0 and ws(2, 3, 5, 20, 0, BF16) == 0

    def f(B=2, H=3, T=5, d=64, act=0, eps=1e-6, dt=BF16, wsp=A, nws=need, **p):
        a = dict(x=A, gate=A + 64, w=A + 128, dy=A + 192, ds=A + 256, dx=A + 320, dgate=A + 384, dw=A + 448)
        a.update(p)
        return lib.kda_rms_norm_backward(*a.values(), None, B, H, T, d, 0, eps, act, dt, wsp, nws, None)
    assert f(B=0) == ERR_SHAPE and f(T=0) == ERR_SHAPE and f(H=0) == OK and f(act=7) == ERR_UNSUPPORTED and f(eps=-1e-9) == ERR_UNSUPPORTED
    for n in ("x", "dy", "dx", "dgate", "dw"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("x", "gate", "w", "dy", "ds", "dx", "dgate"):
        assert f(**{n: A + 8}) == ERR_ALIGN, n
    for g in ("dx", "dgate", "dw"):
        for at in (A, A + 64, A + 128, A + 192, A + 256):
            assert f(**{g: at}) == ERR_UNSUPPORTED, g
    assert f(dgate=A + 320) == ERR_UNSUPPORTED and f(dw=A + 320) == ERR_UNSUPPORTED
    assert f(wsp=None) == ERR_WORKSPACE and f(nws=need - 1) == ERR_WORKSPACE


# ----------------------------------------------------------------- drafts
def test_verify_refusals(lib):
    need = lib.kda_draft_verify_workspace_bytes(2, 3, 40000, F32)
    assert need > 0 and lib.kda_draft_verify_workspace_bytes(0, 3, 40000, F32) == 0
    assert lib.kda_draft_verify_workspace_bytes(2, 3, 1000, F32) == 0  # (short rows need none)

    def f(N=2, K=3, V=40000, dt=F32, ws=A, nws=need, ts=None, qs=None, **p):
        a = dict(p=A + 4, q=A + 8, tok=A + 12, u=A + 16, counts=None, acc=A + 20, out=A + 24)
        a.update(p)
        return lib.kda_draft_verify(a["p"], ts, a["q"], qs, a["tok"], a["u"], a["counts"], a["acc"], a["out"], N, K, V, dt, ws,
                                    nws, None)
    assert f(dt=2) == ERR_UNSUPPORTED and f(N=-1) == ERR_SHAPE and f(K=-1) == ERR_SHAPE and f(V=0) == ERR_SHAPE and f(V=-5) == ERR_SHAPE
    assert f(K=(1 << 16) + 1) == ERR_SHAPE and f(V=(1 << 30) + 1) == ERR_SHAPE and f(N=1 << 20, V=1 << 25) == ERR_SHAPE
    for n in ("p", "tok", "u", "acc", "out"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("p", "q", "tok", "u", "counts", "acc", "out"):
        assert f(**{n: A + 2}) == ERR_ALIGN, n
    assert f(p=A + 2, dt=BF16, acc=A + 1) == ERR_ALIGN and f(p=A + 1, dt=BF16) == ERR_ALIGN
    for o in ("acc", "out"):
        for at in (A + 4, A + 8, A + 12, A + 16):
            assert f(**{o: at}) == ERR_UNSUPPORTED, o
    assert f(acc=A + 24) == ERR_UNSUPPORTED
    assert f(ts=st(-1, 0, 1000)) == ERR_SHAPE and f(qs=st(1000, 0, 1 << 41)) == ERR_SHAPE
    assert f(ws=None) == ERR_WORKSPACE and f(nws=need - 1) == ERR_WORKSPACE and f(ws=A + 8) == ERR_ALIGN
    assert f(N=0) == OK


def test_commit_refusals(lib):
    def f(N=2, ntok=3, H=2, dk=4, dv=4, pos=A, idx=A + 4, S=A + 64):
        return lib.kda_state_commit(pos, idx, S, N, ntok, H, dk, dv, None)
    assert f(N=-1) == ERR_SHAPE and f(ntok=-1) == ERR_SHAPE and f(dk=1 << 13, dv=1 << 13) == ERR_SHAPE
    assert f(H=1, dk=1, dv=3) == ERR_UNSUPPORTED
    assert f(pos=None) == ERR_NULL and f(idx=None) == ERR_NULL and f(S=None) == ERR_NULL
    assert f(pos=A + 8) == ERR_ALIGN and f(S=A + 8) == ERR_ALIGN and f(S=A) == ERR_UNSUPPORTED
    assert f(N=0) == OK and f(ntok=0) == OK and f(H=0) == OK


# --------------------------------------------------------------- bindings
def test_bindings_refuse_host_tensors():
    z = torch.zeros(1, 2, 3, 8)
    for f in (lambda: kda.glr_prefill(z, z), lambda: kda.glr_step(z[:, :, 0], z[:, :, 0], z[:, :, 0]),
              lambda: kda.glr_backward(z, z, None, None, z, z), lambda: kda.rms_norm(z, None),
              lambda: kda.rms_norm_quant(z, None, scales="row"), lambda: kda.rms_norm_backward(z, None, z),
              lambda: kda.draft_verify(z[0], None, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 3)),
              lambda: kda.state_commit(torch.zeros(1, 1, 1, 2, 2), torch.zeros(1, dtype=torch.int32), z)):
        with pytest.raises(kda.KdaError, match="device tensor"):
            f()
    with pytest.raises(kda.KdaError, match="unsupported dtype"):
        kda.glr_prefill(z.half(), z)
    with pytest.raises(kda.KdaError, match="dimensions"):
        kda.rms_norm(z[0], None)
    with pytest.raises(kda.KdaError, match="8-bit output"):
        kda.rms_norm_quant(z, None, fmt="e5m2")
    with pytest.raises(kda.KdaError, match="blocks of 32"):
        kda.rms_norm_quant(z, None)
    with pytest.raises(kda.KdaError, match="h is required"):
        kda.glr_step(z[:, :, 0], z[:, :, 0], None)


# --------------------------------------------------- the references themselves
def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("norm", [False, True])
def test_glr_reference_gradients(norm):
    B, H, T, d = 2, 2, 7, 3
    t = dict(x=rand(B, H, T, d, seed=1), la=-rand(B, H, T, d, seed=2).abs() - 0.01, beta=rand(B, H, T, d, seed=3), h0=rand(B, H, d, seed=4))
    dO, dh = rand(B, H, T, d, seed=5), rand(B, H, d, seed=6)
    leaves = {n: v.clone().requires_grad_() for n, v in t.items()}
    h, rows = leaves["h0"], []
    for i in range(T):
        la = leaves["la"][:, :, i]
        n = torch.sqrt(1 - torch.exp(2 * la)) if norm else 1.0
        h = torch.exp(la) * h + n * leaves["beta"][:, :, i] * leaves["x"][:, :, i]
        rows.append(h)
    y = torch.stack(rows, 2)
    ref = torch.autograd.grad([y, h], list(leaves.values()), [dO, dh])
    o, end = orc.glr(t["x"], t["la"], t["beta"], t["h0"], norm)
    assert torch.allclose(o, y.detach(), rtol=1e-12) and torch.allclose(end, h.detach(), rtol=1e-12)
    got = orc.glr_backward(t["x"], t["la"], t["beta"], t["h0"], o, dO, dh, norm)
    for n, r in zip(("dx", "dlog_alpha", "dbeta", "dh0"), ref):
        assert torch.allclose(got[n], r, rtol=1e-9, atol=1e-11), n


def test_glr_reference_lengths():
    x, la = rand(2, 1, 5, 2, seed=1), -rand(2, 1, 5, 2, seed=2).abs()
    o, h = orc.glr(x, la, lens=[3, 0])
    a, b = orc.glr(x[:1, :, :3], la[:1, :, :3])
    assert torch.equal(o[0, :, :3], a[0]) and torch.equal(h[0], b[0]) and not h[1].any() and torch.isnan(o[1]).all()
    g = orc.glr_backward(x, la, None, None, torch.nan_to_num(o), torch.ones_like(x), torch.ones(2, 1, 2), lens=[3, 0])
    assert not g["dx"][0, :, 3:].any() and not g["dx"][1].any() and torch.equal(g["dh0"][1], torch.ones(1, 2).double())


@pytest.mark.parametrize("act", [None, "sigmoid", "silu"])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_reference_gradients(act, per_head):
    s, w, z = rand(2, 3, 4, 6, seed=1), rand(*((3, 6) if per_head else (6,)), seed=2), rand(2, 3, 4, 6, seed=3)
    dy, ds = rand(2, 3, 4, 6, seed=4), rand(2, 3, 4, 6, seed=5)
    leaves = [t.clone().requires_grad_() for t in (s, w, z)]
    n = leaves[0] * torch.rsqrt(leaves[0].square().mean(-1, keepdim=True) + 1e-3)
    y = n * (leaves[1][:, None] if per_head else leaves[1])
    if act:
        y = y * (torch.sigmoid(leaves[2]) if act == "sigmoid" else torch.nn.functional.silu(leaves[2]))
    ref = torch.autograd.grad((y * dy).sum() + (leaves[0] * ds).sum() + 0 * leaves[2].sum(), leaves)
    gate = z if act else None
    assert torch.allclose(orc.rms_norm(s, w, gate, act, 1e-3), y.detach(), rtol=1e-12, atol=1e-13)
    got = orc.rms_norm_backward(s, w, dy, ds, gate, act, 1e-3)
    for n, r in zip(("dx", "dweight") + (("dgate",) if act else ()), ref):
        assert torch.allclose(got[n], r, rtol=1e-10, atol=1e-12), n


def test_verify_reference_follows_the_target():
    """Accepted and drawn tokens together are distributed as the target's, whatever the draft: over a grid of
    random numbers the first token's frequencies are the target's probabilities."""
    p = torch.tensor([0.5, 0.2, 0.3], dtype=torch.float32)
    q = torch.tensor([0.2, 0.7, 0.1], dtype=torch.float32)
    n = 60
    grid = (torch.arange(n) + 0.5) / n
    freq = torch.zeros(3, dtype=torch.float64)
    for tok in range(3):
        u = torch.stack(torch.meshgrid(grid, grid, indexing="ij"), -1).reshape(-1, 2).float()
        N = u.shape[0]
        _, out = orc.verify(p.expand(N, 2, 3), q.expand(N, 1, 3), torch.full((N, 1), tok), u)
        freq += float(q[tok]) * torch.bincount(out[:, 0].long(), minlength=3).double() / N
    assert (freq - p.double()).abs().max() <= 2.0 / n
