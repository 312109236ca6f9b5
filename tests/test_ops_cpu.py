"""CPU tests of the companion operators: the C-ABI's refusals (on the host, before
anything would be launched), the bindings' refusals of host tensors, and the fp64
references that the GPU tests use against autograd and differences."""
import ctypes

import pytest
import torch

import gated_delta_rule_104_amd as kda
import ops_oracle as orc

OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_PRECONDITION, ERR_HIP = range(8)
F32, BF16 = 0, 1
A = 0x100000  # 16-byte aligned, never dereferenced: these calls are refused or have nothing to do


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def st(b, h, t):
    return kda._Strides(b, h, t)


# ------------------------------------------------------------- convolution
def conv(lib, x=A, xs=None, w=A + 2, bias=None, s_in=None, lens=None, o=A + 64, os_=None, s_out=None, B=1, H=2, T=5,
         d=16, K=4, act=1, dt=BF16):
    return lib.kda_conv_prefill(x, xs, w, bias, s_in, lens, o, os_, s_out, B, H, T, d, K, act, dt, None)


def test_conv_prefill_refusals(lib):
    assert conv(lib, dt=7) == ERR_UNSUPPORTED
    assert conv(lib, act=2) == ERR_UNSUPPORTED
    assert conv(lib, K=1) == ERR_UNSUPPORTED and conv(lib, K=5) == ERR_UNSUPPORTED
    assert conv(lib, d=12) == ERR_UNSUPPORTED and conv(lib, d=6, dt=F32) == ERR_UNSUPPORTED
    assert conv(lib, B=-1) == ERR_SHAPE and conv(lib, T=-1) == ERR_SHAPE and conv(lib, d=-16) == ERR_SHAPE
    assert conv(lib, H=1 << 20, d=1 << 12) == ERR_SHAPE and conv(lib, T=(1 << 30) + 1) == ERR_SHAPE
    assert conv(lib, x=None) == ERR_NULL and conv(lib, w=None) == ERR_NULL and conv(lib, o=None) == ERR_NULL
    assert conv(lib, x=A + 8) == ERR_ALIGN and conv(lib, o=A + 4) == ERR_ALIGN
    assert conv(lib, s_in=A + 8) == ERR_ALIGN and conv(lib, s_out=A + 8) == ERR_ALIGN
    assert conv(lib, s_in=A + 128, s_out=A + 128) == ERR_UNSUPPORTED
    assert conv(lib, o=A) == ERR_UNSUPPORTED
    assert conv(lib, B=0) == OK and conv(lib, H=0) == OK and conv(lib, T=0) == OK


def test_strides_are_checked(lib):
    B = dict(B=2, H=3, T=5)
    good = st(240, 16, 48)
    assert conv(lib, xs=st(240, 12, 48), **B) == ERR_ALIGN
    assert b"dimension 1" in lib.kda_last_error()
    assert conv(lib, xs=st(-240, 16, 48), **B) == ERR_SHAPE
    assert conv(lib, os_=st(240, 16, 0), **B) == ERR_SHAPE
    assert conv(lib, xs=good, os_=st(240, 16, (1 << 23) + 8), **B) == ERR_SHAPE
    # of dimensions of size 1 they are not looked at
    assert conv(lib, xs=st(-1, 3, 7), B=1, H=1, T=0) == OK


def test_conv_step_refusals(lib):
    def f(x=A, state=A + 64, w=A, o=A + 128, N=2, H=1, d=8, K=4, act=0, dt=BF16):
        return lib.kda_conv_step(x, None, state, w, None, o, None, N, H, d, K, act, dt, None)
    assert f(K=9) == ERR_UNSUPPORTED and f(d=4) == ERR_UNSUPPORTED and f(N=-1) == ERR_SHAPE
    assert f(x=None) == ERR_NULL and f(state=None) == ERR_NULL and f(w=None) == ERR_NULL and f(o=None) == ERR_NULL
    assert f(state=A + 2) == ERR_ALIGN
    assert f(N=0) == OK


def test_conv_backward_refusals(lib):
    def f(x=A, w=A, dO=A + 64, dx=A + 128, dw=A, ws=A, nws=1 << 30, B=1, H=2, T=5, d=16, K=4, dt=BF16):
        return lib.kda_conv_backward(x, None, w, None, None, dO, None, None, dx, None, dw, None, None, B, H, T, d, K, 1,
                                     dt, ws, nws, None)
    need = lib.kda_conv_backward_workspace_bytes
    assert need(1, 2, 5, 16, 4, BF16) > 0 and need(1, 2, 5, 16, 9, BF16) == 0 and need(0, 2, 5, 16, 4, BF16) == 0
    assert f(B=0) == ERR_SHAPE and f(T=0) == ERR_SHAPE and f(H=0) == OK
    assert f(x=None) == ERR_NULL and f(dO=None) == ERR_NULL and f(dx=None) == ERR_NULL and f(dw=None) == ERR_NULL
    assert f(dx=A) == ERR_UNSUPPORTED and f(dx=A + 64) == ERR_UNSUPPORTED
    assert f(ws=None) == ERR_WORKSPACE and f(ws=A + 8) == ERR_ALIGN
    assert f(nws=need(1, 2, 5, 16, 4, BF16) - 1) == ERR_WORKSPACE


# --------------------------------------------------------------------- scan
def ssm(lib, q=A, k=A, v=A, la=A + 2, beta=A + 2, D=None, S0=None, lens=None, o=A + 64, S_T=A + 128, strides=None, B=1,
        H=4, G=2, T=70, dk=64, dv=64, dt=BF16, ws=None, nws=0):
    return lib.kda_ssm_prefill(q, k, v, la, beta, D, S0, lens, o, S_T, strides, B, H, G, T, dk, dv, dt, ws, nws, None)


def test_ssm_prefill_refusals(lib):
    assert ssm(lib, dt=2) == ERR_UNSUPPORTED
    assert ssm(lib, dk=96) == ERR_UNSUPPORTED and ssm(lib, dv=32) == ERR_UNSUPPORTED
    assert ssm(lib, G=3) == ERR_SHAPE and ssm(lib, G=0) == ERR_SHAPE and ssm(lib, B=-1) == ERR_SHAPE
    assert ssm(lib, T=(1 << 30) + 1) == ERR_SHAPE and ssm(lib, B=1 << 12, H=1 << 13, G=1) == ERR_SHAPE
    for n in ("q", "k", "v", "la", "beta", "o", "S_T"):
        assert ssm(lib, **{n: None}) == ERR_NULL, n
    for n in ("q", "k", "v", "o", "S_T", "S0"):
        assert ssm(lib, **{n: A + 8}) == ERR_ALIGN, n
    assert ssm(lib, ws=A + 8, nws=64) == ERR_ALIGN
    for n in ("q", "k", "v"):
        assert ssm(lib, **{n: A + 64}) == ERR_UNSUPPORTED, n
    bad = kda._SsmStrides(*(st(4096, 64, 64) for _ in range(6)))
    bad.o = st(4096, 64, 60)
    assert ssm(lib, strides=bad) == ERR_ALIGN
    bad.o = st(4096, 0, 64)
    assert ssm(lib, strides=bad) == ERR_SHAPE
    assert ssm(lib, B=0) == OK and ssm(lib, H=0, G=1) == OK


def test_ssm_workspace_and_plan(lib):
    ws = lib.kda_ssm_prefill_workspace_bytes
    state = 64 * 128 * 64 * 4
    n = ws(1, 64, 8, 65536, 128, 64, BF16)
    # 16 segments (two workgroups of two heads per compute unit, 256 units): their start and end
    # states, and one decay each
    assert n == 17 * state + 16 * 64 * 4
    assert ws(1, 64, 8, 128, 128, 64, BF16) == 0  # too short
    assert ws(64, 64, 8, 8192, 128, 64, BF16) == 0  # enough heads
    assert ws(1, 64, 8, 65536, 96, 64, BF16) == 0 and ws(1, 64, 7, 65536, 128, 64, BF16) == 0


def test_ssm_step_refusals(lib):
    def f(N=2, H=4, G=2, dk=64, dv=128, dt=F32, **p):
        a = dict(q=A, k=A, v=A, la=A + 4, beta=A + 4, D=None, S=A, o=A)
        a.update(p)
        return lib.kda_ssm_step(*a.values(), N, H, G, dk, dv, dt, None)
    assert f(G=3) == ERR_SHAPE and f(N=-1) == ERR_SHAPE and f(dk=16) == ERR_UNSUPPORTED and f(dt=5) == ERR_UNSUPPORTED
    for n in ("q", "k", "v", "la", "beta", "S", "o"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("q", "k", "v", "S", "o"):
        assert f(**{n: A + 4}) == ERR_ALIGN, n
    assert f(N=0) == OK


def test_ssm_backward_refusals(lib):
    need = lib.kda_ssm_backward_workspace_bytes(1, 4, 2, 70, 64, 64, BF16)
    assert need > 0 and lib.kda_ssm_backward_workspace_bytes(1, 4, 2, 0, 64, 64, BF16) == 0

    def f(B=1, H=4, G=2, T=70, dk=64, dv=64, dt=BF16, ws=A, nws=need, gst=None, **p):
        a = dict(q=A, k=A, v=A, la=A + 2, beta=A + 2, D=None, S0=None, dO=A, dS_T=None, dq=A + 64, dk_=A + 128, dv_=A + 192,
                 dla=A + 256, dbeta=A + 320, dD=None, dS0=None)
        a.update(p)
        return lib.kda_ssm_backward(*a.values(), None, gst, B, H, G, T, dk, dv, dt, ws, nws, None)
    assert f(T=0) == ERR_SHAPE and f(B=0) == ERR_SHAPE and f(dk=80) == ERR_UNSUPPORTED and f(H=0, G=1) == OK
    for n in ("q", "k", "v", "la", "beta", "dO", "dq", "dk_", "dv_", "dla", "dbeta"):
        assert f(**{n: None}) == ERR_NULL, n
    assert f(D=A + 2) == ERR_NULL  # its gradient has nowhere to go
    for n in ("dO", "dS_T", "dq", "dS0"):
        assert f(**{n: A + 4}) == ERR_ALIGN, n
    assert f(ws=None) == ERR_WORKSPACE and f(nws=need - 1) == ERR_WORKSPACE and f(ws=A + 8) == ERR_ALIGN
    for n in ("dq", "dk_", "dv_", "dla", "dbeta"):  # a later launch would read what an earlier one wrote
        assert f(**{n: A}) == ERR_UNSUPPORTED, n
    assert f(S0=A + 512, dS0=A + 512) == ERR_UNSUPPORTED and f(dS_T=A + 512, dS0=A + 512) == ERR_UNSUPPORTED
    g = kda._SsmGradStrides(*(st(4096 * 4, 4096, 64) for _ in range(6)))
    g.dbeta = st(280, 70, 0)
    assert f(gst=g) == ERR_SHAPE


# ------------------------------------------- outputs that are inputs, one token
def test_steps_refuse_outputs_that_are_inputs(lib):
    """A head's q and k are read by the workgroups of its whole group, so an output in their place would
    be read by some of them; the calls refuse every such output, as the prompt calls do."""
    def conv_step(x=A, state=A + 64, w=A + 256, bias=A + 320, o=A + 128):
        return lib.kda_conv_step(x, None, state, w, bias, o, None, 2, 1, 8, 4, 0, BF16, None)

    def ssm_step(**p):
        a = dict(q=A, k=A + 4096, v=A + 8192, la=A + 12288, beta=A + 12352, D=A + 12416, S=A + 16384, o=A + 65536 * 8)
        a.update(p)
        return lib.kda_ssm_step(*a.values(), 2, 4, 2, 64, 64, BF16, None)
    assert conv_step(o=A) == ERR_UNSUPPORTED and conv_step(o=A + 64) == ERR_UNSUPPORTED
    assert conv_step(o=A + 256) == ERR_UNSUPPORTED and conv_step(o=A + 320) == ERR_UNSUPPORTED
    assert conv_step(state=A) == ERR_UNSUPPORTED
    for n, at in (("q", A), ("k", A + 4096), ("v", A + 8192), ("la", A + 12288), ("beta", A + 12352), ("S", A + 16384)):
        assert ssm_step(o=at) == ERR_UNSUPPORTED, n
    for n, at in (("q", A), ("k", A + 4096), ("v", A + 8192)):
        assert ssm_step(S=at) == ERR_UNSUPPORTED, n


# -------------------------------------------------------------- state cache
def test_state_cache_refusals(lib):
    def store(S=A, slots=A + 4, c=A, sc=A + 1, n=2, ns=4, H=1, dk=64, dv=64, f=0):
        return lib.kda_state_store(S, slots, c, sc, n, ns, H, dk, dv, f, None)

    def load(c=A, sc=A + 1, slots=A + 4, S=A, n=2, ns=4, H=1, dk=64, dv=64, f=0):
        return lib.kda_state_load(c, sc, slots, S, n, ns, H, dk, dv, f, None)
    for g in (store, load):
        assert g(f=2) == ERR_UNSUPPORTED and g(dv=48) == ERR_UNSUPPORTED
        assert g(n=-1) == ERR_SHAPE and g(ns=-1) == ERR_SHAPE and g(n=(1 << 16) + 1) == ERR_SHAPE
        for p in ("S", "slots", "c", "sc"):
            assert g(**{p: None}) == ERR_NULL, p
        assert g(S=A + 8) == ERR_ALIGN and g(c=A + 8) == ERR_ALIGN
        assert g(n=0) == OK and g(H=0) == OK


def test_bindings_refuse_host_tensors():
    x = torch.zeros(1, 2, 3, 8)
    with pytest.raises(kda.KdaError, match="device tensor"):
        kda.conv_prefill(x, torch.zeros(2, 8, 4))
    with pytest.raises(kda.KdaError, match="unsupported dtype"):
        kda.conv_prefill(x.half(), torch.zeros(2, 8, 4))
    with pytest.raises(kda.KdaError, match="dimensions"):
        kda.conv_step(x, None, torch.zeros(2, 8, 4))
    z = torch.zeros(1, 1, 4, 64)
    with pytest.raises(kda.KdaError, match="device tensor"):
        kda.ssm_prefill(z, z, z, torch.zeros(1, 1, 4), torch.zeros(1, 1, 4))
    with pytest.raises(kda.KdaError, match="format"):
        kda.state_cache(1, 1, 64, 64, "fp4", "cpu")
    with pytest.raises(kda.KdaError, match="blocks of 32"):
        kda.state_cache(1, 1, 64, 48, "int8", "cpu")
    c, s = kda.state_cache(2, 1, 64, 64, "e4m3", "cpu")
    assert c.dtype == torch.float8_e4m3fn and s.shape == (2, 1, 64, 2)
    with pytest.raises(kda.KdaError, match="device tensor"):
        kda.state_load(c, s, torch.zeros(1, dtype=torch.int32))


# --------------------------------------------------- the references themselves
def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("act", [False, True])
def test_conv_reference_gradients(act):
    x, w, b, s = rand(2, 3, 7, 4, seed=1), rand(3, 4, 3, seed=2), rand(3, 4, seed=3), rand(2, 3, 2, 4, seed=4)
    dO, ds = rand(2, 3, 7, 4, seed=5), rand(2, 3, 2, 4, seed=6)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, s)]
    e = torch.cat([leaves[3], leaves[0]], 2)
    y = sum(leaves[1][:, None, :, k] * e[:, :, k:k + 7] for k in range(3)) + leaves[2][:, None]
    y = torch.nn.functional.silu(y) if act else y
    ref = torch.autograd.grad([y, e[:, :, 7:]], leaves, [dO, ds])
    got = orc.conv_backward(x, w, b, s, dO, ds, act)
    o, _ = orc.conv(x, w, b, s, act)
    assert torch.allclose(o, y.detach(), rtol=1e-12, atol=1e-12)
    for n, r in zip(("dx", "dweight", "dbias", "dstate"), ref):
        assert torch.allclose(got[n], r, rtol=1e-12, atol=1e-12), n


def test_ssm_reference_gradients():
    B, H, G, T, dk, dv = 2, 4, 2, 6, 5, 3
    t = dict(q=rand(B, G, T, dk, seed=1), k=rand(B, G, T, dk, seed=2), v=rand(B, H, T, dv, seed=3),
             log_alpha=-rand(B, H, T, seed=4).abs(), beta=rand(B, H, T, seed=5), D=rand(H, seed=6),
             S0=rand(B, H, dk, dv, seed=7))
    dO, dS_T = rand(B, H, T, dv, seed=8), rand(B, H, dk, dv, seed=9)
    got = orc.ssm_backward(*t.values(), dO, dS_T)

    def loss(x):
        o, S = orc.ssm(*x.values())
        return float((o * dO).sum() + (S * dS_T).sum())

    for i, n in enumerate(t):
        u = rand(*t[n].shape, seed=20 + i)
        h = 1e-6
        d = (loss({**t, n: t[n] + h * u}) - loss({**t, n: t[n] - h * u})) / (2 * h)
        assert abs(float((got["d" + n] * u).sum()) - d) <= 1e-7 * max(1.0, abs(d)), n


def test_quantise_reference():
    x = torch.tensor([[127.0] + [0.0] * 31, [127.5] + [1.0] * 31, [0.0] * 32, [2.0 ** -130] * 32])
    p, y = orc.quantise(x, 127.0)
    assert p.flatten().tolist() == [0.0, 1.0, -126.0, -126.0] and float(y.abs().max()) <= 127
