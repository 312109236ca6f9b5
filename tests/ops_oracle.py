"""fp64 references of the companion operators (convolution, scan, state cache),
written token by token from the definitions in include/libkda.h."""
import torch


def conv(x, weight, bias, state, act, lens=None):
    """x [B,H,T,d], weight [H,d,K], state [B,H,K-1,d] or None: (o, state_out), fp64.  Rows
    of o behind lens are NaN."""
    x, w = x.double(), weight.double()
    B, H, T, d = x.shape
    K = w.shape[2]
    st = torch.zeros(B, H, K - 1, d, dtype=torch.float64) if state is None else state.double()
    o = torch.full((B, H, T, d), float("nan"), dtype=torch.float64)
    out = torch.empty(B, H, K - 1, d, dtype=torch.float64)
    for b in range(B):
        n = T if lens is None else max(0, min(T, int(lens[b])))
        e = torch.cat([st[b], x[b, :, :n]], 1)
        for t in range(n):
            s = sum(w[:, :, k] * e[:, t + k] for k in range(K))
            if bias is not None:
                s = s + bias.double()
            o[b, :, t] = s / (1 + torch.exp(-s)) if act else s
        out[b] = e[:, n:n + K - 1]
    return o, out


def conv_backward(x, weight, bias, state, dO, dstate_out, act):
    x, w, g = x.double(), weight.double(), dO.double()
    B, H, T, d = x.shape
    K = w.shape[2]
    st = torch.zeros(B, H, K - 1, d, dtype=torch.float64) if state is None else state.double()
    e = torch.cat([st, x], 2)
    de, dw, db = torch.zeros_like(e), torch.zeros_like(w), torch.zeros(H, d, dtype=torch.float64)
    for t in range(T):
        s = sum(w[:, :, k] * e[:, :, t + k] for k in range(K)) + (0 if bias is None else bias.double())
        p = g[:, :, t]
        if act:
            sig = 1 / (1 + torch.exp(-s))
            p = p * (sig + s * sig * (1 - sig))
        for k in range(K):
            de[:, :, t + k] += w[:, :, k] * p
            dw[:, :, k] += (p * e[:, :, t + k]).sum(0)
        db += p.sum(0)
    if dstate_out is not None:
        de[:, :, T:] += dstate_out.double()
    return dict(dx=de[:, :, K - 1:], dweight=dw, dbias=db, dstate=de[:, :, :K - 1])


def _heads(t, H):
    """[B,G,...] rows of groups as [B,H,...] rows of heads."""
    return t.double().repeat_interleave(H // t.shape[1], 1)


def ssm(q, k, v, la, beta, D=None, S0=None, lens=None):
    """(o, S_T) in fp64; rows of o behind lens are NaN."""
    B, H, T, dv = v.shape
    q, k, v, beta, a = _heads(q, H), _heads(k, H), v.double(), beta.double(), torch.exp(la.double())
    S = torch.zeros(B, H, q.shape[-1], dv, dtype=torch.float64) if S0 is None else S0.double().clone()
    n = torch.full((B,), T) if lens is None else lens.long().clamp(0, T)
    o = torch.full((B, H, T, dv), float("nan"), dtype=torch.float64)
    for t in range(T):
        on = (t < n)[:, None, None]
        Sn = a[:, :, t, None, None] * S + k[:, :, t, :, None] * (beta[:, :, t, None] * v[:, :, t])[:, :, None]
        S = torch.where(on[..., None], Sn, S)
        y = torch.einsum("bhk,bhkv->bhv", q[:, :, t], S)
        if D is not None:
            y = y + D.double()[:, None] * v[:, :, t]
        o[:, :, t] = torch.where(on, y, o[:, :, t])
    return o, S


def ssm_backward(q, k, v, la, beta, D, S0, dO, dS_T):
    """Reverse mode through the token steps, keeping every state."""
    B, H, T, dv = v.shape
    G, dk = k.shape[1], k.shape[3]
    qh, kh, v, beta, a, g = _heads(q, H), _heads(k, H), v.double(), beta.double(), torch.exp(la.double()), dO.double()
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64) if S0 is None else S0.double()
    before, after = [], []
    for t in range(T):
        before.append(S)
        S = a[:, :, t, None, None] * S + kh[:, :, t, :, None] * (beta[:, :, t, None] * v[:, :, t])[:, :, None]
        after.append(S)
    dS = torch.zeros_like(S) if dS_T is None else dS_T.double().clone()
    out = {n: torch.zeros(B, H, T, m, dtype=torch.float64) for n, m in (("dq", dk), ("dk", dk), ("dv", dv))}
    dla, dbeta = torch.zeros(B, H, T, dtype=torch.float64), torch.zeros(B, H, T, dtype=torch.float64)
    for t in reversed(range(T)):
        dS = dS + qh[:, :, t, :, None] * g[:, :, t, None]
        out["dq"][:, :, t] = torch.einsum("bhkv,bhv->bhk", after[t], g[:, :, t])
        z = torch.einsum("bhkv,bhk->bhv", dS, kh[:, :, t])
        out["dv"][:, :, t] = beta[:, :, t, None] * z + (0 if D is None else D.double()[:, None] * g[:, :, t])
        dbeta[:, :, t] = (z * v[:, :, t]).sum(-1)
        out["dk"][:, :, t] = beta[:, :, t, None] * torch.einsum("bhkv,bhv->bhk", dS, v[:, :, t])
        dla[:, :, t] = a[:, :, t] * (dS * before[t]).sum((-1, -2))
        dS = a[:, :, t, None, None] * dS
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(B, G, H // G, T, dk).sum(2)
    out.update(dlog_alpha=dla, dbeta=dbeta, dS0=dS)
    if D is not None:
        out["dD"] = (g * v).sum((0, 2, 3))
    return out


def quantise(S, top):
    """Exponents p [..., dv/32] and scaled values of blocks of 32: the smallest power of two with
    max|x| 2^-p <= top, at least -126."""
    x = S.double().unflatten(-1, (-1, 32))
    m = x.abs().amax(-1)
    p = torch.full(m.shape, -126.0, dtype=torch.float64)
    for e in range(-126, 128):  # the first power that is large enough
        p = torch.where(m > top * 2.0 ** p, torch.full_like(p, e), p)
    return p, (x * torch.exp2(-p)[..., None]).flatten(-2)


def rel(x, ref):
    """Relative L2 distance over the finite places of ref (which are all of x's)."""
    x, ref = x.double().cpu(), ref.double()
    ok = ~torch.isnan(ref)
    n = float((ref[ok]).norm())
    d = float((x[ok] - ref[ok]).norm())
    return d / n if n > 0 else d
