"""fp64 references of the gated linear recurrence, the root-mean-square norm and the verification of
drafted tokens, written from the definitions in include/libkda.h, on the CPU."""
import torch


def _d(t):
    return None if t is None else t.double()


def lengths(lens, B, T):
    return [T] * B if lens is None else [max(0, min(T, int(n))) for n in lens]


def glr(x, la, beta=None, h0=None, norm=False, lens=None):
    """[B,H,T,d]: (o, h_T), fp64, token by token.  Rows of o behind lens are NaN."""
    x, a = x.double(), torch.exp(la.double())
    B, H, T, d = x.shape
    n = torch.sqrt(-torch.expm1(2 * la.double())) if norm else torch.ones_like(a)
    b = n * (x if beta is None else beta.double() * x)
    o = torch.full((B, H, T, d), float("nan"), dtype=torch.float64)
    h = torch.zeros(B, H, d, dtype=torch.float64) if h0 is None else h0.double().clone()
    for s, end in enumerate(lengths(lens, B, T)):
        for t in range(end):
            h[s] = torch.where(a[s, :, t] == 0, 0.0, a[s, :, t] * h[s]) + b[s, :, t]
            o[s, :, t] = h[s]
    return o, h


def glr_backward(x, la, beta, h0, o, dO, dh_T=None, norm=False, lens=None):
    """Gradients with the states before each token read from o."""
    x, la, o, g = x.double(), la.double(), o.double(), dO.double()
    B, H, T, d = x.shape
    a = torch.exp(la)
    bt = torch.ones_like(x) if beta is None else beta.double()
    n = torch.sqrt(-torch.expm1(2 * la)) if norm else torch.ones_like(a)
    out = {k: torch.zeros_like(x) for k in ("dx", "dlog_alpha", "dbeta")}
    lam = torch.zeros(B, H, d, dtype=torch.float64) if dh_T is None else dh_T.double().clone()
    for s, end in enumerate(lengths(lens, B, T)):
        for t in reversed(range(end)):
            l = lam[s] + g[s, :, t]
            before = o[s, :, t - 1] if t else (torch.zeros(H, d).double() if h0 is None else h0[s].double())
            at, nt, bx = a[s, :, t], n[s, :, t], bt[s, :, t] * x[s, :, t]
            out["dx"][s, :, t] = nt * bt[s, :, t] * l
            out["dbeta"][s, :, t] = nt * x[s, :, t] * l
            dl = at * before * l
            if norm:
                dl = dl - torch.where(nt > 0, at * at / nt, torch.zeros_like(nt)) * bx * l
            out["dlog_alpha"][s, :, t] = torch.where(at == 0, torch.zeros_like(dl), dl)
            lam[s] = torch.where(at == 0, torch.zeros_like(l), at * l)
    out["dh0"] = lam
    return out


def gate_factor(z, act):
    s = 1 / (1 + torch.exp(-z))
    return s if act == "sigmoid" else z * s


def _rows(w, x):
    """A weight [d] or [H,d] beside [B,H,T,d]."""
    if w is None:
        return torch.ones(x.shape[-1], dtype=torch.float64)
    return w.double()[:, None] if w.dim() == 2 else w.double()


def rms_norm(s, w=None, gate=None, act="sigmoid", eps=1e-6):
    s = s.double()
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * _rows(w, s)
    return y if gate is None else y * gate_factor(gate.double(), act)


def rms_norm_backward(s, w, dy, ds=None, gate=None, act="sigmoid", eps=1e-6):
    """Gradients of sum(dy y) + sum(ds s) by the chain rule."""
    s, dy = s.double(), dy.double()
    B, H, T, d = s.shape
    r = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    n, k = s * r, _rows(w, s)
    z = None if gate is None else gate.double()
    g = torch.ones_like(s) if z is None else gate_factor(z, act)
    dn = dy * k * g
    out = dict(dx=r * (dn - n * (dn * n).mean(-1, keepdim=True)) + (0 if ds is None else ds.double()))
    per = dy * n * g
    out["dweight"] = per.sum((0, 2)) if w is not None and w.dim() == 2 else per.sum((0, 1, 2))
    if z is not None:
        sig, rest = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))  # (1 - sig would be 0 far from zero)
        dg = sig * rest if act == "sigmoid" else sig * (1 + z * rest)
        out["dgate"] = dy * n * k * dg
    return out


def verify(target, draft, tokens, u, counts=None):
    """(accepted, out) by the definition, running sums in fp64."""
    N, K1, V = target.shape
    K = K1 - 1
    acc, rows = [], []
    for i in range(N):
        cnt = K if counts is None else max(0, min(K, int(counts[i])))
        a = 0
        while a < cnt:
            t = int(tokens[i, a])
            if not 0 <= t < V:
                break
            q = 1.0 if draft is None else float(draft[i, a, t])
            if not float(u[i, a]) * q < float(target[i, a, t]):
                break
            a += 1
        p = target[i, a].double()
        p = torch.where(p > 0, p, torch.zeros_like(p))
        w = p
        if a < cnt:
            q = torch.zeros_like(p)
            if draft is not None:
                q = draft[i, a].double()
                q = torch.where(q > 0, q, torch.zeros_like(q))
            elif 0 <= int(tokens[i, a]) < V:
                q[int(tokens[i, a])] = 1.0
            w = (p - q).clamp(min=0)
        if float(w.sum()) == 0:
            w = p
        cdf = torch.cumsum(w, 0)
        pick = -1
        if float(cdf[-1]) > 0:
            above = (cdf > float(u[i, K]) * cdf[-1]) & (w > 0)
            pick = int(above.nonzero()[0]) if above.any() else int((w > 0).nonzero()[-1])
        acc.append(a)
        rows.append([int(t) for t in tokens[i, :a]] + [pick] + [-1] * (K - a))
    return torch.tensor(acc, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32).reshape(N, K1)
