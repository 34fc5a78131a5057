"""Float64 oracle of linear attention with a decay for each head and of the
block-norm junction: the definitions token by token and row by row (numpy),
with their gradients. Test-only."""
import numpy as np


def _heads(t, rep):
    return np.repeat(np.asarray(t, dtype=np.float64), rep, axis=2)


def _decays(g, B, L, H):
    if g is None:
        return np.zeros((B, L, H))
    g = np.asarray(g, dtype=np.float64)
    return np.broadcast_to(g, (B, L, H)).copy()


def linattn_fwd(q, k, v, g=None, scale=1.0, h0=None, seqlens=None):
    """q, k [B, L, Hq, dk], v [B, L, H, dv], g [B, L, H] or [H]; returns y and
    the state after each row's last token."""
    v = np.asarray(v, dtype=np.float64)
    B, L, H, dv = v.shape
    rep = H // q.shape[2]
    q, k = _heads(q, rep), _heads(k, rep)
    g = _decays(g, B, L, H)
    S = np.zeros((B, H, q.shape[3], dv)) if h0 is None else np.array(h0, dtype=np.float64)
    y = np.zeros_like(v)
    for b in range(B):
        n = L if seqlens is None else min(max(int(seqlens[b]), 0), L)
        for t in range(n):
            a = np.exp(g[b, t])[:, None, None]
            old = np.where(a == 0.0, 0.0, S[b])
            S[b] = a * old + k[b, t][:, :, None] * v[b, t][:, None, :]
            y[b, t] = scale * np.einsum("hk,hkv->hv", q[b, t], S[b])
    return y, S


def linattn_bwd(q, k, v, g=None, scale=1.0, h0=None, seqlens=None, dy=None, dfinal=None):
    """Gradients of Σ dy·y + Σ dfinal·S_last: dict dq, dk, dv, dlog_decay, dh0.
    dlog_decay from its own definition, exp(g_t)·<S_{t−1}, N_t>."""
    v = np.asarray(v, dtype=np.float64)
    dy = np.asarray(dy, dtype=np.float64)
    B, L, H, dv = v.shape
    Hq, dk = q.shape[2], q.shape[3]
    rep = H // Hq
    q, k = _heads(q, rep), _heads(k, rep)
    g = _decays(g, B, L, H)
    dq, dkk, dvv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg = np.zeros_like(g)
    dh0 = np.zeros((B, H, dk, dv))
    for b in range(B):
        n = L if seqlens is None else min(max(int(seqlens[b]), 0), L)
        S = np.zeros((n + 1, H, dk, dv))
        if h0 is not None:
            S[0] = h0[b]
        for t in range(n):
            a = np.exp(g[b, t])[:, None, None]
            S[t + 1] = a * S[t] + k[b, t][:, :, None] * v[b, t][:, None, :]
        N = np.zeros((H, dk, dv)) if dfinal is None else np.array(dfinal[b], dtype=np.float64)
        for t in range(n - 1, -1, -1):
            N = N + scale * q[b, t][:, :, None] * dy[b, t][:, None, :]
            dq[b, t] = scale * np.einsum("hkv,hv->hk", S[t + 1], dy[b, t])
            dkk[b, t] = np.einsum("hkv,hv->hk", N, v[b, t])
            dvv[b, t] = np.einsum("hkv,hk->hv", N, k[b, t])
            a = np.exp(g[b, t])
            dg[b, t] = a * np.einsum("hkv,hkv->h", S[t], N)
            N = a[:, None, None] * N
        dh0[b] = N
    shared = lambda t: t.reshape(B, L, Hq, rep, dk).sum(3)  # noqa: E731
    return dict(dq=shared(dq), dk=shared(dkk), dv=dvv, dlog_decay=dg, dh0=dh0)


def block_norm_fwd(x, z=None, weight=None, residual=None, res_scale=None, next_weight=None,
                   groups=1, eps=1e-5, gate="after"):
    """Rows [R, D]; returns (out, y) and what the gradient needs."""
    f = lambda t: None if t is None else np.asarray(t, dtype=np.float64)  # noqa: E731
    x, z, weight, residual, res_scale, next_weight = map(
        f, (x, z, weight, residual, res_scale, next_weight))
    R, D = x.shape
    c = {}
    sig = None if z is None else 1.0 / (1.0 + np.exp(-z))
    gz = None if z is None else z * sig
    a = x * gz if z is not None and gate == "before" else x
    p = a
    if weight is not None:
        ag = a.reshape(R, groups, -1)
        c["rstd"] = 1.0 / np.sqrt((ag ** 2).mean(2, keepdims=True) + eps)
        c["n"] = (ag * c["rstd"]).reshape(R, D)
        p = c["n"] * weight
    u = p * gz if z is not None and gate == "after" else p
    out = u if res_scale is None else res_scale * u
    if residual is not None:
        out = residual + out
    y = None
    if next_weight is not None:
        c["rstd2"] = 1.0 / np.sqrt((out ** 2).mean(1, keepdims=True) + eps)
        y = out * c["rstd2"] * next_weight
    c.update(sig=sig, gz=gz, p=p, u=u, x=x, z=z)
    return out, y, c


def block_norm_bwd(x, z=None, weight=None, residual=None, res_scale=None, next_weight=None,
                   groups=1, eps=1e-5, gate="after", dout=None, dy=None):
    out, _, c = block_norm_fwd(x, z, weight, residual, res_scale, next_weight, groups, eps, gate)
    R, D = out.shape
    g = {}
    dr = np.zeros((R, D)) if dout is None else np.asarray(dout, dtype=np.float64)
    if next_weight is not None:
        dy = np.asarray(dy, dtype=np.float64)
        m = out * c["rstd2"]
        g["dnext_weight"] = (dy * m).sum(0)
        dm = dy * next_weight
        dr = dr + c["rstd2"] * (dm - m * (dm * m).mean(1, keepdims=True))
    if residual is not None:
        g["dresidual"] = dr
    du = dr
    if res_scale is not None:
        g["dres_scale"] = (dr * c["u"]).sum(0)
        du = dr * res_scale
    dgate = None
    dp = du
    if z is not None and gate == "after":
        dgate, dp = du * c["p"], du * c["gz"]
    da = dp
    if weight is not None:
        g["dweight"] = (dp * c["n"]).sum(0)
        dn = (dp * weight).reshape(R, groups, -1)
        n = c["n"].reshape(R, groups, -1)
        da = (c["rstd"] * (dn - n * (dn * n).mean(2, keepdims=True))).reshape(R, D)
    if z is not None and gate == "before":
        dgate, da = da * c["x"], da * c["gz"]
    g["dx"] = da
    if z is not None:
        g["dz"] = dgate * c["sig"] * (1.0 + c["z"] * (1.0 - c["sig"]))
    return g
