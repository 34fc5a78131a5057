"""Timed cases of the linear-attention and block-norm operators.

Operators (shapes row-major, last index fastest):

  linattn_fwd   y_t = scale·S_tᵀ q_t,  S_t = exp(g_t)·S_{t−1} + k_t v_tᵀ   for every batch row and head,
                whole sequences, with an optional first state, ragged lengths and the state after the last token
  linattn_bwd   its gradient
  linattn_step  the same for one token, the state updated in place
  norm_fwd      p = RMSNorm_groups(x [· silu(z)])·weight [· silu(z)];  out = residual + res_scale·p;
                y = RMSNorm(out)·next_weight
  norm_bwd      its gradient

``listed`` and ``draw`` give cases, ``prepare`` their inputs, ``run`` one pass (``own``: the framework's kernels, else
plain torch operations in float32), ``work`` what a pass cannot do without and ``exact`` the definition in float64.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linattn(name, op, dtype, batch, seqlen, qk_heads, heads, dk, dv, decay="token", ragged=False, init=False,
             final=False, fused=False):
    c = dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, qk_heads=qk_heads, heads=heads, dk=dk, dv=dv,
             decay=decay, ragged=ragged, init=init, final=final, fused=fused)
    return dict(c, name=name) if name else c


def _norm(name, op, dtype, rows, dim, groups=1, gate="after", weight=True, residual="f32", res_scale=True, next=True):
    c = dict(op=op, dtype=dtype, rows=rows, dim=dim, groups=groups, gate=gate, weight=weight, residual=residual,
             res_scale=res_scale, next=next)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt of one user: the call's latency
        _linattn("fwd_prompt100", "linattn_fwd", "bf16", 1, 100, 16, 16, 64, 64, final=True),
        # a layer of the size of the repository's Mamba-2 layer (2 x 4096 tokens, 32 heads), 8 query/key heads
        # shared by 4 value heads each, q, k and v being slices of one projection
        _linattn("fwd_layer", "linattn_fwd", "bf16", 2, 4096, 8, 32, 128, 128, final=True, fused=True),
        # one long document, fixed decays (retention): more tokens than heads to spread over the GPU
        _linattn("fwd_long", "linattn_fwd", "bf16", 1, 65536, 16, 16, 128, 128, decay="fixed", final=True),
        # a padded batch of unequal prompts continued from states, float32, head sizes that fill no tile
        _linattn("fwd_ragged_f32", "linattn_fwd", "f32", 3, 1111, 6, 6, 48, 80, ragged=True, init=True, final=True),
        # the gradient of a training step's layer
        _linattn("bwd_layer", "linattn_bwd", "bf16", 2, 4096, 16, 16, 128, 128),
        # the gradient in float32 with shared heads and an odd length
        _linattn("bwd_shared_f32", "linattn_bwd", "f32", 2, 777, 2, 6, 64, 64, init=True),
        # decoding for one user, and for a full serving batch
        _linattn("step_b1", "linattn_step", "bf16", 1, 1, 32, 32, 128, 128),
        _linattn("step_b256", "linattn_step", "bf16", 256, 1, 8, 32, 128, 128),
        # the junction between two blocks: a decode batch of the 2.8B model's width, and a training batch
        _norm("norm_decode", "norm_fwd", "bf16", 8, 2560),
        _norm("norm_train", "norm_fwd", "bf16", 16384, 5120, residual="bf16"),
        # the gradient of the junction, and of a gated group norm (Mamba-2's) at an odd width in float32
        _norm("norm_bwd_train", "norm_bwd", "bf16", 16384, 2560),
        _norm("norm_bwd_gated_f32", "norm_bwd", "f32", 1001, 1530, groups=6, gate="before", residual="none",
              res_scale=False, next=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linattn_fwd", "linattn_fwd", "linattn_bwd", "linattn_step", "norm_fwd", "norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op.startswith("norm"):
        dim = _log(rng, 64, 8192)
        dim = dim if rng.random() < 0.3 else max(64, dim // 64 * 64)
        gate = rng.choice(("none", "before", "after"))
        weight = rng.random() < 0.8
        groups = rng.choice([n for n in (1, 1, 2, 4, 8) if dim % n == 0]) if weight else 1
        residual = rng.choice(("none", "f32", dtype))
        return _norm("", op, dtype, max(1, _log(rng, 1, 40_000_000 // dim)), dim, groups, gate, weight, residual,
                     residual != "none" and rng.random() < 0.5, rng.random() < 0.7)
    heads = rng.choice((1, 2, 4, 6, 8, 16, 24, 32))
    qk_heads = heads // rng.choice([n for n in (1, 1, 2, 4) if heads % n == 0])
    dk, dv = (rng.choice((16, 32, 48, 64, 64, 80, 96, 128, 128)) if rng.random() < 0.85 else rng.randint(8, 128)
              for _ in range(2))
    decay = rng.choice(("token", "token", "fixed", "none"))
    if op == "linattn_step":
        return _linattn("", op, dtype, _log(rng, 1, 8192 // heads), 1, qk_heads, heads, dk, dv, decay)
    tokens = (1 << 20 if op == "linattn_fwd" else 1 << 17) // (1 if dtype == "bf16" else 8)
    batch = _log(rng, 1, 8)
    seqlen = _log(rng, 1, min(65536, max(1, tokens // (batch * heads))))
    return _linattn("", op, dtype, batch, seqlen, qk_heads, heads, dk, dv, decay, rng.random() < 0.3,
                    rng.random() < 0.3, op == "linattn_fwd" and rng.random() < 0.7, rng.random() < 0.4)


def _decay(c, randn, rand):
    """Log decays: heads remember from 4 to 512 tokens, and a token's decay varies about its head's by a softplus gate."""
    H = c["heads"]
    window = torch.exp(rand(H) * (math.log(512.0) - math.log(4.0)) + math.log(4.0))
    if c["decay"] == "none":
        return None
    if c["decay"] == "fixed":
        return -1.0 / window
    return (-torch.nn.functional.softplus(randn(c["batch"], c["seqlen"], H) + 0.5) / window).to(TYPES[c["dtype"]])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)
    dt = TYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = dict(c)
    if c["op"].startswith("norm"):
        R, D = c["rows"], c["dim"]
        rt = dt if c["residual"] == "none" else TYPES[c["residual"]]
        s["x"] = randn(R, D).to(dt)
        s["z"] = randn(R, D).to(dt) if c["gate"] != "none" else None
        s["weight"] = 1.0 + 0.1 * randn(D) if c["weight"] else None
        s["res"] = (2.0 * randn(R, D)).to(rt) if c["residual"] != "none" else None
        s["res_scale_w"] = 0.3 + 0.05 * randn(D) if c["res_scale"] else None
        s["next_weight"] = 1.0 + 0.1 * randn(D) if c["next"] else None
        if c["op"] == "norm_bwd":
            s["dout"] = randn(R, D).to(rt)
            s["dy"] = randn(R, D).to(dt) if c["next"] else None
        return s
    B, L, Hq, H, dk, dv = c["batch"], c["seqlen"], c["qk_heads"], c["heads"], c["dk"], c["dv"]
    if c["op"] == "linattn_step":
        s["q"], s["k"], s["v"] = (randn(B, h, d).to(dt) for h, d in ((Hq, dk), (Hq, dk), (H, dv)))
        s["state"] = randn(B, H, dk, dv)
        g = _decay(c, randn, rand)
        s["g"] = g[:, 0].contiguous() if c["decay"] == "token" else g
        return s
    if c["fused"]:
        both = randn(B, L, 2 * Hq * dk + H * dv).to(dt)
        q, k, v = both.split((Hq * dk, Hq * dk, H * dv), dim=2)
        s["q"], s["k"], s["v"] = q.unflatten(2, (Hq, dk)), k.unflatten(2, (Hq, dk)), v.unflatten(2, (H, dv))
    else:
        s["q"], s["k"], s["v"] = (randn(B, L, h, d).to(dt) for h, d in ((Hq, dk), (Hq, dk), (H, dv)))
    s["g"] = _decay(c, randn, rand)
    s["h0"] = randn(B, H, dk, dv) if c["init"] else None
    s["seqlens"] = (rand(B) * (L + 1)).to(torch.int32) if c["ragged"] else None
    if c["op"] == "linattn_bwd":
        s["dy"] = randn(B, L, H, dv).to(dt)
    return s


# ---- plain forms ------------------------------------------------------------------------------------------------
def _plain_sweep(q, k, v, g, h0):
    """y_t = S_tᵀ q_t for [B, H, L, d] float32 and log decays [B, H, L] float64, in chunks: products inside a chunk,
    the chunks' own states, and a triangular product that brings the states of the chunks before. Returns y and the
    state after the last token."""
    B, H, L, dk = q.shape
    dv = v.shape[3]
    C = 64
    while C * 128 < L:
        C *= 2
    n = max(1, -(-L // C))
    pad = n * C - L
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).view(B, H, n, C, t.shape[3]) for t in (q, k, v))
    G = torch.nn.functional.pad(g, (0, pad)).view(B, H, n, C).cumsum(3)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).exp().float()
    y = (q @ k.transpose(3, 4) * D) @ v
    U = (k * (G[..., -1:] - G).exp().float()[..., None]).transpose(3, 4) @ v
    A = torch.nn.functional.pad(G[..., -1].cumsum(2), (1, 0))  # log decay of everything before chunk c
    T = (A[:, :, :, None] - A[:, :, None, 1:]).masked_fill(
        ~torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1), -math.inf).exp().float()
    S = (T @ U.reshape(B, H, n, dk * dv)).view(B, H, n + 1, dk, dv)
    if h0 is not None:
        S = S + A.exp().float()[..., None, None] * h0[:, :, None]
    y = y + (q * G.exp().float()[..., None]) @ S[:, :, :n]
    return y.reshape(B, H, n * C, dv)[:, :, :L], S[:, :, n]


def _plain_operands(s):
    """q, k, v as [B, H, L, d] float32 (shared heads repeated, nothing behind a row's length) and g as [B, H, L] float64."""
    c, rep = s, s["heads"] // s["qk_heads"]
    q, k, v = (t.float().transpose(1, 2) for t in (s["q"], s["k"], s["v"]))
    q, k = (t.repeat_interleave(rep, dim=1) for t in (q, k))
    shape = (c["batch"], c["heads"], c["seqlen"])
    if c["decay"] == "none":
        g = torch.zeros(shape, dtype=torch.float64, device=q.device)
    elif c["decay"] == "fixed":
        g = s["g"].double()[None, :, None].expand(shape)
    else:
        g = s["g"].double().transpose(1, 2)
    live = None
    if s["seqlens"] is not None:
        live = (torch.arange(c["seqlen"], device=q.device)[None, :] < s["seqlens"][:, None])[:, None]
        q, k, v = (t * live[..., None] for t in (q, k, v))
        g = g * live
    return q, k, v, g, live


def _plain_fwd(s):
    q, k, v, g, _ = _plain_operands(s)
    y, S = _plain_sweep(q, k, v, g, s["h0"])
    y = (y * s["dk"] ** -0.5).transpose(1, 2).to(s["v"].dtype).contiguous()
    return {"y": y, "state": S.contiguous()} if s["final"] else {"y": y}


def _plain_bwd(s):
    q, k, v, g, live = _plain_operands(s)
    scale = s["dk"] ** -0.5
    do = s["dy"].float().transpose(1, 2) * scale
    if live is not None:
        do = do * live[..., None]
    h0 = s["h0"].transpose(2, 3) if s["h0"] is not None else None
    dq, _ = _plain_sweep(do, v, k, g, h0)
    back = torch.cat([torch.zeros_like(g[..., :1]), g.flip(2)[..., :-1]], 2)  # decays between flipped neighbours
    qf, kf, vf, df = (t.flip(2) for t in (q, k, v, do))
    dk, M = _plain_sweep(vf, df, qf, back, None)
    dv, _ = _plain_sweep(kf, qf, df, back, None)
    dk, dv = dk.flip(2), dv.flip(2)
    dt = s["q"].dtype
    out = {"dv": dv.transpose(1, 2).to(dt).contiguous()}
    if s["decay"] == "token":
        both = (q.double() * dq).sum(3) - (k.double() * dk).sum(3)
        dg = both.flip(2).cumsum(2).flip(2)
        out["dlog_decay"] = (dg if live is None else dg * live).transpose(1, 2).to(dt).contiguous()
    rep = s["heads"] // s["qk_heads"]
    for name, t in (("dq", dq), ("dk", dk)):
        out[name] = t.unflatten(1, (s["qk_heads"], rep)).sum(2).transpose(1, 2).to(dt).contiguous()
    if s["h0"] is not None:
        out["dh0"] = (M * g[..., :1].exp().float()[..., None]).transpose(2, 3).contiguous()
    return out


def _plain_step(s):
    rep = s["heads"] // s["qk_heads"]
    q, k = (t.float().repeat_interleave(rep, dim=1) for t in (s["q"], s["k"]))
    a = 1.0 if s["g"] is None else (s["g"].float().exp()[..., None, None])
    s["state"].copy_(a * s["state"] + k[..., None] * s["v"].float()[..., None, :])
    y = (q[..., None, :] @ s["state"])[..., 0, :] * s["dk"] ** -0.5
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


def _plain_norm_parts(s):
    """The junction's values in float32, named as the gradient needs them."""
    x, D, n = s["x"].float(), s["dim"], s["groups"]
    v = {"x": x}
    if s["z"] is not None:
        z = s["z"].float()
        v["z"], v["sig"] = z, torch.sigmoid(z)
        v["gate"] = z * v["sig"]
    a = x * v["gate"] if s["gate"] == "before" else x
    p = a
    if s["weight"] is not None:
        ag = a.unflatten(1, (n, D // n))
        v["rstd"] = torch.rsqrt(ag.square().mean(2, keepdim=True) + EPS)
        v["n"] = (ag * v["rstd"]).flatten(1)
        p = v["n"] * s["weight"]
    v["p"] = p
    if s["gate"] == "after":
        p = p * v["gate"]
    v["pg"] = p
    r = p if s["res_scale_w"] is None else p * s["res_scale_w"]
    v["r"] = r if s["res"] is None else r + s["res"].float()
    if s["next_weight"] is not None:
        v["rstd2"] = torch.rsqrt(v["r"].square().mean(1, keepdim=True) + EPS)
        v["m"] = v["r"] * v["rstd2"]
    return v


def _plain_norm_fwd(s):
    v = _plain_norm_parts(s)
    rt = s["x"].dtype if s["res"] is None else s["res"].dtype
    out = {"out": v["r"].to(rt)}
    if s["next_weight"] is not None:
        out["y"] = (v["m"] * s["next_weight"]).to(s["x"].dtype)
    return out


def _plain_norm_bwd(s):
    v, D, n = _plain_norm_parts(s), s["dim"], s["groups"]
    out = {}
    dr = s["dout"].float()
    if s["next_weight"] is not None:
        dy = s["dy"].float()
        dm = dy * s["next_weight"]
        dr = dr + v["rstd2"] * (dm - v["m"] * (dm * v["m"]).mean(1, keepdim=True))
        out["dnext_weight"] = (dy * v["m"]).sum(0)
    if s["res"] is not None:
        out["dresidual"] = dr.to(s["res"].dtype)
    dp = dr
    if s["res_scale_w"] is not None:
        out["dres_scale"] = (dr * v["pg"]).sum(0)
        dp = dr * s["res_scale_w"]
    dgate = None
    if s["gate"] == "after":
        dgate = dp * v["p"]
        dp = dp * v["gate"]
    da = dp
    if s["weight"] is not None:
        out["dweight"] = (dp * v["n"]).sum(0)
        dn, nn = (dp * s["weight"]).unflatten(1, (n, D // n)), v["n"].unflatten(1, (n, D // n))
        da = (v["rstd"] * (dn - nn * (dn * nn).mean(2, keepdim=True))).flatten(1)
    if s["gate"] == "before":
        dgate = da * v["x"]
        da = da * v["gate"]
    out["dx"] = da.to(s["x"].dtype)
    if dgate is not None:
        out["dz"] = (dgate * v["sig"] * (1.0 + v["z"] * (1.0 - v["sig"]))).to(s["x"].dtype)
    return out


PLAIN = {"linattn_fwd": _plain_fwd, "linattn_bwd": _plain_bwd, "linattn_step": _plain_step,
         "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


# ---- the framework's calls ----------------------------------------------------------------------------------------
def _own(s):
    import selective_state_space_42_b200 as ss
    op = s["op"]
    if op == "linattn_fwd":
        r = ss.selscan_linattn_fwd(s["q"], s["k"], s["v"], s["g"], initial_state=s["h0"], seqlens=s["seqlens"],
                                   return_final_state=s["final"])
        return {"y": r[0], "state": r[1]} if s["final"] else {"y": r}
    if op == "linattn_bwd":
        r = ss.selscan_linattn_bwd(s["q"], s["k"], s["v"], s["g"], initial_state=s["h0"], seqlens=s["seqlens"],
                                   dy=s["dy"])
        return {n: r[n] for n in ("dq", "dk", "dv", "dlog_decay", "dh0") if r.get(n) is not None}
    if op == "linattn_step":
        y = ss.selscan_linattn_step(s["state"], s["q"], s["k"], s["v"], s["g"])
        return {"y": y, "state": s["state"]}
    kw = dict(z=s["z"], weight=s["weight"], residual=s["res"], res_scale=s["res_scale_w"],
              next_weight=s["next_weight"], groups=s["groups"], eps=EPS,
              gate=s["gate"] if s["z"] is not None else "after")
    if op == "norm_fwd":
        out, y = ss.selscan_block_norm_fwd(s["x"], **kw)
        return {"out": out} if y is None else {"out": out, "y": y}
    r = ss.selscan_block_norm_bwd(s["x"], dout=s["dout"], dy=s["dy"], **kw)
    return {n: t for n, t in r.items() if t is not None}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("norm"):
        n = c["rows"] * c["dim"]
        r = 0 if c["residual"] == "none" else 4 if c["residual"] == "f32" else 2
        ro = r or e
        z = e if c["gate"] != "none" else 0
        y = e if c["next"] else 0
        w = 4 * c["dim"] * (c["weight"] + c["res_scale"] + c["next"])
        if c["op"] == "norm_fwd":
            return {"bytes": n * (e + z + r + ro + y) + w, "flops": 20 * n}
        return {"bytes": n * (2 * e + 2 * z + 2 * r + ro + y) + 2 * w, "flops": 40 * n}
    B, L, Hq, H, dk, dv = c["batch"], c["seqlen"], c["qk_heads"], c["heads"], c["dk"], c["dv"]
    T = B * L
    g = e * T * H if c["decay"] == "token" else 0
    qk, v, st = 2 * e * T * Hq * dk, e * T * H * dv, 4 * B * H * dk * dv
    f = 4 * T * H * dk * dv
    if c["op"] == "linattn_step":
        return {"bytes": qk + 2 * v + g + 2 * st, "flops": f}
    if c["op"] == "linattn_fwd":
        return {"bytes": qk + 2 * v + g + st * (c["init"] + c["final"]), "flops": f}
    return {"bytes": 2 * qk + 3 * v + 2 * g + 2 * st * c["init"], "flops": 3 * f}


# ---- the definitions in float64 ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("norm"):
        return _exact_norm(s)
    if s["op"] == "linattn_step":
        rep = s["heads"] // s["qk_heads"]
        a = torch.ones(1, dtype=torch.float64, device="cuda") if s["g"] is None else torch.exp(s["g"].double())
        a = a.expand(s["batch"], s["heads"])
        q, k = (t.double().repeat_interleave(rep, 1) for t in (s["q"], s["k"]))
        S = a[:, :, None, None] * s["state"].double() + torch.einsum("bhk,bhv->bhkv", k, s["v"].double())
        return {"y": torch.einsum("bhk,bhkv->bhv", q, S) / math.sqrt(s["dk"]), "state": S}
    return _exact_recurrence(s)


def _exact_recurrence(s):
    """Token by token, and for the gradient token by token backwards."""
    B, L, H, rep = s["batch"], s["seqlen"], s["heads"], s["heads"] // s["qk_heads"]
    q, k = (t.double().repeat_interleave(rep, 2).transpose(0, 1).contiguous() for t in (s["q"], s["k"]))
    v = s["v"].double().transpose(0, 1).contiguous()
    if s["g"] is None:
        g = torch.zeros(L, B, H, dtype=torch.float64, device="cuda")
    else:
        g = s["g"].double().expand(B, L, H).transpose(0, 1).contiguous()
    if s["seqlens"] is not None:
        dead = torch.arange(L, device="cuda")[:, None] >= s["seqlens"][None, :]
        g = g.masked_fill(dead[..., None], 0.0)
        q, k, v = (t.masked_fill(dead[..., None, None], 0.0) for t in (q, k, v))
    a = g.exp()[..., None, None]
    scale = 1.0 / math.sqrt(s["dk"])
    S = torch.zeros(B, H, s["dk"], s["dv"], dtype=torch.float64, device="cuda") if s["h0"] is None \
        else s["h0"].double().clone()
    if s["op"] == "linattn_fwd":
        y = torch.empty_like(v)
        for t in range(L):
            S.mul_(a[t]).addcmul_(k[t].unsqueeze(3), v[t].unsqueeze(2))
            torch.matmul(q[t].unsqueeze(2), S, out=y[t].unsqueeze(2))
        y = (y * scale).transpose(0, 1)
        return {"y": y, "state": S} if s["final"] else {"y": y}
    do = s["dy"].double().transpose(0, 1) * scale
    if s["seqlens"] is not None:
        do = do.masked_fill(dead[..., None, None], 0.0)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S.mul_(a[t]).addcmul_(k[t].unsqueeze(3), v[t].unsqueeze(2))
        dq[t] = (S @ do[t].unsqueeze(3)).squeeze(3)
    N = torch.zeros_like(S)  # the loss's gradient with respect to the state, carried backwards
    for t in range(L - 1, -1, -1):
        N.addcmul_(q[t].unsqueeze(3), do[t].unsqueeze(2))
        dk[t] = (N @ v[t].unsqueeze(3)).squeeze(3)
        dv[t] = (k[t].unsqueeze(2) @ N).squeeze(2)
        N.mul_(a[t])
    out = {"dv": dv.transpose(0, 1)}
    for n, t in (("dq", dq), ("dk", dk)):
        out[n] = t.unflatten(2, (s["qk_heads"], rep)).sum(3).transpose(0, 1)
    if s["decay"] == "token":
        dg = torch.flip(torch.cumsum(torch.flip((q * dq).sum(3) - (k * dk).sum(3), (0,)), 0), (0,))
        if s["seqlens"] is not None:
            dg = dg.masked_fill(dead[..., None], 0.0)
        out["dlog_decay"] = dg.transpose(0, 1)
    if s["h0"] is not None:
        out["dh0"] = N
    return out


def _exact_norm(s):
    """The definition in float64, and its gradient by differentiating the definition."""
    names = {"x": "dx", "z": "dz", "res": "dresidual", "weight": "dweight", "res_scale_w": "dres_scale",
             "next_weight": "dnext_weight"}
    v = {n: None if s[n] is None else s[n].double().requires_grad_(s["op"] == "norm_bwd") for n in names}
    p = v["x"]
    gate = None if v["z"] is None else v["z"] / (1.0 + torch.exp(-v["z"]))
    if s["gate"] == "before":
        p = p * gate
    if v["weight"] is not None:
        t = p.reshape(s["rows"], s["groups"], -1)
        t = t / torch.sqrt((t * t).sum(2, keepdim=True) / t.shape[2] + EPS)
        p = t.reshape(s["rows"], s["dim"]) * v["weight"]
    if s["gate"] == "after":
        p = p * gate
    if v["res_scale_w"] is not None:
        p = v["res_scale_w"] * p
    out = p if v["res"] is None else v["res"] + p
    y = None
    if v["next_weight"] is not None:
        y = out / torch.sqrt((out * out).sum(1, keepdim=True) / s["dim"] + EPS) * v["next_weight"]
    if s["op"] == "norm_fwd":
        return {"out": out} if y is None else {"out": out, "y": y}
    loss = (out * s["dout"].double()).sum()
    if y is not None:
        loss = loss + (y * s["dy"].double()).sum()
    have = [n for n in names if v[n] is not None]
    return {names[n]: t for n, t in zip(have, torch.autograd.grad(loss, [v[n] for n in have]))}
