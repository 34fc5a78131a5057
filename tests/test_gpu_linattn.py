"""GPU parity of linear attention with a decay for each head (forward,
gradient, single token) against the float64 recurrence.

Tolerances, |gpu − oracle| ≤ rtol·(|oracle| + rms(oracle)): float32 I/O 1e-4
(sums of up to 192 float32 products a chunk, 2^-24 each against terms of at
most a few rms, weights from ex2.approx at 2^-22, a few tens of chunks).
bfloat16 I/O 2e-2: the output's rounding is at most 2^-8 of it, and the
operands rounded to bfloat16 (weights of the chunk's products, the entering
state) put an error of at most 2^-8 on each of many independent terms, six
standard deviations of whose sum are 6·2^-8/√3·√2 = 1.9e-2 of the rms.
The log decays' gradient is a running sum of q·dq − k·dk whose terms cancel, so
it carries their errors: e of |q||dq| + |k||dk| for each token, with e = 2^-20
in float32 (the weights' 2^-22 and a few sums) and 2^-17 where states enter as
pairs of bfloat16 (8 + 8 bits, half a step off); over up to L tokens these add
up to √L of their rms as independent errors, of which four deviations are
allowed on top of the relative bound.
"""
import math

import numpy as np
import pytest
import torch

import selective_state_space_42_b200 as ss
from oracle import linattn as lo

import gpu_helpers as gh

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, L, Hq, H, dk, dv, dtype, seed, decay="token", h0=False, strength=0.2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    i = dict(q=r(B, L, Hq, dk).to(DT[dtype]), k=r(B, L, Hq, dk).to(DT[dtype]),
             v=r(B, L, H, dv).to(DT[dtype]))
    if decay == "token":
        i["g"] = (-strength * torch.rand(B, L, H, generator=g)).to(DT[dtype])
    elif decay == "fixed":
        i["g"] = -strength * torch.rand(H, generator=g)
    else:
        i["g"] = None
    i["h0"] = r(B, H, dk, dv) if h0 else None
    i["dy"] = r(B, L, H, dv).to(DT[dtype])
    i["dS"] = r(B, H, dk, dv) if h0 else None
    return i


def dev(i):
    return {k: None if v is None else v.to(DEV) for k, v in i.items()}


def check_fwd(i, dtype, seqlens=None, what=""):
    d = dev(i)
    sl = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device=DEV)
    y, S = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                  seqlens=sl, return_final_state=True)
    torch.cuda.synchronize()
    n = gh.to_np
    yo, So = lo.linattn_fwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), i["q"].shape[3] ** -0.5,
                            n(i["h0"]), seqlens)
    gh.compare(n(y), yo, gh.RTOL[dtype], what + " y")
    gh.compare(n(S), So, 1e-4, what + " state")  # float32 whatever the I/O type


def check_bwd(i, dtype, seqlens=None, what=""):
    d = dev(i)
    sl = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device=DEV)
    got = ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                 seqlens=sl, dy=d["dy"], dfinal_state=d["dS"])
    torch.cuda.synchronize()
    n = gh.to_np
    want = lo.linattn_bwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), i["q"].shape[3] ** -0.5,
                          n(i["h0"]), seqlens, n(i["dy"]), n(i["dS"]))
    for k in ("dq", "dk", "dv"):
        gh.compare(n(got[k]), want[k], gh.RTOL[dtype], f"{what} {k}")
    assert (got["dlog_decay"] is not None) == (i["g"] is not None and i["g"].dim() == 3)
    if got["dlog_decay"] is not None:
        o, d = want["dlog_decay"], n(got["dlog_decay"])
        assert np.isfinite(d).all(), what
        per = sum(np.sqrt((n(i[a]) ** 2).sum(3) * (want["d" + a] ** 2).sum(3)) for a in "qk")
        live = per[np.isfinite(per)]
        L = o.shape[1]
        e = {"f32": 2.0 ** -20, "bf16": 2.0 ** -17}[dtype]
        bound = gh.RTOL[dtype] * (np.abs(o) + np.sqrt((o * o).mean())) \
            + 4 * e * math.sqrt(L) * np.sqrt((live * live).mean())
        assert (np.abs(d - o) <= bound).all(), (what, float((np.abs(d - o) / bound).max()))
    assert (got["dh0"] is not None) == (i["h0"] is not None)
    if got["dh0"] is not None:
        gh.compare(n(got["dh0"]), want["dh0"], 1e-4, what + " dh0")


SHAPES = [  # B, L, Hq, H, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 2, 1, 2, 8, 8), (1, 63, 2, 2, 64, 64), (1, 64, 1, 1, 128, 128),
    (2, 65, 2, 4, 64, 128), (1, 129, 3, 3, 128, 64), (2, 200, 1, 4, 16, 24), (1, 130, 5, 5, 7, 33),
    (1, 300, 2, 2, 72, 120), (3, 128, 1, 2, 48, 80), (1, 191, 2, 2, 32, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    check_fwd(make(*shape, dtype, 100 + shape[1]), dtype, what=str(shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "fixed", "none"])
def test_forward_decays_from_a_state(dtype, decay):
    check_fwd(make(2, 150, 2, 4, 64, 64, dtype, 7, decay, h0=True), dtype, what=decay)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(shape, dtype):
    check_bwd(make(*shape, dtype, 200 + shape[1]), dtype, what=str(shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "fixed", "none"])
def test_gradient_decays_from_a_state(dtype, decay):
    check_bwd(make(2, 150, 2, 4, 64, 72, dtype, 8, decay, h0=True), dtype, what=decay)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2100, 1, 1, 64, 64), (1, 2100, 1, 2, 128, 128)], ids=str)
def test_segments(shape, dtype):
    """One or two heads over 33 chunks: the sequence is cut into segments."""
    i = make(*shape, dtype, 9, h0=True, strength=0.05)
    check_fwd(i, dtype, what="segments")
    check_bwd(i, dtype, what="segments")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("strength", [3.0, 40.0])
def test_steep_decays(dtype, strength):
    """Decays whose sums leave float32's exponent range inside a chunk."""
    i = make(1, 200, 2, 2, 64, 64, dtype, 10, h0=True, strength=strength)
    check_fwd(i, dtype, what="steep")
    check_bwd(i, dtype, what="steep")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [-math.inf, torch.finfo(torch.bfloat16).min])
def test_resets(dtype, value):
    """A log decay of −∞ or the type's lowest value: nothing from before counts,
    also when it stands on the first token of a state that holds NaN."""
    i = make(2, 150, 2, 2, 64, 64, dtype, 11, h0=True)
    i["g"][0, [3, 70, 71, 128]] = value
    i["g"][1, :, 1] = value  # every token of a head
    check_fwd(i, dtype, what="resets")
    check_bwd(i, dtype, what="resets")
    i["g"][:, 0] = value
    clean = dev(i)
    y0, S0 = ss.selscan_linattn_fwd(clean["q"], clean["k"], clean["v"], clean["g"],
                                    return_final_state=True)
    y1, S1 = ss.selscan_linattn_fwd(clean["q"], clean["k"], clean["v"], clean["g"],
                                    initial_state=torch.full_like(clean["h0"], math.nan),
                                    return_final_state=True)
    assert torch.equal(y0, y1) and torch.equal(S0, S1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ragged_rows(dtype):
    """Lengths 0, 1, inside a chunk, on its edge, whole; one beyond the tensor
    and one negative are clamped. What stands behind a length may be anything."""
    lens = [0, 1, 77, 128, 200, 999, -5]
    i = make(7, 200, 1, 2, 64, 64, dtype, 12, h0=True)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "dy"):
            i[name][b, max(n, 0):] = [math.nan, math.inf][b % 2]
    n0 = {k: v for k, v in i.items()}
    for name in ("q", "k", "v", "g", "dy"):  # the oracle does not read them either
        n0[name] = i[name]
    check_fwd(n0, dtype, lens, "ragged")
    check_bwd(n0, dtype, lens, "ragged")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ragged_segments(dtype):
    lens = [0, 700, 2100]
    i = make(3, 2100, 1, 1, 64, 64, dtype, 13, h0=True, strength=0.05)
    check_fwd(i, dtype, lens, "ragged segments")
    check_bwd(i, dtype, lens, "ragged segments")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_one_projection(dtype):
    """q, k and v as views of one [B, L, *] tensor give what copies give, bit by bit."""
    B, L, Hq, H, dk, dv = 2, 150, 2, 4, 64, 64
    both = torch.randn(B, L, 2 * Hq * dk + H * dv, device=DEV).to(DT[dtype])
    q, k, v = both.split((Hq * dk, Hq * dk, H * dv), 2)
    q, k, v = q.unflatten(2, (Hq, dk)), k.unflatten(2, (Hq, dk)), v.unflatten(2, (H, dv))
    g = (-0.1 * torch.rand(B, L, H, device=DEV)).to(DT[dtype])
    dy = torch.randn(B, L, H, dv, device=DEV).to(DT[dtype])
    c = [t.contiguous() for t in (q, k, v)]
    assert torch.equal(ss.selscan_linattn_fwd(q, k, v, g), ss.selscan_linattn_fwd(*c, g))
    a = ss.selscan_linattn_bwd(q, k, v, g, dy=dy)
    b = ss.selscan_linattn_bwd(*c, g, dy=dy)
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert torch.equal(a[n], b[n]), n
    with pytest.raises(ValueError, match="contiguous"):
        ss.selscan_linattn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)
    with pytest.raises(ValueError, match="contiguous"):
        ss.selscan_linattn_fwd(c[0][:, :, :1].expand(B, L, Hq, dk), k, v)


def _misaligned(t):
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = buf[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_off_16_bytes(dtype):
    i = make(1, 100, 2, 2, 64, 64, dtype, 14, h0=True)
    d = dev(i)
    for k in ("q", "k", "v"):
        d[k] = _misaligned(d[k])
    y = _misaligned(torch.zeros_like(d["v"]))
    ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"], y=y)
    n = gh.to_np
    yo, _ = lo.linattn_fwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), 0.125, n(i["h0"]))
    gh.compare(n(y), yo, gh.RTOL[dtype], "misaligned y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,heads", [(200, 2), (2100, 1)])
def test_state_in_place_and_repeats(dtype, L, heads):
    """final_state may be the initial state itself; two calls give the same bits."""
    d = dev(make(1, L, heads, heads, 64, 64, dtype, 15, h0=True))
    y0, S0 = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                    return_final_state=True)
    st = d["h0"].clone()
    y1 = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=st, final_state=st)
    assert torch.equal(y0, y1) and torch.equal(S0, st)
    a, b = (ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                   dy=d["dy"], dfinal_state=d["dS"]) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_sizes(dtype):
    z = lambda *s: torch.zeros(*s, device=DEV, dtype=DT[dtype])  # noqa: E731
    h0 = torch.randn(2, 3, 8, 8, device=DEV)
    y, S = ss.selscan_linattn_fwd(z(2, 0, 3, 8), z(2, 0, 3, 8), z(2, 0, 3, 8), initial_state=h0,
                                  return_final_state=True)
    assert y.shape == (2, 0, 3, 8) and torch.equal(S, h0)
    g = ss.selscan_linattn_bwd(z(2, 0, 3, 8), z(2, 0, 3, 8), z(2, 0, 3, 8), initial_state=h0,
                               dy=z(2, 0, 3, 8), dfinal_state=h0)
    assert torch.equal(g["dh0"], h0)
    assert ss.selscan_linattn_fwd(z(0, 4, 3, 8), z(0, 4, 3, 8), z(0, 4, 3, 8)).numel() == 0
    assert ss.selscan_linattn_step(torch.zeros(0, 3, 8, 8, device=DEV), z(0, 3, 8), z(0, 3, 8),
                                   z(0, 3, 8)).numel() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (2, 2, 4, 128, 128), (5, 3, 3, 64, 64),
                                   (3, 1, 2, 17, 33), (300, 1, 2, 32, 16), (160, 2, 4, 128, 120),
                                   (200, 2, 2, 100, 48)], ids=str)
@pytest.mark.parametrize("decay", ["token", "fixed", "none"])
def test_step(shape, dtype, decay):
    B, Hq, H, dk, dv = shape
    i = make(B, 1, Hq, H, dk, dv, dtype, 16, decay, h0=True)
    d = dev(i)
    st = d["h0"].clone()
    g = d["g"][:, 0].contiguous() if decay == "token" else d["g"]
    y = ss.selscan_linattn_step(st, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], g)
    n = gh.to_np
    yo, So = lo.linattn_fwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), dk ** -0.5, n(i["h0"]))
    gh.compare(n(y), yo[:, 0], gh.RTOL[dtype], "step y")
    gh.compare(n(st), So, 1e-5, "step state")  # two products and a sum in float32


def test_step_resets_a_state_of_nan():
    q = torch.randn(2, 2, 16, device=DEV)
    for dv in (16, 15):
        v = torch.randn(2, 2, dv, device=DEV)
        st = torch.full((2, 2, 16, dv), math.nan, device=DEV)
        y = ss.selscan_linattn_step(st, q, q, v, torch.full((2, 2), -math.inf, device=DEV), 1.0)
        want = (q * q).sum(-1, keepdim=True) * v
        assert torch.allclose(y, want, rtol=1e-5, atol=1e-5) and not torch.isnan(st).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens(dtype):
    """A prompt, continued by a second call from its state and then token by
    token, equals the whole sequence in one call."""
    i = make(2, 150, 2, 4, 64, 64, dtype, 17)
    d = dev(i)
    cut = lambda a, b: [d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")]  # noqa: E731
    y1, S = ss.selscan_linattn_fwd(*cut(0, 70), return_final_state=True)
    y2 = ss.selscan_linattn_fwd(*cut(70, 147), initial_state=S, final_state=S)
    ys = [y1, y2]
    for t in range(147, 150):
        q, k, v, g = (x[:, 0].contiguous() for x in cut(t, t + 1))
        ys.append(ss.selscan_linattn_step(S, q, k, v, g)[:, None])
    n = gh.to_np
    yo, So = lo.linattn_fwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), 0.125)
    gh.compare(n(torch.cat(ys, 1)), yo, gh.RTOL[dtype], "continued y")
    gh.compare(n(S), So, 1e-4, "continued state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_on_another_stream(dtype):
    """Captured into a graph and replayed on new inputs, and launched on a
    stream that is not the current one."""
    i, j = (make(1, 700, 2, 2, 64, 64, dtype, s) for s in (18, 19))
    d, e = dev(i), dev(j)

    def both():
        y = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"])
        g = ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], dy=d["dy"])
        return [y, *(g[n] for n in ("dq", "dk", "dv", "dlog_decay"))]

    first = [t.clone() for t in both()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], stream=s)
    y2 = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, first[0]) and torch.equal(y2, first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, first):
        assert torch.equal(a, b)
    for n in ("q", "k", "v", "g", "dy"):
        d[n].copy_(e[n])
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in held]
    for a, b in zip(replayed, both()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_agrees_with_the_one_group_scan(dtype):
    """With k = B, q = C shared by all heads, v = Δ·x and g = Δ·A this is the
    scan with one scalar A per head."""
    B, L, H, P, N = 2, 200, 4, 64, 64
    g = torch.Generator().manual_seed(20)
    x = torch.randn(B, L, H * P, generator=g).to(DT[dtype]).to(DEV)
    Bm, Cm = (torch.randn(B, L, N, generator=g).to(DT[dtype]).to(DEV) for _ in range(2))
    dt = torch.full((B, L, H), 0.5, device=DEV, dtype=DT[dtype])
    A = torch.tensor([-0.25, -0.5, -0.0625, -0.125], device=DEV)
    want, Sw = ss.selscan_ssd_fwd(x, dt, A, Bm, Cm, softplus=False, return_final_state=True)
    y, S = ss.selscan_linattn_fwd(Cm[:, :, None], Bm[:, :, None], (x * 0.5).unflatten(2, (H, P)),
                                  (dt * A).to(DT[dtype]), scale=1.0, return_final_state=True)
    gh.compare(gh.to_np(y.flatten(2)), gh.to_np(want), gh.RTOL[dtype], "scan y")
    gh.compare(gh.to_np(S.transpose(2, 3).reshape(B, H * P, N)), gh.to_np(Sw),
               gh.RTOL[dtype], "scan state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,d", [(330, 64), (330, 128), (2100, 128), (1500, 48)])
def test_chunks_of_unlike_decays(dtype, L, d):
    """Slow and steep stretches that begin and end on chunk edges and inside
    chunks, with resets among them: each kind of chunk follows each other."""
    i = make(1, L, 2, 2, d, d, dtype, 21, h0=True, strength=0.05)
    for a, b in ((64, 128), (192, 200), (250, 320), (640, 896), (1000, 1001)):
        i["g"][:, a:b] *= 400
    i["g"][0, 130::97] = -math.inf
    check_fwd(i, dtype, what="unlike")
    check_bwd(i, dtype, what="unlike")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [130, 2100])
def test_fixed_decays_of_every_size(dtype, L):
    """Fixed decays of nothing, of 1/2 a token, of e^-60 and of a reset at each token."""
    i = make(1, L, 4, 4, 64, 128, dtype, 22, "fixed", h0=True)
    i["g"] = torch.tensor([0.0, -0.6931, -60.0, -math.inf])
    i["v"] *= 0.1
    check_fwd(i, dtype, what="fixed")
    check_bwd(i, dtype, what="fixed")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales(dtype):
    """A scale is a factor of y and of every gradient; zero gives zeros, and the
    state has none. Powers of two: the same bits times the factor."""
    d = dev(make(2, 150, 1, 2, 64, 64, dtype, 23, h0=True))
    a = (d["q"], d["k"], d["v"], d["g"])
    kw = dict(initial_state=d["h0"], return_final_state=True)
    y1, S1 = ss.selscan_linattn_fwd(*a, scale=0.125, **kw)
    g1 = ss.selscan_linattn_bwd(*a, scale=0.125, initial_state=d["h0"], dy=d["dy"])
    for f in (-1.0, 2.0, 0.0):
        y, S = ss.selscan_linattn_fwd(*a, scale=0.125 * f, **kw)
        g = ss.selscan_linattn_bwd(*a, scale=0.125 * f, initial_state=d["h0"], dy=d["dy"])
        assert torch.equal(S, S1) and torch.equal(y, y1 * f)
        for n in ("dq", "dk", "dv", "dh0"):
            assert torch.equal(g[n], g1[n] * f), (f, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_heads_and_ragged_rows(dtype):
    """Heads in groups of four over rows of unequal length, gradients of the
    shared heads summed in float32."""
    lens = [0, 130, 61]
    i = make(3, 130, 2, 8, 64, 128, dtype, 24, h0=True)
    check_fwd(i, dtype, lens, "shared ragged")
    check_bwd(i, dtype, lens, "shared ragged")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("given", ["h0", "dS", "neither"])
def test_growing_states_and_one_state_given(dtype, given):
    """Log decays of both signs, and a first state without a last one's gradient
    and the other way round, over several segments."""
    i = make(1, 1000, 1, 2, 64, 64, dtype, 30, h0=True)
    i["g"] = (i["g"].float() * 0.25 * torch.tensor([1.0, -0.1])).to(DT[dtype])
    for n in {"h0", "dS"} - {given}:
        i[n] = None
    check_fwd(i, dtype, what="growing")
    check_bwd(i, dtype, what="growing")


@pytest.mark.parametrize("d", [48, 64, 128])
def test_states_of_bfloat16_operands_keep_float32(d):
    """The float32 results of bfloat16 operands, the last state and the first
    one's gradient, to 2^-18 of their size: over five chunks the decays and a
    token's weight are ten exponentials of 2^-22 at most, and the sums of 320 terms
    round by less than six more together."""
    i = make(2, 300, 2, 2, d, d, "bf16", 32, h0=True, strength=0.02)
    v = dev(i)
    n = gh.to_np
    a = (n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), d ** -0.5, n(i["h0"]), None)
    _, S = ss.selscan_linattn_fwd(v["q"], v["k"], v["v"], v["g"], initial_state=v["h0"],
                                  return_final_state=True)
    gh.compare(n(S), lo.linattn_fwd(*a)[1], 2.0 ** -18, "state")
    g = ss.selscan_linattn_bwd(v["q"], v["k"], v["v"], v["g"], initial_state=v["h0"],
                               dy=v["dy"], dfinal_state=v["dS"])
    gh.compare(n(g["dh0"]), lo.linattn_bwd(*a, n(i["dy"]), n(i["dS"]))["dh0"], 2.0 ** -18, "dh0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_tensor_for_all_operands(dtype):
    d = dev(make(1, 150, 2, 2, 64, 64, dtype, 31))
    x = d["q"]
    a = ss.selscan_linattn_bwd(x, x, x, d["g"], dy=x)
    b = ss.selscan_linattn_bwd(x.clone(), x.clone(), x.clone(), d["g"], dy=x.clone())
    assert torch.equal(ss.selscan_linattn_fwd(x, x, x, d["g"]),
                       ss.selscan_linattn_fwd(x.clone(), x.clone(), x.clone(), d["g"]))
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_calls_at_once(dtype):
    """Calls on two streams at a time, each with its own workspace, give what
    they give one after the other."""
    ds = [dev(make(1, 1900, 2, 2, 128, 128, dtype, s, h0=True)) for s in (25, 26)]

    def run(d, stream):
        y, S = ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                      return_final_state=True, stream=stream)
        g = ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                   dy=d["dy"], dfinal_state=d["dS"], stream=stream)
        return [y, S, *g.values()]

    want = [[t.clone() for t in run(d, None)] for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[], []]
    for _ in range(3):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                got[n].append(run(ds[n], None))
    torch.cuda.synchronize()
    for n in range(2):
        for again in got[n]:
            for a, b in zip(again, want[n]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_rows_than_a_grid_dimension(dtype):
    check_fwd(make(70001, 1, 1, 1, 8, 8, dtype, 27, h0=True), dtype, what="rows")
    check_bwd(make(70001, 1, 1, 1, 8, 8, dtype, 28, h0=True), dtype, what="rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_beyond_32_bits(dtype):
    """Slices of tokens 2^22 elements apart: the last ones stand past 2^31."""
    L, step = 520, 1 << 22
    i = dev(make(1, L, 1, 1, 64, 64, dtype, 29))
    wide = torch.empty(L * step, device=DEV, dtype=DT[dtype])
    at = lambda o: wide.as_strided((1, L, 1, 64), (L * step, step, 64, 1), o)  # noqa: E731
    q, k, v = at(0), at(64), at(128)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(i[n])
    assert torch.equal(ss.selscan_linattn_fwd(q, k, v, i["g"]),
                       ss.selscan_linattn_fwd(i["q"], i["k"], i["v"], i["g"]))
    a = ss.selscan_linattn_bwd(q, k, v, i["g"], dy=i["dy"])
    b = ss.selscan_linattn_bwd(i["q"], i["k"], i["v"], i["g"], dy=i["dy"])
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert torch.equal(a[n], b[n]), n


def test_no_device_wait_gave_up():
    torch.cuda.synchronize()
    assert ss.selscan_device_status() == 0
