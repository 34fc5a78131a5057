"""GPU parity of the block-norm junction and its gradient against float64.

Tolerances, |gpu − oracle| ≤ rtol·(|oracle| + rms(oracle)): float32 results
1e-5·√(terms / 64) for column sums over many rows and 1e-5 else (a handful of
float32 roundings of 2^-24 and a sum whose terms add up without cancelling;
silu from ex2.approx and rcp.approx, 2^-21 together); bfloat16 results 2^-8
of the value for the store's rounding, on top of that 1e-5. Where a norm's
gradient subtracts dn − n·mean(dn·n), the difference carries the rounding of
its parts: 2^-20 of their size (four roundings of 2^-24 and the statistics'
2^-22), which counts where the two all but cancel (rows of one element).
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


def make(R, D, dtype, seed, z=True, weight=True, res="f32", scale=True, nxt=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rt = DT[dtype if res is None else res]
    i = dict(x=r(R, D).to(DT[dtype]), z=r(R, D).to(DT[dtype]) if z else None,
             weight=1 + 0.1 * r(D) if weight else None,
             residual=r(R, D).to(rt) if res else None,
             res_scale=0.5 + 0.1 * r(D) if scale else None,
             next_weight=1 + 0.1 * r(D) if nxt else None)
    grads = dict(dout=r(R, D).to(rt), dy=r(R, D).to(DT[dtype]) if nxt else None)
    return i, grads


def sizes(n, grads, groups, gate, eps):
    """Sizes of the parts that dresidual, dx and dz are differences of."""
    _, _, c = lo.block_norm_fwd(**n, groups=groups, gate=gate, eps=eps)
    dr = 0.0 if grads["dout"] is None else np.abs(gh.to_np(grads["dout"]))
    if n["next_weight"] is not None:
        dr = dr + c["rstd2"] * np.abs(gh.to_np(grads["dy"]) * n["next_weight"])
    d = dr if n["res_scale"] is None else dr * np.abs(n["res_scale"])
    gz = None if n["z"] is None else np.abs(c["gz"])
    dgate = 0.0
    if n["z"] is not None and gate == "after":
        dgate, d = d * np.abs(c["p"]), d * gz
    if n["weight"] is not None:
        d = (np.abs(d * n["weight"]).reshape(len(d), groups, -1) * c["rstd"]).reshape(d.shape)
    if n["z"] is not None and gate == "before":
        dgate, d = d * np.abs(n["x"]), d * gz
    return {"dresidual": dr, "dx": d, "dz": 1.1 * dgate}


def near(got, want, what, size=0.0):
    assert got is not None, what
    g, o = gh.to_np(got), np.asarray(want)
    assert g.shape == o.shape and np.isfinite(g).all(), what
    rms = math.sqrt(float((o * o).mean())) if o.size else 0.0
    rt = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    bad = np.abs(g - o) > rt * np.abs(o) + 1e-5 * (np.abs(o) + rms) + 2.0 ** -20 * size + 1e-37
    assert not bad.any(), (what, float(np.abs(g - o).max()), rms)


def check(i, grads, groups=1, gate="after", eps=1e-5, what=""):
    d = {k: None if v is None else v.to(DEV) for k, v in i.items()}
    dg = {k: None if v is None else v.to(DEV) for k, v in grads.items()}
    n = {k: gh.to_np(v) for k, v in i.items()}
    kw = dict(groups=groups, gate=gate, eps=eps)
    out, y = ss.selscan_block_norm_fwd(**d, **kw)
    wo, wy, _ = lo.block_norm_fwd(**n, **kw)
    near(out, wo, what + " out")
    assert (y is None) == (wy is None)
    if y is not None:
        near(y, wy, what + " y")
    got = ss.selscan_block_norm_bwd(**d, **dg, **kw)
    want = lo.block_norm_bwd(**n, **{k: gh.to_np(v) for k, v in grads.items()}, **kw)
    assert {k for k, v in got.items() if v is not None} == set(want)
    rows = i["x"].shape[0]
    size = sizes(n, grads, **kw)
    for k in want:
        if k in ("dweight", "dres_scale", "dnext_weight"):
            o, g = want[k], gh.to_np(got[k])
            rms = math.sqrt(float((o * o).mean()))
            assert (np.abs(g - o) <= 1e-5 * max(1.0, math.sqrt(rows / 64)) * (np.abs(o) + rms)
                    + 1e-37).all(), (what, k)
        else:
            near(got[k], want[k], f"{what} {k}", size[k])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["before", "after", None])
@pytest.mark.parametrize("shape", [(1, 1), (3, 8), (5, 30), (7, 64), (130, 256), (33, 1000),
                                   (9, 1530), (4, 2560), (6, 4104), (3, 5120), (2, 8200),
                                   (2, 16384), (2, 12001)], ids=str)
def test_whole_junction(shape, dtype, gate):
    i, g = make(*shape, dtype, shape[1], z=gate is not None)
    check(i, g, gate=gate or "after", what=f"{shape} {gate}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,groups", [(64, 2), (64, 64), (96, 3), (1530, 6), (2048, 8), (2560, 5),
                                      (4096, 512), (1000, 1000), (16000, 100), (15500, 100),
                                      (8192, 2)])
@pytest.mark.parametrize("gate", ["before", "after"])
def test_groups(D, groups, gate, dtype):
    i, g = make(5, D, dtype, D + groups)
    check(i, g, groups=groups, gate=gate, what=f"{D}/{groups}")


@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                       ("f32", None), ("bf16", None)])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("nxt", [True, False])
@pytest.mark.parametrize("z", [True, False])
def test_every_set_of_parts(dtype, res, weight, scale, nxt, z):
    i, g = make(11, 192, dtype, 3, z, weight, res, scale, nxt)
    check(i, g, what=f"{dtype} {res} {weight} {scale} {nxt} {z}")


def test_many_rows():
    """More rows than the gradient has blocks: several rows a block, in each map."""
    for D in (16, 64, 520, 2560):
        i, g = make(1500, D, "f32", D)
        check(i, g, what=f"1500 x {D}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_zeros_and_large_values(dtype):
    """A row of zeros (the norm of nothing: eps alone) and rows near the square
    root of float32's range."""
    i, g = make(4, 128, dtype, 4)
    i["x"][0] = 0
    i["residual"][0] = 0
    i["x"][1] *= 2.0 ** 55
    i["z"][2] = torch.linspace(-300, 300, 128).to(i["z"].dtype)
    check(i, g, what="zeros")


def test_only_one_gradient_comes_in():
    i, g = make(6, 200, "bf16", 6)
    d = {k: v.to(DEV) for k, v in i.items()}
    n = {k: gh.to_np(v) for k, v in i.items()}
    got = ss.selscan_block_norm_bwd(**d, dy=g["dy"].to(DEV))
    want = lo.block_norm_bwd(**n, dy=gh.to_np(g["dy"]))
    for k in ("dx", "dz", "dresidual"):
        near(got[k], want[k], k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_and_leading_dimensions(dtype):
    """x and z as slices of one projection [B, L, 2·D] give what copies give."""
    both = torch.randn(2, 9, 2 * 64, device=DEV).to(DT[dtype])
    x, z = both.split(64, 2)
    w = torch.rand(64, device=DEV)
    a = ss.selscan_block_norm_fwd(x, z, w)[0]
    b = ss.selscan_block_norm_fwd(x.contiguous(), z.contiguous(), w)[0]
    assert a.shape == (2, 9, 64) and torch.equal(a, b)
    dout = torch.randn_like(a)
    ga, gb = (ss.selscan_block_norm_bwd(*t, w, dout=dout)
              for t in ((x, z), (x.contiguous(), z.contiguous())))
    for k in ("dx", "dz", "dweight"):
        assert torch.equal(ga[k], gb[k])
    with pytest.raises(ValueError, match="spaced"):
        ss.selscan_block_norm_fwd(torch.randn(9, 2, 64, device=DEV).to(DT[dtype])
                                  .transpose(0, 1), z, w)
    with pytest.raises(ValueError, match="spaced"):
        ss.selscan_block_norm_fwd(x[:1, :1].expand(2, 9, 64), z, w)


def test_off_16_bytes_in_place_empty_and_repeats():
    i, g = make(7, 256, "bf16", 8, res="bf16")
    d = {k: v.to(DEV) for k, v in i.items()}
    out, y = ss.selscan_block_norm_fwd(**d)
    buf = torch.empty(7 * 256 + 8, device=DEV, dtype=torch.bfloat16)
    xm = buf[1:1 + 7 * 256].view(7, 256)
    xm.copy_(d["x"])
    o2, y2 = ss.selscan_block_norm_fwd(**{**d, "x": xm})
    near(o2, gh.to_np(out), "misaligned out")
    r = d["residual"].clone()
    o3, y3 = ss.selscan_block_norm_fwd(**{**d, "residual": r}, out=r)
    assert o3 is r and torch.equal(r, out) and torch.equal(y3, y)
    e = torch.empty(0, 256, device=DEV, dtype=torch.bfloat16)
    oe, ye = ss.selscan_block_norm_fwd(e, weight=d["weight"], next_weight=d["next_weight"])
    assert oe.shape == ye.shape == (0, 256)
    ge = ss.selscan_block_norm_bwd(e, weight=d["weight"], dout=e)
    assert torch.equal(ge["dweight"], torch.zeros(256, device=DEV))
    a, b = (ss.selscan_block_norm_bwd(**d, dout=g["dout"].to(DEV), dy=g["dy"].to(DEV))
            for _ in range(2))
    for k in a:
        assert torch.equal(a[k], b[k])


def test_captured_and_on_another_stream():
    i, g = make(300, 640, "bf16", 9)
    d = {k: v.to(DEV) for k, v in i.items()}
    dg = {k: v.to(DEV) for k, v in g.items()}

    def both():
        return [*ss.selscan_block_norm_fwd(**d), *ss.selscan_block_norm_bwd(**d, **dg).values()]

    first = [t.clone() for t in both()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, y = ss.selscan_block_norm_fwd(**d, stream=s)
    s.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(y, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    d["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in held]
    for a, b in zip(replayed, both()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,groups,gate,res,parts", [
    (2560, 1, "after", "f32", {}), (2560, 5, "before", "bf16", {}),
    (1536, 48, "before", "bf16", {}), (5120, 8, "before", "bf16", {"res": None}),
    (5120, 1, "after", "f32", {"weight": False}), (10240, 1, "after", "bf16", {"nxt": False}),
    (2048, 1, "after", "f32", {"weight": False, "nxt": False}), (640, 1, "after", "f32", {"z": False}),
    (16384, 1, "after", "bf16", {"scale": False}),
], ids=str)
def test_many_rows_of_bfloat16(D, groups, gate, res, parts):
    """Rows enough for several a block, brought in ahead of their use, with every
    kind of operand there or not."""
    i, g = make(1301, D, "bf16", D + 1, **{"res": res, **parts})
    check(i, g, groups=groups, gate=gate, what=f"1301 x {D} {parts}")


def test_many_rows_of_slices_captured_and_two_at_once():
    """x and z of one projection, replayed in a graph on new inputs and run on
    two streams at a time: the same bits as alone."""
    R, D = 1400, 2048
    i, g = make(R, D, "bf16", 12)
    d = {k: v.to(DEV) for k, v in i.items()}
    dg = {k: v.to(DEV) for k, v in g.items()}
    both = torch.cat([d["x"], d["z"]], 1)
    sliced = {**d, "x": both[:, :D], "z": both[:, D:]}

    def run(a):
        return [*ss.selscan_block_norm_fwd(**a), *ss.selscan_block_norm_bwd(**a, **dg).values()]

    want = [t.clone() for t in run(d)]
    for a, b in zip(run(sliced), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got += [run(sliced), run(sliced)]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(sliced)
    both.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip([t.clone() for t in held], run(sliced)):
        assert torch.equal(a, b)


def test_many_rows_in_place():
    """out in the residual's place, over rows brought ahead."""
    i, _ = make(1400, 1024, "bf16", 13, res="bf16")
    d = {k: v.to(DEV) for k, v in i.items()}
    out, y = ss.selscan_block_norm_fwd(**d)
    r = d["residual"].clone()
    o2, y2 = ss.selscan_block_norm_fwd(**{**d, "residual": r}, out=r)
    assert o2 is r and torch.equal(r, out) and torch.equal(y2, y)


def test_more_rows_than_a_grid_dimension_and_beyond_32_bits():
    """70001 rows of 8, and rows of slices 2^22 elements apart that pass 2^31."""
    i, g = make(70001, 8, "bf16", 14)
    check(i, g, what="70001 x 8")
    i, g = make(1300, 256, "bf16", 15)
    d = {k: v.to(DEV) for k, v in i.items()}
    dg = {k: v.to(DEV) for k, v in g.items()}
    wide = torch.empty(1300 << 22, device=DEV, dtype=torch.bfloat16)
    x = wide.as_strided((1300, 256), (1 << 22, 1), 0)
    z = wide.as_strided((1300, 256), (1 << 22, 1), 1 << 12)
    x.copy_(d["x"])
    z.copy_(d["z"])
    for a, b in zip(ss.selscan_block_norm_fwd(**{**d, "x": x, "z": z}),
                    ss.selscan_block_norm_fwd(**d)):
        assert torch.equal(a, b)
    a = ss.selscan_block_norm_bwd(**{**d, "x": x, "z": z}, **dg)
    b = ss.selscan_block_norm_bwd(**d, **dg)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_block_and_its_gradient(dtype):
    """Norm, linear attention, gated norm and residual sum as a model runs them,
    its gradient chained through the operators, against float64."""
    B, L, H, d = 2, 70, 2, 32
    D = H * d
    t = DT[dtype]
    gen = torch.Generator().manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    res, z = r(B * L, D), r(B * L, D).to(t)
    w0, w1, sc = 1 + 0.1 * r(D), 1 + 0.1 * r(D), 0.5 + 0.1 * r(D)
    q, k = r(B, L, H, d).to(t), r(B, L, H, d).to(t)
    g = (-0.2 * torch.rand(B, L, H, generator=gen)).to(t)
    dout = r(B * L, D)
    c = {n: v.to(DEV) for n, v in dict(res=res, z=z, w0=w0, w1=w1, sc=sc, q=q, k=k, g=g,
                                       dout=dout).items()}
    x0 = c["res"].to(t)
    _, h = ss.selscan_block_norm_fwd(x0, residual=None, next_weight=c["w0"])
    y = ss.selscan_linattn_fwd(c["q"], c["k"], h.view(B, L, H, d), c["g"])
    out, _ = ss.selscan_block_norm_fwd(y.view(B * L, D), c["z"], c["w1"], c["res"], c["sc"])
    gb = ss.selscan_block_norm_bwd(y.view(B * L, D), c["z"], c["w1"], c["res"], c["sc"],
                                   dout=c["dout"])
    ga = ss.selscan_linattn_bwd(c["q"], c["k"], h.view(B, L, H, d), c["g"],
                                dy=gb["dx"].view(B, L, H, d))
    g0 = ss.selscan_block_norm_bwd(x0, next_weight=c["w0"], dout=None,
                                   dy=ga["dv"].view(B * L, D))
    n = gh.to_np
    _, ho, _ = lo.block_norm_fwd(n(x0), next_weight=n(w0))
    yo, _ = lo.linattn_fwd(n(q), n(k), ho.reshape(B, L, H, d), n(g), d ** -0.5)
    oo, _, _ = lo.block_norm_fwd(yo.reshape(B * L, D), n(z), n(w1), n(res), n(sc))
    gbo = lo.block_norm_bwd(yo.reshape(B * L, D), n(z), n(w1), n(res), n(sc), dout=n(dout))
    gao = lo.linattn_bwd(n(q), n(k), ho.reshape(B, L, H, d), n(g), d ** -0.5,
                         dy=gbo["dx"].reshape(B, L, H, d))
    g0o = lo.block_norm_bwd(n(x0), next_weight=n(w0), dy=gao["dv"].reshape(B * L, D))
    # three roundings to bfloat16 in a row, each inside the single operators' bound
    tol = 3 * gh.RTOL[dtype]
    gh.compare(n(out), oo, tol, "block out")
    for name, a, b in (("dz", gb["dz"], gbo["dz"]), ("dq", ga["dq"], gao["dq"]),
                       ("dk", ga["dk"], gao["dk"]), ("dlog_decay", ga["dlog_decay"],
                                                    gao["dlog_decay"]),
                       ("dx", g0["dx"], g0o["dx"]), ("dw0", g0["dnext_weight"],
                                                     g0o["dnext_weight"])):
        gh.compare(n(a), b, tol, "block " + name)
