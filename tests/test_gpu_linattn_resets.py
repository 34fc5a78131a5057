"""Documents packed into one row and set apart by resets (a log decay of −∞, or one
whose factor leaves float32): each gets what it gets alone.

Tolerances as in test_gpu_linattn.py, each document's at its own scale.
"""
import math

import numpy as np
import pytest
import torch

import selective_state_space_42_b200 as ss
from oracle import linattn as lo

import gpu_helpers as gh
from test_gpu_linattn import DEV, dev, make

pytestmark = pytest.mark.gpu


def check_documents(i, cuts, dtype, names=("dq", "dk", "dv", "dlog_decay"), upto=None):
    """The gradients of tokens cuts[n] .. cuts[n + 1] against float64 of these alone."""
    d = dev(i)
    got = ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                 dy=d["dy"], dfinal_state=d["dS"])
    torch.cuda.synchronize()
    n, L = gh.to_np, i["q"].shape[1]
    cuts = [0, *cuts, L]
    for a, b in zip(cuts[:-1], cuts[1:]):
        if upto is not None and b > upto:
            break
        x = {k: n(i[k][:, a:b]) for k in ("q", "k", "v", "g", "dy")}
        want = lo.linattn_bwd(x["q"], x["k"], x["v"], x["g"], i["q"].shape[3] ** -0.5,
                              n(i["h0"]) if a == 0 else None, None, x["dy"],
                              n(i["dS"]) if b == L else None)
        for k in names:
            g, o = n(got[k][:, a:b]), want[k]
            if k != "dlog_decay":
                gh.compare(g, o, gh.RTOL[dtype], f"{k} of {a}..{b}")
                continue
            assert np.isfinite(g).all(), (a, b)
            per = sum(np.sqrt((x[c] ** 2).sum(3) * (want["d" + c] ** 2).sum(3)) for c in "qk")
            e = {"f32": 2.0 ** -20, "bf16": 2.0 ** -17}[dtype]
            bound = gh.RTOL[dtype] * (np.abs(o) + np.sqrt((o * o).mean())) \
                + 4 * e * math.sqrt(b - a) * np.sqrt((per * per).mean())
            assert (np.abs(g - o) <= bound).all(), (a, b, float((np.abs(g - o) / bound).max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [-math.inf, -100.0])
def test_decay_gradient_of_documents_of_unlike_size(dtype, value):
    """A document whose gradients are 10^4 times larger stands behind two others:
    the running sum's errors from there stay there."""
    i = make(1, 300, 2, 2, 64, 64, dtype, 50, h0=True)
    i["g"][:, [100, 200]] = value
    i["dy"][:, 200:] *= 1e4
    i["dS"] *= 1e4
    check_documents(i, [100, 200], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_gradient_before_a_document_of_nan(dtype):
    i = make(1, 300, 2, 2, 64, 64, dtype, 51, h0=True)
    i["g"][:, [100, 190]] = -math.inf
    for k in ("q", "k", "v", "dy"):
        i[k][:, 256:] = math.nan
    i["dS"][:] = math.nan
    check_documents(i, [100, 190], dtype, upto=190)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_gradient_over_many_tiles(dtype):
    """Resets at the edges of the running sum's tiles, threads and warps, and tiles
    with none."""
    L = 13001
    cuts = sorted({1, L - 4096, L - 4095, L - 4097, L - 8192, L - 3, L - 1, L - 128 * 4,
                   L - 128 * 4 - 4, L - 128 * 4 + 1})
    i = make(1, L, 1, 1, 8, 8, dtype, 52, h0=True, strength=0.05)
    i["g"][:, cuts] = -math.inf
    for n, a in enumerate(cuts):  # neighbours of unlike size
        i["dy"][:, a:] = i["dy"][:, a:] * (100.0 if n % 2 else 0.01)
    check_documents(i, cuts, dtype, names=("dlog_decay",))
