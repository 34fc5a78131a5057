"""Calls of the block-norm junction as programs make them side by side: several
host threads, operands off 16 bytes, one gradient alone. Tolerances as in
test_gpu_block_norm.py."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import selective_state_space_42_b200 as ss
from oracle import linattn as lo
from selective_state_space_42_b200.selscan import BlockNormOptions

import gpu_helpers as gh
from test_gpu_block_norm import make, near, sizes

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_host_threads_with_unlike_rows():
    """Host threads at a time, some with a gate and some without: the same kernel
    with rings of unlike size. No launch may fail, and all get what they get alone.
    Calls of the C entry point with arguments made ahead: the threads spend their
    time inside it, where the interpreter lets them run side by side."""
    R, D = 1300, 2560
    lib = ss.load_library()
    want, calls, held = [], [], []
    for n in range(4):
        i, _ = make(R, D, "bf16", 40 + n % 2, z=n % 2 == 0)
        d = {k: None if v is None else v.to(DEV) for k, v in i.items()}
        want.append([t.clone() for t in ss.selscan_block_norm_fwd(**d)])
        out, y = (torch.empty_like(t) for t in want[n])
        p = {k: None if v is None else v.data_ptr() for k, v in d.items()}
        o = BlockNormOptions(p["z"], 0, 0, p["weight"], p["residual"], p["res_scale"],
                             p["next_weight"], 1, 2 if p["z"] else 0, 1, 1e-5)
        stream = torch.cuda.Stream()
        calls.append((p["x"], ctypes.byref(o), out.data_ptr(), y.data_ptr(), R, D, 1,
                      stream.cuda_stream))
        held.append((d, out, y, o, stream))
    torch.cuda.synchronize()
    codes, start = [set() for _ in calls], threading.Barrier(len(calls))

    def work(n):
        start.wait()
        for _ in range(3000):
            codes[n].add(lib.selscan_block_norm_fwd(*calls[n]))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(calls)
    for w, h in zip(want, held):
        assert torch.equal(w[0], h[1]) and torch.equal(w[1], h[2])


def _off(t):
    """The same values one element behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = buf[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def _check_gradient(got, i, g, what, **kw):
    """Against float64, tolerances of test_gpu_block_norm.check."""
    n = {k: gh.to_np(v) for k, v in i.items()}
    want = lo.block_norm_bwd(**n, **{k: gh.to_np(v) for k, v in g.items()}, **kw)
    size = sizes(n, g, kw.get("groups", 1), kw.get("gate", "after"), kw.get("eps", 1e-5))
    rows = i["x"].shape[0]
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k in want:
        if k not in ("dweight", "dres_scale", "dnext_weight"):
            near(got[k], want[k], f"{what} {k}", size[k])
            continue
        o = want[k]
        rms = math.sqrt(float((o * o).mean()))
        assert (np.abs(gh.to_np(got[k]) - o) <= 1e-5 * max(1.0, math.sqrt(rows / 64))
                * (np.abs(o) + rms) + 1e-37).all(), (what, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["x", "z", "residual", "weight", "res_scale", "next_weight",
                                  "dout", "dy", "out", "y"])
def test_operands_off_16_bytes(dtype, name):
    """Each operand and output in turn, over rows enough for the ring."""
    i, g = make(1301, 256, dtype, 41)
    d = {k: v.to(DEV) for k, v in i.items()}
    dg = {k: v.to(DEV) for k, v in g.items()}
    outs = {}
    if name in d:
        d[name] = _off(d[name])
    elif name in dg:
        dg[name] = _off(dg[name])
    else:
        outs[name] = _off(torch.zeros_like(d["residual" if name == "out" else "x"]))
    out, y = ss.selscan_block_norm_fwd(**d, **outs)
    wo, wy, _ = lo.block_norm_fwd(**{k: gh.to_np(v) for k, v in i.items()})
    near(out, wo, name + " out")
    near(y, wy, name + " y")
    _check_gradient(ss.selscan_block_norm_bwd(**d, **dg), i, g, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(6, 200), (1300, 2048)], ids=str)
@pytest.mark.parametrize("name", ["dout", "dy"])
def test_one_gradient_alone(dtype, shape, name):
    """dout or dy alone, over few rows and over rows enough for the ring."""
    i, g = make(*shape, dtype, 42, nxt=name == "dy")
    d = {k: None if v is None else v.to(DEV) for k, v in i.items()}
    g = {"dout": None, "dy": None, name: g[name]}
    dg = {name: g[name].to(DEV)}
    _check_gradient(ss.selscan_block_norm_bwd(**d, **dg), i, g, f"{shape} {name}")
