"""Calls of the block-norm junction as programs make them side by side: several
host threads, operands off 16 bytes, one gradient alone. Tolerances as in
test_gpu_block_norm.py."""
import ctypes
import threading

import pytest
import torch

import selective_state_space_42_b200 as ss
from selective_state_space_42_b200.selscan import BlockNormOptions

from test_gpu_block_norm import make

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
