"""Host-side validation of the linear-attention and block-norm entry points
(CPU only; every check runs before any CUDA call)."""
import ctypes

import pytest
import torch

import selective_state_space_42_b200 as ss
from selective_state_space_42_b200 import build as ssbuild
from selective_state_space_42_b200.selscan import BlockNormOptions, LinattnOptions

P = 1 << 20  # fake, aligned device addresses (never dereferenced)
Q, K, V, Y, G, H0, HF, LENS, GH = (P + i * (1 << 16) for i in range(9))


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return ss.load_library()


def la(lib, opts=None, **kw):
    a = dict(q=Q, k=K, v=V, y=Y, final=None, batch=0, seqlen=8, qk=2, heads=4, dk=16, dv=8,
             dtype=1, ws=None, wsb=0)
    a.update(kw)
    o = None if opts is None else ctypes.byref(LinattnOptions(**opts))
    return lib.selscan_linattn_fwd(a["q"], a["k"], a["v"], 1.0, o, a["y"], a["final"], a["batch"],
                                   a["seqlen"], a["qk"], a["heads"], a["dk"], a["dv"], a["dtype"],
                                   a["ws"], a["wsb"], None)


def test_linattn_fwd_validation(lib):
    assert la(lib) == 0  # batch = 0: nothing to do
    assert la(lib, dtype=2) == -3
    for bad in (dict(batch=-1), dict(seqlen=-1), dict(heads=-4), dict(qk=0), dict(qk=3),
                dict(dk=0), dict(dk=129), dict(dv=0), dict(dv=129), dict(heads=70000, qk=1),
                dict(batch=1 << 22, heads=4), dict(batch=1, seqlen=1 << 40)):
        assert la(lib, **bad) == -2, bad
    assert la(lib, dict(log_decay=G, head_log_decay=GH)) == -2  # one decay at most
    assert la(lib, dict(q_stride=31)) == -2  # shorter than a token's heads
    full = dict(batch=1)
    for n in ("q", "k", "v", "y"):
        assert la(lib, **{n: None}, **full) == -1, n
    assert la(lib, q=Q + 1, **full) == -4
    assert la(lib, final=HF + 2, **full) == -4
    assert la(lib, dict(seqlens=LENS + 2), **full) == -4
    assert la(lib, ws=P + 4, wsb=1 << 20, **full) == -4
    assert la(lib, y=Q, **full) == -7
    assert la(lib, dict(log_decay=Y), **full) == -7
    assert la(lib, dict(seqlens=Y + 4), **full) == -7
    assert la(lib, dict(initial_state=HF + 64), final=HF, **full) == -7  # overlaps, not equal
    # a strided q's reach counts: 8 tokens 4096 elements apart run into y
    assert la(lib, dict(q_stride=4096), q=Y - 2048, **full) == -7


def test_linattn_bwd_validation(lib):
    def call(opts=None, **kw):
        a = dict(dy=Y, dS=None, dq=P + (1 << 20), dk=P + (1 << 21), dv=P + (3 << 20), dg=None,
                 dh0=None, batch=0)
        a.update(kw)
        o = None if opts is None else ctypes.byref(LinattnOptions(**opts))
        return lib.selscan_linattn_bwd(Q, K, V, 1.0, o, a["dy"], a["dS"], a["dq"], a["dk"],
                                       a["dv"], a["dg"], a["dh0"], a["batch"], 8, 2, 4, 16, 8, 1,
                                       a.get("ws"), a.get("wsb", 0), None)
    assert call() == 0
    for n in ("dy", "dq", "dk", "dv"):
        assert call(batch=1, **{n: None}) == -1, n
    assert call(batch=1, dg=HF) == -1  # a decay's gradient needs decays per token
    assert call(dict(head_log_decay=GH), batch=1, dg=HF) == -1
    assert call(batch=1, dq=Q) == -7
    assert call(batch=1, dv=Y) == -7
    assert call(batch=1, dS=HF, dh0=HF) == -7
    assert call(batch=1, dh0=HF + 2) == -4
    assert call(batch=1, ws=P + (1 << 24), wsb=16) == -8


def test_linattn_step_validation(lib):
    def call(**kw):
        a = dict(state=HF, q=Q, k=K, v=V, g=None, gh=None, y=Y, batch=0, qk=2, heads=4, dk=16,
                 dv=8, dtype=1)
        a.update(kw)
        return lib.selscan_linattn_step(a["state"], a["q"], a["k"], a["v"], a["g"], a["gh"], 1.0,
                                        a["y"], a["batch"], a["qk"], a["heads"], a["dk"], a["dv"],
                                        a["dtype"], None)
    assert call() == 0
    assert call(dtype=5) == -3
    assert call(qk=3) == -2
    assert call(dk=129) == -2
    assert call(g=G, gh=GH) == -2
    for n in ("state", "q", "k", "v", "y"):
        assert call(batch=1, **{n: None}) == -1, n
    assert call(batch=1, state=HF + 2) == -4
    assert call(batch=1, y=HF) == -7
    assert call(batch=1, q=HF) == -7


def test_linattn_workspace_bytes(lib):
    f, b = lib.selscan_linattn_workspace_bytes, lib.selscan_linattn_bwd_workspace_bytes
    assert f(0, 8, 2, 4, 16, 8, 1) == 0
    assert f(1, 8, 3, 4, 16, 8, 1) == 0  # invalid sizes
    assert f(1, 8, 2, 4, 16, 8, 1) == 0  # one segment: none needed
    assert f(1, 1 << 16, 4, 4, 128, 128, 1) > 0  # segments
    n = 4 * 8 * 4
    assert b(1, 8, 4, 4, 16, 8, 0) >= 2 * n
    assert b(1, 8, 2, 4, 16, 8, 0) >= b(1, 8, 4, 4, 16, 8, 0)  # shared heads: their partial sums


def bn(lib, opts=None, out=Y, y=None, rows=0, dim=16, dtype=1, x=Q):
    o = ctypes.byref(BlockNormOptions(**{"eps": 1e-5, **(opts or {})}))
    return lib.selscan_block_norm_fwd(x, o, out, y, rows, dim, dtype, None)


def test_block_norm_validation(lib):
    W = dict(weight=G)
    assert bn(lib) == 0
    assert bn(lib, dtype=9) == -3
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=16385)):
        assert bn(lib, **bad) == -2, bad
    assert bn(lib, dict(groups=3, **W)) == -2
    assert bn(lib, dict(groups=2)) == -2  # groups belong to a norm
    assert bn(lib, dict(groups=-1, **W)) == -2
    assert bn(lib, dict(groups=2048, **W), dim=2048) == -2
    assert bn(lib, dict(gate=3)) == -2
    assert bn(lib, dict(eps=-1.0)) == -2
    assert bn(lib, dict(eps=float("nan"))) == -2
    assert bn(lib, dict(x_stride=15)) == -2
    assert bn(lib, rows=2, x=None) == -1
    assert bn(lib, dict(gate=1), rows=2) == -1  # a gate without z
    assert bn(lib, rows=2, out=None) == -1
    assert bn(lib, dict(next_weight=G), rows=2) == -1  # the next norm without y
    assert bn(lib, rows=2, y=K) == -1  # y without the next norm
    assert bn(lib, rows=2, x=Q + 1) == -4
    assert bn(lib, dict(residual=K + 2, residual_f32=1), rows=2) == -4
    assert bn(lib, rows=2, out=Q) == -7
    assert bn(lib, dict(residual=Y + 2), rows=2) == -7  # overlaps, not equal
    assert bn(lib, dict(residual=K, next_weight=G), rows=2, y=K) == -7


def test_block_norm_bwd_validation(lib):
    def call(opts=None, dout=K, dy=None, dx=Y, dz=None, dres=None, dw=None, ws=None, wsb=0,
             rows=2):
        o = ctypes.byref(BlockNormOptions(**{"eps": 1e-5, **(opts or {})}))
        return lib.selscan_block_norm_bwd(Q, o, dout, dy, dx, dz, dres, dw, None, None, rows, 16,
                                          1, ws, wsb, None)
    assert call(rows=0) == 0
    assert call(dx=None) == -1
    assert call(dout=None) == -1  # no gradient comes in
    assert call(dy=V) == -1  # dy without the next norm
    assert call(dict(next_weight=G)) == -1
    assert call(dict(gate=1, z=V)) == -1  # dz is required with a gate
    assert call(dx=K) == -7
    assert call(dict(weight=G), dw=G) == -7
    assert call(ws=P + (1 << 24), wsb=16) == -8
    assert lib.selscan_block_norm_bwd_workspace_bytes(0, 16) == 0
    assert lib.selscan_block_norm_bwd_workspace_bytes(5, 16385) == 0
    assert lib.selscan_block_norm_bwd_workspace_bytes(5, 64) == 5 * 2 * 64 * 4  # a block a row


def test_bindings_refuse_cpu_tensors_and_wrong_shapes(lib):
    t = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        ss.selscan_linattn_fwd(t(1, 4, 2, 8), t(1, 4, 2, 8), t(1, 4, 2, 8))
    with pytest.raises(ValueError, match="batch"):
        ss.selscan_linattn_fwd(t(4, 2, 8), t(4, 2, 8), t(4, 2, 8))
    with pytest.raises(TypeError):
        ss.selscan_linattn_fwd(*(t(1, 4, 2, 8).half() for _ in range(3)))
    with pytest.raises(ValueError, match="state"):
        ss.selscan_linattn_step(t(1, 2, 8), t(1, 2, 8), t(1, 2, 8), t(1, 2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ss.selscan_block_norm_fwd(t(3, 8), weight=t(8))
    with pytest.raises(ValueError, match="gate"):
        ss.selscan_block_norm_fwd(t(3, 8), gate="both")
    with pytest.raises(TypeError):
        ss.selscan_block_norm_fwd(t(3, 8), residual=t(3, 8).half())
