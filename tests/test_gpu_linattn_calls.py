"""Calls of linear attention that its documentation allows and whose answers are
easy to lose. Tolerances as in test_gpu_linattn.py unless stated."""
import math

import pytest
import torch

import selective_state_space_42_b200 as ss

import test_gpu_linattn as t_la
from test_gpu_linattn import DEV, DT, check_bwd, check_fwd, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 0, 3, 8), (0, 4, 3, 8)], ids=str)
def test_empty_decays_have_an_empty_gradient(dtype, shape):
    z = torch.zeros(shape, device=DEV, dtype=DT[dtype])
    g = ss.selscan_linattn_bwd(z, z, z, z[..., 0].contiguous(), dy=z)
    assert g["dlog_decay"] is not None and g["dlog_decay"].shape == shape[:3]
    assert ss.selscan_linattn_bwd(z, z, z, torch.zeros(3, device=DEV), dy=z)["dlog_decay"] is None


def test_heads_without_columns_are_refused():
    """dk or dv of zero: the library's own error, from every entry point."""
    for dk, dv in ((0, 8), (8, 0)):
        q, v = torch.zeros(1, 4, 2, dk, device=DEV), torch.zeros(1, 4, 2, dv, device=DEV)
        with pytest.raises(ss.SelscanError):
            ss.selscan_linattn_fwd(q, q, v)
        with pytest.raises(ss.SelscanError):
            ss.selscan_linattn_bwd(q, q, v, dy=v)
        with pytest.raises(ss.SelscanError):
            ss.selscan_linattn_step(torch.zeros(1, 2, dk, dv, device=DEV), q[:, 0], q[:, 0], v[:, 0])


@pytest.mark.parametrize("op", ["y", "dq"])
def test_weights_behind_many_resets(op):
    """Tokens 45 .. 63 of a chunk whose first 45 all reset, against the same tokens
    behind 44 that do nothing and one that resets. The pairs' weights are the same
    up to 2^-20 (two exponentials of 2^-22 and a difference); at a step of 2^-8 of
    the operand they are rounded to, that turns a rounding in 2^-11 of the pairs, at
    most 19 pairs a row: 1% of the rows, of which twice as many are allowed."""
    i = make(4, 64, 8, 8, 64, 64, "bf16", 61, strength=0.05)
    d = dev(i)
    many, one = d["g"].clone(), d["g"].clone()
    many[:, :45] = -math.inf
    one[:, :44] = 0
    one[:, 44] = -math.inf

    def run(g):
        if op == "y":
            return ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], g)[:, 45:]
        return ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], g, dy=d["dy"])["dq"][:, 45:]

    a, b = run(many), run(one)
    assert (a != b).any(-1).float().mean().item() <= 0.02


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_products_under_decay(dtype):
    """Scores of 2^62 times values of 2^26, and decays of 2^-51 over a chunk: every
    result is within float32's range, so no factor on the way may leave it."""
    i = make(1, 130, 2, 2, 64, 64, dtype, 60)
    for k, e in (("q", 28), ("k", 28), ("v", 26)):
        i[k] = (i[k].float() * 2.0 ** e).to(i[k].dtype)
    i["g"][:] = -0.5546875
    check_fwd(i, dtype, what="large")


def _off(t):
    """The same values one element behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = buf[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "dy", "h0", "dS"])
@pytest.mark.parametrize("heads", [2, 4])
def test_gradient_of_rows_off_16_bytes(dtype, name, heads, monkeypatch):
    """Each operand in turn; heads of their own and shared ones."""
    i = make(2, 150, 2, heads, 64, 64, dtype, 62, h0=True)
    real = t_la.dev

    def dev_off(i):
        d = real(i)
        d[name] = _off(d[name])
        return d

    monkeypatch.setattr(t_la, "dev", dev_off)
    check_bwd(i, dtype, what=f"{name} off")
    check_fwd(i, dtype, what=f"{name} off")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_a_layer_with_shared_heads_and_a_state(dtype):
    """Shared heads and a first state together, over segments."""
    i = make(1, 1500, 2, 4, 128, 128, dtype, 63, h0=True, strength=0.1)
    check_bwd(i, dtype, what="layer")
