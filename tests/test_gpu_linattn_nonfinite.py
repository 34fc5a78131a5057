"""Values that are not finite, in linear attention: they reach what the recurrence
lets them reach and nothing else. What they do not reach keeps its bits.

A value at token t of a row reaches y of the tokens from t on, up to the next
reset, and the state leaving; one of v only its own column. The gradients of q
(sums over earlier tokens) and of k and v (over later ones) likewise. What is
reached is not finite; whether infinite or NaN is not said, except that a state
takes an infinite v as it stands.
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
BAD = [math.inf, -math.inf, math.nan]


def fwd(d, **kw):
    return ss.selscan_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                  return_final_state=True, **kw)


def bwd(d, **kw):
    return ss.selscan_linattn_bwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["h0"],
                                  dy=d["dy"], dfinal_state=d["dS"], **kw)


def changed(d, name, at, value):
    e = dict(d)
    e[name] = d[name].clone()
    e[name][at] = value
    return e


# L, dk, dv, strength of the decays (3.0: chunks whose factors leave their range)
SIZES = [(150, 64, 64, 0.1), (150, 64, 64, 3.0), (300, 128, 128, 0.1), (300, 128, 128, 3.0),
         (130, 48, 80, 0.1), (130, 33, 50, 0.1), (2100, 64, 64, 0.05), (2100, 128, 128, 0.05)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", BAD, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_value_reaches_later_tokens_of_its_column(dtype, value, size):
    L, dk, dv, strength = size
    d = dev(make(1, L, 2, 2, dk, dv, dtype, 70, h0=True, strength=strength))
    y0, S0 = fwd(d)
    for t, c in ((0, 0), (37, dv - 1), (64, 17), (L - 1, 5)):
        y, S = fwd(changed(d, "v", (0, t, 1, c), value))
        others = [n for n in range(dv) if n != c]
        assert torch.equal(y[:, :, 0], y0[:, :, 0]) and torch.equal(S[:, 0], S0[:, 0])
        assert torch.equal(y[0, :, 1, others], y0[0, :, 1, others])
        assert torch.equal(S[0, 1][:, others], S0[0, 1][:, others])
        assert torch.equal(y[0, :t, 1, c], y0[0, :t, 1, c])
        far = L if strength < 1 else min(L, t + 16)  # steep decays end in zero
        assert not torch.isfinite(y[0, t:far, 1, c]).any()
        if strength < 1 or t == L - 1:
            s = S[0, 1, :, c]
            if math.isnan(value):
                assert torch.isnan(s).all()
            else:
                k = d["k"][0, t, 1].float()
                assert torch.equal(s, torch.where(k * value > 0, math.inf, -math.inf))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_value_reaches_later_tokens_in_several_columns(dtype):
    """Several in one chunk and in chunks next to each other."""
    d = dev(make(1, 330, 1, 1, 128, 128, dtype, 71, strength=0.1))
    y0, _ = fwd(d)
    e = dict(d)
    e["v"] = d["v"].clone()
    first = torch.full((128,), 330, device=DEV)
    for t, c in ((3, 0), (9, 0), (63, 40), (64, 41), (65, 0), (100, 127), (128, 90), (128, 91),
                 (200, 64), (329, 10)):
        e["v"][0, t, 0, c] = math.inf
        first[c] = min(first[c].item(), t)
    y, _ = fwd(e)
    reached = torch.arange(330, device=DEV)[:, None] >= first
    y, y0 = y[0, :, 0], y0[0, :, 0]
    assert not torch.isfinite(y[reached]).any()
    assert torch.equal(y[~reached], y0[~reached])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("value", [math.inf, math.nan], ids=str)
@pytest.mark.parametrize("L,dim,cut", [(200, 64, 100), (200, 128, 70), (2100, 64, 1000),
                                       (2100, 128, 1937)])
def test_a_reset_keeps_documents_apart(dtype, name, value, L, dim, cut):
    """A value near the reset in one document and the other's results, both ways
    round, in the forward pass and in every gradient."""
    d = dev(make(1, L, 2, 2, dim, dim, dtype, 72, h0=True, strength=0.1))
    d["g"][:, cut] = -math.inf
    y0, S0 = fwd(d)
    g0 = bwd(d)
    for t in (cut - 3, cut - 1, cut, cut + 2):
        other = slice(cut, L) if t < cut else slice(0, cut)
        e = changed(d, name, (0, t), value)  # all heads, all columns
        y, S = fwd(e)
        assert torch.equal(y[:, other], y0[:, other])
        if t < cut:
            assert torch.equal(S, S0)
        g = bwd(e)
        for n in ("dq", "dk", "dv", "dlog_decay"):
            assert torch.equal(g[n][:, other], g0[n][:, other]), (n, t)
        if t >= cut:
            assert torch.equal(g["dh0"], g0["dh0"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,dim,strength", [(200, 64, 0.1), (200, 128, 0.1), (200, 128, 3.0),
                                            (2100, 64, 0.05)])
@pytest.mark.parametrize("heads", [2, 4])
def test_gradients_on_the_other_side_of_a_value(dtype, L, dim, strength, heads):
    """dq of a token does not depend on later tokens, dk and dv not on earlier ones."""
    d = dev(make(1, L, 2, heads, dim, dim, dtype, 73, h0=True, strength=strength))
    g0 = bwd(d)
    for t in (1, 70, 127, L - 2):
        for name in ("k", "v"):
            g = bwd(changed(d, name, (0, t), math.inf))
            assert torch.equal(g["dq"][:, :t], g0["dq"][:, :t]), (name, t)
            assert not torch.isfinite(g["dq"][:, t]).any()
        for name in ("q", "dy"):
            g = bwd(changed(d, name, (0, t), math.inf))
            for n in ("dk", "dv"):
                assert torch.equal(g[n][:, t + 1:], g0[n][:, t + 1:]), (name, n, t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,dim", [(150, 64), (150, 128), (2100, 64)])
def test_rows_behind_a_length_stay_zero(dtype, L, dim):
    """y and gradients of tokens behind a row's length are zero whatever the states
    hold."""
    d = dev(make(2, L, 1, 2, dim, dim, dtype, 74, h0=True, strength=0.05))
    d["h0"][:, 0] = math.inf
    d["dS"][:, 1] = math.nan
    lens = [77, L - 70]
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    y, _ = fwd(d, seqlens=sl)
    g = bwd(d, seqlens=sl)
    for b, n in enumerate(lens):
        assert not torch.isfinite(y[b, :n, 0]).any() and torch.isfinite(y[b, :n, 1]).all()
        for t in (y, g["dq"], g["dk"], g["dv"], g["dlog_decay"]):
            assert (t[b, n:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(8))
def test_scattered_values_against_the_recurrence(dtype, seed):
    """Values of every kind in q, k and v at random tokens, resets at random tokens,
    rows of unlike length: finite where the float64 recurrence is, and near it
    (tolerances of test_gpu_linattn.py), not finite where it is not."""
    r = np.random.default_rng(seed)
    B, L, Hq, H = 2, int(r.integers(130, 700)), 2, 4
    dk, dv = int(r.choice([40, 64, 128])), int(r.choice([48, 64, 128]))
    i = make(B, L, Hq, H, dk, dv, dtype, 80 + seed, h0=True, strength=0.05)
    for _ in range(12):
        n = ["q", "k", "v"][r.integers(3)]
        x = i[n]
        x[tuple(int(r.integers(s)) for s in x.shape)] = float(r.choice(BAD))
    for _ in range(14):
        i["g"][int(r.integers(B)), int(r.integers(L)), int(r.integers(H))] = -math.inf
    lens = [L, int(r.integers(1, L))]
    d = dev(i)
    y, S = fwd(d, seqlens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    n = gh.to_np
    with np.errstate(invalid="ignore"):
        yo, So = lo.linattn_fwd(n(i["q"]), n(i["k"]), n(i["v"]), n(i["g"]), dk ** -0.5, n(i["h0"]),
                                lens)
    for got, want, tol in ((n(y), yo, gh.RTOL[dtype]), (n(S), So, 1e-4)):
        ok = np.isfinite(want)
        assert (np.isfinite(got) == ok).all()
        gh.compare(np.where(ok, got, 0.0), np.where(ok, want, 0.0), tol, "finite part")
