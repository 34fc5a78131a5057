"""The float64 oracle of linear attention and of the block-norm junction
against independent forms: the dense masked product, finite differences."""
import numpy as np
import pytest

from oracle import linattn as lo


def _inputs(B, L, Hq, H, dk, dv, seed):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, L, Hq, dk)), k=r.standard_normal((B, L, Hq, dk)),
                v=r.standard_normal((B, L, H, dv)), g=-0.3 * r.random((B, L, H)),
                h0=r.standard_normal((B, H, dk, dv)))


def test_forward_is_the_masked_product():
    """y = (D ◦ QKᵀ)V + exp(G)·Q S_0 with D_ij = exp(G_i − G_j), j ≤ i."""
    i = _inputs(2, 9, 2, 4, 3, 5, 1)
    y, S = lo.linattn_fwd(i["q"], i["k"], i["v"], i["g"], 0.7, i["h0"])
    G = np.cumsum(i["g"], 1)
    for b in range(2):
        for h in range(4):
            D = np.tril(np.exp(G[b, :, None, h] - G[b, None, :, h]))
            q, k, v = i["q"][b, :, h // 2], i["k"][b, :, h // 2], i["v"][b, :, h]
            want = 0.7 * ((D * (q @ k.T)) @ v
                          + np.exp(G[b, :, h])[:, None] * (q @ i["h0"][b, h]))
            np.testing.assert_allclose(y[b, :, h], want, rtol=1e-12, atol=1e-12)
            end = np.exp(G[b, -1, h]) * i["h0"][b, h] + (
                k * np.exp(G[b, -1, h] - G[b, :, h])[:, None]).T @ v
            np.testing.assert_allclose(S[b, h], end, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("seqlens", [None, [4, 0]])
def test_linattn_gradient_by_differences(seqlens):
    i = _inputs(2, 6, 1, 2, 3, 2, 2)
    r = np.random.default_rng(3)
    dy, dS = r.standard_normal(i["v"].shape), r.standard_normal(i["h0"].shape)

    def loss(**kw):
        a = {**i, **kw}
        y, S = lo.linattn_fwd(a["q"], a["k"], a["v"], a["g"], 0.7, a["h0"], seqlens)
        return (y * dy).sum() + (S * dS).sum()

    g = lo.linattn_bwd(i["q"], i["k"], i["v"], i["g"], 0.7, i["h0"], seqlens, dy, dS)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("h0", "dh0")):
        for at in np.ndindex(*i[name].shape):
            e = np.zeros_like(i[name])
            e[at] = 1e-5
            d = (loss(**{name: i[name] + e}) - loss(**{name: i[name] - e})) / 2e-5
            # central difference: truncation ~1e-10 of third derivatives of order one
            assert abs(d - g[key][at]) < 1e-7, (name, at)


@pytest.mark.parametrize("gate", ["before", "after"])
@pytest.mark.parametrize("groups", [1, 2])
def test_block_norm_gradient_by_differences(gate, groups):
    r = np.random.default_rng(5)
    R, D = 3, 6
    i = dict(x=r.standard_normal((R, D)), z=r.standard_normal((R, D)),
             weight=1 + 0.1 * r.standard_normal(D), residual=r.standard_normal((R, D)),
             res_scale=0.5 + 0.1 * r.standard_normal(D),
             next_weight=1 + 0.1 * r.standard_normal(D))
    dout, dy = r.standard_normal((R, D)), r.standard_normal((R, D))

    def loss(**kw):
        out, y, _ = lo.block_norm_fwd(**{**i, **kw}, groups=groups, gate=gate)
        return (out * dout).sum() + (y * dy).sum()

    g = lo.block_norm_bwd(**i, groups=groups, gate=gate, dout=dout, dy=dy)
    for name in i:
        for at in np.ndindex(*i[name].shape):
            e = np.zeros_like(i[name])
            e[at] = 1e-5
            d = (loss(**{name: i[name] + e}) - loss(**{name: i[name] - e})) / 2e-5
            assert abs(d - g["d" + name][at]) < 1e-7, (name, at)
