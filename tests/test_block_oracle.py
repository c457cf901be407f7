"""Pins of the oracle of the gate with groups, the fused norms and the checkpoint
against brute force, closed forms and central differences.  CPU only."""
import itertools

import numpy as np
import pytest

import oracle as O

RNG = np.random.default_rng(7)


def rand(*shape, scale=1.0):
    return RNG.standard_normal(shape) * scale


def numeric(f, x, d, step=1e-6):
    """d/dx of sum(d * f(x)) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = ((f(hi) - f(lo)) * d).sum() / (2 * step)
    return g


def test_gate_without_groups_and_bias_is_the_plain_softmax_gate():
    l = rand(50, 12)
    idx, gate = O.gate_group(l, 3, 4, 4)
    assert np.array_equal(idx, O.topk_experts(l, 3))
    assert np.allclose(gate, np.take_along_axis(O.softmax_experts(l), idx.astype(np.int64), axis=1), rtol=1e-14)


@pytest.mark.parametrize("group_max", [False, True])
def test_gate_groups_against_every_choice_of_groups(group_max):
    """The kept groups are the subset with the largest sum of ranks, and the
    experts the best subset inside it, by enumeration."""
    l, b = rand(30, 12), rand(12, scale=0.3)
    idx, _ = O.gate_group(l, 3, 4, 2, sigmoid=True, bias=b, group_max=group_max)
    c = 1 / (1 + np.exp(-l)) + b
    for t in range(30):
        rank = [sorted(c[t, 3 * g:3 * g + 3])[-1:] if group_max else sorted(c[t, 3 * g:3 * g + 3])[-2:] for g in range(4)]
        kept = max(itertools.combinations(range(4), 2), key=lambda p: sum(sum(rank[g]) for g in p))
        allowed = [e for g in kept for e in range(3 * g, 3 * g + 3)]
        best = max(itertools.combinations(allowed, 3), key=lambda p: sum(c[t, e] for e in p))
        assert set(idx[t]) == set(best)
        assert (np.diff(c[t, idx[t]]) <= 0).all()


def test_gate_masked_experts():
    l = np.full((3, 8), -np.inf)
    l[1, 5] = 0.3
    l[2] = np.nan
    idx, gate = O.gate_group(l, 3, 4, 2, sigmoid=True, renorm=True, scale=2.0)
    assert idx.tolist() == [[0, 1, 2], [5, 0, 1], [0, 1, 2]]
    assert gate[0].tolist() == [0, 0, 0] and gate[1].tolist() == [2, 0, 0] and np.isnan(gate[2]).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_backward_against_differences(sigmoid, renorm):
    l, d = rand(4, 8), rand(4, 3)
    kw = dict(sigmoid=sigmoid, renorm=renorm, scale=1.7)
    idx, _ = O.gate_group(l, 3, 2, 1, **kw)

    def gates(x):
        s = 1 / (1 + np.exp(-x)) if sigmoid else O.softmax_experts(x)
        g = np.take_along_axis(s, idx.astype(np.int64), axis=1)
        return 1.7 * (g / g.sum(axis=1, keepdims=True) if renorm else g)
    assert np.allclose(gates(l), O.gate_group(l, 3, 2, 1, **kw)[1], rtol=1e-13)
    assert np.allclose(O.gate_group_bwd(d, l, idx, **kw), numeric(gates, l, d), atol=1e-8)


@pytest.mark.parametrize("post,scale,nxt", [(True, True, True), (False, True, True), (True, False, False), (False, False, True)])
def test_combine_norm_backward_against_differences(post, scale, nxt):
    T, K, H, eps = 3, 2, 5, 1e-3
    h, gate, dst = rand(T * K, H), rand(T, K), RNG.permutation(T * K)
    res, dy, dxn = rand(T, H), rand(T, H), rand(T, H) if nxt else None
    opt = dict(row_scale=rand(T) if scale else None, w_post=rand(H) if post else None,
               res_scale=rand(H) if scale else None, w_next=rand(H) if nxt else None)

    def loss_of(**kw):
        a = dict(h=h, gate=gate, residual=res, **opt)
        a.update(kw)
        y, xn = O.combine_norm(a["h"], a["gate"], dst, K, eps, a["row_scale"], a["residual"], a["w_post"],
                               a["res_scale"], a["w_next"])
        return np.array([(y * dy).sum() + ((xn * dxn).sum() if nxt else 0)])
    y, _ = O.combine_norm(h, gate, dst, K, eps, residual=res, **opt)
    got = O.combine_norm_bwd(dy, dxn, h, gate, dst, K, eps, y, **opt)
    names = {"d_res": ("residual", res), "dh": ("h", h), "d_gate": ("gate", gate)}
    if scale:
        names.update(d_scale=("row_scale", opt["row_scale"]), d_res_scale=("res_scale", opt["res_scale"]))
    if post:
        names["dw_post"] = ("w_post", opt["w_post"])
    if nxt:
        names["dw_next"] = ("w_next", opt["w_next"])
    for out, (name, x) in names.items():
        assert np.allclose(got[out], numeric(lambda v: loss_of(**{name: v}), x, np.ones(1)), atol=1e-7), out


def test_combine_norm_without_a_block_is_the_norm():
    x, w = rand(4, 6), rand(6)
    y, xn = O.combine_norm(None, None, None, 0, 0.0, residual=x, w_next=w)
    assert np.array_equal(y, x) and np.allclose((xn / w) ** 2 @ np.ones(6) / 6, 1)


def test_ckpt_error_and_borders():
    x = rand(20, 70) * np.exp(3 * rand(20, 1))
    q, s = O.ckpt_pack(x)
    assert s.shape == (20, 3) and (np.abs(q.astype(int)) <= 127).all()
    a = np.abs(np.pad(x, ((0, 0), (0, 26))).reshape(20, 3, 32)).max(axis=2)
    step = 2.0 ** (s.astype(float) - 127)
    assert (a <= 127 * step).all() and (a > 63.5 * step).all()
    assert (np.abs(O.ckpt_unpack(q, s) - x) <= np.repeat(step, 32, axis=1)[:, :70] / 2).all()
    # 127 times a power of two is held exactly; a little more takes the next power; halves go to even
    q, s = O.ckpt_pack(np.array([[127.0, 0.5, 1.5, -2.5], [127.5, 1.0, 3.0, 0.0], [0, 0, 0, 0], [1, np.inf, 0, 2]]))
    assert q.tolist() == [[127, 0, 2, -2], [64, 0, 2, 0], [0] * 4, [0] * 4]
    assert s[:, 0].tolist() == [127, 128, 1, 255]
    assert np.isnan(O.ckpt_unpack(q, s)[3]).all()
