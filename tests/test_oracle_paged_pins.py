"""Pins for the oracle's prologue backward and paged-cache functions, each against something other than the oracle
itself: torch.autograd in float64, central differences, hand-picked positions, and the contiguous functions on a cache
laid out as pages.  Planted mistakes in copies must fail them.

Cited page: "Transformers 中的 Doge 小语言模型完全指南" ([Guide]), section "动态掩码注意力（DMA）" forward-chain steps 1-4.
"""
import numpy as np
import pytest
import torch

import oracle


def check_backward(prologue_backward):
    rng = np.random.default_rng(3)
    B, L, Hq, Hkv, d, theta, eps = 2, 3, 2, 1, 8, 300.0, 1e-3
    q, k = rng.standard_normal((B, L, Hq, d)), rng.standard_normal((B, L, Hkv, d))
    qw, kw = rng.uniform(0.5, 1.5, d), rng.uniform(0.5, 1.5, d)
    pos = np.array([2, 11])
    gq, gk = rng.standard_normal(q.shape), rng.standard_normal(k.shape)
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, qw, kw)]
    # an independent forward: complex rotation of the normalised pairs
    ang = (torch.tensor(pos)[:, None] + torch.arange(L))[:, :, None, None] * theta ** (-torch.arange(0, d, 2).double() / d)

    def rotated(x, w):
        y = w * x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps)
        z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * torch.exp(1j * ang)
        return torch.cat([z.real, z.imag], -1)

    loss = (rotated(t[0], t[2]) * torch.tensor(gq)).sum() + (rotated(t[1], t[3]) * torch.tensor(gk)).sum()
    want = torch.autograd.grad(loss, t)
    got = prologue_backward(q, k, qw, kw, eps, theta, pos, gq, gk)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b.numpy(), rtol=1e-11, atol=1e-11)


def test_prologue_backward_equals_autograd():
    check_backward(oracle.prologue_backward)


@pytest.mark.parametrize("wrong", ["sign", "no_mean", "eps", "swapped"])
def test_planted_backward_mistakes_are_found(wrong):
    def broken(q, k, qw, kw, eps, theta, pos, gq, gk):
        if wrong == "sign":
            pos = -np.asarray(pos)
        if wrong == "eps":
            eps = 0.0
        r = oracle.prologue_backward(q, k, qw, kw, eps, theta, pos, gq, gk)
        if wrong == "swapped":
            r = (r[0], r[1], r[3], r[2])
        if wrong == "no_mean":
            rho = np.sqrt((q * q).mean(-1, keepdims=True) + eps)
            dy = np.stack([oracle.rope(gq[b], -(int(pos[b]) + np.arange(q.shape[1])), theta) for b in range(len(pos))])
            r = (qw * dy / rho,) + r[1:]
        return r
    with pytest.raises(AssertionError):
        check_backward(broken)


def test_prologue_backward_by_differences():
    rng = np.random.default_rng(4)
    q, k = rng.standard_normal((1, 2, 2, 6)), rng.standard_normal((1, 2, 1, 6))
    w = rng.uniform(0.5, 1.5, 6)
    gq, gk = rng.standard_normal(q.shape), rng.standard_normal(k.shape)
    z = np.zeros((1, 9, 1, 6))
    f = lambda a: (oracle.prologue(a, k, k, w, w, 1e-6, 50.0, [5], z, z)[0] * gq).sum()
    dq = oracle.prologue_backward(q, k, w, w, 1e-6, 50.0, [5], gq, gk)[0]
    step = rng.standard_normal(q.shape)
    assert (f(q + 1e-5 * step) - f(q - 1e-5 * step)) / 2e-5 == pytest.approx((dq * step).sum(), rel=1e-7)


def test_visible_positions():
    assert oracle.visible_positions(5, 0, 0) == [0, 1, 2, 3, 4]
    assert oracle.visible_positions(5, 2, 1) == [0, 3, 4]
    assert oracle.visible_positions(5, 2, 4) == [0, 1, 2, 3, 4]
    assert oracle.visible_positions(5, 9, 0) == [0, 1, 2, 3, 4]
    assert oracle.visible_positions(0, 2, 1) == []


def paged(rng, cache, lens, page):
    """A contiguous cache [B, Lk, ...] as scattered pages."""
    B, Lk = cache[0].shape[:2]
    n = -(-Lk // page)
    table = rng.permutation(B * n).reshape(B, n)
    pools = []
    for c in cache:
        pool = np.zeros((B * n, page) + c.shape[2:])
        for b in range(B):
            for j in range(lens[b]):
                pool[table[b, j // page], j % page] = c[b, j]
        pools.append(pool)
    return table, pools


@pytest.mark.parametrize("w,page", [(4, 3), (50, 4), (7, 1)])
def test_decode_paged_equals_contiguous_decode(w, page):
    rng = np.random.default_rng(5)
    B, Lk, Hq, Hkv, d = 3, 19, 4, 2, 8
    q = rng.standard_normal((B, Hq, d))
    k, v = rng.standard_normal((2, B, Lk, Hkv, d))
    dt = rng.uniform(0.1, 1.0, (B, Lk, Hkv)).astype(np.float32)
    lens = [19, 1, 8]
    table, (kp, vp, dp) = paged(rng, (k, v, dt), lens, page)
    got = oracle.decode_paged(q, kp, vp, dp.transpose(0, 2, 1), table, lens, w, 0, 0, 0.3)
    want = oracle.decode_step(q, k, v, None, None, lens, w, 0.3, dt=dt.transpose(0, 2, 1))
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-13)


def test_decode_paged_window_equals_masked_softmax():
    rng = np.random.default_rng(6)
    Lk, d = 23, 4
    q, k, v = rng.standard_normal((1, 2, d)), rng.standard_normal((Lk, d)), rng.standard_normal((Lk, d))
    dt = rng.uniform(0.1, 1.0, Lk).astype(np.float32)
    table, (kp, vp, dp) = paged(rng, (k[None, :, None], v[None, :, None], dt[None, :, None]), [Lk], 5)
    got = oracle.decode_paged(q, kp, vp, dp.transpose(0, 2, 1), table, [Lk], 100, 6, 2, 0.5)
    s = torch.tensor(0.5 * q[0] @ k.T + dt)
    s[:, 2:Lk - 6] = -torch.inf
    np.testing.assert_allclose(got[0], (torch.softmax(s, -1) @ torch.tensor(v)).numpy(), rtol=1e-12)
    # the best four of what is seen
    got = oracle.decode_paged(q, kp, vp, dp.transpose(0, 2, 1), table, [Lk], 4, 6, 2, 0.5)
    seen = [0, 1] + list(range(Lk - 6, Lk))
    drop = [j for j in range(Lk) if j not in sorted(seen, key=lambda j: -dt[j])[:4]]
    s = torch.tensor(0.5 * q[0] @ k.T + dt)
    s[:, drop] = -torch.inf
    np.testing.assert_allclose(got[0], (torch.softmax(s, -1) @ torch.tensor(v)).numpy(), rtol=1e-12)


def test_append_paged_equals_prologue_and_scores():
    rng = np.random.default_rng(7)
    Hq, Hkv, d, page = 2, 2, 8, 3
    news, positions = [3, 0, 5], [4, 1, 0]
    T = sum(news)
    q, k, v = rng.standard_normal((T + 1, Hq, d)), *rng.standard_normal((2, T + 1, Hkv, d))
    w, W, A = rng.uniform(0.5, 1.5, d), rng.standard_normal((Hkv * d, Hkv)), -rng.uniform(0.1, 2, Hkv)
    table = rng.permutation(12).reshape(3, 4)
    z = np.full((12, page, Hkv, d), 9.0)
    cu = np.cumsum([0] + news)
    qo, ko, kp, vp, dp = oracle.append_paged(q, k, v, w, w, 1e-6, 100.0, W, A, cu, positions, table, z, z,
                                             np.full((12, Hkv, page), 9.0))
    assert np.isnan(qo[T]).all() and np.isfinite(qo[:T]).all()
    touched = np.zeros((12, page), bool)
    for b, n in enumerate(news):
        if n == 0:
            continue
        t = slice(cu[b], cu[b + 1])
        c = np.zeros((1, 12, Hkv, d))
        wq, wk, wv = oracle.prologue(q[t][None], k[t][None], v[t][None], w, w, 1e-6, 100.0, [positions[b]], c, c)
        np.testing.assert_array_equal(qo[t], wq[0])
        dt = oracle.dt_scores64(v[t][None], W, A)[0]
        for i in range(n):
            j = positions[b] + i
            at = table[b, j // page], j % page
            touched[at] = True
            np.testing.assert_array_equal(kp[at], wk[0, j])
            np.testing.assert_array_equal(vp[at], v[cu[b] + i])
            np.testing.assert_allclose(dp[at[0], :, at[1]], dt[:, i], rtol=1e-14)
    assert (kp[~touched] == 9.0).all() and (vp[~touched] == 9.0).all()
    assert touched.sum() == T
