"""Backward of the prologue's norms and rotation on the GPU, against the float64 oracle, and the training run it is
part of.

Tolerances.  dx is rounded once to bf16 (2^-8 of the value) after fewer than 60
float32 roundings of terms that r |w g|_2 bounds (r the row's inverse root mean
square): 2^-18 of that.  A weight gradient is a float32 sum: at most one
rounding of 2^-24 of sum|dy x r| per added term along the longest chain, and
some 40 more for the terms themselves and the tree above the lanes.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dma():
    from doge_dynamic_mask_b200 import build
    build.build()
    from doge_dynamic_mask_b200 import dma as m
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(B, L, Hq, Hkv, d, positions, seed, small_rows=False):
    gen = torch.Generator().manual_seed(seed)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
    x = {"q": bf(B, L, Hq, d), "k": bf(B, L, Hkv, d), "dq_out": bf(B, L, Hq, d), "dk_out": bf(B, L, Hkv, d),
         "q_w": torch.rand(d, generator=gen) + 0.5, "k_w": torch.rand(d, generator=gen) + 0.5,
         "positions": torch.tensor(positions, dtype=torch.int32)}
    if small_rows:                       # rows whose mean square is near or far below eps
        x["q"][0, 0] *= 1e-3
        x["q"][0, -1] = 0
        x["k"][-1, 0] *= 1e-6
    return x


def check(x, dq, dk, dqw, dkw, theta, eps=1e-6):
    p = x["positions"].numpy()
    want = oracle.prologue_backward(f64(x["q"]), f64(x["k"]), f64(x["q_w"]), f64(x["k_w"]), eps, theta, p,
                                    f64(x["dq_out"]), f64(x["dk_out"]))
    for got, ref, inp, w, g, what in ((dq, want[0], "q", "q_w", "dq_out", "dq"), (dk, want[1], "k", "k_w", "dk_out", "dk")):
        r = 1 / np.sqrt((f64(x[inp]) ** 2).mean(-1, keepdims=True) + eps)
        size = r * np.linalg.norm(f64(x[g]) * f64(x[w]).max(), axis=-1, keepdims=True)
        err = np.abs(f64(got) - ref)
        assert np.isfinite(f64(got)).all()
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size).all(), f"{what}: {err.max():.3e}"
    for got, ref, inp, g, what in ((dqw, want[2], "q", "dq_out", "dq_norm_w"), (dkw, want[3], "k", "dk_out", "dk_norm_w")):
        xi = f64(x[inp])
        xh = xi / np.sqrt((xi ** 2).mean(-1, keepdims=True) + eps)
        terms = np.stack([np.abs(oracle.rope(f64(x[g])[b], -(int(p[b]) + np.arange(xi.shape[1])), theta) * xh[b]).sum((0, 1))
                          for b in range(len(p))]).sum(0)
        # the angles' float32 error turns a channel pair into itself: the partner's term counts as well
        half = xi.shape[-1] // 2
        terms = terms + np.roll(terms, half)
        n = xi.shape[0] * xi.shape[1] * xi.shape[2]
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= (n / 4 + 44) * 2.0 ** -24 * terms).all(), f"{what}: {err.max():.3e}"


@pytest.mark.parametrize("B,L,Hq,Hkv,d,positions,theta", [
    (1, 1, 8, 4, 64, [0], 10000.0),
    (1, 1, 1, 1, 128, [5], 10000.0),
    (2, 37, 8, 4, 64, [0, 9], 10000.0),
    (3, 11, 3, 1, 128, [4, 0, 100], 10000.0),
    (2, 5, 16, 16, 64, [-3, 7], 500.0),                       # positions are only angles here
    (1, 9, 32, 4, 128, [2 ** 30], 500000.0),                  # far positions: angles need double precision
    (1, 700, 16, 8, 128, [0], 10000.0),
    (5, 333, 4, 2, 64, [0, 1, 2, 3, 4], 10000.0),
])
def test_matches_oracle(dma, B, L, Hq, Hkv, d, positions, theta):
    x = inputs(B, L, Hq, Hkv, d, positions, seed=B * 1000 + L, small_rows=L > 1)
    g = {n: t.cuda() for n, t in x.items()}
    call = lambda: dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"],
                                             g["dk_out"], rope_theta=theta)
    r = call()
    check(x, *r, theta)
    for a, b in zip(r, call()):
        assert torch.equal(a, b)                              # the same call, the same bits


@pytest.mark.parametrize("B,L,Hq,Hkv,d", [(1, 3, 3, 1, 64), (3, 7, 5, 1, 128), (1, 33, 6, 2, 64), (1, 1, 1, 1, 64)])
def test_without_eps(dma, B, L, Hq, Hkv, d):
    """eps = 0: heads and tokens that fill up a warp's step must not add to the weights' gradients."""
    x = inputs(B, L, Hq, Hkv, d, list(range(B)), seed=d + L)
    g = {n: t.cuda() for n, t in x.items()}
    r = dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"], eps=0.0)
    check(x, *r, 10000.0, eps=0.0)


def test_slices_of_projection_buffers(dma):
    B, L, Hq, Hkv, d = 2, 19, 8, 4, 64
    x = inputs(B, L, Hq, Hkv, d, [0, 3], seed=5)
    g = {n: t.cuda() for n, t in x.items()}
    qkv = torch.cat([g["q"], g["k"], torch.full_like(g["k"], float("nan"))], 2)
    grads = torch.full_like(qkv, 77.0)
    q, k, _ = torch.split(qkv, [Hq, Hkv, Hkv], 2)
    dq, dk, dv = torch.split(grads, [Hq, Hkv, Hkv], 2)
    r = dma.dma_prologue_backward(q, k, g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"], dq=dq, dk=dk)
    want = dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"])
    for a, b in zip(r, want):
        assert torch.equal(a, b)
    assert (dv == 77.0).all()
    check(x, *r, 10000.0)


def test_more_tokens_than_resident_warps(dma):
    B, L, Hq, Hkv, d = 1, 20000, 2, 1, 64
    x = inputs(B, L, Hq, Hkv, d, [1], seed=6)
    g = {n: t.cuda() for n, t in x.items()}
    check(x, *dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"]), 10000.0)


def test_differences(dma):
    """The gradients against central differences of the prologue itself (in float64, through the oracle)."""
    B, L, Hq, Hkv, d = 1, 3, 2, 1, 64
    x = inputs(B, L, Hq, Hkv, d, [7], seed=8)
    g = {n: t.cuda() for n, t in x.items()}
    dq, dk, dqw, dkw = dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"])
    z = np.zeros((B, 16, Hkv, d))
    args = {n: f64(x[n]) for n in ("q", "k", "q_w", "k_w")}

    def loss(a):
        qo, kc, _ = oracle.prologue(a["q"], a["k"], np.zeros((B, L, Hkv, d)), a["q_w"], a["k_w"], 1e-6, 10000.0, [7], z, z)
        return (qo * f64(x["dq_out"])).sum() + (kc[:, 7:7 + L] * f64(x["dk_out"])).sum()

    rng = np.random.default_rng(0)
    for name, got in (("q", dq), ("k", dk), ("q_w", dqw), ("k_w", dkw)):
        step = rng.standard_normal(args[name].shape)
        hi, lo = dict(args), dict(args)
        hi[name], lo[name] = args[name] + 1e-4 * step, args[name] - 1e-4 * step
        want = (loss(hi) - loss(lo)) / 2e-4
        have = (got.double().cpu().numpy() * step).sum()
        # each rounded gradient entry is off by at most 2^-8 of itself
        assert abs(have - want) <= 2.0 ** -8 * np.abs(f64(got) * step).sum() + 1e-3


def test_captured_and_replayed(dma):
    x, y = (inputs(2, 50, 8, 4, 64, p, seed=s) for p, s in (([0, 1], 1), ([9, 30], 2)))
    g = {n: t.cuda() for n, t in x.items()}
    dq, dk = torch.empty_like(g["q"]), torch.empty_like(g["k"])
    dqw, dkw = torch.empty_like(g["q_w"]), torch.empty_like(g["k_w"])
    ws = dma.new_workspace(dma.dma_prologue_backward_workspace_size(2, 50, 8, 4, 64))
    call = lambda: dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], g["dq_out"], g["dk_out"],
                                             dq=dq, dk=dk, dq_norm_w=dqw, dk_norm_w=dkw, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for z in (y, x):
        for n in g:
            g[n].copy_(z[n].cuda())
        graph.replay()
        torch.cuda.synchronize()
        check(z, dq, dk, dqw, dkw, 10000.0)


def test_training_run(dma):
    """Prologue, attention with row normalisers, attention backward, prologue backward: a training step's attention
    part, its gradients against the oracle's chained in float64.  The intermediate tensors are bf16, so an entry may
    be off by their roundings: 2^-8 each for the rotated inputs, the output, and the gradients in between, carried
    through sums over the keys; 2e-2 of the gradient's largest entry covers them at this size (the attention
    backward's own bar)."""
    B, L, Hq, Hkv, d, w = 2, 96, 4, 2, 64, 40
    x = inputs(B, L, Hq, Hkv, d, [0, 0], seed=13)
    gen = torch.Generator().manual_seed(14)
    v = torch.randn((B, L, Hkv, d), generator=gen).to(torch.bfloat16)
    W = torch.randn((Hkv * d, Hkv), generator=gen) * 0.02
    A = torch.tensor([-0.7, -1.3])
    dout = torch.randn((B, L, Hq, d), generator=gen).to(torch.bfloat16)
    g = {n: t.cuda() for n, t in x.items()}
    kc, vc = (torch.empty((B, L, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qr = dma.dma_prologue(g["q"], g["k"], v.cuda(), g["q_w"], g["k_w"], g["positions"], kc, vc)
    lse = torch.empty((B, Hq, L), device="cuda")
    dt = oracle.dt_scores(f64(v), W.double().numpy(), A.double().numpy())     # one dt, so one kept set, on both sides
    dtg = torch.from_numpy(dt).cuda()
    out = dma.dma_forward_prefill(qr, kc, vc, W.cuda(), A.cuda(), None, w, dt_in=dtg, lse_out=lse)
    dq, dk, dv, dW, dA = dma.dma_backward_prefill(qr, kc, vc, W.cuda(), A.cuda(), None, w, out, dout.cuda(), dt_in=dtg,
                                                  lse_in=lse)
    r = dma.dma_prologue_backward(g["q"], g["k"], g["q_w"], g["k_w"], g["positions"], dq, dk)
    z = np.zeros((B, L, Hkv, d))
    q64, k64, _ = oracle.prologue(f64(x["q"]), f64(x["k"]), f64(v), f64(x["q_w"]), f64(x["k_w"]), 1e-6, 10000.0, [0, 0], z, z)
    grads = oracle.prefill_backward(q64, k64, f64(v), W.double().numpy(), A.double().numpy(), [L] * B, w, d ** -0.5, f64(dout),
                                    dt_fixed=dt)
    want = oracle.prologue_backward(f64(x["q"]), f64(x["k"]), f64(x["q_w"]), f64(x["k_w"]), 1e-6, 10000.0, [0, 0],
                                    grads[0], grads[1])
    for got, ref in zip(r, want):
        assert np.abs(got.double().cpu().numpy() - ref).max() <= 2e-2 * np.abs(ref).max()
