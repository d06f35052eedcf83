"""The prologue's backward over rows at the ends of its range: NaN and infinite entries, and rows of (nearly) nothing
with eps = 0 or the smallest eps."""
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
    return t.detach().double().cpu().numpy()


def inputs(B, L, Hq, Hkv, d, seed):
    gen = torch.Generator().manual_seed(seed)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
    return {"q": bf(B, L, Hq, d), "k": bf(B, L, Hkv, d), "q_w": torch.rand(d, generator=gen) + 0.5,
            "k_w": torch.rand(d, generator=gen) + 0.5, "positions": torch.arange(B, dtype=torch.int32),
            "dq_out": bf(B, L, Hq, d), "dk_out": bf(B, L, Hkv, d)}


def run(dma, x, eps=1e-6):
    return dict(zip(("q", "k", "q_w", "k_w"), dma.dma_prologue_backward(*[t.cuda() for t in x.values()], eps=eps)))


SHAPES = [(1, 1, 8, 4, 64), (2, 5, 3, 1, 64), (1, 7, 5, 1, 128), (3, 40, 16, 8, 128)]


@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("name", ["q", "k"])
@pytest.mark.parametrize("B,L,Hq,Hkv,d", SHAPES)
def test_a_nan_reaches_all_of_its_row_and_of_the_weights(dma, B, L, Hq, Hkv, d, name, eps):
    x = inputs(B, L, Hq, Hkv, d, seed=L)
    clean = run(dma, x, eps)
    x[name][B - 1, L // 2, -1, 3] = float("nan")
    got = run(dma, x, eps)
    row = torch.zeros(x[name].shape, dtype=torch.bool, device="cuda")
    row[B - 1, L // 2, -1] = True
    assert got[name][row].isnan().all()
    assert torch.equal(got[name][~row], clean[name][~row])
    assert got[name + "_w"].isnan().all()
    other = "k" if name == "q" else "q"
    for n in (other, other + "_w"):
        assert torch.equal(got[n], clean[n])


@pytest.mark.parametrize("B,L,Hq,Hkv,d", SHAPES)
def test_an_infinite_entry(dma, B, L, Hq, Hkv, d):
    """The row's norm is infinite: its other entries normalise to 0, inf / inf is NaN."""
    x = inputs(B, L, Hq, Hkv, d, seed=L)
    without = {n: t.clone() for n, t in x.items()}
    x["q"][0, 0, 0, 5] = float("inf")
    without["q"][0, 0, 0] = 0                        # adds nothing to the weights
    got, clean = run(dma, x), run(dma, without)
    assert got["q"][0, 0, 0].isnan().all()
    assert got["q_w"][5].isnan()
    others = torch.arange(d, device="cuda") != 5
    assert torch.equal(got["q_w"][others], clean["q_w"][others])
    assert torch.equal(got["k_w"], clean["k_w"])


def check(x, got, eps, rel):
    """rel: what the float32 mean square of the rows at hand costs, on top of 60 roundings of 2^-24."""
    p = x["positions"].numpy()
    want = oracle.prologue_backward(f64(x["q"]), f64(x["k"]), f64(x["q_w"]), f64(x["k_w"]), eps, 10000.0, p,
                                    f64(x["dq_out"]), f64(x["dk_out"]))
    for n, dx, dw in (("q", want[0], want[2]), ("k", want[1], want[3])):
        xi, g, w = f64(x[n]), f64(x["d%s_out" % n]), f64(x[n + "_w"])
        r = 1 / np.sqrt((xi ** 2).mean(-1, keepdims=True) + eps)
        size = r * np.linalg.norm(g * w.max(), axis=-1, keepdims=True)
        err = np.abs(f64(got[n]) - dx)
        assert (err <= 2.0 ** -8 * np.abs(dx) + (2.0 ** -18 + rel) * size).all(), f"d{n}: {err.max():.3e}"
        turned = np.stack([np.abs(oracle.rope(np.abs(g[b]), 0 * np.arange(xi.shape[1]), 10000.0)) for b in range(len(p))])
        half = xi.shape[-1] // 2
        pair = turned + np.roll(turned, half, -1)    # a rotated entry is at most the pair's sum
        terms = (pair * np.abs(xi) * r).sum((0, 1, 2))
        rows = xi.shape[0] * xi.shape[1] * xi.shape[2]
        err = np.abs(f64(got[n + "_w"]) - dw)
        assert (err <= ((rows + 44) * 2.0 ** -24 + rel) * terms).all(), f"d{n}_norm_w: {err.max():.3e}"


@pytest.mark.parametrize("power,eps", [(-40, 0.0), (-60, 0.0), (-66, 0.0), (-66, 1e-45), (-66, 1e-39), (-60, 1e-37)])
@pytest.mark.parametrize("B,L,Hq,Hkv,d", [(1, 1, 8, 4, 64), (2, 3, 3, 1, 64), (1, 5, 5, 1, 128)])
def test_rows_of_next_to_nothing(dma, B, L, Hq, Hkv, d, power, eps):
    """Entries about 2^power.  Below 2^-63 the squares are subnormal: at 2^-66 the mean square is about 2^-132 and each
    of its d + 1 roundings at most 2^-150 (those of the d terms count 1/d each): 2^-17 of it, half of that in r, three
    factors of r in a gradient."""
    x = inputs(B, L, Hq, Hkv, d, seed=L - power)
    for n in ("q", "k"):                             # entries within a factor of two of 2^power, so the mean square is
        x[n] = ((1 + x[n].float().abs().clamp(max=0.99)) * x[n].float().sign() * 2.0 ** power).to(torch.bfloat16)
    eps = float(np.float32(eps))
    check(x, run(dma, x, eps), eps, 3 * 2.0 ** -18 if power < -63 else 0.0)


@pytest.mark.parametrize("B,L,Hq,Hkv,d", SHAPES)
def test_a_row_of_zeros_has_no_gradient_without_eps(dma, B, L, Hq, Hkv, d):
    """0 / 0, as in the forward; with the smallest eps the row is zeros and adds nothing to the weights."""
    x = inputs(B, L, Hq, Hkv, d, seed=L)
    x["k"][0, L - 1, 0] = 0
    got = run(dma, x, 0.0)
    row = torch.zeros(x["k"].shape, dtype=torch.bool, device="cuda")
    row[0, L - 1, 0] = True
    assert got["k"][row].isnan().all() and got["k_w"].isnan().all()
    assert got["k"][~row].isfinite().all() and got["q"].isfinite().all() and got["q_w"].isfinite().all()
    tiny = run(dma, x, 1e-45)
    assert tiny["k_w"].isfinite().all() and tiny["k"].isfinite().all()
    assert torch.equal(tiny["k"][~row], got["k"][~row]) and torch.equal(tiny["q_w"], got["q_w"])


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 4, 64), (2, 1, 128)])
def test_small_angles_reach_the_weights(dma, Hq, Hkv, d):
    """A gradient of the upper channels only: dw of a lower channel is sum_h g sin(a) x r, all terms positive, so it is
    exact to a few roundings of itself: g sin(a) and its angle 2^-23 each (the angle is below 1, so a relative error of
    it is one of its sine), sin 2^-23, x r 2^-21.5 (the inverse root 2^-22.5, its argument's some ten roundings of
    2^-24, halved), the sum over heads 2^-22: 2^-20 in all.  dw of an upper channel has cos(a) in place of the sine."""
    x = inputs(1, 1, Hq, Hkv, d, seed=d)
    x["positions"] = torch.tensor([1], dtype=torch.int32)
    for n in ("q", "k", "dq_out", "dk_out"):
        x[n] = (x[n].float().abs() + 0.5).to(torch.bfloat16)
    for n in ("dq_out", "dk_out"):
        x[n][..., :d // 2] = 0
    got = run(dma, x)
    want = oracle.prologue_backward(f64(x["q"]), f64(x["k"]), f64(x["q_w"]), f64(x["k_w"]), 1e-6, 10000.0, [1],
                                    f64(x["dq_out"]), f64(x["dk_out"]))
    for n, dw in (("q_w", want[2]), ("k_w", want[3])):
        err = np.abs(f64(got[n]) - dw) / np.abs(dw)
        assert (err <= 2.0 ** -20).all(), f"{n}: {err.max():.2e}"
