"""The weight gradients of the prologue's backward as sums: a bound from the additions that a term goes through, tight
enough that the share of any one warp, left out, breaks it.

A warp step takes four heads of 128 / d tokens; the tokens' items (or parts of them, when they are few) are dealt to the
warps of the grid in turn.  A term passes through
  * its lane's additions: the steps of the warp's items,
  * log2(512 / d) exchanges between the lanes of a channel, eight warps,
  * the blocks, every 2048 / (d / 2)-th or so to a thread, and those threads' sums,
each off by 2^-24 of the terms' sum of magnitudes at most.  The terms themselves: the turned gradient is off by the
angle (2 pi 2^-26, and 2^-23 of its sine and cosine) and two roundings, 6 * 2^-24 of the channel pair's magnitudes;
the normalised entry by half of the mean square's some 14 roundings, the inverse root's 2^-22.5 and a product, 11 *
2^-24: 20 * 2^-24 with the product of both and to spare."""
import numpy as np
import pytest
import torch

import oracle

CASES = [(1, 20000, 2, 1, 64), (3, 3001, 16, 8, 128), (1, 37, 8, 4, 64), (2, 700, 5, 1, 128), (7, 1200, 8, 4, 64)]


def inputs(B, L, Hq, Hkv, d):
    gen = torch.Generator().manual_seed(L + d)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
    return {"q": bf(B, L, Hq, d), "k": bf(B, L, Hkv, d), "q_w": torch.rand(d, generator=gen) + 0.5,
            "k_w": torch.rand(d, generator=gen) + 0.5, "positions": torch.arange(B, dtype=torch.int32) * 11,
            "dq_out": bf(B, L, Hq, d), "dk_out": bf(B, L, Hkv, d)}


class Deal:
    """Which warp of the grid takes which rows."""

    def __init__(self, T, Hq, Hkv, d, sms):
        slots = min(2 * sms, 512)
        self.q_steps, self.steps = -(-Hq // 4), -(-Hq // 4) - (-Hkv // 4)
        self.per_group = 128 // d
        groups = -(-T // self.per_group)
        self.parts = min(max(1, slots * 8 // groups), self.steps)
        self.items = groups * self.parts
        self.blocks = min(-(-self.items // 8), slots)
        lane = -(-self.items // (self.blocks * 8)) * -(-self.steps // self.parts)
        rows = 256 // (2 * d // 4)
        self.depth = lane + int(np.log2(512 // d)) + 8 + -(-self.blocks // rows) + rows

    def warp_of(self, token, head, tensor):
        step = head // 4 + (self.q_steps if tensor == "k" else 0)
        # part p has the steps from p * steps // parts on
        part = next(p for p in range(self.parts - 1, -1, -1) if p * self.steps // self.parts <= step)
        return (token // self.per_group * self.parts + part) % (self.blocks * 8)


def terms_of(x, tensor, eps=1e-6):
    """(terms [T, H, d] whose sum over rows is the weight gradient, magnitudes that bound their errors)"""
    f = lambda t: t.double().numpy()
    xi, g = f(x[tensor]), f(x["d%s_out" % tensor])
    xh = xi / np.sqrt((xi ** 2).mean(-1, keepdims=True) + eps)
    dy = np.stack([oracle.rope(g[b], -(int(x["positions"][b]) + np.arange(xi.shape[1])), 10000.0) for b in range(len(g))])
    half = xi.shape[-1] // 2
    pair = np.abs(g) + np.roll(np.abs(g), half, -1)
    flat = lambda t: t.reshape(-1, *t.shape[2:])
    return flat(dy * xh), flat(pair * np.abs(xh))


def bound(deal, size):
    return (deal.depth + 20) * 2.0 ** -24 * size.sum((0, 1))


@pytest.mark.parametrize("B,L,Hq,Hkv,d", CASES)
def test_a_lost_share_breaks_the_bound(B, L, Hq, Hkv, d):
    """On the host, for 148 SMs: the share of each warp, and so that of each block, is more than twice the bound."""
    x, deal = inputs(B, L, Hq, Hkv, d), Deal(B * L, Hq, Hkv, d, 148)
    for tensor, heads in (("q", Hq), ("k", Hkv)):
        terms, size = terms_of(x, tensor)
        shares = np.zeros((deal.blocks * 8, d))
        warp = np.array([[deal.warp_of(t, h, tensor) for h in range(heads)] for t in range(B * L)])
        np.add.at(shares, warp.reshape(-1), terms.reshape(-1, d))
        has = np.bincount(warp.reshape(-1), minlength=len(shares)) > 0
        seen = (np.abs(shares) / bound(deal, size)).max(-1)
        assert seen[has].min() > 2, f"{tensor}: {seen[has].min():.2f}"
        blocks = shares.reshape(8, deal.blocks, d).sum(0)
        assert (np.abs(blocks) / bound(deal, size)).max(-1)[has.reshape(8, deal.blocks).any(0)].min() > 2


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,Hq,Hkv,d", CASES)
def test_weight_gradients_hold_every_share(B, L, Hq, Hkv, d):
    from doge_dynamic_mask_b200 import dma
    x = inputs(B, L, Hq, Hkv, d)
    deal = Deal(B * L, Hq, Hkv, d, torch.cuda.get_device_properties(0).multi_processor_count)
    _, _, dqw, dkw = dma.dma_prologue_backward(*[t.cuda() for t in x.values()])
    for tensor, got in (("q", dqw), ("k", dkw)):
        terms, size = terms_of(x, tensor)
        err = np.abs(got.double().cpu().numpy() - terms.sum((0, 1)))
        assert (err <= bound(deal, size)).all(), f"{tensor}: {(err / bound(deal, size)).max():.2f} of the bound"
