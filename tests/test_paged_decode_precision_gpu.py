"""The paged decode holds its probabilities in 32 bits: outputs in which the leading bits of a probability cancel.

Three keys, q = 0, so the scores are the keys' dt: 1, x, 1.  With p = e^(x - 1), c1 = bf16(p) and c2 = bf16(p - c1)
the values are -c1, 1 and -c2, so

    o = (p - c1 - c2) / (2 + p),

what two bf16 terms of p leave of it.  x is chosen so that |p - c1 - c2| lies between 0.8 * 2^-18 and 2^-18 (half an
ulp of c2 at most): |o| is above 1.0e-6, and a p of two bf16 terms gives 0.

Tolerance.  Scores in log2 units lie below 1.45: three roundings of at most 2^-24 (the products of both keys, their
difference), times ln 2; the constant log2(e) is off by 2^-25 of itself; 2^x is off by 2^-22 at most.  Together below
3.9e-7 of p.  A product's sum in the tensor core is off by 2^-23 of its largest term (1) at most, three of them: 3.6e-7.
Divided by 2 + p (at least 2.5, the division's own rounding far below): 3e-7.  The output's rounding: 2^-8 of it.
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


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def chosen_dt(n):
    """n float32 dt in (0.36, 0.99) whose probability leaves nearly half an ulp behind its two bf16 terms."""
    x = np.random.default_rng(7).uniform(0.36, 0.99, 4000).astype(np.float32)
    p = np.exp(x.astype(np.float64) - 1)
    c1 = bf16(p)
    c2 = bf16(p - c1)
    at = np.flatnonzero(np.abs(p - c1 - c2) >= 0.8 * 2.0 ** -18)[:n]
    assert len(at) == n
    return x[at], c1[at], c2[at]


@pytest.mark.parametrize("Hq,Hkv,d,w", [(8, 4, 64, 2048), (16, 2, 128, 2048), (4, 4, 128, 3), (3, 1, 64, 3)])
def test_probabilities_hold_what_bf16_terms_leave(dma, Hq, Hkv, d, w):
    """w = 3: a fourth key, of the lowest dt, is not kept, so the kept list is read."""
    B, page, n = 24, 16, 4 if w == 3 else 3
    x, c1, c2 = chosen_dt(B)
    dt = np.full((B, Hkv, page), 0.125, dtype=np.float32)
    dt[:, :, 0], dt[:, :, 1], dt[:, :, 2] = 1.0, x[:, None], 1.0
    v = np.ones((B, page, Hkv, d))
    v[:, 0], v[:, 2] = -c1[:, None, None], -c2[:, None, None]
    kp = torch.randn((B, page, Hkv, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    vp = torch.from_numpy(v).to(torch.bfloat16)
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16)
    table, lens = torch.arange(B, dtype=torch.int32)[:, None], torch.full((B,), n, dtype=torch.int32)
    out = dma.dma_decode_paged(q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(dt).cuda(), table.cuda(), lens.cuda(), w)
    want = oracle.decode_paged(q.double().numpy(), kp.double().numpy(), vp.double().numpy(), dt, table.numpy(),
                               lens.numpy(), w, 0, 0, d ** -0.5)
    assert (np.abs(want) >= 1.0e-6).all()
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 3e-7).all(), f"off by {err.max():.2e} of {np.abs(want).min():.2e}"


@pytest.mark.parametrize("d,warps", [(64, 16), (128, 8)])
def test_long_sums_are_rounded_to_nearest(dma, d, warps):
    """128 rows of 65536 keys: values of 1 and, in three keys at the end, what makes the 64-bit output vanish.  All a
    warp's sums grow one way, so an addition that cuts off bits (as a chain of tensor-core products does) is off by
    2^-24 of the sum on average each time, and the output by 1e-5 and more.

    Tolerance, relative to the sum of the probabilities: every tile's sum enters a warp's by one addition, off by at
    most half an ulp either way: 4 sqrt(tiles) ulps with a probability of 2 e^-32 to be off by more (Hoeffding).  A
    probability: 2^-22 (2^x) and 1.3e-7 (its score), for the keys and for the last three.  The last tile's three products:
    2^-23 each.  Joining: an addition of 2^-24 per warp of the row, and 2^-22 of a piece's weight."""
    page, pages, n, B, Hkv = 64, 9, 65536, 64, 2
    gen = torch.Generator().manual_seed(d)
    dt = 0.2 + 0.8 * torch.rand((pages, page), generator=gen)
    dt[-1, -3:] = 0.7
    table = torch.randint(0, pages - 1, (n // page,), generator=gen)
    table[-1] = pages - 1
    p = torch.exp(dt.double() - 1)[table].flatten()
    v = torch.ones((pages, page), dtype=torch.float64)
    rest = -p[:-3].sum()
    for i in (-3, -2, -1):
        v[-1, i] = (rest / p[-1]).to(torch.bfloat16).double()
        rest -= v[-1, i] * p[-1]
    assert abs(rest) < 1e-7 * p.sum()
    vp = v.to(torch.bfloat16)[:, :, None, None].expand(pages, page, Hkv, d).contiguous().cuda()
    kp = torch.randn((pages, page, Hkv, d), generator=gen).to(torch.bfloat16).cuda()
    dtp = dt[:, None].expand(pages, Hkv, page).contiguous().cuda()
    q = torch.zeros((B, 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    tab = table.to(torch.int32)[None].expand(B, -1).contiguous().cuda()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out = dma.dma_decode_paged(q, kp, vp, dtp, tab, lens, 1 << 20).double().abs().max().item()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_warp = -(-B * Hkv * (n // 16) // (sms * warps))
    ulp = 2.0 ** (np.floor(np.log2(16.0 * per_warp)) - 23)
    total = p.sum().item()
    tol = (4 * np.sqrt(n // 16) * ulp / total + 2 * (2.0 ** -22 + 1.3e-7) + 3 * 2.0 ** -23
           + (n // 16 // per_warp + 2) * 2.0 ** -24 + 2.0 ** -22)
    assert tol < 8e-6 and out <= tol, f"{out:.2e}, tolerance {tol:.2e}"
