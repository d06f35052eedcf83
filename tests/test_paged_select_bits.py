"""The paged selection over dt bits that no score has (dt >= 0 is the contract, but pages may hold what was never
written): the kept lists hold visible positions, each once, ordered by the bits as whole numbers.

On the host: the narrowing of a range of bits to one value, step by step as the kernel does it, in 32 bits."""
import numpy as np
import pytest
import torch

M = 0xFFFFFFFF


def bin_shift(r):
    top = (r | 1).bit_length()
    return top - 11 if top > 11 else 0


def bin_top(lo, shift, hi):
    return hi if (hi - lo) & M < 1 << shift else (lo + (1 << shift) - 1) & M


def narrowed(bits, k, top):
    """(value of the k-th largest, how many of the keys equal to it belong to the k)."""
    lo, hi = min(bits), max(bits)
    while lo < hi:
        s = bin_shift(hi - lo)
        bins = [((x - lo) & M) >> s for x in bits if lo <= x <= hi]
        assert max(bins) < 2048
        hist = np.bincount(bins, minlength=2048)
        above = 0
        for b in range(2047, -1, -1):
            if above + hist[b] >= k:
                break
            above += hist[b]
        else:
            return None
        k -= above
        l2 = (lo + (b << s)) & M
        lo, hi = l2, top(l2, s, hi)
    return lo, k


def wrapping(lo, shift, hi):
    """The sum as 32 bits hold it."""
    return min(hi, (lo + (1 << shift) - 1) & M)


def patterns(n, rng):
    score = np.exp(-rng.uniform(0, 3, n)).astype(np.float32).view(np.uint32)
    high = (0xFFE00000 + rng.integers(0, 0x1FFFFF, n)).astype(np.uint32)
    part = rng.random(n)
    return {"all ones": np.full(n, M, np.uint32),
            "ones over scores": np.where(part < 0.9, np.uint32(M), score),
            "a few ones": np.where(part < 0.001, np.uint32(M), score),
            "near the top": high,
            "scores and near the top": np.where(part < 0.5, high, score),
            "NaN over scores": np.where(part < 0.5, np.uint32(0x7FC00000), score),
            "negative NaN": np.where(part < 0.5, np.uint32(0xFFC00000), score),
            "any": rng.integers(0, 1 << 32, n).astype(np.uint32)}


KINDS = list(patterns(1, np.random.default_rng(0)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,k", [(900, 1), (900, 60), (900, 899)])
def test_narrowing_ends_at_the_kth_value(kind, n, k):
    bits = [int(x) for x in patterns(n, np.random.default_rng(n + k))[kind]]
    want = sorted(bits, reverse=True)[k - 1]
    assert narrowed(bits, k, bin_top) == (want, k - sum(x > want for x in bits))


def test_a_wrapping_sum_would_miss_it():
    """What the kernel's step must not do: the range ends below itself, at a value no key has."""
    bits = [int(x) for x in patterns(900, np.random.default_rng(3))["scores and near the top"]]
    missed = [k for k in (1, 60, 500) if narrowed(bits, k, wrapping)[0] != sorted(bits, reverse=True)[k - 1]]
    assert missed


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,w,window,sinks,page,max_pages", [
    (9001, 600, 0, 0, 16, 563),                  # the table ends with the sequence's last page
    (9001, 600, 8000, 13, 5, 1801),
    (60000, 2048, 0, 0, 64, 938),                # a cluster per row
    (700, 600, 0, 0, 8, 88),
])
def test_kept_lists_of_any_bits(n, w, window, sinks, page, max_pages, kind):
    from doge_dynamic_mask_b200 import dma
    import oracle
    Hkv, d = 2, 64
    rng = np.random.default_rng(n + w)
    pages = -(-n // page)
    bits = np.stack([patterns(n, rng)[kind] for _ in range(Hkv)])
    pool = np.zeros((Hkv, pages * page), np.uint32)
    pool[:, :n] = bits
    dt = torch.from_numpy(pool.view(np.float32).reshape(Hkv, pages, page).transpose(1, 0, 2).copy()).cuda()
    assert np.array_equal(dt.cpu().numpy().view(np.uint32).transpose(1, 0, 2).reshape(Hkv, -1)[:, :n], bits)
    kv = torch.ones((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((1, Hkv, d), dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = dma.new_workspace(dma.dma_decode_paged_workspace_size(1, max_pages, page, Hkv, Hkv, d, w, window, sinks))
    dma.dma_decode_paged(q, kv, kv, dt, table, lens, w, window=window, sinks=sinks, workspace=ws)
    assert dma.dma_check(ws) == 0
    pos, bias = (t.cpu().numpy() for t in dma.paged_list_views(ws, 1, Hkv, Hkv, d, w))
    j = np.array(oracle.visible_positions(n, window, sinks))
    for h in range(Hkv):
        best = j[np.argsort(-(bits[h][j].astype(np.int64)), kind="stable")[:w]]
        got = np.argsort(pos[0, h])
        assert np.array_equal(pos[0, h][got], np.sort(best))
        assert np.array_equal(bias[0, h].view(np.uint32)[got], bits[h][np.sort(best)])
