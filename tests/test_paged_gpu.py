"""The paged cache on the GPU: the append and the decode step, against the float64 oracle.

Tolerances.  bf16 results carry one rounding, at most 2^-8 of the value, plus
float32 arithmetic:

* append: a rotated value is at most about 17 (weights below 1.5, a normalised
  row's largest entry below sqrt(d)) after some eight float32 roundings of
  2^-24 and an angle exact to 2 pi 2^-25: below 2e-5.
* dt: products with the three-term weight are exact, so x = v W differs by the
  float32 additions alone: at most 24 accumulations per warp and 16 warps, each
  off by 2^-23 of a partial sum that sum|v W| bounds; exp, log1p and the product
  with A add a few 2^-23 of the exponent.
* decode: scores in log2 units are sums of d/16 accumulations, off by at most
  2^-23 of the sum of |q k| scale log2(e) (about 10) each: 1e-5; P in two bf16
  terms: 2^-17; so a sum of p v is off by less than 4e-5 of max|v| (below 5).
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
DECODE_ATOL = 2e-4


@pytest.fixture(scope="module")
def dma():
    from doge_dynamic_mask_b200 import build
    build.build()
    from doge_dynamic_mask_b200 import dma as m
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def assert_close(got, want, rtol, atol, what):
    g = got if isinstance(got, np.ndarray) else f64(got)
    assert np.isfinite(g).all(), what
    bad = np.abs(g - want) > rtol * np.abs(want) + atol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside the bound, max err {np.abs(g - want).max():.3e}"


def page_table(counts, max_pages, gen, spare=2):
    """A table of scattered pages; entries no sequence needs hold an invalid page."""
    n = sum(counts) + spare
    perm = torch.randperm(n, generator=gen).to(torch.int32)
    table = torch.full((len(counts), max_pages), -7, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    return table, n


def randn_bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


# ---- append -------------------------------------------------------------------------

def append_inputs(news, positions, Hq, Hkv, d, page, lead=0, pad=0, fused=False, seed=0, max_pages=None):
    gen = torch.Generator().manual_seed(seed)
    T = lead + sum(news) + pad
    if fused:
        qkv = randn_bf16((T, Hq + 2 * Hkv, d), gen)
        q, k, v = torch.split(qkv, [Hq, Hkv, Hkv], 1)
    else:
        q, k, v = randn_bf16((T, Hq, d), gen), randn_bf16((T, Hkv, d), gen), randn_bf16((T, Hkv, d), gen)
    counts = [-(-(p + n) // page) for p, n in zip(positions, news)]
    table, n_pages = page_table(counts, max_pages or max(max(counts), 1), gen)
    return {
        "q": q, "k": k, "v": v, "q_w": torch.rand(d, generator=gen) + 0.5, "k_w": torch.rand(d, generator=gen) + 0.5,
        "W": torch.randn((Hkv * d, Hkv), generator=gen) * 0.02, "A": -(torch.rand(Hkv, generator=gen) * 1.9 + 0.1),
        "cu": torch.tensor([0] + list(news)).cumsum(0).add(lead).to(torch.int32),
        "positions": torch.tensor(positions, dtype=torch.int32), "table": table,
        "k_pages": randn_bf16((n_pages, page, Hkv, d), gen), "v_pages": randn_bf16((n_pages, page, Hkv, d), gen),
        "dt_pages": torch.rand((n_pages, Hkv, page), generator=gen) + 5.0,
    }


def on_gpu(x):
    if x["q"].storage_offset() == 0 and x["q"].stride(0) != x["q"].shape[1] * x["q"].shape[2]:
        heads = [x[n].shape[1] for n in "qkv"]
        whole = torch.cat([x["q"], x["k"], x["v"]], 1).cuda()
        g = dict(zip("qkv", torch.split(whole, heads, 1)))
    else:
        g = {n: x[n].cuda() for n in "qkv"}
    return {**{n: t.cuda() for n, t in x.items() if n not in "qkv"}, **g}


def run_append(dma, x, g, theta=10000.0, with_k=True, **kw):
    T, Hq, d = x["q"].shape
    q_out = torch.full((T, Hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full(x["k"].shape, 77.0, dtype=torch.bfloat16, device="cuda") if with_k else None
    ws = dma.new_workspace(256)
    r = dma.dma_append_paged(g["q"], g["k"], g["v"], g["q_w"], g["k_w"], g["W"], g["A"], g["cu"], g["positions"],
                             g["table"], g["k_pages"], g["v_pages"], g["dt_pages"], rope_theta=theta, q_out=q_out,
                             k_out=k_out, workspace=ws, **kw)
    assert r is q_out
    return q_out, k_out, dma.dma_check(ws)


def check_append(x, g, q_out, k_out, theta=10000.0):
    args = [f64(x[n]) for n in ("q", "k", "v", "q_w", "k_w")]
    W, A = x["W"].double().numpy(), x["A"].double().numpy()
    wq, wk, wkp, wvp, wdp = oracle.append_paged(*args, 1e-6, theta, W, A, x["cu"].numpy(), x["positions"].numpy(),
                                                x["table"].numpy(), f64(x["k_pages"]), f64(x["v_pages"]),
                                                f64(x["dt_pages"]))
    mine = ~np.isnan(wq[:, 0, 0])                     # tokens that belong to a sequence
    for got, want, what in ((q_out, wq, "q_out"), (k_out, wk, "k_out")):
        if got is not None:
            assert_close(f64(got)[mine], want[mine], BF16, 2e-5, what)
            assert (f64(got)[~mine] == 77.0).all(), what + ": rows of no sequence were written"
    written = np.zeros(wkp.shape[:2], bool)
    page = wkp.shape[1]
    cu, pos, table = (x[n].numpy() for n in ("cu", "positions", "table"))
    S = np.zeros(wdp.shape)
    for b in range(len(pos)):
        for t in range(cu[b], cu[b + 1]):
            j = pos[b] + t - cu[b]
            at = table[b][j // page], j % page
            written[at] = True
            S[at[0], :, at[1]] = np.abs(f64(x["v"][t])).reshape(-1) @ np.abs(W)
    assert_close(f64(g["k_pages"])[written], wkp[written], BF16, 2e-5, "k_pages")
    for n in ("k_pages", "v_pages"):                  # every other row untouched, bit for bit
        assert torch.equal(g[n].cpu().view(torch.int16)[~written], x[n].view(torch.int16)[~written]), n
    assert np.array_equal(f64(g["v_pages"])[written], wvp[written])
    w3 = np.broadcast_to(written[:, None, :], wdp.shape)
    got = f64(g["dt_pages"])
    assert np.array_equal(got[~w3], wdp[~w3])
    tol = wdp * (np.abs(A)[None, :, None] * 40 * 2.0 ** -23 * S + (np.abs(np.log(wdp)) + 4) * 2.0 ** -22)
    assert (np.abs(got - wdp) <= tol)[w3].all(), "dt: max err %.3e" % np.abs(got - wdp)[w3].max()


@pytest.mark.parametrize("news,positions,Hq,Hkv,d,page,kw", [
    ([1], [0], 8, 4, 64, 16, {}),                                       # one token, the first of a sequence
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 40], 8, 4, 64, 16, {"pad": 3}),   # a decode step in a padded batch
    ([37, 0, 1, 64], [5, 3, 0, 100], 16, 8, 128, 16, {"fused": True}),  # prompts and single tokens, one sequence idle
    ([3, 40], [7, 0], 3, 1, 128, 5, {"lead": 2, "pad": 1}),             # pages of five, tokens before the first sequence
    ([19], [2], 16, 16, 128, 1, {}),                                    # pages of one token, sixteen kv heads
    ([23, 9], [0, 31], 16, 2, 64, 100, {"fused": True}),                # eight query heads per kv head
    ([11], [0], 1, 1, 64, 8, {}),                                       # one head of each
    ([9, 8], [1, 2], 32, 16, 64, 24, {}),
    ([2, 5], [131000, 90001], 4, 2, 128, 64, {}),                       # far positions: angles need double precision
    ([700], [3], 4, 4, 64, 32, {"fused": True}),
])
def test_append_matches_oracle(dma, news, positions, Hq, Hkv, d, page, kw):
    x = append_inputs(news, positions, Hq, Hkv, d, page, seed=len(news) * 100 + page, **kw)
    g = on_gpu(x)
    q_out, k_out, status = run_append(dma, x, g, theta=500000.0 if max(positions) > 60000 else 10000.0)
    assert status == 0
    check_append(x, g, q_out, k_out, theta=500000.0 if max(positions) > 60000 else 10000.0)


def test_append_more_sequences_than_the_staged_offsets(dma):
    news = [(i * 7) % 4 for i in range(1500)]
    x = append_inputs(news, [i % 23 for i in range(1500)], 2, 1, 64, 8, seed=9)
    g = on_gpu(x)
    q_out, _, status = run_append(dma, x, g, with_k=False)
    assert status == 0
    check_append(x, g, q_out, None)


def test_append_many_tokens_sampled(dma):
    """More tokens than resident warps, so every block takes several tiles; sampled tokens against the oracle."""
    x = append_inputs([5000, 4001], [0, 77], 16, 8, 128, 64, fused=True, seed=4)
    g = on_gpu(x)
    before = {n: g[n].clone() for n in ("k_pages", "v_pages", "dt_pages")}
    q_out, k_out, status = run_append(dma, x, g)
    assert status == 0
    toks = np.unique(np.concatenate([[0, 1, 4999, 5000, 9000], np.random.default_rng(0).integers(0, 9001, 40)]))
    cu, pos = x["cu"].tolist(), x["positions"].tolist()
    W, A = x["W"].double().numpy(), x["A"].double().numpy()
    for t in toks:
        b = 0 if t < cu[1] else 1
        j = pos[b] + int(t) - cu[b]
        one = {n: f64(x[n][t:t + 1]) for n in "qkv"}
        z = np.zeros
        wq, wk, _, _, wd = oracle.append_paged(one["q"], one["k"], one["v"], f64(x["q_w"]), f64(x["k_w"]), 1e-6,
                                               10000.0, W, A, [0, 1], [j], np.zeros((1, j + 1), int),
                                               z((1, 1, 8, 128)), z((1, 1, 8, 128)), z((1, 8, 1)))
        page, off = int(x["table"][b, j // 64]), j % 64
        assert_close(f64(q_out[t]), wq[0], BF16, 2e-5, "q")
        assert_close(f64(k_out[t]), wk[0], BF16, 2e-5, "k_out")
        assert torch.equal(g["k_pages"][page, off], k_out[t])
        assert torch.equal(g["v_pages"][page, off].cpu(), x["v"][t])
        assert_close(f64(g["dt_pages"][page, :, off]), wd[0, :, 0], 4e-5, 0.0, "dt")
    for n in before:                                   # rows no token went to
        rows = torch.ones(before[n].shape[0], before["k_pages"].shape[1], dtype=torch.bool)
        for b in range(2):
            j = torch.arange(pos[b], pos[b] + cu[b + 1] - cu[b])
            rows[x["table"][b].long()[j // 64], j % 64] = False
        rows = rows.cuda()
        if n == "dt_pages":
            assert torch.equal(g[n].transpose(1, 2)[rows], before[n].transpose(1, 2)[rows])
        else:
            assert torch.equal(g[n][rows], before[n][rows])


def test_append_agrees_with_the_contiguous_prologue(dma):
    """Same rows as dma_prologue for equal lengths, the cache being pages of one sequence each."""
    B, L, Lmax, Hq, Hkv, d = 3, 21, 64, 8, 4, 64
    x = append_inputs([L] * B, [4, 0, 43], Hq, Hkv, d, Lmax, seed=2, max_pages=1)
    g = on_gpu(x)
    q_out, k_out, status = run_append(dma, x, g)
    assert status == 0
    kc = torch.zeros((B, Lmax, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    shape = lambda t: t.reshape(B, L, t.shape[1], d).contiguous()
    want = dma.dma_prologue(shape(g["q"]), shape(g["k"]), shape(g["v"]), g["q_w"], g["k_w"], g["positions"], kc, vc)
    assert_close(f64(q_out.view_as(want)), f64(want), 2 * BF16, 4e-5, "q")       # each within its own rounding
    for b in range(B):
        p, n = int(x["positions"][b]), int(x["table"][b, 0])
        assert torch.equal(g["v_pages"][n, p:p + L], vc[b, p:p + L])
        assert_close(f64(g["k_pages"][n, p:p + L]), f64(kc[b, p:p + L]), 2 * BF16, 4e-5, "k")


def test_append_reports_bad_positions_and_pages(dma):
    x = append_inputs([4, 4, 2], [28, 0, 1], 4, 2, 64, 16, seed=6, max_pages=2)     # sequence 0 fits exactly
    g = on_gpu(x)
    g["positions"][0] = 30                       # its last two tokens fall past the table
    before = {n: g[n].clone() for n in ("k_pages", "v_pages", "dt_pages")}
    q_out, k_out, status = run_append(dma, x, g)
    assert dma.STATUS[status] == "DMA_ERR_BAD_POSITION"
    page0 = int(x["table"][0, 1])
    assert not torch.equal(g["v_pages"][page0, 14:], before["v_pages"][page0, 14:])
    assert torch.equal(g["v_pages"][page0, 14:16].cpu(), x["v"][:2])
    assert (f64(q_out) != 77.0).all()            # q rows are written all the same
    for bad in (-1, g["k_pages"].shape[0], 2 ** 31 - 1):
        g = on_gpu(x)
        g["table"][1, 0] = bad
        q_out, k_out, status = run_append(dma, x, g)
        assert dma.STATUS[status] == "DMA_ERR_BAD_PAGE"
        used = [int(x["table"][0, 1]), int(x["table"][2, 0])]
        others = [n for n in range(g["k_pages"].shape[0]) if n not in used]
        for n in before:
            assert torch.equal(g[n][others].cpu(), x[n][others])
        assert (f64(k_out) != 77.0).all()
    g = on_gpu(x)
    g["positions"][2] = -1                       # one of its tokens before the sequence's start
    _, _, status = run_append(dma, x, g)
    assert dma.STATUS[status] == "DMA_ERR_BAD_POSITION"
    assert torch.equal(g["v_pages"][int(x["table"][2, 0]), 0].cpu(), x["v"][9])


# ---- decode -------------------------------------------------------------------------

def decode_inputs(lens, Hq, Hkv, d, page, seed=0, cap=None, dt="random", garbage=True, interleaved=False):
    gen = torch.Generator().manual_seed(seed)
    max_pages = -(-max(cap or max(lens), 1) // page)
    table, n = page_table([-(-k // page) for k in lens], max_pages, gen)
    pool = (n, 2, page, Hkv, d) if interleaved else (2, n, page, Hkv, d)
    kv = randn_bf16(pool, gen)
    k, v = (kv[:, 0], kv[:, 1]) if interleaved else (kv[0], kv[1])
    x = torch.randn((n, Hkv, page), generator=gen) * 0.64
    A = -(torch.rand(Hkv, generator=gen) * 1.9 + 0.1)
    dtp = torch.exp(A[:, None] * torch.nn.functional.softplus(x))
    if dt == "ones":
        dtp = torch.ones_like(dtp)
    if dt == "few":                                       # four values: ties at every threshold
        dtp = torch.randint(1, 5, dtp.shape, generator=gen).float() / 4
    if dt == "outlier":                                   # one key far above, many zeros
        dtp = torch.where(torch.rand(dtp.shape, generator=gen) < 0.9, torch.zeros(()), dtp * 1e-3)
        dtp[table[0, 0], :, 0] = 3.0
    if dt in ("rising", "falling"):                       # the best keys all lie together
        for b, k_len in enumerate(lens):
            j = torch.arange(-(-k_len // page) * page).float()
            r = 0.1 + 0.8 * (j if dt == "rising" else j.flip(0)) / max(1, j.numel())
            dtp[table[b, :j.numel() // page].long()] = r.view(-1, 1, page).expand(-1, Hkv, -1).clone()
    if garbage:                                           # rows past the lengths and pages of nobody
        used = torch.zeros((n, page), dtype=torch.bool)
        for b, k_len in enumerate(lens):
            j = torch.arange(k_len)
            used[table[b].long()[j // page], j % page] = True
        k[~used], v[~used] = float("nan"), float("inf")
        dtp = torch.where(used[:, None], dtp, torch.tensor(float("nan")))
    return {"q": randn_bf16((len(lens), Hq, d), gen), "kv": kv, "k": k, "v": v, "dt": dtp, "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32), "interleaved": interleaved}


def decode_gpu(x):
    g = {n: x[n].cuda() for n in ("q", "kv", "dt", "table", "lens")}
    g["k"], g["v"] = (g["kv"][:, 0], g["kv"][:, 1]) if x["interleaved"] else (g["kv"][0], g["kv"][1])
    return g


def run_decode(dma, g, w, window=0, sinks=0, **kw):
    B, Hq, d = g["q"].shape
    _, page, Hkv, _ = g["k"].shape
    ws = dma.new_workspace(dma.dma_decode_paged_workspace_size(B, g["table"].shape[1], page, Hq, Hkv, d, w, window, sinks))
    out = torch.full((B, Hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
    dma.dma_decode_paged(g["q"], g["k"], g["v"], g["dt"], g["table"], g["lens"], w, window=window, sinks=sinks,
                         out=out, workspace=ws, **kw)
    return out, ws


def check_lists(dma, x, ws, w, window, sinks):
    """The kept lists of rows that see more than w keys: exactly the w best, each once."""
    B, Hq, d = x["q"].shape
    _, page, Hkv, _ = x["k"].shape
    pos, bias = (t.cpu().numpy() for t in dma.paged_list_views(ws, B, Hq, Hkv, d, w))
    for b in range(B):
        j = np.array(oracle.visible_positions(int(x["lens"][b]), window, sinks), dtype=np.int64)
        if len(j) <= w:
            continue
        pg, off = x["table"][b].numpy()[j // page].astype(np.int64), j % page
        for h in range(Hkv):
            dt = x["dt"].numpy()[pg, h, off]
            best = np.sort(np.argsort(-dt, kind="stable")[:w])
            got = np.argsort(pos[b, h])
            assert np.array_equal(pos[b, h][got], j[best]), f"kept set of sequence {b}, kv head {h}"
            assert np.array_equal(bias[b, h][got], dt[best])


def check_decode(x, out, w, window, sinks, scale=None):
    d = x["q"].shape[2]
    clean = lambda t: np.nan_to_num(f64(t), nan=0.0, posinf=0.0)
    want = oracle.decode_paged(f64(x["q"]), clean(x["k"]), clean(x["v"]), np.nan_to_num(x["dt"].numpy()),
                               x["table"].numpy(), x["lens"].numpy(), w, window, sinks, d ** -0.5 if scale is None else scale)
    assert_close(out, want, BF16, DECODE_ATOL, "out")


@pytest.mark.parametrize("lens,w,window,sinks,Hq,Hkv,d,page,kw", [
    ([1], 2048, 0, 0, 8, 4, 64, 16, {}),
    ([0, 1, 2, 15, 16, 17, 33], 2048, 0, 0, 8, 4, 64, 16, {}),              # an empty slot; pages that end in a tile
    ([300, 0, 7, 129], 64, 0, 0, 16, 8, 128, 16, {}),                       # kept lists for some, not for others
    ([100, 5, 64], 2048, 0, 0, 3, 1, 128, 5, {}),                           # pages of five, three heads a group
    ([40, 41], 2048, 0, 0, 16, 16, 64, 1, {}),                              # pages of one
    ([513, 200], 100, 0, 0, 5, 1, 64, 7, {}),                               # odd pages with a kept list
    ([130, 70, 1], 33, 0, 0, 16, 2, 128, 100, {}),                          # eight heads a group
    ([3000], 1, 0, 0, 4, 2, 64, 64, {}),                                    # one kept key
    ([3000, 2500], 2499, 0, 0, 4, 2, 64, 64, {}),                           # nearly all kept
    ([700, 90, 64, 0, 3], 2048, 64, 4, 8, 4, 64, 16, {}),                   # window and sinks, fewer keys than them
    ([700, 91, 12], 40, 100, 7, 8, 4, 128, 8, {}),                          # ... of which the best are kept
    ([700, 64], 2048, 1, 0, 8, 4, 64, 16, {}),                              # a window of one key
    ([900, 80], 50, 75, 1000, 8, 4, 64, 5, {}),                             # more sinks than keys
    ([900], 10, 2 ** 30, 2 ** 30, 8, 4, 64, 32, {}),                        # a window beyond every length
    ([5000, 100], 512, 0, 0, 8, 4, 64, 16, {"cap": 9000}),                  # a table longer than any sequence
    ([400, 33], 128, 0, 0, 6, 2, 64, 16, {"interleaved": True}),            # K and V pages in one block
    ([6000], 2048, 0, 0, 2, 1, 64, 64, {"dt": "ones"}),                     # a model at its start: all dt equal
    ([6000, 2500], 600, 0, 0, 4, 2, 64, 16, {"dt": "few"}),
    ([9000], 600, 0, 0, 4, 2, 64, 16, {"dt": "outlier"}),
    ([9000, 70], 700, 0, 0, 2, 2, 64, 16, {"dt": "rising"}),
    ([9000], 700, 0, 0, 2, 2, 128, 20, {"dt": "falling"}),
    ([12000], 9000, 0, 0, 2, 1, 64, 16, {}),                                # a kept list beyond the collection's buffers
])
def test_decode_matches_oracle(dma, lens, w, window, sinks, Hq, Hkv, d, page, kw):
    x = decode_inputs(lens, Hq, Hkv, d, page, seed=sum(lens) + w, **kw)
    g = decode_gpu(x)
    out, ws = run_decode(dma, g, w, window, sinks)
    assert dma.dma_check(ws) == 0
    if (min(g["table"].shape[1] * page, window + sinks) if window else g["table"].shape[1] * page) > w:
        check_lists(dma, x, ws, w, window, sinks)
    check_decode(x, out, w, window, sinks)
    again, _ = run_decode(dma, g, w, window, sinks)
    assert torch.equal(out, again)                     # the same call, the same bits


@pytest.mark.parametrize("n,w,Hkv,dt", [(70001, 2048, 1, "random"), (70001, 2048, 2, "ones"), (300000, 500, 4, "random"),
                                        (66000, 300, 8, "rising")])
def test_decode_long_rows_split_over_a_cluster(dma, n, w, Hkv, dt):
    x = decode_inputs([n], 2 * Hkv, Hkv, 64, 64, seed=n + w, dt=dt, garbage=False)
    g = decode_gpu(x)
    out, ws = run_decode(dma, g, w)
    assert dma.dma_check(ws) == 0
    check_lists(dma, x, ws, w, 0, 0)
    check_decode(x, out, w, 0, 0)


def dt_pattern(kind, n, Hkv, gen):
    """dt of n consecutive keys: [n, Hkv]."""
    r = torch.rand((n, Hkv), generator=gen)
    part = torch.rand((n, Hkv), generator=gen)
    if kind == "half tied":                     # one value among others, above and below it
        return torch.where(part < 0.5, torch.full_like(r, 0.75), r)
    if kind == "tied under a few":              # all but one key in a hundred hold one value
        return torch.where(part < 0.01, 0.5 + r, torch.full_like(r, 0.25))
    if kind == "zeros":                         # most keys hold nothing
        return torch.where(part < 0.99, torch.zeros(()), r)
    if kind == "neighbours":                    # two values one bit apart
        return torch.where(part < 0.5, torch.tensor(0.5), torch.nextafter(torch.tensor(0.5), torch.tensor(1.0)))
    if kind == "tied at the end":               # the tied keys that count lie in the last ones
        tied = torch.full((n, 1), 0.125).expand(n, Hkv).clone()
        tied[-n // 50:] = 0.5
        return tied
    if kind == "lumps":                         # the best keys in random runs of four
        lump = torch.rand((-(-n // 4), Hkv), generator=gen).repeat_interleave(4, 0)[:n]
        return 0.01 * r + lump
    assert kind == "one lane"                   # ... in every 32nd run of eight
    return torch.where(((torch.arange(n) // 8) % 32 == 5)[:, None], 0.9 + 0.1 * r, 0.5 * r)


@pytest.mark.parametrize("n,w,window,sinks,Hkv,page", [
    (9001, 600, 0, 0, 2, 16),
    (9001, 600, 8000, 13, 2, 16),               # ... under a window with sinks
    (9001, 600, 8000, 13, 2, 5),                # pages that runs of eight cross
    (60000, 2048, 0, 0, 1, 64),                 # a cluster per row
    (60000, 2048, 50000, 100, 4, 20),
])
@pytest.mark.parametrize("kind", ["half tied", "tied under a few", "zeros", "neighbours", "tied at the end", "lumps", "one lane"])
def test_decode_selection_of_hard_rows(dma, n, w, window, sinks, Hkv, page, kind):
    x = decode_inputs([n, n - 7], Hkv, Hkv, 64, page, seed=n + Hkv, garbage=False)
    gen = torch.Generator().manual_seed(n + w)
    for b in range(2):
        j = torch.arange(int(x["lens"][b]))
        x["dt"][x["table"][b].long()[j // page], :, j % page] = dt_pattern(kind, len(j), Hkv, gen)
    g = decode_gpu(x)
    out, ws = run_decode(dma, g, w, window, sinks)
    assert dma.dma_check(ws) == 0
    check_lists(dma, x, ws, w, window, sinks)
    check_decode(x, out, w, window, sinks)
    again, _ = run_decode(dma, g, w, window, sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("w,kind", [(2048, "lumps"), (2048, "half tied"), (8000, "lumps"), (8000, "zeros"), (8000, "one lane")])
def test_decode_selection_of_many_rows(dma, w, kind):
    """More rows than SMs, so that a row has one CTA, or a few for the lists of a large window."""
    lens = [12000, 11111] + [9] * 90 + [w + 1, w, 12000]
    x = decode_inputs(lens, 2, 2, 64, 16, seed=w, garbage=False)
    gen = torch.Generator().manual_seed(w)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        x["dt"][x["table"][b].long()[j // 16], :, j % 16] = dt_pattern(kind, n, 2, gen)
    g = decode_gpu(x)
    out, ws = run_decode(dma, g, w)
    assert dma.dma_check(ws) == 0
    check_lists(dma, x, ws, w, 0, 0)
    check_decode(x, out, w, 0, 0)


@pytest.mark.parametrize("d,lens,w", [(64, [700, 3, 90, 4000], 2048), (128, [2500, 0, 31], 300), (64, [9000], 64)])
def test_workspace_that_held_something_else(dma, d, lens, w):
    """Only the header has to be zero: entry points share a workspace, whatever they left behind it."""
    x = decode_inputs(lens, 8, 4, d, 16, seed=d + w, garbage=False)
    g = decode_gpu(x)
    want, _ = run_decode(dma, g, w)
    size = dma.dma_decode_paged_workspace_size(len(lens), g["table"].shape[1], 16, 8, 4, d, w)
    ws = dma.new_workspace(max(size, dma.dma_prologue_backward_workspace_size(2, 40, 8, 4, d)))
    q, k = (torch.randn((2, 40, h, d), device="cuda").bfloat16() for h in (8, 4))
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    one = torch.ones(d, device="cuda")
    back = lambda ws=None: dma.dma_prologue_backward(q, k, one, one, torch.zeros(2, dtype=torch.int32, device="cuda"), dq,
                                                     dk, workspace=ws)
    grads = back()
    for fill in (0xFF, 0x01, None):
        if fill is not None:
            ws[256:] = fill
        for _ in range(2):
            out = dma.dma_decode_paged(g["q"], g["k"], g["v"], g["dt"], g["table"], g["lens"], w, workspace=ws)
            assert torch.equal(out, want)
            assert not ws[:256].any()
            for a, b in zip(back(ws), grads):
                assert torch.equal(a, b)
            assert not ws[:256].any()


def test_decode_long_row_kept_whole(dma):
    x = decode_inputs([40000, 3], 4, 2, 64, 16, seed=3, garbage=False)
    out, _ = run_decode(dma, decode_gpu(x), 1 << 20)
    check_decode(x, out, 1 << 20, 0, 0)


def test_decode_more_sequences_than_a_scan_step(dma):
    lens = [(i * 37) % 61 for i in range(600)]
    x = decode_inputs(lens, 2, 1, 64, 16, seed=1)
    out, _ = run_decode(dma, decode_gpu(x), 32)
    check_decode(x, out, 32, 0, 0)


@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_decode_scales(dma, scale):
    x = decode_inputs([200, 31], 4, 2, 64, 16, seed=8)
    out, _ = run_decode(dma, decode_gpu(x), 2048, scale=scale)
    # the scores' float32 error grows with the scale: 1e-5 at the usual 1/8
    d = x["q"].shape[2]
    want = oracle.decode_paged(f64(x["q"]), np.nan_to_num(f64(x["k"])), np.nan_to_num(f64(x["v"]), posinf=0.0),
                               np.nan_to_num(x["dt"].numpy()), x["table"].numpy(), x["lens"].numpy(), 2048, 0, 0, scale)
    assert_close(out, want, BF16, DECODE_ATOL * max(1.0, abs(scale) * d ** 0.5), "out")


def test_decode_reports_bad_lengths_and_pages(dma):
    x = decode_inputs([40, 50, 60], 4, 2, 64, 16, seed=5, garbage=False)
    g = decode_gpu(x)
    g["lens"][0], g["lens"][1] = -3, 10 ** 6            # clamped to 0 and to the table's 64 positions
    g["table"][1, 3] = 0
    out, ws = run_decode(dma, g, 2048)
    assert dma.STATUS[dma.dma_check(ws)] == "DMA_ERR_BAD_LENGTH"
    y = dict(x, lens=torch.tensor([0, 64, 60], dtype=torch.int32), table=g["table"].cpu())
    check_decode(y, out, 2048, 0, 0)
    for w in (2048, 20):
        for bad in (-1, g["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
            g = decode_gpu(x)
            g["table"][2, 1] = bad                      # keys 16..31 of sequence 2 are not seen
            out, ws = run_decode(dma, g, w)
            assert dma.STATUS[dma.dma_check(ws)] == "DMA_ERR_BAD_PAGE"
            keep = [j for j in range(60) if not 16 <= j < 32]
            pg = x["table"][2].long()[torch.tensor(keep) // 16]
            off = torch.tensor(keep) % 16
            k, v, dt = x["k"][pg, off][None], x["v"][pg, off][None], x["dt"][pg, :, off].T[None]
            want = oracle.decode_step(f64(x["q"][2:]), f64(k), f64(v), None, None, [len(keep)], w, 0.125, dt=dt.numpy())
            assert_close(out[2:], want, BF16, DECODE_ATOL, "out")


def test_decode_row_whose_pages_are_all_bad(dma):
    x = decode_inputs([40, 50], 4, 2, 64, 16, seed=5, garbage=False)
    for w in (2048, 20):
        g = decode_gpu(x)
        g["table"][1] = -1
        out, ws = run_decode(dma, g, w)
        assert dma.STATUS[dma.dma_check(ws)] == "DMA_ERR_BAD_PAGE"
        assert (out[1] == 0).all()


def test_decode_offsets_past_32_bits(dma):
    """A pool of more than 2^32 elements, the sequence's pages at its far end."""
    page, Hkv, d, n = 64, 8, 128, 66000                 # 4.3e9 elements in each pool
    gen = torch.Generator().manual_seed(0)
    k = torch.empty((n, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    dt = torch.empty((n, Hkv, page), device="cuda")
    tail = 4
    kt, vt = randn_bf16((tail, page, Hkv, d), gen), randn_bf16((tail, page, Hkv, d), gen)
    dtt = torch.rand((tail, Hkv, page), generator=gen)
    k[-tail:], v[-tail:], dt[-tail:] = kt.cuda(), vt.cuda(), dtt.cuda()
    table = torch.arange(n - 1, n - 1 - tail, -1, dtype=torch.int32)[None]
    x = {"q": randn_bf16((1, 16, d), gen), "k": kt, "v": vt, "dt": dtt, "lens": torch.tensor([200], dtype=torch.int32),
         "table": table - (n - tail)}
    for w in (2048, 70):
        g = {"q": x["q"].cuda(), "k": k, "v": v, "dt": dt, "table": table.cuda(), "lens": x["lens"].cuda()}
        out, ws = run_decode(dma, g, w)
        assert dma.dma_check(ws) == 0
        check_decode(x, out, w, 0, 0)
    a = append_inputs([30], [220], 16, Hkv, d, page, seed=1, max_pages=4)
    ga = on_gpu(a)
    ga.update(k_pages=k, v_pages=v, dt_pages=dt, table=table.cuda())
    _, k_out, status = run_append(dma, a, ga)
    assert status == 0
    for t in (0, 29):
        j = 220 + t
        assert torch.equal(k[int(table[0, j // page]), j % page], k_out[t])
        assert torch.equal(v[int(table[0, j // page]), j % page].cpu(), a["v"][t])


def test_binding_names_what_is_wrong(dma):
    """Arguments that do not fit are refused with their name before anything is launched."""
    x = append_inputs([3], [0], 4, 2, 64, 8)
    g = on_gpu(x)
    q_out = torch.full((3, 4, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    names = ["q", "k", "v", "q_w", "k_w", "W", "A", "cu", "positions", "table", "k_pages", "v_pages", "dt_pages"]
    wrong = {"k": g["k"].float(), "v": g["v"][:2], "q_w": g["q_w"][:32], "W": g["W"].T, "A": g["A"].double(),
             "cu": g["cu"].long(), "positions": torch.cat([g["positions"]] * 2), "table": g["table"].long(),
             "k_pages": g["k_pages"].transpose(1, 2), "v_pages": g["v_pages"].half(), "dt_pages": g["dt_pages"].transpose(1, 2),
             "q": g["q"].transpose(1, 2)}
    for name, t in wrong.items():
        with pytest.raises(ValueError):
            dma.dma_append_paged(*[t if n == name else g[n] for n in names], q_out=q_out)
    with pytest.raises(ValueError, match="workspace|must be"):
        dma.dma_append_paged(*[g[n] for n in names], q_out=q_out, workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(dma.DMAError, match="WORKSPACE"):
        dma.dma_append_paged(*[g[n] for n in names], q_out=q_out, workspace=dma.new_workspace(128))
    assert (q_out == 77.0).all()
    y = decode_inputs([40], 4, 2, 64, 16, garbage=False)
    h = decode_gpu(y)
    call = lambda w=2048, **kw: dma.dma_decode_paged(h["q"], kw.pop("k", h["k"]), h["v"], h["dt"], kw.pop("table", h["table"]),
                                                     h["lens"], w, **kw)
    for bad in (dict(w=2 ** 32 + 5), dict(window=2 ** 32 + 5), dict(sinks=2 ** 33), dict(k=h["k"][:, :8]),
                dict(table=h["table"].long()), dict(out=torch.zeros((1, 4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=1e300)):
        with pytest.raises((ValueError, dma.DMAError)):
            call(**bad)
    check_decode(y, call(), 2048, 0, 0)


# ---- streams, graphs, the run together -------------------------------------------------

def test_decode_in_a_graph_follows_its_inputs(dma):
    """Captured once, replayed with other lengths, tables and queries; two graphs on one workspace, one after the other."""
    x = decode_inputs([90, 700, 0], 8, 4, 64, 16, seed=11, garbage=False, cap=1024)
    y = decode_inputs([1, 0, 1000], 8, 4, 64, 16, seed=12, garbage=False, cap=1024)
    n = max(x["k"].shape[0], y["k"].shape[0])
    g = decode_gpu(x)
    for name in ("k", "v", "dt"):
        g[name] = torch.zeros((n,) + tuple(x[name].shape[1:]), dtype=x[name].dtype, device="cuda")
    size = max(dma.dma_decode_paged_workspace_size(3, 64, 16, 8, 4, 64, w, 0, 0) for w in (2048, 100))
    ws = dma.new_workspace(size)
    outs = [torch.zeros((3, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    for w, out in zip((2048, 100), outs):
        call = lambda: dma.dma_decode_paged(g["q"], g["k"], g["v"], g["dt"], g["table"], g["lens"], w, out=out, workspace=ws)
        with torch.cuda.stream(side):
            g["lens"].zero_()
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for z in (x, y, x):
        for name in ("k", "v", "dt"):
            g[name][:z[name].shape[0]] = z[name].cuda()
        for name in ("q", "table", "lens"):
            g[name].copy_(z[name].cuda())
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        check_decode(z, outs[0], 2048, 0, 0)
        check_decode(z, outs[1], 100, 0, 0)


def test_calls_on_another_stream(dma):
    """`stream=` runs everything there, what the binding allocates included, behind that stream's earlier work."""
    s = torch.cuda.Stream()
    x = decode_inputs([500, 77], 8, 4, 64, 16, seed=21, garbage=False)
    g = decode_gpu(x)
    late = {n: torch.zeros_like(g[n]) for n in ("q", "dt")}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
        for n in late:
            late[n].copy_(g[n], non_blocking=True)
    out = dma.dma_decode_paged(late["q"], g["k"], g["v"], late["dt"], g["table"], g["lens"], 100, stream=s)
    s.synchronize()
    check_decode(x, out, 100, 0, 0)


def test_append_and_decode_in_one_graph(dma):
    """A serving step captured once: packed tokens of other sequences, positions and padding on every replay."""
    Hq, Hkv, d, page, T, B = 8, 4, 64, 16, 12, 4
    runs = [([1, 1, 1, 1], [0, 15, 40, 63]), ([3, 0, 1, 8], [2, 9, 79, 16]), ([0, 0, 0, 1], [1, 2, 3, 0])]
    xs = [append_inputs(n, p, Hq, Hkv, d, page, pad=T - sum(n), seed=i, max_pages=5) for i, (n, p) in enumerate(runs)]
    n_pages = max(x["k_pages"].shape[0] for x in xs)
    g = on_gpu(xs[0])
    for n in ("k_pages", "v_pages", "dt_pages"):
        g[n] = torch.zeros((n_pages,) + tuple(xs[0][n].shape[1:]), dtype=xs[0][n].dtype, device="cuda")
    lens, last = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    q_out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    rows, out = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    ws = dma.new_workspace(dma.dma_decode_paged_workspace_size(B, 5, page, Hq, Hkv, d, 20))

    def step():
        dma.dma_append_paged(g["q"], g["k"], g["v"], g["q_w"], g["k_w"], g["W"], g["A"], g["cu"], g["positions"],
                             g["table"], g["k_pages"], g["v_pages"], g["dt_pages"], q_out=q_out, workspace=ws)
        torch.index_select(q_out, 0, last, out=rows)
        dma.dma_decode_paged(rows, g["k_pages"], g["v_pages"], g["dt_pages"], g["table"], lens, 20, out=out, workspace=ws)

    g["cu"].zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 2, 0):
        x, (news, positions) = xs[i], runs[i]
        q_out.fill_(77.0)
        for n in ("q", "k", "v", "q_w", "k_w", "W", "A", "cu", "positions", "table"):
            g[n].copy_(x[n].cuda())
        for n in ("k_pages", "v_pages", "dt_pages"):
            g[n][:x[n].shape[0]] = x[n].cuda()
        lens.copy_(torch.tensor([p + n if n else 0 for n, p in zip(news, positions)], dtype=torch.int32))
        last.copy_((x["cu"][1:] - 1).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        assert dma.dma_check(ws) == 0
        pools = {n: g[n][:x[n].shape[0]].clone() for n in ("k_pages", "v_pages", "dt_pages")}
        check_append(x, pools, q_out, None)
        state = {"q": rows.cpu(), "k": pools["k_pages"].cpu(), "v": pools["v_pages"].cpu(), "dt": pools["dt_pages"].cpu(),
                 "table": x["table"], "lens": lens.cpu()}
        check_decode(state, out, 20, 0, 0)


def test_two_decodes_at_once(dma):
    """Calls on two streams, each with its own workspace, over the same pages."""
    x = decode_inputs([9000, 70, 3000], 8, 4, 64, 16, seed=41, garbage=False)
    g = decode_gpu(x)
    want = {w: run_decode(dma, g, w)[0] for w in (300, 2048)}
    streams = {w: torch.cuda.Stream() for w in want}
    ws = {w: dma.new_workspace(dma.dma_decode_paged_workspace_size(3, g["table"].shape[1], 16, 8, 4, 64, w)) for w in want}
    torch.cuda.synchronize()
    got = {w: [] for w in want}
    for _ in range(20):
        for w in want:
            got[w].append(dma.dma_decode_paged(g["q"], g["k"], g["v"], g["dt"], g["table"], g["lens"], w, workspace=ws[w],
                                               stream=streams[w]))
    torch.cuda.synchronize()
    for w in want:
        for out in got[w]:
            assert torch.equal(out, want[w])


def test_prompt_then_decode_steps(dma):
    """A user's run: prompts enter the pages (and prefill reads their rotated keys), then single tokens are appended
    and decoded; every decode output against the oracle over what the pages hold, the first also against the
    prefill's row for the same token."""
    Hq, Hkv, d, page, w = 8, 4, 64, 16, 48
    prompts, steps = [70, 33], 4
    B = len(prompts)
    gen = torch.Generator().manual_seed(31)
    total = [p + steps for p in prompts]
    x = append_inputs(total, [0] * B, Hq, Hkv, d, page, seed=31)
    cu = x["cu"].tolist()
    table, n = x["table"].cuda(), x["k_pages"].shape[0]
    kp = torch.full((n, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp, dp = torch.full_like(kp, float("nan")), torch.full((n, Hkv, page), float("nan"), device="cuda")
    wts = [x[m].cuda() for m in ("q_w", "k_w", "W", "A")]
    take = lambda lo, hi: [torch.cat([x[m][cu[b] + lo[b]:cu[b] + hi[b]] for b in range(B)]).cuda() for m in "qkv"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ws = dma.new_workspace(dma.dma_decode_paged_workspace_size(B, table.shape[1], page, Hq, Hkv, d, w))
    # all but the last token of each prompt, then the last one as the first decode step
    q, k, v = take([0] * B, [p - 1 for p in prompts])
    k_out = torch.empty_like(k)
    lens = [p - 1 for p in prompts]
    dma.dma_append_paged(q, k, v, *wts, i32([0] + lens).cumsum(0).to(torch.int32), i32([0] * B), table, kp, vp, dp,
                         k_out=k_out, workspace=ws)
    for step in range(steps + 1):
        q, k, v = take(lens, [n + 1 for n in lens])
        q_out = dma.dma_append_paged(q, k, v, *wts, i32(list(range(B + 1))), i32(lens), table, kp, vp, dp, workspace=ws)
        lens = [n + 1 for n in lens]
        out = dma.dma_decode_paged(q_out, kp, vp, dp, table, i32(lens), w, workspace=ws)
        assert dma.dma_check(ws) == 0
        state = {"q": q_out.cpu(), "k": kp.cpu(), "v": vp.cpu(), "dt": dp.cpu(), "table": x["table"],
                 "lens": torch.tensor(lens, dtype=torch.int32), "interleaved": False}
        check_decode(state, out, w, 0, 0)
        if step == 0:
            for b in range(B):                       # the prefill over the same prompt, its last row
                L = prompts[b]
                qa, ka, va = (x[m][cu[b]:cu[b] + L].cuda() for m in "qkv")
                ko = torch.empty_like(ka)
                scratch = [torch.empty((-(-L // page), page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                qo = dma.dma_append_paged(qa, ka, va, *wts, i32([0, L]), i32([0]),
                                          torch.arange(-(-L // page), dtype=torch.int32, device="cuda")[None], *scratch,
                                          torch.empty((-(-L // page), Hkv, page), device="cuda"), k_out=ko)
                pre = dma.dma_forward_prefill(qo[None], ko[None], va[None], wts[2], wts[3], None, w)
                assert_close(f64(out[b]), f64(pre[0, -1]), 2 * BF16, 2e-2, "decode against the prefill's last row")
