"""What the serving and training operators next to the attention are measured on.

Three operators:

* ``append``: new tokens of a ragged batch enter a paged cache.  Q and K pass
  the per-head RMSNorm and the rotary embedding, K and V go to their pages, and
  the tokens' scores dt = exp(A softplus(v_flat W)) go to the page's dt rows.
* ``decode``: one new query per sequence attends to a paged cache under the
  dynamic mask (the best ``w`` visible keys by dt, ties to the lower index),
  with dt as an additive bias; a window and first tokens that stay visible
  (sinks) may limit what is visible.
* ``prologue_backward``: gradients of the per-head RMSNorm and the rotary
  embedding with respect to q, k and the two norm weights.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, calls the library.  ``exact`` computes them again in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
SPARE_PAGES = 3          # pages of the pool that belong to no sequence


def listed():
    return [
        # one step of a full serving batch: a token per sequence, q/k/v slices of one projection's output,
        # seven slots of the captured batch unused
        {"name": "append_batch", "op": "append", "B": 57, "new_lo": 1, "new_hi": 1, "ctx": 1500, "Hq": 16, "Hkv": 8,
         "d": 128, "page": 64, "pad": 7, "fused": True, "k_out": False},
        # ragged prompts and single tokens in one batch, small pages
        {"name": "append_prompts", "op": "append", "B": 9, "new_lo": 1, "new_hi": 2047, "ctx": 300, "Hq": 8, "Hkv": 4,
         "d": 64, "page": 16, "pad": 0, "fused": False, "k_out": True},
        # one long prompt: the projected states of the whole context enter the cache
        {"name": "append_prompt_long", "op": "append", "B": 1, "new_lo": 32768, "new_hi": 32768, "ctx": 0, "Hq": 16,
         "Hkv": 8, "d": 128, "page": 128, "pad": 0, "fused": True, "k_out": True},
        # the first answers of a single user: latency
        {"name": "decode_one", "op": "decode", "B": 1, "len_lo": 301, "len_hi": 301, "w": 2048, "window": 0,
         "sinks": 0, "Hq": 8, "Hkv": 4, "d": 64, "page": 16, "cap": 2048, "a0": False},
        # a batch of conversations no longer than the kept window, one slot empty
        {"name": "decode_batch", "op": "decode", "B": 32, "len_lo": 0, "len_hi": 2048, "w": 2048, "window": 0,
         "sinks": 0, "Hq": 8, "Hkv": 4, "d": 64, "page": 16, "cap": 2048, "a0": False},
        # long contexts, each keeping its best 2048 keys
        {"name": "decode_topk_batch", "op": "decode", "B": 64, "len_lo": 32768, "len_hi": 65536, "w": 2048,
         "window": 0, "sinks": 0, "Hq": 16, "Hkv": 8, "d": 128, "page": 64, "cap": 65536, "a0": False},
        # one very long context: few rows, a long axis to select over
        {"name": "decode_topk_one", "op": "decode", "B": 1, "len_lo": 500001, "len_hi": 500001, "w": 2048,
         "window": 0, "sinks": 0, "Hq": 16, "Hkv": 8, "d": 128, "page": 64, "cap": 524288, "a0": False},
        # every key of long contexts is kept: the whole cache is read
        {"name": "decode_full_long", "op": "decode", "B": 8, "len_lo": 65536, "len_hi": 131072, "w": 131072,
         "window": 0, "sinks": 0, "Hq": 16, "Hkv": 8, "d": 128, "page": 64, "cap": 131072, "a0": False},
        # a sliding window with four first tokens that stay visible, eight query heads per kv head
        {"name": "decode_window", "op": "decode", "B": 48, "len_lo": 1, "len_hi": 32768, "w": 2048, "window": 1024,
         "sinks": 4, "Hq": 16, "Hkv": 2, "d": 128, "page": 32, "cap": 32768, "a0": False},
        # a short training micro-batch: latency
        {"name": "prologue_bwd_small", "op": "prologue_backward", "B": 2, "L": 37, "Hq": 8, "Hkv": 4, "d": 64,
         "pos": 0, "fused": False},
        # the dense training workload's shape
        {"name": "prologue_bwd_dense", "op": "prologue_backward", "B": 8, "L": 2048, "Hq": 8, "Hkv": 4, "d": 64,
         "pos": 0, "fused": False},
        # the long training workload's shape, q/k and their gradients slices of one projection's buffers
        {"name": "prologue_bwd_long", "op": "prologue_backward", "B": 1, "L": 32768, "Hq": 16, "Hkv": 8, "d": 128,
         "pos": 0, "fused": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([r for r in (1, 2, 3, 4, 5, 6, 7, 8) if r * Hkv <= 32])
        page = rng.choice([1, 5, 8, 16, 24, 32, 64, 100, 128, 256])
        op = rng.choice(["append", "decode", "decode", "prologue_backward"])
        if op == "append":
            B = _log_int(rng, 1, 96)
            hi = rng.choice([1, _log_int(rng, 1, max(1, 32768 // B))])
            case = {"op": op, "B": B, "new_lo": rng.choice([1, hi]), "new_hi": hi, "ctx": rng.choice([0, _log_int(rng, 1, 65536)]),
                    "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "pad": rng.choice([0, rng.randint(1, 9)]),
                    "fused": rng.random() < 0.5, "k_out": rng.random() < 0.5}
            held = 8 * B * (case["ctx"] + hi) * Hkv * d * 4
        elif op == "decode":
            B = _log_int(rng, 1, 64)
            hi = _log_int(rng, 1, 400000)
            cap = hi + rng.choice([0, 1, hi // 3])
            window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
            case = {"op": op, "B": B, "len_lo": rng.choice([0, 1, hi // 2, hi]), "len_hi": hi,
                    "w": rng.choice([_log_int(rng, 1, 8192), 2048, cap + page]), "window": window,
                    "sinks": rng.choice([0, 4, rng.randint(1, 70)]) if window else 0, "Hq": Hq, "Hkv": Hkv, "d": d,
                    "page": page, "cap": cap, "a0": rng.random() < 0.15}
            held = B * cap * Hkv * d * 4
        else:
            B = _log_int(rng, 1, 16)
            case = {"op": op, "B": B, "L": _log_int(rng, 1, 32768 // B), "Hq": Hq, "Hkv": Hkv, "d": d,
                    "pos": rng.choice([0, _log_int(rng, 1, 100000)]), "fused": rng.random() < 0.5}
            held = 0
        most = {"append": 6.0e8, "decode": 3.2e9, "prologue_backward": 7.0e8}[op]
        if work(case)["bytes"] <= most and held <= 8e9:
            return case


def _spread(lo, hi, n):
    """n whole numbers spread evenly from lo to hi."""
    return [lo + (hi - lo) * i // (n - 1) if n > 1 else hi for i in range(n)]


def _visible(case, n):
    return min(n, case["sinks"] + case["window"]) if case["window"] else n


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "append":
        T = sum(_spread(case["new_lo"], case["new_hi"], case["B"]))
        rows = 2 * (Hq + 2 * Hkv) + (Hkv if case["k_out"] else 0)            # q, k, v in; q, k, v (and k again) out
        return {"bytes": T * (rows * d * 2 + Hkv * 4) + (Hkv * d * Hkv + Hkv + 2 * d) * 4,
                "flops": T * (2 * Hkv * d * Hkv + 10 * (Hq + Hkv) * d)}
    if case["op"] == "decode":
        total, flops = 0, 0
        for n in _spread(case["len_lo"], case["len_hi"], case["B"]):
            nvis = _visible(case, n)
            kept = min(nvis, case["w"])
            total += Hkv * (nvis * 4 + kept * d * 4) + -(-nvis // case["page"]) * 4 + 4 * Hq * d
            flops += 4 * Hq * kept * d
        return {"bytes": total, "flops": flops}
    T = case["B"] * case["L"]
    return {"bytes": T * (Hq + Hkv) * d * 6 + 16 * d, "flops": T * (Hq + Hkv) * d * 20}


def _randn(shape, gen):
    """N(0, 1) rounded to bf16; large tensors in pieces."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 28):
        flat[s:s + (1 << 28)].normal_(generator=gen)
    return out


def _qkv(T, Hq, Hkv, d, fused, gen, parts):
    """Projected states of T tokens: tensors of their own, or slices of one projection's output."""
    heads = [Hq, Hkv, Hkv][:parts]
    if fused:
        return list(torch.split(_randn((T, sum(heads), d), gen), heads, dim=1))
    return [_randn((T, h, d), gen) for h in heads]


def _table(counts, max_pages, gen):
    """A page table whose pages lie scattered over the pool; entries past a sequence's pages hold -1."""
    counts = torch.tensor(counts)
    perm = torch.randperm(int(counts.sum()) + SPARE_PAGES, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), max_pages), -1, dtype=torch.int32, device="cuda")
    used = (torch.arange(max_pages)[None] < counts[:, None]).cuda()
    table[used] = perm[:int(counts.sum())]
    return table, perm.numel()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    s = {"case": case, "own": {}}
    if case["op"] == "prologue_backward":
        T = B * case["L"]
        q, k = _qkv(T, Hq, Hkv, d, case["fused"], gen, 2)
        s["q"], s["k"] = (x.unflatten(0, (B, case["L"])) for x in (q, k))
        s["dq_out"], s["dk_out"] = (_randn((B, case["L"], h, d), gen) for h in (Hq, Hkv))
        dq, dk = _qkv(T, Hq, Hkv, d, case["fused"], gen, 2)
        s["dq"], s["dk"] = (x.unflatten(0, (B, case["L"])) for x in (dq, dk))
        s["q_w"], s["k_w"] = (torch.rand(d, generator=gen, device="cuda") + 0.5 for _ in range(2))
        s["positions"] = torch.randint(0, case["pos"] + 1, (B,), generator=gen, device="cuda").to(torch.int32)
        return s
    page = case["page"]
    s["A"] = -(torch.rand(Hkv, generator=gen, device="cuda") * 1.9 + 0.1)
    order = torch.randperm(B, generator=gen, device="cuda").cpu().tolist()
    if case["op"] == "append":
        news = _spread(case["new_lo"], case["new_hi"], B)
        news = [news[i] for i in order]
        T = sum(news) + case["pad"]
        s["q"], s["k"], s["v"] = _qkv(T, Hq, Hkv, d, case["fused"], gen, 3)
        s["q_w"], s["k_w"] = (torch.rand(d, generator=gen, device="cuda") + 0.5 for _ in range(2))
        s["W"] = torch.randn((Hkv * d, Hkv), generator=gen, device="cuda") * 0.02
        pos = [_spread(case["ctx"], 0, B)[i] for i in order]
        s["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        s["cu_tokens"] = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
        max_pages = -(-(case["ctx"] + max(news)) // page)
        counts = [-(-(p + n) // page) for p, n in zip(pos, news)]
        s["table"], n_pages = _table(counts, max_pages, gen)
        s["k_pages"] = torch.zeros((n_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        s["dt_pages"] = torch.zeros((n_pages, Hkv, page), device="cuda")
        s["q_out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device="cuda") if case["k_out"] else None
        return s
    lens = _spread(case["len_lo"], case["len_hi"], B)
    lens = [lens[i] for i in order]
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    max_pages = -(-max(case["cap"], 1) // page)
    s["table"], n_pages = _table([-(-n // page) for n in lens], max_pages, gen)
    s["k_pages"], s["v_pages"] = (_randn((n_pages, page, Hkv, d), gen) for _ in range(2))
    if case["a0"]:
        s["A"] = torch.zeros_like(s["A"])            # a model at its start: every dt is 1, ties everywhere
    x = torch.randn((n_pages, Hkv, page), generator=gen, device="cuda") * 0.64
    s["dt_pages"] = torch.exp(s["A"][:, None] * torch.nn.functional.softplus(x))
    s["q"] = _randn((B, Hq, d), gen)
    s["out"] = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    return s


# ---- the plain forms ----------------------------------------------------------------

def _angles(pos, d):
    """cos and sin [..., 1, d/2] (float32) of the positions' rotary angles, formed in 64 bits."""
    freq = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    a = torch.remainder(pos.double()[..., None, None] * freq, 2 * math.pi).float()
    return torch.cos(a), torch.sin(a)


def _norm_rotate(x, w, cos, sin):
    x = x.float()
    y = w * (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS))
    lo, hi = y.chunk(2, -1)
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).bfloat16()


def _append_plain(s):
    c = s["case"]
    cu = s["cu_tokens"].long()
    total = s["q"].shape[0] - c["pad"]
    tok = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = s["positions"].long()[seq] + tok - cu[seq]
    pages, off = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    cos, sin = _angles(pos, c["d"])
    kn = _norm_rotate(s["k"][:total], s["k_w"], cos, sin)
    v = s["v"][:total]
    x = v.reshape(total, -1).float() @ s["W"]
    dt = torch.exp(s["A"] * torch.nn.functional.softplus(x, threshold=60.0))
    s["q_out"][:total] = _norm_rotate(s["q"][:total], s["q_w"], cos, sin)
    s["k_pages"][pages, off] = kn
    s["v_pages"][pages, off] = v
    s["dt_pages"][pages, :, off] = dt
    if s["k_out"] is not None:
        s["k_out"][:total] = kn


def _decode_plain(s):
    c = s["case"]
    B, Hq, Hkv, d, page, w = (c[n] for n in ("B", "Hq", "Hkv", "d", "page", "w"))
    lens = s["lengths"].long()
    # visible keys in order: the sinks and the window, or all of them
    shift = (lens - c["window"] - c["sinks"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    n = max(1, _visible(c, c["len_hi"]))
    i = torch.arange(n, device="cuda")
    j = torch.where(i < c["sinks"], i, i + shift[:, None]) if c["window"] else i.expand(B, n)
    seen = i < (lens - shift)[:, None]                                      # [B, n]
    pages = torch.gather(s["table"].long(), 1, (j // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    off = j % page
    g = torch.arange(Hkv, device="cuda")[None, :, None]
    dt = s["dt_pages"][pages[:, None], g, off[:, None]]                      # [B, Hkv, n]
    keep = seen[:, None].expand(B, Hkv, n)
    if n > w:
        key = dt.view(torch.int32).long() * (1 << 32) + (0xFFFFFFFF - i)     # dt >= 0: its bits order like it
        best = torch.topk(torch.where(keep, key, -1), w, dim=-1).indices     # [B, Hkv, w]
        dt, keep = torch.gather(dt, 2, best), torch.gather(keep, 2, best)
        pages, off = (torch.gather(x[:, None].expand(B, Hkv, n), 2, best) for x in (pages, off))
    else:
        pages, off = pages[:, None], off[:, None]
    k = s["k_pages"][pages, off, g].float()                                  # [B, Hkv, kept, d]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    sc = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5 + dt[:, :, None]
    del k
    sc = sc.masked_fill(~keep[:, :, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    v = s["v_pages"][pages, off, g].float()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    return o.view(B, Hq, d).bfloat16()


def _backward_plain(s):
    c = s["case"]
    pos = s["positions"].long()[:, None] + torch.arange(c["L"], device="cuda")
    cos, sin = _angles(pos, c["d"])

    def one(x, w, dout):
        x, lo, hi = x.float(), *dout.float().chunk(2, -1)
        dy = torch.cat([lo * cos + hi * sin, hi * cos - lo * sin], -1)       # the rotation undone
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * r
        dw = (dy * xh).sum((0, 1, 2))
        dyw = dy * w
        return (r * (dyw - xh * (dyw * xh).mean(-1, keepdim=True))).bfloat16(), dw

    dq, dqw = one(s["q"], s["q_w"], s["dq_out"])
    dk, dkw = one(s["k"], s["k_w"], s["dk_out"])
    return {"dq": dq, "dk": dk, "dq_norm_w": dqw, "dk_norm_w": dkw}


# ---- the library's ------------------------------------------------------------------

def _workspace(s, size):
    """The workspace that a program keeps beside its buffers: made once, zeroed once."""
    from doge_dynamic_mask_b200 import dma
    if "ws" not in s["own"]:
        s["own"]["ws"] = dma.new_workspace(size)
    return s["own"]["ws"]


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            from doge_dynamic_mask_b200 import dma
            dma.dma_append_paged(s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["W"], s["A"], s["cu_tokens"],
                                 s["positions"], s["table"], s["k_pages"], s["v_pages"], s["dt_pages"], eps=EPS,
                                 rope_theta=THETA, q_out=s["q_out"], k_out=s["k_out"], workspace=_workspace(s, 256))
        else:
            _append_plain(s)
        return {n: s[n] for n in ("q_out", "k_out", "k_pages", "v_pages", "dt_pages")}
    if c["op"] == "decode":
        if not own:
            return _decode_plain(s)
        from doge_dynamic_mask_b200 import dma
        if "ws" not in s["own"]:
            _workspace(s, dma.dma_decode_paged_workspace_size(c["B"], s["table"].shape[1], c["page"], c["Hq"], c["Hkv"],
                                                              c["d"], c["w"], c["window"], c["sinks"]))
        return dma.dma_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["dt_pages"], s["table"], s["lengths"], c["w"],
                                    window=c["window"], sinks=c["sinks"], out=s["out"], workspace=s["own"]["ws"])
    if not own:
        return _backward_plain(s)
    from doge_dynamic_mask_b200 import dma
    if "ws" not in s["own"]:
        _workspace(s, dma.dma_prologue_backward_workspace_size(c["B"], c["L"], c["Hq"], c["Hkv"], c["d"]))
    dq, dk, dqw, dkw = dma.dma_prologue_backward(s["q"], s["k"], s["q_w"], s["k_w"], s["positions"], s["dq_out"],
                                                 s["dk_out"], eps=EPS, rope_theta=THETA, dq=s["dq"], dk=s["dk"],
                                                 workspace=s["own"]["ws"])
    return {"dq": dq, "dk": dk, "dq_norm_w": dqw, "dk_norm_w": dkw}


# ---- 64 bits ------------------------------------------------------------------------

def _turn(x, pos, sign):
    """Channel pairs (i, i + d/2) as complex numbers, turned by sign * pos * theta^(-2i/d)."""
    half = x.shape[-1] // 2
    freq = torch.exp(-math.log(THETA) * torch.arange(half, dtype=torch.float64, device="cuda") / half)
    a = pos.double()[:, None, None] * freq * sign
    z = torch.complex(x[..., :half], x[..., half:]) * torch.polar(torch.ones_like(a), a)
    return torch.cat([z.real, z.imag], -1)


def _rms(x):
    return torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "append":
        out = {n: None if s[n] is None else s[n].double() for n in ("q_out", "k_out", "k_pages", "v_pages", "dt_pages")}
        cu, start = s["cu_tokens"].tolist(), s["positions"].tolist()
        for b in range(case["B"]):
            for lo in range(cu[b], cu[b + 1], 4096):
                t = slice(lo, min(lo + 4096, cu[b + 1]))
                pos = torch.arange(start[b] + t.start - cu[b], start[b] + t.stop - cu[b], device="cuda")
                q, k, v = (s[n][t].double() for n in ("q", "k", "v"))
                out["q_out"][t] = _turn(q / _rms(q) * s["q_w"].double(), pos, 1)
                kn = _turn(k / _rms(k) * s["k_w"].double(), pos, 1)
                if out["k_out"] is not None:
                    out["k_out"][t] = kn
                at = s["table"][b].long()[pos // case["page"]], pos % case["page"]
                out["k_pages"][at], out["v_pages"][at] = kn, v
                x = v.flatten(1) @ s["W"].double()
                dt = torch.exp(s["A"].double() * (torch.relu(x) + torch.log1p(torch.exp(-x.abs()))))
                out["dt_pages"][at[0], :, at[1]] = dt
        return out
    if case["op"] == "decode":
        o = torch.zeros((case["B"], Hq, d), dtype=torch.float64, device="cuda")
        rep = Hq // Hkv
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            j = torch.arange(n, device="cuda")
            if case["window"]:
                j = j[(j < case["sinks"]) | (j >= n - case["window"])]
            page, off = s["table"][b].long()[j // case["page"]], j % case["page"]
            for g in range(Hkv):
                dt = s["dt_pages"][page, g, off]
                kept = torch.sort(dt, descending=True, stable=True).indices[:case["w"]]
                k, v = (s[x][page[kept], off[kept], g].double() for x in ("k_pages", "v_pages"))
                sc = s["q"][b, g * rep:(g + 1) * rep].double() @ k.T / math.sqrt(d) + dt[kept].double()
                o[b, g * rep:(g + 1) * rep] = torch.softmax(sc, -1) @ v
        return o
    out = {}
    pos = (s["positions"][:, None] + torch.arange(case["L"], device="cuda")).flatten()
    for n, wn in (("q", "q_w"), ("k", "k_w")):
        grads, dw = [], torch.zeros(d, dtype=torch.float64, device="cuda")
        x_all, g_all = s[n].flatten(0, 1), s["d%s_out" % n].flatten(0, 1)
        for lo in range(0, x_all.shape[0], 4096):
            x, g = x_all[lo:lo + 4096].double(), _turn(g_all[lo:lo + 4096].double(), pos[lo:lo + 4096], -1)
            rms = _rms(x)
            dw += (g * x / rms).sum((0, 1))
            u = g * s[wn].double()
            grads.append(u / rms - x * (u * x).sum(-1, keepdim=True) / (d * rms ** 3))
        out["d" + n] = torch.cat(grads).view(s[n].shape)
        out["d%s_norm_w" % n] = dw
    return out
