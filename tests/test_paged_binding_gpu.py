"""Workspaces that the binding makes for a call: only their header is zeroed, and nothing else is needed."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dma():
    from doge_dynamic_mask_b200 import build
    build.build()
    from doge_dynamic_mask_b200 import dma as m
    return m


def marked(size):
    """Leaves a block of `size` bytes of 0xA5 to the allocator; returns its address."""
    t = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    torch.cuda.synchronize()
    del t
    return at


def what_is_left(size, at):
    t = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert t.data_ptr() == at, "the allocator gave another block: nothing to see here"
    return t


@pytest.mark.parametrize("w", [40, 2048])
def test_decode_without_a_workspace_zeroes_the_header_alone(dma, w):
    B, Hq, Hkv, d, page, pages = 3, 16, 2, 128, 16, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = rand(B, Hq, d), rand(B * pages, page, Hkv, d), rand(B * pages, page, Hkv, d)
    dt = torch.rand((B * pages, Hkv, page), generator=gen, device="cuda")
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    lens = torch.tensor([100, 0, 127], dtype=torch.int32, device="cuda")
    size = dma.dma_decode_paged_workspace_size(B, pages, page, Hq, Hkv, d, w)
    ws, out, want = dma.new_workspace(size), torch.empty_like(q), torch.empty_like(q)
    dma.dma_decode_paged(q, k, v, dt, table, lens, w, out=want, workspace=ws)
    del ws
    torch.cuda.empty_cache()
    at = marked(size)
    dma.dma_decode_paged(q, k, v, dt, table, lens, w, out=out)
    assert torch.equal(out, want)
    t = what_is_left(size, at)
    assert not t[:256].any()
    assert (t[256:] == 0xA5).float().mean() > 0.5


def test_prologue_backward_without_a_workspace_zeroes_the_header_alone(dma):
    B, L, Hq, Hkv, d = 2, 37, 8, 4, 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, gq, gk, dq, dk = (rand(B, L, h, d) for h in (Hq, Hkv) * 3)
    one, pos = torch.ones(d, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    dw = [torch.empty_like(one) for _ in range(4)]
    call = lambda a, b, ws=None: dma.dma_prologue_backward(q, k, one, one, pos, gq, gk, dq=dq, dk=dk, dq_norm_w=a,
                                                           dk_norm_w=b, workspace=ws)
    size = dma.dma_prologue_backward_workspace_size(B, L, Hq, Hkv, d)
    ws = dma.new_workspace(size)
    call(*dw[:2], ws)
    del ws
    torch.cuda.empty_cache()
    at = marked(size)
    call(*dw[2:])
    assert torch.equal(dw[0], dw[2]) and torch.equal(dw[1], dw[3])
    t = what_is_left(size, at)
    assert not t[:256].any()
    assert (t[256:] == 0xA5).float().mean() > 0.5


def test_decode_refuses_to_write_its_query(dma):
    """Blocks that share a row read q until the last one has joined it: in place would be a race."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    q, kv, dt = rand(1, 4, 64), rand(4, 16, 2, 64), torch.rand((4, 2, 16), generator=gen, device="cuda")
    table, lens = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([60], dtype=torch.int32, device="cuda")
    before = q.clone()
    with pytest.raises(ValueError, match="out must not be q"):
        dma.dma_decode_paged(q, kv, kv, dt, table, lens, 2048, out=q)
    assert torch.equal(q, before)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_infinite_values_show_where_they_are_kept_and_nowhere_else(dma, Hq, Hkv, d):
    """A probability's three parts are not negative, so their products with an infinity are it, or NaN where a part is 0."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v, dt = rand(2, Hq, d), rand(8, 16, Hkv, d), rand(8, 16, Hkv, d), torch.rand((8, Hkv, 16), generator=gen, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([60, 60], dtype=torch.int32, device="cuda")
    want = dma.dma_decode_paged(q, k, v, dt, table, lens, 2048)
    v[1, 3, 0, 7] = float("inf")                     # kept by sequence 0
    v[7, 14, 0, 7] = float("inf")                    # past sequence 1's length
    out = dma.dma_decode_paged(q, k, v, dt, table, lens, 2048)
    rep = Hq // Hkv
    got = out[0, :rep, 7]
    assert (got.isnan() | (got == float("inf"))).all()
    others = torch.ones_like(out, dtype=torch.bool)
    others[0, :rep, 7] = False
    assert torch.equal(out[others], want[others])
