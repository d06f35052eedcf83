"""The binding of the paged cache and of the prologue's backward where no GPU is needed: sizes beyond 32 bits."""
import pytest
import torch

from doge_dynamic_mask_b200 import build as dma_build


@pytest.fixture(scope="module")
def dma():
    dma_build.build()
    from doge_dynamic_mask_b200 import dma as m
    return m


BEYOND = [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5, -2 ** 31 - 1, 2 ** 64 + 5, -5]


@pytest.mark.parametrize("bad", BEYOND)
@pytest.mark.parametrize("name", ["keep_window_size", "window", "sinks"])
def test_decode_refuses_sizes_that_32_bits_would_wrap(dma, name, bad):
    """-2^32 + 5 is 5 in a C int."""
    bf = dict(dtype=torch.bfloat16)
    sizes = {"keep_window_size": 64, "window": 8, "sinks": 1, name: bad}
    with pytest.raises(ValueError, match=r"2\^31"):
        dma.dma_decode_paged(torch.zeros((1, 4, 64), **bf), torch.zeros((2, 16, 2, 64), **bf),
                             torch.zeros((2, 16, 2, 64), **bf), torch.zeros((2, 2, 16)),
                             torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32), **sizes)


@pytest.mark.parametrize("bad", BEYOND)
def test_workspace_sizes_are_zero_beyond_32_bits(dma, bad):
    decode = dict(B=2, max_pages=8, page_size=16, Hq=8, Hkv=4, d=64, keep_window_size=64, window=8, sinks=1)
    assert dma.dma_decode_paged_workspace_size(**decode) > 0
    for name in decode:
        assert dma.dma_decode_paged_workspace_size(**dict(decode, **{name: bad})) == 0, name
    backward = dict(B=2, L=5, Hq=8, Hkv=4, d=64)
    assert dma.dma_prologue_backward_workspace_size(**backward) > 0
    for name in backward:
        assert dma.dma_prologue_backward_workspace_size(**dict(backward, **{name: bad})) == 0, name


@pytest.mark.parametrize("Hq,Hkv,d,w", [(8, 4, 64, 100), (16, 2, 128, 2048), (3, 1, 128, 1), (16, 16, 64, 33)])
def test_list_views_are_the_last_parts_of_the_workspace(dma, Hq, Hkv, d, w):
    """Whatever lies before them: both lists, each rounded up to 256 bytes, end the workspace of every table."""
    B = 3
    n, up = B * Hkv * w * 4, lambda x: -(-x // 256) * 256
    for max_pages, page in ((w + 1, 1), (500, 16), (7000, 100)):
        size = dma.dma_decode_paged_workspace_size(B, max_pages, page, Hq, Hkv, d, w)
        ws = torch.zeros(size, dtype=torch.uint8)
        pos, bias = dma.paged_list_views(ws, B, Hq, Hkv, d, w)
        assert pos.dtype == torch.int32 and bias.dtype == torch.float32 and pos.shape == bias.shape == (B, Hkv, w)
        at = [t.data_ptr() - ws.data_ptr() for t in (pos, bias)]
        assert at == [size - 2 * up(n), size - up(n)]
    # without lists the workspace is that much smaller
    assert dma.dma_decode_paged_workspace_size(B, w, 1, Hq, Hkv, d, w) == size - 2 * up(n)
