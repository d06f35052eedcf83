"""Refusals of the paged-cache calls and the prologue's backward, on the host before any device work, and the sizes
they report.  Every call here has one bad argument: nothing is ever launched on the dummy pointers."""
import ctypes

import pytest
import torch

from doge_dynamic_mask_b200 import build as dma_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def dma():
    dma_build.build()
    from doge_dynamic_mask_b200 import dma as m
    return m


P = ctypes.c_void_p(1 << 20)            # aligned dummy address, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)    # misaligned

APPEND = dict(q=P, k=P, v=P, q_stride=512, k_stride=256, v_stride=256, q_norm_w=P, k_norm_w=P, eps=1e-6,
              rope_theta=10000.0, W_dt=P, A=P, cu_tokens=P, positions=P, page_table=P, T=5, B=2, max_pages=8,
              num_pages=20, page_size=16, page_stride=16 * 256, Hq=8, Hkv=4, d=64, q_out=P, k_out=None, k_pages=P,
              v_pages=P, dt_pages=P, workspace=P, ws_bytes=256, stream=None)
DECODE = dict(q=P, k_pages=P, v_pages=P, dt_pages=P, page_table=P, lengths=P, B=2, max_pages=8, num_pages=20,
              page_size=16, page_stride=16 * 256, Hq=8, Hkv=4, d=64, keep_window_size=64, window=0, sinks=0,
              scale=0.125, out=P, workspace=P, ws_bytes=1 << 40, stream=None)
BACKWARD = dict(q=P, k=P, q_stride=512, k_stride=256, q_norm_w=P, k_norm_w=P, eps=1e-6, rope_theta=10000.0,
                positions=P, dq_out=P, dk_out=P, B=2, L=5, Hq=8, Hkv=4, d=64, dq=P, dk=P, dq_stride=512,
                dk_stride=256, dq_norm_w=P, dk_norm_w=P, workspace=P, ws_bytes=1 << 40, stream=None)


def pointers(args):
    return [n for n, v in args.items() if v is P]


def cases(args, more):
    out = [(n, bad, INVALID) for n in pointers(args) for bad in (None, ODD)]
    return out + more


SHAPES = [("Hq", 6, INVALID), ("Hq", 0, INVALID), ("Hkv", 0, INVALID), ("d", 96, UNSUPPORTED), ("Hkv", -4, INVALID)]
PAGES = [("B", 0, INVALID), ("B", 65537, UNSUPPORTED), ("max_pages", 0, INVALID), ("num_pages", 0, INVALID),
         ("page_size", 0, INVALID), ("page_size", -16, INVALID), ("page_stride", 16 * 256 - 8, INVALID),
         ("page_stride", 16 * 256 + 4, INVALID), ("page_stride", 1 << 33, UNSUPPORTED),
         ("page_stride", 1 << 62, UNSUPPORTED), ("max_pages", 65537, UNSUPPORTED), ("ws_bytes", 255, WORKSPACE)]
ROPE = [("eps", -1e-6, INVALID), ("eps", float("nan"), INVALID), ("rope_theta", 1.0, INVALID),
        ("rope_theta", float("inf"), INVALID)]


@pytest.mark.parametrize("name,bad,status", cases(APPEND, SHAPES + PAGES + ROPE + [
    ("k_out", ODD, INVALID), ("T", 0, INVALID), ("T", 1 << 28, UNSUPPORTED), ("q_stride", 504, INVALID),
    ("q_stride", 516, INVALID), ("k_stride", 248, INVALID), ("v_stride", 0, INVALID), ("v_stride", -256, INVALID)]))
def test_append_refuses(dma, name, bad, status):
    assert dma.raw().dma_append_paged(*dict(APPEND, **{name: bad}).values()) == status


@pytest.mark.parametrize("name,bad,status", cases(DECODE, SHAPES + PAGES + [
    ("keep_window_size", 0, INVALID), ("window", -1, INVALID), ("sinks", -1, INVALID), ("scale", float("nan"), INVALID),
    ("scale", float("inf"), INVALID)]))
def test_decode_refuses(dma, name, bad, status):
    assert dma.raw().dma_decode_paged(*dict(DECODE, **{name: bad}).values()) == status


@pytest.mark.parametrize("name,bad,status", cases(BACKWARD, SHAPES + ROPE + [
    ("B", 0, INVALID), ("L", 0, INVALID), ("L", 1 << 30, UNSUPPORTED), ("q_stride", 504, INVALID),
    ("dq_stride", 516, INVALID), ("dk_stride", 8, INVALID), ("ws_bytes", 256, WORKSPACE)]))
def test_backward_refuses(dma, name, bad, status):
    assert dma.raw().dma_prologue_backward(*dict(BACKWARD, **{name: bad}).values()) == status


def test_workspace_sizes(dma):
    f = dma.dma_decode_paged_workspace_size
    short = f(4, 8, 16, 8, 4, 64, 128)                     # 128 positions: no row can see more than it keeps
    assert short > 256
    assert f(4, 8, 16, 8, 4, 64, 127) >= short + 2 * 4 * 4 * 127 * 4
    assert f(4, 80, 16, 8, 4, 64, 128, 100, 28) == short   # nor can it through this window
    assert f(4, 80, 16, 8, 4, 64, 128, 100, 29) > short
    assert f(64, 1024, 64, 16, 8, 128, 1 << 20) == f(1, 1, 1, 16, 8, 128, 1)
    assert f(4, 8, 16, 8, 3, 64, 128) == f(0, 8, 16, 8, 4, 64, 128) == f(4, 8, 16, 8, 4, 80, 128) == 0
    assert f(4, 1 << 20, 2, 8, 4, 64, 128) == 0            # more than 2^20 positions
    assert f(2048, 1 << 16, 16, 16, 16, 64, 1 << 20) == 0  # 2^35 kept keys
    assert f(2047, 1 << 16, 16, 16, 16, 64, 1 << 20) > 0
    assert dma.dma_prologue_backward_workspace_size(1, 1, 8, 4, 64) > 256
    assert dma.dma_prologue_backward_workspace_size(1, 1, 8, 3, 64) == 0
    assert dma.dma_status_string(8) == "DMA_ERR_BAD_PAGE"


def test_binding_refuses_host_tensors(dma):
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    kv = torch.zeros((3, 16, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dma.dma_decode_paged(q, kv, kv, torch.zeros((3, 4, 16)), torch.zeros((2, 1), dtype=torch.int32),
                             torch.ones(2, dtype=torch.int32), 64)


def test_token_stride(dma):
    x = torch.zeros((6, 16, 64))
    assert dma._token_stride("x", x) == 1024
    assert dma._token_stride("x", x[:, :4]) == 1024
    assert dma._token_stride("x", x[:1, :4]) == 256
    assert dma._token_stride("x", x.view(2, 3, 16, 64)[:, :, 4:8]) == 1024
    assert dma._token_stride("x", x.view(6, 1, 16, 64)[:, :, 4:8]) == 1024
    assert dma._token_stride("x", x.view(1, 6, 16, 64)[:, :, 4:8]) == 1024
    for bad in (x[..., ::2], x[:, ::2], x.view(2, 3, 16, 64)[:, :2], x.transpose(0, 1)):
        with pytest.raises(ValueError):
            dma._token_stride("x", bad)


def test_page_stride(dma):
    kv = torch.zeros((5, 2, 16, 4, 64))
    assert dma._page_stride(kv[:, 0], kv[:, 1]) == 2 * 16 * 256
    assert dma._page_stride(kv[:1, 0], kv[:1, 1]) == 16 * 256
    dense = torch.zeros((5, 16, 4, 64))
    assert dma._page_stride(dense, dense) == 16 * 256
    for k, v in ((kv[:, 0], dense), (kv[:, 0, :8], kv[:, 1]), (dense.transpose(1, 2), dense.transpose(1, 2))):
        with pytest.raises(ValueError):
            dma._page_stride(k, v)
