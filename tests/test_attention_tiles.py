"""pre_attn_attention_ext where several rows are one tcgen05 tile (pa_attn_tc.cu), against the 64-bit reference.  Small
calls go to clusters of the other kernel, so these have wide block tables, long sinks or many items, and each says which
kernel and mode it is to reach."""

import numpy as np
import pytest
import torch

from tests import cache_reference as ref
from tests import window_reference as win
from tests.test_cache_readers_host import P, attention_args
from tests.test_window_and_weights import FORMATS, case

WHOLE, SLICED, CLUSTER, TILES = 0, 1, 2, 4
WIDE = 60  # columns of the block table behind a request's blocks, with which few items are cut into slices


@pytest.fixture(scope="module")
def B():
    from indexer_projection_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def path(rd, ext=True):
    """Of the reader's last call to attend."""
    from indexer_projection_gb300 import binding as B
    return B.pre_attn_attention_path(rd._attn, rd._ext if ext else None)


def check(c, mode, lists=None, status=0, sel=None, again=True, **kw):
    """Attention and weights of the call, which is to reach the tiles in that mode; twice the same bits."""
    rd = c.reader(weigh=True, topk=lists[0].shape[-1] if lists else 0)
    out, w = win.attend(c, rd, lists, weights=True, **kw)
    assert path(rd) == TILES | mode
    q = None
    if "q" in kw:
        q = kw["q"].float().cpu() * kw["q_fp8_scale"]
    win.close(out, c.attention(sel, q=q))
    win.close_weights(w, c, c.weights(sel, q=q))
    if again:
        second = win.attend(c, rd, lists, weights=True, **kw)
        assert torch.equal(out, second[0]) and torch.equal(w, second[1])
    assert rd.device_status() == status
    return out, w


# ------------------------------------------------------------ which kernel

def test_path_without_a_gpu(B):
    e = B.pa_attention_ext(0, 0, None, 0, None, 0, 1.0, None, 0)
    assert B.load().pre_attn_attention_path(None, e) == -B.PA_ERR_NULL
    assert B.pre_attn_attention_path(attention_args(B)) == -B.PA_ERR_SHAPE  # no requests
    assert B.pre_attn_attention_path(attention_args(B), e) == -B.PA_ERR_SHAPE
    assert B.pre_attn_attention_path(attention_args(B, q=None)) == -B.PA_ERR_CONFIG
    e.window = -1
    assert B.pre_attn_attention_path(attention_args(B), e) == -B.PA_ERR_CONFIG
    e.window = 5
    assert B.pre_attn_attention_path(attention_args(B, blocks=P, counts=P), e) == -B.PA_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len,tiles", [("fp8", 4, 0), ("fp8", 5, TILES), ("fp8", 8, TILES), ("fp8", 9, TILES), ("nvfp4", 2, 0),
                                             ("nvfp4", 3, TILES), ("nvfp4", 16, TILES)])
def test_path_of_a_call(fmt, q_len, tiles):
    c = case(fmt, [q_len + 300, 0], q_len, 1, 2, seed=q_len, extra_width=WIDE).upload()
    rd = c.reader(weigh=True)
    win.attend(c, rd, weights=True)
    assert path(rd) == tiles | SLICED and path(rd, ext=False) == SLICED  # (without a window and weights: the other kernel)
    c.W, c.dev["bt"] = 4, c.dev["bt"][:, :4].contiguous()
    rd = c.reader(weigh=True)
    win.attend(c, rd, weights=True)
    assert path(rd) == CLUSTER
    many = case(fmt, [q_len + 5] * 2100, q_len, 1, 1, seed=1).upload()
    rd = many.reader(weigh=True)
    win.attend(many, rd, weights=True)
    assert path(rd) == tiles | WHOLE
