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


# ---------------------------------------------------- rows of V that are zero

def zero_value(c, r, j, scale=1.0):
    """Key j of request r: a value row of zeros, whose writer gives it the scale 1 (FP8).  It does not count to the
    largest weight x V scale."""
    slot = int(c.bt[r, j // 128]) * 128 + j % 128
    page, t = slot // 128 * c.kps + slot % 128 // 16, slot % 16
    for h in range(c.nkv):
        c.bytes["v"][(page * c.nkv + h) * 2048 + np.arange(128) * 16 + t] = 0x80 if j % 3 == 0 else 0  # (either zero)
        c.scales["v"][(page * c.nkv + h) * 16 + t] = scale
        c.v[h, slot], c.vs[h, slot] = 0.0, 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [SLICED, WHOLE])
@pytest.mark.parametrize("zeros", ["some", "blocks", "first block", "all"])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 100])
def test_zero_values_beside_small_scales(mode, zeros, scale):
    q_len = 5
    if mode == SLICED:
        c = case("fp8", [700, 130, 512], q_len, 1, 8, seed=70, extra_width=WIDE)
    else:
        c = case("fp8", [700, 130, 512, 300] * 20, q_len, 1, 8, 600, 130, seed=70)
    for w in "kv":
        c.scales[w][np.isfinite(c.scales[w])] *= np.float32(2.0 ** -9 if w == "v" else 1)
    c.v, c.vs = c.v * 2.0 ** -9, c.vs * 2.0 ** -9
    for r, n in enumerate(c.seq.tolist()):
        which = {"some": [j for j in range(n) if j % 7 == 2 or j == n - 1], "blocks": [j for j in range(n) if j // 128 % 2 == 1],
                 "first block": [j for j in range(n) if j < 128], "all": range(n)}[zeros]
        for j in which:
            zero_value(c, r, j, scale)
    c.upload()
    out, _ = check(c, mode)
    if zeros == "all":
        assert (out == 0).all()
