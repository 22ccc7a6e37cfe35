"""Refusals of pre_attn_index_scores_nvfp4, pre_attn_select_blocks and
pre_attn_attention: each documented error comes back before anything touches
a GPU (host-checkable arguments only; the pointers are never followed)."""

import ctypes

import pytest

from tests import cache_reference  # noqa: F401  (importable without a GPU)


@pytest.fixture(scope="module")
def B():
    from indexer_projection_gb300 import binding, build
    build.build()
    binding.load()
    return binding


P = 0x10000  # an aligned address that nothing reads


def scores_args(B, **kw):
    d = dict(iq=P, iq_stride=256, head=1, idx_cache=P, idx_pages=8, idx_page_bytes=1152, block_size=16, block_table=P,
             seq_lens=P, R=0, q_len=2, bt_width=3, init_blocks=1, local_blocks=1, index_scale=0.1, scores=P,
             score_stride=384, status=P)
    d.update(kw)
    return B.pa_index_nvfp4_args(**d)


def select_args(B, **kw):
    d = dict(scores=P, score_stride=384, score_head_stride=384 * 64, n_heads=2, seq_lens=P, R=0, q_len=2, bt_width=3,
             init_blocks=1, local_blocks=1, topk=2, blocks=P, counts=P, status=P)
    d.update(kw)
    return B.pa_select_args(**d)


def attention_args(B, cache_fields=None, **kw):
    c = B.pa_caches()
    c.k_cache = c.v_cache = c.k_scale = c.v_scale = c.kv_cache = P
    c.num_pages16, c.kv_pages, c.kv_page_bytes, c.k_global_scale, c.v_global_scale = 64, 64, 4608, 1.0, 1.0
    for k, v in (cache_fields or {}).items():
        setattr(c, k, v)
    d = dict(q=P, q_fp8=None, q_fp8_scale=1.0, q_stride=4096, n_q_heads=32, n_kv_heads=2, cache_format=B.PA_CACHE_FP8,
             block_size=16, kv_page_stride=0, caches=ctypes.pointer(c), block_table=P, seq_lens=P, blocks=P, counts=P,
             topk=4, R=0, q_len=2, bt_width=3, sm_scale=0.1, out=P + (1 << 24), out_stride=4096, workspace=P,
             workspace_bytes=1 << 30, status=P, flags=0)
    d.update(kw)
    return B.pa_attention_args(**d)


def test_nothing_to_do_is_accepted(B):
    assert B.pre_attn_index_scores_nvfp4(scores_args(B), check=False) == B.PA_OK
    assert B.pre_attn_select_blocks(select_args(B), check=False) == B.PA_OK
    assert B.pre_attn_attention(attention_args(B), check=False) == B.PA_OK
    assert B.pre_attn_attention(attention_args(B, cache_format=B.PA_CACHE_NVFP4), check=False) == B.PA_OK


@pytest.mark.parametrize("kw,err", [
    *[({p: None}, "NULL") for p in ("iq", "idx_cache", "block_table", "seq_lens", "scores", "status")],
    *[({"R": v}, "SHAPE") for v in (-1, 65536)], *[({"q_len": v}, "SHAPE") for v in (0, 17)],
    *[({"bt_width": v}, "SHAPE") for v in (0, 4, 16385)], ({"head": -1}, "SHAPE"), ({"head": 2}, "SHAPE"),
    ({"idx_pages": 0}, "SHAPE"), ({"idx_page_bytes": 1120}, "SHAPE"), ({"init_blocks": -1}, "CONFIG"),
    ({"local_blocks": -1}, "CONFIG"), ({"index_scale": float("nan")}, "CONFIG"),
    *[({"block_size": v}, "CONFIG") for v in (0, 2, 18, 2048)],
    *[({"block_size": v, "idx_page_bytes": 72 * 1024}, "UNSUPPORTED") for v in (12, 96, 192)],
    ({"iq": P + 4}, "ALIGN"), ({"iq_stride": 258}, "ALIGN"), ({"idx_cache": P + 16}, "ALIGN"),
    ({"idx_page_bytes": 1160}, "ALIGN"), ({"scores": P + 8}, "ALIGN"), ({"score_stride": 386}, "ALIGN"),
    ({"block_table": P + 2}, "ALIGN"), ({"seq_lens": P + 1}, "ALIGN"), ({"status": P + 2}, "ALIGN")])
def test_nvfp4_scores_refusals(B, kw, err):
    assert B.pre_attn_index_scores_nvfp4(scores_args(B, **kw), check=False) == getattr(B, "PA_ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    *[({p: None}, "NULL") for p in ("scores", "seq_lens", "blocks", "counts", "status")],
    *[({"R": v}, "SHAPE") for v in (-1, 65536)], *[({"q_len": v}, "SHAPE") for v in (0, 17)],
    *[({"n_heads": v}, "SHAPE") for v in (0, 65)], *[({"bt_width": v}, "SHAPE") for v in (0, 4, 16385)],
    *[({"topk": v}, "SHAPE") for v in (0, 257)], ({"R": 50}, "SHAPE"), ({"init_blocks": -1}, "CONFIG"),
    ({"local_blocks": -1}, "CONFIG"), ({"init_blocks": 2}, "CONFIG"), ({"init_blocks": 2 ** 31 - 1}, "CONFIG"),
    ({"scores": P + 4}, "ALIGN"), ({"score_stride": 385}, "ALIGN"), ({"score_head_stride": 384 * 64 + 2}, "ALIGN"),
    *[({p: P + 2}, "ALIGN") for p in ("seq_lens", "blocks", "counts", "status")]])
def test_selection_refusals(B, kw, err):
    assert B.pre_attn_select_blocks(select_args(B, **kw), check=False) == getattr(B, "PA_ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    *[({p: None}, "NULL") for p in ("caches", "block_table", "seq_lens", "out", "status", "counts")],
    ({"q": None}, "CONFIG"), ({"q_fp8": P}, "CONFIG"), ({"cache_format": 2}, "CONFIG"), ({"n_kv_heads": 3}, "CONFIG"),
    *[({"n_q_heads": v}, "CONFIG") for v in (0, 33, 34)], ({"flags": 1}, "CONFIG"),
    *[({"sm_scale": v}, "CONFIG") for v in (0.0, -1.0, float("inf"), float("nan"))],
    *[({"q": None, "q_fp8": P, "q_fp8_scale": v}, "CONFIG") for v in (0.0, float("inf"), float("nan"))],
    *[({"R": v}, "SHAPE") for v in (-1, 65536)], *[({"q_len": v}, "SHAPE") for v in (0, 17)],
    *[({"bt_width": v}, "SHAPE") for v in (0, 16385)], ({"q_stride": 4080}, "SHAPE"), ({"out_stride": 4088}, "SHAPE"),
    *[({"topk": v}, "SHAPE") for v in (0, 257)], *[({"kv_page_stride": v}, "CONFIG") for v in (-1, 7)],
    ({"block_size": 32}, "CONFIG"), ({"q": P + 8}, "ALIGN"), ({"q_stride": 4104}, "ALIGN"), ({"out": P + 8}, "ALIGN"),
    ({"out_stride": 4100}, "ALIGN"), *[({p: P + 2}, "ALIGN") for p in ("block_table", "seq_lens", "blocks", "counts", "status")]])
def test_attention_refusals(B, kw, err):
    assert B.pre_attn_attention(attention_args(B, **kw), check=False) == getattr(B, "PA_ERR_" + err)


@pytest.mark.parametrize("caches,err", [
    *[({p: None}, "NULL") for p in ("k_cache", "v_cache", "k_scale", "v_scale")],
    *[({p: P + 4}, "ALIGN") for p in ("k_cache", "v_cache", "k_scale", "v_scale")], ({"num_pages16": 0}, "CONFIG")])
def test_attention_refuses_bad_fp8_caches(B, caches, err):
    assert B.pre_attn_attention(attention_args(B, caches), check=False) == getattr(B, "PA_ERR_" + err)


@pytest.mark.parametrize("caches,kw,err", [
    ({"kv_cache": None}, {}, "NULL"), ({"kv_cache": P + 16}, {}, "ALIGN"), ({"kv_page_bytes": 4616}, {}, "ALIGN"),
    ({"kv_page_bytes": 4576}, {}, "CONFIG"), ({"kv_pages": 0}, {}, "CONFIG"), ({"k_global_scale": 0.0}, {}, "CONFIG"),
    ({"v_global_scale": -1.0}, {}, "CONFIG"), ({}, {"block_size": 6}, "CONFIG"), ({}, {"block_size": 2048}, "CONFIG"),
    ({"kv_page_bytes": 1 << 20}, {"block_size": 24}, "UNSUPPORTED"),
    ({"kv_page_bytes": 1 << 20}, {"block_size": 192}, "UNSUPPORTED")])
def test_attention_refuses_bad_nvfp4_caches(B, caches, kw, err):
    a = attention_args(B, caches, cache_format=B.PA_CACHE_NVFP4, **kw)
    assert B.pre_attn_attention(a, check=False) == getattr(B, "PA_ERR_" + err)


def test_out_over_q_is_refused(B):
    a = attention_args(B, R=2)
    for off in (0, 4096 * 2 * 4 - 16, -4096 * 2 * 4 + 16):
        a.out = P + (1 << 20) + off
        a.q = P + (1 << 20)
        assert B.pre_attn_attention(a, check=False) == B.PA_ERR_ALIAS


def test_out_right_behind_a_slice_of_columns_is_not_an_overlap(B):
    # q: the columns 4096 .. 8191 of rows of 8192, its last row ends where out begins
    a = attention_args(B, R=2, q=P + 4096 * 2, q_stride=8192, out=P + 4 * 8192 * 2, workspace=None)
    assert B.pre_attn_attention(a, check=False) in (B.PA_ERR_WORKSPACE, B.PA_ERR_CUDA)  # the next refusal, or no GPU
    a.out -= 16
    assert B.pre_attn_attention(a, check=False) == B.PA_ERR_ALIAS


@pytest.mark.parametrize("field", ["k_global_scale", "v_global_scale"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_attention_refuses_global_scales_without_a_value(B, field, value):
    a = attention_args(B, {field: value}, cache_format=B.PA_CACHE_NVFP4)
    assert B.pre_attn_attention(a, check=False) == B.PA_ERR_CONFIG


def test_workspace_bytes(B):
    n = B.pre_attn_attention_workspace_bytes(64, 7, 2, 152)
    assert n > 0 and B.pre_attn_attention_workspace_bytes(0, 1, 1, 152) > 0
    assert B.pre_attn_attention_workspace_bytes(64, 7, 2, 160) > n
    for bad in ((-1, 1, 1, 152), (65536, 1, 1, 152), (1, 0, 1, 152), (1, 17, 1, 152), (1, 1, 3, 152), (1, 1, 1, 0)):
        assert B.pre_attn_attention_workspace_bytes(*bad) == 0
