"""Scales of the attention whose product is no f32 number, or rounds to one with fewer bits: refused on the host."""

import pytest


@pytest.mark.parametrize("fmt,sm_scale,q8,k_global,ok", [
    ("nvfp4", 1e30, None, 1e30, False), ("nvfp4", 1e-30, None, 1e-30, False), ("nvfp4", 1e30, None, 1e-30, True),
    ("fp8", 1e20, 1e20, 1.0, False), ("fp8", 1e-20, 1e-20, 1.0, False), ("fp8", 1e20, 1e-20, 1.0, True),
    ("nvfp4", 1e15, 1e15, 1e15, False), ("nvfp4", 1e-15, 1e-15, 1e-15, False), ("nvfp4", 1e-15, 1e15, 1e15, True),
    ("fp8", 3e38, None, 1.0, False),  # x log2(e): above the largest f32
    ("fp8", 2e38, None, 1.0, True), ("fp8", 1e-38, None, 1.0, True), ("fp8", 1e-40, None, 1.0, False),
    ("fp8", 1e30, None, 1e30, True)])  # the FP8 caches have no global scale
def test_the_score_scale_is_a_normal_number(fmt, sm_scale, q8, k_global, ok):
    from indexer_projection_gb300 import binding as B, build
    from tests.test_cache_readers_host import P, attention_args

    build.build()
    kw = dict(q=None, q_fp8=P, q_fp8_scale=q8) if q8 else {}
    a = attention_args(B, {"k_global_scale": k_global}, sm_scale=sm_scale,
                       cache_format=B.PA_CACHE_FP8 if fmt == "fp8" else B.PA_CACHE_NVFP4, **kw)
    assert B.pre_attn_attention(a, check=False) == (B.PA_OK if ok else B.PA_ERR_CONFIG)
