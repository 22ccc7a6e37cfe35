"""Refusals of pre_attn_attention_ext, without a GPU: each documented error comes back before anything is launched."""

import pytest

from tests.test_cache_readers_host import P, attention_args


@pytest.fixture(scope="module")
def B():
    from indexer_projection_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def ext(B, **kw):
    d = dict(window=100, sinks=4, weights=P + (1 << 28), weights_stride=3, weights_before=P + (1 << 29), before_stride=3, decay=1.0,
             workspace=P + (1 << 30), workspace_bytes=1 << 30)
    d.update(kw)
    return B.pa_attention_ext(**d)


def call(B, e, **kw):
    return B.pre_attn_attention_ext(attention_args(B, **dict(dict(blocks=None, counts=None), **kw)), e, check=False)


def test_nothing_to_do_is_accepted(B):
    assert call(B, ext(B)) == B.PA_OK
    assert call(B, ext(B, weights=None)) == B.PA_OK
    assert call(B, ext(B, weights=None, window=0, sinks=0)) == B.PA_OK
    assert call(B, ext(B, window=0, sinks=0), blocks=P, counts=P) == B.PA_OK
    assert B.load().pre_attn_attention_ext(None, ext(B), None) == B.PA_ERR_NULL
    assert B.load().pre_attn_attention_ext(attention_args(B), None, None) == B.PA_ERR_NULL


@pytest.mark.parametrize("e,kw,err", [
    (dict(window=-1), {}, "CONFIG"), (dict(sinks=-1), {}, "CONFIG"), (dict(window=0), {}, "CONFIG"),
    *[(dict(decay=v), {}, "CONFIG") for v in (-0.5, float("inf"), float("nan"))], ({}, dict(blocks=P, counts=P), "UNSUPPORTED"),
    (dict(weights_stride=2), {}, "SHAPE"), (dict(before_stride=2), {}, "SHAPE"), (dict(weights=P + (1 << 28) + 2), {}, "ALIGN"),
    (dict(weights_before=P + 2), {}, "ALIGN"), ({}, dict(q=None), "CONFIG"), ({}, dict(seq_lens=None), "NULL"), ({}, dict(R=-1), "SHAPE"),
    ({}, dict(bt_width=16385), "SHAPE"), ({}, dict(out=P + (1 << 24) + 8), "ALIGN")])
def test_refusals(B, e, kw, err):
    assert call(B, ext(B, **e), **kw) == getattr(B, "PA_ERR_" + err)


def test_bytes(B):
    n = B.pre_attn_attention_weights_bytes
    assert n(64, 7, 32, 2, 256) == 64 * 7 * 2 * 256 * 16 * 4
    assert n(8, 1, 5, 1, 10) == 8 * 10 * 4 * 8 * 4  # four parts of a block, five heads in eight places
    assert n(8, 3, 16, 1, 10) == 8 * 3 * 10 * 2 * 16 * 4
    assert n(0, 1, 16, 1, 1) > 0
    for bad in ((-1, 1, 16, 1, 1), (65536, 1, 16, 1, 1), (1, 0, 16, 1, 1), (1, 17, 16, 1, 1), (1, 1, 17, 1, 1), (1, 1, 0, 1, 1),
                (1, 1, 16, 3, 1), (1, 1, 15, 2, 1), (1, 1, 16, 1, 0), (1, 1, 16, 1, 16385)):
        assert n(*bad) == 0


def test_a_packed_struct_holds_what_its_fields_do():
    from indexer_projection_gb300 import binding as B

    for cls in (B.pa_evict_args, B.pa_verify_args):
        fill, args = B.packed(cls)
        values = [2 ** 40 + k if t is B.ctypes.c_void_p else -k if t is B.ctypes.c_int64 else k - 5
                  for k, (_, t) in enumerate(cls._fields_)]
        for _ in range(2):
            fill(*values)
            assert [getattr(args, name) for name, _ in cls._fields_] == values
            values[0] += 1
