"""A CacheReader's life: its caches replaced, made on one stream and used on another, dropped early, on a device."""

import gc
import types

import numpy as np
import pytest
import torch

from tests import cache_reference as ref


def attend(case, rd, **kw):
    out = torch.full((case.M, case.nkv * case.group * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    rd.attend(case.dev["q"], case.dev["bt"], case.dev["seq"], out, **kw)
    return out


def check(out, case, want=None):
    want, tol = want or case.attention()
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_other_caches_are_read_by_every_call(fmt):
    a, b = (ref.Case(fmt, [300, 130], 1, 1, 16, seed=s).upload() for s in (51, 52))
    b.dev["q"], b.q = a.dev["q"], a.q
    rd = a.reader()
    check(attend(a, rd), a)
    assert rd.caches is a.caches
    rd.caches = b.caches
    assert rd.caches is b.caches
    check(attend(b, rd), b)
    assert rd.device_status() == 0
    # the scores of one index cache, then of another
    keys = [torch.randint(0, 0x38, (512, 128 if fmt == "fp8" else 72), dtype=torch.uint8, device="cuda") for _ in "ab"]
    seq, bt = torch.tensor([200], dtype=torch.int32, device="cuda"), torch.tensor([[2, 1]], dtype=torch.int32, device="cuda")
    iq = torch.ones(1, 128, dtype=torch.bfloat16, device="cuda")
    got = []
    from indexer_projection_gb300.runner import CacheReader, PreAttn
    held = [PreAttn.fp8_caches(None, None, None, None, k, 0, 512) if fmt == "fp8" else PreAttn.nvfp4_caches(None, 0, 0, k, 32, 1152)
            for k in keys]
    for first in (0, 1):
        rd = CacheReader(16, 1, cache_format=a.format, caches=held[first], max_requests=1, q_len=1, bt_width=2)
        for k in (first, 1 - first):
            rd.caches = held[k]
            s = torch.zeros(1, 256, device="cuda")
            rd.index_scores(iq, 0, bt, seq, s)
            got.append(s)
    assert torch.equal(got[0], got[3]) and torch.equal(got[1], got[2]) and not torch.equal(got[0], got[1])


@pytest.mark.gpu
def test_made_on_a_busy_stream_and_used_on_another():
    # the status word is clear before the first call of another stream raises a bit in it
    from indexer_projection_gb300 import binding as B

    c = ref.Case("fp8", [300, 500], 1, 1, 16, seed=53).upload()
    c.dev["seq"] = torch.tensor([128 * c.W + 1, 500], dtype=torch.int32, device="cuda")  # longer than its table
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(300_000_000)
    rd = c.reader()
    with torch.cuda.stream(s):
        attend(c, rd)
    torch.cuda.synchronize()
    assert rd.device_status() == B.PA_DEV_SLOT_RANGE


@pytest.mark.gpu
def test_not_made_in_a_capture():
    c = ref.Case("fp8", [300], 1, 1, 16, seed=54).upload()
    x = torch.zeros(8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="capture"):
            c.reader()
        x += 1
    g.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()
    check(attend(c, c.reader()), c)


@pytest.mark.gpu
@pytest.mark.parametrize("made_on_side", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_dropped_while_its_call_runs(made_on_side, given):
    # the workspace goes back to the allocator, but not to another stream's tensors before the call is done
    c = ref.Case("nvfp4", [40000, 300], 1, 1, 16, seed=55).upload()
    want = c.attention()
    side = torch.cuda.Stream()
    used, made = (torch.cuda.default_stream(), side) if made_on_side else (side, torch.cuda.default_stream())
    with torch.cuda.stream(made):
        rd = c.reader()
    at, size = rd.workspace.data_ptr(), rd.workspace.numel()
    warm = c.reader()  # (loading the kernels waits for the device; it stays, so that its workspace is not handed out)
    check(attend(c, warm), c, want)
    out = torch.full((c.M, 2048), float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(used):
        torch.cuda._sleep(300_000_000)
    if given:
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, stream=used)
    else:
        with torch.cuda.stream(used):
            rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out)
    del rd
    gc.collect()
    with torch.cuda.stream(made):
        other = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert not used.query() and other.data_ptr() != at
        other.fill_(0xff)
    torch.cuda.synchronize()
    check(out, c, want)


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_a_device_without_cuda_is_refused(device):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader

    with pytest.raises(ValueError, match="CUDA device"):
        CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), max_requests=1, q_len=1, bt_width=1, device=device)


@pytest.mark.gpu
def test_a_stream_of_another_device_is_refused():
    c = ref.Case("fp8", [300], 1, 1, 16, seed=56).upload()
    rd = c.reader(device="cuda")
    with pytest.raises(ValueError, match="another device"):
        attend(c, rd, stream=types.SimpleNamespace(cuda_stream=0, device_index=1))
    check(attend(c, rd, stream=torch.cuda.current_stream()), c)
    check(attend(c, rd, stream=torch.cuda.current_stream().cuda_stream), c)
