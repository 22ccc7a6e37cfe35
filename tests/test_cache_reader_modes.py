"""The attention in each way its items meet the CTAs: waits that run out, rows of every number, launches in order,
finite values where no key is, caches past 2^32 bytes.

A call takes a cluster of CTAs an item where the table is short; even slices of a persistent grid where it is long (314
blocks: 40 a CTA of the largest cluster, above any limit of blocks times rows); a CTA an item above 2048 items."""

import numpy as np
import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
FORMATS = ["fp8", "nvfp4"]


def attend(case, rd, lists=None):
    out = torch.full((case.M, case.nkv * case.group * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    kw = {} if lists is None else dict(zip(("blocks", "counts"), (torch.from_numpy(x).cuda() for x in lists)))
    rd.attend(case.dev["q"], case.dev["bt"], case.dev["seq"], out, **kw)
    return out


def check(out, case, lists=None, want=None):
    want, tol = want or case.attention(lists)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()


def lengths(mode, q_len):
    if mode == "cluster":
        return [700, 90]
    if mode == "sliced":
        return [40100 + q_len, 23 * 128, 0, 300]
    return list(np.random.default_rng(q_len).integers(q_len, 300, 2100))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("mode", ["cluster", "sliced", "whole"])
@pytest.mark.parametrize("q_len", [1, 2, 4, 7])
def test_a_wait_that_runs_out_in_every_mode(fmt, mode, q_len):
    from indexer_projection_gb300 import binding as B

    c = ref.Case(fmt, lengths(mode, q_len), q_len, 1, 2, seed=60 + q_len).upload()
    rd = c.reader()
    before = attend(c, rd)
    assert rd.device_status() == 0
    late = c.reader(flags=B.PA_FLAG_TEST_WAIT_TIMEOUT)
    out = torch.full_like(before, 3.0)
    late.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out)
    assert late.device_status() == B.PA_DEV_WAIT_TIMEOUT
    assert (out == 3).all()
    after = attend(c, rd)
    assert rd.device_status() == 0 and torch.equal(before, after)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [2, 3, 5, 7, 9])
def test_more_items_than_the_sliced_grid_lists(fmt, q_len):
    g = np.random.default_rng(q_len)
    c = ref.Case(fmt, list(g.integers(q_len, 300, 520 if q_len < 9 else 260)), q_len, 4, 2, seed=70 + q_len).upload()
    rd = c.reader(topk=2)
    check(attend(c, rd), c)
    blocks, counts, lists = ref.random_lists(c, 2, seed=q_len)
    check(attend(c, rd, (blocks, counts)), c, lists)
    assert rd.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("mode", ["cluster", "sliced", "whole"])
@pytest.mark.parametrize("q_len", [1, 3])
def test_launches_in_order_give_the_same_bits(fmt, mode, q_len):
    from indexer_projection_gb300 import binding as B

    c = ref.Case(fmt, lengths(mode, q_len), q_len, 1, 4, seed=80 + q_len).upload()
    early, ordered = c.reader(), c.reader(flags=B.PA_FLAG_NO_PDL)
    outs = [attend(c, rd) for rd in (early, ordered, early, ordered, ordered)]
    assert early.device_status() == 0 and ordered.device_status() == 0
    assert all(torch.equal(outs[0], o) for o in outs[1:]) and outs[0].isfinite().all()


def large_where_no_key_is(case):
    """Largest codes and scales, all finite, in the slots that hold no key (they hold NaN)."""
    if case.fmt == "fp8":
        for w in "kv":
            case.bytes[w][case.bytes[w] == 0x7f] = 0x7e
            case.scales[w][np.isnan(case.scales[w])] = 1e4
    else:
        sf = case.kv[:, :2 * case.nkv * case.bs * 72].reshape(case.pages, 2 * case.nkv, case.bs * 72)[:, :, case.bs * 64:]
        assert (sf == 0xff).any()
        sf[sf == 0xff] = 0x7e
    return case


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,topk", [(1, 1, 0), (1, 2, 3), (3, 1, 0), (4, 2, 3), (7, 1, 4), (9, 1, 0)])
def test_large_finite_values_where_no_key_is(fmt, q_len, nkv, topk):
    c = large_where_no_key_is(ref.Case(fmt, [1000, q_len, 0, 261 + q_len, 128 * 9 + 1], q_len, nkv, 16, seed=90 + q_len)).upload()
    rd = c.reader(topk=topk)
    if topk:
        blocks, counts, lists = ref.random_lists(c, topk, seed=topk)
        check(attend(c, rd, (blocks, counts)), c, lists)
    else:
        check(attend(c, rd), c)
    assert rd.device_status() == 0


def moved(bt, pages, per):
    """A block table's blocks spread over a cache of `pages` pages, `per` a block, from its end down; old -> new ids."""
    old = sorted(set(bt[bt >= 0].tolist()))
    step = pages // per // (2 * len(old))
    return {b: pages // per - 1 - k * step for k, b in enumerate(old)}


def test_fp8_caches_beyond_32_bits():
    from indexer_projection_gb300.runner import PreAttn

    c = ref.Case("fp8", [200, 130], 2, 1, 16, seed=100)
    pages = 2_300_000  # x 2048 bytes = 4.7 GB
    new = moved(c.bt, pages, 8)
    big = {w: torch.zeros(pages, 2048, dtype=torch.uint8, device="cuda") for w in "kv"}
    scales = {w: torch.zeros(pages, 16, device="cuda") for w in "kv"}
    want, bt = c.attention(), c.bt.copy()
    assert max(new.values()) * 8 * 2048 > 2 ** 32
    for old, at in new.items():
        bt[c.bt == old] = at
        for w in "kv":
            big[w][at * 8:at * 8 + 8] = torch.from_numpy(c.bytes[w].reshape(-1, 2048)[old * 8:old * 8 + 8]).cuda()
            scales[w][at * 8:at * 8 + 8] = torch.from_numpy(c.scales[w].reshape(-1, 16)[old * 8:old * 8 + 8]).cuda()
    c.upload()
    c.caches = PreAttn.fp8_caches(big["k"], big["v"], scales["k"], scales["v"], None, pages, 0)
    c.dev["bt"] = torch.from_numpy(bt).cuda()
    rd = c.reader()
    check(attend(c, rd), c, want=want)
    assert rd.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_index_caches_beyond_32_bits(fmt):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader, PreAttn

    block = 128 * (128 if fmt == "fp8" else 72)
    blocks = 4_700_000_000 // block
    small = torch.randint(0, 0x38, (4, block), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).cuda()
    bt = np.array([[3, 0, 1], [2, -1, -1]], np.int32)
    seq = torch.tensor([300, 100], dtype=torch.int32, device="cuda")
    iq = torch.randn(4, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    new = moved(bt, blocks, 1)
    assert max(new.values()) * block > 2 ** 32
    big = torch.zeros(blocks, block, dtype=torch.uint8, device="cuda")
    far = bt.copy()
    for old, at in new.items():
        far[bt == old], big[at] = at, small[old]
    got = []
    for cache, table, n in ((small, bt, 4), (big, far, blocks)):
        caches = (PreAttn.fp8_caches(None, None, None, None, cache, 0, n * 128) if fmt == "fp8" else
                  PreAttn.nvfp4_caches(None, 0, 0, cache, n, block))
        rd = CacheReader(16, 1, cache_format=B.PA_CACHE_FP8 if fmt == "fp8" else B.PA_CACHE_NVFP4, caches=caches, max_requests=2,
                         q_len=2, bt_width=3, block_size=16 if fmt == "fp8" else 128)
        s = torch.zeros(4, 384, device="cuda")
        rd.index_scores(iq, 0, torch.from_numpy(table).cuda(), seq, s)
        assert rd.device_status() == 0
        got.append(s)
    assert torch.equal(got[0], got[1]) and got[0][:, :128].abs().max() > 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,q_len", [(45, 15), (64, 16), (39, 13)])
def test_a_prompt_as_several_requests(fmt, rows, q_len):
    # q_len rows each, the same row of the block table, the length up to their own last row
    from indexer_projection_gb300.runner import CacheReader

    c = ref.Case(fmt, [400 + rows], rows, 2, 8, seed=105).upload()
    n = rows // q_len
    rd = CacheReader(16, 2, cache_format=c.format, caches=c.caches, max_requests=n, q_len=q_len, bt_width=c.W)
    out = torch.full((rows, 16 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    seq = torch.arange(400 + q_len, 400 + rows + 1, q_len, dtype=torch.int32, device="cuda")
    rd.attend(c.dev["q"], c.dev["bt"].repeat(n, 1), seq, out)
    assert rd.device_status() == 0
    check(out, c)
