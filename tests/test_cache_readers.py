"""GPU parity of what is read back of the caches (pre_attn_index_scores_nvfp4,
pre_attn_select_blocks, pre_attn_attention) with the 64-bit reference."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu


def attend(case, lists=None, topk=0, q=None, out=None, reader=None, **kw):
    rd = reader or case.reader(topk=topk)
    wide = case.nkv * case.group * 128
    out = torch.full((case.M, wide), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    q = case.dev["q"] if q is None else q
    if lists is None:
        rd.attend(q, case.dev["bt"], case.dev["seq"], out, **kw)
    else:
        blocks, counts = (torch.from_numpy(x).cuda() for x in lists)
        rd.attend(q, case.dev["bt"], case.dev["seq"], out, blocks=blocks, counts=counts, **kw)
    torch.cuda.synchronize()
    return out[:, :wide].double().cpu().numpy(), rd.device_status()


def close(got, want):
    out, tol = want
    assert np.isfinite(got).all()
    over = np.abs(got - out) - tol
    assert (over <= 0).all(), f"max excess {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"


FORMATS = ["fp8", "nvfp4"]


# ------------------------------------------------------------- the attention

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 700])
def test_one_row_of_every_length(fmt, n):
    c = ref.Case(fmt, [n], 1, seed=n).upload()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,group", [(1, 1, 16), (2, 2, 16), (3, 1, 8), (4, 4, 5), (5, 2, 1), (7, 2, 16),
                                             (8, 1, 13), (9, 1, 16), (13, 2, 4), (16, 1, 16)])
def test_rows_and_heads(fmt, q_len, nkv, group):
    c = ref.Case(fmt, [q_len, 300, 0, 129 + q_len, 640], q_len, nkv, group, seed=q_len, extra_width=2,
                 k_global=0.5, v_global=1.5).upload()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 3), (1, 16), (2, 16), (3, 5), (4, 2), (6, 1), (8, 16), (9, 3), (16, 4)])
def test_requests_that_few_sms_share(fmt, q_len, group):
    # tables of two to thirteen blocks: joined by SMs that meet, two to eight of them, or by a kernel of their own
    for blocks in (2, 3, 5, 7, 8, 9, 13):
        c = ref.Case(fmt, [128 * blocks - 5, max(q_len, 64 * blocks), 0], q_len, 1, group, seed=100 + blocks).upload()
        got, status = attend(c)
        assert status == 0
        close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,topk", [(1, 1, 1), (1, 2, 4), (2, 1, 3), (4, 2, 5), (7, 2, 4), (8, 1, 6), (11, 1, 3)])
def test_selected_blocks(fmt, q_len, nkv, topk):
    c = ref.Case(fmt, [1000, q_len, 0, 260 + q_len, 128 * 9], q_len, nkv, 16, seed=100 + q_len).upload()
    blocks, counts, lists = ref.random_lists(c, topk, seed=topk)
    got, status = attend(c, (blocks, counts), topk)
    assert status == 0
    close(got, c.attention(lists))


@pytest.mark.parametrize("fmt,bs,kps,pad", [("fp8", 16, 16, 0), ("fp8", 16, 9, 0), ("nvfp4", 4, 8, 32), ("nvfp4", 8, 8, 0),
                                            ("nvfp4", 32, 8, 64), ("nvfp4", 64, 8, 0), ("nvfp4", 128, 8, 96),
                                            ("nvfp4", 256, 8, 0), ("nvfp4", 1024, 8, 32)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_page_layouts(fmt, bs, kps, pad, q_len):
    c = ref.Case(fmt, [700, 90, 1300], q_len, 2, 8, bs=bs, kps=kps, pad=pad, seed=bs + kps).upload()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 4, 6])
def test_long_requests_shared_by_every_sm(fmt, q_len):
    # two requests over all SMs: each is split many times and joined
    c = ref.Case(fmt, [40000 + q_len, 23 * 128], q_len, 1, 16, seed=7).upload()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
def test_more_items_than_the_sliced_grid_lists(fmt):
    g = np.random.default_rng(1)
    seq = g.integers(0, 200, 2100)
    c = ref.Case(fmt, list(seq), 1, 1, 2, seed=3).upload()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())
    blocks, counts, lists = ref.random_lists(c, 2, seed=5)
    got, status = attend(c, (blocks, counts), 2)
    assert status == 0
    close(got, c.attention(lists))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 5])
def test_rows_that_select_nothing_or_a_block_twice(fmt, q_len):
    c = ref.Case(fmt, [900, 500], q_len, 1, 16, seed=11).upload()
    blocks = np.full((c.M, 1, 6), -1, np.int32)
    counts = np.zeros((c.M, 1), np.int32)
    lists = [[[]] for _ in range(c.M)]
    blocks[0, 0, :5], counts[0] = [2, 0, 2, 1, 0], 5
    lists[0] = [[0, 1, 2]]
    got, status = attend(c, (blocks, counts), 6)
    assert status == 0
    close(got, c.attention(lists))
    assert (got[1:] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_ids_are_skipped_and_flagged(fmt):
    from indexer_projection_gb300 import binding as B

    c = ref.Case(fmt, [900, 500], 2, 1, 16, seed=12).upload()
    blocks, counts, lists = ref.random_lists(c, 4, seed=2)
    # a block after the row's last, a negative one, a count beyond topk
    blocks[0, 0], counts[0] = [1, 7000, -5, 3], 4
    lists[0] = [[1, 3]]
    counts[1] = 99
    lists[1] = [[int(b) for b in blocks[1, 0]]]
    got, status = attend(c, (blocks, counts), 4)
    assert status == B.PA_DEV_SLOT_RANGE
    close(got, c.attention(lists))
    # a table entry outside the cache: that block is skipped
    c.bt[1, 2] = c.pool + 4
    c.dev["bt"] = torch.from_numpy(c.bt).cuda()
    got, status = attend(c)
    assert status == B.PA_DEV_SLOT_RANGE
    c.bt[1, 2] = -1
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
def test_requests_shorter_than_their_rows_or_longer_than_the_table(fmt):
    from indexer_projection_gb300 import binding as B

    c = ref.Case(fmt, [300, 300, 300], 3, 1, 16, seed=13).upload()
    c.seq[:] = [2, 300, 128 * c.W + 1]
    c.dev["seq"] = torch.from_numpy(c.seq).cuda()
    got, status = attend(c)
    assert status == B.PA_DEV_SLOT_RANGE
    close(got, c.attention())
    assert (got[:3] == 0).all() and (got[6:] == 0).all()
    c.seq[:] = [-4, 300, 0]
    c.dev["seq"] = torch.from_numpy(c.seq).cuda()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


def test_strides_and_columns_behind_the_rows():
    c = ref.Case("fp8", [300, 20], 2, 2, 4, seed=14).upload()
    wide = 8 * 128
    q = torch.full((c.M, wide + 48), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:, :wide] = c.dev["q"]
    out = torch.full((c.M + 1, wide + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    rd = c.reader()
    rd.attend(q, c.dev["bt"], c.dev["seq"], out[:c.M])
    torch.cuda.synchronize()
    close(out[:c.M, :wide].double().cpu().numpy(), c.attention())
    assert (out[:, wide:] == 7).all() and (out[c.M] == 7).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_fp8_queries(fmt):
    c = ref.Case(fmt, [400, 77], 3, 1, 16, seed=15).upload()
    q8 = (c.q.float() / 0.25).to(torch.float8_e4m3fn)
    got, status = attend(c, q=q8.cuda(), q_fp8_scale=0.25)
    assert status == 0
    close(got, c.attention(q=q8.float() * 0.25))


def test_query_magnitudes():
    # head rows from 2^-90 to 2^60, one of zeros: a row's own power of two keeps its values
    c = ref.Case("fp8", [333], 1, 1, 16, seed=16, q_scale=1.0)
    scale = torch.tensor([2.0 ** e for e in (-90, -40, -20, -6, -3, -2, -1, 0, 0, 0, 1, 1, 2, 2, 3, 3)])
    scale[4] = 0.0
    c.q = (c.q.float().view(16, 128) * scale[:, None]).to(torch.bfloat16).view(1, -1)
    c.upload()
    got, status = attend(c)
    close(got, c.attention())
    # and a score scale that undoes a large one
    c.q = (c.q.float() * 2.0 ** 60).to(torch.bfloat16)
    c.upload()
    got, _ = attend(c, reader=c.reader(sm_scale=2.0 ** -60 * 128 ** -0.5))
    close(got, c.attention(sm_scale=2.0 ** -60 * 128 ** -0.5))


@pytest.mark.parametrize("q_len", [1, 3])
def test_value_scales_far_apart(q_len):
    # V scales over 2^24, a zero value row with scale 1 that takes nearly all the weight
    c = ref.Case("fp8", [500], q_len, 1, 16, seed=17, spread=24.0)
    c.upload()
    got, _ = attend(c)
    close(got, c.attention())
    c = ref.Case("fp8", [500], 1, 1, 16, seed=18)
    slot = int(c.bt[0, 0]) * 128
    page, t = slot // 16, 0
    c.bytes["v"][page * 2048 + np.arange(128) * 16 + t] = 0
    c.scales["v"][page * 16 + t] = 1.0
    c.v[0, slot], c.vs[0, slot] = 0.0, 1.0
    c.q = torch.from_numpy(np.tile(c.k[0, slot] * 0.75, 16)[None]).float().to(torch.bfloat16)  # a lead of about 2^12
    c.upload()
    got, _ = attend(c)
    close(got, c.attention())


def test_peaked_rows():
    c = ref.Case("nvfp4", [3000], 1, 1, 16, seed=19, q_scale=12.0).upload()
    got, _ = attend(c)
    close(got, c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_in_a_row_stays_in_it(fmt):
    c = ref.Case(fmt, [300, 200], 2, 1, 16, seed=20)
    c.q[1, 5 * 128 + 3] = float("nan")
    c.upload()
    got, _ = attend(c)
    assert np.isnan(got[1, 5 * 128:6 * 128]).all()
    got[1, 5 * 128:6 * 128] = 0
    c.q[1, 5 * 128 + 3] = 0.0
    out, tol = c.attention()
    out[1, 5 * 128:6 * 128] = 0
    close(got, (out, tol + 1e-30))


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_on_another_stream(fmt):
    c = ref.Case(fmt, [1000, 64, 5000], 2, 2, 16, seed=21).upload()
    blocks, counts, lists = ref.random_lists(c, 5, seed=3)
    tb, tc = torch.from_numpy(blocks).cuda(), torch.from_numpy(counts).cuda()
    rd = c.reader(topk=5)
    dense, sparse = (torch.zeros(c.M, 32 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], dense)
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], sparse, blocks=tb, counts=tc)
    s.synchronize()
    want = (c.attention(), c.attention(lists))
    close(dense.double().cpu().numpy(), want[0])
    close(sparse.double().cpu().numpy(), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], dense)
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], sparse, blocks=tb, counts=tc)
    first = dense.clone(), sparse.clone()
    for _ in range(3):
        dense.fill_(9), sparse.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dense, first[0]) and torch.equal(sparse, first[1])  # the same bits every time


@pytest.mark.parametrize("fmt,q_len", [("fp8", 1), ("fp8", 7), ("nvfp4", 3)])
def test_a_wait_that_runs_out_is_reported(fmt, q_len):
    from indexer_projection_gb300 import binding as B

    c = ref.Case(fmt, [700, 90], q_len, 1, 16, seed=22).upload()
    out = torch.full((c.M, 2048), 3.0, dtype=torch.bfloat16, device="cuda")
    got, status = attend(c, reader=c.reader(flags=B.PA_FLAG_TEST_WAIT_TIMEOUT), out=out)
    assert status == B.PA_DEV_WAIT_TIMEOUT
    assert (got == 3).all()
    got, status = attend(c)
    assert status == 0
    close(got, c.attention())


def test_two_readers_at_once():
    # two host threads, a reader and a stream each: what one does is not seen by the other
    import threading
    cases = [ref.Case(f, [3000, 900], q, 2, 16, seed=90 + q).upload() for f, q in (("fp8", 1), ("nvfp4", 3))]
    outs = [torch.zeros(c.M, 32 * 128, dtype=torch.bfloat16, device="cuda") for c in cases]
    torch.cuda.synchronize()

    def work(c, out):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            rd = c.reader()
            for _ in range(20):
                rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out)
            assert rd.device_status() == 0
        s.synchronize()

    threads = [threading.Thread(target=work, args=(c, o)) for c, o in zip(cases, outs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for c, out in zip(cases, outs):
        close(out.double().cpu().numpy(), c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
def test_what_the_reader_refuses(fmt):
    c = ref.Case(fmt, [300, 20], 2, 1, 16, seed=95).upload()
    rd = c.reader(topk=2)
    out = torch.zeros(c.M, 2048, dtype=torch.bfloat16, device="cuda")
    lists, counts = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((c.M, 1, 2), (c.M, 1)))
    q, bt, seq = c.dev["q"], c.dev["bt"], c.dev["seq"]
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(q=q[1:]), dict(q=q[:, :-128]), dict(bt=bt.cpu()), dict(bt=bt.long()),
                dict(bt=bt[:, 1:]), dict(seq=seq.cpu()), dict(seq=seq.long()), dict(out=out.cpu()), dict(out=out.float()),
                dict(blocks=lists), dict(counts=counts), dict(blocks=lists.cpu(), counts=counts),
                dict(blocks=lists, counts=counts.cpu()), dict(blocks=lists[:, :, :1], counts=counts)):
        a = dict(dict(q=q, bt=bt, seq=seq, out=out), **bad)
        with pytest.raises(ValueError):
            rd.attend(a["q"], a["bt"], a["seq"], a["out"], blocks=a.get("blocks"), counts=a.get("counts"))
    with pytest.raises(ValueError):  # a reader of every block alone
        c.reader().attend(q, bt, seq, out, blocks=lists[:, :, :0], counts=counts)
    scores = torch.zeros(1, c.M, c.W * 128, device="cuda")
    for bad in (dict(scores=scores.cpu()), dict(seq=seq.cpu()), dict(blocks=lists.cpu()), dict(counts=counts.cpu()),
                dict(scores=scores.half()), dict(scores=scores[0])):
        a = dict(dict(scores=scores, seq=seq, blocks=lists, counts=counts), **bad)
        with pytest.raises(ValueError):
            rd.select_blocks(a["scores"], a["seq"], a["blocks"], a["counts"])
    iq = torch.zeros(c.M, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(iq=iq.cpu()), dict(head=1), dict(bt=bt.cpu()), dict(scores=scores[0].cpu())):
        a = dict(dict(iq=iq, head=0, bt=bt, seq=seq, scores=scores[0]), **bad)
        with pytest.raises(ValueError):
            rd.index_scores(a["iq"], a["head"], a["bt"], a["seq"], a["scores"])
    assert rd.device_status() == 0 and not out.any()


def test_a_call_without_requests_does_nothing():
    c = ref.Case("fp8", [300], 1, 1, 16, seed=96).upload()
    rd = c.reader(topk=2)
    none = {k: c.dev[k][:0] for k in ("q", "bt", "seq")}
    out = torch.zeros(0, 2048, dtype=torch.bfloat16, device="cuda")
    lists, counts = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((0, 1, 2), (0, 1)))
    assert rd.attend(none["q"], none["bt"], none["seq"], out) == 0
    assert rd.attend(none["q"], none["bt"], none["seq"], out, blocks=lists, counts=counts) == 0
    scores = torch.zeros(1, 0, c.W * 128, device="cuda")
    assert rd.index_scores(none["q"][:, :128], 0, none["bt"], none["seq"], scores[0]) == 0
    assert rd.select_blocks(scores, none["seq"], lists, counts) == 0
    assert rd.device_status() == 0


def test_the_caches_are_read_at_the_call():
    # a reader whose caches' struct is given its fields after the reader was made
    c = ref.Case("nvfp4", [300, 130], 1, 1, 16, seed=97).upload()
    fields = [f for f, _ in c.caches._fields_]
    kept = {f: getattr(c.caches, f) for f in fields}
    for f in fields:
        setattr(c.caches, f, None if "cache" in f else 0)
    rd = c.reader()
    for f in fields:
        setattr(c.caches, f, kept[f])
    got, status = attend(c, reader=rd)
    assert status == 0
    close(got, c.attention())


def test_offsets_beyond_32_bits():
    # pages past 2^31 bytes of a cache, and past 2^32
    c = ref.Case("nvfp4", [200, 130], 1, 1, 16, bs=128, seed=23, stale="zero")
    pages = 300000  # x 18432 bytes = 5.5 GB
    big = torch.zeros(pages, c.page_bytes, dtype=torch.uint8, device="cuda")
    move = {int(b): pages - 1 - 70000 * k for k, b in enumerate(sorted(set(c.bt[c.bt >= 0].tolist())))}
    for old, new in move.items():
        big[new] = torch.from_numpy(c.kv[old]).cuda()
    want = c.attention()
    bt = c.bt.copy()
    for old, new in move.items():
        bt[c.bt == old] = new
    c.upload()
    from indexer_projection_gb300.runner import PreAttn
    c.caches = PreAttn.nvfp4_caches(big, pages, c.page_bytes, None, 0, 0)
    c.dev["bt"] = torch.from_numpy(bt).cuda()
    got, status = attend(c)
    assert status == 0
    close(got, want)


@pytest.mark.parametrize("fmt,R,q_len,nkv,topk", [("fp8", 48, 1, 2, 0), ("nvfp4", 24, 1, 4, 0), ("fp8", 12, 7, 2, 0),
                                                  ("nvfp4", 12, 4, 2, 0), ("fp8", 64, 7, 2, 16), ("nvfp4", 64, 6, 2, 16),
                                                  ("fp8", 200, 2, 1, 12)])
def test_many_blocks_a_cta(fmt, R, q_len, nkv, topk):
    """Enough blocks that every CTA's ring goes round many times, ragged requests; the reference in 64 bits on the GPU."""
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader, PreAttn

    g = torch.Generator(device="cuda").manual_seed(R + q_len)
    dev, D = "cuda", 128
    seq = torch.randint(q_len, 20000, (R,), generator=g, device=dev, dtype=torch.int32)
    W = (20000 + 127) // 128
    nb = (seq + 127) // 128
    pool = int(nb.sum())
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    bt = torch.full((R, W), -1, dtype=torch.int32, device=dev)
    bt[torch.arange(W, device=dev) < nb[:, None]] = perm
    q = (torch.randn(R * q_len, nkv * 16 * D, generator=g, device=dev) * 0.5).to(torch.bfloat16)
    e4m3 = torch.from_numpy(np.nan_to_num(ref.E4M3)).to(dev)
    slots = pool * 128
    s_ = torch.arange(slots, device=dev)[:, None]
    d = torch.arange(D, device=dev)
    if fmt == "fp8":
        code = [torch.randint(0, 0x70, (slots // 16 * nkv * 2048,), generator=g, device=dev, dtype=torch.uint8) for _ in "kv"]
        for x in code:
            x |= torch.randint(0, 2, x.shape, generator=g, device=dev, dtype=torch.uint8) << 7
        scale = [torch.rand(slots // 16 * nkv * 16, generator=g, device=dev) * 0.02 + 0.001 for _ in "kv"]
        caches, form, bs = PreAttn.fp8_caches(*code, *scale, None, slots // 16, 0), B.PA_CACHE_FP8, 16

        def kv(h, slot):
            p, t = (slot // 16 * nkv + h)[:, None], (slot % 16)[:, None]
            k = e4m3[code[0][p * 2048 + d // 16 * 256 + t * 16 + d % 16].long()] * scale[0][p * 16 + t].double()
            return k, e4m3[code[1][p * 2048 + d * 16 + t].long()] * scale[1][p * 16 + t].double()
    else:
        bs = 32
        page = 2 * nkv * bs * 72
        cache = torch.randint(0, 256, (slots // bs, page), generator=g, device=dev, dtype=torch.uint8)
        sf = cache.view(slots // bs, 2 * nkv, bs * 72)[:, :, bs * 64:]
        sf.copy_(torch.randint(0x20, 0x38, sf.shape, generator=g, device=dev, dtype=torch.uint8))
        caches, form = PreAttn.nvfp4_caches(cache, slots // bs, page, None, 0, 0), B.PA_CACHE_NVFP4
        flat, e2m1 = cache.view(-1), torch.from_numpy(ref.E2M1).to(dev)

        def kv(h, slot):
            out = []
            for sl in (2 * h, 2 * h + 1):
                base, t, grp = (slot // bs * page + sl * bs * 72)[:, None], (slot % bs)[:, None], d // 16
                byte = flat[base + t * 64 + d // 2].long()
                at = (t // 4 * 4 + grp // 2) * 8 + grp % 2 * 4 + t % 4 if sl % 2 else t * 8 + grp
                out.append(e2m1[torch.where(d % 2 == 0, byte & 15, byte >> 4)] * e4m3[flat[base + bs * 64 + at].long()])
            return out
    rd = CacheReader(16 * nkv, nkv, cache_format=form, caches=caches, max_requests=R, q_len=q_len, bt_width=W, topk=topk,
                     block_size=bs)
    kw = {}
    if topk:
        pos = (seq.long()[:, None] - q_len + torch.arange(q_len, device=dev)).view(-1, 1, 1)
        order = torch.rand(R * q_len, nkv, W, generator=g, device=dev)
        order[:, :, :4] += 1  # blocks that most rows share
        order = torch.where(torch.arange(W, device=dev) <= pos // 128, order, -1.0)
        val, top = order.topk(topk, dim=-1)
        kw["blocks"] = torch.where(val >= 0, top, -1).to(torch.int32)
        kw["counts"] = (val >= 0).sum(-1).to(torch.int32)
    outs = []
    for _ in range(3):
        out = torch.full((R * q_len, nkv * 16 * D), float("nan"), dtype=torch.bfloat16, device=dev)
        rd.attend(q, bt, seq, out, **kw)
        outs.append(out)
    torch.cuda.synchronize()
    assert rd.device_status() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for r in range(R):
        n = int(seq[r])
        j = torch.arange(n, device=dev)
        slot = bt[r, j // 128].long() * 128 + j % 128
        for h in range(nkv):
            k, v = kv(h, slot)
            for i in range(q_len):
                m = r * q_len + i
                live = j <= n - q_len + i
                if topk:
                    live = live & torch.isin(j // 128, kw["blocks"][m, h].long())
                w = torch.softmax(q[m].view(nkv, 16, D)[h].double() @ k[live].T * D ** -0.5, -1)
                want, mass = w @ v[live], w @ v[live].abs()
                # as ref.Case.attention's bound: 2^-11 a weight's rounding, 2^-8 the output's, the scores' errors below 2^-12
                tol = 2.0 ** -10 * mass + 2.0 ** -8 * want.abs() + 1e-6 * v.abs().max()
                got = outs[0][m].view(nkv, 16, D)[h].double()
                assert ((got - want).abs() <= tol).all(), (r, h, i, float(((got - want).abs() - tol).max()))


# ------------------------------------------------------------- the selection

def run_select(scores, seq, q_len, init, local, topk, W):
    from indexer_projection_gb300.runner import CacheReader
    from indexer_projection_gb300 import binding as B

    H, M = scores.shape[:2]
    rd = CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), max_requests=max(len(seq), 1), q_len=q_len,
                     bt_width=W, topk=topk, init_blocks=init, local_blocks=local)
    blocks = torch.full((M, H, topk), -77, dtype=torch.int32, device="cuda")
    counts = torch.full((M, H), -77, dtype=torch.int32, device="cuda")
    rd.select_blocks(torch.from_numpy(scores).cuda(), torch.from_numpy(np.array(seq, np.int32)).cuda(), blocks, counts)
    torch.cuda.synchronize()
    return blocks.cpu().numpy(), counts.cpu().numpy(), rd.device_status()


def check_select(scores, seq, q_len, init, local, topk, W, status=0):
    blocks, counts, st = run_select(scores, seq, q_len, init, local, topk, W)
    assert st == status
    want = ref.select(scores, seq, q_len, W, init, local, topk)
    for m, rows in enumerate(want):
        for h, b in enumerate(rows):
            assert counts[m, h] == len(b), (m, h)
            assert blocks[m, h].tolist() == b + [-1] * (topk - len(b)), (m, h)


@pytest.mark.parametrize("q_len,H,init,local,topk,W,spare", [(1, 1, 1, 4, 16, 60, 0), (3, 2, 0, 1, 5, 9, 4), (7, 4, 2, 3, 8, 40, 128),
                                                             (16, 1, 0, 0, 1, 17, 0), (2, 3, 1, 1, 256, 300, 0)])
def test_selection(q_len, H, init, local, topk, W, spare):
    g = np.random.default_rng(topk)
    seq = [W * 128, q_len, 0, 129 + q_len, W * 64 + 5]
    s = g.standard_normal((H, len(seq) * q_len, W * 128 + spare)).astype(np.float32)
    check_select(s, seq, q_len, init, local, topk, W)
    # few values: ties everywhere, both zeros among them
    s = (g.integers(-1, 2, s.shape) * 0.25).astype(np.float32)
    s[s == 0] *= -1.0
    s[..., ::2][s[..., ::2] == 0] = 0.0
    check_select(np.sign(s) * np.abs(s), seq, q_len, init, local, topk, W)


def test_selection_of_extreme_scores():
    W, g = 24, np.random.default_rng(0)
    s = g.standard_normal((1, 6, W * 128)).astype(np.float32)
    big = np.finfo(np.float32).max
    s[0, 0, 128 * 3:128 * 9] = -np.inf               # blocks that are masked
    s[0, 1] = -np.inf                                # a row without any
    s[0, 2] = -big                                   # the type's lowest value is a score
    s[0, 3] = np.nan
    s[0, 3, 128 * 5 + 7] = -3.0                      # one number among NaN
    s[0, 4, 128 * 4 + 1], s[0, 4, 128 * 6 + 1], s[0, 4, 128 * 8 + 9] = np.inf, big, np.nan
    s[0, 5] = np.where(np.arange(W * 128) % 128 == 100, 1e-45, -1e-45)
    for topk in (1, 4, 24, 40):
        check_select(s, [W * 128] * 6, 1, 0, 1, topk, W)


def test_selection_of_long_rows_and_bad_requests():
    from indexer_projection_gb300 import binding as B

    W, g = 2500, np.random.default_rng(5)
    s = g.standard_normal((2, 2, W * 128)).astype(np.float32)
    s = np.round(s * 8) / 8  # thousands of equal maxima
    check_select(s, [W * 128 - 3], 2, 1, 4, 64, W)
    check_select(s[:, :, :4 * 128], [1], 2, 1, 1, 4, 4, status=B.PA_DEV_SLOT_RANGE)
    check_select(s[:, :, :4 * 128], [513], 2, 1, 1, 4, 4, status=B.PA_DEV_SLOT_RANGE)


# ---------------------------------------------------------- the NVFP4 scores

class Keys:
    """An NVFP4 index cache: 64 code and 8 scale bytes a token, NaN scales where no key is."""

    def __init__(self, seq, bs, pad, seed, extra_width=0):
        g = np.random.default_rng(seed)
        self.seq = np.array(seq, np.int32)
        nb = (np.maximum(self.seq, 0) + 127) // 128
        self.W = int(max(nb.max(initial=0), 1)) + extra_width
        per = 1 if bs <= 128 else bs // 128
        pool = (int(nb.sum()) + 2 + per) // per * per
        perm = g.permutation(pool)
        self.bt = np.full((len(seq), self.W), -1, np.int32)
        at = 0
        for r, n in enumerate(nb):
            self.bt[r, :n] = perm[at:at + n]
            at += n
        self.bs, self.page_bytes, self.pages, self.pool = bs, bs * 72 + pad, pool * 128 // bs, pool
        self.cache = np.full((self.pages, self.page_bytes), 0xff, np.uint8)
        self.keys = np.full((pool * 128, 128), np.nan)
        for r, n in enumerate(self.seq):
            j = np.arange(max(int(n), 0))
            slot = self.bt[r, j // 128].astype(np.int64) * 128 + j % 128
            nib = g.integers(0, 16, (len(j), 128)).astype(np.uint8)
            sf = torch.from_numpy(np.exp2(g.random((len(j), 8)) * 6 - 5)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            base = (slot // bs * self.page_bytes)[:, None]
            t = (slot % bs)[:, None]
            flat = self.cache.reshape(-1)
            flat[base + t * 64 + np.arange(64)] = nib[:, 0::2] | (nib[:, 1::2] << 4)
            flat[base + bs * 64 + t * 8 + np.arange(8)] = sf
            self.keys[slot] = ref.E2M1[nib] * np.repeat(ref.E4M3[sf], 16, axis=1)


def check_scores(seq, q_len, init, local, bs=16, pad=0, n_iq=1, head=0, seed=0, spare=0, bad=None, iq_scale=1.0):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader, PreAttn

    k = Keys(seq, bs, pad, seed, extra_width=1)
    if bad is not None:
        k.bt[bad] = k.pool + 3
    g = np.random.default_rng(seed + 1)
    M = len(seq) * q_len
    iq = ref.bf16(g.standard_normal((M, n_iq * 128)) * iq_scale)
    cache = torch.from_numpy(k.cache).cuda()
    rd = CacheReader(16, 1, cache_format=B.PA_CACHE_NVFP4, caches=PreAttn.nvfp4_caches(None, 0, 0, cache, k.pages, k.page_bytes),
                     max_requests=max(len(seq), 1), q_len=q_len, bt_width=k.W, init_blocks=init, local_blocks=local,
                     block_size=bs)
    scores = torch.full((M, k.W * 128 + spare), 77.0, device="cuda")
    rd.index_scores(iq.cuda(), head, torch.from_numpy(k.bt).cuda(), torch.from_numpy(k.seq).cuda(), scores)
    torch.cuda.synchronize()
    got = scores.double().cpu().numpy()
    scale = float(np.float32(128 ** -0.5 * 1.4426950408889634))
    q = iq.double().numpy()[:, head * 128:(head + 1) * 128]
    seen = 0
    for m in range(M):
        r, i = divmod(m, q_len)
        n = int(k.seq[r])
        p = n - q_len + i
        nb = p // 128 + 1 if n >= max(q_len, 1) and (n + 127) // 128 <= k.W else 0
        assert (got[m, nb * 128:] == 77).all()
        j = np.arange(nb * 128)
        b = j // 128
        on = (j <= p) & (b >= init) & (b < nb - local)
        blk = k.bt[r, b].astype(np.int64)
        lost = (b >= init) & (b < nb - local) & (blk >= k.pool)
        assert np.isneginf(got[m, :nb * 128][~on & ~lost]).all()
        assert (got[m, :nb * 128][lost] == 77).all()
        on &= ~lost
        keys = k.keys[blk[on] * 128 + j[on] % 128]
        want = keys @ q[m] * scale
        # 128 products in f32: at most 127 additions, each off by up to 2^-23 of the running sum, and two factors
        tol = 2.0 ** -16 * scale * (np.abs(keys) @ np.abs(q[m])) + 1e-300
        assert (np.abs(got[m, :nb * 128][on] - want) <= tol).all(), m
        seen += int(on.sum())
    return seen, rd.device_status()


@pytest.mark.parametrize("q_len,init,local", [(1, 0, 0), (1, 1, 4), (3, 0, 1), (7, 1, 2), (8, 2, 0), (9, 0, 0), (16, 1, 1)])
def test_nvfp4_scores(q_len, init, local):
    seen, status = check_scores([q_len, 1500, 0, 128 + q_len, 1025], q_len, init, local, n_iq=2, head=1, seed=q_len)
    assert seen > 0 and status == 0


@pytest.mark.parametrize("bs,pad", [(4, 32), (8, 0), (32, 0), (64, 64), (128, 0), (256, 32), (1024, 0)])
def test_nvfp4_scores_page_layouts(bs, pad):
    seen, status = check_scores([700, 130, 2000], 2, 0, 1, bs=bs, pad=pad, seed=bs, spare=64)
    assert seen > 0 and status == 0


def test_nvfp4_scores_bad_blocks_requests_and_magnitudes():
    from indexer_projection_gb300 import binding as B

    seen, status = check_scores([700, 600], 2, 1, 1, seed=31, bad=(1, 2))
    assert seen > 0 and status == B.PA_DEV_SLOT_RANGE
    _, status = check_scores([1, 400], 2, 0, 0, seed=32)
    assert status == B.PA_DEV_SLOT_RANGE
    for s in (2.0 ** -60, 2.0 ** 70):
        seen, status = check_scores([400], 3, 0, 0, seed=33, iq_scale=s)
        assert seen > 0 and status == 0


# ------------------------------------------------------------- all together

@pytest.mark.parametrize("cache_fmt,q_len", [("fp8", 1), ("fp8", 4), ("nvfp4", 1), ("nvfp4", 4)])
def test_step_scores_selection_attention_on_one_stream(cache_fmt, q_len):
    """The step writes its rows' keys into caches that hold the requests' earlier keys; the scores, the selection and
    the attention follow on the same stream, then the reference repeats each from what the one before it left."""
    from tests import harness
    from indexer_projection_gb300.runner import CacheReader

    R, nkv, W, topk, init, local = 6, 2, 12, 6, 1, 1
    M = R * q_len
    wl = workloads.Workload(f"run_{cache_fmt}_{q_len}", H=512, nkv=nkv, M=M, weight_fmt="ptpc", cache_fmt=cache_fmt, seed=41,
                            n_iq=nkv, max_pos=2048, pool_pages16=R * W * 8, pool_pages=R * W * 8)
    st = workloads.host_state(wl)
    rng = np.random.default_rng(8)
    seq = rng.integers(q_len, W * 128, R).astype(np.int32)
    seq[0] = q_len
    bt = rng.permutation(R * W).reshape(R, W).astype(np.int32)
    pos = (seq[:, None] - q_len + np.arange(q_len)).reshape(-1)
    rr = np.repeat(np.arange(R), q_len)
    slots = bt[rr, pos // 128].astype(np.int64) * 128 + pos % 128
    st["positions"], st["slot_mapping"], st["index_slot_mapping"] = pos.astype(np.int64), slots, slots.copy()
    # the earlier keys
    nslots = R * W * 128
    if cache_fmt == "fp8":
        for w in "kv":
            x = torch.from_numpy(rng.standard_normal(nslots * nkv * 128) * 120).clamp(-448, 448)
            st[w + "_cache"] = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(st[w + "_cache"].shape).copy()
            st[w + "_scale"] = np.full(st[w + "_scale"].shape, 0.01, np.float32)
        x = torch.from_numpy(rng.standard_normal(nslots * 128)).to(torch.float8_e4m3fn)
        st["index_cache"] = x.view(torch.uint8).numpy().reshape(st["index_cache"].shape).copy()
    else:
        for w in ("kv_cache", "idx_cache"):
            c = rng.integers(0, 256, st[w].size).astype(np.uint8).reshape(wl.kv_pages, -1)
            for at in range(0, c.shape[1], 16 * 72):  # group scales around 1
                c[:, at + 1024:at + 1152] = rng.integers(0x30, 0x40, (c.shape[0], 128))
            st[w] = c.reshape(st[w].shape)
    run = harness.GpuRun(wl, st)
    d = run.d
    dev = torch.device("cuda")
    t_bt, t_seq = torch.from_numpy(bt).to(dev), torch.from_numpy(seq).to(dev)
    rd = CacheReader(16 * nkv, nkv, cache_format=run.runner.cfg.cache_format, caches=run.caches, max_requests=R, q_len=q_len,
                     bt_width=W, topk=topk, init_blocks=init, local_blocks=local, block_size=16)
    scores = torch.full((nkv, M, W * 128), 55.0, device=dev)
    blocks = torch.zeros(M, nkv, topk, dtype=torch.int32, device=dev)
    counts = torch.zeros(M, nkv, dtype=torch.int32, device=dev)
    out = torch.zeros(M, nkv * 16 * 128, dtype=torch.bfloat16, device=dev)
    q = d["q_bf16"].view(torch.bfloat16).view(M, -1)
    iq = d["iq_bf16"].view(torch.bfloat16).view(M, -1)
    torch.cuda.synchronize()
    assert run.run(check=False) == 0
    for h in range(nkv):
        rd.index_scores(iq, h, t_bt, t_seq, scores[h])
    rd.select_blocks(scores, t_seq, blocks, counts)
    rd.attend(q, t_bt, t_seq, out, blocks=blocks, counts=counts)
    torch.cuda.synchronize()
    assert rd.device_status() == 0 and run.runner.device_status() == 0
    # the selection from the scores that the GPU left
    lists = ref.select(scores.cpu().numpy(), seq, q_len, W, init, local, topk)
    assert [[[int(b) for b in blocks[m, h, :counts[m, h]]] for h in range(nkv)] for m in range(M)] == lists
    # the attention from the step's q, its caches and that selection
    c = ref.Case.__new__(ref.Case)
    c.fmt, c.q_len, c.nkv, c.group, c.R, c.M, c.W, c.seq, c.bt = cache_fmt, q_len, nkv, 16, R, M, W, seq, bt
    c.q, c.vs = q.cpu(), np.zeros((nkv, R * W * 128))
    dd, slot = np.arange(128), np.arange(nslots)[:, None]
    c.k, c.v = np.zeros((nkv, nslots, 128)), np.zeros((nkv, nslots, 128))
    idx = np.zeros((nslots, 128))
    if cache_fmt == "fp8":
        kc, vc = (d[w + "_cache"].view(torch.uint8).cpu().numpy().reshape(-1) for w in "kv")
        ks, vs = (d[w + "_scale"].float().cpu().numpy().reshape(-1).astype(np.float64) for w in "kv")
        for h in range(nkv):
            p = slot // 16 * nkv + h
            c.k[h] = ref.E4M3[kc[p * 2048 + dd // 16 * 256 + slot % 16 * 16 + dd % 16]] * ks[p * 16 + slot % 16]
            c.v[h] = ref.E4M3[vc[p * 2048 + dd * 16 + slot % 16]] * vs[p * 16 + slot % 16]
            c.vs[h] = vs[p * 16 + slot % 16][:, 0]
        idx = ref.E4M3[d["index_cache"].view(torch.uint8).cpu().numpy().reshape(nslots, 128)]
    else:
        def rows(flat, stride, sl, swz):
            b, t = slot // 16 * stride + sl * 16 * 72, slot % 16
            byte = flat[b + t * 64 + dd // 2]
            g = dd // 16
            sf = flat[b + 1024 + ((t // 4 * 4 + g // 2) * 8 + g % 2 * 4 + t % 4 if swz else t * 8 + g)]
            return ref.E2M1[np.where(dd % 2 == 0, byte & 15, byte >> 4)] * ref.E4M3[sf]
        kv = d["kv_cache"].view(torch.uint8).cpu().numpy().reshape(-1)
        for h in range(nkv):
            c.k[h], c.v[h] = rows(kv, wl.kv_page_bytes, 2 * h, False), rows(kv, wl.kv_page_bytes, 2 * h + 1, True)
        idx = rows(d["idx_cache"].view(torch.uint8).cpu().numpy().reshape(-1), wl.idx_page_bytes, 0, False)
    close(out.double().cpu().numpy(), c.attention(lists))
    # the scores from the step's index_q and index cache
    scale = float(np.float32(oracle.index_scale_log2e(128 ** -0.5)))
    for m in range(M):
        j = np.arange(pos[m] + 1)
        nb = pos[m] // 128 + 1
        j = j[(j // 128 >= init) & (j // 128 < nb - local)]
        keys = idx[bt[rr[m], j // 128].astype(np.int64) * 128 + j % 128]
        for h in range(nkv):
            qv = iq[m, h * 128:(h + 1) * 128].double().cpu().numpy()
            err = np.abs(scores[h, m, :].double().cpu().numpy()[j] - keys @ qv * scale)
            assert (err <= 2.0 ** -16 * scale * (np.abs(keys) @ np.abs(qv)) + 1e-30).all()
