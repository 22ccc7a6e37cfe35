"""pre_attn_evict_blocks against its definition, request by request in Python; its refusals without a GPU."""

import math

import numpy as np
import pytest
import torch

P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def B():
    from indexer_projection_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def expected(weights, table, seq, keep, init, local):
    """The outputs for one request: weights, table, length, evicted, count, flagged."""
    w, t, W = list(weights), list(table), len(table)
    nb = (seq + 127) // 128 if seq > 0 else 0
    if nb > W:
        return w, t, seq, [-1] * W, 0, True
    free = [b for b in range(nb) if b >= init and b < nb - max(local, 1)]
    free.sort(key=lambda b: (-math.inf if math.isnan(w[b]) else w[b], -b))
    out = sorted(free[:max(nb - keep, 0)])
    gone = [t[b] for b in out]
    for b in reversed(out):
        del w[b], t[b]
    n = len(out)
    return w + [0.0] * n, t + [-1] * n, seq - 128 * n, gone + [-1] * (W - n), n, False


def reader(W, init, local, R=8):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader
    return CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), max_requests=R, q_len=1, bt_width=W,
                       init_blocks=init, local_blocks=local)


def check(weights, table, seq, keep, init, local, in_place=False, pad=0, rd=None):
    R, W = table.shape
    rd = rd or reader(W, init, local, R)
    wide = torch.full((R, W + pad), 55.0, device="cuda")
    wide[:, :W] = torch.from_numpy(weights).cuda()
    w, t, s = wide[:, :W], torch.from_numpy(table).cuda(), torch.from_numpy(seq).cuda()
    evicted, counts = torch.full_like(t, 77), torch.full_like(s, 77)
    kw = {}
    if not in_place:
        kw = dict(weights_out=torch.full((R, W + 2 * pad), 66.0, device="cuda"), block_table_out=torch.full_like(t, 77),
                  seq_lens_out=torch.full_like(s, 77))
    rd.evict_blocks(w, t, s, evicted, counts, keep=keep, **kw)
    torch.cuda.synchronize()
    status = rd.device_status()
    got = (kw.get("weights_out", w)[:, :W], kw.get("block_table_out", t), kw.get("seq_lens_out", s), evicted, counts)
    got = [x.cpu().numpy() for x in got]
    flagged = False
    for r in range(R):
        *want, bad = expected(weights[r].tolist(), table[r].tolist(), int(seq[r]), keep, init, local)
        flagged |= bad
        for g, v, what in zip(got, want, ("weights", "table", "length", "evicted", "count")):
            assert np.array_equal(g[r], np.array(v, g.dtype), equal_nan=g.dtype == np.float32), (r, what)
    assert status == (1 if flagged else 0)
    if pad:
        assert (wide[:, W:] == 55).all()
        if not in_place:
            assert (kw["weights_out"][:, W:] == 66).all()
    if not in_place:  # the inputs stay as they were
        assert np.array_equal(w.cpu().numpy(), weights, equal_nan=True) and np.array_equal(t.cpu().numpy(), table)


def inputs(R, W, seed, values="random", spare=False):
    g = np.random.default_rng(seed)
    table = g.permutation(R * W).reshape(R, W).astype(np.int32)
    w = g.exponential(size=(R, W)).astype(np.float32)
    if values == "ties":
        w = (g.integers(-1, 3, (R, W)) * 0.5).astype(np.float32)
        w[::2][w[::2] == 0] = -0.0
    elif values == "extreme":
        w = g.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0], np.float32), (R, W))
    elif values == "same":
        w[:] = 0.25
    elif values == "close":  # keys that differ in their lowest bits alone
        w = (np.float32(1.0) + g.integers(0, 7, (R, W)) * np.float32(2.0 ** -23)).astype(np.float32)
    return w, table


@pytest.mark.gpu
@pytest.mark.parametrize("values", ["random", "ties", "extreme", "same", "close"])
@pytest.mark.parametrize("W,keep,init,local", [(1, 1, 0, 0), (2, 1, 0, 1), (5, 3, 1, 1), (31, 7, 0, 2), (33, 9, 2, 7), (64, 5, 1, 4),
                                               (256, 40, 1, 4), (1000, 400, 0, 0), (1024, 1, 0, 0), (1025, 700, 3, 3)])
def test_every_width(W, keep, init, local, values):
    seq = np.array([128 * W, 0, 1, 128 * W - 127, 128 * min(W, keep), 128 * min(W, keep + 1), -3, 64 * W], np.int32)
    w, table = inputs(len(seq), W, W + keep, values)
    check(w, table, seq, keep, init, local)
    check(w, table, seq, keep, init, local, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("W", [2048, 2049, 4096, 5000, 8192, 8193, 16384])
@pytest.mark.parametrize("values", ["random", "ties"])
def test_wide_tables(W, values):
    w, table = inputs(3, W, W, values)
    check(w, table, np.array([128 * W, 100 * W, 128 * W - 5], np.int32), W // 3, 4, 16, in_place=values == "ties")


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_strides_reserved_entries_and_lengths_beyond_the_table(in_place):
    w, table = inputs(5, 40, 3)
    seq = np.array([1000, 128 * 40 + 1, 2 ** 31 - 1, 128 * 40, 128 * 20 + 1], np.int32)  # entries behind the last block move too
    check(w, table, seq, 6, 1, 1, in_place=in_place, pad=3)
    table[:, 30:] = -1
    check(w, table, seq, 6, 1, 1, in_place=in_place, pad=3)


@pytest.mark.gpu
def test_every_number_kept():
    w, table = inputs(4, 37, 9, "ties")
    rd = reader(37, 1, 2)
    for keep in (*range(3, 41), 2 ** 32 + 3):
        check(w, table, np.array([37 * 128, 35 * 128 + 1, 129, 20 * 128], np.int32), keep, 1, 2, rd=rd)


@pytest.mark.gpu
def test_as_many_requests_as_there_can_be():
    w, table = inputs(65535, 6, 11, "ties")
    R = 65535
    rd = reader(6, 1, 1, R)
    seq = (np.arange(R) * 37 % (6 * 128 + 1)).astype(np.int32)
    t = [torch.from_numpy(x).cuda() for x in (w, table, seq)]
    evicted, counts = torch.zeros_like(t[1]), torch.zeros_like(t[2])
    rd.evict_blocks(*t, evicted, counts, keep=3)
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in (*t, evicted, counts)]
    for r in [0, 1, 2, R // 2, *range(R - 300, R)]:
        want = expected(w[r].tolist(), table[r].tolist(), int(seq[r]), 3, 1, 1)
        assert [got[0][r].tolist(), got[1][r].tolist(), int(got[2][r]), got[3][r].tolist(), int(got[4][r])] == list(want[:5])
    assert (got[4] == np.maximum((seq + 127) // 128 - 3, 0)).all()


@pytest.mark.gpu
def test_captured_on_a_stream_and_again_until_nothing_is_left():
    w, table = inputs(2, 50, 4)
    seq = np.array([50 * 128 - 3, 30 * 128], np.int32)
    rd = reader(50, 1, 1)
    t = [torch.from_numpy(x).cuda() for x in (w, table, seq)]
    outs = [torch.zeros_like(t[0]), torch.zeros_like(t[1]), torch.zeros_like(t[2])]
    evicted, counts = torch.zeros_like(t[1]), torch.zeros_like(t[2])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rd.evict_blocks(*t, evicted, counts, keep=20, weights_out=outs[0], block_table_out=outs[1], seq_lens_out=outs[2])
    for _ in range(3):
        for x in (*outs, evicted, counts):
            x.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        for r in range(2):
            want = expected(w[r].tolist(), table[r].tolist(), int(seq[r]), 20, 1, 1)
            assert outs[1][r].tolist() == want[1] and int(outs[2][r]) == want[2] and int(counts[r]) == want[4]
    for _ in range(2):  # in place: the second call finds the request within its budget
        rd.evict_blocks(*t, evicted, counts, keep=20)
    torch.cuda.synchronize()
    assert (counts == 0).all() and (evicted == -1).all() and torch.equal(t[1], outs[1]) and torch.equal(t[2], outs[2])
    assert rd.evict_blocks(*(x[:0] for x in t), evicted[:0], counts[:0], keep=20) == 0
    assert rd.device_status() == 0


@pytest.mark.gpu
def test_what_the_reader_refuses():
    w, table = inputs(2, 8, 4)
    rd = reader(8, 1, 1)
    a = dict(weights=torch.from_numpy(w).cuda(), block_table=torch.from_numpy(table).cuda(),
             seq_lens=torch.tensor([900, 900], dtype=torch.int32, device="cuda"))
    a["evicted"], a["counts"] = torch.zeros_like(a["block_table"]), torch.zeros_like(a["seq_lens"])
    keep = {k: v.clone() for k, v in a.items()}
    for bad in (dict(weights=a["weights"].cpu()), dict(weights=a["weights"].double()), dict(weights=a["weights"][:, 1:]),
                dict(weights=a["weights"].t().contiguous().t()), dict(block_table=a["block_table"].long()),
                dict(seq_lens=a["seq_lens"].cpu()), dict(evicted=a["evicted"][:1]), dict(counts=a["counts"].long()),
                dict(weights_out=a["weights"][:1]), dict(block_table_out=a["block_table"][:, :7]),
                dict(seq_lens_out=a["seq_lens"].cpu())):
        with pytest.raises(ValueError):
            rd.evict_blocks(**dict(a, **bad), keep=4)
    from indexer_projection_gb300.binding import PreAttnError
    for bad in (dict(keep=1), dict(evicted=a["block_table"]), dict(weights_out=torch.zeros(3, 8, device="cuda")[1:], keep=-5)):
        with pytest.raises(PreAttnError):
            rd.evict_blocks(**dict(dict(a, keep=4), **bad))
    torch.cuda.synchronize()
    assert all(torch.equal(keep[k], a[k]) for k in a) and rd.device_status() == 0


def args(B, **kw):
    at = iter(range(P, P + (100 << 20), 1 << 20))
    d = dict(weights=next(at), weights_stride=40, block_table=next(at), seq_lens=next(at), R=2, bt_width=40, keep=6, init_blocks=1,
             local_blocks=2, weights_out=next(at), weights_out_stride=40, block_table_out=next(at), seq_lens_out=next(at),
             evicted=next(at), counts=next(at), status=next(at))
    d.update(kw)
    return B.pa_evict_args(**d)


POINTERS = ("weights", "block_table", "seq_lens", "weights_out", "block_table_out", "seq_lens_out", "evicted", "counts", "status")


@pytest.mark.parametrize("kw,err", [
    *[({p: None}, "NULL") for p in POINTERS], *[({p: P + 2}, "ALIGN") for p in POINTERS],
    *[({"R": v}, "SHAPE") for v in (-1, 65536)], *[({"bt_width": v}, "SHAPE") for v in (0, 41, 16385)],
    ({"weights_stride": 39}, "SHAPE"), ({"weights_out_stride": 39}, "SHAPE"), ({"keep": 2}, "CONFIG"), ({"keep": -1}, "CONFIG"),
    ({"init_blocks": -1}, "CONFIG"), ({"local_blocks": -1}, "CONFIG"), ({"init_blocks": 6, "local_blocks": 0}, "CONFIG"),
    ({"init_blocks": 2 ** 31 - 1}, "CONFIG"), ({"evicted": P}, "ALIAS"), ({"counts": P + (1 << 20) + 4}, "ALIAS"),
    ({"weights_out": P + 4}, "ALIAS"), ({"weights_out": P, "weights_out_stride": 41}, "ALIAS"),
    ({"weights_out": P + (1 << 20)}, "ALIAS"), ({"block_table_out": P + (1 << 20) + 8}, "ALIAS")])
def test_refusals(B, kw, err):
    assert B.pre_attn_evict_blocks(args(B, **kw), check=False) == getattr(B, "PA_ERR_" + err)


def test_no_requests_is_accepted(B):
    assert B.pre_attn_evict_blocks(args(B, R=0), check=False) == B.PA_OK
