"""GPU parity of pre_attn_attention_ext (the window with sinks, the blocks' weights) with the 64-bit reference, and a
speculative step on caches of bounded size: attention and weights, verification, eviction, attention."""

import numpy as np
import pytest
import torch

from tests import cache_reference as ref
from tests import window_reference as win
from tests.test_evict_blocks import expected as evicted_of
from tests.test_verify_drafts import expected as verified

pytestmark = pytest.mark.gpu
FORMATS = ["fp8", "nvfp4"]


def case(fmt, seq, q_len, nkv=1, group=16, window=0, sinks=0, **kw):
    c = win.Case(fmt, seq, q_len, nkv, group, **kw)
    c.window, c.sinks = window, sinks
    return c


# ---------------------------------------------------------------- the window

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (15, 3), (16, 0), (127, 1), (128, 0), (129, 4), (130, 127), (300, 128),
                                          (1, 129), (700, 300), (5000, 7), (200, 5000)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_every_window(fmt, window, sinks, q_len):
    c = case(fmt, [q_len, 128, 129, 300, 0, 1100, 1029], q_len, 1, 16, window, sinks, seed=window + sinks).poison().upload()
    rd = c.reader()
    win.close(win.attend(c, rd), c.attention())
    assert rd.device_status() == 0  # (the blocks that no row sees are not asked for)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,group", [(1, 1, 16), (2, 2, 16), (3, 1, 8), (4, 4, 5), (5, 2, 1), (7, 2, 16), (8, 1, 13), (9, 1, 16),
                                             (13, 2, 4), (16, 1, 16)])
def test_rows_and_heads(fmt, q_len, nkv, group):
    c = case(fmt, [q_len, 300, 0, 129 + q_len, 940], q_len, nkv, group, 200, 5, seed=q_len, extra_width=2, k_global=0.5,
             v_global=1.5).poison().upload()
    rd = c.reader()
    win.close(win.attend(c, rd), c.attention())
    assert rd.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,group", [(1, 16), (2, 4), (4, 2), (6, 1)])
@pytest.mark.parametrize("mode", ["cluster", "sliced", "whole"])
def test_every_way_of_dealing_blocks(fmt, q_len, group, mode):
    if mode == "whole":
        seq = list(np.random.default_rng(q_len).integers(q_len, 500, 2100))
        c = case(fmt, seq, q_len, 1, min(group, 2), 60, 130, seed=q_len)
    else:
        seq = [9000 + q_len, 90, 0, 23 * 128, 5000]
        window = 150 if mode == "cluster" else 7000
        c = case(fmt, seq, q_len, 1, group, window, 260, seed=40 + q_len, extra_width=0 if mode == "cluster" else 250)
    c.poison().upload()
    rd = c.reader()
    win.close(win.attend(c, rd), c.attention())
    assert rd.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 4, 6])
def test_long_windows_shared_by_every_sm(fmt, q_len):
    c = case(fmt, [60000 + q_len, 23 * 128], q_len, 1, 16, 33333, 300, seed=7).upload()
    rd = c.reader()
    win.close(win.attend(c, rd), c.attention())
    assert rd.device_status() == 0


@pytest.mark.parametrize("fmt,bs,kps,pad", [("fp8", 16, 16, 0), ("fp8", 16, 9, 0), ("nvfp4", 4, 8, 32), ("nvfp4", 32, 8, 64),
                                            ("nvfp4", 128, 8, 96), ("nvfp4", 256, 8, 0), ("nvfp4", 1024, 8, 32)])
def test_page_layouts(fmt, bs, kps, pad):
    c = case(fmt, [700, 90, 1300], 2, 2, 8, 333, 70, bs=bs, kps=kps, pad=pad, seed=bs + kps).upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_window_as_wide_as_the_table_is_none(fmt):
    c = case(fmt, [900, 300], 2, 1, 16, seed=5).upload()
    rd = c.reader()
    want = win.attend(c, rd)
    for c.window, c.sinks in ((c.W * 128, 3), (2 ** 31 - 1, 2 ** 31 - 1), (c.W * 128 - 1, 0), (2 ** 32 + 2, 2 ** 32)):
        assert torch.equal(win.attend(c, rd), want)
    c.window, c.sinks = 2, 2 ** 31 - 1  # sinks past every key
    win.close(win.attend(c, rd), c.attention())


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_blocks_and_requests_within_a_window(fmt):
    c = case(fmt, [900, 500, 2, 128 * 8 + 1], 3, 1, 16, 300, 130, seed=6)
    c.W, c.bt = 8, c.bt[:, :8].copy()
    c.upload()
    c.bt[0, 5], c.bt[1, 1] = -1, c.pool  # a block of the window, one of the sinks'
    c.dev["bt"] = torch.from_numpy(c.bt).cuda()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    assert rd.device_status() == 1
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())
    assert (out[6:] == 0).all()


# --------------------------------------------------------------- the weights

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,group", [(1, 1, 16), (1, 4, 1), (2, 2, 16), (3, 1, 8), (4, 4, 5), (5, 2, 1), (7, 2, 16), (8, 1, 13),
                                             (9, 1, 16), (13, 2, 4), (16, 4, 3)])
@pytest.mark.parametrize("window", [0, 200])
def test_weights_of_rows_and_heads(fmt, q_len, nkv, group, window):
    c = case(fmt, [q_len, 300, 0, 129 + q_len, 940, 128], q_len, nkv, group, window, 5 if window else 0, seed=q_len, extra_width=2,
             k_global=0.5, v_global=1.5)
    c.seq[5] = q_len - 1 if q_len > 1 else 0
    c.upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    assert rd.device_status() == (1 if q_len > 1 else 0)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())
    total = w[[0, 1, 3, 4]].double().sum(1).cpu()  # a softmax for each row and head
    assert torch.allclose(total, torch.full_like(total, float(q_len * nkv * group)), rtol=2.0 ** -12)
    # the attention is the one without weights, to the bit where the kernel is the same
    if window:
        assert torch.equal(out, win.attend(c, rd))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv,topk", [(1, 1, 1), (1, 2, 4), (2, 1, 3), (1, 1, 40), (4, 2, 5), (7, 2, 4), (8, 1, 6), (11, 1, 3)])
def test_weights_of_selected_blocks(fmt, q_len, nkv, topk):
    c = case(fmt, [1000, q_len, 0, 260 + q_len, 128 * 9], q_len, nkv, 16, seed=100 + q_len).upload()
    blocks, counts, lists = ref.random_lists(c, topk, seed=topk)
    # a block twice, one outside the request, a negative one
    if topk >= 4:
        blocks[0, 0, :4], counts[0, 0] = [1, 3, 1, 3], 4
        lists[0][0] = [1, 3]
    rd = c.reader(topk=topk, weigh=True)
    out, w = win.attend(c, rd, (blocks, counts), weights=True)
    assert rd.device_status() == 0
    win.close(out, c.attention(lists))
    win.close_weights(w, c, c.weights(lists))
    if topk >= 4:
        blocks[0, 0, :4] = [1, 7000, -5, 3]
        out, w = win.attend(c, rd, (blocks, counts), weights=True)
        assert rd.device_status() == 1
        win.close(out, c.attention(lists))
        win.close_weights(w, c, c.weights(lists))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,group", [(1, 16), (2, 4), (4, 2), (6, 1)])
@pytest.mark.parametrize("mode", ["cluster", "sliced", "whole"])
def test_weights_in_every_way_of_dealing_blocks(fmt, q_len, group, mode):
    if mode == "whole":
        c = case(fmt, list(np.random.default_rng(q_len).integers(q_len, 500, 2100)), q_len, 1, min(group, 2), seed=q_len)
    elif mode == "cluster":
        c = case(fmt, [700, 90, 1100], q_len, 1, group, seed=60 + q_len)
    else:
        c = case(fmt, [40100 + q_len, 23 * 128, 0, 300], q_len, 1, group, seed=60 + q_len)
    c.upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())
    again = win.attend(c, rd, weights=True)
    assert torch.equal(out, again[0]) and torch.equal(w, again[1]) and rd.device_status() == 0  # the same bits


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("W", [4096, 4097, 16384])
def test_lists_of_wide_tables(fmt, W):
    c = case(fmt, [1000, 700, 129], 7, 1, 16, seed=W).upload()
    blocks, counts, lists = ref.random_lists(c, 4, seed=3)
    narrow = c.attention(lists), c.weights(lists)
    c.bt = np.concatenate((c.bt, np.full((3, W), -1, np.int32)), 1)[:, :W].copy()
    c.W, c.dev["bt"] = W, torch.from_numpy(c.bt).cuda()
    rd = c.reader(topk=4, weigh=True)
    out, w = win.attend(c, rd, (blocks, counts), weights=True)
    assert rd.device_status() == 0
    win.close(out, narrow[0])
    k = narrow[1][0].shape[1]
    assert (w[:, k:] == 0).all()
    over = np.abs(w[:, :k].double().cpu().numpy() - narrow[1][0]) - narrow[1][1]
    assert (over <= 0).all()


@pytest.mark.parametrize("W", [33, 64, 2049, 16384])
def test_weights_of_wide_tables(W):
    # short requests in wide tables: each cluster size, columns of zeros behind the last block
    c = case("nvfp4", [1000, 4100, 129], 2, 2, 4, seed=W)
    c.bt = np.concatenate((c.bt, np.full((3, W), -1, np.int32)), 1)[:, :W].copy()
    c.W = W
    c.upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_that_fade_in_place_and_strides(fmt):
    c = case(fmt, [700, 0, 1300], 2, 2, 8, seed=8, extra_width=1).upload()
    rd = c.reader(weigh=True)
    g = np.random.default_rng(3)
    before = g.exponential(size=(3, c.W)).astype(np.float32)
    wide = torch.full((3, c.W + 5), 3.0, device="cuda")
    wide[:, :c.W] = torch.from_numpy(before).cuda()
    old = wide[:, :c.W]
    new = torch.full((3, c.W + 2), 7.0, device="cuda")
    for decay in (1.0, 0.75, 2.0, 0.0):
        win.attend(c, rd, weights=new[:, :c.W], weights_before=old, decay=decay)
        win.close_weights(new[:, :c.W], c, c.weights(before=before, decay=decay))
    assert (new[:, c.W:] == 7).all() and torch.equal(old.cpu(), torch.from_numpy(before))
    old[:, 1] = float("nan")  # not read
    win.attend(c, rd, weights=new[:, :c.W], weights_before=old, decay=0.0)
    win.close_weights(new[:, :c.W], c, c.weights())
    old[:] = torch.from_numpy(before).cuda()
    for k in range(3):  # a layer after the other into the same rows
        win.attend(c, rd, weights=old, weights_before=old)
    mine, tol = c.weights()
    win.close_weights(old, c, (before + 3 * mine, 3 * tol + 2.0 ** -20 * (before + 3 * mine)), untouched=before[1])
    assert (wide[:, c.W:] == 3).all() and rd.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_of_peaked_rows_and_far_magnitudes(fmt):
    c = case(fmt, [3000, 700], 1, 1, 16, seed=19, q_scale=12.0)
    c.q = (c.q.float().view(2, 16, 128) * torch.tensor([2.0 ** e for e in range(-12, 4)])[:, None]).to(torch.bfloat16).view(2, -1)
    c.upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 3, 5, 8])
@pytest.mark.parametrize("window", [0, 260])
def test_far_scales_and_peaked_rows(fmt, q_len, window):
    # V scales over 2^24, a zero value row with scale 1 that takes nearly all the weight (FP8); head rows of queries from
    # 2^-30 to 2^5: nearly even weights and a single one
    c = case(fmt, [700, 130, 512], q_len, 2, 16, window, 4 if window else 0, seed=30 + q_len, spread=24.0)
    c.q = (c.q.float().view(-1, 2, 16, 128) * torch.tensor([2.0 ** e for e in range(-30, 6, 9)] * 4)[:, None]).to(torch.bfloat16).view(c.M, -1)
    if fmt == "fp8":
        n = 700
        slot = int(c.bt[0, (n - q_len) // 128]) * 128 + (n - q_len) % 128
        page, t = slot // 128 * c.kps + slot % 128 // 16, slot % 16
        for h in range(2):
            base = (page * 2 + h) * 2048
            c.bytes["v"][base + np.arange(128) * 16 + t] = 0
            c.scales["v"][(page * 2 + h) * 16 + t] = 1.0
            c.v[h, slot], c.vs[h, slot] = 0.0, 1.0
    c.upload()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())
    assert rd.device_status() == 0


def put_nan(c, what, r, j):
    """NaN in key j of request r, KV head 0: a value's code (FP8) or the scale of its dims 32 .. 47 (NVFP4), a scale of FP8."""
    slot = int(c.bt[r, j // 128]) * 128 + j % 128
    if c.fmt == "fp8":
        page, t = slot // 128 * c.kps + slot % 128 // 16, slot % 16
        if what == "value":
            c.bytes["v"][page * c.nkv * 2048 + 37 * 16 + t] = 0xff
        else:
            c.scales[what][page * c.nkv * 16 + t] = float("nan")
    else:
        flat, t = c.kv.reshape(-1), slot % c.bs
        base = slot // c.bs * c.page_bytes + c.bs * 64
        flat[base + t * 8 + 2 if what == "k" else base + c.bs * 72 + (t // 4 * 4 + 1) * 8 + t % 4] = 0x7f


@pytest.mark.parametrize("fmt,what", [("fp8", "value"), ("fp8", "k"), ("fp8", "v"), ("nvfp4", "value"), ("nvfp4", "k")])
@pytest.mark.parametrize("q_len", [2, 4, 7])
@pytest.mark.parametrize("lists", [False, True])
def test_a_nan_reaches_the_rows_that_see_it(fmt, what, q_len, lists):
    n, window = 700, 0 if lists else 260
    c = case(fmt, [n, 300], q_len, 1, 16, window, 2 if window else 0, seed=50 + q_len)
    sel = None
    if lists:  # rows of even number attend block 1
        blocks, counts = np.tile(np.array([0, 2, 5], np.int32), (c.M, 1, 1)), np.full((c.M, 1), 3, np.int32)
        blocks[::2, 0, 1] = 1
        sel = [[[b for b in blocks[m, 0] if b * 128 < (n if m < q_len else 300)]] for m in range(c.M)]
        blocks[q_len:, 0, 2], counts[q_len:] = -1, 2
        keys = [130, n - 2]
    else:
        keys = [n - q_len + 1 - window, n - 2, 300]  # the window's end, the rows' own keys, one that none sees
    want = c.attention(sel)
    for j in keys:
        put_nan(c, what, 0, j)
    c.upload()
    got = win.attend(c, c.reader(topk=3 if lists else 0), (blocks, counts) if lists else None)
    got = got.double().cpu().numpy().reshape(c.M, 16, 128)
    dims = np.ones(128, bool)
    if what == "value":
        dims[:] = False
        dims[37 if fmt == "fp8" else slice(32, 48)] = True
    nan = np.zeros(got.shape, bool)
    for i in range(q_len):
        if set(keys) & set(c.row_positions(0, i, None if sel is None else sel[i][0]).tolist()):
            nan[i][:, dims] = True
    assert nan[:q_len].any() and (q_len == 2 or not nan[:q_len].all())
    assert (np.isnan(got) == nan).all()
    over = np.where(nan, -1.0, np.abs(got - want[0].reshape(got.shape)) - want[1].reshape(got.shape))
    assert (over <= 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_row_of_nan_stays_in_its_request(fmt):
    c = case(fmt, [300, 200], 2, 1, 16, seed=20)
    c.q[1, 5 * 128 + 3] = float("nan")
    c.upload()
    rd = c.reader(weigh=True)
    _, w = win.attend(c, rd, weights=True)
    assert w[0, :3].isnan().all() and (w[0, 3:] == 0).all()
    c.q[1, 5 * 128 + 3] = 0.0
    got = w.clone()
    got[0] = torch.from_numpy(c.weights()[0][0]).cuda()
    win.close_weights(got, c, c.weights())


@pytest.mark.parametrize("fmt", FORMATS)
def test_fp8_queries(fmt):
    c = case(fmt, [400, 77], 3, 1, 16, 100, 2, seed=15).upload()
    q8 = (c.q.float() / 0.25).to(torch.float8_e4m3fn)
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, q=q8.cuda(), q_fp8_scale=0.25, weights=True)
    win.close(out, c.attention(q=q8.float() * 0.25))
    win.close_weights(w, c, c.weights(q=q8.float() * 0.25))


@pytest.mark.parametrize("fmt,q_len", [("fp8", 1), ("fp8", 7), ("nvfp4", 3)])
def test_a_wait_that_runs_out_is_reported(fmt, q_len):
    from indexer_projection_gb300 import binding as B

    c = case(fmt, [700, 90], q_len, 1, 16, 200, 4, seed=22).upload()
    late = c.reader(flags=B.PA_FLAG_TEST_WAIT_TIMEOUT, weigh=True)
    out, w = torch.full((c.M, 2048), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, c.W), 3.0, device="cuda")
    late.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, window=200, sinks=4, weights=w)
    assert late.device_status() == B.PA_DEV_WAIT_TIMEOUT
    assert (out == 3).all() and (w == 3).all()
    rd = c.reader(weigh=True)
    out, w = win.attend(c, rd, weights=True)
    win.close(out, c.attention())
    win.close_weights(w, c, c.weights())


@pytest.mark.parametrize("fmt,q_len,seq", [("fp8", 7, [20000, 700]), ("nvfp4", 3, [20000, 700]), ("nvfp4", 7, [300] * 2100)])
def test_a_wait_that_runs_out_while_items_are_cut_or_whole(fmt, q_len, seq):
    from indexer_projection_gb300 import binding as B

    c = case(fmt, seq, q_len, 1, 2, 0, 0, seed=24).upload()
    late, rd = c.reader(flags=B.PA_FLAG_TEST_WAIT_TIMEOUT, weigh=True), c.reader(weigh=True)
    out, w = torch.full((c.M, 256), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((c.R, c.W), 3.0, device="cuda")
    late.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, weights=w)
    assert late.device_status() == B.PA_DEV_WAIT_TIMEOUT and (w == 3).all()
    first = win.attend(c, rd, weights=True)
    again = win.attend(c, rd, weights=True)
    assert rd.device_status() == 0 and torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    some = [0, 1, c.R - 1]
    total = first[1][some].double().sum(1).cpu()
    assert torch.allclose(total, torch.full_like(total, q_len * 2.0), rtol=2.0 ** -12)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_readers_at_once(fmt):
    # on two streams, each with a workspace of its own, one of them in a graph: the results of one at a time
    cases = [case(fmt, [9000, 300, 77], 7, 2, 16, 2000, 4, seed=25).upload(), case(fmt, [500, 12000], 2, 2, 16, 0, 0, seed=26).upload()]
    readers = [c.reader(weigh=True) for c in cases]
    want = [win.attend(c, rd, weights=True) for c, rd in zip(cases, readers)]
    got = [[torch.zeros_like(x) for x in pair] for pair in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    go = lambda k: readers[k].attend(*(cases[k].dev[n] for n in ("q", "bt", "seq")), got[k][0], window=cases[k].window,  # noqa: E731
                                     sinks=cases[k].sinks, weights=got[k][1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        go(0)
    for turn in range(6):
        for pair in got:
            for x in pair:
                x.fill_(9)
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(streams[0]):
                g.replay()
            with torch.cuda.stream(streams[1]):
                go(1)
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][1], want[k][1])
    assert all(rd.device_status() == 0 for rd in readers)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seq", [[1000, 64, 5000], [40000, 700, 64]])
@pytest.mark.parametrize("q_len", [2, 7])
def test_captured_in_order_and_on_another_stream(fmt, seq, q_len):
    from indexer_projection_gb300 import binding as B

    c = case(fmt, seq, q_len, 2, 16, 900, 130, seed=21).upload()
    rd, ordered = c.reader(weigh=True), c.reader(weigh=True, flags=B.PA_FLAG_NO_PDL)
    out, w = torch.zeros(c.M, 32 * 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.R, c.W, device="cuda")
    want = c.attention(), c.weights()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda r: r.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, window=900, sinks=130, weights=w)  # noqa: E731
    with torch.cuda.stream(s):
        call(rd)
    s.synchronize()
    win.close(out, want[0])
    win.close_weights(w, c, want[1])
    first = out.clone(), w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(rd)
    for run in (g.replay, g.replay, lambda: call(ordered), lambda: call(rd)):
        out.fill_(9), w.fill_(9)
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(w, first[1])
    assert rd.device_status() == 0 and ordered.device_status() == 0


def test_offsets_beyond_32_bits():
    # pages past 2^32 bytes of a cache, and sums of weights past 2^31 bytes of scratch
    c = case("nvfp4", [40000, 130], 4, 1, 16, 300, 4, bs=128, seed=23, stale="zero")
    pages = 300000  # x 18432 bytes = 5.5 GB
    big = torch.zeros(pages, c.page_bytes, dtype=torch.uint8, device="cuda")
    bt = c.bt.copy()
    for k, old in enumerate(sorted(set(c.bt[c.bt >= 0].tolist()))):
        big[pages - 1 - 900 * k] = torch.from_numpy(c.kv[old]).cuda()
        bt[c.bt == old] = pages - 1 - 900 * k
    want = c.attention(), c.weights()
    R, W = 300, 16384  # 300 x 4 x 16384 x 2 x 16 x 4 bytes = 2.5 GB
    seq, wide = np.zeros(R, np.int32), np.full((R, W), -1, np.int32)
    wide[[1, R - 1], :bt.shape[1]], seq[[1, R - 1]] = bt, c.seq
    q = torch.zeros(R * 4, 16 * 128, dtype=torch.bfloat16, device="cuda")
    q[4:8], q[-4:] = c.q[:4].cuda(), c.q[4:].cuda()
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader, PreAttn
    rd = CacheReader(16, 1, cache_format=B.PA_CACHE_NVFP4, caches=PreAttn.nvfp4_caches(big, pages, c.page_bytes, None, 0, 0), max_requests=R,
                     q_len=4, bt_width=W, block_size=128, weigh=True)
    out, w = torch.zeros_like(q), torch.full((R, W), 7.0, device="cuda")
    rd.attend(q, torch.from_numpy(wide).cuda(), torch.from_numpy(seq).cuda(), out, window=300, sinks=4, weights=w)
    assert rd.device_status() == 0
    win.close(torch.cat((out[4:8], out[-4:])), want[0])
    win.close_weights(w[[1, R - 1]][:, :c.W], c, want[1])
    assert (w[0] == 7).all() and (w[[1, R - 1]][:, c.W:] == 0).all()


@pytest.mark.parametrize("fmt,q_len", [("fp8", 1), ("fp8", 7), ("nvfp4", 1), ("nvfp4", 7)])
def test_as_many_requests_as_there_can_be(fmt, q_len):
    # 65535 requests that share a block, 129 lengths in turn
    R, lengths = 65535, 129
    c = case(fmt, [128], q_len, 1, 2, 50, 3, seed=61)
    block = int(c.bt[0, 0])
    c.R, c.M, c.seq, c.bt = lengths, lengths * q_len, np.arange(lengths, dtype=np.int32), np.full((lengths, 1), block, np.int32)
    c.q = ref.bf16(np.random.default_rng(62).standard_normal((c.M, 2 * 128)))
    c.upload()
    of = torch.arange(R) % lengths
    rows = (of[:, None] * q_len + torch.arange(q_len)).flatten()
    rd = c.reader(weigh=True, max_requests=R)
    q, seq, table = c.q[rows].cuda(), of.int().cuda(), torch.full((R, 1), block, dtype=torch.int32, device="cuda")
    out, w = torch.full_like(q, float("nan")), torch.full((R, 1), 7.0, device="cuda")
    rd.attend(q, table, seq, out, window=50, sinks=3, weights=w)
    assert rd.device_status() == (1 if q_len > 1 else 0)  # (lengths below q_len)
    want, tol = c.attention()
    over = (out.double().cpu() - torch.from_numpy(want)[rows]).abs() - torch.from_numpy(tol)[rows]
    assert (over <= 0).all()  # (a NaN is not)
    have = of >= max(q_len, 1)
    assert (w.cpu()[~have] == 7).all() and torch.allclose(w.cpu()[have], torch.tensor(2.0 * q_len), rtol=2.0 ** -12)


def test_what_the_reader_refuses():
    from indexer_projection_gb300 import binding as B

    c = case("fp8", [300, 20], 2, 1, 16, seed=95).upload()
    rd, plain = c.reader(topk=2, weigh=True), c.reader()
    out = torch.zeros(c.M, 2048, dtype=torch.bfloat16, device="cuda")
    lists, counts = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((c.M, 1, 2), (c.M, 1)))
    w = torch.zeros(2, c.W, device="cuda")
    go = lambda r, **kw: r.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, **kw)  # noqa: E731
    for kw in (dict(weights=w.cpu()), dict(weights=w.double()), dict(weights=w[:1]), dict(weights=w[:, 1:]), dict(weights_before=w),
               dict(weights=w, weights_before=w.cpu()), dict(weights=w, weights_before=w[:, 1:]), dict(window=5, weights_before=w)):
        with pytest.raises(ValueError):
            go(rd, **kw)
    with pytest.raises(ValueError, match="weigh=True"):
        go(plain, weights=w)
    for kw, err in ((dict(window=-1), B.PA_ERR_CONFIG), (dict(sinks=4), B.PA_ERR_CONFIG), (dict(window=4, sinks=-1), B.PA_ERR_CONFIG),
                    (dict(window=4, blocks=lists, counts=counts), B.PA_ERR_UNSUPPORTED), (dict(weights=w, decay=-1.0), B.PA_ERR_CONFIG),
                    (dict(weights=w, decay=float("nan")), B.PA_ERR_CONFIG), (dict(weights=w, decay=float("inf")), B.PA_ERR_CONFIG),
                    (dict(weights=out.view(torch.float32)[:2, :c.W]), B.PA_ERR_ALIAS)):
        with pytest.raises(B.PreAttnError) as e:
            go(rd, **kw)
        assert e.value.status == err
    torch.cuda.synchronize()
    assert rd.device_status() == 0 and not out.any() and not w.any()
    none = {k: c.dev[k][:0] for k in ("q", "bt", "seq")}
    assert rd.attend(none["q"], none["bt"], none["seq"], out[:0], window=3, weights=w[:0]) == 0


# -------------------------------------------------------------- all together

@pytest.mark.parametrize("fmt", FORMATS)
def test_a_speculative_step_on_caches_of_bounded_size(fmt):
    """Verify rows attend every block and leave the blocks' weights, a second layer's rows within a window add theirs; the
    drafts are verified, the blocks with the least weight evicted, and the next rows attend what is left."""
    from indexer_projection_gb300.runner import DraftVerifier

    q_len, V, keep, init, local = 4, 500, 5, 1, 2
    c = case(fmt, [1500, 700, 0, 300, 1281], q_len, 2, 16, seed=77, extra_width=1).upload()
    rd = c.reader(weigh=True, init_blocks=init, local_blocks=local)
    s = torch.cuda.Stream()
    g = torch.Generator().manual_seed(5)
    target = torch.softmax(torch.randn(c.M, V, generator=g) * 2, -1)
    draft = torch.softmax(torch.randn(c.R * (q_len - 1), V, generator=g) * 2, -1) * 0.4 + 0.6 * target.view(c.R, q_len, V)[:, :-1].reshape(-1, V)
    x = torch.multinomial(draft, 1, generator=g).int().view(c.R, q_len - 1)
    u = torch.rand(c.R, q_len, generator=g)
    dev = [y.cuda() for y in (target, x, u, draft)]
    ver = DraftVerifier(V, q_len)
    out, second = (torch.zeros(c.M, 32 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.full((c.R, c.W), 7.0, device="cuda")
    tokens, accepted = torch.zeros(c.R, q_len, dtype=torch.int32, device="cuda"), torch.zeros(c.R, dtype=torch.int32, device="cuda")
    table, lens = torch.zeros_like(c.dev["bt"]), torch.zeros_like(c.dev["seq"])
    evicted, counts, left = torch.zeros_like(table), torch.zeros_like(lens), torch.zeros_like(w)
    last = torch.zeros_like(out)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, weights=w)
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], second, window=400, sinks=4, weights=w, weights_before=w, decay=0.5)
        ver.verify(dev[0], dev[1], dev[2], tokens, accepted, draft_probs=dev[3])
        rd.evict_blocks(w, c.dev["bt"], c.dev["seq"], evicted, counts, keep=keep, weights_out=left, block_table_out=table, seq_lens_out=lens)
        rd.attend(c.dev["q"], table, lens, last)
    torch.cuda.synchronize()
    assert rd.device_status() == 0 and ver.device_status() == 0
    win.close(out, c.attention())
    first, tol = c.weights()
    c.window, c.sinks = 400, 4
    win.close(second, c.attention())
    more, tol2 = c.weights()
    win.close_weights(w, c, (0.5 * first + more, 0.5 * tol + tol2 + 2.0 ** -22 * (first + more)))
    for r in range(c.R):
        want = verified(target.view(c.R, q_len, V)[r].double().numpy(), draft.view(c.R, q_len - 1, V)[r].double().numpy(), x[r].tolist(),
                        u[r].numpy(), V)
        assert (tokens[r].tolist(), int(accepted[r])) == want[:2]
        kept = evicted_of(w[r].tolist(), c.bt[r].tolist(), int(c.seq[r]), keep, init, local)
        assert left[r].tolist() == kept[0] and table[r].tolist() == kept[1] and int(lens[r]) == kept[2]
        assert evicted[r].tolist() == kept[3] and int(counts[r]) == kept[4]
    assert counts.tolist()[0] == 7
    c.window, c.sinks = 0, 0
    c.bt, c.seq = table.cpu().numpy(), lens.cpu().numpy()
    win.close(last, c.attention())
