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


# ----------------------------------------------------------- padded batches

def padded(fmt, q_len, R, window, sinks, nkv, group, seed):
    """Requests of a block or two between, behind and in runs of such without keys, many of them a CTA."""
    g = np.random.default_rng(seed)
    seq = np.where(g.random(R) < 0.5, 0, g.integers(q_len, 300, R))
    seq[:5], seq[R // 2:R // 2 + 40], seq[-9:] = [200, 0, 0, 0, 131], 0, 0
    seq[R // 3:R // 3 + 30] = np.tile([260, 0, 0], 10)
    return case(fmt, seq.tolist(), q_len, nkv, group, window, sinks, seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len", [("fp8", 5), ("fp8", 8), ("nvfp4", 3), ("nvfp4", 7)])
@pytest.mark.parametrize("R,nkv,window", [(1000, 2, 0), (300, 1, 0), (2000, 1, 1000), (160, 4, 1000)])
def test_padded_batches(fmt, q_len, R, nkv, window):
    c = padded(fmt, q_len, R, window, 2 if window else 0, nkv, 1, R + q_len)
    if window:
        c.W += 10  # (a window wider than the table is none)
        c.bt = np.concatenate((c.bt, np.full((R, 10), -1, np.int32)), 1)
    c.upload()
    out, w = check(c, SLICED)
    rd = c.reader(weigh=True)
    for _ in range(30):  # back to back
        rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, window=c.window, sinks=c.sinks, weights=w)
    assert rd.device_status() == 0
    second = win.attend(c, rd, weights=True)
    assert torch.equal(out, second[0]) and torch.equal(w, second[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len", [("fp8", 5), ("fp8", 8), ("nvfp4", 3), ("nvfp4", 7)])
def test_nan_values_behind_requests_without_keys(fmt, q_len):
    # in every second request the last key's value has a NaN, which its last row alone sees
    c = padded(fmt, q_len, 1000, 0, 0, 2, 1, 7 + q_len)
    want = c.attention()
    nan = np.zeros((c.M, 2, 128), bool)
    for r, n in enumerate(c.seq.tolist()):
        if n >= q_len and r % 2 == 0:
            put_nan(c, "value", r, n - 1)
            nan[r * q_len + q_len - 1, 0, 37 if fmt == "fp8" else slice(32, 48)] = True
    assert 100 < nan.any((1, 2)).sum() < c.R
    c.upload()
    rd = c.reader(weigh=True)
    for _ in range(5):
        out, w = win.attend(c, rd, weights=True)
        assert path(rd) == TILES | SLICED and rd.device_status() == 0
        got = out.double().cpu().numpy().reshape(nan.shape)
        assert (np.isnan(got) == nan).all()
        over = np.where(nan, -1.0, np.abs(got - want[0].reshape(got.shape)) - want[1].reshape(got.shape))
        assert (over <= 0).all()
    win.close_weights(w, c, c.weights())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len", [("fp8", 5), ("nvfp4", 7)])
def test_a_padded_batch_in_a_graph(fmt, q_len):
    # captured once, replayed with other lengths: every request there, some, one, none
    c = padded(fmt, q_len, 700, 0, 0, 1, 2, 90 + q_len)
    full = c.seq.copy()
    c.upload()
    rd = c.reader(weigh=True)
    out, w = torch.zeros(c.M, 2 * 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.R, c.W, device="cuda")
    call = lambda: rd.attend(c.dev["q"], c.dev["bt"], c.dev["seq"], out, weights=w)  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert path(rd) == TILES | SLICED
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    live = np.nonzero(full)[0]
    for kept in (live, live[::3], live[:1], live[-1:], live[:0], live):
        c.seq = np.zeros_like(full)
        c.seq[kept] = full[kept]
        c.dev["seq"].copy_(torch.from_numpy(c.seq))
        out.fill_(3), w.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        win.close(out, c.attention())
        win.close_weights(w, c, c.weights())
    assert rd.device_status() == 0


# ----------------------------------------------------- windows, rows, layouts

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k,window,sinks", [(k, *x) for k, x in enumerate([
    (1, 0), (1, 1), (2, 0), (15, 3), (16, 0), (127, 1), (128, 0), (129, 4), (130, 127), (300, 128), (1, 129), (700, 300)])])
def test_every_window_a_cta_an_item(fmt, k, window, sinks):
    q_len = ((5, 8, 6) if fmt == "fp8" else (3, 8, 5))[k % 3]
    lengths = [q_len, 128, 129, 300, 0, 1100, 1029, 128 + q_len]
    c = case(fmt, lengths * 5, q_len, 2, (4, 16, 1)[k % 3], window, sinks, seed=k).poison().upload()
    check(c, WHOLE)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len", [("fp8", 5), ("fp8", 8), ("nvfp4", 5), ("nvfp4", 8)])
@pytest.mark.parametrize("window,sinks", [(1, 2000), (15, 2100), (129, 1999), (4000, 0)])
def test_every_window_in_slices(fmt, q_len, window, sinks):
    c = case(fmt, [6000 + q_len, 0, 2500, q_len, 4097], q_len, 1, 8, window, sinks, seed=window + q_len).poison().upload()
    check(c, SLICED)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len,nkv,group", [
    ("nvfp4", 3, 1, 8), ("nvfp4", 4, 4, 5), ("fp8", 5, 2, 1), ("nvfp4", 5, 2, 1), ("fp8", 6, 4, 3), ("fp8", 7, 2, 16), ("nvfp4", 7, 2, 16),
    ("fp8", 8, 1, 13), ("fp8", 9, 1, 16), ("nvfp4", 9, 1, 16), ("nvfp4", 10, 2, 11), ("fp8", 13, 2, 4), ("nvfp4", 13, 2, 4), ("fp8", 16, 4, 16),
    ("nvfp4", 16, 1, 16)])
@pytest.mark.parametrize("window", [0, 200])
def test_rows_and_heads(fmt, q_len, nkv, group, window):
    lengths = [q_len, 300, 0, 129 + q_len, 940, 128]
    if window:  # as many items as are not dealt to clusters
        lengths = (lengths * 14)[:-(-77 // (nkv * (2 if q_len > 8 else 1)))]
    c = case(fmt, lengths, q_len, nkv, group, window, 5 if window else 0, seed=q_len, extra_width=2 if window else WIDE, k_global=0.5,
             v_global=1.5)
    if window:
        c.poison()
    check(c.upload(), WHOLE if window else SLICED)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,bs,kps,pad", [("fp8", 16, 8, 0), ("fp8", 16, 16, 0), ("fp8", 16, 9, 0), ("nvfp4", 4, 8, 32),
                                            ("nvfp4", 8, 8, 0), ("nvfp4", 32, 8, 64), ("nvfp4", 64, 8, 0), ("nvfp4", 128, 8, 96),
                                            ("nvfp4", 256, 8, 0), ("nvfp4", 1024, 8, 32)])
def test_page_layouts(fmt, bs, kps, pad):
    c = case(fmt, [700, 90, 1300], 5, 2, 8, bs=bs, kps=kps, pad=pad, seed=bs + kps, extra_width=WIDE).upload()
    check(c, SLICED)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [6, 9])
def test_fp8_queries(fmt, q_len):
    c = case(fmt, [400, 77, 0, 1000], q_len, 2, 16, seed=15, extra_width=WIDE).upload()
    q8 = (c.q.float() / 0.25).to(torch.float8_e4m3fn).cuda()
    check(c, SLICED, q=q8, q_fp8_scale=0.25)
    wide = torch.full((c.M, q8.shape[1] + 48), float("nan"), device="cuda").to(torch.float8_e4m3fn)  # rows with a stride
    wide[:, :q8.shape[1]] = q8
    rd = c.reader(weigh=True)
    got = win.attend(c, rd, q=wide, q_fp8_scale=0.25, weights=True)
    want = win.attend(c, rd, q=q8, q_fp8_scale=0.25, weights=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 4000])
def test_bad_blocks_and_requests(fmt, window):
    c = case(fmt, [900, 500, 2, 128 * 8 + 1, 6000], 5, 1, 16, window, 130 if window else 0, seed=6, extra_width=WIDE)
    c.seq[3] = 128 * c.W + 1
    c.upload()
    c.bt[0, 5], c.bt[1, 1], c.bt[4, 40], c.bt[4, 3] = -1, c.pool, 2 ** 31 - 1, -7
    c.dev["bt"] = torch.from_numpy(c.bt).cuda()
    out, _ = check(c, SLICED, status=1)
    assert (out[10:20] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_every_block_outside_the_cache(fmt):
    c = case(fmt, [700, 300, 513], 5, 2, 4, seed=16, extra_width=WIDE).upload()
    c.bt[1] = -1
    c.dev["bt"] = torch.from_numpy(c.bt).cuda()
    out, w = check(c, SLICED, status=1)
    assert (out[5:10] == 0).all() and (w[1] == 0).all()


# ------------------------------------------------------------- lists of blocks

@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q_len,nkv,topk,mode", [("fp8", 7, 2, 4, WHOLE), ("nvfp4", 7, 2, 4, WHOLE), ("fp8", 8, 1, 40, SLICED),
                                                     ("nvfp4", 8, 1, 40, SLICED), ("fp8", 11, 1, 8, SLICED), ("nvfp4", 4, 1, 64, SLICED)])
def test_lists_of_blocks(fmt, q_len, nkv, topk, mode):
    c = case(fmt, [3000, q_len, 0, 260 + q_len, 128 * 9], q_len, nkv, 8, seed=100 + q_len, extra_width=WIDE).upload()
    blocks, counts, lists = ref.random_lists(c, topk, seed=topk)
    blocks[0, 0, :4], counts[0, 0], lists[0][0] = [1, 3, 1, 3], 4, [1, 3]  # a block twice
    check(c, mode, (blocks, counts), sel=lists)
    blocks[0, 0, :4] = [1, 7000, -5, 3]  # outside the request
    check(c, mode, (blocks, counts), sel=lists, status=1)
    counts[:q_len] = 0  # a request whose lists are empty
    for m in range(q_len):
        lists[m] = [[] for _ in range(nkv)]
    out, _ = check(c, mode, (blocks, counts), sel=lists)
    assert (out[:q_len] == 0).all()


# -------------------------------------------------------- far values, NaN

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [5, 8])
@pytest.mark.parametrize("spread", [2.0, 24.0, 60.0])
@pytest.mark.parametrize("mode", [SLICED, WHOLE])
def test_far_scales_and_peaked_rows(fmt, q_len, spread, mode):
    # V scales near each other and over 2^24 and 2^60; head rows of queries from 2^-30 to 2^5: nearly even weights and a single one
    if mode == SLICED:
        c = case(fmt, [700, 130, 512], q_len, 2, 16, seed=30 + q_len, spread=spread, extra_width=WIDE)
    else:
        c = case(fmt, [700, 130, 512, 0] * 10, q_len, 2, 16, 260, 4, seed=30 + q_len, spread=spread)
    if fmt == "fp8":  # (K scales stay near each other)
        even = np.float32(0.01)
        c.scales["k"][np.isfinite(c.scales["k"])] = even
        for r, n in enumerate(c.seq.tolist()):
            j = np.arange(n)
            slot = c.bt[r, j // 128].astype(np.int64) * 128 + j % 128
            page, t = slot // 128 * c.kps + slot % 128 // 16, slot % 16
            for h in range(c.nkv):
                code = c.bytes["k"].reshape(-1, 2048)[page * c.nkv + h].reshape(-1, 8, 16, 16)[np.arange(n), :, t].reshape(n, 128)
                c.k[h, slot] = ref.E4M3[code] * np.float64(even)
    c.q = (c.q.float().view(-1, 2, 16, 128) * torch.tensor([2.0 ** e for e in range(-30, 6, 9)] * 4)[:, None]).to(torch.bfloat16).view(c.M, -1)
    check(c.upload(), mode)


def put_nan(c, what, r, j):
    """NaN in key j of request r, KV head 0: a value's code (FP8) or the scale of its dims 32 .. 47 (NVFP4), a scale of FP8."""
    from tests.test_window_and_weights import put_nan as put
    put(c, what, r, j)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,what", [("fp8", "value"), ("fp8", "k"), ("fp8", "v"), ("nvfp4", "value"), ("nvfp4", "k")])
@pytest.mark.parametrize("q_len,mode", [(7, "window, sliced"), (7, "window, whole"), (5, "window, whole"), (7, "lists"), (8, "lists")])
def test_a_nan_reaches_the_rows_that_see_it(fmt, what, q_len, mode):
    lists, sel = mode == "lists", None
    if lists:  # rows of even number attend block 1
        c = case(fmt, [700, 300], q_len, 1, 16, seed=50 + q_len, extra_width=WIDE)
        blocks, counts = np.tile(np.array([0, 2, 5], np.int32), (c.M, 1, 1)), np.full((c.M, 1), 3, np.int32)
        blocks[::2, 0, 1] = 1
        sel = [[[b for b in blocks[m, 0] if b * 128 < (700 if m < q_len else 300)]] for m in range(c.M)]
        blocks[q_len:, 0, 2], counts[q_len:] = -1, 2
        keys = [130, 698]
    elif mode == "window, sliced":
        c = case(fmt, [6700, 300], q_len, 1, 16, 260, 2000, seed=50 + q_len)
        keys = [6700 - q_len + 1 - 260, 6698, 3000]
    else:
        c = case(fmt, [700, 300] * 39, q_len, 1, 16, 260, 2, seed=50 + q_len)
        keys = [700 - q_len + 1 - 260, 698, 300]  # the window's end, the rows' own keys, one that none sees
    want = c.attention(sel)
    for j in keys:
        put_nan(c, what, 0, j)
    c.upload()
    rd = c.reader(topk=3 if lists else 0, weigh=True)
    got, w = win.attend(c, rd, (blocks, counts) if lists else None, weights=True)
    assert path(rd) == TILES | (SLICED if mode == "window, sliced" else WHOLE)
    got = got.double().cpu().numpy().reshape(c.M, 16, 128)
    dims = np.ones(128, bool)
    if what == "value":
        dims[:] = False
        dims[37 if fmt == "fp8" else slice(32, 48)] = True
    nan = np.zeros(got.shape, bool)
    for i in range(q_len):
        if set(keys) & set(c.row_positions(0, i, None if sel is None else sel[i][0]).tolist()):
            nan[i][:, dims] = True
    assert nan[:q_len].any() and not nan[:q_len].all()
    assert (np.isnan(got) == nan).all()
    over = np.where(nan, -1.0, np.abs(got - want[0].reshape(got.shape)) - want[1].reshape(got.shape))
    assert (over <= 0).all()
    assert torch.isfinite(w[1:]).all() and (what == "k" or torch.isfinite(w).all())
