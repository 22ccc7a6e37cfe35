"""The readers at the largest sizes that the header allows: tables of 16384 blocks, lists of 256, 16 rows, 65535 requests.
Block tables name the blocks of a small cache many times over; the references are in 64 bits on the GPU."""

import numpy as np
import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
FORMATS = ["fp8", "nvfp4"]
W, POOL, D = 16384, 40, 128


def pool(fmt, nkv, group, bs=16):
    """A case whose one request owns every block of a cache of POOL (and its K, V by block, f64 on the GPU)."""
    c = ref.Case(fmt, [POOL * 128], 1, nkv, group, bs=bs, seed=110 + nkv).upload()
    kv = []
    for x in (c.k, c.v):  # [nkv, slots, 128] in the request's order
        s = c.bt[0].astype(np.int64)[:, None] * 128 + np.arange(128)
        kv.append(torch.from_numpy(x[:, s]).cuda())  # [nkv, POOL, 128 keys, 128]
    return c, torch.from_numpy(c.bt[0]).cuda(), *kv


def reader(c, q_len, width, topk, R):
    from indexer_projection_gb300.runner import CacheReader
    return CacheReader(c.nkv * c.group, c.nkv, cache_format=c.format, caches=c.caches, max_requests=R, q_len=q_len,
                       bt_width=width, topk=topk, block_size=c.bs)


def check_row(got, q, k, v, n_last, copies):
    """One row and KV head: got, q [group, 128]; k, v [blocks, 128, 128]; the last block's keys from n_last on are masked.
    copies [blocks]: how often a block is looked at.  The bound as in ref.Case.attention, its parts summed over the row."""
    x = torch.einsum("gd,bkd->gbk", q, k) * (D ** -0.5 * 1.4426950408889634)
    x[:, -1, n_last:] = -torch.inf
    w = torch.exp2(x - x.amax((1, 2), keepdim=True)) * copies[:, None]
    l = w.sum((1, 2))[:, None]
    want, mass = torch.einsum("gbk,bkd->gd", w, v) / l, torch.einsum("gbk,bkd->gd", w, v.abs()) / l
    n = float(copies.sum()) * 128
    # f16 weights 2^-11, ex2 2^-21, scores below 2^-12 here, sums n 2^-23 at most 2^-2 of .. in order of slices of at most
    # 2^14 keys each: 2^-9; twice (numerator and sum); bf16 output 2^-8; weights below f16's range 2^-34 of the largest value
    rel = 2.0 ** -11 + 2.0 ** -12 + min(n, 2.0 ** 14) * 2.0 ** -23
    tol = rel * (mass + want.abs()) + 2.0 ** -8 * want.abs() + n * 2.0 ** -34 * v.abs().amax() / l
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() - tol).max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len", [1, 16])
def test_every_block_of_the_widest_table(fmt, q_len):
    c, ids, k, v = pool(fmt, 1, 16)
    g = torch.Generator(device="cuda").manual_seed(q_len)
    order = torch.randint(0, POOL, (W,), generator=g, device="cuda")
    bt = ids[order][None].contiguous()
    n = W * 128 - 3
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn(q_len, 16 * D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((q_len, 16 * D), torch.nan, dtype=torch.bfloat16, device="cuda")
    rd = reader(c, q_len, W, 0, 1)
    rd.attend(q, bt, seq, out)
    assert rd.device_status() == 0
    counts = torch.bincount(order[:-1], minlength=POOL).double()
    for i in range(q_len):
        blocks = torch.cat((torch.arange(POOL, device="cuda"), order[-1:]))
        copies = torch.cat((counts, counts.new_ones(1)))
        check_row(out[i].view(16, D), q[i].view(16, D).double(), k[0][blocks], v[0][blocks],
                  n - q_len + i + 1 - (W - 1) * 128, copies)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_len,nkv", [(1, 2), (8, 1), (16, 1)])
def test_the_longest_lists(fmt, q_len, nkv):
    c, ids, k, v = pool(fmt, nkv, 4)
    R, topk = 3, 256
    g = torch.Generator(device="cuda").manual_seed(q_len)
    order = torch.randint(0, POOL, (R, W), generator=g, device="cuda")
    bt = ids[order].contiguous()
    seq = torch.tensor([W * 128, 300 * 128 + 5, 7000 * 128 + 64], dtype=torch.int32, device="cuda")
    q = torch.randn(R * q_len, nkv * 4 * D, generator=g, device="cuda").to(torch.bfloat16)
    blocks = torch.empty(R * q_len, nkv, topk, dtype=torch.int32, device="cuda")
    counts = torch.full((R * q_len, nkv), topk, dtype=torch.int32, device="cuda")
    last = [(int(seq[m // q_len]) - q_len + m % q_len) // 128 for m in range(R * q_len)]
    for m in range(R * q_len):
        for h in range(nkv):  # distinct blocks, the row's last among them
            b = torch.randperm(last[m], generator=g, device="cuda")[:topk].to(torch.int32)
            b[int(torch.randint(0, topk, (1,), generator=g, device="cuda"))] = last[m]
            blocks[m, h] = b
    out = torch.full_like(q, torch.nan)
    rd = reader(c, q_len, W, topk, R)
    rd.attend(q, bt, seq, out, blocks=blocks, counts=counts)
    assert rd.device_status() == 0
    for m in range(R * q_len):
        r, p = m // q_len, int(seq[m // q_len]) - q_len + m % q_len
        for h in range(nkv):
            b = blocks[m, h].long()
            b = torch.cat((b[b != last[m]], b[b == last[m]]))
            at = order[r, b]
            check_row(out[m].view(nkv, 4, D)[h], q[m].view(nkv, 4, D)[h].double(), k[h][at], v[h][at], p % 128 + 1,
                      torch.ones(topk, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("fmt", FORMATS)
def test_as_many_requests_as_allowed(fmt):
    # most of them padded; the others share one block
    c, ids, k, v = pool(fmt, 4, 1)
    R, width = 65535, 2
    bt = ids[:2].repeat(R, 1)
    seq = torch.zeros(R, dtype=torch.int32, device="cuda")
    live = {0: 1, 1: 130, 30000: 256, 65534: 77}
    for r, n in live.items():
        seq[r] = n
    q = torch.randn(R, 4 * D, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, torch.nan)
    rd = reader(c, 1, width, 1, R)
    rd.attend(q, bt, seq, out)
    assert rd.device_status() == 0
    for r, n in live.items():
        nb = (n + 127) // 128
        for h in range(4):
            check_row(out[r].view(4, 1, D)[h], q[r].view(4, 1, D)[h].double(), k[h, :nb], v[h, :nb], (n - 1) % 128 + 1,
                      torch.ones(nb, dtype=torch.float64, device="cuda"))
    rows = torch.ones(R, dtype=torch.bool)
    rows[list(live)] = False
    assert not out[rows.cuda()].any()
    # their scores and selection
    from indexer_projection_gb300.runner import CacheReader, PreAttn
    idx = torch.randint(0, 0x38, (2, 128 * (128 if fmt == "fp8" else 72)), dtype=torch.uint8, device="cuda")
    caches = PreAttn.fp8_caches(None, None, None, None, idx, 0, 256) if fmt == "fp8" else PreAttn.nvfp4_caches(None, 0, 0, idx, 2, 9216)
    ri = CacheReader(4, 4, cache_format=c.format, caches=caches, max_requests=R, q_len=1, bt_width=width, topk=1,
                     block_size=16 if fmt == "fp8" else 128)
    tb = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(R, 1)
    scores = torch.full((1, R, 256), 5.0, device="cuda")
    ri.index_scores(q, 0, tb, seq, scores[0])
    blocks, counts = (torch.full(s, -3, dtype=torch.int32, device="cuda") for s in ((R, 1, 1), (R, 1)))
    ri.select_blocks(scores, seq, blocks, counts, block_table=tb)
    assert ri.device_status() == 0
    assert (scores[0, rows.cuda()] == 5).all() and not counts[rows.cuda()].any() and (blocks[rows.cuda()] == -1).all()
    for r, n in live.items():
        assert (scores[0, r, (n + 127) // 128 * 128:] == 5).all() and counts[r] == 1
        top = scores[0, r, :(n + 127) // 128 * 128].view(-1, 128).amax(-1)
        assert blocks[r, 0, 0] == int(top.argmax())


@pytest.mark.parametrize("q_len,heads,topk,init,local", [(1, 1, 256, 1, 4), (2, 64, 7, 0, 1), (16, 1, 256, 200, 56)])
def test_the_widest_selection(q_len, heads, topk, init, local):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader

    width = W if heads == 1 else 500
    seq = np.array([width * 128 - 60], np.int32)
    s = torch.randn(heads, q_len, width * 128, generator=torch.Generator(device="cuda").manual_seed(topk), device="cuda")
    s = torch.round(s * 4) / 4
    rd = CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), max_requests=1, q_len=q_len, bt_width=width,
                     topk=topk, init_blocks=init, local_blocks=local)
    blocks, counts = (torch.full(x, -3, dtype=torch.int32, device="cuda") for x in ((q_len, heads, topk), (q_len, heads)))
    rd.select_blocks(s, torch.from_numpy(seq).cuda(), blocks, counts)
    assert rd.device_status() == 0
    top = s.view(heads, q_len, width, 128).amax(-1).double()
    b = torch.arange(width, device="cuda")
    for i in range(q_len):
        nb = (int(seq[0]) - q_len + i) // 128 + 1
        t = top[:, i].clone()
        t[:, (b < init) | (b >= nb - local)] = torch.inf
        t[:, b >= nb] = -torch.inf
        want = torch.sort(t, dim=-1, descending=True, stable=True).indices[:, :topk].sort(-1).values
        assert (counts[i] == topk).all() and torch.equal(blocks[i], want.to(torch.int32))
