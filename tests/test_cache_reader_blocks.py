"""The selection behind scores of blocks that lie outside the index cache: their columns hold what an earlier step left."""

import numpy as np
import pytest
import torch

from tests import cache_reference as ref


def test_refusals_of_the_block_table():
    from indexer_projection_gb300 import binding as B, build
    from tests.test_cache_readers_host import P, select_args

    build.build()
    for kw, err in ((dict(block_table=P, num_blocks=1), B.PA_OK), (dict(block_table=P, num_blocks=0), B.PA_ERR_SHAPE),
                    (dict(block_table=P + 2, num_blocks=1), B.PA_ERR_ALIGN), (dict(num_blocks=0), B.PA_OK)):
        assert B.pre_attn_select_blocks(select_args(B, **kw), check=False) == err


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("q_len,bs", [(1, 16), (3, 256)])
def test_a_block_outside_the_cache_is_not_selected(fmt, q_len, bs):
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import CacheReader, PreAttn

    g = np.random.default_rng(q_len)
    seq, W, topk, init, local, heads = np.array([1500, 900, 0, 128 * 40], np.int32), 40, 5, 1, 1, 2
    R, M, blocks_held = len(seq), len(seq) * q_len, 48
    bt = g.permutation(blocks_held)[None, :W].repeat(R, 0).astype(np.int32)
    bt[0, 3], bt[1, 2], bt[3, 17], bt[3, 30] = blocks_held, -1, 2 ** 31 - 1, blocks_held + 7
    bt[0, 11] = -9  # a pinned block: selected all the same
    cache = torch.from_numpy(g.integers(0, 0x38, (blocks_held * 128, 128 if fmt == "fp8" else 72)).astype(np.uint8)).cuda()
    if fmt == "fp8":
        caches = PreAttn.fp8_caches(None, None, None, None, cache, 0, blocks_held * 128)
    else:
        caches = PreAttn.nvfp4_caches(None, 0, 0, cache, blocks_held * 128 // bs, bs * 72)
    rd = CacheReader(16, 1, cache_format=B.PA_CACHE_FP8 if fmt == "fp8" else B.PA_CACHE_NVFP4, caches=caches, max_requests=R,
                     q_len=q_len, bt_width=W, topk=topk, init_blocks=init, local_blocks=local, block_size=bs)
    iq = torch.randn(M, heads * 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    t_bt, t_seq = torch.from_numpy(bt).cuda(), torch.from_numpy(seq).cuda()
    scores = torch.full((heads, M, W * 128), 1e30, device="cuda")  # what an earlier step left
    picked = torch.full((M, heads, topk), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((M, heads), -7, dtype=torch.int32, device="cuda")
    for h in range(heads):
        rd.index_scores(iq, h, t_bt, t_seq, scores[h])
    assert rd.device_status() == B.PA_DEV_SLOT_RANGE
    rd.select_blocks(scores, t_seq, picked, counts, block_table=t_bt)
    assert rd.device_status() == B.PA_DEV_SLOT_RANGE
    left = scores.cpu().numpy()
    for m in range(M):
        r = m // q_len
        for b in np.nonzero((bt[r] < 0) | (bt[r] >= blocks_held))[0]:
            left[:, m, b * 128:(b + 1) * 128] = -np.inf
    want = ref.select(left, seq, q_len, W, init, local, topk)
    for m in range(M):
        for h in range(heads):
            n = int(counts[m, h])
            assert picked[m, h].tolist() == want[m][h] + [-1] * (topk - n) and n == len(want[m][h])
    # with every id inside, the table changes nothing and nothing is flagged
    t_bt = torch.from_numpy(np.where((bt < 0) | (bt >= blocks_held), 0, bt)).cuda()
    for h in range(heads):
        rd.index_scores(iq, h, t_bt, t_seq, scores[h])
    rd.select_blocks(scores, t_seq, picked, counts, block_table=t_bt)
    first = picked.clone(), counts.clone()
    rd.select_blocks(scores, t_seq, picked, counts)
    assert torch.equal(first[0], picked) and torch.equal(first[1], counts) and rd.device_status() == 0
    assert rd.select_blocks(scores[:, :0], t_seq[:0], picked[:0], counts[:0], block_table=t_bt[:0]) == B.PA_OK
    for bad in (t_bt.cpu(), t_bt.long(), t_bt[:, 1:]):
        with pytest.raises(ValueError):
            rd.select_blocks(scores, t_seq, picked, counts, block_table=bad)
