"""The operators behind the pre-attention step, as cases to be measured.

The step leaves q, index_q and paged FP8 or NVFP4 caches; what a sparse
layer then does with them is measured here: the indexer scores over an NVFP4
index cache, the selection of each row's blocks from those scores, and the
attention over the FP8 or NVFP4 caches, on the selected blocks or on all.

Each case runs in one of two forms: `own` false computes it with elementary
torch operations in 32 bits, `own` true calls the framework.  `exact` is the
definition in 64 bits, from the cache formats' byte offsets.
"""

import math

import torch

own = False

D = 128          # head dim
BLOCK = 128      # keys a block
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def _scores(name, R, q_len, lo, hi, bs, n_iq, head, init=1, local=4):
    return dict(name=name, op="scores", R=R, q_len=q_len, lo=lo, hi=hi, bs=bs, n_iq=n_iq, head=head, init=init,
                local=local)


def _select(name, R, q_len, lo, hi, heads, topk, init=1, local=4):
    return dict(name=name, op="select", R=R, q_len=q_len, lo=lo, hi=hi, heads=heads, topk=topk, init=init, local=local)


def _attn(name, fmt, R, q_len, lo, hi, nkv, group=16, topk=0, own_blocks=0, init=1, local=4, bs=16, pad=0):
    # topk = 0: every block; otherwise own_blocks of a row's topk are its own, the others shared by its request's rows
    return dict(name=name, op="attn", fmt=fmt, R=R, q_len=q_len, lo=lo, hi=hi, nkv=nkv, group=group, topk=topk,
                own_blocks=own_blocks, init=init, local=local, bs=bs, pad=pad)


def listed():
    return [
        # one decode step of a small batch, ragged lengths: latency counts
        _scores("scores_nvfp4_decode", 8, 1, 1, 32768, 16, 1, 0),
        # 64 requests of 7 speculative verify rows
        _scores("scores_nvfp4_spec", 64, 7, 1024, 32767, 64, 2, 1),
        # the selection behind each of the two
        _select("select_decode", 8, 1, 1, 32768, 1, 16),
        _select("select_spec", 64, 7, 1024, 32767, 2, 16),
        # one request with a long context, all index heads
        _select("select_long", 1, 3, 130001, 131072, 4, 64),
        # a decode step's attention on its 16 selected blocks: the smallest call
        _attn("fp8_sparse_decode", "fp8", 8, 1, 1, 32768, 1, topk=16),
        # verify rows, each with four blocks of its own beside the shared ones
        _attn("fp8_sparse_spec", "fp8", 64, 7, 1024, 32767, 2, topk=16, own_blocks=4),
        # a dense layer's decode step, ragged lengths
        _attn("fp8_dense_decode", "fp8", 32, 1, 1, 32768, 2),
        # the same sparse calls on 4-bit caches, with pages longer than 16 tokens and eight query heads a KV head
        _attn("nvfp4_sparse_decode", "nvfp4", 5, 1, 4097, 131072, 4, group=8, topk=24, bs=64),
        _attn("nvfp4_sparse_spec", "nvfp4", 64, 7, 1024, 32767, 2, topk=16, own_blocks=4),
        # a large batch on a dense layer with every KV head
        _attn("nvfp4_dense_decode", "nvfp4", 64, 1, 1, 32768, 4),
        # one request's verify rows over a long context
        _attn("nvfp4_dense_long", "nvfp4", 1, 4, 131001, 131072, 4, bs=128, pad=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scores", "select", "attn", "attn", "attn", "attn"])
    R, q_len, hi = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 13]), _log(rng, 200, 32768)
    lo = rng.choice([q_len, max(q_len, hi // 32), max(q_len, hi - 77)])
    init, local = rng.choice([(1, 4), (0, 1), (1, 1), (2, 3)])
    if op == "scores":
        n_iq = rng.choice([1, 2, 4])
        return _nameless(_scores("", R, q_len, lo, hi, rng.choice([16, 32, 64, 128]), n_iq, rng.randrange(n_iq), init, local))
    if op == "select":
        return _nameless(_select("", R, q_len, lo, hi, rng.choice([1, 2]), rng.choice([8, 13, 16, 32, 48]), init, local))
    fmt, nkv, group = rng.choice(["fp8", "nvfp4"]), rng.choice([1, 2, 4]), rng.choice([16, 16, 8, 5, 1])
    topk = rng.choice([0, 0, 8, 16, 16, 24, 33])
    rows_own = min(rng.randrange(0, max(1, topk - init - local)), 6) if q_len > 1 else 0
    c = _nameless(_attn("", fmt, R, q_len, lo, hi, nkv, group, topk, rows_own, init, local,
                        16 if fmt == "fp8" else rng.choice([16, 32, 64, 128]), 0 if fmt == "fp8" else rng.choice([0, 64])))
    most = [max(x) for x in zip(*((w["bytes"], w["flops"]) for w in map(work, listed())))]
    while c["R"] > 1 and (work(c)["bytes"] > most[0] or work(c)["flops"] > most[1]):
        c["R"] -= (c["R"] + 3) // 4  # no more work than the largest listed case
    return c


def _nameless(c):
    c.pop("name")
    return c


def _mean_keys(c):
    return (max(c["lo"], c["q_len"]) + c["hi"]) / 2


def work(case):
    c = case
    keys, M = _mean_keys(c), c["R"] * c["q_len"]
    if c["op"] == "scores":
        pinned = min(keys, (c["init"] + c["local"] - 0.5) * BLOCK)
        return {"bytes": c["R"] * (keys - pinned) * 72 + M * (256 + 4 * keys), "flops": 2 * D * M * (keys - pinned)}
    if c["op"] == "select":
        return {"bytes": M * c["heads"] * (4 * keys + 4 * (c["topk"] + 1)), "flops": M * c["heads"] * keys}
    token = 264 if c["fmt"] == "fp8" else 144
    hq = c["nkv"] * c["group"]
    if c["topk"]:
        blocks = keys / BLOCK
        union = min(blocks, c["topk"] + (c["q_len"] - 1) * c["own_blocks"])
        read, seen = union * BLOCK, min(keys, c["topk"] * BLOCK)
    else:
        read, seen = keys, keys
    return {"bytes": c["R"] * c["nkv"] * read * token + 4 * D * M * hq, "flops": 4 * D * M * hq * seen}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _requests(c, g):
    """seq_lens [R] and a block table of distinct random blocks, -1 past a request's last."""
    R, W = c["R"], (c["hi"] + BLOCK - 1) // BLOCK
    lo = max(c["lo"], c["q_len"])
    seq = torch.randint(lo, max(c["hi"], lo) + 1, (R,), generator=g, device="cuda")
    W = max(W, (max(c["hi"], lo) + BLOCK - 1) // BLOCK)
    nb = (seq + BLOCK - 1) // BLOCK
    held = torch.arange(W, device="cuda")[None, :] < nb[:, None]
    pool = int(held.sum()) + 3
    perm = torch.randperm(pool, generator=g, device="cuda")
    bt = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    bt[held] = perm[: pool - 3].to(torch.int32)
    return seq.to(torch.int32), bt, pool


def _e2m1_groups(x):
    """Values [..., 128] as packed E2M1 bytes [..., 64] and the E4M3 codes of 8 group scales."""
    v = x.view(*x.shape[:-1], 8, 16)
    sf = (v.abs().amax(-1) / 6).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    y = v / sf.float().unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edges).to(torch.uint8)
    code = code | (((y < 0) & (code > 0)).to(torch.uint8) << 3)
    code = code.reshape(*x.shape[:-1], 64, 2)
    return code[..., 0] | (code[..., 1] << 4), sf.view(torch.uint8)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _fp8_caches(c, g, pool):
    pages = pool * 8
    out = {}
    for what in ("k", "v"):
        x = _randn(g, pages, 16, c["nkv"], D)
        s = x.abs().amax(-1) / 448  # per token and head
        code = (x / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        if what == "k":  # [page, head, d / 16, token, d % 16]
            code = code.view(pages, 16, c["nkv"], 8, 16).permute(0, 2, 3, 1, 4)
        else:            # [page, head, d, token]
            code = code.permute(0, 2, 3, 1)
        out[what + "_cache"] = code.contiguous()
        out[what + "_scale"] = s.permute(0, 2, 1).contiguous()
    return out


def _nvfp4_pages(x, bs, slot, swizzled, into):
    """Token rows x [tokens, 128] of one head into `slot` of the pages `into` [pages, page bytes]."""
    pages = x.shape[0] // bs
    data, sf = _e2m1_groups(x)
    at = slot * bs * 72
    into[:, at:at + bs * 64] = data.view(pages, bs * 64)
    if swizzled:  # scale of (token t, group g) at (t / 4) * 32 + 4 g + t % 4
        sf = sf.view(pages, bs // 4, 4, 8).permute(0, 1, 3, 2)
    into[:, at + bs * 64:at + bs * 72] = sf.reshape(pages, bs * 8)


def _select_blocks_for(c, g, seq):
    """Blocks as a selection leaves them: pinned ones, ones that a request's rows share, and own_blocks of a row alone."""
    R, q_len, nkv, topk = c["R"], c["q_len"], c["nkv"], c["topk"]
    W = (max(c["hi"], c["lo"], q_len) + BLOCK - 1) // BLOCK
    p = (seq.long()[:, None] - q_len + torch.arange(q_len, device="cuda"))          # [R, q_len]
    nb = (p // BLOCK + 1)[:, :, None, None]
    b = torch.arange(W, device="cuda")
    pinned = (b < c["init"]) | (b >= nb - c["local"])
    rank = torch.rand(R, 1, nkv, W, generator=g, device="cuda").argsort(-1).argsort(-1)
    shared = max(0, topk - c["init"] - c["local"] - c["own_blocks"])
    i = torch.arange(q_len, device="cuda")[None, :, None, None]
    mine = (rank >= shared + i * c["own_blocks"]) & (rank < shared + (i + 1) * c["own_blocks"])
    value = torch.where(rank < shared, 2.0, torch.where(mine, 1.0, 0.0)) - rank * 1e-4
    value = torch.where(pinned, 3.0, value)
    value = torch.where(b < nb, value, -math.inf).expand(R, q_len, nkv, W)
    k = min(topk, W)
    top, at = value.topk(k, dim=-1)
    at = torch.where(top > -math.inf, at, W).sort(-1).values
    blocks = torch.full((R * q_len, nkv, topk), -1, dtype=torch.int32, device="cuda")
    blocks[:, :, :k] = torch.where(at < W, at, -1).reshape(R * q_len, nkv, k).to(torch.int32)
    return blocks, (blocks >= 0).sum(-1).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    M = c["R"] * c["q_len"]
    s = {"case": c}
    if c["op"] == "scores":
        s["seq"], s["bt"], pool = _requests(c, g)
        bs = c["bs"]
        s["idx_cache"] = torch.empty(pool * BLOCK // bs, bs * 72, dtype=torch.uint8, device="cuda")
        _nvfp4_pages(_randn(g, pool * BLOCK, D), bs, 0, False, s["idx_cache"])
        s["iq"] = _randn(g, M, c["n_iq"] * D).to(torch.bfloat16)  # a normed index_q has unit RMS
        s["scale"] = float(torch.tensor(D ** -0.5 * math.log2(math.e), dtype=torch.float32))
        # columns that no row owns keep what an earlier step left there
        s["scores"] = torch.full((M, s["bt"].shape[1] * BLOCK), -5.0, device="cuda")
    elif c["op"] == "select":
        s["seq"], s["bt"], _ = _requests(c, g)
        W = s["bt"].shape[1]
        x = _randn(g, c["heads"], M, W * BLOCK) * 1.4427
        x = torch.round(x * 64) / 64  # near scores tie
        p = (s["seq"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device="cuda")).view(M, 1)
        j = torch.arange(W * BLOCK, device="cuda")
        nb = p // BLOCK + 1
        x = torch.where((j <= p) & (j // BLOCK >= c["init"]) & (j // BLOCK < nb - c["local"]), x, -math.inf)
        s["scores"] = torch.where(j // BLOCK < nb, x, 1e30)  # stale past a row's last block
        s["blocks"] = torch.zeros(M, c["heads"], c["topk"], dtype=torch.int32, device="cuda")
        s["counts"] = torch.zeros(M, c["heads"], dtype=torch.int32, device="cuda")
    else:
        s["seq"], s["bt"], pool = _requests(c, g)
        nkv, hq = c["nkv"], c["nkv"] * c["group"]
        s["q"] = (_randn(g, M, hq * D) * 1.5).to(torch.bfloat16)
        if c["fmt"] == "fp8":
            s.update(_fp8_caches(c, g, pool))
        else:
            bs = c["bs"]
            stride = 2 * nkv * bs * 72 + c["pad"]
            s["kv_cache"] = torch.zeros(pool * BLOCK // bs, stride, dtype=torch.uint8, device="cuda")
            for slot in range(2 * nkv):
                _nvfp4_pages(_randn(g, pool * BLOCK, D), bs, slot, slot % 2 == 1, s["kv_cache"])
            s["k_global"], s["v_global"] = 0.75, 1.25
        if c["topk"]:
            s["blocks"], s["counts"] = _select_blocks_for(c, g, s["seq"])
        s["out"] = torch.zeros(M, hq * D, dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _positions(s):
    c = s["case"]
    return s["seq"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device="cuda")  # [R, q_len]


def _unpack(data, sf):
    """Packed E2M1 [..., 64] and E4M3 group scales [..., 8] as f32 [..., 128]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
    code = torch.stack((data & 15, data >> 4), -1).flatten(-2)
    x = lut.index_select(0, code.reshape(-1).int()).view(*code.shape[:-1], 8, 16)
    return (x * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _linear_head(pages, bs, slot):
    """Pages [..., bytes] of bs tokens: the data [..., bs, 64] and scales [..., bs, 8] of a slot with linear scales."""
    at = slot * bs * 72
    return (pages[..., at:at + bs * 64].unflatten(-1, (bs, 64)),
            pages[..., at + bs * 64:at + bs * 72].unflatten(-1, (bs, 8)))


def _plain_scores(s):
    c = s["case"]
    R, q_len, W, bs = c["R"], c["q_len"], s["bt"].shape[1], c["bs"]
    blocks = s["idx_cache"].view(-1, BLOCK // bs, bs * 72)[s["bt"].clamp(min=0).long()]
    keys = _unpack(*_linear_head(blocks, bs, 0)).view(R, W * BLOCK, D)
    iq = s["iq"].view(R, q_len, c["n_iq"], D)[:, :, c["head"]].float()
    x = torch.matmul(iq, keys.transpose(1, 2)) * s["scale"]
    p = _positions(s)[:, :, None]
    j = torch.arange(W * BLOCK, device="cuda")
    nb = p // BLOCK + 1
    x = torch.where((j <= p) & (j // BLOCK >= c["init"]) & (j // BLOCK < nb - c["local"]), x, -math.inf)
    old = s["scores"].view(R, q_len, -1)
    old.copy_(torch.where(j // BLOCK < nb, x, old))
    return s["scores"]


def _plain_select(s):
    c = s["case"]
    H, M = c["heads"], c["R"] * c["q_len"]
    W = s["scores"].shape[2] // BLOCK
    nb = (_positions(s).view(M, 1) // BLOCK + 1)
    b = torch.arange(W, device="cuda")
    top = s["scores"].view(H, M, W, BLOCK).nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf).amax(-1)
    pinned = (b < c["init"]) | (b >= nb - c["local"])
    top = torch.where(b < nb, torch.where(pinned, math.inf, top), -math.inf)
    k = min(c["topk"], W)
    # pinned first, then by score; a stable sort leaves ties in block order
    first, at = torch.sort(top, dim=-1, descending=True, stable=True)
    at = torch.where(first[..., :k] > -math.inf, at[..., :k], W).sort(-1).values
    at = torch.where(at < W, at, -1).permute(1, 0, 2).to(torch.int32)
    s["blocks"].fill_(-1)
    s["blocks"][:, :, :k] = at
    s["counts"].copy_((at >= 0).sum(-1))
    return s["blocks"], s["counts"]


def _plain_kv(s, ids, head):
    """K and V in f32, [*ids.shape, 128 keys, 128], of physical blocks `ids` and KV heads `head` (broadcast against ids)."""
    c, nkv = s["case"], s["case"]["nkv"]
    if c["fmt"] == "fp8":
        k = s["k_cache"].view(-1, 8, nkv, 8, 16, 16)[ids, :, head].view(torch.float8_e4m3fn).float()  # [.., page, d / 16, t, d % 16]
        k = k.transpose(-3, -2).reshape(*ids.shape, BLOCK, D)
        v = s["v_cache"].view(-1, 8, nkv, D, 16)[ids, :, head].view(torch.float8_e4m3fn).float()
        v = v.transpose(-2, -1).reshape(*ids.shape, BLOCK, D)
        ks = s["k_scale"].view(-1, 8, nkv, 16)[ids, :, head].reshape(*ids.shape, BLOCK, 1)
        vs = s["v_scale"].view(-1, 8, nkv, 16)[ids, :, head].reshape(*ids.shape, BLOCK, 1)
        return k * ks, v * vs
    bs = c["bs"]
    slots = s["kv_cache"][:, :2 * nkv * bs * 72].unflatten(1, (nkv, 2, bs * 72)).unflatten(0, (-1, BLOCK // bs))
    kp, vp = slots[ids, :, head, 0], slots[ids, :, head, 1]
    k = _unpack(kp[..., :bs * 64].unflatten(-1, (bs, 64)), kp[..., bs * 64:].unflatten(-1, (bs, 8)))
    vf = vp[..., bs * 64:].unflatten(-1, (bs // 4, 8, 4)).transpose(-2, -1).reshape(*vp.shape[:-1], bs, 8)
    v = _unpack(vp[..., :bs * 64].unflatten(-1, (bs, 64)), vf)
    return (k.reshape(*ids.shape, BLOCK, D) * s["k_global"], v.reshape(*ids.shape, BLOCK, D) * s["v_global"])


def _softmax_v(x, v):
    """softmax(x) v with the maximum taken out, zeros for a row of -inf alone."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total == 0, 1.0, total)


def _plain_attn(s):
    c = s["case"]
    R, q_len, nkv, G, W = c["R"], c["q_len"], c["nkv"], c["group"], s["bt"].shape[1]
    M, scale, p = R * q_len, D ** -0.5, _positions(s)
    heads = torch.arange(nkv, device="cuda")
    q = s["q"].float().view(R, q_len, nkv, G, D)
    if c["topk"]:
        chosen = s["blocks"].long()                                              # [M, nkv, topk], -1 past the last
        r = torch.arange(M, device="cuda")[:, None, None] // q_len
        ids = s["bt"].long()[r, chosen.clamp(min=0)].clamp(min=0)
        k, v = _plain_kv(s, ids, heads[None, :, None].expand_as(ids))
        x = torch.matmul(q.view(M, nkv, G, D), k.flatten(2, 3).transpose(2, 3)) * scale
        j = chosen[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
        live = (chosen[..., None] >= 0) & (j <= p.view(M, 1, 1, 1))
        out = _softmax_v(torch.where(live.flatten(2)[:, :, None], x, -math.inf), v.flatten(2, 3))
    else:
        ids = s["bt"].long().clamp(min=0)[:, None, :].expand(R, nkv, W)
        k, v = _plain_kv(s, ids, heads[None, :, None].expand_as(ids))
        rows = q.permute(0, 2, 1, 3, 4).reshape(R, nkv, q_len * G, D)
        x = torch.matmul(rows, k.flatten(2, 3).transpose(2, 3)).view(R, nkv, q_len, G, W * BLOCK) * scale
        live = torch.arange(W * BLOCK, device="cuda") <= p[:, None, :, None, None]
        x = torch.where(live, x, -math.inf).view(R, nkv, q_len * G, W * BLOCK)
        out = _softmax_v(x, v.flatten(2, 3)).view(R, nkv, q_len, G, D).permute(0, 2, 1, 3, 4)
    s["out"].copy_(out.reshape(M, nkv * G * D))
    return s["out"]


# ---------------------------------------------------------- the framework's

def _front_end(s):
    """The handle that a program keeps for a layer: its shapes, its caches and a workspace."""
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300 import runner

    c = s["case"]
    kw = dict(max_requests=c["R"], q_len=c["q_len"], bt_width=s["bt"].shape[1], init_blocks=c["init"],
              local_blocks=c["local"])
    if c["op"] == "scores":
        caches = runner.PreAttn.nvfp4_caches(None, 0, 0, s["idx_cache"], s["idx_cache"].shape[0], c["bs"] * 72)
        return runner.CacheReader(16, 1, cache_format=B.PA_CACHE_NVFP4, caches=caches, block_size=c["bs"], **kw)
    if c["op"] == "select":
        return runner.CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), topk=c["topk"], **kw)
    if c["fmt"] == "fp8":
        caches = runner.PreAttn.fp8_caches(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], None,
                                           s["k_cache"].shape[0], 0)
        fmt = B.PA_CACHE_FP8
    else:
        caches = runner.PreAttn.nvfp4_caches(s["kv_cache"], s["kv_cache"].shape[0], s["kv_cache"].shape[1], None, 0, 0,
                                             s["k_global"], s["v_global"])
        fmt = B.PA_CACHE_NVFP4
    return runner.CacheReader(c["nkv"] * c["group"], c["nkv"], cache_format=fmt, caches=caches, block_size=c["bs"],
                              topk=c["topk"], sm_scale=D ** -0.5, **kw)


def _own(s):
    if "front" not in s:
        s["front"] = _front_end(s)
    f, op = s["front"], s["case"]["op"]
    if op == "scores":
        f.index_scores(s["iq"], s["case"]["head"], s["bt"], s["seq"], s["scores"], scale=s["scale"])
        return s["scores"]
    if op == "select":
        f.select_blocks(s["scores"], s["seq"], s["blocks"], s["counts"])
        return s["blocks"], s["counts"]
    if s["case"]["topk"]:
        f.attend(s["q"], s["bt"], s["seq"], s["out"], blocks=s["blocks"], counts=s["counts"])
    else:
        f.attend(s["q"], s["bt"], s["seq"], s["out"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "scores":
        return _plain_scores(state)
    if op == "select":
        return _plain_select(state)
    return _plain_attn(state)


# ------------------------------------------------------------------- exact

def _e4m3_table():
    """The value of each E4M3 code, from its fields."""
    out = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v = math.nan if code & 127 == 127 else v
        out.append(-v if code & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _nvfp4_rows(flat, page_bytes, bs, slot, tokens, swizzled, e4m3):
    """Token slots `tokens` [n] of a head's cache slot in 64 bits [n, 128], byte by byte."""
    page, t = (tokens // bs)[:, None], (tokens % bs)[:, None]
    d = torch.arange(D, device="cuda")
    base = page * page_bytes + slot * bs * 72
    byte = flat[base + t * 64 + (d // 64) * 32 + (d % 64) // 2].long()
    nib = torch.where(d % 2 == 0, byte & 15, byte >> 4)
    grp = d // 16
    at = (t // 4 * 4 + grp // 2) * 8 + (grp % 2) * 4 + t % 4 if swizzled else t * 8 + grp
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[nib & 7]
    return torch.where(nib >= 8, -mag, mag) * e4m3[flat[base + bs * 64 + at].long()]


def exact(case, seed):
    c = case
    if c["op"] == "select":
        return None
    s = prepare(case, seed)
    e4m3, q_len = _e4m3_table(), c["q_len"]
    seqs, bt = s["seq"].tolist(), s["bt"].long()
    if c["op"] == "scores":
        out, flat = s["scores"].double(), s["idx_cache"].view(-1)
        for r, n in enumerate(seqs):
            j = torch.arange((n + BLOCK - 1) // BLOCK * BLOCK, device="cuda")
            keys = _nvfp4_rows(flat, c["bs"] * 72, c["bs"], 0, bt[r, j // BLOCK] * BLOCK + j % BLOCK, False, e4m3)
            for i in range(q_len):
                p = n - q_len + i
                nb = p // BLOCK + 1
                x = (keys @ s["iq"][r * q_len + i, c["head"] * D:(c["head"] + 1) * D].double())[:nb * BLOCK] * s["scale"]
                b = j[:nb * BLOCK] // BLOCK
                x[(j[:nb * BLOCK] > p) | (b < c["init"]) | (b >= nb - c["local"])] = -math.inf
                out[r * q_len + i, :nb * BLOCK] = x
        return out
    nkv, G = c["nkv"], c["group"]
    out = torch.zeros(len(seqs) * q_len, nkv * G * D, dtype=torch.float64, device="cuda")
    d = torch.arange(D, device="cuda")
    for r, n in enumerate(seqs):
        for h in range(nkv):
            j = torch.arange(n, device="cuda")
            if c["topk"]:
                mine = s["blocks"][r * q_len:(r + 1) * q_len, h].long()
                union = mine[mine >= 0].unique()
                j = (union[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(-1)
                j = j[j < n]
            slot = bt[r, j // BLOCK] * BLOCK + j % BLOCK
            if c["fmt"] == "fp8":
                page, t = (slot // 16)[:, None], (slot % 16)[:, None]
                head = page * nkv + h
                k = e4m3[s["k_cache"].view(-1)[head * 2048 + (d // 16) * 256 + t * 16 + d % 16].long()]
                v = e4m3[s["v_cache"].view(-1)[head * 2048 + d * 16 + t].long()]
                k = k * s["k_scale"].view(-1)[head * 16 + t].double()
                v = v * s["v_scale"].view(-1)[head * 16 + t].double()
            else:
                flat, stride = s["kv_cache"].view(-1), s["kv_cache"].shape[1]
                k = _nvfp4_rows(flat, stride, c["bs"], 2 * h, slot, False, e4m3) * s["k_global"]
                v = _nvfp4_rows(flat, stride, c["bs"], 2 * h + 1, slot, True, e4m3) * s["v_global"]
            for i in range(q_len):
                m = r * q_len + i
                live = j <= n - q_len + i
                if c["topk"]:
                    live = live & torch.isin(j // BLOCK, s["blocks"][m, h].long())
                q = s["q"][m].view(nkv, G, D)[h].double()
                w = torch.softmax((q @ k[live].T) / math.sqrt(D), -1)
                out[m].view(nkv, G, D)[h] = w @ v[live]
    return out
