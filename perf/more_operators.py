"""Serving with caches of bounded size and with drafted tokens, as cases to be measured.

Beside the attention over the step's paged caches: the attention within a
sliding window with first tokens that stay visible, the weight that each block
of the cache got from a step's rows, the eviction of the blocks with the least
of it, and the verification of drafted tokens.

Each case runs in one of two forms: `own` false computes it with elementary
torch operations in 32 bits (the verification's sums in 64), `own` true calls
the framework.  `exact` is the definition in 64 bits, from the cache formats'
byte offsets.
"""

import math

import torch

own = False

D = 128          # head dim
BLOCK = 128      # keys a block
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def _attn(name, op, fmt, R, q_len, lo, hi, nkv, group=16, window=0, sinks=0, topk=0, bs=16, decay=1.0):
    # window = 0: every key; topk: the keys of that many blocks of each row and KV head
    return dict(name=name, op=op, fmt=fmt, R=R, q_len=q_len, lo=lo, hi=hi, nkv=nkv, group=group, window=window,
                sinks=sinks, topk=topk, bs=bs, decay=decay)


def _evict(name, R, lo, hi, keep, init=1, local=4):
    return dict(name=name, op="evict", R=R, lo=lo, hi=hi, keep=keep, init=init, local=local)


def _verify(name, R, drafts, vocab, accept, dtype="f32", draft_probs=True):
    # accept: the chance of a draft to be accepted, about
    return dict(name=name, op="verify", R=R, drafts=drafts, vocab=vocab, accept=accept, dtype=dtype,
                draft_probs=draft_probs)


def listed():
    return [
        # a decode step of a small batch within a short window: latency counts
        _attn("window_fp8_decode", "window", "fp8", 8, 1, 1, 32768, 1, window=1000, sinks=4),
        # 64 requests of 7 speculative verify rows, a window that ends inside blocks
        _attn("window_fp8_spec", "window", "fp8", 64, 7, 1024, 32767, 2, window=2047, sinks=5),
        # a large batch on 4-bit caches with every KV head
        _attn("window_nvfp4_decode", "window", "nvfp4", 64, 1, 1, 32768, 4, window=4096, sinks=128),
        # one request's verify rows, a long window
        _attn("window_nvfp4_long", "window", "nvfp4", 1, 4, 131001, 131072, 4, group=8, window=40000, sinks=130, bs=64),
        # a small decode batch, on every key, that keeps the blocks' weights for evictions
        _attn("weights_fp8_decode", "weights", "fp8", 8, 1, 1, 8192, 1),
        # a larger one, with older steps' weights fading
        _attn("weights_fp8_batch", "weights", "fp8", 32, 1, 1, 32768, 2, decay=0.98),
        # verify rows that read 16 selected blocks each
        _attn("weights_nvfp4_spec", "weights", "nvfp4", 64, 7, 1024, 32767, 2, topk=16),
        # every request of a batch over its budget
        _evict("evict_batch", 64, 1, 32768, 64),
        # few requests with very long contexts
        _evict("evict_long", 3, 500000, 1048576, 1000, init=4, local=16),
        # one request's six drafts
        _verify("verify_one", 1, 6, 32000, 0.8),
        # a batch's, over a large odd vocabulary
        _verify("verify_batch", 64, 6, 129281, 0.7),
        # a drafter without probabilities (each draft certain to it), 16-bit target probabilities
        _verify("verify_certain_bf16", 128, 3, 200064, 0.7, dtype="bf16", draft_probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "weights", "weights", "evict", "verify", "verify"])
    if op == "evict":
        R, hi = _log(rng, 1, 64), _log(rng, 1000, 1048576)
        init, local = rng.choice([(1, 4), (0, 1), (2, 3), (0, 0)])
        c = _evict("", R, rng.choice([1, hi // 2, max(1, hi - 700)]), hi, 8, init, local)
        c["keep"] = min(_log(rng, 8, 2000), (hi + BLOCK - 1) // BLOCK + 3)
        c["keep"] = max(c["keep"], init + max(local, 1))
        return _nameless(c)
    if op == "verify":
        c = _verify("", _log(rng, 1, 128), rng.choice([0, 1, 2, 3, 4, 6, 7, 15]), _log(rng, 500, 200064),
                    rng.choice([0.2, 0.5, 0.7, 0.9, 0.99]), rng.choice(["f32", "f32", "bf16"]), rng.random() < 0.7)
        while c["R"] > 1 and c["R"] * (c["drafts"] + 1) * c["vocab"] > 64 * 7 * 129281:
            c["R"] -= (c["R"] + 3) // 4
        return _nameless(c)
    fmt, nkv, group = rng.choice(["fp8", "nvfp4"]), rng.choice([1, 2, 4]), rng.choice([16, 16, 8, 5, 1])
    R, q_len, hi = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 13]), _log(rng, 200, 32768)
    lo = rng.choice([q_len, max(q_len, hi // 32), max(q_len, hi - 77)])
    window = _log(rng, 1, 8192) if op == "window" else rng.choice([0, 0, _log(rng, 64, 8192)])
    topk = 0 if window else rng.choice([0, 8, 16, 24])
    sinks = rng.choice([0, 1, 4, 100, 300]) if window else 0
    c = _nameless(_attn("", op, fmt, R, q_len, lo, hi, nkv, group, window, sinks, topk,
                        16 if fmt == "fp8" else rng.choice([16, 32, 64, 128]), rng.choice([1.0, 0.9, 0.0])))
    if op == "window":
        c["decay"] = 1.0
    most = [max(x) for x in zip(*((w["bytes"], w["flops"]) for w in map(work, listed())))]
    while c["R"] > 1 and (work(c)["bytes"] > most[0] or work(c)["flops"] > most[1]):
        c["R"] -= (c["R"] + 3) // 4  # no more work than the largest listed case
    return c


def _nameless(c):
    c.pop("name")
    return c


def work(case):
    c = case
    if c["op"] == "evict":
        entries = c["R"] * ((c["lo"] + c["hi"]) / 2 / BLOCK)
        return {"bytes": entries * 16, "flops": entries}  # the table and the weights, read and written
    if c["op"] == "verify":
        es = 4 if c["dtype"] == "f32" else 2
        # the row that the token is drawn from, its draft row where a draft was rejected, and the drafts' own values
        rows = 1 + (1 - c["accept"] ** c["drafts"] if c["draft_probs"] else 0)
        n = c["R"] * c["vocab"] * rows
        return {"bytes": n * es + c["R"] * (c["drafts"] + 1) * (2 * es + 12), "flops": 2 * n}
    keys, M = (max(c["lo"], c["q_len"]) + c["hi"]) / 2, c["R"] * c["q_len"]
    token, hq = 264 if c["fmt"] == "fp8" else 144, c["nkv"] * c["group"]
    if c["topk"]:
        read = seen = min(keys, c["topk"] * BLOCK)
    elif c["window"]:
        read, seen = min(keys, c["window"] + c["q_len"] - 1 + c["sinks"]), min(keys, c["window"] + c["sinks"])
    else:
        read = seen = keys
    return {"bytes": c["R"] * c["nkv"] * read * token + 4 * D * M * hq +
            (c["R"] * keys / BLOCK * 8 if c["op"] == "weights" else 0), "flops": 4 * D * M * hq * seen}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _requests(c, g, q_len=1):
    """seq_lens [R] and a block table of distinct random blocks, -1 past a request's last."""
    R, lo = c["R"], max(c["lo"], q_len)
    hi = max(c["hi"], lo)
    seq = torch.randint(lo, hi + 1, (R,), generator=g, device="cuda")
    W = (hi + BLOCK - 1) // BLOCK
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


def _select_blocks_for(c, g, seq, W):
    """Blocks as a selection leaves them: the first, the last four and others that a request's rows share."""
    R, q_len, nkv, topk = c["R"], c["q_len"], c["nkv"], c["topk"]
    p = (seq.long()[:, None] - q_len + torch.arange(q_len, device="cuda"))          # [R, q_len]
    nb = (p // BLOCK + 1)[:, :, None, None]
    b = torch.arange(W, device="cuda")
    rank = torch.rand(R, 1, nkv, W, generator=g, device="cuda")
    value = torch.where((b < 1) | (b >= nb - 4), 3.0, rank.expand(R, q_len, nkv, W))
    value = torch.where(b < nb, value, -math.inf)
    k = min(topk, W)
    top, at = value.topk(k, dim=-1)
    at = torch.where(top > -math.inf, at, W).sort(-1).values
    blocks = torch.full((R * q_len, nkv, topk), -1, dtype=torch.int32, device="cuda")
    blocks[:, :, :k] = torch.where(at < W, at, -1).reshape(R * q_len, nkv, k).to(torch.int32)
    return blocks, (blocks >= 0).sum(-1).to(torch.int32)


def _verify_inputs(c, g):
    R, k, V = c["R"], c["drafts"], c["vocab"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = {}
    target = torch.softmax(_randn(g, R, k + 1, V) * 3.0, -1)
    if c["draft_probs"]:
        # the drafter agrees with the target on `accept` of its mass
        draft = target[:, :k] * c["accept"] + torch.softmax(_randn(g, R, k, V) * 3.0, -1) * (1 - c["accept"])
        s["draft_probs"] = draft.to(dtype).view(R * k, V)
        draft = s["draft_probs"].float().view(R, k, V)
    else:
        draft = target[:, :k]
    # drawn from it: the largest of p / e, e exponential
    e = torch.empty(R, k, V, device="cuda").exponential_(generator=g)
    x = (draft / e).argmax(-1) if k else torch.zeros(R, 0, device="cuda", dtype=torch.long)
    if not c["draft_probs"] and k:  # certain drafts are likely ones
        target = target * (1 - c["accept"])
        target[:, :k].scatter_add_(2, x[..., None], torch.full((R, k, 1), c["accept"], device="cuda"))
        target[:, k] /= 1 - c["accept"]
    s["drafts"] = x.to(torch.int32)
    s["target"] = target.to(dtype).view(R * (k + 1), V)
    s["uniforms"] = torch.rand(R, k + 1, generator=g, device="cuda")
    s["tokens"] = torch.zeros(R, k + 1, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "verify":
        s.update(_verify_inputs(c, g))
        return s
    if c["op"] == "evict":
        s["seq"], s["bt"], _ = _requests(c, g)
        R, W = s["bt"].shape
        x = torch.empty(R, W, device="cuda").exponential_(generator=g)
        s["weights"] = torch.where(s["bt"] >= 0, torch.round(x * 256) / 256, 0.0)  # some are equal
        s["new_bt"], s["evicted"] = torch.zeros_like(s["bt"]), torch.zeros_like(s["bt"])
        s["new_seq"], s["counts"] = torch.zeros_like(s["seq"]), torch.zeros_like(s["seq"])
        s["new_weights"] = torch.zeros_like(s["weights"])
        return s
    s["seq"], s["bt"], pool = _requests(c, g, c["q_len"])
    nkv, hq, M = c["nkv"], c["nkv"] * c["group"], c["R"] * c["q_len"]
    s["q"] = (_randn(g, M, hq * D) * 1.5).to(torch.bfloat16)
    if c["fmt"] == "fp8":
        s.update(_fp8_caches(c, g, pool))
    else:
        bs = c["bs"]
        s["kv_cache"] = torch.zeros(pool * BLOCK // bs, 2 * nkv * bs * 72, dtype=torch.uint8, device="cuda")
        for slot in range(2 * nkv):
            _nvfp4_pages(_randn(g, pool * BLOCK, D), bs, slot, slot % 2 == 1, s["kv_cache"])
        s["k_global"], s["v_global"] = 0.75, 1.25
    if c["topk"]:
        s["blocks"], s["counts"] = _select_blocks_for(c, g, s["seq"], s["bt"].shape[1])
    s["out"] = torch.zeros(M, hq * D, dtype=torch.bfloat16, device="cuda")
    if c["op"] == "weights":
        s["before"] = torch.empty(*s["bt"].shape, device="cuda").exponential_(generator=g) * (s["bt"] >= 0)
        s["weights"] = torch.zeros_like(s["before"])
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


def _plain_kv(s, slots):
    """K and V in f32, [*slots.shape, KV heads, 128], of the token slots."""
    c, nkv = s["case"], s["case"]["nkv"]
    if c["fmt"] == "fp8":
        p, t = slots // 16, slots % 16
        k = s["k_cache"].view(-1, nkv, 8, 16, 16)[p, :, :, t].view(torch.float8_e4m3fn).float().flatten(-2)
        v = s["v_cache"].view(-1, nkv, D, 16)[p, :, :, t].view(torch.float8_e4m3fn).float()
        return (k * s["k_scale"].view(-1, nkv, 16)[p, :, t].unsqueeze(-1),
                v * s["v_scale"].view(-1, nkv, 16)[p, :, t].unsqueeze(-1))
    bs = c["bs"]
    p, t = slots // bs, slots % bs
    pages = s["kv_cache"].unflatten(1, (nkv, 2, bs * 72))
    codes, scales = pages[..., :bs * 64].unflatten(-1, (bs, 64)), pages[..., bs * 64:]
    k = _unpack(codes[:, :, 0][p, :, t], scales[:, :, 0].unflatten(-1, (bs, 8))[p, :, t])
    v = _unpack(codes[:, :, 1][p, :, t], scales[:, :, 1].unflatten(-1, (bs // 4, 8, 4))[p, :, t // 4, :, t % 4])
    return k * s["k_global"], v * s["v_global"]


def _softmax(x):
    """softmax over the last axis, zeros for a row of -inf alone."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _keys_of(s):
    """Positions of the keys that a request's rows see between them [R, N], -1 past the last."""
    c, n = s["case"], s["seq"].long()[:, None]
    if not c["window"]:
        j = torch.arange(s["bt"].shape[1] * BLOCK, device="cuda")[None, :]
        return torch.where(j < n, j, -1)
    first = (n - c["q_len"] - c["window"] + 1).clamp(min=0)
    j = first + torch.arange(c["window"] + c["q_len"] - 1, device="cuda")
    sink = torch.arange(c["sinks"], device="cuda").expand(c["R"], -1)
    return torch.cat((torch.where(sink < n, sink, -1), torch.where((j >= c["sinks"]) & (j < n), j, -1)), 1)


def _plain_attn(s):
    c = s["case"]
    R, q_len, nkv, G, W = c["R"], c["q_len"], c["nkv"], c["group"], s["bt"].shape[1]
    M, scale, p = R * q_len, D ** -0.5, _positions(s)
    got = torch.zeros(R, W, device="cuda")
    if c["topk"]:
        chosen = s["blocks"].long()                                              # [M, nkv, topk], -1 past the last
        j = (chosen[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(2)
        live = (j >= 0) & (j <= p.view(M, 1, 1))
        r = torch.arange(M, device="cuda")[:, None, None] // q_len
        slots = s["bt"].long()[r, (j // BLOCK).clamp(min=0)].clamp(min=0) * BLOCK + j % BLOCK
        out = torch.zeros(M, nkv, G, D, device="cuda")
        q = s["q"].float().view(M, nkv, G, D)
        for h in range(nkv):  # each head has blocks of its own
            k, v = (x[:, :, h] for x in _plain_kv(s, slots[:, h]))
            x = torch.matmul(q[:, h], k.transpose(1, 2)) * scale
            w = _softmax(torch.where(live[:, h, None], x, -math.inf))
            out[:, h] = torch.matmul(w, v)
            mine = w.sum(1).view(M, c["topk"], BLOCK).sum(-1)
            at = chosen[:, h].clamp(min=0)
            rows = torch.zeros(M, W, device="cuda").scatter_add_(1, at, torch.where(chosen[:, h] >= 0, mine, 0.0))
            got += rows.view(R, q_len, W).sum(1)
        out = out.view(M, nkv * G * D)
    else:
        j = _keys_of(s)
        slots = torch.gather(s["bt"].long(), 1, (j // BLOCK).clamp(min=0)).clamp(min=0) * BLOCK + j % BLOCK
        k, v = (x.transpose(1, 2) for x in _plain_kv(s, slots))                  # [R, nkv, N, D]
        rows = s["q"].float().view(R, q_len, nkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, nkv, q_len * G, D)
        x = torch.matmul(rows, k.transpose(2, 3)).view(R, nkv, q_len, G, -1) * scale
        at, pr = j[:, None, None, None], p[:, None, :, None, None]
        live = (at >= 0) & (at <= pr)
        if c["window"]:
            live = live & ((at > pr - c["window"]) | (at < c["sinks"]))
        w = _softmax(torch.where(live, x, -math.inf))
        out = torch.matmul(w.view(R, nkv, q_len * G, -1), v).view(R, nkv, q_len, G, D)
        out = out.permute(0, 2, 1, 3, 4).reshape(M, nkv * G * D)
        if c["op"] == "weights":
            got.scatter_add_(1, (j // BLOCK).clamp(min=0), torch.where(j >= 0, w.sum((1, 2, 3)), 0.0))
    s["out"].copy_(out)
    if c["op"] == "window":
        return s["out"]
    held = torch.arange(W, device="cuda") * BLOCK < s["seq"][:, None]
    s["weights"].copy_(torch.where(held, s["before"] * c["decay"] + got, 0.0))
    return s["out"], s["weights"]


def _plain_evict(s):
    c = s["case"]
    W, init, local = s["bt"].shape[1], c["init"], max(c["local"], 1)
    b = torch.arange(W, device="cuda")
    nb = ((s["seq"] + BLOCK - 1) // BLOCK)[:, None]
    pinned = ((b < init) | (b >= nb - local)) & (b < nb)
    value = torch.where(pinned, math.inf, torch.where(b < nb, s["weights"], -math.inf))
    # the largest first; a stable sort leaves ties in block order
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, b.expand_as(order))
    out = (b < nb) & (rank >= c["keep"])
    n = out.sum(-1, keepdim=True)
    # the row without them, moved up; then the evicted ones
    at = torch.sort(out.int(), dim=-1, stable=True).indices
    bt, w = s["bt"].gather(1, at), s["weights"].gather(1, at)
    s["new_bt"].copy_(torch.where(b < W - n, bt, -1))
    s["new_weights"].copy_(torch.where(b < W - n, w, 0.0))
    gone = s["bt"].gather(1, torch.sort(out.int(), dim=-1, descending=True, stable=True).indices)
    s["evicted"].copy_(torch.where(b < n, gone, -1))
    s["counts"].copy_(n[:, 0])
    s["new_seq"].copy_(s["seq"] - BLOCK * s["counts"])
    return s["new_bt"], s["new_seq"], s["new_weights"], s["evicted"], s["counts"]


def _plain_verify(s):
    c = s["case"]
    R, k, V = c["R"], c["drafts"], c["vocab"]
    target, x = s["target"].view(R, k + 1, V), s["drafts"].long()
    p = torch.gather(target[:, :k], 2, x[..., None])[..., 0].double()
    if c["draft_probs"]:
        q = torch.gather(s["draft_probs"].view(R, k, V), 2, x[..., None])[..., 0].double()
    else:
        q = torch.ones_like(p)
    good = s["uniforms"][:, :k].double() * q < p
    a = good.int().cumprod(-1).sum(-1)                                           # drafts accepted
    r = torch.arange(R, device="cuda")
    row = target[r, a].double()
    w = row
    if k:
        last = a.clamp(max=k - 1)
        if c["draft_probs"]:
            left = (row - s["draft_probs"].view(R, k, V)[r, last].double()).clamp(min=0)
        else:
            left = row.scatter(1, x[r, last][:, None], 0.0)
        left = torch.where(left.sum(-1, keepdim=True) > 0, left, row)
        w = torch.where((a < k)[:, None], left, row)
    run = w.cumsum(-1)
    token = (run <= s["uniforms"][:, k:].double() * run[:, -1:]).sum(-1)
    i = torch.arange(k + 1, device="cuda")
    drafts = torch.cat((x, x.new_zeros(R, 1)), 1)
    tokens = torch.where(i < a[:, None], drafts, torch.where(i == a[:, None], token[:, None], -1))
    s["tokens"].copy_(tokens)
    s["accepted"].copy_(a)
    return s["tokens"], s["accepted"]


# ---------------------------------------------------------- the framework's

def _front_end(s):
    """The handle that a program keeps: for a layer its shapes, its caches and a workspace."""
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300 import runner

    c = s["case"]
    if c["op"] == "verify":
        return runner.DraftVerifier(c["vocab"], c["drafts"] + 1)
    kw = dict(max_requests=c["R"], bt_width=s["bt"].shape[1])
    if c["op"] == "evict":
        return runner.CacheReader(16, 1, cache_format=B.PA_CACHE_FP8, caches=B.pa_caches(), q_len=1,
                                  init_blocks=c["init"], local_blocks=c["local"], **kw)
    if c["fmt"] == "fp8":
        caches = runner.PreAttn.fp8_caches(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], None,
                                           s["k_cache"].shape[0], 0)
        fmt = B.PA_CACHE_FP8
    else:
        caches = runner.PreAttn.nvfp4_caches(s["kv_cache"], s["kv_cache"].shape[0], s["kv_cache"].shape[1], None, 0, 0,
                                             s["k_global"], s["v_global"])
        fmt = B.PA_CACHE_NVFP4
    return runner.CacheReader(c["nkv"] * c["group"], c["nkv"], cache_format=fmt, caches=caches, block_size=c["bs"],
                              q_len=c["q_len"], topk=c["topk"], weigh=c["op"] == "weights", **kw)


def _own(s):
    if "front" not in s:
        s["front"] = _front_end(s)
    f, c = s["front"], s["case"]
    if c["op"] == "verify":
        f.verify(s["target"], s["drafts"], s["uniforms"], s["tokens"], s["accepted"], draft_probs=s.get("draft_probs"))
        return s["tokens"], s["accepted"]
    if c["op"] == "evict":
        f.evict_blocks(s["weights"], s["bt"], s["seq"], s["evicted"], s["counts"], keep=c["keep"],
                       weights_out=s["new_weights"], block_table_out=s["new_bt"], seq_lens_out=s["new_seq"])
        return s["new_bt"], s["new_seq"], s["new_weights"], s["evicted"], s["counts"]
    kw = {}
    if c["window"]:
        kw.update(window=c["window"], sinks=c["sinks"])
    if c["topk"]:
        kw.update(blocks=s["blocks"], counts=s["counts"])
    if c["op"] == "weights":
        kw.update(weights=s["weights"], weights_before=s["before"], decay=c["decay"])
    f.attend(s["q"], s["bt"], s["seq"], s["out"], **kw)
    return (s["out"], s["weights"]) if c["op"] == "weights" else s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_verify(state) if op == "verify" else _plain_evict(state) if op == "evict" else _plain_attn(state)


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
    if c["op"] == "verify":  # whole numbers
        return None
    s = prepare(case, seed)
    if c["op"] == "evict":  # the weights that stay, row by row; the rest are whole numbers
        rows = s["weights"].double().tolist()
        for row, n in zip(rows, s["seq"].tolist()):
            nb = (n + BLOCK - 1) // BLOCK
            free = [b for b in range(nb) if b >= c["init"] and b < nb - max(c["local"], 1)]
            free.sort(key=lambda b: (row[b], -b))
            for b in sorted(free[:max(nb - c["keep"], 0)], reverse=True):
                row.append(0.0)
                del row[b]
        return None, None, torch.tensor(rows, dtype=torch.float64, device="cuda"), None, None
    e4m3, q_len = _e4m3_table(), c["q_len"]
    seqs, bt = s["seq"].tolist(), s["bt"].long()
    nkv, G = c["nkv"], c["group"]
    out = torch.zeros(len(seqs) * q_len, nkv * G * D, dtype=torch.float64, device="cuda")
    total = torch.zeros(*bt.shape, dtype=torch.float64, device="cuda")
    d = torch.arange(D, device="cuda")
    for r, n in enumerate(seqs):
        if c["op"] == "weights":
            nb = (n + BLOCK - 1) // BLOCK
            total[r, :nb] = s["before"][r, :nb].double() * c["decay"]
        for h in range(nkv):
            j = torch.arange(n, device="cuda")
            if c["window"]:
                j = j[(j < c["sinks"]) | (j > n - q_len - c["window"])]
            if c["topk"]:
                mine = s["blocks"][r * q_len:(r + 1) * q_len, h].long()
                j = j[torch.isin(j // BLOCK, mine)]
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
                m, p = r * q_len + i, n - q_len + i
                live = j <= p
                if c["window"]:
                    live = live & ((j < c["sinks"]) | (j > p - c["window"]))
                if c["topk"]:
                    live = live & torch.isin(j // BLOCK, s["blocks"][m, h].long())
                q = s["q"][m].view(nkv, G, D)[h].double()
                w = torch.softmax((q @ k[live].T) / math.sqrt(D), -1)
                out[m].view(nkv, G, D)[h] = w @ v[live]
                if c["op"] == "weights":
                    total[r].index_add_(0, j[live] // BLOCK, w.sum(0))
    return (out, total) if c["op"] == "weights" else out
