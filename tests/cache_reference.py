"""A plain 64-bit reference of what is read back of the caches: the NVFP4
indexer scores, the block selection and the attention, from the byte offsets
that include/pre_attn.h gives, row by row, with the worst-case error that the
kernels' arithmetic allows beside each attention value.

Cache bytes that no key of a request owns hold NaN: FP8 pages NaN scales and,
with stale "nan", NaN codes; NVFP4 pages NaN scales and codes of -6 whatever
`stale` says.  A kernel that looks at them fails.
"""

import math

import numpy as np
import torch

D = 128
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3_table():
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


E4M3 = e4m3_table()


def bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16)


class Case:
    """Requests with their block tables, K / V (or index) caches, and the decoded K and V of every key.

    fp8: random codes with per-token scales around `scale` (spread over `spread` powers of two); nvfp4: random codes and
    group scales.  seq_lens: a list of R lengths."""

    def __init__(self, fmt, seq_lens, q_len, nkv=1, group=16, bs=16, kps=8, pad=0, seed=0, stale="nan", spread=2.0,
                 extra_width=0, q_scale=1.0, k_global=1.0, v_global=1.0):
        g = np.random.default_rng(seed)
        self.fmt, self.q_len, self.nkv, self.group, self.bs, self.kps = fmt, q_len, nkv, group, bs, kps
        self.seq = np.array(seq_lens, np.int32)
        self.R, self.M = len(seq_lens), len(seq_lens) * q_len
        self.k_global, self.v_global = k_global, v_global
        nb = (np.maximum(self.seq, 0) + 127) // 128
        self.W = int(max(nb.max(initial=0), 1)) + extra_width
        per = 1 if bs <= 128 else bs // 128
        pool = (int(nb.sum()) + 3 + per) // per * per
        perm = g.permutation(pool)
        self.bt = np.full((self.R, self.W), -1, np.int32)
        at = 0
        for r in range(self.R):
            self.bt[r, :nb[r]] = perm[at:at + nb[r]]
            at += nb[r]
        self.pool = pool
        self.q = bf16(g.standard_normal((self.M, nkv * group * D)) * q_scale)
        fill = 0x7f if stale == "nan" else 0xA5
        ns = pool * 128  # slots
        used = np.zeros(ns, bool)
        for r in range(self.R):
            j = np.arange(max(int(self.seq[r]), 0))
            used[self.bt[r, j // 128].astype(np.int64) * 128 + j % 128] = True
        self.k = np.full((nkv, ns, D), math.nan)
        self.v = np.full((nkv, ns, D), math.nan)
        self.vs = np.zeros((nkv, ns))  # fp8: the V scales
        n = int(used.sum())
        slot = np.nonzero(used)[0].astype(np.int64)
        d = np.arange(D)
        if fmt == "fp8":
            pages = pool * kps
            self.bytes = {w: np.full(pages * nkv * 2048, fill, np.uint8) for w in "kv"}
            self.scales = {w: np.full(pages * nkv * 16, math.nan, np.float32) for w in "kv"}
            self.pages = pages
            page, t = slot // 128 * kps + slot % 128 // 16, slot % 16
            for h in range(nkv):
                for w, dst in (("k", self.k), ("v", self.v)):
                    code = torch.from_numpy(g.standard_normal((n, D)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                    code = code.view(torch.uint8).numpy()
                    sc = (0.01 * 2.0 ** (g.random(n) * spread - spread / 2)).astype(np.float32)
                    base = (page * nkv + h)[:, None]
                    off = base * 2048 + (d // 16 * 256 + d % 16 + t[:, None] * 16 if w == "k" else d * 16 + t[:, None])
                    self.bytes[w][off] = code
                    self.scales[w][(page * nkv + h) * 16 + t] = sc
                    dst[h, slot] = E4M3[code] * sc[:, None].astype(np.float64)
                    if w == "v":
                        self.vs[h, slot] = sc
        else:
            self.page_bytes = 2 * nkv * bs * 72 + pad
            npages = ns // bs
            self.pages = npages
            kv = np.full((npages, self.page_bytes), 0xff, np.uint8)  # nibble -6, scale NaN
            flat = kv.reshape(-1)
            page, t = (slot // bs)[:, None], (slot % bs)[:, None]
            grp = np.arange(8)
            for sl in range(2 * nkv):
                h, isv = sl // 2, sl % 2
                nib = g.integers(0, 16, (n, D)).astype(np.uint8)
                sf = torch.from_numpy(np.exp2(g.random((n, 8)) * 4 - 4)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                base = page * self.page_bytes + sl * bs * 72
                flat[base + t * 64 + np.arange(64)] = nib[:, 0::2] | (nib[:, 1::2] << 4)
                so = (t // 4 * 4 + grp // 2) * 8 + grp % 2 * 4 + t % 4 if isv else t * 8 + grp
                flat[base + bs * 64 + so] = sf
                val = E2M1[nib] * np.repeat(E4M3[sf], 16, axis=1)
                (self.v if isv else self.k)[h, slot] = val * (v_global if isv else k_global)
            self.kv = kv

    # -------------------------------------------------------------- to the GPU
    def upload(self):
        from indexer_projection_gb300 import binding as B
        from indexer_projection_gb300.runner import PreAttn

        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.dev = {"bt": t(self.bt), "seq": t(self.seq), "q": self.q.cuda()}
        if self.fmt == "fp8":
            for w in "kv":
                self.dev[w], self.dev[w + "s"] = t(self.bytes[w]), t(self.scales[w])
            self.caches = PreAttn.fp8_caches(self.dev["k"], self.dev["v"], self.dev["ks"], self.dev["vs"], None, self.pages, 0)
            self.format = B.PA_CACHE_FP8
        else:
            self.dev["kv"] = t(self.kv)
            self.caches = PreAttn.nvfp4_caches(self.dev["kv"], self.pages, self.page_bytes, None, 0, 0, self.k_global,
                                               self.v_global)
            self.format = B.PA_CACHE_NVFP4
        return self

    def reader(self, topk=0, flags=0, max_requests=None, **kw):
        from indexer_projection_gb300.runner import CacheReader
        return CacheReader(self.nkv * self.group, self.nkv, cache_format=self.format, caches=self.caches,
                           max_requests=max_requests or max(self.R, 1), q_len=self.q_len, bt_width=self.W, topk=topk,
                           block_size=self.bs if self.fmt == "nvfp4" else 16,
                           kv_page_stride=self.kps if self.fmt == "fp8" else 0, flags=flags, **kw)

    # -------------------------------------------------------------- reference
    def row_keys(self, r, i, blocks=None):
        """Slots of the keys that row i of request r sees (blocks: its list, or None for all)."""
        n = int(self.seq[r])
        if n < max(self.q_len, 1) or (n + 127) // 128 > self.W:
            return np.zeros(0, np.int64)
        p = n - self.q_len + i
        j = np.arange(p + 1)
        if blocks is not None:
            j = j[np.isin(j // 128, [b for b in blocks if 0 <= b <= p // 128])]
        blk = self.bt[r, j // 128].astype(np.int64)
        return (blk * 128 + j % 128)[blk >= 0]

    def attention(self, lists=None, q=None, sm_scale=D ** -0.5):
        """out [M, heads * 128] and the bound on the kernel's error, both f64.

        The bound, with w_j the weights exp2(s_j - max): the score's error is at most 2^-21 of scale * sum |q k| (128
        f32 products and sums, two f32 factors) plus 2^-21 (|s| + 16) for the subtraction of the reference; a weight's
        relative error ln 2 of that, 2^-21 for ex2, 2^-11 for its rounding to f16, and where f16 is subnormal half its
        step, 2^-25, against a largest weight of 2^9 or more and in units of a power of two up to the largest V scale; the sums of n terms n 2^-23; the output's bf16 rounding 2^-8."""
        q = (self.q if q is None else q).double().numpy().reshape(self.M, self.nkv, self.group, D)
        out = np.zeros((self.M, self.nkv, self.group, D))
        tol = np.zeros_like(out)
        c = sm_scale * math.log2(math.e)
        for r in range(self.R):
            for i in range(self.q_len):
                m = r * self.q_len + i
                for h in range(self.nkv):
                    s = self.row_keys(r, i, None if lists is None else lists[m][h])
                    if s.size == 0:
                        continue
                    k, v = self.k[h, s], self.v[h, s]
                    x = q[m, h] @ k.T * c
                    top = x.max(1, keepdims=True)
                    w = np.exp2(x - top)
                    l = w.sum(1, keepdims=True)
                    out[m, h] = w @ v / l
                    ds = 2.0 ** -21 * (np.abs(q[m, h]) @ np.abs(k).T * c + np.abs(x) + np.abs(top) + 16)
                    rel = math.log(2) * ds + 2.0 ** -21 + 2.0 ** -11 + s.size * 2.0 ** -23
                    err = (w * rel) @ np.abs(v) / l
                    err += np.abs(out[m, h]) * ((w * rel).sum(1, keepdims=True) / l)
                    err += s.size * 2.0 ** -34 * max(np.abs(v).max(), 448 * self.vs[h, s].max()) / l
                    tol[m, h] = err * 1.01 + 2.0 ** -8 * (np.abs(out[m, h]) + err) + 1e-30
        return out.reshape(self.M, -1), tol.reshape(self.M, -1)


def select(scores, seq, q_len, W, init, local, topk):
    """scores [H, M, cols] (any float array): lists [M][H] in ascending order."""
    H, M = scores.shape[:2]
    out = []
    for m in range(M):
        n = int(seq[m // q_len])
        p = n - q_len + m % q_len
        nb = 0 if n < max(q_len, 1) or (n + 127) // 128 > W else p // 128 + 1
        rows = []
        for h in range(H):
            pinned = [b for b in range(nb) if b < init or b >= nb - local]
            best = []
            for b in range(nb):
                if b in pinned:
                    continue
                x = scores[h, m, b * 128:(b + 1) * 128]
                x = x[~np.isnan(x)]
                if x.size and x.max() > -np.inf:
                    best.append((-x.max(), b))
            best.sort()
            rows.append(sorted(pinned + [b for _, b in best[:max(0, topk - len(pinned))]]))
        out.append(rows)
    return out


def random_lists(case, topk, seed):
    """blocks [M, nkv, topk], counts [M, nkv] and the lists: random distinct blocks of each row, in random order."""
    g = np.random.default_rng(seed)
    blocks = np.full((case.M, case.nkv, topk), -1, np.int32)
    counts = np.zeros((case.M, case.nkv), np.int32)
    lists = []
    for m in range(case.M):
        p = int(case.seq[m // case.q_len]) - case.q_len + m % case.q_len
        nb = p // 128 + 1 if p >= 0 else 0
        rows = []
        for h in range(case.nkv):
            n = int(g.integers(0, min(topk, nb) + 1)) if m % 3 == 2 else min(topk, nb)
            b = g.permutation(nb)[:n]
            blocks[m, h, :n], counts[m, h] = b, n
            rows.append([int(y) for y in b])
        lists.append(rows)
    return blocks, counts, lists
