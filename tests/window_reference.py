"""The 64-bit reference of the attention within a window and of the blocks' weights, on tests/cache_reference.py."""

import math

import numpy as np
import torch

from tests import cache_reference as ref

D = 128


class Case(ref.Case):
    """A ref.Case whose rows see `window` keys and the first `sinks` (window 0: all)."""

    window, sinks = 0, 0

    def seen(self, r, i):
        """Positions that row i of request r sees by its place alone, as a mask over the request's keys up to it."""
        p = int(self.seq[r]) - self.q_len + i
        j = np.arange(p + 1)
        return np.ones(p + 1, bool) if not self.window else (j > p - self.window) | (j < self.sinks)

    def row_positions(self, r, i, blocks=None):
        n = int(self.seq[r])
        if n < max(self.q_len, 1) or (n + 127) // 128 > self.W:
            return np.zeros(0, np.int64)
        j = np.nonzero(self.seen(r, i))[0]
        if blocks is not None:
            j = j[np.isin(j // 128, [b for b in blocks if 0 <= b])]
        return j[(self.bt[r, j // 128] >= 0) & (self.bt[r, j // 128] < self.pool)]

    def row_keys(self, r, i, blocks=None):
        j = self.row_positions(r, i, blocks)
        return self.bt[r, j // 128].astype(np.int64) * 128 + j % 128

    def poison(self):
        """Everything that no row sees: NaN key and value scales, codes of NaN, table entries outside the cache."""
        for r in range(self.R):
            n = int(self.seq[r])
            if n < self.q_len:
                continue
            any_row = np.zeros(n, bool)
            for i in range(self.q_len):
                m = self.seen(r, i)
                any_row[:m.size] |= m
            j = np.nonzero(~any_row)[0]
            slot = self.bt[r, j // 128].astype(np.int64) * 128 + j % 128
            if self.fmt == "fp8":
                page, t = slot // 128 * self.kps + slot % 128 // 16, slot % 16
                d = np.arange(D)
                for h in range(self.nkv):
                    base = page * self.nkv + h
                    for w in "kv":
                        off = base[:, None] * 2048 + (d // 16 * 256 + d % 16 + t[:, None] * 16 if w == "k" else d * 16 + t[:, None])
                        self.bytes[w][off] = 0x7f
                        self.scales[w][base * 16 + t] = math.nan
            else:
                flat, bs, g = self.kv.reshape(-1), self.bs, np.arange(8)
                page, t = (slot // bs)[:, None], (slot % bs)[:, None]
                for sl in range(2 * self.nkv):
                    base = page * self.page_bytes + sl * bs * 72
                    flat[base + t * 64 + np.arange(64)] = 0xff
                    flat[base + bs * 64 + ((t // 4 * 4 + g // 2) * 8 + g % 2 * 4 + t % 4 if sl % 2 else t * 8 + g)] = 0xff
            whole = np.nonzero(~np.array([any_row[b * 128:(b + 1) * 128].any() for b in range((n + 127) // 128)]))[0]
            self.bt[r, whole] = np.where(whole % 2 == 0, 2 ** 31 - 1, -1)
        return self

    def weights(self, lists=None, q=None, sm_scale=D ** -0.5, before=None, decay=1.0):
        """[R, W] and the bound on the kernel's error, f64.

        The bound: a score is off by ds as in ref.Case.attention; log2 of a block's sum and that of all blocks' round at
        2^-24 of up to |top| + 16 each, and lg2 and ex2 are off by up to 2^-21 in all; a sum of n terms by n 2^-24; with
        the rows' and heads' sum and the decayed weight one more rounding a term, 2^-24 each."""
        q = (self.q if q is None else q).double().numpy().reshape(self.M, self.nkv, self.group, D)
        out, tol = np.zeros((self.R, self.W)), np.zeros((self.R, self.W))
        c = sm_scale * math.log2(math.e)
        for r in range(self.R):
            nb = (int(self.seq[r]) + 127) // 128
            for i in range(self.q_len):
                m = r * self.q_len + i
                for h in range(self.nkv):
                    j = self.row_positions(r, i, None if lists is None else lists[m][h])
                    if j.size == 0:
                        continue
                    k = self.k[h, self.bt[r, j // 128].astype(np.int64) * 128 + j % 128]
                    x = q[m, h] @ k.T * c
                    top = x.max(1, keepdims=True)
                    w = np.exp2(x - top)
                    w /= w.sum(1, keepdims=True)
                    ds = 2.0 ** -21 * (np.abs(q[m, h]) @ np.abs(k).T * c + np.abs(x) + np.abs(top) + 16)
                    rel = math.log(2) * (ds + ds.max(1, keepdims=True) + 2.0 ** -22 * (np.abs(top) + 16)) + 2.0 ** -19
                    rel = rel + j.size * 2.0 ** -23
                    np.add.at(out[r], j // 128, w.sum(0))
                    np.add.at(tol[r], j // 128, (w * rel).sum(0) + 2.0 ** -24 * self.group)
            if before is not None and decay != 0 and nb <= self.W:
                old = decay * before[r, :nb].astype(np.float64)
                out[r, :nb] += old
                tol[r, :nb] += 2.0 ** -23 * np.abs(old)
            tol[r] = tol[r] * 1.01 + 2.0 ** -23 * np.abs(out[r])
        return out, tol


def attend(case, rd, lists=None, q=None, **kw):
    """out [M, heads * 128] and, with weights=True, the weights [R, W]; finite where nothing was written would show."""
    out = torch.full((case.M, case.nkv * case.group * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    if lists is not None:
        kw.update(zip(("blocks", "counts"), (torch.from_numpy(x).cuda() for x in lists)))
    if kw.get("weights") is True:
        kw["weights"] = torch.full((case.R, case.W), 7.0, device="cuda")
    rd.attend(case.dev["q"] if q is None else q, case.dev["bt"], case.dev["seq"], out, window=case.window, sinks=case.sinks, **kw)
    torch.cuda.synchronize()
    return (out, kw["weights"]) if "weights" in kw else out


def close(got, want):
    out, tol = want
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - out) - tol
    assert (over <= 0).all(), f"max excess {over.max():.3g} at {np.unravel_index(over.argmax(), over.shape)}"


def close_weights(got, case, want, untouched=7.0):
    """Rows of requests without keys hold what was there, columns behind a request's last block 0."""
    out, tol = want
    for r in range(case.R):
        n = int(case.seq[r])
        nb = (n + 127) // 128
        row = got[r].double().cpu().numpy()
        if n < max(case.q_len, 1) or nb > case.W:
            assert (row == untouched).all(), r
            continue
        assert (row[nb:] == 0).all() and np.isfinite(row).all(), r
        over = np.abs(row[:nb] - out[r, :nb]) - tol[r, :nb]
        assert (over <= 0).all(), (r, int(over.argmax()), float(over.max()))
