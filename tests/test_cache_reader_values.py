"""FP8 attention where the V scales and the weights lie far apart: zero rows
with the scale 1 that the step's writer gives them, rows of large values that
no query looks at, values near the largest that bf16 holds."""

import math

import numpy as np
import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)  # with this sm_scale a score is q . k, a weight 2^(score - largest)


class Scored(ref.Case):
    """A request whose key j has the score q[head][0] * k0[j]: K codes are zeros but for dim 0, all K scales 1."""

    def __init__(self, n, q_len, k0, v_scale, seed, zero=(), group=16):
        super().__init__("fp8", [n], q_len, 1, group, seed=seed)
        g = np.random.default_rng(seed + 1)
        j, d = np.arange(n), np.arange(128)
        slot = self.bt[0, j // 128].astype(np.int64) * 128 + j % 128
        page, t = slot // 128 * self.kps + slot % 128 // 16, slot % 16
        self.k[0, slot] = 0
        self.k[0, slot, 0] = k0
        k = torch.from_numpy(self.k[0, slot]).to(torch.float8_e4m3fn)
        assert (k.double().numpy() == self.k[0, slot]).all()
        self.bytes["k"][page[:, None] * 2048 + d // 16 * 256 + d % 16 + t[:, None] * 16] = k.view(torch.uint8).numpy()
        self.scales["k"][page * 16 + t] = 1.0
        # values as the writer leaves them: the largest of a row is code 448; of one sign, so that nothing cancels
        v = g.random((n, 128)) * 400 + 40
        v[j, g.integers(0, 128, n)] = 448
        v[list(zero)] = 0
        code = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        self.bytes["v"][page[:, None] * 2048 + d * 16 + t[:, None]] = code
        self.scales["v"][page * 16 + t] = v_scale
        self.v[0, slot] = ref.E4M3[code] * np.asarray(v_scale, np.float32).astype(np.float64)[:, None]
        self.amax = np.zeros(self.vs.shape[1])
        self.amax[slot] = np.where(code.any(1), 448.0 * v_scale, 0.0)
        q = np.zeros((self.M, group, 128))
        q[:, :, 0] = g.choice([1.0, 0.9375, 0.875, 1.0625], (self.M, group))
        self.q = ref.bf16(q.reshape(self.M, -1))

    def wanted(self):
        """The 64-bit result and the bound: as ref.Case.attention's, but what f16 loses below its normal range is half
        its smallest step, 2^-25, where the largest weight x V scale of a row that is not all zeros stands at 2^9 or
        more; times a code up to 448."""
        out = np.zeros((self.M, self.group, 128))
        tol = np.zeros_like(out)
        for m in range(self.M):
            s = self.row_keys(0, m)
            q = self.q[m].double().numpy().reshape(self.group, 128)
            k, v = self.k[0, s], self.v[0, s]
            x = q @ k.T
            top = x.max(1, keepdims=True)
            w = np.exp2(x - top)
            l = w.sum(1, keepdims=True)
            out[m] = w @ v / l
            ds = 2.0 ** -21 * (np.abs(q) @ np.abs(k).T + np.abs(x) + np.abs(top) + 16)
            rel = LN2 * ds + 2.0 ** -21 + 2.0 ** -11 + s.size * 2.0 ** -23
            err = (w * rel) @ np.abs(v) / l + np.abs(out[m]) * ((w * rel).sum(1, keepdims=True) / l)
            err += s.size * 2.0 ** -34 * (w * self.amax[s]).max(1, keepdims=True) / l
            tol[m] = err * 1.01 + 2.0 ** -8 * (np.abs(out[m]) + err) + 2.0 ** -133
        return out.reshape(self.M, -1), tol.reshape(self.M, -1)

    def check(self, copies):
        """`copies` requests with the same keys and queries, each against the bound."""
        from indexer_projection_gb300.runner import CacheReader

        self.upload()
        dev = self.dev
        rd = CacheReader(self.group, 1, cache_format=self.format, caches=self.caches, max_requests=copies,
                         q_len=self.q_len, bt_width=self.W, sm_scale=LN2)
        out = torch.full((copies * self.M, self.group * 128), math.nan, dtype=torch.bfloat16, device="cuda")
        rd.attend(dev["q"].repeat(copies, 1), dev["bt"].repeat(copies, 1), dev["seq"].repeat(copies), out)
        assert rd.device_status() == 0
        want, tol = self.wanted()
        got = out.double().cpu().numpy().reshape(copies, *want.shape)
        assert np.isfinite(got).all()
        over = np.abs(got - want) - tol
        assert (over <= 0).all(), (f"max excess {over.max():.3g} where {np.abs(want).max():.3g} is the largest",
                                   np.unravel_index(over.argmax(), over.shape))


# one request on a cluster of SMs; many on even slices of the SMs, several rows too; a CTA a request
SHAPES = [(1, 1, 1100), (1, 2, 700), (200, 1, 4096), (90, 3, 3000), (60, 7, 2500), (2100, 1, 300)]


@pytest.mark.parametrize("copies,q_len,n", SHAPES)
@pytest.mark.parametrize("where", ["first", "middle"])
@pytest.mark.parametrize("live", [-16, -24])
@pytest.mark.parametrize("weight", ["all", "none"])
def test_a_zero_row_of_scale_one(copies, q_len, n, where, live, weight):
    # one V row of zeros with the scale 1, with the largest weight or none; the others' weights 2^-13 of it, or all there is
    at = 0 if where == "first" else n // 2
    k0 = np.zeros(n)
    k0[at] = 13.0 if weight == "all" else -64.0
    vs = np.full(n, 2.0 ** live, np.float32)
    vs[at] = 1.0
    Scored(n, q_len, k0, vs, seed=n, zero=[at]).check(copies)


@pytest.mark.parametrize("copies,q_len,n", SHAPES)
@pytest.mark.parametrize("order", [1, -1])
def test_large_values_that_have_no_weight(copies, q_len, n, order):
    # scores rise (or fall) over 120 powers of two along the keys, the V scales fall (rise) over 30: the keys that
    # count have the small values
    step = np.arange(n) * 15 // n
    k0 = (8.0 * step - 56)[::order]
    vs = (2.0 ** (8.0 - 2 * step)).astype(np.float32)[::order]
    Scored(n, q_len, k0, vs, seed=n + 1).check(copies)


@pytest.mark.parametrize("copies,q_len,n", SHAPES)
def test_large_values_with_little_weight(copies, q_len, n):
    # half the keys at weight 1 with values of 2^-20, half at 2^-22 with values up to 1: both show in the result
    g = np.random.default_rng(n)
    big = g.permutation(n) < n // 2
    Scored(n, q_len, np.where(big, -22.0, 0.0), np.where(big, 2.0 ** -9, 2.0 ** -29).astype(np.float32), seed=n + 2).check(copies)


@pytest.mark.parametrize("copies,q_len,n", SHAPES)
@pytest.mark.parametrize("live", [118, -110])
def test_values_near_the_largest_and_the_smallest(copies, q_len, n, live):
    # values up to 448 * 2^118, a quarter of the largest bf16 (and down to 2^-105): the sums stay in range
    Scored(n, q_len, np.zeros(n), np.full(n, 2.0 ** live, np.float32), seed=n + 3).check(copies)
