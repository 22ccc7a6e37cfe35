"""pre_attn_verify_drafts against its definition in exact integers; its refusals without a GPU."""

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


def units(p, bits=62):
    """Probabilities in whole units of 2^-bits (what is below is dropped), as uint64."""
    p = np.nan_to_num(np.asarray(p, np.float64), nan=0.0)
    return np.floor(np.clip(p, 0.0, 1.0) * 2.0 ** bits).astype(np.uint64)  # exact: a power of two times 24 bits


def expected(target, q, drafts, u, V, bits=62):
    """One request: target [q_len, V], q [q_len - 1, V] or None, as f64 arrays, in units of 2^-bits: (tokens, accepted, status)."""
    k, status = len(drafts), 0
    n = next((i for i, x in enumerate(drafts) if x < 0), k)
    if any(x >= V for x in drafts[:n]):
        status |= 8
    a = 0
    while a < n and drafts[a] < V:
        x = drafts[a]
        if not float(u[a]) * (float(q[a][x]) if q is not None else 1.0) < float(target[a][x]):
            break
        a += 1
    w = units(target[a], bits)
    if a < n:
        if q is not None:
            d = units(q[a], bits)
            w = np.where(w > d, w - d, np.uint64(0))
        elif drafts[a] < V:
            w = w.copy()
            w[drafts[a]] = 0
        if not w.any():
            w = units(target[a], bits)
    total = int(w.sum(dtype=np.uint64))
    if total == 0:
        return list(drafts[:a]) + [-1] * (k + 1 - a), a, status | 16
    f = float(u[k])
    frac = 2 ** 64 - 1 if f >= 1 else 0 if not f > 0 else int(f * 2.0 ** 64)
    token = int(np.searchsorted(np.cumsum(w, dtype=np.uint64), np.uint64(frac * total >> 64), side="right"))
    return list(drafts[:a]) + [token] + [-1] * (k - a), a, status


def check(target, q, drafts, u, V, verifier=None, stride=None, status=None):
    """target [R, q_len, V] and q [R, q_len - 1, V] torch CPU tensors of their types (q: or None)."""
    from indexer_projection_gb300.runner import DraftVerifier

    R, n = target.shape[:2]
    ver = verifier or DraftVerifier(V, n)

    def rows(x, extra):
        wide = torch.full((x.shape[0] * x.shape[1], V + extra), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, :V] = x.reshape(-1, V).cuda()
        return wide
    t = rows(target, stride or 0)
    d = rows(q, 2 * (stride or 0)) if q is not None else None
    tokens = torch.full((R, n), -7, dtype=torch.int32, device="cuda")
    accepted = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    drafts = np.asarray(drafts, np.int32).reshape(R, n - 1)
    u = np.asarray(u, np.float32).reshape(R, n)
    ver.verify(t, torch.from_numpy(drafts).cuda(), torch.from_numpy(u).cuda(), tokens, accepted, draft_probs=d)
    torch.cuda.synchronize()
    got, acc, st = tokens.tolist(), accepted.tolist(), ver.device_status()
    want_st = 0
    bits = 46 if target.dtype is torch.bfloat16 and (q is None or q.dtype is torch.bfloat16) else 62
    for r in range(R):
        tok, a, s = expected(target[r].double().numpy(), q[r].double().numpy() if q is not None else None,
                             drafts[r].tolist(), u[r], V, bits)
        assert (got[r], acc[r]) == (tok, a), r
        want_st |= s
    assert st == want_st and (status is None or st == status)
    return acc


def case(R, n, V, seed, agree=0.6, dtype=(torch.float32, torch.float32), sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    target = torch.softmax(torch.randn(R, n, V, generator=g) * sharp, -1)
    q = target[:, :n - 1] * agree + (1 - agree) * torch.softmax(torch.randn(R, n - 1, V, generator=g) * sharp, -1)
    target, q = target.to(dtype[0]), q.to(dtype[1])
    x = torch.multinomial(q.float().reshape(-1, V), 1, generator=g).view(R, n - 1) if n > 1 else torch.zeros(R, 0)
    return target, q, x.int().numpy(), torch.rand(R, n, generator=g).numpy()


F, H = torch.float32, torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("n,V,stride,dtype", [(1, 1, 0, (F, F)), (2, 1, 1, (F, F)), (2, 2, 0, (H, H)), (3, 31, 0, (F, H)), (4, 32, 3, (H, F)),
                                              (5, 33, 0, (F, F)), (7, 63, 1, (H, H)), (8, 64, 0, (F, F)), (16, 65, 5, (F, H)), (2, 500, 0, (H, F)),
                                              (3, 1000, 0, (F, F)), (4, 4097, 0, (H, H)), (7, 20011, 0, (F, F)), (3, 20480, 8, (H, H)),
                                              (2, 65537, 0, (F, F)), (1, 65536, 0, (H, H))])
@pytest.mark.parametrize("certain", [False, True])
def test_every_size(n, V, stride, dtype, certain):
    target, q, x, u = case(40 if V < 5000 else 9, n, V, V + n, dtype=dtype)
    acc = check(target, None if certain else q, x, u, V, stride=stride)
    if n > 2 and V > 8 and not certain:
        assert len(set(acc)) > 1


@pytest.mark.gpu
def test_one_request_and_many():
    for R in (1, 2, 333):
        check(*case(R, 5, 777, R), 777)


@pytest.mark.gpu
@pytest.mark.parametrize("R,V", [(3, 12345), (20, 12345), (60, 12345), (100, 20000), (152, 2100), (153, 20000), (200, 30000)])
def test_every_split_of_a_vocabulary(R, V):
    check(*case(R, 2, V, R + V), V)  # (CTAs a request: 8 and fewer)


@pytest.mark.gpu
def test_as_many_requests_as_there_can_be():
    from indexer_projection_gb300.runner import DraftVerifier

    R, few, n, V = 65535, 257, 3, 40
    target, q, x, u = (torch.as_tensor(y) for y in case(few, n, V, 71))
    of = torch.arange(R) % few
    dev = [y[of].contiguous().cuda() for y in (target, x, u, q)]
    ver = DraftVerifier(V, n)
    tokens, accepted = torch.full((R, n), -7, dtype=torch.int32, device="cuda"), torch.full((R,), -7, dtype=torch.int32, device="cuda")
    ver.verify(dev[0].view(-1, V), dev[1], dev[2], tokens, accepted, draft_probs=dev[3].view(-1, V))
    assert ver.device_status() == 0
    want = [expected(target[r].double().numpy(), q[r].double().numpy(), x[r].tolist(), u[r].numpy(), V) for r in range(few)]
    assert torch.equal(tokens.cpu(), torch.tensor([y[0] for y in want], dtype=torch.int32)[of])
    assert torch.equal(accepted.cpu(), torch.tensor([y[1] for y in want], dtype=torch.int32)[of])


@pytest.mark.gpu
@pytest.mark.parametrize("certain", [False, True])
def test_uniforms_at_their_ends(certain):
    target, q, x, u = case(12, 3, 300, 5)
    u[:, 0] = 0.0  # accepted
    u[:, 2] = [0.0, 1e-30, 2.0 ** -40, 1 - 2.0 ** -24, 1.0, 7.0, np.inf, -0.5, np.nan, 0.5, 2.0 ** -24, 0.25]
    check(target, None if certain else q, x, u, 300)
    u[:, 1] = 0.0
    check(target, None if certain else q, x, u, 300)
    u[:, 1] = np.nan  # never accepted
    assert set(check(target, None if certain else q, x, u, 300)) == {1}


@pytest.mark.gpu
@pytest.mark.parametrize("certain", [False, True])
def test_drafts_that_end_early_or_lie_outside_the_vocabulary(certain):
    target, q, x, u = case(8, 5, 130, 6, agree=0.95)
    u[:, :4] *= 0.2
    x[0, 2], x[1, 0], x[2, 3], x[3, 1:] = -1, -5, -2 ** 31, -1
    check(target, None if certain else q, x, u, 130, status=0)
    x[4, 1], x[5, 0], x[6, 2] = 130, 2 ** 31 - 1, 1000
    x[7, 1], x[7, 2] = -1, 5000  # behind the end: not looked at
    check(target, None if certain else q, x, u, 130, status=8)


@pytest.mark.gpu
def test_rows_that_leave_nothing():
    V = 100
    target, q, x, u = case(6, 3, V, 7)
    q[0, 0] = 1.0                      # nothing above the drafter's: drawn from the target's own
    u[0, 0] = 0.99
    target[1] = 0.0                    # no probability at all
    target[2, 0], u[2, 0] = 0.0, 0.0   # the draft has none: 0 < 0 is false; then nothing to draw
    target[3, 0] = float("nan")
    u[4, 0], q[4, 0], x[4, 0] = 0.5, 0.0, 3    # q of zero: accepted where p is above zero
    check(target, q, x, u, V, status=16)
    one = torch.zeros(1, 2, V)
    one[0, 0, 9], one[0, 1, 4] = 1.0, 1.0  # a target that is certain
    check(one, None, [[9]], [[0.999, 0.7]], V, status=0)
    check(one, None, [[8]], [[0.0, 0.7]], V, status=0)
    one[0, 0, 9] = 0.25                # the drafted token alone has probability and is rejected
    check(one, None, [[9]], [[0.3, 0.7]], V, status=0)


@pytest.mark.gpu
def test_values_that_are_no_probabilities():
    V = 90
    g = torch.Generator().manual_seed(3)
    target = torch.rand(20, 3, V, generator=g) / V
    bad = torch.tensor([float("nan"), -0.25, float("-inf"), -0.0, 1e-45, 2.0 ** -63, 2.0 ** -62, 2.0 ** -38])
    at = torch.rand(target.shape, generator=g) < 0.5
    target = torch.where(at, bad[torch.randint(0, len(bad), target.shape, generator=g)], target)
    q = torch.where(torch.rand(20, 2, V, generator=g) < 0.3, float("nan"), torch.rand(20, 2, V, generator=g) / V)
    x = torch.randint(0, V, (20, 2), generator=g).int().numpy()
    check(target, q, x, torch.rand(20, 3, generator=g).numpy(), V)
    target[0, 0, 5] = float("inf")   # counts as 1
    check(target, q, x, torch.rand(20, 3, generator=g).numpy(), V)
    check(target.bfloat16(), q.bfloat16(), x, torch.rand(20, 3, generator=g).numpy(), V)
    tiny = torch.exp2(-60 * torch.rand(20, 3, V, generator=g))  # over all of the units
    check(tiny / V, tiny[:, :2] / V * 0.9, x, torch.rand(20, 3, generator=g).numpy(), V)
    check((tiny / V).bfloat16(), (tiny[:, :2] / V * 0.9).bfloat16(), x, torch.rand(20, 3, generator=g).numpy(), V)


@pytest.mark.gpu
def test_rows_of_whatever_values_stay_in_range():
    # sums of 4 and more: any token or none, inside the vocabulary
    from indexer_projection_gb300.runner import DraftVerifier

    V, R, n = 1000, 50, 3
    ver = DraftVerifier(V, n)
    target = torch.rand(R * n, V, device="cuda") * 3
    tokens, accepted = torch.zeros(R, n, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    drafts = torch.randint(0, V, (R, n - 1), device="cuda", dtype=torch.int32)
    ver.verify(target, drafts, torch.rand(R, n, device="cuda"), tokens, accepted)
    assert ((tokens >= -1) & (tokens < V)).all() and ((accepted >= 0) & (accepted < n)).all()


@pytest.mark.gpu
def test_the_distribution_of_accepted_and_drawn_tokens():
    # many requests with the same rows: the first token's frequencies are the target's.  Each of 6 counts is binomial;
    # the chance that one of them is off by 6 standard deviations is below 2e-8
    V, R = 6, 40000
    p = torch.tensor([0.05, 0.3, 0.2, 0.15, 0.2, 0.1])
    q = torch.tensor([0.3, 0.1, 0.05, 0.35, 0.15, 0.05])
    from indexer_projection_gb300.runner import DraftVerifier

    g = torch.Generator(device="cuda").manual_seed(0)
    target, draft = p.cuda().expand(R * 2, V).contiguous(), q.cuda().expand(R, V).contiguous()
    x = torch.multinomial(draft, 1, generator=g).int()
    u = torch.rand(R, 2, generator=g, device="cuda")
    tokens, accepted = torch.zeros(R, 2, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    DraftVerifier(V, 2).verify(target, x, u, tokens, accepted, draft_probs=draft)
    freq = torch.bincount(tokens[:, 0].long(), minlength=V).cpu().double()
    p = p.double()
    assert ((freq - R * p).abs() <= 6 * (R * p * (1 - p)).sqrt()).all()
    rate = float(accepted.double().mean())
    want = float(torch.minimum(p, q.double()).sum())
    assert abs(rate - want) <= 6 * (want * (1 - want) / R) ** 0.5


@pytest.mark.gpu
def test_captured_and_on_two_streams():
    from indexer_projection_gb300.runner import DraftVerifier

    V, R, n = 5000, 6, 4
    cases = [case(R, n, V, s) for s in (1, 2)]
    vers = [DraftVerifier(V, n) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [(t.cuda().view(-1, V), torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(), torch.zeros(R, n, dtype=torch.int32, device="cuda"),
            torch.zeros(R, dtype=torch.int32, device="cuda"), q.cuda().view(-1, V)) for t, q, x, u in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for ver, s, d in zip(vers, streams, dev):
            with torch.cuda.stream(s):
                ver.verify(*d[:5], draft_probs=d[5])
    torch.cuda.synchronize()
    want = [[expected(t[r].double().numpy(), q[r].double().numpy(), x[r].tolist(), u[r], V) for r in range(R)] for t, q, x, u in cases]
    for d, w in zip(dev, want):
        assert d[3].tolist() == [y[0] for y in w] and d[4].tolist() == [y[1] for y in w]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        vers[0].verify(*dev[0][:5], draft_probs=dev[0][5])
    for _ in range(3):
        dev[0][3].fill_(9), dev[0][4].fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert dev[0][3].tolist() == [y[0] for y in want[0]]
    assert all(v.device_status() == 0 for v in vers)


@pytest.mark.gpu
def test_rows_past_32_bits():
    # a row of the target's that begins past 2^32 bytes
    from indexer_projection_gb300.runner import DraftVerifier

    V, R, n, stride = 1000, 300, 4, 1 << 20
    target, q, x, u = case(R, n, V, 11)
    big = torch.zeros(R * n, stride, device="cuda")[:, :V]
    big.copy_(target.view(-1, V))
    tokens, accepted = torch.zeros(R, n, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    DraftVerifier(V, n).verify(big, torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(), tokens, accepted, draft_probs=q.cuda().view(-1, V))
    for r in (0, 1, R // 2, R - 1):
        want = expected(target[r].double().numpy(), q[r].double().numpy(), x[r].tolist(), u[r], V)
        assert tokens[r].tolist() == want[0] and int(accepted[r]) == want[1]


@pytest.mark.gpu
def test_what_the_verifier_refuses():
    from indexer_projection_gb300 import binding as B
    from indexer_projection_gb300.runner import DraftVerifier

    V, R, n = 64, 2, 3
    ver = DraftVerifier(V, n)
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    a = dict(target=z(R * n, V), drafts=z(R, n - 1, dtype=torch.int32), uniforms=z(R, n), tokens=z(R, n, dtype=torch.int32),
             accepted=z(R, dtype=torch.int32), draft_probs=z(R * (n - 1), V))
    for bad in (dict(target=a["target"].cpu()), dict(target=a["target"].half()), dict(target=a["target"][1:]),
                dict(target=a["target"][:, 1:]), dict(target=z(V, R * n).t()), dict(draft_probs=a["target"]),
                dict(draft_probs=a["draft_probs"].double()), dict(drafts=a["drafts"].long()), dict(drafts=a["tokens"]),
                dict(uniforms=a["uniforms"].double()), dict(uniforms=a["uniforms"][:, 1:]), dict(tokens=a["drafts"]),
                dict(tokens=a["tokens"].cpu()), dict(accepted=a["accepted"].long()), dict(accepted=a["tokens"])):
        with pytest.raises(ValueError):
            ver.verify(**dict(a, **bad))
    with pytest.raises(B.PreAttnError):
        ver.verify(**dict(a, accepted=a["tokens"].view(-1)[:R]))
    for bad in ((0, 3), (2 ** 24 + 1, 3), (64, 0), (64, 17)):
        with pytest.raises(ValueError):
            DraftVerifier(*bad)
    none = dict(target=z(0, V), drafts=z(0, n - 1, dtype=torch.int32), uniforms=z(0, n), tokens=z(0, n, dtype=torch.int32),
                accepted=z(0, dtype=torch.int32))
    assert ver.verify(**none) == 0 and ver.device_status() == 0


def args(B, **kw):
    at = iter(range(P, P + (1 << 30), 1 << 24))
    d = dict(target=next(at), target_stride=100, target_type=0, draft_probs=next(at), draft_stride=100, draft_type=1, drafts=next(at),
             uniforms=next(at), R=2, q_len=3, vocab=100, tokens=next(at), accepted=next(at), status=next(at))
    d.update(kw)
    return B.pa_verify_args(**d)


@pytest.mark.parametrize("kw,err", [
    *[({p: None}, "NULL") for p in ("target", "drafts", "uniforms", "tokens", "accepted", "status")],
    *[({p: P + 2}, "ALIGN") for p in ("target", "drafts", "uniforms", "tokens", "accepted", "status")],
    ({"draft_probs": P + 1}, "ALIGN"), *[({"R": v}, "SHAPE") for v in (-1, 65536)], *[({"q_len": v}, "SHAPE") for v in (0, 17)],
    *[({"vocab": v}, "SHAPE") for v in (0, 101, 2 ** 24 + 1)], ({"target_stride": 99}, "SHAPE"), ({"draft_stride": 99}, "SHAPE"),
    ({"target_type": 2}, "CONFIG"), ({"target_type": -1}, "CONFIG"), ({"draft_type": 2}, "CONFIG"), ({"tokens": P + 400}, "ALIAS"),
    ({"accepted": P + (1 << 24) + 4}, "ALIAS"), ({"tokens": P + (2 << 24)}, "ALIAS"), ({"accepted": P + (4 << 24) + 20}, "ALIAS")])
def test_refusals(B, kw, err):
    assert B.pre_attn_verify_drafts(args(B, **kw), check=False) == getattr(B, "PA_ERR_" + err)


def test_no_requests_is_accepted(B):
    assert B.pre_attn_verify_drafts(args(B, R=0), check=False) == B.PA_OK
    assert B.pre_attn_verify_drafts(args(B, R=0, q_len=1, drafts=None, draft_probs=None), check=False) == B.PA_OK
