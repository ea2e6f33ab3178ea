"""Log probabilities, entropy and alternatives against 64 bits, at vocabularies, orders and masks where they can go wrong."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402

INF = float("inf")


def rows_of(kind, S, V, seed):
    """float64 [S, V] that bf16 holds exactly, or nearly."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2.5, (S, V))
    if kind == "equal":
        x[:] = 1.5
    elif kind == "up":
        x = np.sort(x, 1)
    elif kind == "down":
        x = -np.sort(-x, 1)
    elif kind == "levels":
        x = np.round(x * 2) / 2
    elif kind == "zeros":  # both signs of zero are one value
        x = np.where(rng.random((S, V)) < 0.5, 0.0, -0.0)
    elif kind == "negative":
        x = -np.abs(x) - 3
    elif kind == "sure":
        x[np.arange(S), rng.integers(0, V, S)] = 40
    elif kind == "few":  # all but a few are masked out
        x = np.where(rng.random((S, V)) < 3.0 / V, x, -INF)
        x[:, V // 2] = -1.0
    elif kind == "cluster":  # the large ones side by side
        at = rng.integers(0, max(1, V - 300))
        x[:, at:at + 300] += 12
    elif kind == "stripes":  # the large ones all with the same few threads
        x[:, (np.arange(V) // 8) % 256 < 3] += 12
    return x


def run(X, xt, S, V, ld, scale, ids, K, ent=True):
    M = 0 if ids is None else ids.shape[1]
    LP = poisoned((S, M), torch.float32) if M else None
    ENT = poisoned((S,), torch.float32) if ent else None
    TV, TI = (poisoned((S, K), torch.float32), poisoned((S, K), torch.int32)) if K else (None, None)
    n = osc.osc_logprobs_workspace(S, V, K)
    WS = poisoned((n,), torch.uint8) if n else None
    osc.osc_logprobs(X, xt, S, V, ld, scale, ids, M, K, LP, ENT, TV, TI, WS)
    return LP, ENT, TV, TI


def check(x, dt, scale, M, K, pad, seed):
    """x: float64 [S, V]"""
    S, V = x.shape
    ld = V + pad
    bf = dt == torch.bfloat16
    held = torch.from_numpy(x).to(DEV).to(dt)
    buf = torch.full(((S - 1) * ld + V,), 3.0e38, dtype=dt, device=DEV)  # nothing behind the last row, the columns between are large
    for s in range(S):
        buf[s * ld:s * ld + V] = held[s]
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.randint(0, V, (S, M), generator=g, device=DEV).to(torch.int32) if M else None
    if M > 1:
        ids[:, 0], ids[::2, 1], ids[1::2, 1] = V - 1, -1, V
    LP, ENT, TV, TI = run(buf, osc.OSC_Y_BF16 if bf else osc.OSC_Y_F32, S, V, ld, scale, ids, K)
    y = held.double() * scale
    lse = torch.logsumexp(y, 1, keepdim=True)
    # A thread takes n = V / 256 values one behind the other, in chunks of 2048 and more too, and sums are joined over 22 steps at most:
    # each sum is off by n + 22 units of 2^-24, its terms by 4 for exp2 and by 2^-24 of the exponent's size for the product before; scale log2 e
    # is rounded twice, which shifts a log probability by 2^-23 of scale times (its logit less the mean one).  With `size` the largest |scale x|:
    size = y[torch.isfinite(y)].abs().max()
    eps, n = 2.0 ** -24, V / 256 + 22
    tol = eps * (n + 8 + 8 * size)
    assert bool((ENT >= 0).all())
    if M:
        assert bool((LP <= 0).all())
        want = torch.gather(y, 1, ids.clamp(0, V - 1).long()) - lse
        want[(ids < 0) | (ids >= V)] = -INF
        assert torch.equal(torch.isinf(LP), torch.isinf(want))
        f = torch.isfinite(want)
        assert bool(((LP.double() - want).abs() <= tol)[f].all()), float((LP.double() - want)[f].abs().max() / tol)
    # the entropy's two parts carry the sums' errors; around a reference up to 4 off the largest value, each is at most H + 6 (in bits)
    p = y - lse
    H = -(p.exp() * torch.where(torch.isfinite(p), p, 0.0)).sum(1)
    assert bool(((ENT.double() - H).abs() <= tol * (2 * H + 10)).all()), float(((ENT.double() - H).abs() / tol).max())
    if K:
        h = held.float().cpu().numpy()
        for s in range(S):
            order = np.lexsort((np.arange(V), -h[s]))[:K]
            order = order[np.isfinite(h[s][order])]
            k = len(order)
            assert TI[s].tolist() == order.tolist() + [-1] * (K - k), s
            want = y[s][torch.from_numpy(order).to(DEV)] - lse[s]
            assert bool(((TV[s, :k].double() - want).abs() <= tol).all())
            assert bool((TV[s, k:] == -INF).all())


KINDS = ("normal", "equal", "up", "down", "levels", "zeros", "negative", "sure", "few", "cluster", "stripes")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,V,K,pad", [(3, 70001, 64, 3), (40, 32001, 20, 0), (1, 16385, 5, 0), (2, 9000, 64, 1), (5, 400, 64, 7)])
def test_logprobs_orders(kind, dt, S, V, K, pad):
    check(rows_of(kind, S, V, S + V), dt, 1.0, 2, K, pad, V)


@pytest.mark.parametrize("kind", ["up", "equal", "normal", "stripes"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [33000, 100003])
def test_logprobs_rows_in_one_part(kind, dt, V):
    """As many rows as there are workgroups: a row is not cut, and its list runs over where the order is a bad one."""
    x = np.tile(rows_of(kind, 2, V, V), (512, 1))
    x[5] = rows_of("normal", 1, V, 5)[0]
    S = x.shape[0]
    held = torch.from_numpy(x).to(DEV).to(dt)
    _, _, TV, TI = run(held, osc.OSC_Y_BF16 if dt == torch.bfloat16 else osc.OSC_Y_F32, S, V, V, 1.0, None, 64)
    h = held.float().cpu().numpy()
    for s in (0, 1, 5, S - 1):
        assert TI[s].tolist() == np.lexsort((np.arange(V), -h[s]))[:64].tolist(), s
    assert bool((TI[6::2] == TI[0]).all()) and bool((TI[7::2] == TI[1]).all())
    assert torch.equal(TV[16::16], TV[:1].expand(TV[16::16].shape))  # rows that begin at the same place of 16 bytes are summed in the same order


@pytest.mark.parametrize("kind", ["equal", "zeros", "up"])
@pytest.mark.parametrize("dt,V", [(torch.bfloat16, 2047 * 8 + 2), (torch.bfloat16, 2047 * 8 + 9), (torch.float32, 2047 * 4 + 2), (torch.float32, 2047 * 4 + 5)])
def test_logprobs_most_that_a_part_holds(kind, dt, V):
    """rows that begin and end inside a vector, of 2047 whole ones: the most that are chosen from at once"""
    check(rows_of(kind, 260, V, V), dt, 1.0, 2, 64, 1, V)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 2047, 2048, 2049, 4096, 4097, 16384, 16400])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_logprobs_vocabularies(V, dt):
    for S, K, M, pad, scale in ((1, 1, 1, 0, 1.0), (7, 64, 3, 1, 0.7), (3, 0, 2, 5, 3.0), (4, 20, 0, 8, 1.25)):
        check(rows_of("normal", S, V, V + S), dt, scale, M, K, pad, V)


@pytest.mark.parametrize("S,V", [(1, 151936), (300, 151936), (1025, 3001), (5000, 130)])
def test_logprobs_rows(S, V):
    check(rows_of("normal", min(S, 37), V, S)[np.arange(S) % min(S, 37)], torch.bfloat16, 1.0, 1, 8, 0, S)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,V", [(6, 60000), (6, 300)])
def test_logprobs_rows_without_a_distribution(dt, S, V):
    """A NaN, +inf, or -inf alone: NaN and -1 there, and the other rows as they are."""
    x = rows_of("normal", S, V, 4)
    good = torch.from_numpy(x).to(DEV).to(dt)
    bad = good.clone()
    bad[0, V - 1], bad[2, 17], bad[3, :] = float("nan"), INF, -INF
    bad[5, :], bad[5, 3] = -INF, float("nan")
    xt = osc.OSC_Y_BF16 if dt == torch.bfloat16 else osc.OSC_Y_F32
    ids = torch.tensor([[3, -1, V]] * S, dtype=torch.int32, device=DEV)
    a, b = run(good, xt, S, V, V, 1.0, ids, 6), run(bad, xt, S, V, V, 1.0, ids, 6)
    for r in (0, 2, 3, 5):
        assert bool(torch.isnan(b[0][r]).all()) and bool(torch.isnan(b[1][r])) and bool(torch.isnan(b[2][r]).all()) and bool((b[3][r] == -1).all())
    for r in (1, 4):
        for p, q in zip(a, b):
            assert torch.equal(p[r], q[r])


def test_logprobs_parts_that_are_not_asked_for():
    x = torch.from_numpy(rows_of("normal", 5, 9001, 1)).to(DEV).bfloat16()
    ids = torch.zeros((5, 2), dtype=torch.int32, device=DEV)
    every = run(x, osc.OSC_Y_BF16, 5, 9001, 9001, 1.0, ids, 7)
    assert torch.equal(run(x, osc.OSC_Y_BF16, 5, 9001, 9001, 1.0, ids, 0, ent=False)[0], every[0])
    only = run(x, osc.OSC_Y_BF16, 5, 9001, 9001, 1.0, None, 7, ent=False)
    assert torch.equal(only[2], every[2]) and torch.equal(only[3], every[3])
    assert torch.equal(run(x, osc.OSC_Y_BF16, 5, 9001, 9001, 1.0, None, 0)[1], every[1])


def test_logprobs_binding_refuses():
    x = torch.zeros((3, 100), dtype=torch.bfloat16, device=DEV)
    ids, lp, ent = torch.zeros((3, 1), dtype=torch.int32, device=DEV), torch.zeros((3, 1), device=DEV), torch.zeros(3, device=DEV)
    f = lambda x=x, xt=osc.OSC_Y_BF16, S=3, ids=ids, lp=lp, ent=ent: osc.osc_logprobs(x, xt, S, 100, 100, 1.0, ids, 1, 0, lp, ent, None, None, None)
    f()
    for bad, status in ((dict(xt=osc.OSC_Y_F32), 5), (dict(x=x.float()), 5), (dict(ids=ids.long()), 5), (dict(lp=lp.double()), 5), (dict(ent=ent.half()), 5),
                        (dict(x=x[:2]), 2), (dict(x=x.t().contiguous().t()), 2), (dict(ent=ent[:2]), 2), (dict(ids=ids.cpu()), 2), (dict(xt=7), 5)):
        with pytest.raises(osc.OscError) as e:
            f(**bad)
        assert e.value.status == status, bad
    big = torch.zeros((2, 50000), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(osc.OscError) as e:  # cut rows need a workspace
        osc.osc_logprobs(big, osc.OSC_Y_BF16, 2, 50000, 50000, 1.0, None, 0, 0, None, ent, None, None, None)
    assert e.value.status == 1


def test_logprobs_replayed():
    """Captured once, replayed on other inputs, with eager work between."""
    S, V, K = 9, 40001, 10
    x = torch.zeros((S, V), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((S, 2), dtype=torch.int32, device=DEV)
    out = [torch.zeros((S, 2), device=DEV), torch.zeros(S, device=DEV), torch.zeros((S, K), device=DEV), torch.zeros((S, K), dtype=torch.int32, device=DEV)]
    ws = torch.empty((osc.osc_logprobs_workspace(S, V, K),), dtype=torch.uint8, device=DEV)
    call = lambda: osc.osc_logprobs(x, osc.OSC_Y_BF16, S, V, V, 0.8, ids, 2, K, *out, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for it in range(4):
        x.copy_(torch.from_numpy(rows_of(KINDS[it], S, V, it)))
        ids.random_(0, V)
        want = run(x, osc.OSC_Y_BF16, S, V, V, 0.8, ids, K)
        for t in out:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_logprobs_behind_32_bits():
    """More than 2^32 bytes of logits: rows at both ends against 64 bits, all of them against rows with the same logits."""
    V, S = 151936, 15000
    few = torch.from_numpy(rows_of("normal", 8, V, 3)).to(DEV).bfloat16()
    x = torch.empty((S, V), dtype=torch.bfloat16, device=DEV)
    for s in range(0, S, 8):
        x[s:s + 8] = few[:min(8, S - s)]
    ids = torch.full((S, 1), V - 1, dtype=torch.int32, device=DEV)
    LP, ENT, TV, TI = run(x, osc.OSC_Y_BF16, S, V, V, 1.0, ids, 3)
    want = torch.log_softmax(few.double(), 1)
    size = float(few.double().abs().max())
    tol = 2.0 ** -24 * (V / 256 + 22 + 8 + 8 * size)
    assert bool(((LP[:8, 0].double() - want[:, -1]).abs() <= tol).all())
    for t in (LP, ENT, TV, TI):
        for s in range(8):
            assert bool((t[s::8] == t[s]).all())


@pytest.mark.parametrize("S", [3, 300])
def test_logprobs_on_another_stream(S):
    V, K = 30001, 9
    x = torch.from_numpy(rows_of("normal", S, V, 3)).to(DEV).bfloat16()
    ids = torch.zeros((S, 1), dtype=torch.int32, device=DEV)
    want = run(x, osc.OSC_Y_BF16, S, V, V, 1.0, ids, K)
    out = [torch.zeros_like(t) for t in want]
    ws = torch.zeros((max(osc.osc_logprobs_workspace(S, V, K), 16),), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    osc.osc_logprobs(x, osc.OSC_Y_BF16, S, V, V, 1.0, ids, 1, K, *out, ws.data_ptr(), stream=side)
    side.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("S,V,M", [(2, 30001, 700), (257, 900, 257), (3, 200, 1000)])
def test_logprobs_many_given_tokens(S, V, M):
    """more given tokens than a workgroup has threads"""
    check(rows_of("normal", S, V, M), torch.bfloat16, 1.0, M, 4, 3, M)


def test_logprobs_most_rows():
    """2^24 - 1 rows of one token: its log probability is 0 but for roundings, whatever the logit, and no workspace is needed"""
    S = 2 ** 24 - 1
    x = torch.arange(S, dtype=torch.int32, device=DEV).remainder_(251).float()
    assert osc.osc_logprobs_workspace(S, 1, 1) == 0
    x[S - 2] = -INF
    ids = torch.zeros((S, 1), dtype=torch.int32, device=DEV)
    ids[S - 1] = 1
    LP, ENT, TV, TI = run(x, osc.OSC_Y_F32, S, 1, 1, 1.0, ids, 1)
    assert bool(torch.isnan(LP[S - 2]).all()) and float(LP[S - 1]) == -INF and int(TI[S - 2]) == -1
    keep = torch.ones(S, dtype=torch.bool, device=DEV)
    keep[S - 2] = False
    tol = 2.0 ** -24 * (1 + 22 + 8 + 8 * 250)  # as in check()
    assert bool((TI[keep] == 0).all())
    for t, most in ((TV[keep], tol), (LP[:S - 2], tol), (ENT[keep], 10 * tol)):
        assert bool((t.abs() <= most).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,V", [(6, 4001), (300, 30001), (5, 300)])
@pytest.mark.parametrize("scale", [1e-37, 1e-39, 1e-45])
def test_logprobs_without_a_distribution_at_the_smallest_scales(dt, S, V, scale):
    """+inf behind a thread's first values, where no finite logit moves the reference any more: NaN and -1, as at any scale."""
    x = rows_of("normal", S, V, 4)
    good = torch.from_numpy(x).to(DEV).to(dt)
    bad = good.clone()
    bad[0, V - 1], bad[2, V - 500 if V > 500 else 17], bad[3, V // 2] = INF, INF, float("nan")
    xt = osc.OSC_Y_BF16 if dt == torch.bfloat16 else osc.OSC_Y_F32
    ids = torch.tensor([[3, -1, V]] * S, dtype=torch.int32, device=DEV)
    a, b = run(good, xt, S, V, V, scale, ids, 6), run(bad, xt, S, V, V, scale, ids, 6)
    for r in (0, 2, 3):
        assert bool(torch.isnan(b[0][r]).all()) and bool(torch.isnan(b[1][r])) and bool(torch.isnan(b[2][r]).all()) and bool((b[3][r] == -1).all()), r
    for r in (1, 4):
        for p, q in zip(a, b):
            assert torch.equal(p[r], q[r])
    # every token is as likely as any: sums and logarithm as in check(), the largest |scale x| below 2^-90
    tol = 2.0 ** -24 * (V / 256 + 22 + 8 + 4 * np.log(V))
    assert bool(((a[0][:, 0].double() + np.log(V)).abs() <= tol).all()) and bool(((a[1].double() - np.log(V)).abs() <= 2 * tol * np.log(V)).all())
