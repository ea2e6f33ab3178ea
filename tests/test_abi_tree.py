"""Refusals of the calls of a step with drafted tokens (tree plan, tree attention, log probabilities, acceptance and cache
move): every invalid argument returns the documented status before any HIP call, so the fake addresses
are never touched.  No GPU needed."""
import ctypes

import pytest

osc = pytest.importorskip("w4a4_outlier_split_amd", reason="libosc.so not built")

A = 0x10000  # 16-byte aligned fake device address
U = 0x10008  # 8-byte aligned
H = 0x10004  # 4-byte aligned
V = 0x10002  # 2-byte aligned
FAR = [(1 << 40) + (i << 34) for i in range(300)]  # operands apart from each other


def call(fn, *args):
    return getattr(osc._lib, fn)(*args)


def plan(PARENT=FAR[0], CU=FAR[1], CTX=FAR[2], R=4, T=16, N=8, POS=FAR[3], MASK=FAR[4]):
    return call("osc_tree_plan", PARENT, CU, CTX, R, T, N, POS, MASK, None)


def test_tree_plan_refusals():
    assert plan(R=-1) == 2 and plan(R=4097) == 2 and plan(T=-1) == 2 and plan(N=0) == 2 and plan(N=257) == 2 and plan(N=-64) == 2
    assert plan(T=1 << 30, N=256) == 2                                  # mask words past 31 bits
    for k in ("PARENT", "CU", "CTX", "POS", "MASK"):
        assert plan(**{k: None}) == 1, k
        assert plan(**{k: V}) == 4, k
    assert plan(MASK=H) == 4                                            # 64-bit words
    assert plan(T=0, PARENT=None, POS=None, MASK=None) == 0
    assert plan(T=0, CU=None) == 1 and plan(R=0, CU=None) == 1          # the offsets are required
    assert plan(POS=FAR[0]) == 2 and plan(MASK=FAR[2] - 8) == 2 and plan(MASK=FAR[3] + 56) == 2


def ws(S=4, R=2, HQ=4, HKV=2, D=128, page=16, MB=4, N=4):
    n = ctypes.c_int64(-1)
    return call("osc_attn_tree_workspace", S, R, HQ, HKV, D, page, MB, N, ctypes.byref(n)), n.value


def attn(Q=FAR[0], KC=FAR[1], VC=FAR[2], S=4, R=2, HQ=4, HKV=2, D=128, page=16, MB=4, NP=8, T=FAR[3], CU=FAR[4], KV=FAR[5], MASK=FAR[6], N=4,
         scale=0.1, O=FAR[7], WS=FAR[8], n=1 << 33):
    return call("osc_attn_tree", Q, KC, VC, S, R, HQ, HKV, D, page, MB, NP, T, CU, KV, MASK, N, scale, O, WS, n, None)


def test_attn_tree_refusals():
    for f in (lambda **k: ws(**k)[0], attn):
        assert f(page=20) == 2 and f(S=-1) == 2 and f(S=1 << 24) == 2 and f(R=-1) == 2 and f(R=4097) == 2 and f(MB=0) == 2
        assert f(HQ=5) == 2 and f(HQ=0) == 2 and f(HKV=0) == 2 and f(D=32) == 2 and f(MB=(1 << 26) + 1) == 2
        assert f(S=(1 << 24) - 1, HQ=16) == 2 and f(N=0) == 2 and f(N=257) == 2
    assert call("osc_attn_tree_workspace", 4, 2, 4, 2, 128, 16, 4, 4, None) == 1
    assert attn(NP=0) == 2 and attn(NP=1 << 27) == 2
    for s in (0.0, -1.0, float("inf"), float("nan"), 3e38):            # the last: over the range times log2 e
        assert attn(scale=s) == 2, s
    for k in ("Q", "KC", "VC", "T", "CU", "KV", "MASK", "O", "WS"):
        assert attn(**{k: None}) == 1, k
    for k in ("Q", "KC", "VC", "O", "WS"):
        assert attn(**{k: U}) == 4, k
    for k in ("T", "CU", "KV"):
        assert attn(**{k: V}) == 4, k
    assert attn(MASK=H) == 4
    assert attn(S=0, Q=None) == 0 and attn(R=0, Q=None) == 0
    need = ws()[1]
    assert ws() == (0, need) and need > 0 and ws(S=0) == (0, 0) and ws(R=0) == (0, 0)
    assert attn(n=need - 1) == 2 and attn(n=-1) == 2
    # operands on an output: its first bytes, its last, and their last bytes on its first
    q, cache = 2 * 4 * 4 * 128, 2 * 8 * 2 * 128 * 16
    size = dict(Q=q, KC=cache, VC=cache, T=4 * 2 * 4, CU=16, KV=16, MASK=32)
    for o, at, n in (("O", FAR[7], q), ("WS", FAR[8], need)):
        for k, b in size.items():
            for d in {0, (n - 1) // 16 * 16, -((b - 1) // 16 * 16)}:
                assert attn(**{k: at + d}) == 2, (o, k, d)
    assert attn(O=FAR[8]) == 2


def lws(S=4, V=1000, K=5):
    n = ctypes.c_int64(-1)
    return call("osc_logprobs_workspace", S, V, K, ctypes.byref(n)), n.value


def lp(X=FAR[0], xt=0, S=4, V=1000, ld=1000, scale=1.0, ID=FAR[1], M=2, K=5, LP=FAR[2], ENT=FAR[3], TOPV=FAR[4], TOPI=FAR[5], WS=FAR[6], n=1 << 33):
    return call("osc_logprobs", X, xt, S, V, ld, scale, ID, M, K, LP, ENT, TOPV, TOPI, WS, n, None)


def test_logprobs_refusals():
    assert lp(xt=2) == 5 and lp(xt=-1) == 5
    for f in (lambda **k: lws(**k)[0], lp):
        assert f(S=-1) == 2 and f(S=1 << 24) == 2 and f(V=0) == 2 and f(K=-1) == 2 and f(K=65) == 2
    assert lws(V=1 << 24)[0] == 2 and lp(V=1 << 24, ld=1 << 24) == 2
    assert lp(ld=999) == 2 and lp(S=1 << 20, ld=1 << 14, V=1 << 14) == 2 and lp(M=-1) == 2 and lp(M=65537) == 2 and lp(S=1 << 16, M=1 << 15) == 2
    for s in (0.0, -1.0, float("inf"), float("nan"), 3e38):
        assert lp(scale=s) == 2, s
    assert call("osc_logprobs_workspace", 4, 1000, 5, None) == 1
    for k in ("X", "ID", "LP", "TOPV", "TOPI"):
        assert lp(**{k: None}) == 1, k
    assert lp(X=U) == 4
    for k in ("ID", "LP", "ENT", "TOPV", "TOPI"):
        assert lp(**{k: V}) == 4, k
    big = dict(S=2, V=100000, K=5)
    need = lws(**big)[1]
    assert need > 0 and lp(**big, ld=100000, WS=None) == 1 and lp(**big, ld=100000, n=need - 1) == 2 and lp(**big, ld=100000, WS=U) == 4
    assert lws(S=0) == (0, 0) and lp(S=0, X=None) == 0
    assert lp(M=0, K=0, ID=None, LP=None, TOPV=None, TOPI=None, ENT=None) == 0  # nothing is asked for
    rows = 2 * (3 * 1000 + 1000)
    for k, b in (("X", rows), ("ID", 32)):
        for o, at, m in (("LP", FAR[2], 32), ("ENT", FAR[3], 16), ("TOPV", FAR[4], 80), ("TOPI", FAR[5], 80)):
            for d in {0, (m - 1) // 16 * 16, -((b - 1) // 16 * 16)}:
                assert lp(**{k: at + d}) == 2, (k, o, d)
    assert lp(**big, ld=100000, X=FAR[6] + (need - 1) // 16 * 16) == 2
    assert lp(ENT=FAR[2] + 28) == 2 and lp(TOPI=FAR[4] + 76) == 2


def accept(TOKEN=FAR[0], PARENT=FAR[1], CHOICE=FAR[2], ldc=3, SLOT=FAR[3], POS=FAR[4], P=9, CU=FAR[5], R=4, T=16, N=8, ACC=FAR[6], PATH=FAR[7],
           NEXT=FAR[8]):
    return call("osc_tree_accept", TOKEN, PARENT, CHOICE, ldc, SLOT, POS, P, CU, R, T, N, ACC, PATH, NEXT, None)


def test_tree_accept_refusals():
    assert accept(R=-1) == 2 and accept(R=4097) == 2 and accept(T=-1) == 2 and accept(N=0) == 2 and accept(N=257) == 2 and accept(P=-1) == 2
    assert accept(ldc=0) == 2 and accept(T=1 << 24, ldc=1024) == 2
    ptrs = ("TOKEN", "PARENT", "CHOICE", "SLOT", "POS", "CU", "ACC", "PATH", "NEXT")
    for k in ptrs:
        assert accept(**{k: None}) == 1, k
        assert accept(**{k: V}) == 4, k
    assert accept(R=0, TOKEN=None, CU=None) == 0
    size = dict(TOKEN=64, PARENT=64, CHOICE=4 * (15 * 3 + 1), SLOT=64, POS=64, CU=20)
    for o, at, m in (("ACC", FAR[6], 16), ("PATH", FAR[7], 128), ("NEXT", FAR[8], 16)):
        for k, b in size.items():
            for d in {0, m - 4, -(b - 4)}:
                assert accept(**{k: at + d}) == 2, (o, k, d)
    assert accept(ACC=FAR[8] + 12) == 2


def commit(KC=None, VC=None, layers=3, NP=8, HKV=2, D=64, page=16, SLOT=FAR[0], CU=FAR[1], ACC=FAR[2], PATH=FAR[3], R=4, T=16, N=8):
    k = [FAR[10 + i] for i in range(max(layers, 0))] if KC is None else KC
    v = [FAR[150 + i] for i in range(max(layers, 0))] if VC is None else VC
    arr = lambda x: None if x == 0 else (ctypes.c_void_p * max(1, len(x)))(*x)
    return call("osc_tree_commit", arr(k), arr(v), layers, NP, HKV, D, page, SLOT, CU, ACC, PATH, R, T, N, None)


def test_tree_commit_refusals():
    assert commit(page=48) == 2 and commit(layers=-1) == 2 and commit(layers=129) == 2 and commit(HKV=0) == 2 and commit(HKV=1025) == 2
    assert commit(D=96) == 2 and commit(NP=0) == 2 and commit(NP=1 << 27) == 2
    assert commit(R=-1) == 2 and commit(R=4097) == 2 and commit(T=-1) == 2 and commit(N=0) == 2 and commit(N=257) == 2
    for k in ("SLOT", "CU", "ACC", "PATH"):
        assert commit(**{k: None}) == 1, k
        assert commit(**{k: V}) == 4, k
    assert commit(KC=0) == 1 and commit(VC=0) == 1
    assert commit(KC=[FAR[10], None, FAR[12]]) == 1 and commit(VC=[FAR[10], FAR[20], U]) == 4
    assert commit(R=0, SLOT=None) == 0 and commit(T=0, SLOT=None) == 0 and commit(layers=0, SLOT=None) == 0
    cache = 2 * 8 * 2 * 64 * 16
    assert commit(KC=[FAR[10], FAR[11], FAR[10]]) == 2 and commit(VC=[FAR[10], FAR[150], FAR[151]]) == 2   # a layer twice
    assert commit(KC=[FAR[10], FAR[10] + cache - 16, FAR[12]]) == 2 and commit(VC=[FAR[12] - cache + 16, FAR[150], FAR[151]]) == 2
    for k, b in (("SLOT", 64), ("CU", 20), ("ACC", 16), ("PATH", 128)):
        for at in (FAR[11], FAR[151]):
            for d in (0, cache - 4, -(b - 4)):
                assert commit(**{k: at + d}) == 2, (k, d)
