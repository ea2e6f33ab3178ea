"""Refusals of the calls between the projections (norm, page plan, cache write, paged attention):
every invalid argument returns the documented status before any HIP call, so the fake addresses
are never touched.  No GPU needed."""
import ctypes

import numpy as np
import pytest

osc = pytest.importorskip("w4a4_outlier_split_amd", reason="libosc.so not built")

A = 0x10000  # 16-byte aligned fake device address
U = 0x10008  # 8-byte aligned
V = 0x10002  # 2-byte aligned


def call(fn, *args):
    return getattr(osc._lib, fn)(*args)


TAB = np.full(1024, -1, np.int32)
LP = TAB.ctypes.data_as(ctypes.c_void_p)


def norm_quant(X=A, RES=A, W=A, S=16, H=256, eps=1e-6, G=32, L=LP, m=1, fmt=0, RO=A, QX=A, SX=A, B=A):
    return call("osc_rmsnorm_quant", X, RES, W, S, H, eps, G, L, m, fmt, RO, QX, SX, B, None)


def test_rmsnorm_quant_refusals():
    assert norm_quant(fmt=7) == 5 and norm_quant(fmt=2) == 5          # unknown; pairs need G = 16
    assert norm_quant(fmt=1) == 5                                      # E4M3 takes no table
    assert norm_quant(G=8) == 2 and norm_quant(H=384) == 2 and norm_quant(H=0) == 2 and norm_quant(S=-1) == 2
    assert norm_quant(H=65536, G=32) == 2                              # over OSC_MAX_GROUPS groups
    assert norm_quant(m=0) == 2 and norm_quant(m=4) == 2
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert norm_quant(eps=eps) == 2, eps
    for k in ("X", "W", "QX", "SX"):
        assert norm_quant(**{k: None}) == 1, k
    assert norm_quant(RES=None) == 1 and norm_quant(RO=None) == 1      # both or neither
    assert norm_quant(B=None) == 1 and norm_quant(L=None) == 1
    for k in ("X", "RES", "W", "RO", "QX", "SX", "B"):
        assert norm_quant(**{k: U}) == 4, k
    bad = np.full(8, 32, np.int32)
    assert norm_quant(L=bad.ctypes.data_as(ctypes.c_void_p)) == 3
    assert norm_quant(S=0, X=None, QX=None) == 0


def norm(X=A, RES=A, W=A, S=16, H=256, eps=1e-6, RO=A, Y=A):
    return call("osc_rmsnorm", X, RES, W, S, H, eps, RO, Y, None)


def test_rmsnorm_refusals():
    assert norm(H=300) == 2 and norm(H=65536 + 256) == 2 and norm(S=-1) == 2 and norm(S=1 << 24) == 2 and norm(eps=0.0) == 2
    assert norm(X=None) == 1 and norm(W=None) == 1 and norm(Y=None) == 1 and norm(RES=None) == 1 and norm(RO=None) == 1
    for k in ("X", "RES", "W", "RO", "Y"):
        assert norm(**{k: U}) == 4, k
    assert norm(S=0, Y=None) == 0


def plan(CTX=A, NEW=A, R=4, page=16, NP=8, FREE=A, F=8, HEAD=A, T=8, TABLE=A, MB=4, CU=A, KV=A, SLOT=A, POS=A, USED=A):
    return call("osc_page_plan", CTX, NEW, R, page, NP, FREE, F, HEAD, T, TABLE, MB, CU, KV, SLOT, POS, USED, None)


def test_page_plan_refusals():
    for p in (0, 8, 24, 512, -16):
        assert plan(page=p) == 2, p
    assert plan(R=-1) == 2 and plan(R=4097) == 2 and plan(F=-1) == 2 and plan(T=-1) == 2 and plan(NP=0) == 2 and plan(MB=0) == 2
    assert plan(NP=1 << 27) == 2 and plan(MB=1 << 27) == 2             # slots past 31 bits
    assert plan(R=4096, MB=1 << 19) == 2                               # table entries past 31 bits
    for k in ("CTX", "NEW", "FREE", "TABLE", "CU", "KV", "SLOT", "POS", "USED"):
        assert plan(**{k: None}) == 1, k
        assert plan(**{k: V}) == 4, k
    assert plan(HEAD=V) == 4
    assert plan(R=0, T=0, F=0, CU=None) == 1 and plan(R=0, USED=None) == 1
    # written while other workgroups read: lengths and the list's head are not updated in place
    B, C = 0x20000, 0x30000
    assert plan(CTX=B, KV=B) == 2 and plan(NEW=B, KV=B) == 2 and plan(KV=B, HEAD=C, USED=C) == 2


def append(QKV=A, S=4, HQ=4, HKV=2, D=128, WQ=A, WK=A, eps=1e-6, CS=A, P=8, POS=A, SLOT=A, Q=A, KC=A, VC=A, NP=8, page=16):
    return call("osc_qkv_append", QKV, S, HQ, HKV, D, WQ, WK, eps, CS, P, POS, SLOT, Q, KC, VC, NP, page, None)


def test_qkv_append_refusals():
    assert append(page=48) == 2 and append(S=-1) == 2 and append(S=1 << 24) == 2 and append(D=96) == 2 and append(HQ=0) == 2
    assert append(HKV=0) == 2 and append(HQ=1025) == 2 and append(HKV=1025) == 2 and append(NP=0) == 2 and append(NP=1 << 27) == 2
    assert append(S=(1 << 24) - 1, HQ=16) == 2                         # 2^34 elements
    assert append(eps=0.0) == 2 and append(eps=float("nan")) == 2 and append(P=0) == 2
    for k in ("QKV", "SLOT", "Q", "KC", "VC", "POS"):
        assert append(**{k: None}) == 1, k
    assert append(WQ=None) == 1 and append(WK=None) == 1
    for k in ("QKV", "WQ", "WK", "CS", "Q", "KC", "VC"):
        assert append(**{k: U}) == 4, k
    assert append(POS=V) == 4 and append(SLOT=V) == 4
    assert append(S=0, QKV=None) == 0
    # without a norm, eps is not looked at; without a rotation, P is not
    assert append(WQ=None, WK=None, eps=0.0, QKV=None) == 1 and append(CS=None, P=0, QKV=None) == 1


def ws(S=4, R=2, HQ=4, HKV=2, D=128, page=16, MB=4):
    n = ctypes.c_int64(-1)
    return call("osc_attn_workspace", S, R, HQ, HKV, D, page, MB, ctypes.byref(n)), n.value


def attn(Q=A, KC=A, VC=A, S=4, R=2, HQ=4, HKV=2, D=128, page=16, MB=4, NP=8, T=A, CU=A, KV=A, scale=0.1, O=A, WS=A, n=1 << 40):
    return call("osc_attn_paged", Q, KC, VC, S, R, HQ, HKV, D, page, MB, NP, T, CU, KV, scale, O, WS, n, None)


def test_attn_refusals():
    for f in (lambda **k: ws(**k)[0], attn):
        assert f(page=20) == 2 and f(S=-1) == 2 and f(S=1 << 24) == 2 and f(R=-1) == 2 and f(R=4097) == 2 and f(MB=0) == 2
        assert f(HQ=5) == 2 and f(HQ=0) == 2 and f(HKV=0) == 2 and f(D=32) == 2 and f(MB=(1 << 26) + 1) == 2
        assert f(S=(1 << 24) - 1, HQ=16) == 2
    assert call("osc_attn_workspace", 4, 2, 4, 2, 128, 16, 4, None) == 1
    assert attn(NP=0) == 2 and attn(NP=1 << 27) == 2
    for s in (0.0, -1.0, float("inf"), float("nan"), 3e38):            # the last: over the range times log2 e
        assert attn(scale=s) == 2, s
    for k in ("Q", "KC", "VC", "T", "CU", "KV", "O"):
        assert attn(**{k: None}) == 1, k
    for k in ("Q", "KC", "VC", "O", "WS"):
        assert attn(**{k: U}) == 4, k
    for k in ("T", "CU", "KV"):
        assert attn(**{k: V}) == 4, k
    assert attn(S=0, Q=None) == 0 and attn(R=0, Q=None) == 0


def test_attn_workspace():
    assert ws(S=0) == (0, 0) and ws(R=0) == (0, 0)
    # none is cut: many tiles, a prompt that fills its table, short requests
    assert ws(S=8192, R=1, HQ=32, HKV=8, page=64, MB=128) == (0, 0) and ws(S=2000, R=1, HQ=32, HKV=8, page=64, MB=32) == (0, 0)
    assert ws(S=9, R=3, D=64) == (0, 0)
    for sizes in (dict(S=1, R=1, HQ=32, HKV=8, page=64, MB=128), dict(S=1024, R=1, HQ=32, HKV=8, page=64, MB=640), dict(S=9, R=3, D=64, MB=640)):
        st, need = ws(**sizes)
        assert st == 0 and 0 < need < 1 << 28  # two tiles for each workgroup, whatever the lengths
        assert attn(**sizes, WS=None) == 1 and attn(**sizes, n=need - 1) == 2 and attn(**sizes, n=-1) == 2


def test_a_short_table_is_refused_by_the_binding():
    with pytest.raises(osc.OscError) as e:
        osc.osc_rmsnorm_quant(A, None, A, 16, 256, 1e-6, 32, [-1] * 7, 1, 0, None, A, A, A, stream=0)
    assert e.value.status == 3
