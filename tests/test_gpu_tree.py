"""Token trees: positions and masks, the accepted path, and the move of its keys and values, against plain implementations
that take one node after the other."""
import numpy as np
import pytest
import torch

import tree_ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402

KINDS = ("chain", "star", "roots", "near", "wild")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def offsets(parents, gap=0):
    return np.concatenate([[gap], gap + np.cumsum([len(p) for p in parents])]).astype(int).tolist()


def words(mask, W):
    return [[m >> 64 * w & (2 ** 64 - 1) for w in range(W)] for m in mask]


def check_plan(parents, ctx, T, N, gap=0):
    R, W = len(parents), -(-N // 64)
    rows = [0] * gap + [p for q in parents for p in q]
    rows = (rows + [5] * max(0, T - len(rows)))[:T]
    pos, mask = poisoned((T + 2,), torch.int32), poisoned((T + 2, W), torch.int64)
    osc.osc_tree_plan(i32(rows), i32(offsets(parents, gap)), i32(ctx), R, T, N, pos, mask)
    want_pos, want_mask = tree_ref.plan(parents, ctx, T, N, gap)
    assert pos[:T].tolist() == want_pos
    got = [[w & (2 ** 64 - 1) for w in row] for row in mask[:T].tolist()]
    assert got == words(want_mask, W)
    assert bool((pos[T:] == -1).all()) and bool((mask[T:] == -1).all())  # behind the rows: as it was


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 128, 130, 192, 200, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_tree_plan(N, kind):
    rng = np.random.default_rng(N + len(kind))
    parents = [tree_ref.tree(rng, n, kind) for n in (N, 0, 1, N // 2, N, N + 3)]
    ctx = [0, 5, 1000, 2 ** 31 - 2, -7, 4]
    total = sum(map(len, parents))
    check_plan(parents, ctx, total + 300, N)
    check_plan(parents, ctx, total, N, gap=0)
    check_plan(parents, ctx, total + 9, N, gap=4)
    check_plan(parents, ctx, max(1, total - 2 * N // 3), N)  # the last tokens have no row


def test_tree_plan_many_requests():
    rng = np.random.default_rng(3)
    parents = [tree_ref.tree(rng, int(rng.integers(0, 9)), KINDS[int(rng.integers(0, 5))]) for _ in range(4096)]
    check_plan(parents, rng.integers(0, 9000, 4096).tolist(), sum(map(len, parents)) + 40000, 8)
    check_plan([], [], 70, 8)
    check_plan([[]] * 5, [1] * 5, 0, 8)


def run_accept(parents, token, choice, slot, pos, P, N, T, ldc=1, gap=0):
    R = len(parents)
    rows = [0] * gap + [p for q in parents for p in q]
    rows = (rows + [0] * max(0, T - len(rows)))[:T]
    acc, path, after = poisoned((R + 1,), torch.int32), poisoned((R + 1, N), torch.int32), poisoned((R + 1,), torch.int32)
    wide = torch.full((max(T, 1), ldc), 77, dtype=torch.int32, device=DEV)
    wide[:T, 0] = i32(choice[:T])
    osc.osc_tree_accept(i32(token[:T]), i32(rows), wide, ldc, i32(slot[:T]), None if pos is None else i32(pos[:T]), P, i32(offsets(parents, gap)), R, T, N, acc,
                        path, after)
    assert acc[R] == -1 and after[R] == -1 and bool((path[R] == -1).all())
    return acc[:R], path[:R], after[:R]


def check_accept(seed, sizes, N, kind, alphabet, P, ldc, cut=0, gap=0):
    rng = np.random.default_rng(seed)
    parents = [tree_ref.tree(rng, n, kind) for n in sizes]
    total = gap + sum(sizes)
    T = max(0, total - cut)
    draw = lambda lo, hi: rng.integers(lo, hi, total).tolist()
    token, choice, slot, pos = draw(-1, alphabet), draw(-1, alphabet), draw(-1, 40), draw(-1, 12)
    for c0, p in zip(offsets(parents, gap), parents):  # most are written, and node 0 nearly always
        for i in range(len(p)):
            if rng.random() < (0.95 if i == 0 else 0.8):
                slot[c0 + i], pos[c0 + i] = abs(slot[c0 + i]), 3
    written = [s >= 0 and (P == 0 or 0 <= x < P) for s, x in zip(slot, pos)][:T]
    got = run_accept(parents, token, choice, slot, pos if P else None, P, N, T, ldc, gap)
    want = tree_ref.accept(parents, token[:T], choice[:T], written, N, offsets(parents, gap))
    for g, w in zip(got, want):
        assert g.tolist() == w
    return want[0]


@pytest.mark.parametrize("N", [1, 3, 64, 65, 129, 200, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_tree_accept(N, kind):
    took = check_accept(N, [N, 0, 1, N // 2, N, N + 4], N, kind, 3, 0, 1)
    took += check_accept(N + 1, [N] * 9, N, kind, 1, 10, 5)  # one token: every child agrees
    took += check_accept(N + 2, [N, 1, N], N, kind, 2, 0, 64, cut=N // 2 + 1, gap=3)
    assert max(took) > (1 if N > 2 and kind != "wild" else 0)


def test_tree_accept_a_chain_of_all_nodes():
    for N in (64, 200, 256):
        p = [[i - 1 for i in range(N)]]
        acc, path, after = run_accept(p, list(range(N)), list(range(1, N + 1)), [0] * N, None, 0, N, N)
        assert acc.tolist() == [N] and path[0].tolist() == list(range(N)) and after.tolist() == [N]


def test_tree_accept_nothing_chosen_agrees_with_nothing():
    # a row without a distribution has the alternative -1; a node whose token is -1 is none of its children
    acc, path, after = run_accept([[-1, 0, 0]], [5, -1, -1], [-1, 3, 3], [0, 1, 2], None, 0, 4, 3)
    assert acc.tolist() == [1] and after.tolist() == [-1] and path.tolist() == [[0, -1, -1, -1]]


def test_tree_accept_many_requests():
    rng = np.random.default_rng(9)
    check_accept(9, rng.integers(0, 7, 4096).tolist(), 6, "near", 2, 0, 1)


def caches(L, NP, HKV, page, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    bits = lambda *n: torch.randint(-2 ** 15, 2 ** 15, n, generator=g, device=DEV).to(torch.int16)
    return bits(L, NP, HKV, page, D), bits(L, NP, HKV, D, page)


def check_commit(L, HKV, D, page, slot, cu, acc, path, R, T, N, NP, seed=1):
    KC, VC = caches(L, NP, HKV, page, D, seed)
    k, v = KC.clone(), VC.clone()
    osc.osc_tree_commit(osc.LayerCaches(list(KC), list(VC), NP, HKV, D, page), i32(slot), i32(cu), i32(acc), i32(path), R, T, N)
    clamp = lambda x: min(max(x, 0), T)
    for r in range(R):
        c0, n = clamp(cu[r]), max(0, clamp(cu[r + 1]) - clamp(cu[r]))
        for i in range(1, min(max(acc[r], 0), n, N)):
            p = path[r][i]
            if i < p < min(n, N):
                s, d = slot[c0 + p], slot[c0 + i]
                if 0 <= s < NP * page and 0 <= d < NP * page:
                    k[:, d // page, :, d % page] = k[:, s // page, :, s % page].clone()
                    v[:, d // page, :, :, d % page] = v[:, s // page, :, :, s % page].clone()
    assert torch.equal(KC, k) and torch.equal(VC, v)


@pytest.mark.parametrize("HKV,D,page", [(8, 128, 64), (1, 64, 16), (3, 64, 256), (2, 128, 32), (17, 128, 16)])
@pytest.mark.parametrize("L", [1, 5])
def test_tree_commit(HKV, D, page, L):
    rng = np.random.default_rng(HKV + page + L)
    N, sizes = 40, [40, 0, 1, 17, 40, 33]
    cu, T = offsets([[0] * n for n in sizes]), sum(sizes)
    NP = sum(-(-n // page) + 2 for n in sizes) + 1
    pool, slot = rng.permutation(NP).tolist(), []
    for n in sizes:
        first, used = int(rng.integers(0, page)), pool[:-(-n // page) + 2]
        pool = pool[len(used):]
        slot += [used[(first + i) // page] * page + (first + i) % page for i in range(n)]
    path, acc = [], []
    for n in sizes:  # the whole tree, none of it, some of it
        took = sorted(rng.choice(n, int(rng.integers(0, n + 1)), replace=False).tolist()) if n else []
        took = [0] + [t for t in took if t] if n else []
        acc.append(len(took))
        path.append(took + [-1] * (N - len(took)))
    check_commit(L, HKV, D, page, slot, cu, acc, path, 6, T, N, NP)
    acc[4], path[4] = 40, list(range(40))               # all stay where they are
    acc[0], path[0] = 20, list(range(20, 40)) + [-1] * 20   # all move, from right behind what is written
    check_commit(L, HKV, D, page, slot, cu, acc, path, 6, T, N, NP, 2)
    acc[4], path[4] = 39, [0] + list(range(2, 40)) + [-1]   # each to the slot that the one before it left
    acc[5], path[5] = 2, [0, 32] + [-1] * 38
    check_commit(L, HKV, D, page, slot, cu, acc, path, 6, T, N, NP, 3)


def test_tree_commit_what_names_nothing_moves_nothing():
    N, page, NP = 8, 16, 3
    slot, cu = [0, 1, -1, 3, 48, 5, 6, 7], [0, 8]  # a node without a slot, one outside the pool
    for acc, path in [(5, [0, 3, 4, 5, 6, 7, 7, 7]), (99, [0, 5, 6, 7, 8, 2 ** 31 - 1, -2 ** 31, 9]), (-3, [0] * 8), (4, [0, 0, 1, 2, 0, 0, 0, 0]), (3, [0, 2, 4, 0, 0, 0, 0, 0])]:
        check_commit(2, 2, 64, page, slot, cu, [acc], [path], 1, 8, N, NP)
    check_commit(2, 2, 64, page, slot, [0, 99], [4], [[0, 5, 6, 7, 0, 0, 0, 0]], 1, 8, N, NP)
    check_commit(2, 2, 64, page, slot, [5, 2], [4], [[0, 5, 6, 7, 0, 0, 0, 0]], 1, 8, N, NP)


def test_tree_commit_behind_32_bits():
    """A cache of more than 2^32 bytes: the last page's slots."""
    HKV, D, page = 8, 128, 256
    NP = 2 ** 32 // (2 * HKV * D * page) + 3
    KC, VC = torch.zeros((NP, HKV, page, D), dtype=torch.int16, device=DEV), torch.zeros((NP, HKV, D, page), dtype=torch.int16, device=DEV)
    last = NP - 1
    KC[last, :, 200], VC[last, :, :, 200] = 7, 9
    slot = [last * page + s for s in (10, 11, 200)]
    osc.osc_tree_commit(osc.LayerCaches([KC], [VC], NP, HKV, D, page), i32(slot), i32([0, 3]), i32([2]), i32([[0, 2, -1]]), 1, 3, 3)
    assert bool((KC[last, :, 11] == 7).all()) and bool((VC[last, :, :, 11] == 9).all())
    assert int((KC != 0).sum()) == 2 * HKV * D and int((VC != 0).sum()) == 2 * HKV * D


def test_layer_caches_are_checked():
    KC, VC = caches(2, 3, 2, 16, 64, 1)
    for k, v, n in ((list(KC), list(VC)[:1], 3), (list(KC), list(VC), 4), (list(KC.float()), list(VC), 3), (list(KC.transpose(3, 4)), list(VC), 3)):
        with pytest.raises(osc.OscError):
            osc.LayerCaches(k, v, n, 2, 64, 16)
    with pytest.raises(osc.OscError) as e:  # a layer twice
        osc.osc_tree_commit(osc.LayerCaches([KC[0], KC[0]], list(VC), 3, 2, 64, 16), i32([0]), i32([0, 1]), i32([1]), i32([[0]]), 1, 1, 1)
    assert e.value.status == 2


def test_tree_commit_all_layers_replayed():
    """128 layers, whose addresses a captured call keeps; other paths in each replay, with eager work between."""
    L, NP, HKV, page, D, N, R = 128, 6, 2, 16, 64, 16, 2
    KC, VC = caches(L, NP, HKV, page, D, 5)
    slot, cu = i32([16 * 3 + (5 + i) % 16 if i < 11 else 16 + i for i in range(16)] + list(range(64, 80))), i32([0, 16, 32])
    acc, path = i32([0, 0]), i32([[-1] * N] * R)
    held = osc.LayerCaches(list(KC), list(VC), NP, HKV, D, page)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        osc.osc_tree_commit(held, slot, cu, acc, path, R, 32, N)
    del held  # the call read the addresses; the caches live
    rng = np.random.default_rng(1)
    for it in range(4):
        took = [[0] + sorted(rng.choice(np.arange(1, 16), 7, replace=False).tolist()) for _ in range(R)]
        acc.copy_(i32([8, 8 - it])), path.copy_(i32([t + [-1] * 8 for t in took]))
        k, v = KC.clone(), VC.clone()
        osc.osc_tree_commit(osc.LayerCaches(list(k), list(v), NP, HKV, D, page), slot, cu, acc, path, R, 32, N)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(KC, k) and torch.equal(VC, v)
