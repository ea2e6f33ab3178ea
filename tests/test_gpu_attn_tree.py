"""Attention of token trees over the paged cache against 64 bits, at the lengths, masks and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

import tree_ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402

NAN = float("nan")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def signed(m):
    return m - 2 ** 64 if m >> 63 else m


def build(reqs, HQ, HKV, D, page, N, seed, masks=None, MB=None, pad=0, lead=0):
    """reqs: (context, masks of the new tokens as whole numbers) each, or (context, parents) with masks None."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = -(-N // 64)
    bits = [m if masks else tree_ref.ancestors(m) for _, m in reqs]
    total = [max(c + len(m), 0) for c, m in reqs]
    MB = MB or max(1, max([-(-t // page) for t in total], default=1)) + 1
    used = [-(-min(t, MB * page) // page) for t in total]
    NP = sum(used) + 3
    pool = rng.permutation(NP).tolist()
    table = np.full((max(1, len(reqs)), MB), -1, np.int32)
    for r, u in enumerate(used):
        table[r, :u], pool = pool[:u], pool[u:]
    cu = np.concatenate([[lead], lead + np.cumsum([len(m) for _, m in reqs])]).astype(int).tolist()
    S = cu[-1] + pad
    rows = [[0] * W] * lead + [[signed(m >> 64 * w & (2 ** 64 - 1)) for w in range(W)] for b in bits for m in b] + [[-1] * W] * pad
    randn = lambda *n: torch.randn(n, generator=g, device=DEV, dtype=torch.bfloat16)
    KC, VC = randn(NP, HKV, page, D), randn(NP, HKV, D, page)
    # behind a request's keys, and in pages that nobody has: whatever memory holds
    for r, t in enumerate(total):
        if used[r] and t < used[r] * page:
            KC[table[r, used[r] - 1], :, t % page or page:] = NAN
            VC[table[r, used[r] - 1], :, :, t % page or page:] = NAN
    for p in pool:
        KC[p], VC[p] = NAN, NAN
    return dict(Q=randn(S, HQ, D) * 1.5, KC=KC, VC=VC, S=S, R=len(reqs), HQ=HQ, HKV=HKV, D=D, page=page, MB=MB, NP=NP, table=table, cu=cu, kv=[c + len(m) for c, m in reqs],
                mask=torch.tensor(rows, dtype=torch.int64, device=DEV).reshape(S, W), bits=bits, N=N, scale=D ** -0.5)


def attend(p, S=None, ws=None, out=None, stream=None):
    S = p["S"] if S is None else S
    sizes = (S, p["R"], p["HQ"], p["HKV"], p["D"], p["page"], p["MB"])
    if ws is None:
        ws = poisoned((osc.osc_attn_tree_workspace(*sizes, p["N"]),), torch.uint8)
    if out is None:
        out = poisoned((p["S"], p["HQ"], p["D"]), torch.bfloat16)
    osc.osc_attn_tree(p["Q"], p["KC"], p["VC"], *sizes, p["NP"], torch.from_numpy(p["table"]).to(DEV) if "dev" not in p else p["dev"][0],
                      i32(p["cu"]) if "dev" not in p else p["dev"][1], i32(p["kv"]) if "dev" not in p else p["dev"][2], p["mask"], p["N"], p["scale"], out, ws,
                      stream)
    return out


def check(p, got, S=None, what=""):
    """Against 64 bits, row by row of a key head; every row that the call may not touch still holds its 0xFF bytes."""
    S = p["S"] if S is None else S
    HQ, HKV, D, page, W = p["HQ"], p["HKV"], p["D"], p["page"], p["mask"].shape[1]
    g, cap = HQ // HKV, p["MB"] * p["page"]
    # The weights are two bf16 (2^-16) up to 16 rows a tree, else one (2^-8); scores and exponents as D products of the terms' size in
    # binary32 (2^-24 each), the sums as much again; the output is rounded to bf16 (2^-8 of it).
    wide = 2.0 ** -8 if p["N"] * g > 16 else 2.0 ** -16
    raw, got = got.view(torch.int16), got.double()
    covered = torch.zeros(p["S"], dtype=torch.bool, device=DEV)
    for r in range(p["R"]):
        c0, n, kv = p["cu"][r], p["cu"][r + 1] - p["cu"][r], max(p["kv"][r], 0)
        rows = [i for i in range(n) if c0 + i < S]
        covered[[c0 + i for i in rows]] = True
        if not rows:
            continue
        ctx = p["kv"][r] - n
        end = min(max(ctx + len(rows), 0), cap)  # tokens without a row have no key either
        key = np.arange(end)
        ids = p["table"][r][key // page]
        there = (ids >= 0) & (ids < p["NP"])
        see = np.zeros((len(rows), end), bool)
        for i in rows:
            see[i] = (key < ctx) & there
            for b in range(64 * W):
                if p["bits"][r][i] >> b & 1 and 0 <= ctx + b < end:
                    see[i, ctx + b] = there[ctx + b]
        see = torch.from_numpy(see).to(DEV)
        at, off = torch.from_numpy(np.where(there, ids, 0)).to(DEV).long(), torch.from_numpy(key % page).to(DEV)
        for h in range(HKV):
            k, v = p["KC"][at, h, off].double(), p["VC"][at, h, :, off].double()
            bad = ~torch.isfinite(k).all(1) | ~torch.isfinite(v).all(1)
            hit = (see & bad).any(1)  # rows that see a key or value that is not finite
            k, v = torch.where(bad[:, None], 0.0, k), torch.where(bad[:, None], 0.0, v)
            q = p["Q"][c0:c0 + len(rows), h * g:(h + 1) * g].double()
            s = torch.matmul(q, k.T.contiguous()) * p["scale"] if end else q.new_zeros(len(rows), g, 0)
            s = s.masked_fill(~see[:, None, :], -float("inf"))
            w = torch.softmax(s, 2) if end else s
            w = torch.where(see.any(1)[:, None, None], w, 0.0)
            ref = w @ v
            size = torch.where(torch.isfinite(s), q.abs() @ k.abs().T * p["scale"], 0.0).amax(2, keepdim=True) if end else 0.0
            tol = (wide + 2 * 2.0 ** -24 * (D * size + 64)) * (w @ v.abs()) + 2.0 ** -8 * ref.abs()
            o = got[c0:c0 + len(rows), h * g:(h + 1) * g]
            assert bool(torch.isnan(o[hit]).all()), (what, r, h)
            e = ((o - ref).abs() <= tol)[~hit]
            assert bool(e.all()), (what, r, h, int((~e).sum()), float((o - ref)[~hit].abs().max()))
    assert bool((raw[~covered] == -1).all()), what


# (context, nodes) of each request
REQS = {"alone": [(0, 1)], "no context": [(0, None), (0, 5)], "short": [(3, 4), (0, 0), (17, None), (31, 1), (64, 9)], "ends of pages": [(63, 2), (64, 1), (255, None), (256, 3), (1, 31)],
        "long": [(3000, None)], "mixed": [(2500, 3), (10, None), (0, 0), (900, 12), (0, 2), (5000, 1)]}


@pytest.mark.parametrize("HQ,HKV,D,page", [(32, 8, 128, 64), (4, 4, 64, 16), (8, 1, 128, 256), (5, 1, 64, 32), (17, 17, 128, 128), (48, 2, 128, 16)])
@pytest.mark.parametrize("N", [1, 4, 8, 16, 33, 64, 100, 256])
@pytest.mark.parametrize("reqs", list(REQS))
def test_attn_tree(HQ, HKV, D, page, N, reqs):
    rng = np.random.default_rng(N + HQ)
    size = [(c, N if n is None else min(n, N)) for c, n in REQS[reqs]]
    p = build([(c, tree_ref.tree(rng, n, ("chain", "near", "roots", "star")[i % 4])) for i, (c, n) in enumerate(size)], HQ, HKV, D, page, N, N + page, pad=3, lead=N % 3)
    check(p, attend(p))


@pytest.mark.parametrize("HQ,HKV,D,page,N", [(32, 8, 128, 64, 16), (4, 4, 64, 16, 8), (8, 1, 128, 256, 64), (4, 1, 64, 32, 256), (1, 1, 128, 16, 64)])
def test_attn_tree_any_mask(HQ, HKV, D, page, N):
    """Masks that are no trees: rows that see nothing, everything, what is behind them, and tokens that the request does not have."""
    rng = np.random.default_rng(N)
    whole = (1 << 64 * -(-N // 64)) - 1
    draw = lambda n: [[0, whole, int.from_bytes(rng.bytes(32), "little") & whole, 1 << int(rng.integers(0, n))][int(rng.integers(0, 4))] for _ in range(n)]
    reqs = [(0, draw(N)), (0, [0] * min(N, 5)), (40, draw(N)), (1000, draw(N - 1 or 1)), (0, []), (7, [whole] * N)]
    p = build(reqs, HQ, HKV, D, page, N, N, masks=True, pad=2)
    check(p, attend(p))


@pytest.mark.parametrize("N,HQ,HKV", [(8, 32, 8), (64, 32, 8), (256, 8, 8), (16, 16, 16)])
def test_attn_tree_pages_that_do_not_exist(N, HQ, HKV):
    rng = np.random.default_rng(N)
    p = build([(700, tree_ref.tree(rng, N, "near")), (130, tree_ref.tree(rng, N, "near")), (0, tree_ref.tree(rng, N, "near")), (200, tree_ref.tree(rng, N // 2, "near"))], HQ, HKV, 128, 32, N, 4)
    p["table"][0, 3], p["table"][0, 9], p["table"][1, :] = -1, p["NP"], 2 ** 31 - 1
    p["table"][2, :], p["table"][3, 6] = -5, -1
    check(p, attend(p))


def test_attn_tree_rows_and_keys_beyond():
    rng = np.random.default_rng(1)
    for N, HQ, HKV in ((8, 8, 2), (64, 8, 8), (128, 8, 2)):
        # fewer rows than tokens, keys that the table has no room for, fewer keys than tokens
        p = build([(90, tree_ref.tree(rng, N, "near")), (500, tree_ref.tree(rng, N, "near")), (100, tree_ref.tree(rng, N, "near"))], HQ, HKV, 128, 16, N, 2)
        check(p, attend(p, S=p["S"] - N // 2), S=p["S"] - N // 2, what="rows")
        p = build([(90, tree_ref.tree(rng, N, "near")), (500, tree_ref.tree(rng, N, "near"))], HQ, HKV, 128, 16, N, 2, MB=20)
        check(p, attend(p), what="table")
        p["kv"] = [N // 2, -4]
        check(p, attend(p), what="kv")
        p["kv"] = [2 ** 31 - 1, N]
        check(p, attend(p), what="largest kv")


@pytest.mark.parametrize("N,HQ,HKV", [(8, 32, 8), (16, 64, 8), (64, 32, 8), (64, 4, 4)])
def test_attn_tree_more_tokens_than_nodes(N, HQ, HKV):
    """A request of more tokens than N: right, though its rows see new keys below 64 W only."""
    rng = np.random.default_rng(N)
    p = build([(50, [m & (2 ** 64 - 1) for m in tree_ref.ancestors(tree_ref.tree(rng, 3 * N + 1, "near"))]), (9, [1])], HQ, HKV, 128, 16, N, 3, masks=True)
    check(p, attend(p))


@pytest.mark.parametrize("HQ,HKV,N", [(32, 8, 8), (32, 8, 16), (8, 8, 64), (32, 4, 40), (32, 8, 64), (8, 2, 200)])
def test_attn_tree_not_finite_reaches_only_rows_that_see_it(HQ, HKV, N):
    rng = np.random.default_rng(N)
    for kind in ("near", "star", "roots"):
        parents = [tree_ref.tree(rng, N, kind), tree_ref.tree(rng, N, "chain")]
        p = build(list(zip((333, 64), parents)), HQ, HKV, 128, 32, N, 7)
        for r, j, what, value in ((0, N // 2, "VC", NAN), (0, N - 1, "VC", float("inf")), (0, N // 3, "KC", NAN), (1, N - 1, "VC", -float("inf")), (1, N // 2, "KC", NAN)):
            at = p["kv"][r] - N + j
            t, id = p[what], p["table"][r, at // 32]
            if what == "KC":
                t[id, :, at % 32, 77] = value
            else:
                t[id, :, 5, at % 32] = value
        check(p, attend(p), what=kind)
        # beside pages that do not exist one to four tiles ahead, and values of the context that are not finite behind one
        for page in (4, 5, 6, 8):
            p["table"][0, page] = -1
            check(p, attend(p), what=(kind, page))


@pytest.mark.parametrize("reqs,HQ,HKV,N", [([(60000, 16)], 8, 1, 16), ([(60000, 64)], 4, 1, 64), ([(33000, 256)], 32, 8, 256), ([(9000, 8)] * 3 + [(5, 8)] * 60, 32, 8, 8),
                                           ([(300, 7)] * 200, 16, 4, 8), ([(40, 3)] * 700, 8, 8, 4), ([(100, 1)] * 4096, 4, 4, 1), ([(2000, 60)] * 40, 32, 8, 64)])
def test_attn_tree_cuts(reqs, HQ, HKV, N):
    rng = np.random.default_rng(len(reqs))
    p = build([(c, tree_ref.tree(rng, n, "near")) for c, n in reqs], HQ, HKV, 64, 64, N, 5)
    got = attend(p)
    if len(reqs) > 100:  # the reference of a few
        keep = sorted(rng.choice(len(reqs), 12, replace=False).tolist() + [0, len(reqs) - 1])
        assert not bool((got.view(torch.int16) == -1).all(2).any())
        for r in keep:
            sub = dict(p, R=1, cu=[0, len(p["bits"][r])], kv=[p["kv"][r]], table=p["table"][r:r + 1], bits=[p["bits"][r]], S=len(p["bits"][r]),
                       Q=p["Q"][p["cu"][r]:p["cu"][r + 1]])
            check(sub, got[p["cu"][r]:p["cu"][r + 1]], what=r)
    else:
        check(p, got)
    again = attend(p)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))  # a fixed order


def test_attn_tree_heads():
    for HQ, HKV, N in ((1024, 1, 2), (1024, 1024, 3), (1000, 8, 5), (3, 3, 256)):
        rng = np.random.default_rng(HQ)
        p = build([(70, tree_ref.tree(rng, N, "near")), (3, tree_ref.tree(rng, 1, "near"))], HQ, HKV, 64, 16, N, 5)
        check(p, attend(p), what=(HQ, HKV))


def test_attn_tree_agrees_with_a_run_of_tokens():
    """A chain is a run of tokens: osc_attn_paged's rows, by its own rounding of the weights."""
    p = build([(1000, list(range(-1, 15))), (20, list(range(-1, 15)))], 32, 8, 128, 64, 16, 9)
    got, run = attend(p), poisoned((32, 32, 128), torch.bfloat16)
    ws = poisoned((osc.osc_attn_workspace(32, 2, 32, 8, 128, 64, p["MB"]) + 16,), torch.uint8)
    osc.osc_attn_paged(p["Q"], p["KC"], p["VC"], 32, 2, 32, 8, 128, 64, p["MB"], p["NP"], torch.from_numpy(p["table"]).to(DEV), i32(p["cu"]), i32(p["kv"]), p["scale"], run, ws)
    # both within their bounds of the exact rows: 2^-8 of the weights and twice the output's rounding, of values up to 5
    assert float((got.double() - run.double()).abs().max()) <= 2.0 ** -8 * 5 * 3


def test_attn_tree_behind_32_bits():
    """A cache of more than 2^32 bytes, whose last pages hold the request."""
    HQ, HKV, D, page, N = 8, 8, 128, 256, 8
    p = build([(600, [-1, 0, 0, 1, 1, 2, 3, 3])], HQ, HKV, D, page, N, 3)
    NP = 2 ** 32 // (2 * HKV * D * page) + 8
    KC, VC = torch.zeros((NP, HKV, page, D), dtype=torch.bfloat16, device=DEV), torch.zeros((NP, HKV, D, page), dtype=torch.bfloat16, device=DEV)
    KC[-p["NP"]:], VC[-p["NP"]:] = p["KC"], p["VC"]
    table = np.where(p["table"] >= 0, p["table"] + NP - p["NP"], -1).astype(np.int32)
    p = dict(p, KC=KC, VC=VC, NP=NP, table=table)
    check(p, attend(p))


def test_attn_tree_replayed():
    """Two graphs on two streams, each with its workspace, replayed on changing lengths with eager calls between."""
    ps, graphs = [], []
    rng = np.random.default_rng(2)
    for seed, (HQ, HKV, N) in enumerate(((32, 8, 16), (32, 8, 64))):
        p = build([(2000, tree_ref.tree(rng, N, "near")), (300, tree_ref.tree(rng, N, "near"))], HQ, HKV, 128, 64, N, seed)
        p["dev"] = [torch.from_numpy(p["table"]).to(DEV), i32(p["cu"]), i32(p["kv"])]
        ws = poisoned((osc.osc_attn_tree_workspace(p["S"], 2, HQ, HKV, 128, 64, p["MB"], N),), torch.uint8)
        out = poisoned((p["S"], HQ, 128), torch.bfloat16)
        attend(p, ws=ws, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attend(p, ws=ws, out=out)
        ps.append((p, out, torch.cuda.Stream(), ws)), graphs.append(graph)  # a graph's workspace lives as long as the graph
    for it in range(4):
        for p, out, *_ in ps:
            N = p["N"]
            p["kv"] = [2000 + N - 100 * it, 300 + N - 70 * it]
            p["dev"][2].copy_(i32(p["kv"]))
            out.view(torch.int16).fill_(-1)
        torch.cuda.synchronize()
        for (_, _, s, _), graph in zip(ps, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for p, out, *_ in ps:
            assert torch.equal(out.view(torch.int16), attend(p).view(torch.int16)), it
            check(p, out, what=it)


@pytest.mark.parametrize("N,HQ,HKV", [(4, 4, 1), (64, 32, 8)])
def test_attn_tree_idle_requests(N, HQ, HKV):
    """Requests without a token among others, and no other at all: nothing of O is written for them."""
    rng = np.random.default_rng(N)
    for reqs in ([(50, 0)] * 70, [(50, 0)] * 70 + [(300, N)] + [(0, 0)] * 200, [(0, 0)]):
        p = build([(c, tree_ref.tree(rng, n, "near")) for c, n in reqs], HQ, HKV, 128, 32, N, 6, pad=5)
        check(p, attend(p))


def test_attn_tree_on_another_stream():
    rng = np.random.default_rng(8)
    for N in (4, 40):
        p = build([(700, tree_ref.tree(rng, N, "near")), (64, tree_ref.tree(rng, N, "near"))], 16, 4, 128, 64, N, 6)
        p["dev"] = [torch.from_numpy(p["table"]).to(DEV), i32(p["cu"]), i32(p["kv"])]
        want = attend(p)
        ws = poisoned((osc.osc_attn_tree_workspace(p["S"], 2, 16, 4, 128, 64, p["MB"], N),), torch.uint8)
        out = poisoned((p["S"], 16, 128), torch.bfloat16)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        attend(p, ws=ws, out=out, stream=side)
        side.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("HQ,HKV,N,D,page", [(4, 1, 4, 128, 32), (16, 16, 16, 64, 16), (8, 8, 8, 128, 64), (8, 1, 2, 64, 32), (3, 1, 5, 128, 16), (2, 2, 1, 64, 256), (16, 1, 1, 128, 32)])
def test_attn_tree_not_finite_in_tiles_of_16_rows(HQ, HKV, N, D, page):
    """The same where a tree's rows fit into one tile, over contexts that leave it whole and that cut it: the join takes NaN parts too."""
    assert N * HQ // HKV <= 16
    rng = np.random.default_rng(N + D)
    for kind in ("near", "star", "roots"):
        parents = [tree_ref.tree(rng, N, kind), tree_ref.tree(rng, N, "chain"), tree_ref.tree(rng, N, kind), tree_ref.tree(rng, N, kind)]
        p = build(list(zip((333, 64, 9000, 0), parents)), HQ, HKV, D, page, N, 7)
        for r, j, what, value in ((0, N // 2, "VC", NAN), (0, N - 1, "VC", float("inf")), (0, N // 3, "KC", NAN), (1, N - 1, "VC", -float("inf")), (1, N // 2, "KC", NAN),
                                  (2, N // 2, "VC", NAN), (2, N - 1, "KC", NAN), (3, N // 3, "VC", float("inf"))):
            at = p["kv"][r] - N + j
            t, id = p[what], p["table"][r, at // page]
            if what == "KC":
                t[id, :, at % page, D - 3] = value
            else:
                t[id, :, 5, at % page] = value
        check(p, attend(p), what=kind)
        # beside pages that do not exist: the first, one ahead of the new keys, and the last, of the new keys themselves
        for r, at in ((0, 0), (2, 3000), (2, 8999), (0, 332), (2, 9000 + N - 1)):
            p["table"][r, at // page] = -1
            check(p, attend(p), what=(kind, r, at))
