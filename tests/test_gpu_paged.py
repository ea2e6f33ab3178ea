"""Page plan, head norm / rotary / cache write, and attention over the paged cache against plain
implementations in 64 bits, at the lengths, layouts and masks where they can go wrong."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402

EPS = 1e-6


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ------------------------------------------------------------------ page plan

def plan_reference(ctx, new, page, NP, free, head, T, table, MB):
    """One request and one token after the other."""
    table = [list(r) for r in table]
    cu, kv, slot, pos, used = [0], [], [], [], 0
    head = max(head, 0)
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        have = min(-(-c // page), MB)
        want = min(-(-(c + n) // page), MB)
        for q in range(have, want):
            id = free[head + used] if head + used < len(free) else -1
            table[r][q] = id if 0 <= id < NP else -1
            used += 1
        for i in range(n):
            at = c + i
            id = table[r][at // page] if at < MB * page else -1
            pos.append(at)
            slot.append(id * page + at % page if 0 <= id < NP else -1)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = [-1] * max(0, T - len(slot))
    return cu, kv, table, (slot + pad)[:T], (pos + pad)[:T], used


def run_plan(ctx, new, page, NP, free, head, T, table, MB, R=None):
    R = len(ctx) if R is None else R
    out = dict(cu=poisoned((R + 3,), torch.int32), kv=poisoned((R + 2,), torch.int32), slot=poisoned((T + 2,), torch.int32),
               pos=poisoned((T + 2,), torch.int32), used=poisoned((2,), torch.int32))
    tab = i32(table).reshape(R, MB) if R else i32([0])
    osc.osc_page_plan(i32(ctx or [0]), i32(new or [0]), R, page, NP, i32(free or [0]), len(free), None if head is None else i32([head]), T, tab,
                      MB, out["cu"], out["kv"], out["slot"], out["pos"], out["used"])
    torch.cuda.synchronize()
    return {k: v.tolist() for k, v in out.items()}, tab.tolist()


def check_plan(ctx, new, page, NP, free, head, T, table, MB):
    out, tab = run_plan(ctx, new, page, NP, free, head, T, table, MB)
    cu, kv, rt, slot, pos, used = plan_reference(ctx, new, page, NP, free, head or 0, T, table, MB)
    R = len(ctx)
    assert out["cu"] == cu + [-1] * 2 and out["kv"] == kv + [-1] * 2  # and what stands behind is untouched
    assert out["slot"] == slot + [-1] * 2 and out["pos"] == pos + [-1] * 2 and out["used"] == [used, -1]
    if R:
        assert tab == rt


def started(rng, ctx, page, MB, NP):
    """Tables of the tokens in the cache and the free list behind them."""
    ids = rng.permutation(NP).tolist()
    table = []
    for c in ctx:
        k = min(-(-max(c, 0) // page), MB)
        table.append(ids[:k] + [-7] * (MB - k))
        ids = ids[k:]
    return table, ids


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("R,most,T", [(1, 1, 1), (1, 3000, 3000), (3, 40, 200), (64, 1, 64), (257, 5, 2000), (1000, 70, 40000)])
def test_page_plan(page, R, most, T):
    rng = np.random.default_rng(R + most + page)
    ctx = [int(v) for v in rng.integers(0, 600, R)]
    ctx[0] = page * 3  # a request that stands at a page's end
    new = [int(v) for v in rng.integers(0, most + 1, R)]
    new[-1] = most
    MB = -(-(600 + most) // page)
    NP = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) + 5
    table, free = started(rng, ctx, page, MB, NP)
    check_plan(ctx, new, page, NP, free, 0, T, table, MB)
    check_plan(ctx, new, page, NP, [9999999, -4] + free, 2, T, table, MB)  # the list's head is where the step starts
    check_plan(ctx, new, page, NP, free, None, T, table, MB)


def test_page_plan_what_does_not_fit():
    page, MB, NP = 16, 4, 50
    rng = np.random.default_rng(3)
    ctx, new = [0, 30, 60, 64, -5, 200], [40, 40, 10, 3, -9, 1]  # past the row, at its end, below 0
    table, free = started(rng, ctx, page, MB, NP)
    check_plan(ctx, new, page, NP, free, 0, 100, table, MB)
    check_plan(ctx, new, page, NP, free[:2], 0, 100, table, MB)          # the free list ends inside the step
    check_plan(ctx, new, page, NP, free, len(free) + 3, 100, table, MB)  # starts behind its end
    check_plan(ctx, new, page, NP, free, -2, 100, table, MB)
    check_plan(ctx, new, page, NP, [], 0, 100, table, MB)
    check_plan(ctx, new, page, NP, [NP, -1, 2 ** 31 - 1] + free, 0, 100, table, MB)  # ids off the pool
    check_plan(ctx, new, page, NP, free, 0, 50, table, MB)               # more tokens than rows
    check_plan(ctx, new, page, NP, free, 0, 0, table, MB)
    check_plan([], [], page, NP, free, 0, 7, [], MB)
    bad = [r[:] for r in table]
    bad[1][1] = NP  # the page that request 1 stands in
    check_plan(ctx, new, page, NP, free, 0, 100, bad, MB)


def test_page_plan_sums_saturate():
    big = 2 ** 31 - 1
    out, _ = run_plan([big, 5, big], [big, big, 3], 16, 8, [1, 2], 0, 6, [[0] * 2] * 3, 2)
    assert out["cu"][:4] == [0, big, big, big] and out["kv"][:3] == [big] * 3
    assert out["slot"][:6] == [-1] * 6 and out["pos"][:6] == [big] * 6


def test_page_plan_most_requests():
    R = osc.OSC_MAX_REQUESTS
    check_plan([16] * R, [1] * R, 16, 2 * R, list(range(R, 2 * R)), 0, R, [[r, -1] for r in range(R)], 2)


# ------------------------------------------------------------------ cache write

def append_reference(qkv, HQ, HKV, D, wq, wk, cs, pos):
    """64-bit q, k (before rounding) and the size of the rotation's terms."""
    S = qkv.shape[0]
    x = qkv.double().reshape(S, HQ + 2 * HKV, D)
    qk = x[:, :HQ + HKV]
    if wq is not None:
        w = torch.cat([wq.double().expand(HQ, D), wk.double().expand(HKV, D)])
        qk = qk / torch.sqrt((qk * qk).mean(2, keepdim=True) + EPS) * w
    size = qk.abs()
    if cs is not None:
        c = cs.double()[pos.clamp(0, cs.shape[0] - 1).long()][:, None]
        co, si = c[..., :D // 2], c[..., D // 2:]
        a, b = qk[..., :D // 2], qk[..., D // 2:]
        size = torch.cat([(a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs()], 2)
        qk = torch.cat([a * co - b * si, b * co + a * si], 2)
    return qk[:, :HQ], qk[:, HQ:], x[:, HQ + HKV:], size


# rounded once, half a step of 2^-8; ahead of that at most 40 binary32 roundings (a lane's 16 squares, 3 sums across
# lanes, division, root, reciprocal, two products, two of the rotation): under 2^-18 of the terms' size
def close(got, ref, size):
    return bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * size).all())


@pytest.mark.parametrize("S", [1, 5, 64, 131])
@pytest.mark.parametrize("HQ,HKV,D,page", [(32, 8, 128, 64), (4, 4, 64, 16), (5, 1, 128, 256), (3, 2, 64, 32)])
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False), (False, False)])
def test_qkv_append(S, HQ, HKV, D, page, norm, rope):
    g = gen(S + HQ + D)
    r = lambda *n: torch.randn(n, generator=g, device=DEV)
    NP, P = -(-S // page) + 3, 500
    qkv = (r(S, (HQ + 2 * HKV) * D) * 3).bfloat16()
    wq, wk = ((1 + 0.3 * r(D)).bfloat16(), (1 + 0.3 * r(D)).bfloat16()) if norm else (None, None)
    cs = torch.cat([a.reshape(P, D // 2) for a in (torch.cos(r(P * D // 2) * 100), torch.sin(r(P * D // 2) * 100))], 1).contiguous() if rope else None
    slots = torch.randperm(NP * page, generator=g, device=DEV)[:S].to(torch.int32)
    if S == 131:  # consecutive slots inside shuffled pages, as a chunk has them
        slots = ((torch.arange(S, device=DEV) + 7) + page).to(torch.int32)
    pos = torch.randint(0, P, (S,), generator=g, device=DEV, dtype=torch.int32)
    skip = torch.zeros(S, dtype=torch.bool, device=DEV)
    if S >= 64:
        slots[3], slots[10], slots[20] = -1, NP * page, -2 ** 31
        skip[[3, 10, 20]] = True
        if rope:
            pos[30], pos[31] = P, -1
            skip[[30, 31]] = True
    Q, KC, VC = poisoned((S, HQ, D), torch.bfloat16), poisoned((NP, HKV, page, D), torch.bfloat16), poisoned((NP, HKV, D, page), torch.bfloat16)
    osc.osc_qkv_append(qkv, S, HQ, HKV, D, wq, wk, EPS, cs, P if rope else 0, pos if rope else None, slots, Q, KC, VC, NP, page)
    q, k, v, size = append_reference(qkv, HQ, HKV, D, wq, wk, cs, pos)
    keep = ~skip
    assert close(Q[keep], q[keep], size[keep][:, :HQ])
    assert bool((Q[skip].view(torch.int16) == -1).all())
    sl = slots[keep].long()
    assert close(KC[sl // page, :, sl % page], k[keep], size[keep][:, HQ:])
    assert torch.equal(VC[sl // page, :, :, sl % page].double(), v[keep])
    rest = torch.ones(NP * page, dtype=torch.bool, device=DEV)
    rest[sl] = False
    assert bool((KC.view(torch.int16).permute(0, 2, 1, 3).reshape(NP * page, -1)[rest] == -1).all())
    assert bool((VC.view(torch.int16).permute(0, 3, 1, 2).reshape(NP * page, -1)[rest] == -1).all())


# ------------------------------------------------------------------ attention

def build(reqs, HQ, HKV, D, page, seed, spread=1.5, slack=2, garbage=float("nan"), MB=None, NP=None):
    """reqs: (keys, new tokens) of each request.  What no request holds is garbage."""
    g = gen(seed)
    need = [-(-kv // page) for kv, _ in reqs]
    MB = max(need + [1]) + 1 if MB is None else MB
    NP = sum(need) + slack if NP is None else NP
    ids = torch.randperm(NP, generator=g, device=DEV).tolist() if NP < 100000 else list(range(NP - 1, NP - 1 - sum(need), -1))
    KC = torch.full((NP, HKV, page, D), garbage, dtype=torch.bfloat16, device=DEV) if NP < 100000 else torch.empty((NP, HKV, page, D), dtype=torch.bfloat16, device=DEV)
    VC = torch.full((NP, HKV, D, page), garbage, dtype=torch.bfloat16, device=DEV) if NP < 100000 else torch.empty((NP, HKV, D, page), dtype=torch.bfloat16, device=DEV)
    table, at = [], 0
    for (kv, _), k in zip(reqs, need):
        row = ids[at:at + k]
        at += k
        for i, id in enumerate(row):
            n = min(page, kv - i * page)
            KC[id, :, :n] = torch.randn((HKV, n, D), generator=g, device=DEV).bfloat16()
            VC[id, :, :, :n] = torch.randn((HKV, D, n), generator=g, device=DEV).bfloat16()
        table.append(row + [-1] * (MB - k))
    S = sum(n for _, n in reqs)
    Q = (torch.randn((S, HQ, D), generator=g, device=DEV) * spread).bfloat16()
    cu = [0]
    for _, n in reqs:
        cu.append(cu[-1] + n)
    return dict(Q=Q, KC=KC, VC=VC, S=S, R=len(reqs), HQ=HQ, HKV=HKV, D=D, page=page, MB=MB, NP=NP, table=table, cu=cu, kv=[k for k, _ in reqs],
                scale=D ** -0.5)


def attend(p, S=None, O=None, stream=None, ws=None):
    S = p["S"] if S is None else S
    sizes = (S, p["R"], p["HQ"], p["HKV"], p["D"], p["page"], p["MB"])
    O = poisoned((S, p["HQ"], p["D"]), torch.bfloat16) if O is None else O
    if ws is None:
        ws = poisoned((osc.osc_attn_workspace(*sizes),), torch.uint8)
    osc.osc_attn_paged(p["Q"], p["KC"], p["VC"], *sizes, p["NP"], i32(p["table"]), i32(p["cu"]), i32(p["kv"]), p["scale"], O, ws, stream)
    return O


def attn_reference(p):
    """Each token and key head by itself in 64 bits: output, and how far a right one may be from it."""
    S, HQ, HKV, D, page = p["S"], p["HQ"], p["HKV"], p["D"], p["page"]
    g = HQ // HKV
    out = torch.zeros(S, HQ, D, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for r in range(p["R"]):
        a, b = (min(max(c, 0), S) for c in p["cu"][r:r + 2])
        n, first = b - a, max(p["kv"][r], 0) - (b - a) - max(p["cu"][r + 1] - S, 0)  # token i sees keys up to first + i
        kv = min(max(first + n, 0), p["MB"] * page)
        ids = torch.tensor(p["table"][r], device=DEV)[torch.arange(kv, device=DEV) // page]
        ok = (ids >= 0) & (ids < p["NP"])
        ids = ids.clamp(0, p["NP"] - 1)
        off = torch.arange(kv, device=DEV) % page
        hidden = torch.arange(kv, device=DEV)[None] > (first + torch.arange(n, device=DEV))[:, None]
        hidden = hidden | ~ok[None]
        for h in range(HKV):
            k = p["KC"][ids, h, off].double()
            v = torch.where(ok[:, None], p["VC"][ids, h, :, off].double(), 0.0)
            for hq in range(h * g, (h + 1) * g):
                q = p["Q"][a:a + n, hq].double()
                s = (q @ k.T * p["scale"]).masked_fill(hidden, -float("inf"))
                w = torch.softmax(s, 1).nan_to_num(0.0)  # a row that sees nothing: zeros
                out[a:a + n, hq] = w @ v
                # Weights rounded to bf16 (half a step, 2^-8, of each), scores summed in binary32 (D products, 2^-24 of
                # the terms' size each, and as much for the exponent and the sums), the output rounded once more.
                size = torch.where(hidden, 0.0, q.abs() @ k.abs().nan_to_num(0.0).T * p["scale"]).amax(1, keepdim=True) if kv else q.new_zeros(n, 1)
                tol[a:a + n, hq] = (2.0 ** -8 + 2 * 2.0 ** -24 * (D * size + 64)) * (w @ v.abs()) + 2.0 ** -8 * out[a:a + n, hq].abs()
    return out, tol


def check_attn(p, O=None):
    O = attend(p) if O is None else O
    ref, tol = attn_reference(p)
    err = (O[:p["S"]].double() - ref).abs()
    assert bool(torch.isfinite(O.float()).all())
    assert bool((err <= tol).all()), (float((err / tol.clamp(min=1e-30)).max()), int((err > tol).sum()))


HEADS = [(8, 2, 128), (4, 4, 128), (5, 1, 64), (16, 1, 128), (33, 1, 64), (6, 2, 64)]


@pytest.mark.parametrize("HQ,HKV,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attn_decode(HQ, HKV, D, page):
    check_attn(build([(1, 1), (31, 1), (32, 1), (33, 1), (500, 1), (257, 1), (16, 1)], HQ, HKV, D, page, HQ + page))


@pytest.mark.parametrize("HQ,HKV,D", HEADS)
@pytest.mark.parametrize("page,MB", [(16, None), (32, None), (128, None), (16, 300), (64, 100)])
def test_attn_chunks_of_uneven_lengths(HQ, HKV, D, page, MB):
    check_attn(build([(40, 40), (300, 7), (65, 64), (1, 1), (200, 0), (0, 0), (333, 129), (64, 3)], HQ, HKV, D, page, HQ * page, MB=MB))


@pytest.mark.parametrize("kv,n", [(1, 1), (2, 2), (17, 9), (63, 63), (64, 64), (129, 33), (700, 1), (700, 32), (1500, 300), (4100, 40)])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("room", [0, 40000])
def test_attn_one_request(kv, n, D, page, room):
    check_attn(build([(kv, n)], 8, 2, D, page, kv + n, MB=-(-(kv + room) // page)))


@pytest.mark.parametrize("reqs", [[(2000, 2000)], [(6000, 600)], [(2200, 1100)], [(9000, 700), (300, 300)], [(700, 700)] * 3, [(700, 700), (0, 0), (1, 1), (15000, 90)]])
def test_attn_whole_or_cut_as_the_lengths_are(reqs):
    """A table with room for 60 thousand keys: only the lengths on the device tell."""
    p = build(reqs, 8, 2, 128, 64, 25, MB=940)
    a = attend(p)
    check_attn(p, a)
    assert torch.equal(attend(p), a)


@pytest.mark.parametrize("reqs", [[(5000, 1)], [(3, 1), (5012, 1), (0, 0)], [(5012, 60), (1, 1)], [(128, 128), (4000, 9)], [(20000, 1)],
                                  [(9000, 300), (64, 64), (1, 1), (700, 0)], [(1, 1)] * 70, [(300, 1), (0, 0)] * 40, [(2000, 2000)],
                                  [(260, 2)] * 130])
@pytest.mark.parametrize("HQ,HKV", [(4, 1), (6, 3)])
def test_attn_cuts(reqs, HQ, HKV):
    """Tiles cut into many parts, parts of many tiles, idle requests in between; more key heads than 1 and not 8."""
    check_attn(build(reqs, HQ, HKV, 64, 64, len(reqs) + HQ, MB=330))


@pytest.mark.parametrize("reqs,D,page", [([(3300, 3300)], 64, 16), ([(2100, 1700)], 128, 64), ([(1500, 1500), (0, 0), (900, 700), (601, 600), (1, 1), (520, 520)], 64, 64),
                                         ([(30, 30)] * 112, 64, 32), ([(900, 1), (1700, 1700)], 128, 256), ([(1700, 1700), (30000, 1), (70, 60)], 128, 64),
                                         ([(20000, 20), (3300, 3300)], 64, 128)])
def test_attn_many_tiles(reqs, D, page):
    """Tiles enough to leave them whole: one request, several, and such with a context so long that they are cut all the same."""
    p = build(reqs, 64 if D == 64 else 128, 8, D, page, len(reqs) + D)
    if len(reqs) > 3:
        p["table"][0][3 if len(reqs) < 20 else 0] = -1
    check_attn(p)


def test_attn_rows_that_see_nothing_are_zero():
    p = build([(5, 5), (40, 40), (70, 2)], 4, 2, 128, 16, 7)
    p["kv"] = [3, 0, 70]  # fewer keys than tokens: the first ones see none
    p["table"][2] = [-1, p["NP"], -5, 2 ** 31 - 1, -2 ** 31] + p["table"][2][5:]
    p["table"][2] = p["table"][2][:p["MB"]]
    O = attend(p)
    ref, tol = attn_reference(p)
    assert bool(((O.double() - ref).abs() <= tol).all())
    assert bool((O[:2] == 0).all()) and bool((O[5:47] == 0).all()) and bool((O[2:5] != 0).any())


@pytest.mark.parametrize("n", [2, 90])
def test_attn_leaves_out_pages_that_do_not_exist(n):
    p = build([(300, n), (100, 1)], 4, 1, 128, 16, n, MB=300 if n == 90 else None)
    p["table"][0][2] = -1
    p["table"][0][7] = p["NP"]
    p["KC"][0], p["VC"][0] = float("nan"), float("inf")  # what stands in for them is never used
    for r in range(2):
        p["table"][r] = [-1 if id == 0 else id for id in p["table"][r]]
    check_attn(p)


def test_attn_rows_outside_the_requests_stay_as_they_were():
    p = build([(50, 9), (20, 3)], 4, 2, 128, 16, 1)
    full = poisoned((p["S"] + 6, 4, 128), torch.bfloat16)
    Q = torch.cat([torch.full((2, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV), p["Q"],
                   torch.full((4, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)])
    for MB in (p["MB"], 300):
        q = dict(p, Q=Q, cu=[c + 2 for c in p["cu"]], table=[r + [-1] * (MB - len(r)) for r in p["table"]], MB=MB)
        O = attend(q, S=p["S"] + 6, O=full)
        assert bool((O[:2].view(torch.int16) == -1).all()) and bool((O[-4:].view(torch.int16) == -1).all())
        check_attn(p, O[2:-4])


def test_attn_lengths_off_their_ranges_stay_inside():
    """Counts past S and lengths past the table: the other tokens' keys are as if all had been there."""
    p = build([(64, 8), (64, 8)], 4, 2, 128, 16, 2, MB=4)
    for cu, kv in (([-3, 8, 10 ** 9], [10 ** 9, -7]), ([0, 8, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1]), ([-2 ** 31, 8, 16], [-2 ** 31, 64])):
        check_attn(dict(p, cu=cu, kv=kv))


@pytest.mark.parametrize("idle", [0, 40])
def test_attn_tokens_that_the_plan_does_not_map_change_nothing_for_the_others(idle):
    """5 tokens too many for the table's pages, and 5 for the call's rows: what is left is the request without them."""
    p = build([(70, 1), (512, 30), *[(0, 0)] * idle], 4, 2, 64, 64, 21, MB=8)
    ref, tol = attn_reference(p)
    ok = lambda O, n: bool(((O[:n].double() - ref[:n]).abs() <= tol[:n]).all())
    long = dict(p, Q=torch.cat([p["Q"], p["Q"][:5]]), S=36, cu=[0, 1] + [36] * (idle + 1), kv=[70, 517] + [0] * idle)
    O = attend(long)
    assert ok(O, 31) and bool(torch.isfinite(O.float()).all())
    O = attend(dict(p, S=26), S=26)
    assert ok(O, 26)


def test_attn_chunk_and_tokens_among_idle_requests():
    """As many requests as a call may have, most of them idle, and fewer tokens than requests: a chunk on single-token tiles."""
    reqs = [(0, 0)] * 4096
    reqs[5], reqs[70], reqs[71], reqs[4095] = (900, 1), (300, 200), (17, 0), (65, 65)
    check_attn(build(reqs, 8, 2, 64, 64, 22, MB=16))


def test_attn_chunks_of_the_most_requests():
    """More tokens than the 4096 requests: large tiles of one or two tokens, found among many."""
    rng = np.random.RandomState(23)
    check_attn(build([(int(k), min(int(k), 2)) for k in rng.randint(0, 40, 4096)], 2, 1, 64, 16, 23, MB=3))


def test_attn_large_scores_and_growing_maximum():
    """Scores whose maximum grows from tile to tile, by little and by much, and scores far below."""
    for step in (0.002, 0.05, 1.0):
        p = build([(600, 70), (333, 1)], 4, 1, 128, 64, 3, spread=1.0, MB=64)
        for r in range(2):
            for i in range(p["kv"][r]):
                id, off = p["table"][r][i // 64], i % 64
                p["KC"][id, :, off] += i * step
        p["Q"] = p["Q"].abs()
        ref, tol = attn_reference(p)
        O = attend(p)
        assert bool(((O.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("n", [1, 40])
def test_attn_large_values_under_a_growing_maximum(n):
    """Values close to 2^80, and scores that grow by less than what the running maximum may lag behind."""
    p = build([(600, n), (601, 1)], 4, 1, 64, 64, 24, spread=0.0)
    p["Q"][..., 0] = 4.0
    for r in range(2):
        for i in range(p["kv"][r]):
            p["KC"][p["table"][r][i // 64], :, i % 64, 0] = i * 0.04  # scores up to 12, 17 in the exponent of 2
    p["VC"] *= 2.0 ** 76
    check_attn(p)


def test_attn_infinite_and_nan_inputs_stay_in_their_rows():
    p = build([(200, 60)], 4, 1, 128, 64, 4)
    ref, tol = attn_reference(p)
    p["Q"][10, 1] = float("nan")
    p["Q"][20, 3, 0] = float("inf")
    O = attend(p)
    assert bool(torch.isnan(O[10, 1].float()).all()) and bool(torch.isnan(O[20, 3].float()).any())
    O[10, 1], O[20, 3] = ref[10, 1].bfloat16(), ref[20, 3].bfloat16()
    assert bool(((O.double() - ref).abs() <= tol).all())


def test_attn_a_key_of_nan_reaches_only_rows_that_see_it():
    p = build([(200, 60)], 4, 1, 128, 64, 5)
    ref, tol = attn_reference(p)
    at = 170
    p["KC"][p["table"][0][at // 64], :, at % 64] = float("nan")
    O = attend(p)
    first = at - 140  # token i sees keys up to 140 + i
    assert bool(((O.double() - ref).abs() <= tol)[:first].all()) and bool(torch.isnan(O[first:].float()).all())


def test_attn_cache_past_31_bits_of_elements():
    """10^5 pages of 2^17 elements: the pages in use stand at the end, far past 2^31 elements."""
    p = build([(600, 1), (300, 50)], 8, 8, 64, 256, 6, NP=100000)
    assert p["KC"].numel() > 2 ** 31 * 4 or p["KC"].numel() > 2 ** 31
    assert min(i for r in p["table"] for i in r if i >= 0) * 8 * 256 * 64 > 2 ** 31
    check_attn(p)


def test_append_cache_past_31_bits_of_elements():
    NP, HKV, page, D = 17000, 8, 256, 64
    KC = torch.zeros((NP, HKV, page, D), dtype=torch.bfloat16, device=DEV)
    VC = torch.zeros((NP, HKV, D, page), dtype=torch.bfloat16, device=DEV)
    S = 70
    qkv = torch.randn((S, 3 * HKV * D), generator=gen(1), device=DEV).bfloat16()
    slots = (NP * page - 100 + torch.arange(S, device=DEV)).to(torch.int32)
    Q = poisoned((S, HKV, D), torch.bfloat16)
    osc.osc_qkv_append(qkv, S, HKV, HKV, D, None, None, 0.0, None, 0, None, slots, Q, KC, VC, NP, page)
    x = qkv.reshape(S, 3, HKV, D)
    sl = slots.long()
    assert torch.equal(Q, x[:, 0]) and torch.equal(KC[sl // page, :, sl % page], x[:, 1]) and torch.equal(VC[sl // page, :, :, sl % page], x[:, 2])
    assert int((KC != 0).sum()) == int((x[:, 1] != 0).sum()) and int((VC != 0).sum()) == int((x[:, 2] != 0).sum())


def test_attn_is_the_same_every_time_and_in_other_company():
    p = build([(900, 1), (900, 70), (64, 64)], 8, 2, 128, 64, 8, MB=40)
    a = attend(p)
    for _ in range(3):
        assert torch.equal(attend(p), a)
    # alone on the device or with the workspace's old contents, a request's rows do not change
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = attend(p)
    c = attend(p)
    torch.cuda.synchronize()
    assert torch.equal(b, a) and torch.equal(c, a)


def test_attn_binding_refuses_short_and_strided_buffers():
    p = build([(900, 1)], 8, 2, 128, 64, 8, MB=40)
    need = osc.osc_attn_workspace(1, 1, 8, 2, 128, 64, 40)
    for ws in (None, torch.empty(need - 16, dtype=torch.uint8, device=DEV)):
        with pytest.raises(osc.OscError):
            attend(p, ws=ws) if ws is not None else osc.osc_attn_paged(p["Q"], p["KC"], p["VC"], 1, 1, 8, 2, 128, 64, 40, p["NP"], i32(p["table"]),
                                                                     i32(p["cu"]), i32(p["kv"]), 0.1, p["Q"].clone(), None)
    for bad in (dict(KC=p["KC"].transpose(1, 2)), dict(VC=p["VC"][:-1]), dict(Q=p["Q"][..., ::2])):
        with pytest.raises(osc.OscError) as e:
            attend(dict(p, **bad))
        assert e.value.status == 2


# ------------------------------------------------------------------ the step in a graph

def test_steps_in_a_graph():
    """Plan, cache write and attention captured once and replayed as a decode loop: lengths, list head and
    tables live on the device and move on between replays.  Checked against the whole history at once."""
    HQ, HKV, D, page, R, MB, T = 8, 2, 128, 16, 5, 8, 8
    NP = R * MB
    g = gen(11)
    free = torch.randperm(NP, generator=g, device=DEV).to(torch.int32)
    table = torch.full((R, MB), -1, dtype=torch.int32, device=DEV)
    ctx, new, head = i32([0] * R), i32([1] * R), i32([0])
    cu, kv, slot, pos, used = i32([0] * (R + 1)), i32([0] * R), i32([0] * T), i32([0] * T), i32([0])
    KC = torch.full((NP, HKV, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    VC = torch.full((NP, HKV, D, page), float("nan"), dtype=torch.bfloat16, device=DEV)
    qkv = torch.zeros((T, (HQ + 2 * HKV) * D), dtype=torch.bfloat16, device=DEV)
    Q, O = poisoned((T, HQ, D), torch.bfloat16), poisoned((T, HQ, D), torch.bfloat16)
    ws = torch.empty(osc.osc_attn_workspace(T, R, HQ, HKV, D, page, MB), dtype=torch.uint8, device=DEV)

    def step():
        osc.osc_page_plan(ctx, new, R, page, NP, free, NP, head, T, table, MB, cu, kv, slot, pos, used)
        osc.osc_qkv_append(qkv, T, HQ, HKV, D, None, None, 0.0, None, 0, None, slot, Q, KC, VC, NP, page)
        osc.osc_attn_paged(Q, KC, VC, T, R, HQ, HKV, D, page, MB, NP, table, cu, kv, D ** -0.5, O, ws)
        ctx.add_(new)
        head.add_(used)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    history = [[] for _ in range(R)]
    for it in range(40):
        counts = [1, 0 if it % 3 else 1, 2 if it % 7 == 0 else 1, 1, 0 if it < 20 else 3]
        new.copy_(i32(counts))
        rows = (torch.randn((T, (HQ + 2 * HKV) * D), generator=g, device=DEV)).bfloat16()
        qkv.copy_(rows)
        O.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        x = rows.reshape(T, -1, D)
        t = 0
        for r in range(R):
            history[r] += [x[t + i] for i in range(counts[r])]
            t += counts[r]
        assert bool((O[t:] == 7.0).all())
        if it % 8 == 7 or it == 39:
            t = 0
            for r in range(R):
                n = counts[r]
                for i in range(n):
                    seen = torch.stack(history[r][:len(history[r]) - n + i + 1]).double()
                    for hq in range(HQ):
                        h = hq // (HQ // HKV)
                        w = torch.softmax(seen[:, HQ + h] @ x[t + i, hq].double() * D ** -0.5, 0)
                        ref = w @ seen[:, HQ + HKV + h]
                        tol = (2.0 ** -8 + 2.0 ** -13) * (w @ seen[:, HQ + HKV + h].abs()) + 2.0 ** -8 * ref.abs()
                        assert bool(((O[t + i, hq].double() - ref).abs() <= tol).all()), (it, r, i, hq)
                t += n
    assert ctx.tolist() == [len(h) for h in history] and int(head) == sum(-(-len(h) // page) for h in history)
