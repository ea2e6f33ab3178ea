"""What the operators of a step with drafted tokens are measured on: the plan of the requests' token trees,
attention of the trees over the paged cache, log probabilities of the logits behind the last block, and the
acceptance of a path of each tree with the move of its keys and values.

Each case names an operator, its sizes, and the seed of its request lengths and trees.  ``run`` computes it in
elementary torch operations, or, where ``own`` is set, by the calls of w4a4_outlier_split_amd that a serving
step makes.  A tree's nodes come after their parents; a parent of -1 is the request's context.  The cache is
K [page][head][slot][D] and V [page][head][D][slot], of all layers in one tensor where a call takes all.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"


def listed():
    return [
        # trees of 16 nodes for a batch of 16 requests: latency
        dict(name="plan_r16_n16", op="plan", R=16, N=16, ragged=False, shape="wide", lens=1),
        # many requests whose trees differ, deep ones among them, in a padded step
        dict(name="plan_r512_n200", op="plan", R=512, N=200, ragged=True, shape="mixed", lens=2),
        # a single user's step: 16 drafted tokens over one long request, where latency counts
        dict(name="attn_r1_n16", op="attn", R=1, N=16, HQ=32, HKV=8, D=128, page=64, ragged=False, ctx_lo=4000, ctx_hi=4000, shape="wide", lens=3),
        # a batch of small trees at lengths that differ, small pages: the cache's bytes
        dict(name="attn_r32_n8", op="attn", R=32, N=8, HQ=32, HKV=8, D=128, page=16, ragged=True, ctx_lo=1, ctx_hi=8192, shape="mixed", lens=4),
        # the same with the trees of most drafting schemes, where bytes and products weigh alike
        dict(name="attn_r32_n64", op="attn", R=32, N=64, HQ=32, HKV=8, D=128, page=64, ragged=True, ctx_lo=1, ctx_hi=8192, shape="mixed", lens=5),
        # the largest tree over one long request
        dict(name="attn_r1_n256", op="attn", R=1, N=256, HQ=32, HKV=8, D=128, page=64, ragged=False, ctx_lo=32700, ctx_hi=32700, shape="mixed", lens=6),
        # one row of logits, as a single user's decode has
        dict(name="lp_s1", op="lp", S=1, V=151936, pad=0, dt="bf16", K=20, M=1, scale=1.0),
        # the nodes of 32 trees of 16: each node's most likely tokens, and the log probability of its children
        dict(name="lp_s512", op="lp", S=512, V=151936, pad=0, dt="bf16", K=8, M=4, scale=1.0),
        # a prompt's tokens scored, with the alternatives that an interface shows
        dict(name="lp_s2048", op="lp", S=2048, V=151936, pad=0, dt="bf16", K=5, M=1, scale=1.0),
        # an odd vocabulary in rows padded behind it, 32-bit logits at a temperature, many alternatives to draw from
        dict(name="lp_s48_f32", op="lp", S=48, V=100003, pad=29, dt="f32", K=50, M=3, scale=1.0 / 0.7),
        # a single user's tree: a path taken, its keys and values moved in all layers
        dict(name="accept_r1_n16", op="accept", R=1, N=16, layers=36, HKV=8, D=128, page=64, ragged=False, shape="wide", rate=0.9, lens=7),
        # a batch's
        dict(name="accept_r32_n64", op="accept", R=32, N=64, layers=36, HKV=8, D=128, page=64, ragged=True, shape="mixed", rate=0.8, lens=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "attn", "attn", "attn", "lp", "lp", "lp", "accept"])
    lens = rng.randrange(1 << 20)
    shape = rng.choice(["chain", "wide", "mixed", "roots"])
    if op == "plan":
        return dict(op=op, R=_log(rng, 1, 512), N=_log(rng, 1, 200), ragged=rng.random() < 0.7, shape=shape, lens=lens)
    HQ, HKV = rng.choice([(32, 8), (32, 8), (16, 8), (8, 8), (32, 4), (24, 8), (8, 1), (5, 1)])
    D = rng.choice([128, 128, 64])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "attn":
        # queries x keys is kept under that of the largest listed case, requests x keys too
        N, ctx = _log(rng, 1, 256), _log(rng, 16, 32768)
        R = max(1, min(_log(rng, 1, 64), 128000 // ctx, 8_000_000 // (N * (ctx + N))))
        return dict(op=op, R=R, N=N, HQ=HQ, HKV=HKV, D=D, page=page, ragged=rng.random() < 0.7, ctx_lo=ctx // 3, ctx_hi=ctx, shape=shape, lens=lens)
    if op == "lp":
        V = _log(rng, 1000, 160000)
        dt = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, S=_log(rng, 1, min(8192, (300_000_000 if dt == "bf16" else 150_000_000) // V)), V=V, pad=rng.choice([0, 0, 1, 24, 100]),
                    dt=dt, K=rng.choice([0, 1, 5, 20, 64]), M=rng.choice([1, 1, 4, 8]), scale=rng.choice([1.0, 1.0, 1.25, 0.5]))
    N = _log(rng, 1, 200)
    return dict(op=op, R=max(1, min(_log(rng, 1, 128), 2000 // N)), N=N, layers=rng.choice([1, 12, 36]), HKV=rng.choice([1, 2, 4, 8]), D=D, page=page,
                ragged=rng.random() < 0.7, shape=shape, rate=rng.choice([0.5, 0.8, 1.0]), lens=lens)


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The case's requests: tokens in the cache before the step, and nodes of their trees."""
    r = random.Random(c["lens"])
    lo, hi = c.get("ctx_lo", 0), c.get("ctx_hi", 3000)
    ctx = [r.randint(lo, hi) for _ in range(c["R"])]
    if not c["ragged"]:
        return ctx, [c["N"]] * c["R"]
    new = [r.choice([0, 1, c["N"]]) if r.random() < 0.3 else r.randint(max(1, c["N"] // 2), c["N"]) for _ in range(c["R"])]
    new[-1] = c["N"]
    return ctx, new


def _parents(c, new):
    """Parents of all nodes in turn, numbered inside their request."""
    r = random.Random(c["lens"] + 1)
    out = []
    for n in new:
        kind = c["shape"] if c["shape"] != "mixed" else r.choice(["chain", "wide", "any", "any"])
        for i in range(n):
            if i == 0 or (kind == "roots" and r.random() < 0.2):
                out.append(-1)
            elif kind == "chain":
                out.append(i - 1)
            elif kind == "wide":
                out.append((i - 1) // 3)  # three drafted tokens behind each node
            else:
                out.append(r.randrange(max(0, i - 6), i))
    return out


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _up(a, b):
    return -(-a // b)


def _sums(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    g = _gen(seed)
    return {"plan": _prepare_plan, "attn": _prepare_attn, "lp": _prepare_lp, "accept": _prepare_accept}[case["op"]](case, g, seed)


def _prepare_plan(c, g, seed):
    ctx, new = _lengths(c)
    up = random.Random(seed).randrange(1000)  # the requests are further on
    T = sum(new) + (sum(new) % 5)  # a step padded behind its last node
    W = _up(c["N"], 64)
    parent = _parents(c, new) + [0] * (T - sum(new))
    return dict(c=c, T=T, W=W, ctx=_i32([v + up for v in ctx]), cu=_i32(_sums(new)), parent=_i32(parent), pos=torch.zeros(T, dtype=torch.int32, device=DEV),
                mask=torch.zeros(T, W, dtype=torch.int64, device=DEV))


def _bits(c, new, W):
    """int64 [sum(new), W]: each node's ancestors and itself."""
    parent, rows, at = _parents(c, new), [], 0
    for n in new:
        seen = []
        for i in range(n):
            p = parent[at + i]
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        rows += seen
        at += n
    words = [[(v >> 64 * w) & (2 ** 64 - 1) for w in range(W)] for v in rows]
    return torch.tensor([[x - 2 ** 64 if x >> 63 else x for x in row] for row in words], dtype=torch.int64, device=DEV).reshape(len(rows), W)


def _prepare_attn(c, g, seed):
    ctx, new = _lengths(c)
    HQ, HKV, D, page = c["HQ"], c["HKV"], c["D"], c["page"]
    total = [a + b for a, b in zip(ctx, new)]
    S, MB, NP, W = sum(new), max(1, _up(max(total), page)) + 1, sum(_up(t, page) for t in total) + 3, _up(c["N"], 64)
    pool = torch.randperm(NP, generator=g, device=DEV).to(torch.int32)
    need = torch.tensor([_up(t, page) for t in total], device=DEV)
    at = torch.arange(MB, device=DEV)
    table = torch.where(at[None, :] < need[:, None], pool[((need.cumsum(0) - need)[:, None] + at[None, :]).clamp(max=NP - 1)], -1)
    return dict(c=c, S=S, W=W, q=_randn(g, S, HQ, D) * 1.5, kc=_randn(g, NP, HKV, page, D), vc=_randn(g, NP, HKV, D, page),
                table=table.to(torch.int32).contiguous(), MB=MB, NP=NP, cu=_i32(_sums(new)), kv=_i32(total), mask=_bits(c, new, W), most_new=max(new),
                most_kv=max(total), scale=D ** -0.5, o=torch.zeros(S, HQ, D, dtype=torch.bfloat16, device=DEV))


def _prepare_lp(c, g, seed):
    S, V, ld, K, M = c["S"], c["V"], c["V"] + c["pad"], c["K"], c["M"]
    # a spread of unlikely tokens, a few dozen likely ones, and rows that are sure of one
    x = torch.randn((S, ld), generator=g, device=DEV, dtype=torch.bfloat16) * 2
    likely = torch.randint(0, V, (S, 24), generator=g, device=DEV)
    lift = torch.rand((S, 24), generator=g, device=DEV) * 6 + 6 + 4 * torch.rand((S, 1), generator=g, device=DEV)
    lift[:, 0] += 12 * (torch.rand(S, generator=g, device=DEV) < 0.2)
    x.scatter_(1, likely, lift.to(torch.bfloat16))
    if c["dt"] == "f32":
        x = x.float() + torch.rand((S, ld), generator=g, device=DEV) * 2.0 ** -8
    ids = torch.where(torch.rand((S, M), generator=g, device=DEV) < 0.7, likely[:, :M], torch.randint(0, V, (S, M), generator=g, device=DEV))
    f32 = dict(dtype=torch.float32, device=DEV)
    return dict(c=c, x=x, ld=ld, ids=ids.to(torch.int32), lp=torch.zeros(S, M, **f32), ent=torch.zeros(S, **f32), topv=torch.zeros(S, K, **f32) if K else None,
                topi=torch.zeros(S, K, dtype=torch.int32, device=DEV) if K else None)


def _prepare_accept(c, g, seed):
    ctx, new = _lengths(c)
    R, N, L, HKV, D, page = c["R"], c["N"], c["layers"], c["HKV"], c["D"], c["page"]
    T, cu, parent = sum(new), _sums(new), _parents(c, new)
    # the model's choice at a node is one of its children's tokens as often as drafts are good
    r = random.Random(c["lens"] + 2)
    token, choice, at = [], [], 0
    for n in new:
        drafted = [r.randrange(150000) for _ in range(n)]
        for i in range(n):
            children = [j for j in range(i + 1, n) if parent[at + j] == i]
            choice.append(drafted[r.choice(children)] if children and r.random() < c["rate"] else r.randrange(150000))
        token += drafted
        at += n
    # the pages of the last tokens are all that the call touches: two and more for each request
    NP = sum(_up(n + page, page) for n in new) + 3
    pool, slot, used = torch.randperm(NP, generator=g, device=DEV).tolist(), [], 0
    for a, n in zip(ctx, new):
        slot += [pool[used + (a % page + i) // page] * page + (a + i) % page for i in range(n)]
        used += _up(n + page, page)
    pos = [ctx[i] + j for i, n in enumerate(new) for j in range(n)]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(c=c, T=T, NP=NP, token=_i32(token), parent=_i32(parent), choice=_i32(choice), slot=_i32(slot), pos=_i32(pos), cu=_i32(cu), spare=pool[-1] * page,
                kc=_randn(g, L, NP, HKV, page, D), vc=_randn(g, L, NP, HKV, D, page), acc=torch.zeros(R, **i32), path=torch.zeros(R, N, **i32),
                next=torch.zeros(R, **i32))


# ------------------------------------------------------------------ the operators in their plain form

def run(state):
    op = state["c"]["op"]
    if own:
        return {"plan": _own_plan, "attn": _own_attn, "lp": _own_lp, "accept": _own_accept}[op](state)
    return {"plan": _plan, "attn": _attn, "lp": _lp, "accept": _accept}[op](state)


def _nodes(s):
    """[R, N]: the row of each node and whether there is one, its parent (-1: the context), and [R, N, N] its ancestors and itself."""
    c = s["c"]
    N, T = c["N"], s["T"]
    cu = s["cu"].long()
    i = torch.arange(N, device=cu.device)
    row = cu[:-1, None] + i[None, :]
    there = row < cu[1:, None]
    p = s["parent"].long()[row.clamp(max=T - 1)]
    p = torch.where(there & (p >= 0) & (p < i[None, :]), p, -1)
    up = (p[:, :, None] == i[None, None, :]).float() + torch.eye(N, device=cu.device)
    for _ in range((N - 1).bit_length()):  # ancestors 2, 4, 8 ... steps away
        up = torch.bmm(up, up).clamp(max=1.0)
    return row, there, p, up > 0


def _plan(s):
    T, W = s["T"], s["W"]
    row, there, _, up = _nodes(s)
    pos = s["ctx"].long()[:, None] + up.sum(2) - 1
    bits = torch.nn.functional.pad(up.long(), (0, 64 * W - up.shape[2])).reshape(*up.shape[:2], W, 64)
    words = (bits << torch.arange(64, device=bits.device)).sum(3)
    at = torch.where(there, row, T).reshape(-1)  # rows that are none go behind the last
    out = torch.full((T + 1,), -1, dtype=torch.int32, device=at.device).scatter_(0, at, pos.to(torch.int32).reshape(-1))
    mask = torch.zeros(T + 1, W, dtype=torch.int64, device=at.device)
    mask[at] = words.reshape(-1, W)
    return dict(pos=out[:T], mask=mask[:T])


def _attn(s):
    c = s["c"]
    S, R, HQ, HKV, D, page = s["S"], c["R"], c["HQ"], c["HKV"], c["D"], c["page"]
    g, N, nb = HQ // HKV, s["most_new"], _up(s["most_kv"], page)
    at = s["table"][:, :nb].clamp(min=0).long()
    k = s["kc"][at].permute(0, 2, 1, 3, 4).reshape(R, HKV, nb * page, D).float()
    v = s["vc"][at].permute(0, 2, 1, 4, 3).reshape(R, HKV, nb * page, D).float()
    cu, kv = s["cu"].long(), s["kv"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(N, device=k.device)
    row = (cu[:-1, None] + i[None, :]).clamp(max=S - 1)  # rows behind a request's last are not used
    q = s["q"][row].float()
    q = q.reshape(R, N, HKV, g, D).permute(0, 2, 1, 3, 4).reshape(R, HKV, N * g, D) * s["scale"]
    w = torch.matmul(q, k.transpose(2, 3).contiguous()).reshape(R, HKV, N, g, nb * page)
    key = torch.arange(nb * page, device=k.device)[None, :] - (kv - n)[:, None]  # < 0: the context, else a node
    bit = key.clamp(0, 64 * s["W"] - 1)
    word = torch.gather(s["mask"][row], 2, (bit // 64)[:, None, :].expand(-1, N, -1))
    seen = ((word >> (bit % 64)[:, None, :]) & 1).bool() & (key < n[:, None])[:, None, :] | (key < 0)[:, None, :]
    w.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    w.sub_(w.amax(4, keepdim=True)).exp_()
    total = w.sum(4, keepdim=True)
    o = torch.matmul(w.reshape(R, HKV, N * g, nb * page), v).reshape(R, HKV, N, g, D) / total
    t = torch.arange(S, device=k.device)
    r = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=R - 1)
    return o.permute(0, 2, 1, 3, 4)[r, t - cu[r]].reshape(S, HQ, D).to(torch.bfloat16)


def _lp(s):
    c = s["c"]
    V, K = c["V"], c["K"]
    x = s["x"][:, :V].float()
    y = x * c["scale"]
    most = y.amax(1, keepdim=True)
    d = y - most
    e = d.exp()
    total = e.sum(1, keepdim=True)
    ent = total.log() - (e * d).sum(1, keepdim=True) / total
    lse = total.log()
    lp = torch.gather(d, 1, s["ids"].long()) - lse
    topv = topi = None
    if K:
        bits = (x + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7fffffff)).long() << 32  # whole numbers in the order of the values,
        order += 0xffffffff - torch.arange(V, device=x.device)     # and the lower index first
        pick = 0xffffffff - (torch.topk(order, K, dim=1).values & 0xffffffff)
        topv, topi = torch.gather(d, 1, pick) - lse, pick.to(torch.int32)
    return dict(lp=lp, ent=ent[:, 0], topv=topv, topi=topi)


def _accept(s):
    c = s["c"]
    R, N, T, page = c["R"], c["N"], s["T"], c["page"]
    row, there, p, up = _nodes(s)
    row = row.clamp(max=T - 1)
    i = torch.arange(N, device=row.device)
    token, choice, slot = s["token"].long()[row], s["choice"].long()[row], s["slot"].long()[row]
    hit = there & (p >= 0) & (torch.gather(choice, 1, p.clamp(min=0)) == token)
    # of siblings with the chosen token the first
    twin = (p[:, :, None] == p[:, None, :]) & hit[:, None, :] & (i[None, None, :] < i[None, :, None])
    hit = (hit & ~twin.any(2)) | (there & (i == 0)[None, :])
    taken = there & ~(up & ~hit[:, None, :]).any(2) & up[:, :, 0]
    acc = taken.sum(1)
    place = torch.where(taken, taken.cumsum(1) - 1, N)
    path = torch.full((R, N + 1), -1, dtype=torch.int64, device=row.device).scatter_(1, place, i.expand(R, N).contiguous())[:, :N]
    last = torch.gather(path, 1, (acc - 1).clamp(min=0)[:, None]).clamp(min=0)
    after = torch.where(acc > 0, torch.gather(choice, 1, last)[:, 0], -1)
    move = path > i[None, :]
    frm = torch.where(move, torch.gather(slot, 1, path.clamp(min=0)), s["spare"]).reshape(-1)
    to = torch.where(move, slot, s["spare"]).reshape(-1)
    s["kc"][:, to // page, :, to % page] = s["kc"][:, frm // page, :, frm % page]
    s["vc"][:, to // page, :, :, to % page] = s["vc"][:, frm // page, :, :, frm % page]
    i32 = torch.int32
    return dict(acc=acc.to(i32), path=path.to(i32), next=after.to(i32), kc=s["kc"], vc=s["vc"])


# ------------------------------------------------------------------ the framework's calls

def _own_plan(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    osc.osc_tree_plan(s["parent"], s["cu"], s["ctx"], c["R"], s["T"], c["N"], s["pos"], s["mask"])
    return dict(pos=s["pos"], mask=s["mask"])


def _own_attn(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    sizes = (s["S"], c["R"], c["HQ"], c["HKV"], c["D"], c["page"], s["MB"])
    if "ws" not in s:  # the step's workspace, kept with its buffers
        s["ws"] = torch.empty(osc.osc_attn_tree_workspace(*sizes, c["N"]), dtype=torch.uint8, device=DEV)
    osc.osc_attn_tree(s["q"], s["kc"], s["vc"], *sizes, s["NP"], s["table"], s["cu"], s["kv"], s["mask"], c["N"], s["scale"], s["o"], s["ws"])
    return s["o"]


def _own_lp(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    if "ws" not in s:
        s["ws"] = torch.empty(osc.osc_logprobs_workspace(c["S"], c["V"], c["K"]), dtype=torch.uint8, device=DEV)
    osc.osc_logprobs(s["x"], osc.OSC_Y_BF16 if c["dt"] == "bf16" else osc.OSC_Y_F32, c["S"], c["V"], s["ld"], c["scale"], s["ids"], c["M"], c["K"], s["lp"],
                     s["ent"], s["topv"], s["topi"], s["ws"])
    return dict(lp=s["lp"], ent=s["ent"], topv=s["topv"], topi=s["topi"])


def _own_accept(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    R, N, T, HKV, D, page = c["R"], c["N"], s["T"], c["HKV"], c["D"], c["page"]
    if "caches" not in s:  # the layers' caches, checked once and kept as the model's are
        s["caches"] = osc.LayerCaches(list(s["kc"]), list(s["vc"]), s["NP"], HKV, D, page)
    osc.osc_tree_accept(s["token"], s["parent"], s["choice"], 1, s["slot"], s["pos"], 0, s["cu"], R, T, N, s["acc"], s["path"], s["next"])
    osc.osc_tree_commit(s["caches"], s["slot"], s["cu"], s["acc"], s["path"], R, T, N)
    return dict(acc=s["acc"], path=s["path"], next=s["next"], kc=s["kc"], vc=s["vc"])


# ------------------------------------------------------------------ work and exact values

def _moved(c, new):
    """Nodes that a path of the usual length moves: about two levels of each tree in every three."""
    return sum(min(n, 3) for n in new) - sum(1 for n in new if n)


def work(case):
    c = case
    if c["op"] == "lp":
        size = 2 if c["dt"] == "bf16" else 4
        return dict(bytes=c["S"] * (c["V"] * size + 8 * c["M"] + 8 * c["K"] + 4), flops=4 * c["S"] * c["V"])
    ctx, new = _lengths(c)
    if c["op"] == "plan":
        return dict(bytes=8 * c["R"] + sum(new) * (8 + 8 * _up(c["N"], 64)), flops=0)
    if c["op"] == "accept":
        return dict(bytes=20 * sum(new) + 8 * c["R"] + 8 * _moved(c, new) * c["layers"] * c["HKV"] * c["D"], flops=0)
    HQ, HKV, D = c["HQ"], c["HKV"], c["D"]
    seen, parent, at = 0, _parents(c, new), 0
    for a, n in zip(ctx, new):
        depth = []
        for i in range(n):
            depth.append(1 + (depth[parent[at + i]] if parent[at + i] >= 0 else 0))
        at += n
        seen += n * a + sum(depth)
    keys = sum(a + n for a, n in zip(ctx, new) if n)
    return dict(bytes=4 * keys * HKV * D + 4 * sum(new) * HQ * D, flops=4 * HQ * D * seen)


def exact(case, seed):
    if case["op"] in ("plan", "accept"):  # whole numbers, and values that are copied
        return None
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_lp(s)


def _exact_attn(s):
    c = s["c"]
    HQ, HKV, D, page = c["HQ"], c["HKV"], c["D"], c["page"]
    g = HQ // HKV
    out = torch.empty(s["S"], HQ, D, dtype=torch.float64, device=DEV)
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    _, new = _lengths(c)
    parent = _parents(c, new)
    for r, total in enumerate(kv):
        a, n = cu[r], cu[r + 1] - cu[r]
        if not n:
            continue
        hidden = torch.zeros(n, total, dtype=torch.bool)
        hidden[:, total - n:] = True
        for i in range(n):
            j = i
            while j >= 0:  # from the node up to the context
                hidden[i, total - n + j] = False
                j = parent[a + j]
        hidden = hidden.to(DEV)
        pages = s["table"][r, :_up(total, page)].long()
        for h in range(HKV):
            k = s["kc"][pages, h].reshape(-1, D)[:total].double()
            v = s["vc"][pages, h].permute(1, 0, 2).reshape(D, -1)[:, :total].double()
            for j in range(h * g, (h + 1) * g):
                p = torch.softmax((s["q"][a:a + n, j].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf), 1)
                out[a:a + n, j] = p @ v.T
    return out


def _exact_lp(s):
    c = s["c"]
    got = dict(lp=[], ent=[], topv=[])
    step = max(1, 60_000_000 // c["V"])
    for a in range(0, c["S"], step):
        y = torch.log_softmax(s["x"][a:a + step, :c["V"]].double() * c["scale"], 1)
        got["lp"].append(torch.gather(y, 1, s["ids"][a:a + step].long()))
        got["ent"].append(-(y * y.exp()).sum(1))
        if c["K"]:
            got["topv"].append(torch.topk(y, c["K"], dim=1).values)
    return dict(lp=torch.cat(got["lp"]), ent=torch.cat(got["ent"]), topv=torch.cat(got["topv"]) if c["K"] else None, topi=None)
