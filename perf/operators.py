"""What the block-step operators are measured on: add + RMS norm + quantization, the page plan, the
per-head norm / rotary / cache write, and attention of new tokens over the paged cache.

Each case names an operator, its sizes, and the seed of its request lengths.  ``run`` computes it in
elementary torch operations, or, where ``own`` is set, by the calls of w4a4_outlier_split_amd that a
serving step makes.  Both give the outputs in the library's own layouts: quantized rows in panels of
128 channels (E4M3 elements as they are, E2M1 elements as the values they stand for, E8M0 scales in
panels of 4 groups, 8 for groups of 16), the cache as K [page][head][slot][D] and V [page][head][D][slot].
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


def listed():
    return [
        # one decode step of 16 requests: the norm ahead of the QKV projection, on the 4-bit path
        # with the table's channel split off; a call whose latency is what counts
        dict(name="norm_s16_fp4", op="norm", S=16, H=4096, G=32, fmt="mxfp4", m=1),
        # a prefill batch ahead of a projection on the 8-bit path
        dict(name="norm_s4096_fp8", op="norm", S=4096, H=4096, G=32, fmt="mxfp8", m=0),
        # a ragged prefill batch of wide rows at the largest group size
        dict(name="norm_s1537_h8192_fp8", op="norm", S=1537, H=8192, G=64, fmt="mxfp8", m=0),
        # one decode step of 64 requests: a token each, some at a page's first slot
        dict(name="plan_r64_decode", op="plan", R=64, page=16, new=1, ragged=False, ctx_lo=1, ctx_hi=8192, lens=1),
        # a large step of decodes and prompt chunks together
        dict(name="plan_r512_mixed", op="plan", R=512, page=64, new=96, ragged=True, ctx_lo=0, ctx_hi=8192, lens=2),
        # a decode step's query and key heads, rotated, keys and values written to the cache
        dict(name="append_s16", op="append", S=16, HQ=32, HKV=8, D=128, page=64, norm=True, rope=True),
        # a prefill batch's, with an odd number of tokens
        dict(name="append_s4097", op="append", S=4097, HQ=32, HKV=8, D=128, page=64, norm=True, rope=True),
        # a single user's decode step: one token over one long request
        dict(name="attn_r1_decode", op="attn", R=1, HQ=32, HKV=8, D=128, page=64, new=1, ragged=False, ctx_lo=4000, ctx_hi=4000, lens=3),
        # a batch of decodes at lengths that differ, small pages
        dict(name="attn_r64_decode", op="attn", R=64, HQ=32, HKV=8, D=128, page=16, new=1, ragged=False, ctx_lo=1, ctx_hi=8192, lens=4),
        # a short chunk at the end of a long request
        dict(name="attn_r1_chunk33", op="attn", R=1, HQ=32, HKV=8, D=128, page=64, new=33, ragged=False, ctx_lo=32700, ctx_hi=32700, lens=5),
        # four chunks of uneven lengths over caches of uneven lengths
        dict(name="attn_r4_chunks", op="attn", R=4, HQ=32, HKV=8, D=128, page=32, new=1024, ragged=True, ctx_lo=0, ctx_hi=8192, lens=6),
        # a whole prompt
        dict(name="attn_r1_s8192", op="attn", R=1, HQ=32, HKV=8, D=128, page=64, new=8192, ragged=False, ctx_lo=0, ctx_hi=0, lens=7),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "plan", "append", "append", "attn", "attn", "attn", "attn"])
    lens = rng.randrange(1 << 20)
    if op == "norm":
        fmt = rng.choice(["mxfp8", "mxfp8", "mxfp4"])
        G = rng.choice([16, 32, 64]) if fmt == "mxfp4" else rng.choice([32, 64])
        return dict(op=op, S=_log(rng, 1, 8192), H=256 * rng.randrange(2, 33), G=G, fmt=fmt,
                    m=rng.choice([0, 1, 2]) if fmt == "mxfp4" else 0)
    if op == "plan":
        return dict(op=op, R=_log(rng, 1, 1024), page=rng.choice([16, 32, 64, 128, 256]), new=rng.choice([1, 7, 64, 200]),
                    ragged=True, ctx_lo=0, ctx_hi=_log(rng, 1, 16384), lens=lens)
    HQ, HKV = rng.choice([(32, 8), (32, 8), (16, 8), (8, 8), (32, 4), (24, 8), (8, 1), (5, 1)])
    D = rng.choice([128, 128, 64])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        return dict(op=op, S=_log(rng, 1, 8192), HQ=HQ, HKV=HKV, D=D, page=page, norm=rng.random() < 0.7, rope=True)
    # queries x keys is kept under that of the largest listed case, requests x keys under that of the largest batch
    kind = rng.choice(["decode", "chunk", "chunk", "prompt"])
    if kind == "decode":
        R, ctx = _log(rng, 1, 128), _log(rng, 16, 32768)
        return dict(op=op, R=min(R, max(1, 300000 // ctx)), HQ=HQ, HKV=HKV, D=D, page=page, new=1, ragged=False, ctx_lo=ctx // 3,
                    ctx_hi=ctx, lens=lens)
    if kind == "chunk":
        new, ctx = _log(rng, 2, 1024), _log(rng, 16, 16384)
        return dict(op=op, R=max(1, min(rng.randrange(1, 17), 30_000_000 // (new * (ctx + new)))), HQ=HQ, HKV=HKV, D=D, page=page,
                    new=new, ragged=rng.random() < 0.7, ctx_lo=0, ctx_hi=ctx, lens=lens)
    return dict(op=op, R=1, HQ=HQ, HKV=HKV, D=D, page=page, new=_log(rng, 100, 6000), ragged=False, ctx_lo=0, ctx_hi=0, lens=lens)


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The case's requests: tokens in the cache before the step, and new ones."""
    r = random.Random(c["lens"])
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["R"])]
    if not c["ragged"]:
        return ctx, [c["new"]] * c["R"]
    new = [r.choice([0, 1, c["new"]]) if r.random() < 0.4 else r.randint(1, c["new"]) for _ in range(c["R"])]
    if not any(new):
        new[0] = 1
    return ctx, new


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _up(a, b):
    return -(-a // b)


def _pages(c, g):
    """Page tables over a shuffled pool: the entries of the tokens in the cache, or of all of them."""
    ctx, new = _lengths(c)
    page = c["page"]
    total = [a + b for a, b in zip(ctx, new)]
    MB = max(1, _up(max(total), page)) + 1
    NP = sum(_up(t, page) for t in total) + 3
    pool = torch.randperm(NP, generator=g, device=DEV).to(torch.int32)
    return ctx, new, total, MB, NP, pool


def _fill(lens, page, MB, pool):
    """int32 [R, MB]: each request's pages in turn from the pool, -1 behind them; and the pages taken."""
    need = torch.tensor([_up(t, page) for t in lens], device=DEV)
    start = need.cumsum(0) - need
    at = torch.arange(MB, device=DEV)
    table = pool[(start[:, None] + at[None, :]).clamp(max=pool.numel() - 1)]
    return torch.where(at[None, :] < need[:, None], table, -1).to(torch.int32).contiguous(), int(sum(_up(t, page) for t in lens))


def prepare(case, seed):
    g = _gen(seed)
    return {"norm": _prepare_norm, "plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn}[case["op"]](case, g, seed)


def _prepare_norm(c, g, seed):
    S, H, G, m = c["S"], c["H"], c["G"], c["m"]
    K = H // G
    # a residual stream with persistent large channels in most groups, as the table indexes them
    host = random.Random(seed)
    off = [[-1] * max(m, 1) for _ in range(K)]
    gain = torch.ones(H)
    for k in range(K):
        for e in range(max(m, 1)):
            if host.random() < 0.7:
                o = host.randrange(G)
                if o not in off[k]:
                    off[k][e] = o
                    gain[k * G + o] = host.uniform(20.0, 60.0)
    gain = gain.to(DEV).to(torch.bfloat16)
    w = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    fp4 = c["fmt"] == "mxfp4"
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV).to(torch.bfloat16)
    both = torch.stack([values.repeat(16), values.repeat_interleave(16)], 1).contiguous()  # byte -> its low and its high code's value
    byte = dict(dtype=torch.uint8, device=DEV)
    return dict(c=c, x=_randn(g, S, H), res=_randn(g, S, H) * gain, w=w, res_out=torch.zeros(S, H, dtype=torch.bfloat16, device=DEV),
                L=np.asarray(off, np.int32) if m else None, Ld=torch.tensor(off, device=DEV),
                Q=torch.zeros(S * H // 2 if fp4 else S * H, **byte), SC=torch.zeros(S * K, **byte),
                B=torch.zeros(_up(m * K, 32), S, 32, dtype=torch.bfloat16, device=DEV) if m else None,
                pair=both.view(torch.int32).reshape(-1))


def _prepare_plan(c, g, seed):
    ctx, new, total, MB, NP, pool = _pages(c, g)
    R, page = c["R"], c["page"]
    table, used = _fill(ctx, page, MB, pool)
    T = sum(new) + (sum(new) % 5)  # a step padded behind its last token
    return dict(c=c, ctx=_i32(ctx), new=_i32(new), table=table, free=pool, head=_i32([used]), T=T, MB=MB, NP=NP, cu=_i32([0] * (R + 1)),
                kv=_i32([0] * R), slot=torch.zeros(T, dtype=torch.int32, device=DEV), pos=torch.zeros(T, dtype=torch.int32, device=DEV),
                used=_i32([0]))


def _prepare_append(c, g, seed):
    S, HQ, HKV, D, page = c["S"], c["HQ"], c["HKV"], c["D"], c["page"]
    # tokens of a few requests: runs of consecutive slots inside pages of a shuffled pool
    host = random.Random(seed)
    P = 8192
    base = host.randrange(0, P - (S if S < P else P - 1))
    pos = (base + torch.arange(S, device=DEV)) % P
    NP = _up(S + page, page) + 2
    pool = torch.randperm(NP, generator=g, device=DEV)
    first = host.randrange(page)
    at = first + torch.arange(S, device=DEV)
    slot = pool[at // page] * page + at % page
    angle = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * torch.pow(
        torch.tensor(1e6, dtype=torch.float64, device=DEV), -torch.arange(D // 2, device=DEV, dtype=torch.float64) * 2 / D)[None, :]
    wq = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    wk = (1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    empty = dict(dtype=torch.bfloat16, device=DEV)
    return dict(c=c, qkv=_randn(g, S, (HQ + 2 * HKV) * D) * 2, wq=wq if c["norm"] else None, wk=wk if c["norm"] else None,
                cs=torch.cat([angle.cos(), angle.sin()], 1).float() if c["rope"] else None, P=P, pos=pos.to(torch.int32),
                slot=slot.to(torch.int32), NP=NP, q=torch.zeros(S, HQ, D, **empty), kc=torch.zeros(NP, HKV, page, D, **empty),
                vc=torch.zeros(NP, HKV, D, page, **empty))


def _prepare_attn(c, g, seed):
    ctx, new, total, MB, NP, pool = _pages(c, g)
    HQ, HKV, D, page = c["HQ"], c["HKV"], c["D"], c["page"]
    S = sum(new)
    table, _ = _fill(total, page, MB, pool)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(c=c, S=S, q=_randn(g, S, HQ, D) * 1.5, kc=_randn(g, NP, HKV, page, D), vc=_randn(g, NP, HKV, D, page), table=table, MB=MB,
                NP=NP, cu=_i32(cu), kv=_i32(total), most_new=max(new), most_kv=max(total), scale=D ** -0.5,
                o=torch.zeros(S, HQ, D, dtype=torch.bfloat16, device=DEV))


# ------------------------------------------------------------------ the operators in their plain form

def run(state):
    op = state["c"]["op"]
    if own:
        return {"norm": _own_norm, "plan": _own_plan, "append": _own_append, "attn": _own_attn}[op](state)
    return {"norm": _norm, "plan": _plan, "append": _append, "attn": _attn}[op](state)


def _panels(t, width):
    """[S, C] -> [C / width, S, width], the tiled operand layout."""
    return t.reshape(t.shape[0], -1, width).transpose(0, 1).contiguous()


def _norm(s):
    c = s["c"]
    S, H, G, m = c["S"], c["H"], c["G"], c["m"]
    r = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    # the quantization that follows steps at its borders: the norm is taken in 64 bits
    rd = r.double()
    y = (rd / torch.sqrt((rd * rd).mean(1, keepdim=True) + EPS) * s["w"].double()).to(torch.bfloat16).float().reshape(S, H // G, G)
    B = None
    if m:
        at = s["Ld"][None].expand(S, -1, -1)
        side = torch.where(at >= 0, torch.gather(y, 2, at.clamp(min=0)), 0.0)
        y = y * (torch.arange(G, device=y.device)[:, None] != s["Ld"][:, None, :]).all(2)[None]
        side = torch.nn.functional.pad(side.reshape(S, -1), (0, -(H // G * m) % 32))
        B = _panels(side.to(torch.bfloat16), 32)
    amax = y.abs().amax(2, keepdim=True)
    top = 2 if c["fmt"] == "mxfp4" else 8
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - top, -127).clamp(-127, 127)
    v = torch.ldexp(y, -e)
    if c["fmt"] == "mxfp4":
        a = v.abs()
        step = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).long()
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=v.device)
        codes = torch.copysign(grid[step], v).to(torch.bfloat16)
    else:
        codes = v.clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (e + 127).to(torch.uint8).reshape(S, -1)
    return dict(res=r, codes=_panels(codes.reshape(S, H), 128), scales=_panels(scales, 8 if G == 16 else 4).view(torch.float8_e8m0fnu), side=B)


def _plan(s):
    c = s["c"]
    R, page, T, MB, NP = c["R"], c["page"], s["T"], s["MB"], s["NP"]
    ctx, new = s["ctx"].long(), s["new"].long()
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    start = s["head"].long() + (want - have).cumsum(0) - (want - have)
    at = torch.arange(MB, device=ctx.device)[None, :]
    fresh = (at >= have[:, None]) & (at < want[:, None])
    pick = (start[:, None] + at - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    t = torch.arange(T, device=ctx.device)
    r = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=R - 1)
    real = t < cu[-1]
    pos = torch.where(real, ctx[r] + t - cu[r], -1)
    slot = torch.where(real, table[r, pos.clamp(min=0) // page].long() * page + pos % page, -1)
    i32 = torch.int32
    return dict(cu=cu.to(i32), kv=(ctx + new).to(i32), table=table, slot=slot.to(i32), pos=pos.to(i32),
                used=(want - have).sum(0, keepdim=True).to(i32))


def _append(s):
    c = s["c"]
    S, HQ, HKV, D, page = c["S"], c["HQ"], c["HKV"], c["D"], c["page"]
    x = s["qkv"].float().reshape(S, HQ + 2 * HKV, D)
    qk = x[:, :HQ + HKV]
    if c["norm"]:
        w = torch.cat([s["wq"].float().expand(HQ, D), s["wk"].float().expand(HKV, D)])
        qk = qk * torch.rsqrt((qk * qk).mean(2, keepdim=True) + EPS) * w
    if c["rope"]:
        cs = s["cs"][s["pos"].long()][:, None, :]
        cos, sin = cs[..., :D // 2], cs[..., D // 2:]
        a, b = qk[..., :D // 2], qk[..., D // 2:]
        qk = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    qk = qk.to(torch.bfloat16)
    s["q"].copy_(qk[:, :HQ])
    slot = s["slot"].long()
    s["kc"][slot // page, :, slot % page] = qk[:, HQ:]
    s["vc"][slot // page, :, :, slot % page] = x[:, HQ + HKV:].to(torch.bfloat16)
    return dict(q=s["q"], kc=s["kc"], vc=s["vc"])


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
    q = s["q"][(cu[:-1, None] + i[None, :]).clamp(max=S - 1)].float()  # [R, N, HQ, D], rows behind a request's last are not used
    q = q.reshape(R, N, HKV, g, D).permute(0, 2, 1, 3, 4).reshape(R, HKV, N * g, D) * s["scale"]
    w = torch.matmul(q, k.transpose(2, 3).contiguous()).reshape(R, HKV, N, g, nb * page)
    last = (kv - n)[:, None] + i[None, :]  # the last key that a token sees
    hidden = torch.arange(nb * page, device=k.device)[None, None, :] > last[:, :, None]
    w.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    w.sub_(w.amax(4, keepdim=True)).exp_()
    total = w.sum(4, keepdim=True)
    o = torch.matmul(w.reshape(R, HKV, N * g, nb * page), v).reshape(R, HKV, N, g, D) / total
    t = torch.arange(S, device=k.device)
    r = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=R - 1)
    return o.permute(0, 2, 1, 3, 4)[r, t - cu[r]].reshape(S, HQ, D).to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's calls

def _own_norm(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    S, H, G, m = c["S"], c["H"], c["G"], c["m"]
    fp4 = c["fmt"] == "mxfp4"
    osc.osc_rmsnorm_quant(s["x"], s["res"], s["w"], S, H, EPS, G, s["L"], max(m, 1), osc.OSC_MXFP4 if fp4 else osc.OSC_MXFP8,
                          s["res_out"], s["Q"], s["SC"], s["B"])
    if fp4:  # two codes a byte, as their values
        codes = s["pair"].index_select(0, s["Q"].int()).view(torch.bfloat16)
    else:
        codes = s["Q"].view(torch.float8_e4m3fn)
    spg = 8 if G == 16 else 4
    return dict(res=s["res_out"], codes=codes.view(H // 128, S, 128), scales=s["SC"].view(H // G // spg, S, spg).view(torch.float8_e8m0fnu),
                side=s["B"])


def _own_plan(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    osc.osc_page_plan(s["ctx"], s["new"], c["R"], c["page"], s["NP"], s["free"], s["free"].numel(), s["head"], s["T"], s["table"], s["MB"],
                      s["cu"], s["kv"], s["slot"], s["pos"], s["used"])
    return dict(cu=s["cu"], kv=s["kv"], table=s["table"], slot=s["slot"], pos=s["pos"], used=s["used"])


def _own_append(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    osc.osc_qkv_append(s["qkv"], c["S"], c["HQ"], c["HKV"], c["D"], s["wq"], s["wk"], EPS, s["cs"], s["P"], s["pos"], s["slot"], s["q"],
                       s["kc"], s["vc"], s["NP"], c["page"])
    return dict(q=s["q"], kc=s["kc"], vc=s["vc"])


def _own_attn(s):
    import w4a4_outlier_split_amd as osc
    c = s["c"]
    sizes = (s["S"], c["R"], c["HQ"], c["HKV"], c["D"], c["page"], s["MB"])
    if "ws" not in s:  # the step's workspace, kept with its buffers
        s["ws"] = torch.empty(osc.osc_attn_workspace(*sizes), dtype=torch.uint8, device=DEV)
    osc.osc_attn_paged(s["q"], s["kc"], s["vc"], *sizes, s["NP"], s["table"], s["cu"], s["kv"], s["scale"], s["o"], s["ws"])
    return s["o"]


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    if c["op"] == "norm":
        S, H, K = c["S"], c["H"], c["H"] // c["G"]
        out = S * (H // 2 if c["fmt"] == "mxfp4" else H) + S * K + 2 * S * K * c["m"]
        return dict(bytes=6 * S * H + 2 * H + out, flops=10 * S * H)
    if c["op"] == "plan":
        ctx, new = _lengths(c)
        fresh = sum(_up(a + b, c["page"]) - _up(a, c["page"]) for a, b in zip(ctx, new))
        return dict(bytes=4 * (4 * c["R"] + 2 * fresh + 2 * sum(new)), flops=0)
    if c["op"] == "append":
        S, D, W = c["S"], c["D"], (c["HQ"] + 2 * c["HKV"])
        return dict(bytes=4 * S * W * D + 8 * S + min(S, 8192) * 4 * D, flops=10 * S * W * D)
    ctx, new = _lengths(c)
    HQ, HKV, D = c["HQ"], c["HKV"], c["D"]
    seen = sum(n * a + n * (n + 1) // 2 for a, n in zip(ctx, new))
    keys = sum(a + n for a, n in zip(ctx, new) if n)
    return dict(bytes=4 * keys * HKV * D + 4 * sum(new) * HQ * D, flops=4 * HQ * D * seen)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "plan": lambda s: None, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _exact_norm(s):
    """E4M3 elements as the values ahead of their rounding; E2M1 elements and the scales are steps and have none."""
    c = s["c"]
    S, H, G, m = c["S"], c["H"], c["G"], c["m"]
    res = s["x"].double() + s["res"].double()
    h = res.bfloat16().double()  # the residual stream is held in 16 bits, and the norm is that of what is held
    inv = (h.pow(2).sum(-1) / H + EPS).rsqrt()
    y = h * inv[:, None] * s["w"].double()
    side = None
    if m:
        side = torch.zeros(_up(m * (H // G), 32) * 32, S, dtype=torch.float64, device=y.device)
        for k, offsets in enumerate(s["L"].tolist()):
            for e, o in enumerate(offsets):
                if o >= 0:
                    side[k * m + e] = y[:, k * G + o]
        side = side.reshape(-1, 32, S).transpose(1, 2).contiguous()
    if c["fmt"] == "mxfp4":
        return dict(res=res, codes=None, scales=None, side=side)
    most = y.bfloat16().reshape(S, -1, G).abs().max(2).values.double()
    e = torch.where(most > 0, (torch.floor(torch.log2(most.clamp(min=2.0 ** -140))) - 8).clamp(-127, 127), torch.full_like(most, -127.0))
    codes = y * torch.exp2(-e).repeat_interleave(G, 1)
    return dict(res=res, codes=codes.reshape(S, H // 128, 128).permute(1, 0, 2).contiguous(), scales=None, side=side)


def _exact_append(s):
    c = s["c"]
    S, HQ, HKV, D, page = c["S"], c["HQ"], c["HKV"], c["D"], c["page"]
    x = s["qkv"].double().view(S, -1, D)
    heads = []
    for h in range(HQ + HKV):
        v = x[:, h]
        if c["norm"]:
            v = v / (v.square().sum(1, keepdim=True) / D + EPS).sqrt() * (s["wq"] if h < HQ else s["wk"]).double()
        if c["rope"]:
            z = torch.complex(v[:, :D // 2], v[:, D // 2:])
            turn = s["cs"].double()[s["pos"].long()]
            z = z * torch.complex(turn[:, :D // 2], turn[:, D // 2:])
            v = torch.cat([z.real, z.imag], 1)
        heads.append(v)
    kc, vc = s["kc"].double(), s["vc"].double()
    at, off = torch.div(s["slot"].long(), page, rounding_mode="floor"), s["slot"].long() % page
    for h in range(HKV):
        kc[at, h, off] = heads[HQ + h]
        vc.select(1, h).transpose(1, 2)[at, off] = x[:, HQ + HKV + h]
    return dict(q=torch.stack(heads[:HQ], 1), kc=kc, vc=vc)


def _exact_attn(s):
    c = s["c"]
    HQ, HKV, D, page = c["HQ"], c["HKV"], c["D"], c["page"]
    g = HQ // HKV
    out = torch.empty(s["S"], HQ, D, dtype=torch.float64, device=DEV)
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    for r, total in enumerate(kv):
        a, n = cu[r], cu[r + 1] - cu[r]
        if not n:
            continue
        pages = s["table"][r, :_up(total, page)].long()
        hidden = torch.arange(total, device=DEV)[None, :] > total - n + torch.arange(n, device=DEV)[:, None]
        for h in range(HKV):
            k = s["kc"][pages, h].reshape(-1, D)[:total].double()
            v = s["vc"][pages, h].permute(1, 0, 2).reshape(D, -1)[:, :total].double()
            for j in range(h * g, (h + 1) * g):
                p = torch.softmax((s["q"][a:a + n, j].double() @ k.T * s["scale"]).masked_fill(hidden, -math.inf), 1)
                out[a:a + n, j] = p @ v.T
    return out
