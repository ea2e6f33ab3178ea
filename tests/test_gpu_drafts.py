"""Steps with trees of drafted tokens through the executor: a block whose tokens are trees, accepted paths in the cache against the same
tokens given one behind the other, whole steps captured, and the head behind the last block."""
import numpy as np
import pytest
import torch

import tree_ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from w4a4_outlier_split_amd import block as blk  # noqa: E402
from gpu_util import DEV, dev_bits16  # noqa: E402
from test_gpu_block_step import D, EPS, G, H, HKV, HQ, MB, PAGE, R, T, make_block, make_pages  # noqa: E402
import synth  # noqa: E402

N = 16


def trees(rng, sizes):
    """Parents, tokens and choices of a step's nodes: small alphabets, so that paths of several nodes are accepted."""
    parents = [tree_ref.tree(rng, n, ("near", "star", "chain")[int(rng.integers(0, 3))]) for n in sizes]
    flat = [p for q in parents for p in q]
    fit = lambda v: torch.tensor((list(v) + [0] * T)[:T], dtype=torch.int32)
    return parents, fit(flat), fit(rng.integers(0, 2, len(flat)).tolist()), fit(rng.integers(0, 2, len(flat)).tolist())


def turned(x, w, cs):
    """Heads normed and rotated, in 64 bits, as the cache holds them: in 16."""
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    a, b = x[..., :D // 2], x[..., D // 2:]
    c, s = cs[:, None, :D // 2].double(), cs[:, None, D // 2:].double()
    return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16().double()


def check_attention(att, history, qkv, parents, got):
    """got [T, HQ, D] against 64 bits: history[r] holds the QKV rows of request r's accepted tokens so far."""
    t0 = 0
    for r, q in enumerate(parents):
        n, ctx = len(q), len(history[r])
        if n:
            anc = tree_ref.ancestors(q)
            pos = torch.tensor([ctx + bin(a).count("1") - 1 for a in anc], device=DEV)
            new = qkv[t0:t0 + n].double().reshape(n, HQ + 2 * HKV, D)
            old = torch.stack(history[r]).double().reshape(ctx, HQ + 2 * HKV, D) if ctx else new[:0]
            x, at = torch.cat([old, new]), torch.cat([torch.arange(ctx, device=DEV), pos])
            qs, ks, vs = turned(new[:, :HQ], att.wq, att.cs[pos]), turned(x[:, HQ:HQ + HKV], att.wk, att.cs[at]), x[:, HQ + HKV:]
            hidden = torch.tensor([[j >= ctx and not anc[i] >> (j - ctx) & 1 for j in range(ctx + n)] for i in range(n)], device=DEV)
            for h in range(HQ):
                s = (qs[:, h] @ ks[:, h // (HQ // HKV)].T * att.scale).masked_fill(hidden, -float("inf"))
                w, v = torch.softmax(s, 1), vs[:, h // (HQ // HKV)]
                ref = w @ v
                # weights rounded to bf16 at worst (2^-8), the output too; the reference's q and k may round the other way where the device's
                # binary32 lies across a half step, which moves a score by a step, 2^-7, of one of D products
                size = (qs[:, h].abs() @ ks[:, h // (HQ // HKV)].abs().T * att.scale).amax(1, keepdim=True) * 2.0 ** -7 / D ** 0.5
                tol = (2.0 ** -8 + 2.0 ** -13 + 2 * size) * (w @ v.abs()) + 2.0 ** -8 * ref.abs()
                assert bool(((got[t0:t0 + n, h].double() - ref).abs() <= tol).all()), (r, h)
        t0 += n


@pytest.mark.parametrize("path", ["osc", "fp8"])
def test_block_steps_with_trees(path):
    b, pages = make_block(11, path), make_pages()
    cache = blk.LayerCache(torch, pages, HKV, D, DEV)
    drafts = blk.Drafts(torch, pages, N, [cache], DEV)
    bufs = b.buffers(T, pages, DEV, N)
    a = bufs["attn"]
    g = torch.Generator(device=DEV).manual_seed(5)
    rng = np.random.default_rng(6)
    history, rows, held = [[] for _ in range(R)], [[] for _ in range(R)], 0
    for it, sizes in enumerate([(20, 7, 0), (16, 16, 16), (3, 16, 1), (16, 0, 16), (16, 16, 16), (1, 1, 1), (16, 16, 5)]):
        x = torch.randn((T, H), generator=g, device=DEV).bfloat16()
        Y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        pages.new.copy_(torch.tensor(sizes, dtype=torch.int32))
        t0 = np.concatenate([[0], np.cumsum(sizes)])
        if it == 0:  # the prompts
            pages.plan()
            b.forward(x.clone(), None, T, pages, cache, bufs, Y)
            pages.advance()
            took = [list(range(n)) for n in sizes]
        else:
            parents, parent, token, choice = trees(rng, sizes)
            drafts.parent.copy_(parent), drafts.token.copy_(token)
            pages.plan(), drafts.plan()
            b.forward(x.clone(), None, T, pages, cache, bufs, Y, drafts=drafts)
            check_attention(b.attention, history, a["qkv"], parents, a["o"])
            drafts.accept(choice.to(DEV)), drafts.commit(), drafts.advance()
            want = tree_ref.accept(parents, token.tolist(), choice.tolist(), [True] * T, N, t0.tolist())
            assert drafts.acc.tolist() == want[0] and drafts.path.tolist() == want[1] and drafts.next.tolist() == want[2]
            took = [p[:n] for n, p in zip(*want[:2])]
            assert max(want[0]) > 1 or it == 5
        for r in range(R):
            history[r] += [a["qkv"][t0[r] + i].clone() for i in took[r]]
            rows[r] += [x[t0[r] + i] for i in took[r]]
        assert pages.ctx.tolist() == [len(h) for h in history]
        used = int(pages.head)
        assert used == sum(-(-len(h) // PAGE) for h in history)
        taken = [id for r in range(R) for id in pages.table[r, :-(-len(history[r]) // PAGE)].tolist()]
        assert sorted(taken + pages.free[used:].tolist()) == list(range(pages.NP))
    pages.check()
    # the same tokens as ordinary ones, in steps of as many rows: keys and values are the same bits
    other = make_pages()
    plain = blk.LayerCache(torch, other, HKV, D, DEV)
    left = [list(q) for q in rows]
    while any(left):
        now = [q[:T // R] for q in left]
        left = [q[T // R:] for q in left]
        x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        flat = [v for q in now for v in q]
        x[:len(flat)] = torch.stack(flat)
        other.new.copy_(torch.tensor([len(q) for q in now], dtype=torch.int32))
        other.plan()
        b.forward(x, None, T, other, plain, bufs, torch.empty_like(x))
        other.advance()
    at = lambda p, c, r, i: (c.KC[p.table[r, i // PAGE], :, i % PAGE], c.VC[p.table[r, i // PAGE], :, :, i % PAGE])
    for r in range(R):
        assert len(rows[r]) <= MB * PAGE
        for i in range(len(rows[r])):
            for u, v in zip(at(pages, cache, r, i), at(other, plain, r, i)):
                assert torch.equal(u, v), (r, i)


def make_head(seed, V=None, path="osc"):
    w = dev_bits16(synth.draw_w(1024, H, seed)).view(torch.bfloat16)
    L = np.random.default_rng(seed).integers(-1, G, (H // G, 1)).astype(np.int32)
    gain = (1 + 0.2 * torch.randn(H, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)).bfloat16()
    return blk.Head(blk.Linear(torch, w, 1024, H, G, path, L if path == "osc" else None), gain, EPS, V)


@pytest.mark.parametrize("V,path", [(None, "osc"), (1001, "fp8")])
def test_head(V, path):
    S = 37
    head = make_head(3, V, path)
    V = V or 1024
    bufs = head.buffers(S, DEV, M=2, K=4)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, res = torch.randn((S, H), generator=g, device=DEV).bfloat16(), torch.randn((S, H), generator=g, device=DEV).bfloat16()
    want = (x.float() + res.float()).bfloat16()
    y, logits = torch.empty_like(x), torch.empty((S, 1024), dtype=torch.bfloat16, device=DEV)
    osc.osc_rmsnorm(want, None, head.w, S, H, EPS, None, y)
    head.proj.forward(y, S, head.proj.act_buffers(S, DEV), logits)
    ids = torch.randint(0, V, (S, 2), generator=g, device=DEV).to(torch.int32)
    head.forward(x, res, S, bufs)
    head.logprobs(S, bufs, ids, 0.8)
    assert torch.equal(res, want) and torch.equal(bufs["logits"], logits)
    p = torch.log_softmax(logits[:, :V].double() * 0.8, 1)
    # sums of at most 4 values a thread, joined over 22 steps, terms off by 8 units and the exponents' size (below 64): 2^-24 of each
    tol = 2.0 ** -24 * (26 + 8 + 8 * 64)
    assert bool(((bufs["lp"].double() - p.gather(1, ids.long())).abs() <= tol).all())
    H_ = -(p * p.exp()).sum(1)
    assert bool(((bufs["ent"].double() - H_).abs() <= tol * (2 * H_ + 10)).all())
    order = np.stack([np.lexsort((np.arange(V), -row))[:4] for row in logits[:, :V].float().cpu().numpy()])
    assert bufs["topi"].tolist() == order.tolist()
    for s in (1, 8, S):  # fewer rows in the same buffers
        head.logprobs(s, bufs, None)
        assert bufs["topi"][:s].tolist() == order[:s].tolist()


def test_speculative_steps_captured():
    """Plan, two blocks, head, acceptance and advance in one graph: replays equal eager steps from the same state."""
    K = 3

    def run(captured):
        blocks, pages, head = [make_block(21, "osc"), make_block(31, "fp8")], make_pages(), make_head(5)
        caches = [blk.LayerCache(torch, pages, HKV, D, DEV) for _ in blocks]
        drafts = blk.Drafts(torch, pages, N, caches, DEV)
        bufs = [b.buffers(T, pages, DEV, N) for b in blocks]
        hb = head.buffers(T, DEV, M=1, K=K)
        x, ids = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV), torch.zeros((T, 1), dtype=torch.int32, device=DEV)
        ys = [torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in blocks]

        def step():
            pages.plan()
            drafts.plan()
            rows = blocks[0].forward(x, None, T, pages, caches[0], bufs[0], ys[0], drafts=drafts)
            blocks[1].forward(ys[0], rows, T, pages, caches[1], bufs[1], ys[1], drafts=drafts)
            head.forward(ys[1], rows, T, hb)
            head.logprobs(T, hb, ids)
            hb["topi"][:, 0].remainder_(2)  # as good as a draft: the small alphabet's
            drafts.accept(hb["topi"], K)
            drafts.commit()
            drafts.advance()

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                step()
        g = torch.Generator(device=DEV).manual_seed(77)
        rng = np.random.default_rng(7)
        got = []
        for sizes in ((16, 3, 0), (16, 16, 16), (1, 1, 5), (0, 16, 9), (16, 16, 16), (16, 16, 16), (2, 16, 3)):
            _, parent, token, _ = trees(rng, sizes)
            drafts.parent.copy_(parent), drafts.token.copy_(token)
            pages.new.copy_(torch.tensor(sizes, dtype=torch.int32))
            x.copy_(torch.randn((T, H), generator=g, device=DEV).bfloat16())
            ids.copy_(torch.randint(0, 1024, (T, 1), generator=g, device=DEV))
            torch.cuda.synchronize()
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            n = sum(sizes)
            got += [t.clone() for t in (hb["logits"][:n], hb["lp"][:n], hb["ent"][:n], hb["topv"][:n], hb["topi"][:n], drafts.acc, drafts.path, drafts.next, pages.ctx,
                                        pages.free, pages.head, pages.pos, drafts.mask, caches[1].KC, caches[0].VC)]
        assert sum(pages.ctx.tolist()) > 15  # paths of more than a node each
        return got

    for i, (a, b) in enumerate(zip(run(False), run(True))):
        assert torch.equal(a, b), i


def test_refusals():
    with pytest.raises(ValueError):
        blk.Head(make_head(1).proj, None, EPS, 1025)
    pages = make_pages()
    small = blk.LayerCache(torch, make_pages(), HKV, D, DEV)
    small.KC = small.KC[:2].contiguous()
    with pytest.raises(osc.OscError):
        blk.Drafts(torch, pages, N, [small], DEV)


def test_step_binding_refuses():
    """Too small, of another type, on another device, not contiguous: refused by the binding, named by the status."""
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)
    mask = torch.zeros((4, 1), dtype=torch.int64, device=DEV)
    calls = [(osc.osc_tree_plan, [i32(4), i32(3), i32(2), 2, 4, 8, i32(4), mask]),
             (osc.osc_tree_accept, [i32(4), i32(4), i32(4, 3), 3, i32(4), i32(4), 9, i32(3), 2, 4, 8, i32(2), i32(2, 8), i32(2)])]
    for f, args in calls:
        f(*args)
        for i, t in enumerate(args):
            if not torch.is_tensor(t):
                continue
            for bad, status in ((t.cpu(), 2), (t.float(), 5), (t.to(torch.int64 if t.dtype == torch.int32 else torch.int32), 5),
                                (t.flatten()[:-1].clone() if t.shape != (4, 3) else t[:3].clone(), 2)):
                with pytest.raises(osc.OscError) as e:
                    f(*[bad if j == i else a for j, a in enumerate(args)])
                assert e.value.status == status, (f.__name__, i, status)
    osc.osc_tree_plan(*calls[0][1][:-1], mask.view(torch.uint64))
    cache = lambda: torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    bf = lambda: torch.zeros((4, 4, 64), dtype=torch.bfloat16, device=DEV)
    n = osc.osc_attn_tree_workspace(4, 2, 4, 2, 64, 16, 2, 8)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    args = [bf(), cache(), cache(), 4, 2, 4, 2, 64, 16, 2, 3, i32(2, 2), i32(3), i32(2), mask, 8, 0.1, bf(), ws]
    osc.osc_attn_tree(*args)
    osc.osc_attn_tree(*args[:-1], ws.data_ptr())
    for i, t in enumerate(args):
        if torch.is_tensor(t):
            for bad, status in ((t.cpu(), 2), (t.double(), 5), (t.flatten()[:-1].clone(), 2)):
                if t is ws and status == 5:
                    continue
                with pytest.raises(osc.OscError) as e:
                    osc.osc_attn_tree(*[bad if j == i else a for j, a in enumerate(args)])
                assert e.value.status == status, (i, status)


def test_commit_in_layers_of_other_heads():
    """Layers with heads of their own, some of as many bytes as others: in each the path's nodes move, and nothing else."""
    pages = make_pages()
    heads = [(2, 128), (4, 64), (4, 128), (2, 128), (1, 64)]
    caches = [blk.LayerCache(torch, pages, h, d, DEV) for h, d in heads]
    g = torch.Generator(device=DEV).manual_seed(3)
    for c in caches:
        for t in (c.KC, c.VC):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    drafts = blk.Drafts(torch, pages, N, caches, DEV)
    sizes = (16, 9, 0)
    pages.new.copy_(torch.tensor(sizes, dtype=torch.int32))
    rng = np.random.default_rng(1)
    parents, parent, token, choice = trees(rng, sizes)
    drafts.parent.copy_(parent), drafts.token.copy_(token)
    pages.plan(), drafts.plan()
    drafts.accept(choice.to(DEV))
    want = [(c.KC.clone(), c.VC.clone()) for c in caches]
    slot, acc, path, moved = pages.slot.tolist(), drafts.acc.tolist(), drafts.path.tolist(), 0
    for r, t0 in enumerate((0, 16, 25)):
        for k in range(acc[r]):
            a, b = slot[t0 + path[r][k]], slot[t0 + k]
            moved += a != b
            for kc, vc in want:
                kc[b // PAGE, :, b % PAGE] = kc[a // PAGE, :, a % PAGE].clone()
                vc[b // PAGE, :, :, b % PAGE] = vc[a // PAGE, :, :, a % PAGE].clone()
    assert moved > 0
    drafts.commit()
    for i, (c, (kc, vc)) in enumerate(zip(caches, want)):
        assert torch.equal(c.KC, kc) and torch.equal(c.VC, vc), i
