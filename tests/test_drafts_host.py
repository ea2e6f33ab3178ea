"""The bookkeeping of steps with drafted tokens (block.Drafts) on host tensors, plan and acceptance taken one node after the other: what a
request's row says is in the cache is the path that was accepted, and no page is lost or held twice."""
import numpy as np
import pytest
import torch

import tree_ref
from test_pages_host import HostPages

blk = pytest.importorskip("w4a4_outlier_split_amd.block", reason="libosc.so not built")
osc = pytest.importorskip("w4a4_outlier_split_amd")


class HostDrafts(blk.Drafts):
    """``plan``, ``accept`` and ``commit`` as osc_tree_plan, osc_tree_accept and osc_tree_commit document them."""

    def trees(self):
        p = self.pages
        cu, rows = p.cu.tolist(), self.parent.tolist()
        return cu, [rows[cu[r]:cu[r + 1]] for r in range(p.R)]

    def plan(self, stream=None):
        p = self.pages
        cu, trees = self.trees()
        pos, mask = tree_ref.plan(trees, p.ctx.tolist(), p.T, self.N, cu[0])
        p.pos.copy_(torch.tensor(pos, dtype=torch.int32))

    def accept(self, choice, ldc=1, stream=None):
        p = self.pages
        T, end = p.rows, p.positions if p.positions < p.MB * p.page else 0
        cu, trees = self.trees()
        written = [s >= 0 and (end == 0 or 0 <= x < end) for s, x in zip(p.slot.tolist()[:T], p.pos.tolist()[:T])]
        acc, path, after = tree_ref.accept(trees, self.token.tolist()[:T], choice.reshape(-1)[::ldc].tolist()[:T], written, self.N, cu)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)
        self.acc.copy_(i32(acc)), self.path.copy_(i32(path)), self.next.copy_(i32(after))

    def move(self, cache):
        """``commit`` on a dict of slots."""
        p = self.pages
        slot, cu = p.slot.tolist(), p.cu.tolist()
        for r in range(p.R):
            for k, at in enumerate(self.path[r, :int(self.acc[r])].tolist()):
                cache[slot[cu[r] + k]] = cache[slot[cu[r] + at]]


def make(R, NP, page, MB, T, N):
    p = HostPages(torch, R, NP, page, MB, T, "cpu")
    p.free.copy_(torch.randperm(NP, generator=torch.Generator().manual_seed(NP)).to(torch.int32))
    return p, HostDrafts(torch, p, N, [blk.LayerCache(torch, p, 1, 64, "cpu")], "cpu"), {}, [[] for _ in range(R)]


def step(p, d, cache, text, sizes, rng, rows=None, rate=0.7):
    """One step: trees of these sizes, some of whose tokens the model chooses; text: each request's tokens so far."""
    parents = [tree_ref.tree(rng, n, ("near", "chain", "star", "roots")[int(rng.integers(0, 4))]) for n in sizes]
    flat = [x for q in parents for x in q]
    token, choice = rng.integers(0, 1000, max(len(flat), 1)).tolist(), rng.integers(0, 1000, max(len(flat), 1)).tolist()
    at = 0
    for q in parents:
        for i in range(len(q)):
            children = [j for j in range(len(q)) if q[j] == i]
            if children and rng.random() < rate:
                choice[at + i] = token[at + int(rng.choice(children))]
        at += len(q)
    fit = lambda v: torch.tensor((v + [0] * p.T)[:p.T], dtype=torch.int32)
    p.new.copy_(torch.tensor(sizes, dtype=torch.int32))
    d.parent.copy_(fit(flat)), d.token.copy_(fit(token))
    p.plan(), d.plan()
    p.rows = p.T if rows is None else rows
    slot, cu, pos = p.slot.tolist(), p.cu.tolist(), p.pos.tolist()
    before, lost = p.ctx.tolist(), int(p.lost)
    for r in range(p.R):
        for i in range(sizes[r]):
            t = cu[r] + i
            if t < p.rows and slot[t] >= 0 and pos[t] < p.positions:
                cache[slot[t]] = (r, pos[t], token[t])
    d.accept(fit(choice)), d.move(cache), d.advance()
    for r in range(p.R):
        took = d.path[r, :int(d.acc[r])].tolist()
        text[r] += [token[cu[r] + x] for x in took]
        assert p.ctx.tolist()[r] == before[r] + len(took) == len(text[r])
    assert int(p.lost) - lost == sum(1 for r in range(p.R) if sizes[r] and not int(d.acc[r]))


def check(p, cache, text):
    ctx, table, head = p.ctx.tolist(), p.table.tolist(), int(p.head)
    held = [table[r][:-(-c // p.page)] for r, c in enumerate(ctx)]
    for r, c in enumerate(ctx):
        for at in range(c):
            assert cache[held[r][at // p.page] * p.page + at % p.page] == (r, at, text[r][at])
    pages = [id for h in held for id in h]
    assert sorted(pages + p.free.tolist()[head:]) == list(range(p.NP))  # each held once or free


@pytest.mark.parametrize("page,N", [(16, 40), (16, 8), (64, 64), (32, 256)])
def test_steps(page, N):
    rng = np.random.default_rng(N)
    R, MB = 5, 2 + 600 // page
    p, d, cache, text = make(R, R * MB, page, MB, R * N, N)
    for it in range(12):
        step(p, d, cache, text, [int(v) for v in rng.integers(0, N + 1, R)], rng, rate=(0.0, 0.5, 1.0)[it % 3])
        check(p, cache, text)


def test_ordinary_steps_between():
    rng = np.random.default_rng(2)
    p, d, cache, text = make(3, 40, 16, 12, 60, 20)
    for it in range(6):
        new = [int(v) for v in rng.integers(0, 20, 3)]
        p.new.copy_(torch.tensor(new, dtype=torch.int32))
        p.plan()
        slot, cu = p.slot.tolist(), p.cu.tolist()
        for r in range(3):
            for i in range(new[r]):
                cache[slot[cu[r] + i]] = (r, len(text[r]), -it)
                text[r].append(-it)
        p.advance()
        step(p, d, cache, text, [20, 0, 7], rng)
        check(p, cache, text)
        if it == 3:
            p.release([1])
            text[1] = []
            check(p, cache, text)


def test_the_free_list_ends_inside_the_step():
    for seed in range(20):
        rng = np.random.default_rng(seed)
        p, d, cache, text = make(4, 9, 16, 6, 160, 40)
        for _ in range(4):
            step(p, d, cache, text, [int(v) for v in rng.integers(0, 41, 4)], rng, rate=1.0)
            check(p, cache, text)


def test_no_row_no_room_no_position():
    rng = np.random.default_rng(5)
    p, d, cache, text = make(3, 30, 16, 4, 30, 20)  # trees of 60 nodes on 30 rows, tables of 64 tokens
    for _ in range(9):
        step(p, d, cache, text, [20, 20, 20], rng, rate=1.0)
        check(p, cache, text)
    p, d, cache, text = make(3, 30, 16, 8, 60, 20)
    p.positions = 0
    for _ in range(9):
        plan = p.plan
        p.plan = lambda: (plan(), setattr(p, "positions", 50))  # a rotary table shorter than the requests' tables
        step(p, d, cache, text, [20, 20, 1], rng, rate=1.0)
        p.plan = plan
        check(p, cache, text)
        assert max(p.ctx.tolist()) <= 50
    for _ in range(3):
        step(p, d, cache, text, [3, 3, 3], rng, rows=4)
        check(p, cache, text)


def test_sizes_are_checked():
    p = HostPages(torch, 2, 4, 16, 2, 8, "cpu")
    for N in (0, 257):
        with pytest.raises(ValueError):
            blk.Drafts(torch, p, N, [], "cpu")
    assert len(blk.Drafts(torch, p, 4, [blk.LayerCache(torch, p, 1, 64, "cpu") for _ in range(130)], "cpu").groups) == 2


def test_layers_of_other_heads():
    """Each commit is told the heads that its layers have, whatever the layers' order; caches of another layout or that share bytes are refused."""
    p = HostPages(torch, 2, 4, 16, 2, 8, "cpu")
    heads = [(2, 128), (4, 64), (2, 128), (4, 128), (4, 64), (1, 64)]  # (2, 128) and (4, 64) have the same bytes
    caches = [blk.LayerCache(torch, p, h, d, "cpu") for h, d in heads]
    d = blk.Drafts(torch, p, 4, caches, "cpu")
    place = {t.data_ptr(): t.shape for c in caches for t in (c.KC, c.VC)}
    assert sum(g.layers for g in d.groups) == len(caches) and len(place) == 2 * len(caches)
    for g in d.groups:
        for i in range(g.layers):
            assert place.pop(g._kc[i]) == (4, g.HKV, 16, g.D) and place.pop(g._vc[i]) == (4, g.HKV, g.D, 16)
    assert not place
    other = HostPages(torch, 2, 4, 32, 2, 8, "cpu")  # larger pages, as many of them
    turned = blk.LayerCache(torch, p, 2, 128, "cpu")
    turned.VC = turned.VC.transpose(2, 3).contiguous()
    for bad in (blk.LayerCache(torch, other, 2, 128, "cpu"), turned):
        with pytest.raises(osc.OscError) as e:
            blk.Drafts(torch, p, 4, [caches[0], bad], "cpu")
        assert e.value.status == 2
    half = blk.LayerCache(torch, p, 1, 64, "cpu")
    half.KC = caches[5].KC.clone()
    half.VC = caches[3].VC.view(-1)[4096:4096 + half.VC.numel()].view(half.VC.shape)  # among another layer's, of other heads
    many = [blk.LayerCache(torch, p, 1, 64, "cpu") for _ in range(129)]
    for bad in (caches + [half], [caches[1], caches[1]], many + [many[0]]):  # the last is of another commit than the first
        with pytest.raises(ValueError):
            blk.Drafts(torch, p, 4, bad, "cpu")
    pool = blk.LayerCache(torch, HostPages(torch, 2, 9, 16, 2, 8, "cpu"), 2, 128, "cpu")  # of more pages than are dealt out
    assert blk.Drafts(torch, p, 4, [pool], "cpu").groups[0].layers == 1


def test_what_is_counted_as_lost():
    """An ordinary step's lost tokens and the trees without a written node 0, one each, in one number; drafts without a place are none."""
    rng = np.random.default_rng(3)
    p, d, cache, text = make(3, 30, 16, 8, 12, 20)
    step(p, d, cache, text, [5, 20, 4], rng)  # the second tree loses 13 drafts, the third its node 0
    assert int(p.lost) == 1 and int(d.acc[2]) == 0 and int(d.next[2]) == -1
    p.new.copy_(torch.tensor([8, 6, 0], dtype=torch.int32))
    p.plan(), p.advance()  # two tokens more than rows
    with pytest.raises(RuntimeError, match=r"^3 tokens \(of a tree of drafted ones its node 0 alone counts\) found no row"):
        p.check()
    p.check()
    step(p, d, cache, [[0] * n for n in p.ctx.tolist()], [5, 5, 2], rng)
    p.check()
