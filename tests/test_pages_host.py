"""The page tables' bookkeeping between steps (block.Pages) on host tensors, the plan taken one token after the
other: what a request's row says is in the cache has been written there, and no page is lost or held twice."""
import numpy as np
import pytest
import torch

blk = pytest.importorskip("w4a4_outlier_split_amd.block", reason="libosc.so not built")


class HostPages(blk.Pages):
    """``plan`` as osc_page_plan documents it."""

    def plan(self, stream=None):
        ctx, new, free = self.ctx.tolist(), self.new.tolist(), self.free.tolist()
        table, head = self.table.tolist(), max(int(self.head), 0)
        cap, cu, slot, pos, used = self.MB * self.page, [0], [], [], 0
        for r, (c, n) in enumerate(zip(ctx, new)):
            c, n = max(c, 0), max(n, 0)
            have, want = (-(-min(v, cap) // self.page) for v in (c, c + n))
            for q in range(have, want):
                table[r][q] = free[head + used] if head + used < len(free) else -1
                used += 1
            for at in range(c, c + n):
                id = table[r][at // self.page] if at < cap else -1
                pos.append(at)
                slot.append(id * self.page + at % self.page if id >= 0 else -1)
            cu.append(cu[-1] + n)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)
        pad = [-1] * max(0, self.T - len(slot))
        self.table.copy_(i32(table)), self.cu.copy_(i32(cu)), self.used.copy_(i32([used]))
        self.kv.copy_(i32([max(c, 0) + max(n, 0) for c, n in zip(ctx, new)]))
        self.slot.copy_(i32((slot + pad)[:self.T])), self.pos.copy_(i32((pos + pad)[:self.T]))


def step(p, cache, new, rows=None):
    """One step: plan, the write of the rows' tokens into ``cache`` (slot -> request and position), advance."""
    p.new.copy_(torch.tensor(new, dtype=torch.int32))
    p.plan()
    n = p.rows = p.T if rows is None else rows
    slot, pos, cu = p.slot.tolist(), p.pos.tolist(), p.cu.tolist()
    for t in range(min(n, cu[-1])):
        if slot[t] >= 0:
            cache[slot[t]] = (next(r for r in range(p.R) if cu[r] <= t < cu[r + 1]), pos[t])
    p.advance()


def check(p, cache):
    ctx, table, head = p.ctx.tolist(), p.table.tolist(), int(p.head)
    held = [table[r][:-(-c // p.page)] for r, c in enumerate(ctx)]
    for r, c in enumerate(ctx):
        assert 0 <= c <= p.MB * p.page
        for at in range(c):
            assert cache[held[r][at // p.page] * p.page + at % p.page] == (r, at)
    pages = [id for h in held for id in h]
    assert sorted(pages + p.free.tolist()[head:]) == list(range(p.NP))  # each held once or free


def test_more_tokens_than_rows():
    p, cache = HostPages(torch, 3, 12, 16, 4, 20, "cpu"), {}
    step(p, cache, [10, 25, 30])
    check(p, cache)
    assert p.ctx.tolist() == [10, 10, 0] and int(p.lost) == 45
    step(p, cache, [1, 15, 4])
    check(p, cache)
    assert p.ctx.tolist() == [11, 25, 4]
    with pytest.raises(RuntimeError, match="45 tokens"):
        p.check()
    p.check()


def test_fewer_rows_than_tokens():
    p, cache = HostPages(torch, 2, 12, 16, 6, 64, "cpu"), {}
    step(p, cache, [20, 20], rows=30)
    check(p, cache)
    assert p.ctx.tolist() == [20, 10] and int(p.lost) == 10
    step(p, cache, [5, 5], rows=10)
    check(p, cache)
    step(p, cache, [5, 5], rows=0)
    check(p, cache)
    assert p.ctx.tolist() == [25, 15] and int(p.lost) == 20


def test_negative_counts_are_idle():
    p, cache = HostPages(torch, 2, 12, 16, 6, 64, "cpu"), {}
    step(p, cache, [33, 20])
    step(p, cache, [-30, 1])
    check(p, cache)
    assert p.ctx.tolist() == [33, 21]
    step(p, cache, [10, -2 ** 31])
    check(p, cache)
    assert p.ctx.tolist() == [43, 21]
    p.check()


def test_positions_behind_the_rotary_table():
    """The blocks wrote nothing for them: ``lost`` says so, and the request keeps its pages."""
    p = HostPages(torch, 2, 12, 16, 4, 100, "cpu")

    def run(new, rows=100):
        p.new.copy_(torch.tensor(new, dtype=torch.int32))
        p.plan()
        p.rows, p.positions = rows, 40
        p.advance()

    run([30, 40])
    p.check()
    run([15, 2])
    assert p.ctx.tolist() == [45, 42] and int(p.lost) == 5 + 2 and int(p.head) == 6
    run([3, 60], rows=10)
    assert p.ctx.tolist() == [48, 49] and int(p.lost) == 7 + 3 + 60 and int(p.head) == 7
    p.release([1])
    run([0, 50])
    assert p.ctx.tolist() == [48, 50] and int(p.lost) == 70 + 10 and int(p.head) == 7


def test_pool_and_row_run_out():
    p, cache = HostPages(torch, 3, 5, 16, 4, 200, "cpu"), {}
    step(p, cache, [30, 70, 5])  # two pages, then room for 64 and pages for 48, then none
    check(p, cache)
    assert p.ctx.tolist() == [30, 48, 0] and int(p.head) == 5 and int(p.lost) == 27
    step(p, cache, [2, 1, 1])  # the rest of a page is there
    check(p, cache)
    assert p.ctx.tolist() == [32, 48, 0]
    p.release([1])
    check(p, cache)
    step(p, cache, [0, 3, 20])
    check(p, cache)
    assert p.ctx.tolist() == [32, 3, 20] and int(p.head) == 5
    p, cache = HostPages(torch, 1, 9, 16, 4, 200, "cpu"), {}
    step(p, cache, [60])
    step(p, cache, [9])
    step(p, cache, [1])
    check(p, cache)
    assert p.ctx.tolist() == [64] and int(p.lost) == 6


@pytest.mark.parametrize("seed", range(20))
def test_any_steps(seed):
    rng = np.random.default_rng(seed)
    R, page, MB, T = int(rng.integers(1, 6)), 16, int(rng.integers(1, 6)), int(rng.integers(1, 120))
    p, cache = HostPages(torch, R, int(rng.integers(1, R * MB + 3)), page, MB, T, "cpu"), {}
    p.free.copy_(torch.from_numpy(rng.permutation(p.NP)))
    lost = 0
    for _ in range(25):
        new = [int(v) for v in rng.integers(-3, rng.choice([2, 20, 60]), R)]
        rows = None if rng.random() < 0.5 else int(rng.integers(0, T + 1))
        before = p.ctx.tolist()
        step(p, cache, new, rows)
        check(p, cache)
        took = [b - a for a, b in zip(before, p.ctx.tolist())]
        assert all(0 <= k <= max(n, 0) for k, n in zip(took, new))
        lost += sum(max(n, 0) for n in new) - sum(took)
        assert int(p.lost) == lost
        if rng.random() < 0.3:
            gone = sorted(rng.choice(R, int(rng.integers(1, R + 1)), replace=False).tolist())
            p.release(gone)
            check(p, cache)
            assert all(p.ctx.tolist()[r] == 0 for r in gone)
