"""Steps of which some tokens find no row, page or room in their table row: the requests go on without them, over what
was written and nothing else.  Checked against 64 bits over the tokens that the lengths say are there."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from w4a4_outlier_split_amd import block as blk  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_block_step import D, H, HKV, MB, PAGE, R, T, attention_reference, make_block  # noqa: E402

# counts, rows of the call, and how many of them are to be written: more tokens than rows, negative counts, fewer rows than
# the plan, a pool of 7 pages that ends inside a request, rows of 6 pages
STEPS = [((30, 40, 5), 48, (30, 18, 0)), ((1, -9, 3), 48, (1, 0, 3)), ((1, 30, 9), 20, (1, 19, 0)), ((-1, 1, 1), 48, (0, 1, 1)),
         ((15, 30, 2), 48, (15, 10, 2)), ((5, 1, 1), 48, (1, 0, 1))]


@pytest.mark.parametrize("captured", [False, True])
def test_steps_that_lose_tokens(captured):
    b = make_block(41, "osc").attention
    pages = blk.Pages(torch, R, 7, PAGE, MB, T, DEV)
    cache = blk.LayerCache(torch, pages, HKV, D, DEV)
    cache.KC.fill_(1000.0), cache.VC.fill_(1000.0)  # what no step has written
    bufs, y = b.buffers(T, pages, DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)

    def step(S):
        pages.plan()
        b.qkv.quantize(x, S, bufs["x"])
        b.forward_quantized(S, pages, cache, bufs, y)
        pages.advance()

    graphs = {}
    if captured:
        for S in sorted({S for _, S, _ in STEPS}):
            graphs[S] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[S], stream=torch.cuda.Stream()):
                step(S)
    g = torch.Generator(device=DEV).manual_seed(8)
    history, lost = [[] for _ in range(R)], 0
    for counts, S, wrote in STEPS:
        pages.new.copy_(torch.tensor(counts, dtype=torch.int32))
        x.copy_(torch.randn((T, H), generator=g, device=DEV).bfloat16())
        torch.cuda.synchronize()
        graphs[S].replay() if captured else step(S)
        torch.cuda.synchronize()
        t0 = np.concatenate([[0], np.cumsum(np.maximum(counts, 0))])
        for r in range(R):
            history[r] += list(bufs["qkv"][t0[r]:t0[r] + wrote[r]].clone())
        lost += sum(max(c, 0) for c in counts) - sum(wrote)
        assert pages.ctx.tolist() == [len(h) for h in history] and int(pages.lost) == lost
        ref, tol = attention_reference(b, history, bufs["qkv"], wrote, t0)
        ok = (bufs["o"].double() - ref).abs() <= tol
        for r in range(R):
            assert bool(ok[t0[r]:t0[r] + wrote[r]].all()), (counts, r)
    used = int(pages.head)
    held = [id for r in range(R) for id in pages.table[r, :-(-len(history[r]) // PAGE)].tolist()]
    assert sorted(held + pages.free[used:].tolist()) == list(range(7))
    with pytest.raises(RuntimeError, match=f"{lost} tokens"):
        pages.check()
    pages.check()


@pytest.mark.parametrize("handle", [False, True])
def test_steps_on_another_stream(handle):
    """A step on a stream that lags behind torch's current one: advance goes with it, check and release wait for it."""
    pages, side = blk.Pages(torch, 2, 8, PAGE, 4, 64, DEV), torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    pages.new.copy_(torch.tensor([40, 3], dtype=torch.int32))
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        pages.plan(stream)
        pages.advance(stream)
    pages.release([1])
    assert pages.ctx.tolist() == [64, 0] and int(pages.head) == 4
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    pages.plan(stream)
    pages.advance(stream)
    with pytest.raises(RuntimeError, match=f"{16 + 40} tokens"):
        pages.check()
    assert pages.ctx.tolist() == [64, 3] and int(pages.head) == 5


@pytest.mark.parametrize("captured", [False, True])
def test_positions_behind_the_rotary_table(captured):
    """The table ends at 40 of 96 positions: check says how many tokens are behind it, the others are as ever."""
    b = make_block(43, "osc").attention
    b.cs = b.cs[:40]
    pages = blk.Pages(torch, R, 18, PAGE, MB, T, DEV)
    cache, bufs = blk.LayerCache(torch, pages, HKV, D, DEV), b.buffers(T, pages, DEV)
    x, y = (torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        pages.plan()
        b.qkv.quantize(x, T, bufs["x"])
        b.forward_quantized(T, pages, cache, bufs, y)
        pages.advance()

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            step()
    g = torch.Generator(device=DEV).manual_seed(9)
    history, seen = [[] for _ in range(R)], [0] * R
    for counts, lost in (((30, 5, 2), 0), ((8, 1, 38), 0), ((5, 20, 1), 3 + 1), ((1, 13, 0), 1)):
        pages.new.copy_(torch.tensor(counts, dtype=torch.int32))
        x.copy_(torch.randn((T, H), generator=g, device=DEV).bfloat16())
        torch.cuda.synchronize()
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        t0 = np.concatenate([[0], np.cumsum(counts)])
        good = [min(n, max(0, 40 - seen[r])) for r, n in enumerate(counts)]
        for r in range(R):
            history[r] += list(bufs["qkv"][t0[r]:t0[r] + good[r]].clone())
            seen[r] += counts[r]
        ref, tol = attention_reference(b, history, bufs["qkv"], good, t0)
        ok = (bufs["o"].double() - ref).abs() <= tol
        for r in range(R):
            assert bool(ok[t0[r]:t0[r] + good[r]].all()), (counts, r)
        assert pages.ctx.tolist() == seen
        if lost:
            with pytest.raises(RuntimeError, match=f"{lost} tokens"):
                pages.check()
        pages.check()


@pytest.mark.parametrize("requests,pool,rows", [(4096, 9000, 5000), (513, 700, 20000), (1, 40, 8192)])
def test_many_requests_replayed(requests, pool, rows):
    """Plan and advance in one graph, replayed with eager work in between, against the same steps on the host."""
    from test_pages_host import HostPages
    args = (requests, pool, 16, 40, rows)
    pages, host = blk.Pages(torch, *args, DEV), HostPages(torch, *args, "cpu")
    pages.plan(), pages.advance()  # what the first call of a library loads
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pages.plan()
        pages.advance()
    g = torch.Generator().manual_seed(requests)
    for it in range(6):
        new = torch.randint(-1, 3 if requests > 1 else 300, (requests,), generator=g, dtype=torch.int32)
        pages.new.copy_(new), host.new.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        host.plan(), host.advance()
        for name in ("ctx", "head", "lost", "slot", "pos", "cu", "kv"):
            assert torch.equal(getattr(pages, name).cpu(), getattr(host, name)), (it, name)
        held = -(-host.ctx // 16)
        own = torch.arange(40)[None] < held[:, None]
        assert torch.equal(pages.table.cpu()[own], host.table[own])
