"""A transformer block through the executor, step after step over the paged cache: prompt chunks and
decodes of several requests in one batch, padded, eager and captured.  Each stage is checked on the
device's own previous output: the projections bit for bit against the separate calls, the attention
against 64 bits over the whole history."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from w4a4_outlier_split_amd import block as blk  # noqa: E402
from gpu_util import DEV, dev_bits16  # noqa: E402

H, HQ, HKV, D, F, G, EPS = 512, 8, 2, 64, 512, 32, 1e-6
R, PAGE, MB, T = 3, 16, 6, 48


def make_block(seed, path):
    w = lambda n, k, s: dev_bits16(synth.draw_w(n, k, s)).view(torch.bfloat16)
    rng = np.random.default_rng(seed)
    L = lambda k: rng.integers(-1, G, (k // G, 1)).astype(np.int32)
    lin = lambda n, k, s, p: blk.Linear(torch, w(n, k, s), n, k, G, p, L(k) if p == "osc" else None)
    g = torch.Generator(device=DEV).manual_seed(seed)
    gain = lambda n: (1 + 0.2 * torch.randn(n, generator=g, device=DEV)).bfloat16()
    att = blk.Attention(lin((HQ + 2 * HKV) * D, H, seed, path), lin(H, HQ * D, seed + 1, "osc"), HQ, HKV, D, gain(D), gain(D),
                        blk.rope_table(torch, MB * PAGE, D, 1e4, DEV), EPS)
    mlp = blk.MLP(lin(2 * F, H, seed + 2, path), lin(H, F, seed + 3, "fp8"))
    return blk.Block(att, mlp, gain(H), gain(H), EPS)


def make_pages():
    p = blk.Pages(torch, R, R * MB, PAGE, MB, T, DEV)
    p.free.copy_(torch.randperm(R * MB, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV))
    return p


def normed(b, x, w):
    y = torch.empty_like(x)
    osc.osc_rmsnorm(x, None, w, T, H, EPS, None, y)
    return y


def attention_reference(att, history, qkv, counts, t0):
    """history[r]: the QKV rows of request r so far, with this step's."""
    out, tol = torch.zeros(T, HQ, D, dtype=torch.float64, device=DEV), torch.ones(T, HQ, D, dtype=torch.float64, device=DEV)

    def turned(x, w):
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
        cs = att.cs.double()[:x.shape[0], None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        c, s = cs[..., :D // 2], cs[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16().double()  # held in 16 bits

    for r, n in enumerate(counts):
        if not n:
            continue
        x = torch.stack(history[r]).double().reshape(len(history[r]), HQ + 2 * HKV, D)
        q, k, v = turned(x[:, :HQ], att.wq)[-n:], turned(x[:, HQ:HQ + HKV], att.wk), x[:, HQ + HKV:]
        kv = x.shape[0]
        hidden = torch.arange(kv, device=DEV)[None] > (kv - n + torch.arange(n, device=DEV))[:, None]
        for h in range(HQ):
            s = (q[:, h] @ k[:, h // 4].T * att.scale).masked_fill(hidden, -float("inf"))
            w = torch.softmax(s, 1)
            out[t0[r]:t0[r] + n, h] = w @ v[:, h // 4]
            # Weights rounded to bf16 (2^-8), the output too.  The reference's q and k may round the other way where the
            # device's binary32 lies across a half step: a score then moves by one step, 2^-7, of a product's share; sized
            # at the whole row, sum |q k| scale 2^-7 / sqrt(D) (one of D products).
            size = (q[:, h].abs() @ k[:, h // 4].abs().T * att.scale).amax(1, keepdim=True) * 2.0 ** -7 / D ** 0.5
            tol[t0[r]:t0[r] + n, h] = (2.0 ** -8 + 2.0 ** -13 + 2 * size) * (w @ v[:, h // 4].abs()) + 2.0 ** -8 * out[t0[r]:t0[r] + n, h].abs()
    return out, tol


@pytest.mark.parametrize("path", ["osc", "fp8"])
def test_block_steps(path):
    b, pages = make_block(11, path), make_pages()
    cache = blk.LayerCache(torch, pages, HKV, D, DEV)
    bufs = b.buffers(T, pages, DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    history = [[] for _ in range(R)]
    for it, counts in enumerate([(20, 7, 0), (1, 16, 30), (1, 0, 1), (27, 1, 17), (1, 1, 1)]):
        pages.new.copy_(torch.tensor(counts, dtype=torch.int32))
        x, res = torch.randn((T, H), generator=g, device=DEV).bfloat16(), torch.randn((T, H), generator=g, device=DEV).bfloat16() * 4
        if it == 1:
            res = None  # as the first block of a model is called
        x0, res0 = x.clone(), None if res is None else res.clone()
        Y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        pages.plan()
        rows = b.forward(x, res, T, pages, cache, bufs, Y)
        pages.advance()
        torch.cuda.synchronize()
        n = sum(counts)
        a = bufs["attn"]
        stream = x0 if res0 is None else (x0.float() + res0.float()).bfloat16()
        act, want = b.attention.qkv.act_buffers(T, DEV), torch.empty_like(a["qkv"])
        b.attention.qkv.forward(normed(b, stream, b.w_attn), T, act, want)
        assert torch.equal(a["qkv"], want)
        t0 = np.concatenate([[0], np.cumsum(counts)])
        for r in range(R):
            history[r] += list(a["qkv"][t0[r]:t0[r + 1]].clone())
        ref, tol = attention_reference(b.attention, history, a["qkv"], counts, t0)
        assert bool(((a["o"].double() - ref).abs() <= tol)[:n].all())
        want = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        b.attention.out.forward(a["o"], T, b.attention.out.act_buffers(T, DEV), want)
        assert torch.equal(bufs["y"], want)
        stream = (want.float() + stream.float()).bfloat16()
        assert torch.equal(rows, stream) and rows is (x if res0 is None else res)
        b.mlp.forward(normed(b, stream, b.w_mlp), T, b.mlp.buffers(T, DEV), want)
        assert torch.equal(Y, want)
    assert pages.ctx.tolist() == [len(h) for h in history]
    # a finished request's pages serve the next
    held = pages.table[1].clone()
    pages.release([1])
    used = int(pages.head)
    assert pages.ctx.tolist()[1] == 0 and bool((pages.table[1] == -1).all())
    assert used == sum(-(-len(history[r]) // PAGE) for r in (0, 2))
    free = set(pages.free[used:].tolist())
    assert free >= set(held[held >= 0].tolist()) and len(free) == R * MB - used
    assert not free & set(pages.table[pages.table >= 0].tolist())
    pages.new.copy_(torch.tensor([0, 33, 0], dtype=torch.int32))
    pages.plan()
    assert len(set(pages.table[pages.table >= 0].tolist())) == used + 3


def test_two_blocks_captured():
    """Plan, two blocks and the lengths' advance in one graph: replays equal eager steps from the same state."""
    def run(captured):
        blocks, pages = [make_block(21, "osc"), make_block(31, "fp8")], make_pages()
        caches = [blk.LayerCache(torch, pages, HKV, D, DEV) for _ in blocks]
        bufs = [b.buffers(T, pages, DEV) for b in blocks]
        x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        ys = [torch.zeros((T, H), dtype=torch.bfloat16, device=DEV) for _ in blocks]

        def step():
            pages.plan()
            rows = blocks[0].forward(x, None, T, pages, caches[0], bufs[0], ys[0])
            blocks[1].forward(ys[0], rows, T, pages, caches[1], bufs[1], ys[1])
            pages.advance()

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                step()
        g = torch.Generator(device=DEV).manual_seed(77)
        got = []
        for counts in ((30, 3, 0), (1, 1, 5), (1, 1, 1), (0, 40, 1), (1, 1, 1), (1, 1, 1)):
            pages.new.copy_(torch.tensor(counts, dtype=torch.int32))
            x.copy_(torch.randn((T, H), generator=g, device=DEV).bfloat16())
            torch.cuda.synchronize()
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            n = sum(counts)
            got += [x[:n].clone(), ys[1][:n].clone(), caches[1].KC.clone(), pages.table.clone(), pages.ctx.clone()]
        return got

    for i, (a, b) in enumerate(zip(run(False), run(True))):
        assert torch.equal(a, b), i


def test_buffers_hold_for_steps_of_fewer_rows():
    """One set of buffers, steps of every kernel: a prompt, a chunk, single tokens, a padded chunk."""
    t, mb = 2400, 2048
    b = make_block(12, "osc")
    pages = blk.Pages(torch, R, 400, PAGE, mb, t, DEV)
    cache, bufs = blk.LayerCache(torch, pages, HKV, D, DEV), b.buffers(t, pages, DEV)
    assert all(osc.osc_attn_workspace(s, R, HQ, HKV, D, PAGE, mb) <= bufs["attn"]["ws"].numel() for s in range(t + 1))
    g = torch.Generator(device=DEV).manual_seed(6)
    for S, counts in ((2400, (2300, 0, 90)), (65, (0, 64, 1)), (3, (1, 1, 1)), (2, (1, 0, 1)), (48, (1, 0, 30)), (4, (2, 1, 1))):
        pages.new.copy_(torch.tensor(counts, dtype=torch.int32))
        x, Y = torch.randn((S, H), generator=g, device=DEV).bfloat16(), torch.empty((S, H), dtype=torch.bfloat16, device=DEV)
        other = {**bufs["attn"], "ws": torch.empty((osc.osc_attn_workspace(S, R, HQ, HKV, D, PAGE, mb),), dtype=torch.uint8, device=DEV)}
        pages.plan()
        b.forward(x.clone(), None, S, pages, cache, bufs, Y)
        again = torch.empty_like(Y)
        b.forward(x.clone(), None, S, pages, cache, {**bufs, "attn": other}, again)
        pages.advance()
        n = sum(counts)
        assert torch.equal(Y[:n], again[:n]) and bool(torch.isfinite(Y[:n].float()).all())


def test_refusals():
    b, pages = make_block(11, "osc"), make_pages()
    with pytest.raises(ValueError):
        b.attention.forward_quantized(T + 1, pages, None, None, None)
    with pytest.raises(ValueError):
        pages.release([0, 0])
    with pytest.raises(ValueError):
        pages.release([R])
    x = torch.zeros((1, H), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        b.forward(x, None, 1, pages, None, None, x)
    with pytest.raises(ValueError):
        blk.Attention(b.attention.qkv, b.attention.out, HQ, HKV + 1, D)
    with pytest.raises(ValueError):
        blk.Block(b.attention, blk.MLP(blk.Linear(torch, torch.zeros(512, 256, dtype=torch.bfloat16, device=DEV), 512, 256, G, "fp8"),
                                       blk.Linear(torch, torch.zeros(256, 256, dtype=torch.bfloat16, device=DEV), 256, 256, G, "fp8")), b.w_attn, b.w_mlp)
