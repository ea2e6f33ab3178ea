"""A Qwen3-8B-shaped transformer block run through libosc, each linear layer on the path its input
calls for (OSC page "W4A4量化技术：OSC框架如何实现高效LLM部署", §2.3 Table 1 and the per-module rule
that follows it, §4 for W2).

Host-side orchestration only: buffers are torch tensors (device memory), every step of every
layer runs in the library's kernels through the C ABI.  ``Linear`` and ``MLP`` are the projections;
``Pages``, ``LayerCache``, ``Attention`` and ``Block`` put the residual adds, the norms and the attention
over the paged cache between them, ``Drafts`` lets a step's tokens be trees of drafted ones, and ``Head`` gives
log probabilities behind the last block.

Per-module rule (§2.3): a module input's clustering density C is the share of a group's outlier
events captured by its statically indexed channel (§2.2), averaged over the groups that saw an
event; C >= 35 % keeps the 4-bit OSC path with the table, C < 35 % switches the module to FP8
microscaling activations (the §4 fallback; weights stay MXFP4 unless asked otherwise).  C is
measured on calibration rows of the module's own input; for the down-projection W2 those rows are
the glue output h = silu(gate) * up of the calibration rows pushed through the up-projection.
"""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass
from typing import Optional

import numpy as np

from . import (OSC_MAX_GROUPS, OSC_MAX_LAYERS, OSC_MAX_TREE, OSC_MXFP4, OSC_MXFP8, OSC_Y_BF16, LayerCaches, code_bytes,
               osc_attn_paged, osc_attn_tree, osc_attn_tree_workspace, osc_attn_workspace, osc_build_table_multi, osc_gemm_fp8,
               osc_gemm_multi, osc_logprobs, osc_logprobs_workspace, osc_pack_weights_multi, osc_page_plan, osc_qkv_append,
               osc_quant_act_multi, osc_rmsnorm_quant, osc_swiglu, osc_swiglu_quant, osc_tree_accept, osc_tree_commit, osc_tree_plan,
               scale_bytes, side_elems)

DENSITY_THRESHOLD = 0.35  # §2.3: below it the module falls back to FP8 microscaling
ALPHA, RHO = 5.0, 0.35    # table-builder defaults (§3.1 / §5.2; rho: the 35 % line of §2.3)


def mean_density(hits: np.ndarray, events: np.ndarray) -> float:
    """§2.2's C averaged over the groups that saw an event (0 if none did); hits: the kept
    entry's count per group (first column when the table has m entries per group)."""
    hits = np.asarray(hits).reshape(len(events), -1)[:, 0].astype(np.float64)
    events = np.asarray(events).astype(np.float64)
    seen = events > 0
    return float(np.mean(hits[seen] / events[seen])) if seen.any() else 0.0


@dataclass
class Calibration:
    L: np.ndarray        # int32[K, m] table slice
    hits: np.ndarray     # int32[K, m]
    events: np.ndarray   # int32[K]
    density: float       # mean C over the groups with events
    path: str            # "osc" or "fp8"


def calibrate(torch, Xcal, H: int, G: int = 32, m: int = 1, stream=None,
              threshold: float = DENSITY_THRESHOLD) -> Calibration:
    """Build the table slice on the device from calibration rows Xcal [R, H] (bf16 device tensor)
    and apply the per-module rule."""
    R = Xcal.shape[0]
    K = H // G
    dev = Xcal.device
    L = torch.empty((K * m,), dtype=torch.int32, device=dev)
    hits = torch.empty((K * m,), dtype=torch.int32, device=dev)
    ev = torch.empty((K,), dtype=torch.int32, device=dev)
    osc_build_table_multi(Xcal, R, H, G, ALPHA, RHO, m, L, hits, ev, stream)
    torch.cuda.synchronize()
    Lh = L.cpu().numpy().reshape(K, m)
    hh = hits.cpu().numpy().reshape(K, m)
    eh = ev.cpu().numpy()
    c = mean_density(hh, eh)
    return Calibration(Lh, hh, eh, c, "osc" if c >= threshold else "fp8")


# ------------------------------------------------------------------ per-layer group size (§6)
# §6 names "dynamic group size" (G adapted per layer among 16 / 32 / 64) as a direction only.
# Reading: a larger G is faster (Table 2), but a group can protect only the channels its table
# entries list; G is too large for a layer when its groups often hold two persistent outlier
# channels.  For each candidate G, fastest first, the table is built with two entries per group on
# the layer's calibration rows; two_share = the share of the protected groups whose second entry
# is also kept (a second consistent channel).  The layer takes the largest G whose two_share is at
# most `tolerance`, else the G with the smallest two_share (larger G on ties).

GROUP_SIZES = (64, 32, 16)
TWO_SHARE_TOLERANCE = 0.10


def two_share(L2: np.ndarray) -> float:
    """L2: int[K, 2] table slice built with two entries per group."""
    L2 = np.asarray(L2).reshape(-1, 2)
    protected = L2[:, 0] >= 0
    if not protected.any():
        return 0.0
    return float(np.mean(L2[protected, 1] >= 0))


def choose_group_size(shares: dict, tolerance: float = TWO_SHARE_TOLERANCE) -> int:
    """shares: {G: two_share}.  The rule above."""
    for G in sorted(shares, reverse=True):
        if shares[G] <= tolerance:
            return G
    return min(sorted(shares, reverse=True), key=lambda g: shares[g])


def calibrate_group_size(torch, Xcal, H: int, sizes=GROUP_SIZES, tolerance: float = TWO_SHARE_TOLERANCE,
                         stream=None):
    """-> (chosen G, {G: two_share}) for one layer's calibration rows Xcal [R, H] (device bf16)."""
    shares = {}
    for G in sizes:
        if H % 256 == 0 and H // G * 2 <= OSC_MAX_GROUPS:
            shares[G] = two_share(calibrate(torch, Xcal, H, G, m=2, stream=stream).L)
    return choose_group_size(shares, tolerance), shares


class Linear:
    """One linear layer y = x W^T with W [N, H] bf16, packed once (offline, §3.3) for its path:
    "osc" (MXFP4 activations with the table's channels split off into B, MXFP4 weights and W_L)
    or "fp8" (MXFP8 activations, no split; weights in wfmt)."""

    def __init__(self, torch, W, N: int, H: int, G: int, path: str, L: Optional[np.ndarray] = None, m: int = 1,
                 wfmt: int = OSC_MXFP4, stream=None):
        if path not in ("osc", "fp8"):
            raise ValueError(f"unknown path {path!r}")
        if path == "osc" and L is None:
            raise ValueError("the OSC path needs a table slice")
        self.torch, self.N, self.H, self.G, self.path, self.m = torch, N, H, G, path, m
        self.L = None if path == "fp8" else np.ascontiguousarray(L, np.int32).reshape(H // G, m)
        self.afmt = OSC_MXFP4 if path == "osc" else OSC_MXFP8
        self.wfmt = OSC_MXFP4 if path == "osc" else wfmt
        dev = W.device
        u8 = lambda n: torch.empty((n,), dtype=torch.uint8, device=dev)
        self.QW, self.SW = u8(code_bytes(N, H, self.wfmt)), u8(scale_bytes(N, H, G))
        self.WL = (torch.empty((side_elems(N, H, G, m),), dtype=torch.int16, device=dev)
                   if self.L is not None else None)
        osc_pack_weights_multi(W, N, H, G, self.L, m, self.wfmt, self.QW, self.SW, self.WL, stream)

    def act_buffers(self, S: int, device):
        """Device buffers of the quantized activation operand for S rows."""
        t = self.torch
        QX = t.empty((code_bytes(S, self.H, self.afmt),), dtype=t.uint8, device=device)
        SX = t.empty((scale_bytes(S, self.H, self.G),), dtype=t.uint8, device=device)
        B = (t.empty((side_elems(S, self.H, self.G, self.m),), dtype=t.int16, device=device)
             if self.L is not None else None)
        return QX, SX, B

    def quantize(self, X, S: int, act, stream=None) -> None:
        QX, SX, B = act
        osc_quant_act_multi(X, S, self.H, self.G, self.L, self.m, self.afmt, QX, SX, B, stream)

    def norm_quantize(self, X, res, w, eps: float, S: int, act, stream=None) -> None:
        """Residual add (in place on ``res``, or none) and RMS norm on the way into the quantization."""
        QX, SX, B = act
        osc_rmsnorm_quant(X, res, w, S, self.H, eps, self.G, self.L, self.m, self.afmt, res, QX, SX, B, stream)

    def gemm(self, act, S: int, Y, yt: int = OSC_Y_BF16, stream=None) -> None:
        QX, SX, B = act
        if self.path == "osc":
            osc_gemm_multi(QX, SX, B, self.QW, self.SW, self.WL, S, self.N, self.H, self.G, self.m, Y, yt, stream)
        else:
            osc_gemm_fp8(QX, SX, self.QW, self.SW, self.wfmt, S, self.N, self.H, self.G, Y, yt, stream)

    def forward(self, X, S: int, act, Y, yt: int = OSC_Y_BF16, stream=None) -> None:
        self.quantize(X, S, act, stream)
        self.gemm(act, S, Y, yt, stream)


class MLP:
    """Gated MLP: up-projection with W1 (gate) and W3 (up) stacked as one [2F, H] weight, the glue
    h = silu(gate) * up fused into the quantization of W2's input, then the down-projection W2
    [H, F]."""

    def __init__(self, up: Linear, down: Linear):
        if up.N != 2 * down.H:
            raise ValueError("the up-projection must produce [gate | up], twice W2's input width")
        self.up, self.down = up, down
        self.F = down.H

    def buffers(self, S: int, device):
        t = self.up.torch
        return {"x": self.up.act_buffers(S, device),
                "gu": t.empty((S, 2 * self.F), dtype=t.bfloat16, device=device),
                "h": self.down.act_buffers(S, device)}

    def forward(self, X, S: int, bufs, Y, yt: int = OSC_Y_BF16, stream=None) -> None:
        self.up.quantize(X, S, bufs["x"], stream)
        self.forward_quantized(S, bufs, Y, yt, stream)

    def forward_quantized(self, S: int, bufs, Y, yt: int = OSC_Y_BF16, stream=None) -> None:
        """From the up-projection's quantized input in bufs["x"]."""
        self.up.gemm(bufs["x"], S, bufs["gu"], OSC_Y_BF16, stream)
        QX, SX, B = bufs["h"]
        d = self.down
        osc_swiglu_quant(bufs["gu"], S, self.F, d.G, d.L, d.m, d.afmt, QX, SX, B, stream)
        d.gemm(bufs["h"], S, Y, yt, stream)

    def glue_rows(self, torch, Xcal, stream=None):
        """W2's calibration rows: Xcal [R, H] pushed through the up-projection and the glue."""
        R = Xcal.shape[0]
        dev = Xcal.device
        act = self.up.act_buffers(R, dev)
        gu = torch.empty((R, 2 * self.F), dtype=torch.bfloat16, device=dev)
        self.up.forward(Xcal, R, act, gu, OSC_Y_BF16, stream)
        h = torch.empty((R, self.F), dtype=torch.bfloat16, device=dev)
        osc_swiglu(gu, R, self.F, h, stream)
        return h

    def calibrate_down(self, torch, Xcal, G: int = 32, m: int = 1, stream=None,
                       threshold: float = DENSITY_THRESHOLD) -> Calibration:
        """The per-module rule on W2's calibration rows (glue_rows)."""
        return calibrate(torch, self.glue_rows(torch, Xcal, stream), self.F, G, m, stream, threshold)


# ------------------------------------------------------------------ the rest of the block


def rope_table(torch, P: int, D: int, theta: float, device):
    """fp32 [P, D]: D/2 cosines and D/2 sines of each position's angles p * theta^(-2i/D), taken in
    64 bits (at position 10^5 a 32-bit angle is off by 2^-8 already)."""
    i = torch.arange(D // 2, dtype=torch.float64, device=device)
    angle = torch.arange(P, dtype=torch.float64, device=device)[:, None] * theta ** (-2.0 * i / D)[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _on(torch, stream):
    """torch's own work on ``stream`` (a Stream or a handle; None: torch's current stream)."""
    if stream is None:
        return nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class Pages:
    """The page tables of R requests, shared by all layers: NP pages of ``page`` tokens, at most MB
    pages a request, steps of at most T new tokens.  One step: set ``new`` (int32 [R], device), call
    ``plan``, run the blocks, call ``advance``, all on one stream.  All three are captureable in a graph.

    New tokens that find no row of the step, no free page or no room in their request's MB pages are
    lost: nothing of them is written, their rows of the step's output mean nothing, ``ctx`` does not count
    them, and ``lost`` (int32 [1], device) does.  They are a request's last ones, so ``ctx`` tells what is
    left to be given again.  A request that passes the end of the blocks' rotary table cannot go on: ``ctx``
    does count those tokens, with their pages, and so does ``lost``.  After a step with trees of drafted tokens (Drafts)
    ``lost`` counts a tree whose node 0 was not written as one token, that node; other nodes that find no place are drafts
    that cannot be accepted, and are not counted.  ``rows`` is how many rows the blocks
    ran with since the plan (T until then), ``positions`` how many their rotary table has.  Table entries
    behind a request's ceil(ctx / page) first mean nothing."""

    def __init__(self, torch, R: int, NP: int, page: int, MB: int, T: int, device):
        self.torch, self.R, self.NP, self.page, self.MB, self.T, self.rows = torch, R, NP, page, MB, T, T
        self.positions = MB * page
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)
        self.ctx, self.new, self.kv, self.cu = i32(R), i32(R), i32(R), i32(R + 1)
        self.slot, self.pos, self.used, self.head, self.lost = i32(T), i32(T), i32(1), i32(1), i32(1)
        self.placed = i32(2, T + 1)  # advance's: which rows have a slot, and which were written
        self.table = torch.full((R, MB), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(NP, dtype=torch.int32, device=device)

    def plan(self, stream=None) -> None:
        self.rows, self.positions = self.T, self.MB * self.page
        osc_page_plan(self.ctx, self.new, self.R, self.page, self.NP, self.free, self.free.numel(), self.head, self.T, self.table,
                      self.MB, self.cu, self.kv, self.slot, self.pos, self.used, stream)

    def advance(self, stream=None) -> None:
        """The step's tokens are in the cache now."""
        torch, rows = self.torch, self.rows
        with _on(torch, stream):
            # tokens with a slot, and written tokens, ahead of each row.  (A single line would be scanned by a library
            # call whose fitness for a graph is not known.)
            flags = self.placed[:, :rows + 1]
            torch.ge(self.slot[:rows], 0, out=flags[0, 1:])
            short = self.positions < self.MB * self.page
            if short:
                torch.mul(flags[0, 1:], self.pos[:rows] < self.positions, out=flags[1, 1:])
            sums = flags.cumsum(1, dtype=torch.int32)
            ahead = sums[0].index_select(0, self.cu.clamp(max=rows))
            # a request's tokens with a slot are its first ones, and their pages the first of those that the step took
            wrote = ahead[1:] - ahead[:-1]
            in_last = (self.ctx - 1) & (self.page - 1)  # of a request's last page, less one; a whole page where there is none
            self.head.add_(((in_last + wrote) >> (self.page.bit_length() - 1)).sum(0, keepdim=True, dtype=torch.int32))
            self.ctx.add_(wrote)
            self.lost.add_(self.cu[-1:]).sub_(sums[1 if short else 0, -1:])

    def check(self) -> None:
        """Raises if tokens were lost since the last check.  Waits for the device; not inside a captured graph."""
        self._wait()
        n = int(self.lost)
        if n:
            self.lost.zero_()
            self._wait()
            raise RuntimeError(f"{n} tokens (of a tree of drafted ones its node 0 alone counts) found no row, free page, "
                               f"room in their request's {self.MB} pages or rotary table")

    def _wait(self) -> None:
        """For the device's work on every stream: a step may run on another than torch's current one."""
        if self.ctx.is_cuda:
            self.torch.cuda.synchronize(self.ctx.device)

    def release(self, rows) -> None:
        """The pages of the finished requests ``rows`` go back to the free list and their rows become
        empty.  Waits for the device; not inside a captured graph."""
        t = self.torch
        rows = [int(r) for r in rows]
        if len(set(rows)) != len(rows) or any(not 0 <= r < self.R for r in rows):
            raise ValueError("rows are distinct requests of this table")
        self._wait()
        ctx, head = self.ctx.tolist(), int(self.head)
        back = [self.table[r, :-(-ctx[r] // self.page)] for r in rows]
        left = t.cat([self.free[head:], *[b[b >= 0] for b in back]])
        # the list keeps its address and length (a captured plan reads them): the pages in use stand first
        used = self.free.numel() - left.numel()
        self.free[used:] = left
        self.free[:used] = -1
        self.head.fill_(used)
        at = t.tensor(rows, dtype=t.long, device=self.ctx.device)
        self.table[at] = -1
        self.ctx[at] = 0
        self._wait()


class LayerCache:
    """One layer's keys and values: KC [NP, HKV, page, D] and VC [NP, HKV, D, page] bf16."""

    def __init__(self, torch, pages: Pages, HKV: int, D: int, device):
        self.KC = torch.zeros((pages.NP, HKV, pages.page, D), dtype=torch.bfloat16, device=device)
        self.VC = torch.zeros((pages.NP, HKV, D, pages.page), dtype=torch.bfloat16, device=device)


class Drafts:
    """Trees of drafted tokens for steps on ``pages``, of at most N nodes a request, over the LayerCache of each layer, whose heads may
    differ.  A tree's node 0 is the request's last certain token, which is not in the cache yet.  One step: set ``pages.new`` to the trees' sizes,
    ``token`` and ``parent`` (int32 [T], request by request as the plan has them; a parent is a node's number in its request, -1
    the context); call ``pages.plan`` and ``plan``; run the blocks with ``drafts``; call ``accept`` with the token chosen behind
    each node, ``commit`` and ``advance`` (not the pages' own), all on one stream.  All of it is captureable in a graph.

    ``acc`` (int32 [R]) nodes of each request are in the cache then, those of ``path`` [R, N] in order, and ``next`` [R] is the
    token behind them, the next tree's node 0 (-1 for a request without a tree, or whose node 0 found no row, page, room
    or position: ``pages.lost`` counts one token for each, and the tree is to be given again)."""

    def __init__(self, torch, pages: Pages, N: int, caches, device):
        if not 1 <= N <= OSC_MAX_TREE:
            raise ValueError(f"a tree of {N} nodes, 1 to {OSC_MAX_TREE} are possible")
        self.torch, self.pages, self.N = torch, pages, N
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)
        self.token, self.parent = i32(pages.T), i32(pages.T)
        self.mask = torch.zeros((pages.T, (N + 63) // 64), dtype=torch.int64, device=device)
        self.acc, self.path, self.next = i32(pages.R), i32(pages.R, N), i32(pages.R)
        self.at = torch.arange(pages.free.numel(), dtype=torch.int32, device=device)
        self.layers = list(caches)
        alike = {}  # one commit moves layers of the same heads
        for c in self.layers:
            alike.setdefault((c.KC.shape[1], c.KC.shape[3]), []).append(c)
        self.groups = [LayerCaches([c.KC for c in g], [c.VC for c in g], pages.NP, HKV, D, pages.page)
                       for (HKV, D), all_of in alike.items()
                       for g in (all_of[i:i + OSC_MAX_LAYERS] for i in range(0, len(all_of), OSC_MAX_LAYERS))]
        # a commit refuses caches that share bytes; two commits would move those twice
        held = sorted((t for c in self.layers for t in (c.KC, c.VC)), key=lambda t: t.data_ptr())
        if any(_meet(a, b) for a, b in zip(held, held[1:])):
            raise ValueError("two caches share bytes; one that several layers read is given once")

    def plan(self, stream=None) -> None:
        """Behind the pages' plan: the nodes' positions into ``pages.pos``, and their masks."""
        p = self.pages
        osc_tree_plan(self.parent, p.cu, p.ctx, p.R, p.T, self.N, p.pos, self.mask, stream)

    def accept(self, choice, ldc: int = 1, stream=None) -> None:
        """choice: int32, the token chosen behind row t at choice[t * ldc] (Head's ``topi`` with ldc = K: the most likely one)."""
        p = self.pages
        end = p.positions if p.positions < p.MB * p.page else 0  # of the rotary table, if it is the shorter
        osc_tree_accept(self.token, self.parent, choice, ldc, p.slot, p.pos, end, p.cu, p.R, p.rows, self.N, self.acc, self.path, self.next, stream)

    def commit(self, stream=None) -> None:
        p = self.pages
        for g in self.groups:
            osc_tree_commit(g, p.slot, p.cu, self.acc, self.path, p.R, p.rows, self.N, stream)

    def advance(self, stream=None) -> None:
        """The accepted nodes are in the cache now; pages that the step took for others go back to the free list."""
        torch, p = self.torch, self.pages
        sh = p.page.bit_length() - 1
        with _on(torch, stream):
            new = p.new.clamp(min=0)
            pages_of = lambda n: (n + (p.page - 1)) >> sh
            had = pages_of(p.ctx)
            # 32-bit sums do: a table row holds fewer than 2^31 tokens
            took = pages_of(torch.minimum(new, p.MB * p.page - p.ctx) + p.ctx) - had
            kept = pages_of(p.ctx + self.acc) - had
            ends = torch.stack([took, kept]).cumsum(1, dtype=torch.int32)
            # The step's pages stand in the free list request by request, from its head on: those kept come first now.  (They may be more
            # than the list has: what is behind its end was never taken.)
            j = self.at - p.head
            r = torch.searchsorted(ends[0], j, right=True).clamp(max=p.R - 1)
            e, k, t = ends[:, r], kept[r], took[r]
            nth = j - (e[0] - t)  # of its request's pages
            to = torch.where(nth < k, e[1] - k + nth, ends[1, -1:] + j - e[1])
            to = torch.where((j >= 0) & (j < ends[0, -1:]), to + p.head, self.at)
            p.free.copy_(torch.empty_like(p.free).index_copy_(0, to.long(), p.free))
            p.head.add_(ends[1, -1:])
            p.ctx.add_(self.acc)
            p.lost.add_(((new > 0) & (self.acc == 0)).sum(0, keepdim=True, dtype=torch.int32))


class Attention:
    """QKV projection -> head norms, rotary embedding, cache write -> attention over the paged cache
    -> output projection.  qkv: [(HQ + 2 HKV) D, H], out: [H, HQ D]; wq, wk: [D] bf16 head norm weights
    or None; cs: rope_table or None."""

    def __init__(self, qkv: Linear, out: Linear, HQ: int, HKV: int, D: int, wq=None, wk=None, cs=None, eps: float = 1e-6):
        if qkv.N != (HQ + 2 * HKV) * D or out.H != HQ * D:
            raise ValueError("the projections do not have these heads")
        self.qkv, self.out, self.HQ, self.HKV, self.D = qkv, out, HQ, HKV, D
        self.wq, self.wk, self.cs, self.eps = wq, wk, cs, eps
        self.scale = D ** -0.5

    def buffers(self, S: int, pages: Pages, device, N: int = 0):
        """Buffers for steps of up to S rows, with trees of up to N nodes (0: without)."""
        t = self.qkv.torch
        bf = lambda *n: t.zeros(n, dtype=t.bfloat16, device=device)  # padding rows stay finite through the output projection
        # steps of fewer rows may need more of a workspace than those of many: single tokens, and the fewest rows of the other kernel
        ws = max(osc_attn_workspace(s, pages.R, self.HQ, self.HKV, self.D, pages.page, pages.MB) for s in {S, min(S, pages.R), min(S, pages.R + 1)})
        if N > 0:
            ws = max(ws, osc_attn_tree_workspace(S, pages.R, self.HQ, self.HKV, self.D, pages.page, pages.MB, N))
        return {"x": self.qkv.act_buffers(S, device), "qkv": bf(S, self.qkv.N), "q": bf(S, self.HQ, self.D), "o": bf(S, self.HQ, self.D),
                "ws": t.empty((ws,), dtype=t.uint8, device=device), "ox": self.out.act_buffers(S, device)}

    def forward_quantized(self, S: int, pages: Pages, cache: LayerCache, bufs, Y, stream=None, drafts=None) -> None:
        """From the QKV projection's quantized input in bufs["x"], by the plan in ``pages``, and that of the trees in ``drafts``."""
        if S > pages.T:
            raise ValueError(f"{S} rows, and a plan of {pages.T}")
        pages.rows = min(pages.rows, S)
        if self.cs is not None:  # tokens behind its end are passed over by the append
            pages.positions = min(pages.positions, self.cs.shape[0])
        self.qkv.gemm(bufs["x"], S, bufs["qkv"], OSC_Y_BF16, stream)
        osc_qkv_append(bufs["qkv"], S, self.HQ, self.HKV, self.D, self.wq, self.wk, self.eps, self.cs,
                       0 if self.cs is None else self.cs.shape[0], pages.pos, pages.slot, bufs["q"], cache.KC, cache.VC, pages.NP,
                       pages.page, stream)
        if drafts is None:
            osc_attn_paged(bufs["q"], cache.KC, cache.VC, S, pages.R, self.HQ, self.HKV, self.D, pages.page, pages.MB, pages.NP, pages.table,
                           pages.cu, pages.kv, self.scale, bufs["o"], bufs["ws"], stream)
        else:
            osc_attn_tree(bufs["q"], cache.KC, cache.VC, S, pages.R, self.HQ, self.HKV, self.D, pages.page, pages.MB, pages.NP, pages.table,
                          pages.cu, pages.kv, drafts.mask, drafts.N, self.scale, bufs["o"], bufs["ws"], stream)
        self.out.forward(bufs["o"], S, bufs["ox"], Y, OSC_Y_BF16, stream)


def _meet(a, b) -> bool:
    """Do two contiguous tensors (of an address, its first byte) share bytes?"""
    (at, an), (bt, bn) = ((t, 1) if isinstance(t, int) else (t.data_ptr(), t.nbytes) for t in (a, b))
    return at < bt + bn and bt < at + an


class Block:
    """One pre-norm transformer block on the residual stream: stream += x; attention(norm(stream));
    stream += that; MLP(norm(stream)), whose output is the next block's x."""

    def __init__(self, attention: Attention, mlp: MLP, w_attn, w_mlp, eps: float = 1e-6):
        if attention.out.N != mlp.up.H or attention.qkv.H != mlp.up.H or mlp.down.N != mlp.up.H:
            raise ValueError("the projections do not share the residual stream's width")
        self.attention, self.mlp, self.w_attn, self.w_mlp, self.eps = attention, mlp, w_attn, w_mlp, eps

    def buffers(self, S: int, pages: Pages, device, N: int = 0):
        t = self.mlp.up.torch
        return {"attn": self.attention.buffers(S, pages, device, N), "mlp": self.mlp.buffers(S, device),
                "y": t.empty((S, self.mlp.up.H), dtype=t.bfloat16, device=device)}

    def forward(self, X, res, S: int, pages: Pages, cache: LayerCache, bufs, Y, stream=None, drafts=None):
        """X: [S, H] bf16, the block before's Y; res: the residual stream, updated in place.  The first
        block takes res = None: X is the stream then, and is updated in place.  Writes the MLP's
        output to Y (neither X nor res) and returns the stream.  drafts: the Drafts whose trees the step's tokens are."""
        if any(t is not None and _meet(Y, t) for t in (X, res)):
            raise ValueError("Y is written while X and the residual stream are in use")
        self.attention.qkv.norm_quantize(X, res, self.w_attn, self.eps, S, bufs["attn"]["x"], stream)
        stream_rows = X if res is None else res
        self.attention.forward_quantized(S, pages, cache, bufs["attn"], bufs["y"], stream, drafts)
        self.mlp.up.norm_quantize(bufs["y"], stream_rows, self.w_mlp, self.eps, S, bufs["mlp"]["x"], stream)
        self.mlp.forward_quantized(S, bufs["mlp"], Y, OSC_Y_BF16, stream)
        return stream_rows


class Head:
    """Behind the last block: its output joins the residual stream, the final norm (w: [H] bf16), the projection onto the vocabulary, and
    from its logits log probabilities.  V: tokens that there are, if the projection has rows behind them."""

    def __init__(self, proj: Linear, w, eps: float = 1e-6, V: Optional[int] = None):
        self.proj, self.w, self.eps, self.V = proj, w, eps, proj.N if V is None else V
        if not 1 <= self.V <= proj.N:
            raise ValueError(f"{self.V} tokens from a projection of {proj.N} rows")

    def buffers(self, S: int, device, M: int = 0, K: int = 1):
        """For steps of up to S rows, with M given tokens a row and the K most likely ones."""
        t = self.proj.torch
        f32 = lambda *n: t.zeros(n, dtype=t.float32, device=device)
        # steps of fewer rows may need more of a workspace: rows are cut then
        ws = max((osc_logprobs_workspace(s, self.V, K) for s in range(1, min(S, 255) + 1)), default=0)
        return {"x": self.proj.act_buffers(S, device), "logits": t.empty((S, self.proj.N), dtype=t.bfloat16, device=device), "M": M, "K": K,
                "lp": f32(S, M), "ent": f32(S), "topv": f32(S, K), "topi": t.zeros((S, K), dtype=t.int32, device=device),
                "ws": t.empty((ws,), dtype=t.uint8, device=device)}

    def forward(self, X, res, S: int, bufs, stream=None) -> None:
        """X: [S, H] bf16, the last block's Y; res: the residual stream, updated in place (None: X is the stream).  Logits to
        bufs["logits"]."""
        self.proj.norm_quantize(X, res, self.w, self.eps, S, bufs["x"], stream)
        self.proj.gemm(bufs["x"], S, bufs["logits"], OSC_Y_BF16, stream)

    def logprobs(self, S: int, bufs, ids=None, scale: float = 1.0, stream=None) -> None:
        """Of p = softmax(scale logits): log p of the tokens ids (int32 [S, M] with the buffers' M, or more rows; None: without) to bufs["lp"],
        the entropy to bufs["ent"], the most likely tokens' log p and ids to bufs["topv"] and bufs["topi"] [S, K]."""
        M = bufs["M"] if ids is not None else 0
        if ids is not None and not isinstance(ids, int):  # too few rows are refused by the call
            n = ids.dim()
            if ids.shape[1] != M if n == 2 else n != 1 or M == 0 or (M > 1 and ids.numel() > S * M):
                raise ValueError(f"given tokens of shape {tuple(ids.shape)} where rows of {M} are read")
        osc_logprobs(bufs["logits"], OSC_Y_BF16, S, self.V, self.proj.N, scale, ids, M, bufs["K"], bufs["lp"], bufs["ent"], bufs["topv"],
                     bufs["topi"], bufs["ws"], stream)
