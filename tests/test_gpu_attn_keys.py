"""Attention over the paged cache, key by key: queries of zero weigh all visible keys alike, and the values mark eight
neighbouring keys in a channel, so that each key left out or taken twice changes an output by an eighth, whatever
the context's length.  All keys are marked in turn."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402

RUN = 8  # keys marked in a channel


def check_every_key(reqs, HQ, HKV, D, page, room=0, pad=0, idle=0):
    """reqs: (keys, new tokens).  room: keys that the table's rows hold beyond the longest; pad: rows of the call that no
    request has; idle: requests without tokens."""
    reqs = list(reqs) + [(0, 0)] * idle
    R, n = len(reqs), sum(c for _, c in reqs)
    S, longest = n + pad, max(kv for kv, _ in reqs)
    need = [-(-kv // page) for kv, _ in reqs]
    MB, NP = -(-(longest + room) // page) + 1, sum(need) + 1
    ids = torch.randperm(NP, generator=torch.Generator().manual_seed(longest + n)).tolist()
    table = torch.full((R, MB), -1, dtype=torch.int32)
    where = []  # request and its keys' places in the cache
    for r, (kv, _) in enumerate(reqs):
        row, ids = ids[:need[r]], ids[need[r]:]
        table[r, :need[r]] = torch.tensor(row, dtype=torch.int32)
        key = torch.arange(kv)
        where.append((torch.tensor(row + [0], device=DEV)[key.to(DEV) // page], (key % page).to(DEV)))
    cu = np.concatenate([[0], np.cumsum([c for _, c in reqs])])
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32).to(DEV)
    table, cu_d, kv_d = table.to(DEV), i32(cu), i32([kv for kv, _ in reqs])
    g = torch.Generator(device=DEV).manual_seed(n)
    KC = torch.randn((NP, HKV, page, D), generator=g, device=DEV).bfloat16()
    VC = torch.full((NP, HKV, D, page), float("nan"), dtype=torch.bfloat16, device=DEV)
    Q = torch.zeros((S, HQ, D), dtype=torch.bfloat16, device=DEV)
    ws = poisoned((osc.osc_attn_workspace(S, R, HQ, HKV, D, page, MB),), torch.uint8)
    seen = torch.cat([torch.arange(kv - c, kv) + 1 for kv, c in reqs]).to(DEV)  # keys of each row
    mark = torch.tensor([1.0, -2.0, 0.5, 4.0], device=DEV)[:min(HKV, 4)].bfloat16()  # of each key head
    heads = mark[torch.arange(HKV, device=DEV) % len(mark)]
    channel = torch.arange(D, device=DEV)
    for first in range(0, longest, RUN * D):
        for id, off in where:
            k = torch.arange(len(id), device=DEV) - first
            hit = (k[:, None] // RUN == channel[None]).bfloat16()  # [keys, D]
            VC[id, :, :, off] = hit[:, None, :] * heads[None, :, None]
        O = poisoned((S, HQ, D), torch.bfloat16)
        osc.osc_attn_paged(Q, KC, VC, S, R, HQ, HKV, D, page, MB, NP, table, cu_d, kv_d, D ** -0.5, O, ws)
        count = (seen[:, None] - first - channel[None] * RUN).clamp(0, RUN).double()  # marked keys that a row sees
        ref = (count / seen[:, None].double())[:, None, :] * heads.double().repeat_interleave(HQ // HKV)[None, :, None]
        # weights of 1 and their sums are exact; the quotient is rounded in binary32 twice and to bf16 once
        bad = (O[:n].double() - ref).abs() > (2.0 ** -8 + 2.0 ** -20) * ref.abs()
        assert not bool(bad.any()), (first, [v.tolist() for v in torch.nonzero(bad)[:3]])
        assert bool((O[n:].view(torch.int16) == -1).all())


DECODES = [[(1, 1)], [(5000, 1)], [(20000, 1)], [(5000, 1), (17, 1), (1, 1), (2048, 1)], [(k, 1) for k in range(1, 1500, 49)]]


@pytest.mark.parametrize("reqs", DECODES)
@pytest.mark.parametrize("HQ,HKV,D,page,room", [(4, 1, 64, 64, 0), (6, 3, 128, 16, 30000), (32, 8, 128, 256, 30000), (17, 1, 64, 16, 0)])
def test_decodes(reqs, HQ, HKV, D, page, room):
    check_every_key(reqs, HQ, HKV, D, page, room)


CHUNKS = [[(5000, 33)], [(20000, 20)], [(300, 300)], [(1000, 1000)], [(2200, 2200)], [(500, 500)] * 2, [(300, 300)] * 3, [(100, 100)] * 20,
          [(2344, 1024), (8711, 765), (5186, 900), (1103, 500)], [(9000, 300), (64, 64), (1, 1), (700, 0)], [(4100, 4000), (12000, 1)]]


@pytest.mark.parametrize("reqs", CHUNKS)
@pytest.mark.parametrize("HQ,HKV,D,page", [(8, 1, 64, 64), (6, 3, 128, 16), (32, 8, 128, 64)])
@pytest.mark.parametrize("room", [0, 40000])
def test_chunks_and_prompts(reqs, HQ, HKV, D, page, room):
    check_every_key(reqs, HQ, HKV, D, page, room)


@pytest.mark.parametrize("reqs,pad", [([(5000, 1)], 4000), ([(20000, 1)], 300), ([(5000, 1)], 8191), ([(700, 1), (9000, 2)], 5000), ([(1, 1)], 2100),
                                      ([(3000, 1000)], 3000)])
@pytest.mark.parametrize("HQ,HKV,D,page", [(8, 1, 64, 64), (32, 8, 128, 64)])
@pytest.mark.parametrize("room,idle", [(0, 0), (40000, 0), (40000, 3)])
def test_calls_with_room_for_more_rows(reqs, pad, HQ, HKV, D, page, room, idle):
    check_every_key(reqs, HQ, HKV, D, page, room, pad, idle)


@pytest.mark.parametrize("reqs", [[(130, 2)] * 300, [(40, 1)] * 290 + [(700, 400)] * 2, [(500, 1), (0, 0)] * 150 + [(4000, 300)]])
@pytest.mark.parametrize("HQ,HKV,D", [(8, 1, 64), (32, 8, 128)])
@pytest.mark.parametrize("room", [0, 40000])
def test_more_tiles_than_workgroups(reqs, HQ, HKV, D, room):
    check_every_key(reqs, HQ, HKV, D, 64, room)


@pytest.mark.parametrize("HQ,HKV", [(40, 40), (600, 300), (1024, 1), (1024, 1024)])
@pytest.mark.parametrize("reqs,room", [([(900, 1), (33, 1)], 0), ([(900, 3), (70, 70)], 0), ([(900, 3), (70, 70)], 9000), ([(1100, 9)], 9000)])
def test_many_heads(HQ, HKV, reqs, room):
    check_every_key(reqs, HQ, HKV, 64, 16, room)


@pytest.mark.parametrize("seed", range(24))
def test_any_lengths(seed):
    rng = np.random.default_rng(seed)
    HQ, HKV = [(8, 1), (6, 3), (32, 8), (4, 4), (40, 2)][seed % 5]
    reqs = []
    for _ in range(int(rng.integers(1, 10))):
        kv = int(np.exp(rng.uniform(0, np.log(9000))))
        reqs.append((kv, int(rng.choice([0, 1, min(kv, 33), int(rng.integers(0, min(kv, 1200) + 1))]))))
    reqs.append((50, 3))
    check_every_key(reqs, HQ, HKV, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256])), int(rng.choice([0, 30000])))


@pytest.mark.parametrize("reqs", [[(9000, 1)], [(5000, 40)], [(700, 700)]])
@pytest.mark.parametrize("HQ,HKV,D", [(32, 8, 128), (8, 1, 64)])
def test_room_for_more_rows_changes_no_bit(reqs, HQ, HKV, D):
    """A call's rows without a token neither change how the others' work is cut, nor the results."""
    (kv, n), page, MB = reqs[0], 64, 640
    g = torch.Generator(device=DEV).manual_seed(kv)
    NP = -(-kv // page)
    KC, VC = (torch.randn((NP, HKV, page * D), generator=g, device=DEV).bfloat16() for _ in range(2))
    Q = torch.randn((8192, HQ, D), generator=g, device=DEV).bfloat16()
    table = torch.full((1, MB), -1, dtype=torch.int32, device=DEV)
    table[0, :NP] = torch.arange(NP, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    got = []
    for S in (max(n, 2), n + 300, 8192):
        O = poisoned((S, HQ, D), torch.bfloat16)
        ws = poisoned((osc.osc_attn_workspace(S, 1, HQ, HKV, D, page, MB),), torch.uint8)
        osc.osc_attn_paged(Q, KC, VC, S, 1, HQ, HKV, D, page, MB, NP, table, i32(0, n), i32(kv), D ** -0.5, O, ws)
        got.append(O[:n])
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])
