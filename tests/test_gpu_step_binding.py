"""What the Python binding of the calls between the projections takes and refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, poisoned  # noqa: E402
from test_gpu_paged import attend, build  # noqa: E402


@pytest.mark.parametrize("reqs,MB", [([(900, 1)], 40), ([(900, 70), (30, 30)], 40), ([(100, 100)], 2)])
def test_workspace_by_its_address(reqs, MB):
    p = build(reqs, 8, 2, 128, 64, 8, MB=MB)
    want = attend(p)
    ws = poisoned((osc.osc_attn_workspace(p["S"], p["R"], 8, 2, 128, 64, MB) + 16,), torch.uint8)
    assert torch.equal(attend(p, ws=ws.data_ptr()), want)


def refused(f, args, i, t):
    with pytest.raises(osc.OscError) as e:
        f(*[t if j == i else a for j, a in enumerate(args)])
    assert e.value.status == 5, i


def test_elements_of_another_type_are_refused():
    """Long enough in bytes, they would be read as what they are not; bits of bf16 in 16-bit integers are taken."""
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)
    S, H, HQ, HKV, D, page, NP, MB, R, P = 4, 512, 4, 2, 64, 16, 3, 2, 2, 8
    cache = lambda: bf(NP, HKV, page, D)
    calls = [
        (osc.osc_rmsnorm, [bf(S, H), bf(S, H), bf(H), S, H, 1e-6, bf(S, H), bf(S, H)]),
        (osc.osc_rmsnorm_quant, [bf(S, H), bf(S, H), bf(H), S, H, 1e-6, 32, [-1] * (H // 32), 1, osc.OSC_MXFP4, bf(S, H), u8(S * H // 2),
                                 u8(S * H // 32), bf(S, 32)]),
        (osc.osc_page_plan, [i32(R), i32(R), R, page, NP, i32(NP), NP, i32(1), S, i32(R, MB), MB, i32(R + 1), i32(R), i32(S), i32(S), i32(1)]),
        (osc.osc_qkv_append, [bf(S, (HQ + 2 * HKV) * D), S, HQ, HKV, D, bf(D), bf(D), 1e-6, i32(P, D).float(), P, i32(S), i32(S) - 1,
                              bf(S, HQ, D), cache(), cache(), NP, page]),
        (osc.osc_attn_paged, [bf(S, HQ, D), cache(), cache(), S, R, HQ, HKV, D, page, MB, NP, i32(R, MB), i32(R + 1), i32(R), 0.1,
                              bf(S, HQ, D), None])]
    for f, args in calls:
        f(*args)
        for i, a in enumerate(args):
            if not torch.is_tensor(a) or a.dtype == torch.uint8:
                continue
            others = {torch.bfloat16: (torch.float32, torch.float16, torch.float64), torch.int32: (torch.int64, torch.float32),
                      torch.float32: (torch.float64, torch.bfloat16)}[a.dtype]
            for t in others:
                refused(f, args, i, torch.zeros(a.numel() * 2, dtype=t, device=DEV))
            if a.dtype == torch.bfloat16:
                f(*[x.view(torch.int16) if x is a else x for x in args])


def test_block_refuses_an_output_inside_its_inputs():
    from test_gpu_block_step import H, T, make_block, make_pages
    b, pages = make_block(51, "osc"), make_pages()
    both = torch.zeros((2 * T, H), dtype=torch.bfloat16, device=DEV)
    x, res = both[:T], both[T:]
    for y in (x, x.view(-1).view(T, H), both[1:T + 1], res, both[T - 1:2 * T - 1]):
        with pytest.raises(ValueError):
            b.forward(x, res, T, pages, None, None, y)
    with pytest.raises(ValueError):
        b.forward(x, None, T, pages, None, None, both[T - 1:2 * T - 1])
    with pytest.raises(ValueError):
        b.forward(x.data_ptr(), None, T, pages, None, None, x)
