"""Single tokens over the paged cache: nothing of a softmax weight is lost ahead of the second product but what two bf16
leave out, so the output's own rounding is all that counts."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_util import DEV  # noqa: E402
from test_gpu_paged import attend, build  # noqa: E402


@pytest.mark.parametrize("HQ,HKV,D,page", [(32, 8, 128, 64), (4, 4, 64, 16), (17, 1, 128, 256)])
@pytest.mark.parametrize("reqs", [[(2, 1), (3, 1), (7, 1), (40, 1)], [(130, 1), (600, 1), (0, 0)], [(3000, 1)] * 3, [(9000, 1)]])
def test_decode_weights(HQ, HKV, D, page, reqs):
    p = build(reqs, HQ, HKV, D, page, HQ + len(reqs))
    got, g, t = attend(p).double(), HQ // HKV, 0
    for r, (kv, n) in enumerate(reqs):
        if not n:
            continue
        key = torch.arange(kv, device=DEV)
        ids, off = torch.tensor(p["table"][r], device=DEV)[key // page], key % page
        for h in range(HKV):
            k, v = p["KC"][ids, h, off].double(), p["VC"][ids, h, :, off].double()
            q = p["Q"][t, h * g:(h + 1) * g].double()
            w = torch.softmax(q @ k.T * p["scale"], 1)
            ref, size = w @ v, (q.abs() @ k.abs().T * p["scale"]).amax(1, keepdim=True)
            # Two bf16 hold a weight to 2^-8 of 2^-8 of it; scores and exponents as D products of the terms' size in binary32
            # (2^-24 each), the sums as much again; the output is rounded to bf16 (2^-8 of it).
            tol = (2.0 ** -16 + 2 * 2.0 ** -24 * (D * size + 64)) * (w @ v.abs()) + 2.0 ** -8 * ref.abs()
            assert bool(((got[t, h * g:(h + 1) * g] - ref).abs() <= tol).all()), (r, h)
        t += 1
