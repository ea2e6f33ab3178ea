"""What the Python binding of the calls between the projections takes and refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import poisoned  # noqa: E402
from test_gpu_paged import attend, build  # noqa: E402


@pytest.mark.parametrize("reqs,MB", [([(900, 1)], 40), ([(900, 70), (30, 30)], 40), ([(100, 100)], 2)])
def test_workspace_by_its_address(reqs, MB):
    p = build(reqs, 8, 2, 128, 64, 8, MB=MB)
    want = attend(p)
    ws = poisoned((osc.osc_attn_workspace(p["S"], p["R"], 8, 2, 128, 64, MB) + 16,), torch.uint8)
    assert torch.equal(attend(p, ws=ws.data_ptr()), want)
