"""Residual add + RMS norm (osc_rmsnorm) against the formula in 64 bits, and osc_rmsnorm_quant bit for
bit against the oracle's quantization of osc_rmsnorm's rows."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import w4a4_outlier_split_amd as osc  # noqa: E402
from gpu_util import DEV, _tiled_outputs, codes6_rm, codes_rm, host_bits16, poisoned, scales_rm, side_rm  # noqa: E402

EPS = 1e-6
# y is rounded once: half a bf16 step (2^-8 of the value).  Ahead of that, in steps of 2^-24: the sum of
# squares is at most 256 sequential additions of a lane and 8 across lanes, half of whose relative error
# reaches the root; division, root, reciprocal and the two products add 5: under 140 * 2^-24 < 2^-16.
Y_REL = 2.0 ** -8 + 2.0 ** -16


def inputs(S, H, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *n: torch.randn(n, generator=g, device=DEV)
    gain = torch.ones(H, device=DEV)
    gain[::37] = 40.0
    return ((r(S, H) * spread).bfloat16(), (r(S, H) * gain * spread).bfloat16(), (1 + 0.2 * r(H)).bfloat16())


def rmsnorm(x, res, w, eps=EPS, in_place=False):
    S, H = x.shape
    y = poisoned((S, H), torch.bfloat16)
    out = None if res is None else res.clone() if in_place else poisoned((S, H), torch.bfloat16)
    osc.osc_rmsnorm(x, out if in_place else res, w, S, H, eps, out, y)
    return out, y


def check_y(y, r, w, eps=EPS):
    rd = r.double()
    ref = rd / torch.sqrt((rd * rd).mean(1, keepdim=True) + eps) * w.double()
    err = (y.double() - ref).abs()
    assert bool((err <= Y_REL * ref.abs() + 2.0 ** -133).all()), float((err / (Y_REL * ref.abs() + 2.0 ** -133)).max())


@pytest.mark.parametrize("S", [1, 3, 77, 2050])
@pytest.mark.parametrize("H", [256, 1024, 4096, 4352, 8192])
def test_rmsnorm(S, H):
    x, res, w = inputs(S, H, S + H)
    for in_place in (False, True):
        out, y = rmsnorm(x, res, w, in_place=in_place)
        r = (x.float() + res.float()).bfloat16()
        assert torch.equal(out, r)
        check_y(y, r, w)
    _, y = rmsnorm(x, None, w)
    check_y(y, x, w)


@pytest.mark.parametrize("H", [8448, 32768, 65536])
def test_rmsnorm_wide_rows(H):
    x, res, w = inputs(5, H, H)
    out, y = rmsnorm(x, res, w)
    r = (x.float() + res.float()).bfloat16()
    assert torch.equal(out, r)
    check_y(y, r, w)


def test_rmsnorm_zero_tiny_and_large_rows():
    x = torch.zeros(6, 512, dtype=torch.bfloat16, device=DEV)
    x[1], x[2], x[3] = 1e-30, 1e17, 2.0 ** -140
    x[4, 100], x[5, ::2] = 7.0, -0.0
    w = inputs(1, 512, 5)[2]
    for eps in (1e-6, 1e-30):
        _, y = rmsnorm(x, None, w, eps)
        check_y(y, x, w, eps)
        assert bool((y[0] == 0).all())


def check_quant(S, H, G, fmt, m, seed, with_res=True):
    x, res, w = inputs(S, H, seed)
    if not with_res:
        res = None
    L = None
    if m:
        rng = np.random.default_rng(seed)
        L = np.stack([rng.choice(G, m, replace=False) for _ in range(H // G)]).astype(np.int32)
        L[rng.random(H // G) < 0.25, -1] = -1
    Q, SC, B = _tiled_outputs(S, H, G, fmt, m > 0, max(m, 1))
    out = None if res is None else poisoned((S, H), torch.bfloat16)
    osc.osc_rmsnorm_quant(x, res, w, S, H, EPS, G, L, max(m, 1), fmt, out, Q, SC, B)
    ref_out, y = rmsnorm(x, res, w)
    if res is not None:
        assert torch.equal(out, ref_out)
    # the device's own quantization of y, byte for byte (unwritten places keep the poison on both sides)
    Q2, SC2, B2 = _tiled_outputs(S, H, G, fmt, m > 0, max(m, 1))
    osc.osc_quant_act_multi(y, S, H, G, L, max(m, 1), fmt, Q2, SC2, B2)
    assert torch.equal(Q, Q2) and torch.equal(SC, SC2) and (B is None or torch.equal(B, B2))
    if fmt == osc.OSC_FP6P:
        return
    yb = host_bits16(y.view(torch.int16))
    if m:
        rq, rs, rb = oracle.quant_act_multi(yb, G, L, m, fmt)
        np.testing.assert_array_equal(side_rm(B, S, H, G, m), rb)
    else:
        rq, rs, _ = oracle.quant_act(yb, G, None, fmt)
    np.testing.assert_array_equal(codes_rm(Q, S, H, fmt), rq)
    np.testing.assert_array_equal(scales_rm(SC, S, H, G), rs)


@pytest.mark.parametrize("S", [1, 37, 2049])
@pytest.mark.parametrize("G,fmt,m", [(32, 0, 0), (32, 0, 1), (16, 0, 2), (64, 0, 1), (64, 0, 3), (32, 1, 0), (64, 1, 0), (16, 1, 0),
                                     (16, 2, 0), (16, 2, 1), (16, 2, 3)])
def test_rmsnorm_quant(S, G, fmt, m):
    check_quant(S, 1024, G, fmt, m, S + G + m)


@pytest.mark.parametrize("S,H,G,fmt,m", [(16, 4096, 32, 0, 1), (2048, 4096, 32, 1, 0), (2500, 8192, 64, 0, 2), (3, 16384, 32, 0, 1),
                                         (2, 65536, 64, 1, 0), (4, 256, 16, 0, 1)])
def test_rmsnorm_quant_shapes(S, H, G, fmt, m):
    check_quant(S, H, G, fmt, m, H + S, with_res=S != 2500)


def test_rows_behind_the_last_stay_as_they_were():
    S, H = 2049, 512
    x, res, w = inputs(S + 3, H, 9)
    y, out = poisoned((S + 3, H), torch.bfloat16), poisoned((S + 3, H), torch.bfloat16)
    osc.osc_rmsnorm(x, res, w, S, H, EPS, out, y)
    assert bool((y[S:].view(torch.int16) == -1).all()) and bool((out[S:].view(torch.int16) == -1).all())


def test_binding_refuses_strided_short_and_host_tensors():
    x, res, w = inputs(8, 512, 1)
    y = poisoned((8, 512), torch.bfloat16)
    wide = poisoned((8, 1024), torch.bfloat16)
    for bad in ((wide[:, :512], res, w, res, y), (x[:4], res, w, res, y), (x, res.cpu(), w, res, y), (x, res, w[:256], res, y),
                (x, res, w, res, wide[:, ::2])):
        with pytest.raises(osc.OscError) as e:
            osc.osc_rmsnorm(bad[0], bad[1], bad[2], 8, 512, EPS, bad[3], bad[4])
        assert e.value.status == 2
