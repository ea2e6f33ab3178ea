"""Operands of the calls between the projections that share bytes with an output are refused before any HIP call, so the
fake addresses are never touched.  No GPU needed."""
import pytest

osc = pytest.importorskip("w4a4_outlier_split_amd", reason="libosc.so not built")

BASE, STEP = 1 << 40, 1 << 32  # operands apart from each other
S, H, HQ, HKV, D, PAGE, NP, MB, R, F, T, P = 8, 512, 4, 2, 64, 16, 9, 5, 3, 9, 8, 32
ROWS = 2 * S * H
CACHE = 2 * NP * HKV * PAGE * D

# call, its operands with their bytes (sizes and the like as they are), the outputs, pairs that may be one
CALLS = {
    "osc_rmsnorm": ([("X", ROWS), ("RES", ROWS), ("W", 2 * H), S, H, 1e-6, ("RES_OUT", ROWS), ("Y", ROWS)], ("RES_OUT", "Y"),
                    ("RES", "RES_OUT")),
    "osc_rmsnorm_quant": ([("X", ROWS), ("RES", ROWS), ("W", 2 * H), S, H, 1e-6, 32, None, 1, osc.OSC_MXFP8, ("RES_OUT", ROWS), ("QX", S * H),
                           ("SX", S * H // 32), None], ("RES_OUT", "QX", "SX"), ("RES", "RES_OUT")),
    "osc_page_plan": ([("CTX", 4 * R), ("NEW", 4 * R), R, PAGE, NP, ("FREE", 4 * F), F, ("HEAD", 4), T, ("TABLE", 4 * R * MB), MB,
                       ("CU", 4 * R + 4), ("KV", 4 * R), ("SLOT", 4 * T), ("POS", 4 * T), ("USED", 4)],
                      ("TABLE", "CU", "KV", "SLOT", "POS", "USED"), ()),
    "osc_qkv_append": ([("QKV", 2 * S * (HQ + 2 * HKV) * D), S, HQ, HKV, D, ("WQ", 2 * D), ("WK", 2 * D), 1e-6, ("CS", 4 * P * D), P,
                        ("POS", 4 * S), ("SLOT", 4 * S), ("Q", 2 * S * HQ * D), ("KC", CACHE), ("VC", CACHE), NP, PAGE],
                       ("Q", "KC", "VC"), ()),
    "osc_attn_paged": ([("Q", 2 * S * HQ * D), ("KC", CACHE), ("VC", CACHE), S, R, HQ, HKV, D, PAGE, 600, NP, ("TABLE", 4 * R * 600),
                        ("CU", 4 * R + 4), ("KV", 4 * R), 0.1, ("O", 2 * S * HQ * D), ("WS", None), 1 << 40], ("O", "WS"), ())}


@pytest.mark.parametrize("name", CALLS)
def test_an_output_shares_no_bytes(name):
    args, outs, one = CALLS[name]
    if name == "osc_attn_paged":
        need = osc.osc_attn_workspace(S, R, HQ, HKV, D, PAGE, 600)
        assert need > 0
        args = [("WS", need) if a == ("WS", None) else a for a in args]
    size = dict(a for a in args if isinstance(a, tuple))
    at = {k: BASE + i * STEP for i, k in enumerate(size)}

    def status(**moved):
        where = {**at, **moved}
        return getattr(osc._lib, name)(*[where[a[0]] if isinstance(a, tuple) else a for a in args], None)

    for o in outs:
        for k in size:
            # k on o's first bytes, on its last, and k's last bytes on o's first (16-byte steps)
            for d in {0, (size[o] - 1) // 16 * 16, -((size[k] - 1) // 16 * 16)}:
                if k != o and not (d == 0 and {o, k} == set(one)):  # updated in place: allowed
                    assert status(**{k: at[o] + d}) == 2, (o, k, d)


def test_in_place_is_for_the_residual_alone():
    at = lambda i: BASE + i * STEP
    lib = osc._lib
    # X on RES_OUT, with the residual updated in place and not
    assert lib.osc_rmsnorm(at(0), at(0), at(1), S, H, 1e-6, at(0), at(2), None) == 2
    assert lib.osc_rmsnorm(at(0), at(3), at(1), S, H, 1e-6, at(0), at(2), None) == 2
    # the residual shifted by a row against its output
    assert lib.osc_rmsnorm(at(0), at(3), at(1), S, H, 1e-6, at(3) + 2 * H, at(2), None) == 2
    # without a residual, the written rows on X
    assert lib.osc_rmsnorm(at(0), None, at(1), S, H, 1e-6, None, at(0), None) == 2
