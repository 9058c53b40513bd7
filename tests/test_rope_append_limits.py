"""GPU tests of the rotated paged append at the ends of what it accepts."""
import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_rows_of_the_widest_ranges():
    """4-bit rows whose range times 15 passes fp32's largest number: every code is the nearest of the sixteen in 64 bits
    (no element of these rows is within an fp32 rounding of two codes' middle)."""
    from flashattention_attention_b200 import fa
    d = 64
    unit = torch.linspace(0, 1, d, dtype=torch.float64)
    rows = torch.stack([unit * 3e38, unit * 3e38 - 1.5e38, unit.flip(0) * 1e38 - 2e38, unit * 2.5e37, unit * 2.2e37 - 1e37,
                        torch.where(unit > 0.5, 1.0, -1.0) * 1.6e38]).float()[:, None]
    c = plain.Cache(700, "int4", [len(rows)], 1, d, 16, poison=False).cuda()
    fa.kv_append_rope_paged(rows.cuda(), rows.cuda(), c.kp_, c.vp_, _i32(0), c.table_, k_scales=c.ks_, v_scales=c.vs_,
                            cu_seqlens=_i32(0, len(rows)))
    assert fa.check_device_error() == fa.FA_OK
    p = int(c.table[0, 0])
    x = rows[:, 0].double().numpy()
    lo, r = x.min(-1, keepdims=True), x.max(-1, keepdims=True) - x.min(-1, keepdims=True)
    exact = 15 * (x - lo) / r
    assert np.abs(exact - np.floor(exact) - 0.5).min() > 1e-4
    for pool, scales in ((c.kp_, c.ks_), (c.vp_, c.vs_)):
        assert np.array_equal(plain.unpack4(pool[p, 0, : len(rows)].cpu().numpy()), np.rint(exact).astype(np.uint8))
        step, low = scales[p, 0, : len(rows)].double().cpu().numpy().T
        assert np.array_equal(low, lo[:, 0])
        assert (np.abs(step - r[:, 0] / 15) <= 2.0 ** -23 * r[:, 0] / 15).all()  # the range and the quotient, rounded


@pytest.mark.parametrize("bounds", [False, True])
def test_tokens_past_the_rotation_table_do_not_count(bounds):
    """A sequence whose new tokens pass the table's last row keeps its old length, as one that passes the capacity does;
    without a rotation, or without a new token, there is no table to pass."""
    from flashattention_attention_b200 import fa
    c = plain.Cache(701, "int8", [64] * 5, 2, 64, 32, poison=False).cuda()
    x = torch.randn((9, 2, 64), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    cur, cu = _i32(10, 9, 11, 12, 62), _i32(0, 3, 6, 7, 7, 9)

    def call(rope):
        lens = torch.full((5,), -1, dtype=torch.int32, device="cuda")
        fa.kv_append_rope_paged(x, x, c.kp_, c.vp_, cur, c.table_, rope_table=rope, k_scales=c.ks_, v_scales=c.vs_,
                                key_bounds=c.bounds_ if bounds else None, cu_seqlens=cu, cache_seqlens=lens)
        return lens.tolist(), fa.check_device_error()

    # slots 10 .. 12, 9 .. 11, 11, none (at 12), 62 .. 63; the table ends with position 11
    assert call(fa.rope_table(12, 64).cuda()) == ([-1, 12, 12, 12, -1], fa.FA_ERR_INVALID)
    assert call(fa.rope_table(64, 64).cuda()) == ([13, 12, 12, 12, 64], fa.FA_OK)
    assert call(None) == ([13, 12, 12, 12, 64], fa.FA_OK)
