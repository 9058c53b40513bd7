"""GPU test of the 4-bit paged attention with a window: only the pages that hold
attended keys are looked up, so the table's entries in front of them may name
no page."""
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 64, 96])
@pytest.mark.parametrize("window,long", [(1, 0), (33, 0), (100, 0), (640, 9000), (30001, 70000)])
def test_pages_in_front_of_the_window_are_not_looked_up(page, d, window, long):
    """Lengths that put the window's first key anywhere in a tile; with a long sequence the tiles are dealt over the
    device.  Entries in front of the window's first page: outside the pool."""
    from flashattention_attention_b200 import fa
    lens = [100, 1, window + 31, long, 0] if long else [100, 1, window, window + 1, window + 31, window + 32, window + 33,
                                                        window + 64, 0, 799]
    hq, hkv = 4, 1 if long else 2
    c = plain.Cache(500 + page, "int4", lens, hkv, d, page)
    for b, n in enumerate(lens):
        c.table[b, :max(0, n - window) // page] = -1 if b % 2 else c.num
    c.cuda()
    q = (torch.randn((len(lens) * hq, d), generator=torch.Generator().manual_seed(page)) * 1.5).bfloat16()
    out = fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, hq=hq, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_,
                                    window=window)
    assert fa.check_device_error() == fa.FA_OK
    ref, tol = plain.attend(c, q.double().numpy().reshape(len(lens), hq, d), hq,
                            lambda b, g: np.arange(max(0, lens[b] - window), lens[b]), 1 / math.sqrt(d))
    assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
