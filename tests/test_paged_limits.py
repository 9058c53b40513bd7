"""GPU test of the 4-bit paged attention at the largest lengths."""
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def test_lengths_next_to_two_to_the_31():
    """A table of 8193 entries that all name one page of 262112 keys: lengths up to 2^31 - 32, of which a window is
    attended, or the last page."""
    from flashattention_attention_b200 import fa
    page, width, d, hq = 32 * 8191, 8193, 64, 2
    top = page * width
    assert top == 2 ** 31 - 32
    lens = [top, top - 1, top - 31, top - 32, top - 63, top - 64, 40]
    c = plain.Cache(600, "int4", [page], 1, d, page, poison=False, spare=0)
    c.lens, c.width, c.table = lens, width, torch.zeros((len(lens), width), dtype=torch.int32)
    c.cuda()
    q = torch.randn((len(lens) * hq, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    qn = q.double().numpy().reshape(len(lens), hq, d)
    kw = dict(hq=hq, hkv=1, k_scales=c.ks_, v_scales=c.vs_)
    for window in (1, 64, 1000):
        out = fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, window=window, **kw)
        ref, tol = plain.attend(c, qn, hq, lambda b, g: np.arange(max(0, lens[b] - window), lens[b]), 1 / math.sqrt(d))
        assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    c.bounds_ = torch.stack([c.bounds_[:, :, 0], c.bounds_[:, :, 1]], 2)
    sel = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=hq, hkv=1, page_size=page, top_k=1, n_first=0, n_recent=1)
    assert sel.flatten().tolist() == [(n - 1) // page for n in lens]
    assert fa.check_device_error() == fa.FA_OK
