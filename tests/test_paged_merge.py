"""The split and merge of long caches: values whose mean jumps from one 64-key
stretch to the next under nearly equal weights, so that a tile or a record that
is lost, taken twice or weighed wrongly moves the answer by more than the
tolerance."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_norms as norms
import paged_plain as plain

# lens, hq, hkv, d, page, pages chosen (0: the 4-bit attention over all)
CASES = [
    ([30011], 4, 1, 128, 96, 0),
    ([17000, 0, 33, 23456, 1], 16, 2, 128, 128, 0),
    ([40000, 7], 24, 1, 64, 64, 0),
    ([25001, 12000], 2, 1, 32, 64, 0),
    ([20000, 9001], 8, 1, 256, 32, 0),
    ([33000], 8, 1, 128, 32, 900),
    ([30000, 5, 26000], 3, 1, 64, 64, 420),
    ([16000, 12000], 2, 1, 256, 32, 350),
    ([25000], 1, 1, 96, 96, 250),
]


SPAN = 512  # keys of a warp at most: all cases' tiles are dealt to 148 SMs of at least four warps


def _case(case, kind):
    lens, hq, hkv, d, page, top = CASES[case]
    c = plain.Cache(900 + case, kind, lens, hkv, d, page, poison=False)
    g = torch.Generator().manual_seed(case)
    for b, n in enumerate(lens):
        jump = torch.randint(0, 2, (hkv, (n + 63) // 64, 1), generator=g) * 16.0 - 8.0
        v = jump.repeat_interleave(64, 1)[:, :n] + 0.25 * torch.randn((hkv, n, d), generator=g)
        norms.repack(c, 0.5 * torch.randn((hkv, n, d), generator=g), v, b)
    q = (0.1 * torch.randn((len(lens) * hq, d), generator=g)).bfloat16()
    chosen = None
    if top:
        chosen = torch.full((len(lens), hkv, top), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            pages = -(-n // page)
            for h in range(hkv):
                few = min(top, pages)
                chosen[b, h, :few] = torch.randperm(pages, generator=g)[:few].int()
    return c, q, chosen


def _keys(c, chosen):
    def keys(b, g):
        n = c.lens[b]
        if chosen is None:
            return np.arange(n)
        at = [np.arange(p * c.page, min(n, (p + 1) * c.page)) for p in chosen[b, g].tolist() if p >= 0]
        return np.concatenate(at)
    return keys


def _reference(case, kind):
    lens, hq, hkv, d, page, top = CASES[case]
    c, q, chosen = _case(case, kind)
    some = [b for b, n in enumerate(lens) if n > 0]
    keys = _keys(c, chosen)
    qn = q.double().numpy().reshape(len(lens), hq, d)
    ref, tol = np.zeros(qn.shape), np.zeros(qn.shape)
    for b in some:
        one = plain.Cache.__new__(plain.Cache)
        one.__dict__.update(c.__dict__, table=c.table[b:b + 1], lens=[lens[b]])
        r, t = norms.attend(one, qn[b:b + 1], hq, lambda _, g, b=b: keys(b, g), 1 / math.sqrt(d), SPAN)
        ref[b], tol[b] = r[0], t[0]
    return c, q, chosen, keys, qn, ref, tol


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_lost_tile_would_show(case, kind):
    """On the oracle: a tile left out at the start, the middle or the end (of a selection a run of 32 keys) moves every
    long sequence's answer past the tolerance, in nearly every channel and by half of it or more."""
    lens, hq, hkv, d, page, top = CASES[case]
    if not top and kind != "int4":
        return
    c, _, _, keys, qn, ref, tol = _reference(case, kind)
    for b, n in enumerate(lens):
        if n < 1000:
            continue
        at = keys(b, 0)
        k, v = c.rows(b, 0, at)
        x = qn[b, 0] @ k.T / math.sqrt(d)
        w = np.exp(x - x.max())
        w /= w.sum()
        size = 32 if top else 64
        starts = np.flatnonzero(at % size == 0)
        for start in starts[[0, len(starts) // 2, -2]]:
            lost = slice(start, start + size)
            part = w[lost] @ v[lost]
            moved = np.abs((ref[b, 0] - part) / (1 - w[lost].sum()) - ref[b, 0])
            assert np.quantile(moved / tol[b, 0], 0.05) > 1.5, (b, start, np.median(moved / tol[b, 0]))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_split_and_merged(case, kind):
    from flashattention_attention_b200 import fa
    lens, hq, hkv, d, page, top = CASES[case]
    if not top and kind != "int4":
        return
    c, q, chosen, _, _, ref, tol = _reference(case, kind)
    c.cuda()
    kw = dict(hq=hq, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_)
    if top:
        out = fa.attention_decode_selected(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, chosen.cuda(), **kw)
    else:
        out = fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, **kw)
    p = fa.DecodeParams(kv_dtype=fa._CACHE_DT[c.kp.dtype], batch=len(lens), hq=hq, hkv=hkv, head_dim=d,
                        capacity=c.width * page)
    pages = fa.KvPages(None, c.width, page, c.num)
    assert fa.lib.fa_decode_pages_workspace_size(ctypes.byref(p), ctypes.byref(pages), top) > 0  # dealt, not clustered
    got = out.double().cpu().numpy().reshape(ref.shape)
    over = np.abs(got - ref) - tol
    assert over.max() <= 0, over.max()
    assert fa.check_device_error() == fa.FA_OK
