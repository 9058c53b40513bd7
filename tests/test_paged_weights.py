"""GPU tests of the quantised paged attention where weights and V's steps differ
by many powers of two, with tolerances that follow the answer and not the
widest row."""
import math

import numpy as np
import pytest
import torch

import paged_norms as norms
import paged_plain as plain

pytestmark = pytest.mark.gpu


def _sink_cache(kind, n, hkv, d, page, gap_bits, wide, seed=0):
    """Key 0 weighs 2^gap_bits times an ordinary key, key 1's V is `wide` times as wide as the others', and every V
    channel has a mean of its own (centred by the channels of a row: the rows' middle is not the channels' mean)."""
    g = torch.Generator().manual_seed(seed)
    c = plain.Cache(seed, kind, [n], hkv, d, page, poison=False)
    q = torch.full((1, hkv, d), 0.5)
    k = torch.randn((hkv, n, d), generator=g)
    k[:, 0] = gap_bits * math.log(2) * math.sqrt(d) / (0.5 * d)
    v = torch.randn((hkv, n, d), generator=g) + 2 * torch.randn((hkv, 1, d), generator=g)
    v[:, 0] = torch.randn((hkv, d), generator=g)
    v[:, 1] = wide * torch.randn((hkv, d), generator=g)
    return norms.repack(c, k, v), q.bfloat16()


def _many(c, q, batch):
    """Queries, lengths, table and a selection of every page for `batch` sequences that are all the cache's first one."""
    return (q[0].cuda().repeat(batch, 1), c.lens_.repeat(batch), c.table_.repeat(batch, 1),
            torch.arange(c.width, dtype=torch.int32, device="cuda").repeat(batch, c.hkv, 1))


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("gap_bits,wide", [(18, 64), (20, 64), (22, 1024), (14, 2 ** 14)])
def test_small_weights_after_a_sink_and_a_wide_row(kind, gap_bits, wide):
    """A key that weighs 2^14 to 2^22 others and a row of wide values come first; tens of thousands of keys follow whose
    weights are small beside theirs but whose sum is not.  More (sequence, head) pairs than warps: a warp serves most
    of a sequence."""
    from flashattention_attention_b200 import fa
    n, hkv, d, page, batch = 32768, 2, 64, 64, 1000
    c, q = _sink_cache(kind, n, hkv, d, page, gap_bits, wide)
    c.cuda()
    qs, lens, table, every = _many(c, q, batch)
    kw = dict(hq=hkv, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_)
    if kind == "int4":
        out = fa.attention_decode_paged(qs, c.kp_, c.vp_, lens, table, **kw)
    else:
        out = fa.attention_decode_selected(qs, c.kp_, c.vp_, lens, table, every, **kw)
    ref, tol = norms.attend(c, q.double().numpy(), hkv, lambda b, g: np.arange(n), 1 / math.sqrt(d))
    # per head, in the L2 norm (most channels' error is far below their bound)
    err = np.linalg.norm(out.double().cpu().numpy().reshape(batch, hkv, d) - ref, axis=-1)
    bound = np.linalg.norm(tol, axis=-1)
    size = np.linalg.norm(ref, axis=-1)
    assert (bound <= 0.02 * size).all()  # the tolerance does not follow the widest row
    assert (err <= bound).all(), (err / size).max()
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_weights_that_fall_and_rise_along_the_cache(kind):
    """Logits that wander over some 60 powers of two, V steps over 40 others: the unit of the weights goes up and down
    again, and the accumulators with it."""
    from flashattention_attention_b200 import fa
    n, hkv, d, page, batch = 4096, 1, 128, 32, 600  # enough sequences that a warp serves a third of one
    g = torch.Generator().manual_seed(7)
    c = plain.Cache(7, kind, [n], hkv, d, page, poison=False)
    q = torch.full((1, 4, d), 0.25) * torch.tensor([1.0, -1.0, 0.5, 0.01])[:, None]
    at = torch.arange(n)
    k = torch.randn((hkv, n, d), generator=g) + (8 * torch.sin(at / 150.0))[None, :, None]
    v = torch.randn((hkv, n, d), generator=g) * torch.exp2(20 * torch.sin(at / 77.0))[None, :, None]
    norms.repack(c, k, v).cuda()
    kw = dict(hq=4, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_)
    qs, lens, table, every = _many(c, q.bfloat16(), batch)
    outs = [fa.attention_decode_selected(qs, c.kp_, c.vp_, lens, table, every, **kw)]
    if kind == "int4":
        outs.append(fa.attention_decode_paged(qs, c.kp_, c.vp_, lens, table, **kw))
    ref, tol = norms.attend(c, q.bfloat16().double().numpy(), 4, lambda b, g: np.arange(n), 1 / math.sqrt(d))
    for out in outs:
        over = np.abs(out.double().cpu().numpy().reshape(batch, 4, d) - ref) - tol
        assert over.max() <= 0, over.max()
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("gain", [2.0 ** -110, 2.0 ** 118])
@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_steps_at_the_ends_of_fp32(kind, gain):
    """V's steps near the ends of fp32's range, in a tile of their own and after ordinary ones."""
    from flashattention_attention_b200 import fa
    n, d, page, batch = 1024, 64, 32, 1000
    for ordinary in (0, 64):
        c = plain.Cache(9, kind, [n], 1, d, page, poison=False)
        at = np.arange(ordinary, n)
        p, o = c.table[0].numpy()[at // page], at % page
        c.vs[p, :, o] = c.vs[p, :, o] * gain
        c.cuda()
        q = torch.randn((1, 2, d), generator=torch.Generator().manual_seed(3)).bfloat16()
        qs, lens, table, every = _many(c, q, batch)
        out = fa.attention_decode_selected(qs, c.kp_, c.vp_, lens, table, every, hq=2, hkv=1, k_scales=c.ks_, v_scales=c.vs_)
        ref, tol = norms.attend(c, q.double().numpy(), 2, lambda b, g: np.arange(n), 1 / math.sqrt(d))
        assert (np.abs(out.double().cpu().numpy().reshape(batch, 2, d) - ref) <= tol).all()
