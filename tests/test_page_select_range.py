"""GPU test of the page selection where products or sums leave fp32's range."""
import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _select(bounds, q, pages, hq, top, seed):
    """The kernel's choice and the definition's among `pages` pages of one sequence and KV head, the last of them kept
    whatever the others' scores (infinite ones too), sums in fp64 and rounded once."""
    from flashattention_attention_b200 import fa
    d = bounds.shape[-1]
    c = plain.Cache(seed, "bf16", [32], 1, d, 32, spare=0)
    c.lens, c.bounds = [32 * pages], bounds
    c.table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()[None]
    got = fa.page_select(q.cuda(), bounds.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(), c.table.cuda(), hq=hq,
                         hkv=1, page_size=32, top_k=top, n_first=0, n_recent=1)
    assert fa.check_device_error() == fa.FA_OK
    qn, lim = q.double().numpy(), bounds[c.table[0].long(), 0].double().numpy()
    with np.errstate(over="ignore"):
        score = np.maximum(qn[:, None] * lim[:-1, 0], qn[:, None] * lim[:-1, 1]).sum(-1).astype(np.float32).max(0)
    best = np.sort(np.argsort(-score, kind="stable")[: top - 1])
    return got.flatten().tolist(), best.tolist() + [pages - 1]


@pytest.mark.parametrize("pages,top", [(60, 20), (900, 400), (3000, 900)])
@pytest.mark.parametrize("gain", [2.0 ** -70, 2.0 ** -64, 2.0 ** 61, 2.0 ** 64])
def test_products_past_fp32(pages, top, gain):
    """Queries and bounds of 2^-70 each give scores among fp32's subnormal numbers, of 2^64 infinite ones: ties, and the
    lower page first."""
    g = torch.Generator().manual_seed(pages)
    k = torch.randn((pages, 1, 1, 64), generator=g) + torch.randn((pages, 1, 2, 64), generator=g)
    bounds = torch.stack([k.amin(2), k.amax(2)], 2) * gain
    q = torch.randn((2, 64), generator=g) * gain
    got, want = _select(bounds.bfloat16().contiguous(), q.bfloat16(), pages, 2, top, 800)
    assert got == want


@pytest.mark.parametrize("pages,top", [(60, 20), (900, 400), (3000, 900)])
def test_products_past_fp32_that_cancel(pages, top):
    """Terms of 2^140 and -2^140: the score is what is left, small numbers that differ from page to page."""
    g = torch.Generator().manual_seed(pages)
    bounds = torch.zeros((pages, 1, 2, 64))
    bounds[..., 0], bounds[..., 1] = 2.0 ** 120, -2.0 ** 120
    bounds[..., 2] = torch.randint(0, 50, (pages, 1, 1), generator=g).float()
    bounds[::5, ..., 1] = 0  # some are infinite
    q = torch.ones((1, 64))
    q[:, :2] = 2.0 ** 20
    got, want = _select(bounds.bfloat16(), q.bfloat16(), pages, 1, top, 801)
    assert got == want
