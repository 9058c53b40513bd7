"""CPU checks of the paged serving operators' limits: refused before a launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fa():
    from flashattention_attention_b200 import fa
    return fa


def test_selection_over_more_pages_than_an_int_counts_is_refused(fa):
    """1024 sequences of a launch times KV heads times groups of 16 pages: up to 2^31, less a round of the device's
    warps, which count past the last group."""
    def call(batch, hkv, max_pages):
        p = fa.PageSelectParams()
        p.q, p.key_bounds, p.cache_seqlens, p.selected = 0x10000, 0x20000, 0x30000, 0x40000
        p.batch, p.hq, p.hkv, p.head_dim, p.top_k, p.n_first, p.n_recent = batch, hkv, hkv, 128, 4, 1, 1
        pages = fa.KvPages(0x90000, max_pages, 32, 16)
        return fa.lib.fa_page_select(ctypes.byref(p), ctypes.byref(pages), None)  # without a workspace

    assert call(1024, 511, 65536) == fa.FA_ERR_WORKSPACE
    assert call(1024, 512, 65536) == fa.FA_ERR_UNSUPPORTED
    assert call(2048, 512, 65536) == fa.FA_ERR_UNSUPPORTED
    assert call(906, 651, 3641 * 16) == fa.FA_ERR_UNSUPPORTED  # 2^31 - 2 groups
    assert call(906, 651, 3640 * 16) == fa.FA_ERR_WORKSPACE
