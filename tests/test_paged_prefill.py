"""GPU test of a chunk of queries over a 4-bit prefix: the rows read back feed
the prefill, against 64 bits over the very values that were read."""
import math

import numpy as np
import pytest
import torch

import paged_plain as plain
from conftest import assert_close_bf16

pytestmark = pytest.mark.gpu


def test_a_chunk_of_queries_over_a_4_bit_prefix():
    """The last 40 positions of 150 cached keys and the last 7 of 64, causal.  The values read back are the cache's,
    code * step + offset, rounded to fp32 twice and to bf16 once; the prefill over them passes the bf16 gate."""
    from flashattention_attention_b200 import fa
    hq, hkv, d, lens, new = 8, 2, 128, [150, 64], [40, 7]
    c = plain.Cache(1100, "int4", lens, hkv, d, 32).cuda()
    cu = torch.tensor([0, 150, 214], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor([0, 40, 47], dtype=torch.int32, device="cuda")
    q = torch.randn((hq, sum(new), d), generator=torch.Generator().manual_seed(9)).bfloat16()
    k, v = fa.kv_read_paged(c.kp_, c.vp_, cu, c.table_, total=214, k_scales=c.ks_, v_scales=c.vs_)
    out = fa.attention_fwd(q.cuda(), k, v, hq=hq, hkv=hkv, causal=True, cu_seqlens_q=cu_q, cu_seqlens_k=cu, max_seqlen_q=40,
                           max_seqlen_k=150)
    assert fa.check_device_error() == fa.FA_OK
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    ref = np.zeros((hq, sum(new), d))
    at = 0
    for b in range(2):
        for g in range(hkv):
            rows = slice(150 * b, 150 * b + lens[b])
            for got, want in zip((kn[g, rows], vn[g, rows]), c.rows(b, g, np.arange(lens[b]))):
                assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * 16).all()
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                for i in range(new[b]):
                    n = lens[b] - new[b] + i + 1
                    x = kn[g, rows][:n] @ q[h, at + i].double().numpy() / math.sqrt(d)
                    w = np.exp(x - x.max())
                    ref[h, at + i] = w @ vn[g, rows][:n] / w.sum()
        at += new[b]
    assert_close_bf16(out.float().cpu().numpy(), ref, what="chunk over a 4-bit prefix")
