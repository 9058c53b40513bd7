"""GPU tests of the paged serving operators at shapes and layouts that the other
tests do not reach: wide groups, every head size, pages of any size, the widest
tables, projections in any layout."""
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _fa():
    from flashattention_attention_b200 import fa
    return fa


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("group,hkv,d,lens", [(11, 1, 64, [700, 0, 33]), (71, 2, 128, [300]), (128, 1, 128, [1000, 65]),
                                              (24, 3, 32, [500, 1]), (12, 2, 256, [260, 90]), (40, 1, 96, [30000, 64])])
def test_wide_groups(kind, group, hkv, d, lens):
    """Groups beyond eight heads run as several passes over their KV head, prime ones head by head."""
    fa, hq, page, top = _fa(), group * hkv, 32, 7
    c = plain.Cache(1200 + group, kind, lens, hkv, d, page).cuda()
    q = (torch.randn((len(lens) * hq, d), generator=torch.Generator().manual_seed(group)) * 1.5).bfloat16()
    qn = q.double().numpy().reshape(len(lens), hq, d)
    kw = dict(hq=hq, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_)
    sel = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=hq, hkv=hkv, page_size=page, top_k=top)
    want = plain.select(c, qn, hq, top, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)

    def keys(b, g):
        at = [np.arange(p * page, min(lens[b], (p + 1) * page)) for p in want[b, g] if p >= 0]
        return np.concatenate(at) if at else np.arange(0)

    calls = [(fa.attention_decode_selected(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, sel, **kw), keys)]
    if kind == "int4":
        calls.append((fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, **kw),
                      lambda b, g: np.arange(lens[b])))
    for out, seen in calls:
        ref, tol = plain.attend(c, qn, hq, seen, 1 / math.sqrt(d))
        assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("d", [16, 48, 80, 112, 144, 208, 240])
def test_select_at_any_head_and_page_size(d, page):
    fa, hq, hkv, top = _fa(), 6, 2, 9
    lens = [page * 300, page * 8 + 1, 1, 0, page * 129]
    c = plain.Cache(1300 + d, "bf16", lens, hkv, d, page).cuda()
    q = torch.randn((len(lens) * hq, d), generator=torch.Generator().manual_seed(d)).bfloat16()
    sel = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=hq, hkv=hkv, page_size=page, top_k=top, n_first=2)
    assert np.array_equal(sel.cpu().numpy(), plain.select(c, q.double().numpy().reshape(len(lens), hq, d), hq, top, 2, 1))
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("top,first,recent", [(4096, 100, 200), (4096, 4096, 0), (4096, 0, 4096), (1, 0, 0)])
def test_select_from_the_widest_table(top, first, recent):
    fa, pages, d = _fa(), 65536, 32
    g = torch.Generator().manual_seed(top + first)
    c = plain.Cache(1400, "bf16", [32], 1, d, 32)
    c.lens, c.table = [32 * pages - 5, 32 * 5000, 7], torch.stack([torch.randperm(pages, generator=g) for _ in range(3)]).int()
    k = torch.randn((pages, 1, 2, d), generator=g)
    c.bounds = torch.stack([k.amin(2), k.amax(2)], 2).bfloat16()
    q = torch.randn((6, d), generator=g).bfloat16()
    sel = fa.page_select(q.cuda(), c.bounds.cuda(), _i32(c.lens), c.table.cuda(), hq=2, hkv=1, page_size=32, top_k=top,
                         n_first=first, n_recent=recent)
    assert np.array_equal(sel.cpu().numpy(), plain.select(c, q.double().numpy().reshape(3, 2, d), 2, top, first, recent))
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("page", [1, 7])
@pytest.mark.parametrize("d", [16, 32, 112, 256])
def test_append_and_read_at_small_pages(kind, page, d):
    """Pages that end after one token or seven, rows appended in two calls, read back from any slot."""
    fa, hq, hkv, lens = _fa(), 3, 5, [40, 0, 9, 23]
    c = plain.Cache(1500 + d, kind, lens, hkv, d, page, poison=False).cuda()
    g = torch.Generator().manual_seed(page)
    table = plain.rope_table(40, 16)
    names = ["kp", "vp", "bounds"] + ([] if kind == "bf16" else ["ks", "vs"])
    for cur, new in (([0, 0, 0, 0], [17, 0, 8, 20]), ([17, 0, 8, 20], [23, 0, 1, 3])):
        total = sum(new)
        x = [torch.randn((total, h, d), generator=g).bfloat16() for h in (hq, hkv, hkv)]
        q_ref, ends = plain.append(c, plain.f32(x[1]), plain.f32(x[2]), plain.f32(x[0]), cur, new, table, True)
        after = _i32([-1] * 4)
        q = fa.kv_append_rope_paged(x[1].cuda(), x[2].cuda(), c.kp_, c.vp_, _i32(cur), c.table_, q=x[0].cuda(), interleaved=True,
                                    rope_table=torch.from_numpy(table).cuda(), k_scales=c.ks_, v_scales=c.vs_,
                                    key_bounds=c.bounds_, cu_seqlens=_i32([0] + list(np.cumsum(new))), cache_seqlens=after)
        assert torch.equal(q.cpu(), q_ref.transpose(0, 1)) and after.tolist() == ends
        for name in names:
            assert torch.equal(getattr(c, name + "_").cpu() + 0, getattr(c, name) + 0), name
    start, n = [3, 0, 8, 0], [37, 0, 1, 23]
    k, v = fa.kv_read_paged(c.kp_, c.vp_, _i32([0] + list(np.cumsum(n))), c.table_, total=sum(n), start=_i32(start),
                            k_scales=c.ks_, v_scales=c.vs_, out_dtype=torch.float32)
    at = 0
    for b in range(4):
        for h in range(hkv):
            for got, want in zip((k, v), c.rows(b, h, np.arange(start[b], start[b] + n[b]))):
                y = got[h, at:at + n[b]].double().cpu().numpy()
                assert (np.abs(y - want) <= 2.0 ** -24 * 4 * (np.abs(want) + 16)).all()
        at += n[b]
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_takes_projections_in_any_layout(dtype):
    """Heads before tokens, gaps between rows, one row for every token or head, one head of many: the same as contiguous
    rows."""
    fa, total, hq, hkv, d = _fa(), 37, 6, 2, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((h, total, d + 16), generator=g).to(dtype).cuda() for h in (hq, hkv, hkv))
    one = torch.randn((1, 1, d), generator=g).to(dtype).cuda()
    layouts = [tuple(x[..., :d].transpose(0, 1) for x in (q, k, v)),
               (q[..., :d].transpose(0, 1), one.expand(total, hkv, d), k[:1, :, 16:].transpose(0, 1).expand(total, hkv, d)),
               (one.expand(total, hq, d), v[:, :1, :d].transpose(0, 1).expand(total, hkv, d), v[..., 8:d + 8].transpose(0, 1))]
    for x in layouts:
        caches = [plain.Cache(1600, "int4", [total], hkv, d, 32, poison=False).cuda() for _ in range(2)]
        outs = []
        for c, rows in zip(caches, (x, [t.contiguous() for t in x])):
            outs.append(fa.kv_append_rope_paged(rows[1], rows[2], c.kp_, c.vp_, _i32([0]), c.table_, q=rows[0],
                                                rope_table=fa.rope_table(64, d).cuda(), k_scales=c.ks_, v_scales=c.vs_,
                                                key_bounds=c.bounds_, cu_seqlens=_i32([0, total])))
        assert torch.equal(*outs)
        for name in ("kp_", "vp_", "ks_", "vs_", "bounds_"):
            assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    assert fa.check_device_error() == fa.FA_OK
