"""GPU parity of the attention over 4-bit pools and over selected pages, and
of the page selection, against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _fa():
    from flashattention_attention_b200 import fa
    return fa


def _queries(seed, B, hq, d, gain=1.5):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn((B * hq, d), generator=g) * gain).bfloat16()


def _check(out, ref, tol, what=""):
    got = out.float().cpu().numpy().reshape(ref.shape).astype(np.float64)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    assert over.max() <= 0, f"{what}: {over.max():.3e} past the tolerance, error {np.abs(got - ref).max():.3e}"


def _decode(c, q, hq, selected=None, **kw):
    fa = _fa()
    c.cuda()
    if selected is None:
        out = fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, hq=hq, hkv=c.hkv, k_scales=c.ks_,
                                        v_scales=c.vs_, **kw)
    else:
        out = fa.attention_decode_selected(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, selected.cuda(), hq=hq, hkv=c.hkv,
                                           k_scales=c.ks_, v_scales=c.vs_, **kw)
    torch.cuda.synchronize()
    return out


def _all_keys(c, window=0):
    return lambda b, g: np.arange(max(0, c.lens[b] - window) if window > 0 else 0, c.lens[b])


INT4_CASES = [
    # lens, hq, hkv, d, page, window
    ([1], 1, 1, 128, 32, 0),
    ([0, 1, 2, 31, 32, 33], 8, 2, 128, 32, 0),
    ([257], 32, 8, 128, 64, 0),
    ([1000, 0, 77, 640], 8, 8, 128, 64, 0),      # G = 1
    ([700, 100], 16, 2, 128, 256, 0),            # G = 8
    ([500, 77], 32, 2, 128, 128, 0),             # G = 16: two passes of 8 heads
    ([400], 9, 1, 64, 96, 0),                    # G = 9: three passes of 3
    ([999, 64, 3], 4, 2, 64, 32, 0),
    ([1000, 33, 512], 8, 2, 32, 64, 0),
    ([999, 100], 6, 2, 96, 64, 0),               # G = 3
    ([700, 1024, 1], 8, 2, 256, 64, 0),
    ([300], 32, 2, 256, 32, 0),
    ([2000, 300, 1025, 5], 8, 2, 128, 64, 700),
    ([2000, 90, 31], 4, 4, 256, 32, 1),          # a window of one key
    ([129] * 40, 4, 2, 64, 64, 100),
    ([9000, 1, 4097], 4, 1, 128, 128, 0),
    # long enough that all tiles are dealt over the device and split segments merged by a second kernel
    ([30011], 4, 1, 128, 96, 0),
    ([17000, 0, 33, 23456, 1], 16, 2, 128, 128, 0),
    ([40000, 7], 24, 1, 64, 64, 0),              # three passes of 8 heads
    ([25001, 12000], 2, 1, 32, 64, 0),
    ([25001, 64], 3, 1, 96, 32, 0),
    ([20000, 9001], 8, 1, 256, 32, 0),
    ([30000, 20000], 4, 2, 128, 64, 15000),
    ([300, 64], 4, 2, 128, 64, 2 ** 31 - 1),     # a window past every key
]


@pytest.mark.parametrize("case", range(len(INT4_CASES)))
def test_int4_decode(case):
    lens, hq, hkv, d, page, window = INT4_CASES[case]
    c = plain.Cache(case, "int4", lens, hkv, d, page, width=-(-max(lens) // page) + 3)
    q = _queries(case, len(lens), hq, d)
    out = _decode(c, q, hq, window=window)
    ref, tol = plain.attend(c, q.double().numpy().reshape(len(lens), hq, d), hq, _all_keys(c, window), 1 / math.sqrt(d))
    _check(out, ref, tol, str(INT4_CASES[case]))
    assert _fa().check_device_error() == _fa().FA_OK


def test_int4_epilogue_scale_and_empty_rows():
    epi = [("mul", -2.0), ("add", 0.5)]
    c = plain.Cache(50, "int4", [0, 100, 0], 2, 128, 32, width=4)
    q = _queries(50, 3, 4, 128)
    out = _decode(c, q.view(-1, 1, 128), 4, scale=0.3, epilogue=epi)
    assert out.shape == (12, 1, 128)
    ref, tol = plain.attend(c, q.double().numpy().reshape(3, 4, 128), 4, _all_keys(c), 0.3, epi)
    _check(out, ref, tol)
    assert (out.view(3, 4, 128)[[0, 2]] == 0.5).all()


@pytest.mark.parametrize("v_gain", [1e-6, 3e4])
def test_int4_values_far_from_one(v_gain):
    """Steps below fp16's normal range and products above its largest number."""
    c = plain.Cache(51, "int4", [600, 40], 2, 128, 64, poison=False)
    c.vs = c.vs * v_gain
    q = _queries(51, 2, 8, 128)
    out = _decode(c, q, 8)
    ref, tol = plain.attend(c, q.double().numpy().reshape(2, 8, 128), 8, _all_keys(c), 1 / math.sqrt(128))
    _check(out, ref, tol)


def test_int4_rows_without_range_and_large_queries():
    """Equal channels (step 0), queries from 2^-10 to 2^10, one far outlier key."""
    c = plain.Cache(52, "int4", [300], 1, 64, 32, poison=False)
    c.ks[:, :, ::3, 0] = 0
    c.vs[:, :, ::5, 0] = 0
    q = _queries(52, 1, 4, 64) * torch.tensor([2.0 ** -10, 1.0, 16.0, 2.0 ** 10]).bfloat16()[:, None]
    out = _decode(c, q, 4)
    ref, tol = plain.attend(c, q.double().numpy().reshape(1, 4, 64), 4, _all_keys(c), 1 / 8)
    _check(out, ref, tol)


SELECT_CASES = [
    # lens, hq, hkv, d, page, top, first, recent
    ([1], 1, 1, 128, 32, 4, 1, 1),
    ([0, 1, 64, 65, 1000], 8, 2, 128, 32, 4, 1, 2),
    ([3000, 2111, 640], 16, 2, 128, 64, 8, 0, 1),
    ([2500, 2], 12, 4, 64, 32, 16, 2, 2),
    ([4000], 32, 2, 128, 32, 7, 0, 0),
    ([1500, 700], 6, 2, 96, 64, 5, 1, 1),
    ([1500, 31], 8, 1, 256, 32, 9, 3, 3),
    ([777, 1024], 4, 4, 32, 32, 1, 0, 1),
    ([9999], 2, 1, 64, 32, 200, 1, 1),
    # selections long enough to be dealt over the device
    ([33000], 8, 1, 128, 32, 900, 2, 2),
    ([30000, 5, 26000], 3, 1, 64, 64, 420, 0, 1),
    ([16000, 12000], 2, 1, 256, 32, 350, 1, 1),
    ([25000], 1, 1, 96, 96, 250, 1, 1),
    ([33000], 4, 1, 32, 32, 1000, 1, 1),
    # many sequences, one of them long: pages dealt evenly to the device, then a block per sequence and KV head
    ([9700] + [(977 * i) % 1500 for i in range(39)], 4, 2, 64, 32, 9, 1, 2),
]


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("case", range(len(SELECT_CASES)))
def test_select_and_attend(case, kind):
    fa = _fa()
    lens, hq, hkv, d, page, top, first, recent = SELECT_CASES[case]
    c = plain.Cache(100 + case, kind, lens, hkv, d, page, width=-(-max(lens) // page) + 1).cuda()
    q = _queries(100 + case, len(lens), hq, d)
    qn = q.double().numpy().reshape(len(lens), hq, d)
    got = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=hq, hkv=hkv, page_size=page, top_k=top, n_first=first,
                         n_recent=recent)
    want = plain.select(c, qn, hq, top, first, recent)
    assert np.array_equal(got.cpu().numpy(), want)
    out = _decode(c, q, hq, selected=got)

    def keys(b, g):
        at = [np.arange(p * page, min(lens[b], (p + 1) * page)) for p in want[b, g] if p >= 0]
        return np.concatenate(at) if at else np.arange(0)

    ref, tol = plain.attend(c, qn, hq, keys, 1 / math.sqrt(d))
    _check(out, ref, tol, f"{kind} {SELECT_CASES[case]}")
    assert fa.check_device_error() == fa.FA_OK


def test_select_ties_go_to_the_lowest_page():
    """Pages with equal bounds everywhere, and scores of -0 and +0."""
    fa = _fa()
    c = plain.Cache(120, "bf16", [64 * 40], 1, 64, 64)
    c.bounds[:] = 1.0
    c.bounds[c.table[0, 7].item()] = 2.0
    c.cuda()
    q = torch.ones(1, 64, dtype=torch.bfloat16)
    got = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=1, hkv=1, page_size=64, top_k=6, n_first=0, n_recent=2)
    assert got.cpu().tolist() == [[[0, 1, 2, 7, 38, 39]]]
    q[:] = 0.0
    c.bounds_[::2] = -1.0
    got = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=1, hkv=1, page_size=64, top_k=6, n_first=0, n_recent=2)
    assert got.cpu().tolist() == [[[0, 1, 2, 3, 38, 39]]]


@pytest.mark.parametrize("pages,top", [(700, 300), (5000, 40), (5000, 4000)])
def test_select_among_many_equal_pages(pages, top):
    """More pages next to the border than are ranked directly, and more than are held in shared memory."""
    fa = _fa()
    c = plain.Cache(122, "bf16", [32], 1, 64, 32, spare=1).cuda()
    c.lens = [32 * pages]
    g = torch.Generator().manual_seed(pages)
    c.bounds = (torch.randint(0, 3, (pages, 1, 2, 64), generator=g) == 0).bfloat16()
    c.bounds[:, :, 0] = -c.bounds[:, :, 0]
    c.bounds[::3] = c.bounds[0]
    c.table = torch.randperm(pages, generator=g).int()[None]
    q = torch.where(torch.arange(64) % 2 == 0, 1.0, -1.0).bfloat16()[None]
    got = fa.page_select(q.cuda(), c.bounds.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(), c.table.cuda(), hq=1,
                         hkv=1, page_size=32, top_k=top, n_first=1, n_recent=1)
    assert np.array_equal(got.cpu().numpy(), plain.select(c, q.double().numpy().reshape(1, 1, 64), 1, top, 1, 1))


def test_select_with_infinite_bounds_stays_inside():
    """An unspecified choice, but of the sequence's pages, ascending and distinct."""
    fa = _fa()
    c = plain.Cache(123, "bf16", [32 * 300], 2, 64, 32)
    c.bounds[::5, 0, 1] = float("inf")
    c.bounds[::7, 1] = float("nan")
    c.cuda()
    got = fa.page_select(_queries(123, 1, 4, 64).cuda(), c.bounds_, c.lens_, c.table_, hq=4, hkv=2, page_size=32, top_k=50)
    for row in got[0].tolist():
        assert row == sorted(set(row)) and 0 <= row[0] and row[-1] == 299 and len(row) == 50


def test_select_near_ties_are_told_apart():
    """Two pages whose scores differ by less than fp32 sums of their terms are good for."""
    fa = _fa()
    c = plain.Cache(121, "bf16", [32 * 64], 1, 128, 32)
    base = torch.randn(128, generator=torch.Generator().manual_seed(5)).bfloat16()
    c.bounds[:] = base * 64
    for p in range(64):  # big terms that cancel, and a small one that decides
        row = c.bounds[c.table[0, p].item(), 0]
        row[:, 0], row[:, 1], row[:, 2] = 4096.0, -4096.0, float(p % 7) * 2.0 ** -9
    c.cuda()
    q = torch.ones(1, 128, dtype=torch.bfloat16)
    got = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=1, hkv=1, page_size=32, top_k=12, n_first=0, n_recent=0)
    assert np.array_equal(got.cpu().numpy(), plain.select(c, q.double().numpy().reshape(1, 1, 128), 1, 12, 0, 0))


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_selection_of_the_callers_own(kind):
    """-1 and pages past the end stand for no key, order does not matter, a page named twice counts twice, and a head
    with nothing selected gets the epilogue of 0."""
    c = plain.Cache(130, kind, [200, 333, 40], 2, 128, 32)
    q = _queries(130, 3, 4, 128)
    sel = torch.tensor([[[5, -1, 2, 0], [6, 1, 99, -7]], [[3, 3, -1, 10], [-1, -1, -1, -1]], [[1, 0, 5, 5], [0, -1, 0, 0]]],
                       dtype=torch.int32)

    def keys(b, g):
        n, pages = c.lens[b], -(-c.lens[b] // 32)
        at = [np.arange(p * 32, min(n, (p + 1) * 32)) for p in sel[b, g, : min(4, pages)].tolist() if 0 <= p < pages]
        return np.concatenate(at) if at else np.arange(0)

    epi = [("mul", 3.0), ("add", -1.0)]
    out = _decode(c, q, 4, selected=sel, epilogue=epi)
    ref, tol = plain.attend(c, q.double().numpy().reshape(3, 4, 128), 4, keys, 1 / math.sqrt(128), epi)
    _check(out, ref, tol, kind)
    assert (out.view(3, 4, 128)[1, 2:] == -1.0).all()
    assert _fa().check_device_error() == _fa().FA_OK


def test_selecting_every_page_is_the_whole_attention():
    fa = _fa()
    c = plain.Cache(131, "int4", [500, 64, 1], 2, 128, 64)
    q = _queries(131, 3, 8, 128)
    sel = torch.arange(8, dtype=torch.int32).expand(3, 2, 8).contiguous()
    a, b = _decode(c, q, 8).float(), _decode(c, q, 8, selected=sel).float()
    # both are roundings of the same sums: a bf16 step apart where the sums straddle a border
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs().clamp(min=2.0 ** -6)).all()


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_bad_lengths_and_pages_are_reported(kind):
    fa = _fa()
    c = plain.Cache(140, kind, [64, 100, 32], 2, 64, 32, poison=False, width=4).cuda()
    c.lens_[0], c.lens_[2] = -5, 10 ** 6  # clamped to 0 and to the capacity of 128
    c.table_[2] = c.table_[1]
    q = _queries(140, 3, 4, 64).cuda()
    sel = torch.zeros((3, 2, 2), dtype=torch.int32, device="cuda")
    kw = dict(hq=4, hkv=2, k_scales=c.ks_, v_scales=c.vs_)
    calls = [lambda: fa.attention_decode_selected(q, c.kp_, c.vp_, c.lens_, c.table_, sel, **kw),
             lambda: fa.page_select(q, c.bounds_, c.lens_, c.table_, hq=4, hkv=2, page_size=32, top_k=2)]
    if kind == "int4":
        calls.append(lambda: fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, **kw))
    for call in calls:
        out = call()
        assert fa.check_device_error() == fa.FA_ERR_INVALID
        assert fa.check_device_error() == fa.FA_OK
    assert (calls[0]()[:4] == 0).all()
    assert fa.check_device_error() == fa.FA_ERR_INVALID
    # a page id outside the pool: reported, nothing read outside
    c.lens_.copy_(torch.tensor([64, 100, 32]))
    good = calls[0]()
    assert fa.check_device_error() == fa.FA_OK
    c.table_[0, 0] = c.num
    c.table_[1, 0] = -1
    bad = calls[0]()
    assert fa.check_device_error() == fa.FA_ERR_INVALID
    assert torch.equal(good[8:], bad[8:])


def test_int4_same_result_run_after_run_and_with_any_workspace():
    fa = _fa()
    c = plain.Cache(150, "int4", [30000, 77, 15000], 1, 128, 64).cuda()
    q = _queries(150, 3, 8, 128).cuda()
    kw = dict(hq=8, hkv=1, k_scales=c.ks_, v_scales=c.vs_)
    need = fa.decode_workspace_size(3, 8, c.width * 64, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a = fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, workspace=ws, **kw)
    for fill in (0, 127):
        ws.fill_(fill)
        assert torch.equal(a, fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, workspace=ws, **kw))
    with pytest.raises(fa.FAError) as e:
        fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, workspace=ws[:-16], **kw)
    assert e.value.status == fa.FA_ERR_WORKSPACE


def test_int4_many_short_sequences():
    c = plain.Cache(151, "int4", [(37 * i) % 150 for i in range(300)], 1, 64, 32)
    q = _queries(151, 300, 2, 64)
    out = _decode(c, q, 2)
    ref, tol = plain.attend(c, q.double().numpy().reshape(300, 2, 64), 2, _all_keys(c), 1 / 8)
    _check(out, ref, tol)


def test_int4_batch_past_a_grid_dimension():
    """More (sequence, KV head) pairs than a grid's second dimension holds."""
    fa = _fa()
    B, hkv, page, d = 70000, 1, 32, 64
    c = plain.Cache(152, "int4", [40], hkv, d, page).cuda()
    lens = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    lens[1::2] = 7
    lens[-3] = 0
    table = c.table_.expand(B, 2).contiguous()
    q = _queries(152, 1, 1, d).cuda().expand(B, d).contiguous()
    out = fa.attention_decode_paged(q, c.kp_, c.vp_, lens, table, hq=1, hkv=1, k_scales=c.ks_, v_scales=c.vs_)
    qn = q[:1].double().cpu().numpy().reshape(1, 1, d)
    for n, rows in ((40, out[0::2]), (7, out[1::2][:-2])):
        c.lens = [n]
        ref, tol = plain.attend(c, qn, 1, _all_keys(c), 1 / 8)
        _check(rows[:1], ref, tol)
        assert (rows == rows[:1]).all()
    assert (out[-3] == 0).all()
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_pages_past_two_to_the_31_elements(kind):
    """A pool whose last pages start past 2^31 elements (and bytes)."""
    fa = _fa()
    hkv, d, page = 1, 256, 256
    num = (2 ** 31 // (page * d)) + 40
    c = plain.Cache(160, kind, [600], hkv, d, page, spare=0).cuda()
    shape = list(c.kp_.shape)
    big = {}
    for name in ("kp_", "vp_", "ks_", "vs_", "bounds_"):
        t = getattr(c, name)
        if t is not None:
            big[name] = torch.empty((num * (2 if kind == "int4" and t.dtype == torch.uint8 else 1),) + tuple(t.shape[1:]),
                                    dtype=t.dtype, device="cuda")
    total = big["kp_"].shape[0]
    for name in list(big):
        t = getattr(c, name)
        if big[name].shape[0] != total:
            big[name] = torch.empty((total,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        big[name][total - shape[0]:] = t
    table = c.table_ + (total - shape[0])
    q = _queries(160, 1, 4, d)
    kw = dict(hq=4, hkv=1, k_scales=big.get("ks_"), v_scales=big.get("vs_"))
    sel = fa.page_select(q.cuda(), big["bounds_"], c.lens_, table, hq=4, hkv=1, page_size=page, top_k=3)
    out = fa.attention_decode_selected(q.cuda(), big["kp_"], big["vp_"], c.lens_, table, sel, **kw)
    ref, tol = plain.attend(c, q.double().numpy().reshape(1, 4, d), 4, _all_keys(c), 1 / 16)
    _check(out, ref, tol)
    if kind == "int4":
        _check(fa.attention_decode_paged(q.cuda(), big["kp_"], big["vp_"], c.lens_, table, **kw), ref, tol)
    assert fa.check_device_error() == fa.FA_OK
