"""GPU parity of the rotated paged append, the read-back, and a run of the
paged serving operators together, bit for bit where the definition rounds
every operation, else against 64 bits."""
import copy
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _fa():
    from flashattention_attention_b200 import fa
    return fa


def _tokens(seed, total, hq, hkv, d, dtype):
    """Q, K and V as slices of one projection's output."""
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((total, (hq + 2 * hkv) * d), generator=g) * 2).to(dtype)
    return (qkv, qkv[:, :hq * d].view(total, hq, d), qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d),
            qkv[:, (hq + hkv) * d:].view(total, hkv, d))


def _cuda_slices(qkv, hq, hkv, d):
    qkv = qkv.cuda()
    n = qkv.shape[0]
    return (qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d),
            qkv[:, (hq + hkv) * d:].view(n, hkv, d))


def _same_cache(c, kind):
    """The pools on the GPU equal the plain ones bit for bit (NaN rows included)."""
    def bits(t):
        t = t.cpu().contiguous()
        return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32) if t.dtype == torch.float32 else t
    names = ["kp", "vp", "bounds"] + ([] if kind == "bf16" else ["ks", "vs"])
    for name in names:
        got, want = getattr(c, name + "_").cpu(), getattr(c, name)
        if got.is_floating_point():
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan), name
            got, want = torch.where(nan, 0, got), torch.where(nan, 0, want)
            got, want = got + 0.0, want + 0.0  # -0 and +0 are one value
        assert torch.equal(bits(got), bits(want)), name


CASES = [
    # cur, new (None: one each), hq, hkv, d, page, rot, interleaved, x dtype
    ([0], None, 4, 2, 128, 32, 128, False, torch.bfloat16),
    ([63, 64, 0, 17], None, 8, 2, 128, 64, 128, False, torch.bfloat16),
    ([5, 0, 31], [40, 0, 1], 4, 4, 64, 32, 64, False, torch.bfloat16),
    ([0, 7, 100], [33, 64, 29], 2, 1, 128, 32, 64, True, torch.float32),
    ([1], [200], 3, 3, 48, 16, 32, False, torch.bfloat16),
    ([0, 250], [300, 7], 8, 8, 256, 128, 256, True, torch.bfloat16),
    ([9], [50], 1, 1, 16, 8, 16, False, torch.float32),
    ([2, 0], [3, 70], 6, 2, 96, 48, 16, False, torch.float32),
    ([12, 3], [5, 90], 5, 5, 80, 40, 0, False, torch.bfloat16),   # no rotation
    ([30] * 20, None, 2, 2, 240, 32, 160, True, torch.bfloat16),
]


@pytest.mark.parametrize("bounds", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_is_bit_exact(case, kind, bounds):
    fa = _fa()
    cur, new, hq, hkv, d, page, rot, inter, dtype = CASES[case]
    n = new or [1] * len(cur)
    total = sum(n)
    c = plain.Cache(case, kind, [a + b for a, b in zip(cur, n)], hkv, d, page, poison=False).cuda()
    qkv, q, k, v = _tokens(case, total, hq, hkv, d, dtype)
    table = plain.rope_table(max(a + b for a, b in zip(cur, n)), rot) if rot else None
    before = c.bounds.clone()
    q_ref, lens = plain.append(c, plain.f32(k), plain.f32(v), plain.f32(q), cur, n, table, inter)
    if not bounds:
        c.bounds = before
    qg, kg, vg = _cuda_slices(qkv, hq, hkv, d)
    cu = None if new is None else torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
    seqlens = torch.full((len(cur),), -1, dtype=torch.int32, device="cuda")
    out = fa.kv_append_rope_paged(kg, vg, c.kp_, c.vp_, torch.tensor(cur, dtype=torch.int32, device="cuda"), c.table_, q=qg,
                                  rope_table=None if table is None else torch.from_numpy(table).cuda(), interleaved=inter,
                                  k_scales=c.ks_, v_scales=c.vs_, key_bounds=c.bounds_ if bounds else None,
                                  cu_seqlens=cu, cache_seqlens=seqlens)
    assert fa.check_device_error() == fa.FA_OK
    want = q_ref.reshape(-1, d) if new is None else q_ref.transpose(0, 1)
    assert torch.equal(out.cpu(), want)
    assert seqlens.tolist() == lens
    _same_cache(c, kind)


def test_rotation_against_64_bits_at_far_positions():
    """The table and the rotation against cos and sin in 64 bits: a table entry is off by half an fp32 step (2^-24) plus
    the error of the 64-bit angle (position 2^-52); a rotated channel by at most four such roundings of |a| + |b|, and
    half a bf16 step."""
    fa = _fa()
    rows, d = 300000, 128
    table = fa.rope_table(rows, d, 500000.0)
    w = 500000.0 ** (-2.0 * np.arange(d // 2) / d)
    pos = np.array([0, 1, 4095, 131071, rows - 1])
    a = pos[:, None] * w
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.abs(table.numpy()[pos] - want).max() <= 2.0 ** -24 + rows * 2.0 ** -52
    x = torch.randn((5, 1, d), generator=torch.Generator().manual_seed(3)).bfloat16()
    page = 4096
    num = -(-rows // page)
    pool = torch.zeros((num, 1, page, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(num, dtype=torch.int32, device="cuda").expand(5, num).contiguous()
    out = fa.kv_append_rope_paged(x.cuda(), x.cuda(), pool, pool.clone(), torch.from_numpy(pos).int().cuda(), ids, q=x.cuda(),
                                  rope_table=table.cuda())
    xd = x.double().numpy()[:, 0]
    u, v = xd[:, :d // 2], xd[:, d // 2:]
    c, s = want[:, :d // 2], want[:, d // 2:]
    ref = np.concatenate([u * c - v * s, v * c + u * s], 1)
    tol = 2.0 ** -8 * np.abs(ref) + 4 * (2.0 ** -24 + rows * 2.0 ** -52) * np.tile(np.abs(u) + np.abs(v), 2)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    for i, p in enumerate(pos):  # the slot's key is the same rotation
        assert torch.equal(pool[p // page, 0, p % page], out[i])
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_quantised_rows_are_within_half_a_step(kind):
    """Against 64 bits: half a step, and the roundings of the row's range (three), of the code's quotient (two, 15 steps
    wide) and of the value (two)."""
    fa = _fa()
    c = plain.Cache(300, kind, [97], 2, 128, 32, poison=False).cuda()
    qkv, q, k, v = _tokens(300, 97, 2, 2, 128, torch.float32)
    _, kg, vg = _cuda_slices(qkv, 2, 2, 128)
    cu = torch.tensor([0, 97], dtype=torch.int32, device="cuda")
    fa.kv_append_rope_paged(kg, vg, c.kp_, c.vp_, torch.zeros(1, dtype=torch.int32, device="cuda"), c.table_,
                            k_scales=c.ks_, v_scales=c.vs_, cu_seqlens=cu)
    got = fa.kv_read_paged(c.kp_, c.vp_, cu, c.table_, total=97, k_scales=c.ks_, v_scales=c.vs_, out_dtype=torch.float32)
    for x, y in ((k, got[0]), (v, got[1])):
        x = x.double().transpose(0, 1)
        top = x.abs().amax(-1, keepdim=True)
        step = top / 127 if kind == "int8" else (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15
        codes = 127 if kind == "int8" else 15
        assert ((y.double().cpu() - x).abs() <= step / 2 + 2.0 ** -24 * (5 * codes * step + 2 * top)).all()


def test_rows_without_range_and_extreme_rows():
    fa = _fa()
    d = 64
    rows = torch.zeros((6, 1, d))
    rows[1] = 3.25
    rows[2, 0, 5] = -1e-30
    rows[3] = torch.linspace(-1e30, 1e30, d)
    rows[4] = torch.arange(d) % 16
    rows[5] = torch.linspace(0, 1, d) * 2.0 ** -140
    for kind in ("int8", "int4"):
        c = plain.Cache(301, kind, [6], 1, d, 16, poison=False).cuda()
        plain.append(c, rows.numpy(), rows.numpy(), None, [0], [6], None, False)
        fa.kv_append_rope_paged(rows.cuda(), rows.cuda(), c.kp_, c.vp_, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                c.table_, k_scales=c.ks_, v_scales=c.vs_, key_bounds=c.bounds_,
                                cu_seqlens=torch.tensor([0, 6], dtype=torch.int32, device="cuda"))
        _same_cache(c, kind)
    assert plain.unpack4(c.kp_.cpu().numpy())[int(c.table[0, 0]), 0, 4].tolist() == [i % 16 for i in range(d)]


def test_non_finite_rows_leave_the_other_rows_alone():
    fa = _fa()
    for kind in ("bf16", "int8", "int4"):
        c = plain.Cache(302, kind, [8], 1, 64, 8, poison=False).cuda()
        x = torch.randn((8, 1, 64), generator=torch.Generator().manual_seed(1))
        y = x.clone()
        y[3] = float("nan")
        y[5, 0, 7] = float("inf")
        d = copy.copy(c)
        for name in ("kp_", "vp_", "ks_", "vs_"):
            t = getattr(c, name)
            setattr(d, name, None if t is None else t.clone())
        cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
        pos = torch.zeros(1, dtype=torch.int32, device="cuda")
        for cache, rows in ((c, x), (d, y)):
            fa.kv_append_rope_paged(rows.cuda(), rows.cuda(), cache.kp_, cache.vp_, pos, c.table_, k_scales=cache.ks_,
                                    v_scales=cache.vs_, cu_seqlens=cu)
        keep = [0, 1, 2, 4, 6, 7]
        p = int(c.table[0, 0])
        for name in ("kp_", "vp_") + (("ks_", "vs_") if kind != "bf16" else ()):
            assert torch.equal(getattr(c, name)[p, 0, keep], getattr(d, name)[p, 0, keep])
        assert fa.check_device_error() == fa.FA_OK


def test_padding_and_bad_tokens_write_nothing():
    """Rows behind the last sequence, slots past the capacity or the table's rows, pages outside the pool and a broken
    cu_seqlens: skipped; everything but padding is reported."""
    fa = _fa()
    c = plain.Cache(303, "int4", [64, 64, 64, 64], 2, 64, 32, poison=False).cuda()
    qkv, *_ = _tokens(303, 12, 2, 2, 64, torch.bfloat16)
    qg, kg, vg = _cuda_slices(qkv, 2, 2, 64)
    names = ("kp_", "vp_", "ks_", "vs_", "bounds_")

    def call(cur, cu, rows=64, table=None):
        before = {n: getattr(c, n).clone() for n in names}
        lens = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        q_out = torch.full((2, 12, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fa.kv_append_rope_paged(kg, vg, c.kp_, c.vp_, torch.tensor(cur, dtype=torch.int32, device="cuda"),
                                c.table_ if table is None else table, q=qg, q_out=q_out,
                                rope_table=fa.rope_table(rows, 64).cuda(), k_scales=c.ks_, v_scales=c.vs_,
                                key_bounds=c.bounds_, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                cache_seqlens=lens)
        status = fa.check_device_error()
        changed = {n: (getattr(c, n) != before[n]).flatten(1).any(1).nonzero().flatten().tolist() for n in names}
        written = (q_out != 7.0).any(-1).any(0).tolist()
        for n in names:
            getattr(c, n).copy_(before[n])
        return status, changed, written, lens.tolist()

    ids = c.table.tolist()
    ok, changed, written, lens = call([3, 0, 9, 1], [0, 2, 2, 5, 6])  # six rows of padding
    assert ok == fa.FA_OK and written == [True] * 6 + [False] * 6 and lens == [5, 0, 12, 2]
    assert set(changed["kp_"]) == {ids[0][0], ids[2][0], ids[3][0]}
    st, changed, written, lens = call([62, -2, 10 ** 9, 64], [0, 4, 8, 10, 12])  # two past the end, two before 0, all outside
    assert st == fa.FA_ERR_INVALID and written == [True, True, False, False, False, False, True, True] + [False] * 4
    assert lens == [-1] * 4 and set(changed["kp_"]) == {ids[0][1], ids[1][0]}
    st, _, written, lens = call([10, 0, 0, 0], [0, 3, 3, 3, 3], rows=12)  # the table ends at position 11
    assert st == fa.FA_ERR_INVALID and written == [True, True] + [False] * 10
    table = c.table_.clone()
    table[0, 0], table[1, 0] = c.num, -1
    st, changed, written, _ = call([0, 0, 0, 0], [0, 3, 6, 9, 12], table=table)
    assert st == fa.FA_ERR_INVALID and written == [False] * 6 + [True] * 6
    assert set(changed["vs_"]) == {ids[2][0], ids[3][0]}
    st, changed, written, lens = call([0, 0, 0, 0], [0, 5, 3, 40, 12])  # not ascending, past the rows
    assert st == fa.FA_ERR_INVALID and lens[1] == -1 and lens[2] == -1
    assert fa.check_device_error() == fa.FA_OK


def test_empty_calls():
    """No sequence, or sequences without a new token: nothing moves but the lengths."""
    fa = _fa()
    c = plain.Cache(304, "int4", [64, 30], 2, 64, 32, poison=False).cuda()
    before = [getattr(c, n).clone() for n in ("kp_", "vp_", "ks_", "vs_", "bounds_")]
    kw = dict(k_scales=c.ks_, v_scales=c.vs_)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens = i32(-1, -1)
    q = fa.kv_append_rope_paged(none, none, c.kp_, c.vp_, i32(5, 64), c.table_, q=none, key_bounds=c.bounds_,
                                rope_table=fa.rope_table(64, 64).cuda(), cu_seqlens=i32(0, 0, 0), cache_seqlens=lens, **kw)
    assert q.shape == (2, 0, 64) and lens.tolist() == [5, 64]
    no = torch.empty((0,), dtype=torch.int32, device="cuda")
    no_table = c.table_[:0].contiguous()
    assert fa.kv_append_rope_paged(none, none, c.kp_, c.vp_, no, no_table, q=none, **kw).shape == (0, 64)
    k, v = fa.kv_read_paged(c.kp_, c.vp_, i32(0, 0, 0), c.table_, total=0, **kw)
    assert k.shape == v.shape == (2, 0, 64)
    nq = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert fa.attention_decode_paged(nq, c.kp_, c.vp_, no, no_table, hq=4, hkv=2, **kw).shape == (0, 64)
    sel = fa.page_select(nq, c.bounds_, no, no_table, hq=4, hkv=2, page_size=32, top_k=3)
    assert sel.shape == (0, 2, 3)
    assert fa.attention_decode_selected(nq, c.kp_, c.vp_, no, no_table, sel, hq=4, hkv=2, **kw).shape == (0, 64)
    assert fa.check_device_error() == fa.FA_OK
    for n, b in zip(("kp_", "vp_", "ks_", "vs_", "bounds_"), before):
        assert torch.equal(getattr(c, n), b)


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_many_tokens_and_heads(x_dtype):
    """More tokens than a block per token would take, decode steps between prompts, heads beyond one block's groups."""
    fa = _fa()
    cur = [0, 61, 7, 0, 130] + [3 * i for i in range(60)]
    new = [700, 1, 90, 0, 33] + [1] * 60
    hq, hkv, d, page = 5, 40, 32, 32
    c = plain.Cache(305, "int4", [a + b for a, b in zip(cur, new)], hkv, d, page, poison=False).cuda()
    total = sum(new)
    qkv, q, k, v = _tokens(305, total, hq, hkv, d, x_dtype)
    table = plain.rope_table(800, d)
    q_ref, lens = plain.append(c, plain.f32(k), plain.f32(v), plain.f32(q), cur, new, table, False)
    qg, kg, vg = _cuda_slices(qkv, hq, hkv, d)
    out = fa.kv_append_rope_paged(kg, vg, c.kp_, c.vp_, torch.tensor(cur, dtype=torch.int32).cuda(), c.table_, q=qg,
                                  rope_table=torch.from_numpy(table).cuda(), k_scales=c.ks_, v_scales=c.vs_,
                                  key_bounds=c.bounds_,
                                  cu_seqlens=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda())
    assert fa.check_device_error() == fa.FA_OK
    assert torch.equal(out.cpu(), q_ref.transpose(0, 1))
    _same_cache(c, "int4")


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_read_back(kind, out_dtype):
    fa = _fa()
    c = plain.Cache(310, kind, [100, 0, 33, 257], 3, 80, 24).cuda()
    start, n = [10, 0, 32, 0], [90, 0, 1, 257]
    total = sum(n) + 5  # the last five rows belong to no sequence
    cu = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")
    ko = torch.full((3, total, 80), 9.0, dtype=out_dtype, device="cuda")
    vo = ko.clone()
    k, v = fa.kv_read_paged(c.kp_, c.vp_, cu, c.table_, total=total, start=torch.tensor(start, dtype=torch.int32).cuda(),
                            k_scales=c.ks_, v_scales=c.vs_, out_dtype=out_dtype, k_out=ko, v_out=vo)
    assert k is ko and v is vo and fa.check_device_error() == fa.FA_OK
    at = 0
    for b in range(4):
        for g in range(3):
            want = c.rows(b, g, np.arange(start[b], start[b] + n[b]))
            for got, ref in ((k, want[0]), (v, want[1])):
                y = got[g, at:at + n[b]].double().cpu().numpy()
                # code * step + offset: two fp32 roundings of terms no larger than 16 steps; then out_dtype's
                tol = 2.0 ** -24 * 4 * (np.abs(ref) + 16) + (2.0 ** -8 * np.abs(ref) if out_dtype == torch.bfloat16 else 0)
                assert (np.abs(y - ref) <= tol).all()
                if kind == "int4" and out_dtype == torch.float32:  # each of the two rounded, no fused operation
                    keys = np.arange(start[b], start[b] + n[b])
                    p, o = c.table[b].numpy()[keys // 24], keys % 24
                    pool, sc = (c.kp, c.ks) if got is k else (c.vp, c.vs)
                    sc = sc[p, g, o].numpy()
                    want32 = plain.unpack4(pool[p, g, o].numpy()).astype(np.float32) * sc[:, :1] + sc[:, 1:]
                    assert np.array_equal(got[g, at:at + n[b]].cpu().numpy(), want32)
        at += n[b]
    assert (k[:, at:] == 9).all() and (v[:, at:] == 9).all()
    # from the start, and past what the table covers
    far = torch.tensor([0, 0, 0, 0, 30], dtype=torch.int32, device="cuda")
    fa.kv_read_paged(c.kp_, c.vp_, far, c.table_, total=30, start=torch.tensor([0, 0, 0, 264 - 10], dtype=torch.int32).cuda(),
                     k_scales=c.ks_, v_scales=c.vs_)
    assert fa.check_device_error() == fa.FA_ERR_INVALID


def _serve(kind, steps=3, hq=8, hkv=2, d=128, page=32):
    """A prompt appended, then decode steps: append, select, attend; every step's outputs."""
    fa = _fa()
    lens0 = [70, 33, 1]
    cap = 6
    num = 3 * cap
    c = plain.Cache(400, kind, [cap * page] * 3, hkv, d, page, poison=False, spare=0).cuda()
    for name in ("kp_", "vp_", "ks_", "vs_", "bounds_"):
        t = getattr(c, name)
        if t is not None and t.is_floating_point():
            t.fill_(float("nan"))  # nothing of the old cache may count
    assert c.num == num
    rope = fa.rope_table(cap * page, d).cuda()
    qkv, *_ = _tokens(400, sum(lens0), hq, hkv, d, torch.bfloat16)
    q, k, v = _cuda_slices(qkv, hq, hkv, d)
    cu = torch.tensor([0, 70, 103, 104], dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    kw = dict(k_scales=c.ks_, v_scales=c.vs_)
    fa.kv_append_rope_paged(k, v, c.kp_, c.vp_, torch.zeros_like(lens), c.table_, q=q, rope_table=rope, key_bounds=c.bounds_,
                            cu_seqlens=cu, cache_seqlens=lens, **kw)
    return fa, c, rope, lens, kw, hq, hkv, d, page


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_append_select_attend_together(kind):
    """A prompt and decode steps, eagerly and as one captured graph replayed, against the definition over the values that
    were appended."""
    fa, c, rope, lens, kw, hq, hkv, d, page = _serve(kind)
    snapshot = [None if t is None else t.clone() for t in (c.kp_, c.vp_, c.ks_, c.vs_, c.bounds_, lens)]
    cur, nxt = torch.empty_like(lens), torch.empty_like(lens)
    buf = torch.empty((3, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device="cuda")
    qv, kv, vv = buf[:, :hq * d].view(3, hq, d), buf[:, hq * d:(hq + hkv) * d].view(3, hkv, d), \
        buf[:, (hq + hkv) * d:].view(3, hkv, d)

    def step():
        cur.copy_(lens)
        q = fa.kv_append_rope_paged(kv, vv, c.kp_, c.vp_, cur, c.table_, q=qv, rope_table=rope, key_bounds=c.bounds_,
                                    cache_seqlens=nxt, **kw)
        lens.copy_(nxt)
        sel = fa.page_select(q, c.bounds_, lens, c.table_, hq=hq, hkv=hkv, page_size=page, top_k=2, n_first=0)
        return q, sel, fa.attention_decode_selected(q, c.kp_, c.vp_, lens, c.table_, sel, hq=hq, hkv=hkv, **kw)

    tokens = [_tokens(410 + i, 3, hq, hkv, d, torch.bfloat16)[0].cuda() for i in range(5)]
    eager = []
    for x in tokens:
        buf.copy_(x)
        q, sel, out = step()
        eager.append([t.clone() for t in (q, sel, out)])
        c.lens = lens.tolist()
        host = copy.copy(c)
        for name in ("kp", "vp", "ks", "vs", "bounds"):
            t = getattr(c, name + "_")
            setattr(host, name, None if t is None else t.cpu())
        qn = q.double().cpu().numpy().reshape(3, hq, d)
        assert np.array_equal(sel.cpu().numpy(), plain.select(host, qn, hq, 2, 0, 1))

        def keys(b, g):
            return np.concatenate([np.arange(p * page, min(c.lens[b], (p + 1) * page)) for p in sel[b, g].tolist() if p >= 0])

        ref, tol = plain.attend(host, qn, hq, keys, 1 / math.sqrt(d))
        got = out.double().cpu().numpy().reshape(ref.shape)
        assert (np.abs(got - ref) <= tol).all()
    assert fa.check_device_error() == fa.FA_OK
    # the same steps as a graph
    for t, s in zip((c.kp_, c.vp_, c.ks_, c.vs_, c.bounds_, lens), snapshot):
        if t is not None:
            t.copy_(s)
    buf.copy_(tokens[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    for x, want in zip(tokens, eager):
        buf.copy_(x)
        graph.replay()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)
    assert fa.check_device_error() == fa.FA_OK


def test_chunked_prefill_over_a_4_bit_prefix():
    """Cached rows read back as bf16 K and V feed the prefill; its last query agrees with the decode over the same cache:
    both are within their roundings of the same attention (values rounded to bf16 once more on the prefill's side)."""
    fa = _fa()
    c = plain.Cache(420, "int4", [150, 64], 2, 128, 32).cuda()
    q = (torch.randn((16, 128), generator=torch.Generator().manual_seed(9))).bfloat16().cuda()
    cu = torch.tensor([0, 150, 214], dtype=torch.int32, device="cuda")
    k, v = fa.kv_read_paged(c.kp_, c.vp_, cu, c.table_, total=214, k_scales=c.ks_, v_scales=c.vs_)
    cu_q = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    qv = q.view(2, 8, 128).transpose(0, 1).contiguous()
    o = fa.attention_fwd(qv, k, v, hq=8, hkv=2, causal=True, cu_seqlens_q=cu_q, cu_seqlens_k=cu, max_seqlen_q=1,
                         max_seqlen_k=150)
    dec = fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, hq=8, hkv=2, k_scales=c.ks_, v_scales=c.vs_)
    a, b = o.transpose(0, 1).reshape(16, 128).float(), dec.float()
    assert (a - b).norm() <= 2e-2 * b.norm()
    assert fa.check_device_error() == fa.FA_OK


def test_two_streams_at_once():
    """The same operators on two streams with tensors of their own, and on a stream the tensors were not made on."""
    fa = _fa()
    want, runs = [], []
    for i in range(2):
        c = plain.Cache(430 + i, "int4", [3000, 500 + i], 2, 128, 64).cuda()
        q = (torch.randn((16, 128), generator=torch.Generator().manual_seed(i)) * 1.5).bfloat16().cuda()
        runs.append((c, q))
        want.append(fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, hq=8, hkv=2, k_scales=c.ks_,
                                              v_scales=c.vs_))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, q) in enumerate(runs):
            got[i].append(fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, hq=8, hkv=2, k_scales=c.ks_,
                                                    v_scales=c.vs_, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


def test_two_graphs_replayed_in_turn():
    """Two captured calls with workspaces of their own, replayed on two streams."""
    fa = _fa()
    graphs = []
    for i in range(2):
        c = plain.Cache(440 + i, "int4", [2000, 100], 2, 128, 64).cuda()
        q = (torch.randn((16, 128), generator=torch.Generator().manual_seed(i)) * 1.5).bfloat16().cuda()
        kw = dict(hq=8, hkv=2, k_scales=c.ks_, v_scales=c.vs_)
        want = fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, **kw)
        sel = fa.page_select(q, c.bounds_, c.lens_, c.table_, hq=8, hkv=2, page_size=64, top_k=5)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, **kw)
            picked = fa.page_select(q, c.bounds_, c.lens_, c.table_, hq=8, hkv=2, page_size=64, top_k=5)
        graphs.append((graph, out, want, picked, sel, c, q, torch.cuda.Stream()))
    for _ in range(5):
        for graph, *_, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, picked, sel, *_ in graphs:
        assert torch.equal(out, want) and torch.equal(picked, sel)
