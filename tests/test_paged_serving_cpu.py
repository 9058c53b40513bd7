"""CPU checks of the paged serving operators: every refusal happens on the host
before a launch (C ABI and binding), and the rotation table's host function."""
import ctypes

import numpy as np
import pytest
import torch

import paged_plain as plain

CUDA0 = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def fa():
    from flashattention_attention_b200 import fa
    return fa


class Fake:
    """Shape, type and address of a tensor that no GPU holds."""

    def __init__(self, addr, shape, dtype, device=CUDA0, contiguous=True, strides=None):
        self.addr, self.shape, self.dtype, self.device = addr, torch.Size(shape), dtype, device
        self.is_cuda, self._contiguous = device.type == "cuda", contiguous
        self._strides = strides or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))

    def data_ptr(self):
        return self.addr

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def is_contiguous(self):
        return self._contiguous

    def stride(self):
        return self._strides

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


def pages(fa, **kw):
    p = fa.KvPages(0x90000, 4, 32, 16)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_append_rope_refusals(fa):
    def call(pg=None, **kw):
        p = fa.KvAppendRopeParams()
        p.k_new, p.v_new, p.q, p.q_out = 0x10000, 0x20000, 0x30000, 0x40000
        p.k_token_stride = p.v_token_stride = p.q_token_stride = p.q_out_token_stride = 1024
        p.k_head_stride = p.v_head_stride = p.q_head_stride = p.q_out_head_stride = 128
        p.rope_table, p.k_cache, p.v_cache, p.cur_pos = 0x50000, 0x60000, 0x70000, 0x80000
        p.x_dtype, p.cache_dtype = fa.FA_BF16, fa.FA_BF16
        p.batch, p.total, p.hq, p.hkv, p.head_dim, p.rot_dim, p.rope_rows = 2, 2, 8, 2, 128, 128, 4096
        for k, v in kw.items():
            setattr(p, k, v)
        return fa.lib.fa_kv_append_rope_paged(ctypes.byref(p), ctypes.byref(pg or pages(fa)), None)

    assert fa.lib.fa_kv_append_rope_paged(None, None, None) == fa.FA_ERR_INVALID
    for bad in (dict(head_dim=120), dict(head_dim=0), dict(x_dtype=fa.FA_I8), dict(cache_dtype=fa.FA_F32),
                dict(cache_dtype=fa.FA_I4), dict(cache_dtype=fa.FA_I8, k_scales=0x1000), dict(total=3), dict(total=-1),
                dict(cu_seqlens=0x1000, total=-1), dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=-16),
                dict(interleaved=2), dict(rope_table=None), dict(rope_table=0x50008), dict(rope_rows=0), dict(hkv=0),
                dict(batch=-1), dict(k_new=None), dict(v_new=0x20004), dict(k_cache=None), dict(v_cache=0x70002),
                dict(cur_pos=None), dict(cur_pos=0x80004), dict(cu_seqlens=0x1004), dict(cache_seqlens=0x80000),
                dict(cu_seqlens=0x1000, cache_seqlens=0x1000), dict(k_token_stride=1020), dict(v_head_stride=4),
                dict(q_token_stride=3), dict(q_out_head_stride=4), dict(q_out=None), dict(hq=0), dict(key_bounds=0x8),
                dict(x_dtype=fa.FA_F32, k_head_stride=130), dict(batch=0)):
        assert call(**bad) == fa.FA_ERR_INVALID, bad
    assert call(head_dim=272) == fa.FA_ERR_UNSUPPORTED
    for bad in (dict(max_pages=0), dict(num_pages=0), dict(page_size=0), dict(block_table=None), dict(block_table=0x8)):
        assert call(pages(fa, **bad)) == fa.FA_ERR_INVALID, bad
    assert call(pages(fa, num_pages=1 << 25)) == fa.FA_ERR_UNSUPPORTED       # rows past 2^31
    assert call(pages(fa, max_pages=1 << 26)) == fa.FA_ERR_UNSUPPORTED       # slots past 2^31
    assert call(batch=0, total=0, k_new=None) == fa.FA_OK                    # nothing to do


def test_read_refusals(fa):
    def call(pg=None, **kw):
        p = fa.KvReadParams()
        p.k_cache, p.v_cache, p.k_out, p.v_out, p.cu_seqlens = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
        p.cache_dtype, p.out_dtype, p.batch, p.total, p.hkv, p.head_dim = fa.FA_BF16, fa.FA_BF16, 2, 10, 2, 128
        for k, v in kw.items():
            setattr(p, k, v)
        return fa.lib.fa_kv_read_paged(ctypes.byref(p), ctypes.byref(pg or pages(fa)), None)

    assert fa.lib.fa_kv_read_paged(None, None, None) == fa.FA_ERR_INVALID
    for bad in (dict(out_dtype=fa.FA_I8), dict(cache_dtype=fa.FA_F32), dict(cache_dtype=fa.FA_I4), dict(total=-1),
                dict(k_out=None), dict(v_cache=0x20008), dict(cu_seqlens=None), dict(start=0x4), dict(head_dim=40),
                dict(hkv=0), dict(batch=-1)):
        assert call(**bad) == fa.FA_ERR_INVALID, bad
    assert call(head_dim=512) == fa.FA_ERR_UNSUPPORTED
    assert call(total=0, k_out=None) == fa.FA_OK


def test_page_select_refusals(fa):
    def call(pg=None, **kw):
        p = fa.PageSelectParams()
        p.q, p.key_bounds, p.cache_seqlens, p.selected = 0x10000, 0x20000, 0x30000, 0x40000
        p.batch, p.hq, p.hkv, p.head_dim, p.top_k, p.n_first, p.n_recent = 2, 8, 2, 128, 4, 1, 1
        p.workspace, p.workspace_bytes = 0x50000, 1 << 20
        for k, v in kw.items():
            setattr(p, k, v)
        return fa.lib.fa_page_select(ctypes.byref(p), ctypes.byref(pg or pages(fa)), None)

    assert fa.lib.fa_page_select(None, None, None) == fa.FA_ERR_INVALID
    for bad in (dict(hq=7), dict(hq=0), dict(top_k=0), dict(top_k=4097), dict(n_first=-1), dict(n_recent=-1),
                dict(n_first=3, n_recent=2), dict(n_first=2 ** 31 - 1, n_recent=2 ** 31 - 1), dict(q=None),
                dict(key_bounds=0x20008), dict(cache_seqlens=None), dict(selected=0x40004), dict(head_dim=100)):
        assert call(**bad) == fa.FA_ERR_INVALID, bad
    for bad in (dict(workspace=None), dict(workspace=0x50008), dict(workspace_bytes=16)):
        assert call(pages(fa, max_pages=5000), **bad) == fa.FA_ERR_WORKSPACE, bad
    assert call(pages(fa, max_pages=65537, page_size=1)) == fa.FA_ERR_UNSUPPORTED
    assert call(head_dim=320) == fa.FA_ERR_UNSUPPORTED
    assert call(batch=0, q=None) == fa.FA_OK
    assert fa.lib.fa_page_select_workspace_size(0, 1, 1) == 0
    assert fa.lib.fa_page_select_workspace_size(4, 8, 1024) == 0  # one kernel
    assert fa.lib.fa_page_select_workspace_size(1000, 8, 128) == 0
    assert fa.lib.fa_page_select_workspace_size(4, 8, 5000) >= 4 * 4 * 8 * 5000


def test_decode_refusals(fa):
    long = 100000 * 32  # a capacity whose work is spread over the device, with a workspace
    need = fa.decode_workspace_size(2, 8, long, 128)

    def params(**kw):
        p = fa.DecodeParams()
        p.q, p.k_cache, p.v_cache, p.k_scales, p.v_scales = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
        p.cache_seqlens, p.out, p.kv_dtype = 0x60000, 0x70000, fa.FA_I4
        p.batch, p.hq, p.hkv, p.head_dim, p.capacity, p.softmax_scale = 2, 8, 2, 128, 128, 0.1
        p.workspace, p.workspace_bytes = 0x80000, need
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def paged(pg=None, **kw):
        return fa.lib.fa_attention_decode_paged(ctypes.byref(params(**kw)), ctypes.byref(pg or pages(fa)), None)

    def selected(sel=0xa0000, top_k=3, pg=None, **kw):
        return fa.lib.fa_attention_decode_selected(ctypes.byref(params(**kw)), ctypes.byref(pg or pages(fa)), sel, top_k,
                                                   None)

    # a 4-bit cache is paged only
    assert fa.lib.fa_attention_decode(ctypes.byref(params()), None) == fa.FA_ERR_INVALID
    assert fa.lib.fa_attention_decode_noalloc(ctypes.byref(params()), None) == fa.FA_ERR_INVALID
    for call in (paged, selected):
        for bad in (dict(k_scales=None), dict(v_scales=0x50008), dict(capacity=96), dict(head_dim=100), dict(hq=7),
                    dict(kv_dtype=fa.FA_F32), dict(softmax_scale=float("nan")), dict(n_epilogue=9), dict(out=None)):
            assert call(**bad) == fa.FA_ERR_INVALID, bad
        assert call(head_dim=160) == fa.FA_ERR_UNSUPPORTED
        far = dict(pg=pages(fa, max_pages=100000), capacity=long)
        if call is selected:
            far["top_k"] = 4096
        for bad in (dict(workspace_bytes=need - 1), dict(workspace=None), dict(workspace=0x80008)):
            assert call(**far, **bad) == fa.FA_ERR_WORKSPACE, bad
        assert call(pg=pages(fa, page_size=48), capacity=192) == fa.FA_ERR_INVALID
        assert call(pg=pages(fa, num_pages=1 << 25)) == fa.FA_ERR_UNSUPPORTED
        assert call(batch=0) == fa.FA_OK
    size = lambda top_k, **kw: fa.lib.fa_decode_pages_workspace_size(
        ctypes.byref(params(**kw)), ctypes.byref(pages(fa, max_pages=kw.get("capacity", 128) // 32)), top_k)
    assert size(0) == 0 and size(3) == 0 and size(3, capacity=long) == 0 and size(0, batch=0) == 0
    assert size(0, capacity=long) == need and size(4096, capacity=long) == need
    assert selected(window=4) == fa.FA_ERR_INVALID
    assert selected(top_k=0) == fa.FA_ERR_INVALID and selected(top_k=4097) == fa.FA_ERR_INVALID
    assert selected(sel=None) == fa.FA_ERR_INVALID and selected(sel=0xa0004) == fa.FA_ERR_INVALID
    assert fa.lib.fa_attention_decode_selected(None, None, None, 1, None) == fa.FA_ERR_INVALID


def test_rope_table(fa):
    for rows, rot, base in ((1, 16, 10000.0), (5000, 64, 10000.0), (33, 256, 1e6)):
        assert np.abs(fa.rope_table(rows, rot, base).numpy().astype(np.float64)
                      - plain.rope_table(rows, rot, base)).max() <= 2.0 ** -23
    assert fa.rope_table(0, 16).shape == (0, 16)
    for bad in ((4, 24, 1e4), (4, 272, 1e4), (4, 16, 0.0), (4, 16, float("inf")), (4, 16, float("nan"))):
        with pytest.raises(fa.FAError):
            fa.rope_table(*bad)
    with pytest.raises(ValueError):
        fa.rope_table(-1, 16)
    assert fa.lib.fa_rope_table(4, 16, 1e4, None) == fa.FA_ERR_INVALID


def _append_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(k_new=Fake(0x1000, (3, 2, 128), bf), v_new=Fake(0x2000, (3, 2, 128), bf),
                k_pages=Fake(0x3000, (9, 2, 32, 128), bf), v_pages=Fake(0x4000, (9, 2, 32, 128), bf),
                cur_pos=Fake(0x5000, (3,), i32), block_table=Fake(0x6000, (3, 4), i32), q=Fake(0x7000, (3, 8, 128), bf),
                q_out=Fake(0x8000, (24, 128), bf), rope_table=Fake(0x9000, (64, 128), torch.float32),
                key_bounds=Fake(0xa000, (9, 2, 2, 128), bf), cache_seqlens=Fake(0xb000, (3,), i32))


def test_binding_refuses_append_tensors_that_do_not_fit(fa):
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    cpu, other = torch.device("cpu"), torch.device("cuda", 1)
    for bad in (dict(k_new=Fake(0x1000, (3, 2, 64), bf)), dict(k_new=Fake(0x1000, (6, 128), bf)),
                dict(v_new=Fake(0x2000, (2, 2, 128), bf)), dict(v_new=Fake(0x2000, (3, 2, 128), f32)),
                dict(k_new=Fake(0x1000, (3, 2, 128), torch.float16), v_new=Fake(0x2000, (3, 2, 128), torch.float16)),
                dict(k_new=Fake(0x1000, (3, 2, 128), bf, strides=(512, 1, 2))),
                dict(k_pages=Fake(0x3000, (9, 2, 32, 128), f32)), dict(k_pages=Fake(0x3000, (9, 2, 32, 128), bf, cpu)),
                dict(v_pages=Fake(0x4000, (8, 2, 32, 128), bf)), dict(v_pages=Fake(0x4000, (9, 2, 32, 128), bf, other)),
                dict(v_pages=Fake(0x4000, (9, 2, 32, 128), bf, contiguous=False)),
                dict(k_pages=Fake(0x3000, (9, 2, 32, 64), torch.uint8), v_pages=Fake(0x4000, (9, 2, 32, 64), torch.uint8)),
                dict(k_pages=Fake(0x3000, (9, 2, 32, 128), torch.int8), v_pages=Fake(0x4000, (9, 2, 32, 128), torch.int8),
                     k_scales=Fake(0x1, (9, 2, 32), f32), v_scales=Fake(0x1, (9, 2, 31), f32)),
                dict(k_scales=Fake(0x1, (9, 2, 32), f32)), dict(cur_pos=Fake(0x5000, (3,), torch.int64)),
                dict(cur_pos=Fake(0x5000, (2,), i32)), dict(block_table=Fake(0x6000, (2, 4), i32)),
                dict(q=Fake(0x7000, (3, 8, 64), bf)), dict(q_out=Fake(0x8000, (8, 3, 128), bf)),
                dict(q=None), dict(rope_table=Fake(0x9000, (64, 128), bf)), dict(rope_table=Fake(0x9000, (64,), f32)),
                dict(key_bounds=Fake(0xa000, (9, 2, 128), bf)), dict(key_bounds=Fake(0xa000, (9, 2, 2, 128), f32)),
                dict(cache_seqlens=Fake(0xb000, (4,), i32)), dict(cu_seqlens=Fake(0xc000, (3,), i32))):
        kw = dict(_append_tensors(), **bad)
        args = [kw.pop(n) for n in ("k_new", "v_new", "k_pages", "v_pages", "cur_pos", "block_table")]
        with pytest.raises(ValueError):
            fa.kv_append_rope_paged(*args, **kw)


def test_binding_refuses_decode_tensors_that_do_not_fit(fa, monkeypatch):
    bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    other = torch.device("cuda", 1)

    def good():
        return dict(q=Fake(0x1000, (24, 128), bf), k_pages=Fake(0x2000, (9, 2, 32, 64), u8),
                    v_pages=Fake(0x3000, (9, 2, 32, 64), u8), cache_seqlens=Fake(0x4000, (3,), i32),
                    block_table=Fake(0x5000, (3, 4), i32), k_scales=Fake(0x6000, (9, 2, 32, 2), f32),
                    v_scales=Fake(0x7000, (9, 2, 32, 2), f32), out=Fake(0x8000, (24, 128), bf),
                    workspace=Fake(0x9000, (1 << 24,), u8))

    for bad in (dict(q=Fake(0x1000, (24, 128), f32)), dict(q=Fake(0x1000, (23, 128), bf)),
                dict(q=Fake(0x1000, (24, 2, 128), bf)), dict(q=Fake(0x1000, (24, 128), bf, other)),
                dict(k_pages=Fake(0x2000, (9, 2, 32, 128), u8)), dict(v_pages=Fake(0x3000, (9, 2, 32, 64), torch.int8)),
                dict(k_scales=None), dict(k_scales=Fake(0x6000, (9, 2, 32), f32)),
                dict(v_scales=Fake(0x7000, (9, 2, 32, 2), bf)), dict(cache_seqlens=Fake(0x4000, (3,), torch.int64)),
                dict(cache_seqlens=Fake(0x4000, (3, 1), i32)), dict(block_table=Fake(0x5000, (4, 3), i32)),
                dict(block_table=Fake(0x5000, (12,), i32)), dict(out=Fake(0x8000, (24, 64), bf)),
                dict(out=Fake(0x8000, (24, 128), f32)), dict(workspace=Fake(0x9000, (1 << 24,), u8, other)),
                dict(hq=7), dict(hkv=0)):
        kw = dict(good(), hq=8, hkv=2)
        kw.update(bad)
        args = [kw.pop(n) for n in ("q", "k_pages", "v_pages", "cache_seqlens", "block_table")]
        with pytest.raises(ValueError):
            fa.attention_decode_paged(*args, **kw)
        for sel in (Fake(0xa000, (3, 2, 4), i32),):
            with pytest.raises(ValueError):
                fa.attention_decode_selected(*args, sel, **kw)
    kw = dict(good(), hq=8, hkv=2)
    args = [kw.pop(n) for n in ("q", "k_pages", "v_pages", "cache_seqlens", "block_table")]
    with pytest.raises(ValueError):
        fa.attention_decode_paged(*args, split_keys=256, **kw)
    for sel in (Fake(0xa000, (3, 2, 4), torch.int64), Fake(0xa000, (3, 1, 4), i32), Fake(0xa000, (3, 8), i32),
                Fake(0xa000, (3, 2, 4), i32, other)):
        with pytest.raises(ValueError):
            fa.attention_decode_selected(*args, sel, **kw)


    # a scale that fp32 does not hold is the library's to refuse
    for scale in (1e39, float("inf"), float("nan")):
        with monkeypatch.context() as m:
            m.setattr(fa, "_on_device", lambda dev, stream, what, fn, *a: statuses.append(fn(*a, None)))
            statuses = []
            fa.attention_decode_paged(*args, scale=scale, **kw)
            assert statuses == [fa.FA_ERR_INVALID]


def test_packed_arguments_have_the_structures_layout(fa):
    for cls, pack in ((fa.KvAppendRopeParams, fa._pack_append), (fa.KvReadParams, fa._pack_read),
                      (fa.PageSelectParams, fa._pack_select), (fa.DecodeParams, fa._pack_decode),
                      (fa.KvPages, fa._pack_pages)):
        values = []
        for i, (_, c) in enumerate(cls._fields_):
            whole = c in (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t)
            values.append(i + 1 if whole else i + 0.5 if c is ctypes.c_float
                          else bytes((7 * i + j) % 251 for j in range(ctypes.sizeof(c))))
        packed = cls.from_buffer_copy(pack(*values))
        for (name, _), v in zip(cls._fields_, values):
            got = getattr(packed, name)
            assert (bytes(got) if isinstance(v, bytes) else got) == v, (cls, name)


def test_binding_refuses_select_and_read_tensors_that_do_not_fit(fa):
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8

    def select(**bad):
        kw = dict(q=Fake(0x1000, (24, 128), bf), key_bounds=Fake(0x2000, (9, 2, 2, 128), bf),
                  cache_seqlens=Fake(0x3000, (3,), i32), block_table=Fake(0x4000, (3, 4), i32),
                  out=Fake(0x5000, (3, 2, 4), i32), workspace=Fake(0x6000, (1 << 20,), u8), hq=8, hkv=2, page_size=32,
                  top_k=4)
        kw.update(bad)
        args = [kw.pop(n) for n in ("q", "key_bounds", "cache_seqlens", "block_table")]
        return fa.page_select(*args, **kw)

    for bad in (dict(key_bounds=Fake(0x2000, (9, 2, 128), bf)), dict(key_bounds=Fake(0x2000, (9, 1, 2, 128), bf)),
                dict(q=Fake(0x1000, (24, 128), torch.float32)), dict(out=Fake(0x5000, (3, 2, 5), i32)),
                dict(out=Fake(0x5000, (3, 2, 4), torch.int64)), dict(block_table=Fake(0x4000, (2, 4), i32)),
                dict(out=None, top_k=0), dict(top_k=2 ** 32 + 4, out=Fake(0x5000, (3, 2, 2 ** 32 + 4), i32)),
                dict(page_size=2 ** 32 + 32), dict(n_first=2 ** 32)):
        with pytest.raises(ValueError):
            select(**bad)
    pools = [Fake(0x1000, (9, 2, 32, 128), bf), Fake(0x2000, (9, 2, 32, 128), bf)]
    table, cu = Fake(0x4000, (3, 4), i32), Fake(0x3000, (4,), i32)
    out = Fake(0x5000, (2, 10, 128), bf)
    for bad in (dict(start=Fake(0x6000, (4,), i32)), dict(k_out=Fake(0x5000, (2, 9, 128), bf)),
                dict(out_dtype=torch.float16), dict(total=2 ** 32 + 10), dict(total=-1)):
        with pytest.raises(ValueError):
            fa.kv_read_paged(*pools, cu, table, **dict(dict(total=10, k_out=out, v_out=out), **bad))
