"""GPU tests of the paged calls that use a workspace: captured, on two streams,
one workspace for several calls, and in launches over more sequences than one
holds, each row against the definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu


def _fa():
    from flashattention_attention_b200 import fa
    return fa


def _decode_bytes(c, batch, hq, top=0):
    fa = _fa()
    p = fa.DecodeParams(kv_dtype=fa._CACHE_DT[c.kp.dtype], batch=batch, hq=hq, hkv=c.hkv, head_dim=c.d,
                        capacity=c.table.shape[1] * c.page)
    pages = fa.KvPages(None, c.table.shape[1], c.page, c.num)
    return fa.lib.fa_decode_pages_workspace_size(ctypes.byref(p), ctypes.byref(pages), top)


def _run(i):
    """Two calls with workspaces over a cache and queries of their own: an attention and a selection."""
    fa = _fa()
    c = plain.Cache(1000 + i, "int4", [30000, 5000 + 777 * i], 1, 128, 32).cuda()
    c.table_ = torch.nn.functional.pad(c.table_, (0, 5000 - c.width), value=-1).contiguous()
    c.table = c.table_.cpu()
    q = (torch.randn((16, 128), generator=torch.Generator().manual_seed(i)) * 1.5).bfloat16().cuda()
    need = _decode_bytes(c, 2, 8), fa.lib.fa_page_select_workspace_size(2, 1, 5000)
    assert min(need) > 0

    def call(workspace=None, **kw):
        dec, sel = (None, None) if workspace is None else workspace
        out = fa.attention_decode_paged(q, c.kp_, c.vp_, c.lens_, c.table_, hq=8, hkv=1, k_scales=c.ks_, v_scales=c.vs_,
                                        workspace=dec, **kw)
        return out, fa.page_select(q, c.bounds_, c.lens_, c.table_, hq=8, hkv=1, page_size=32, top_k=100, workspace=sel, **kw)

    want = [t.clone() for t in call()]
    qn = q.double().cpu().numpy().reshape(2, 8, 128)
    ref, tol = plain.attend(c, qn, 8, lambda b, g: np.arange(c.lens[b]), 1 / math.sqrt(128))
    assert (np.abs(want[0].double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    assert np.array_equal(want[1].cpu().numpy(), plain.select(c, qn, 8, 100, 1, 1))
    return call, want, need, (c, q)


def test_graphs_with_workspaces_of_their_own_on_two_streams():
    fa, runs = _fa(), []
    for i in range(2):
        call, want, _, hold = _run(i)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        runs.append((graph, out, want, torch.cuda.Stream(), hold))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, *_, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, *_ in runs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert fa.check_device_error() == fa.FA_OK


def test_calls_on_two_streams_at_once():
    fa = _fa()
    runs = [_run(i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (call, *_) in enumerate(runs):
            got[i].append(call(stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, want, *_) in enumerate(runs):
        assert all(torch.equal(a, b) for out in got[i] for a, b in zip(out, want))
    assert fa.check_device_error() == fa.FA_OK


def test_graphs_that_share_a_workspace_on_one_stream():
    """What a serving loop does: one workspace for all its calls, captured or not, one after the other on a stream."""
    fa = _fa()
    runs = [_run(i) for i in range(2)]
    need = [max(r[2][x] for r in runs) for x in range(2)]
    shared = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in need]
    torch.cuda.synchronize()
    graphs = []
    for call, want, *_ in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(shared)
        graphs.append((graph, out, want))
    torch.cuda.synchronize()
    for _ in range(5):
        for (graph, out, want), (call, *_) in zip(graphs, runs):
            graph.replay()
            copies = [t.clone() for t in out] + list(call(shared))
            assert all(torch.equal(a, b) for a, b in zip(copies, want + want))
    assert fa.check_device_error() == fa.FA_OK


@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_more_sequences_than_a_launch_holds(kind):
    """300 sequences with queries, tables and lengths of their own, tiles dealt over the device: launches of 256."""
    fa = _fa()
    hq, hkv, d, page, batch, width = 2, 1, 64, 32, 300, 170
    c = plain.Cache(1010, kind, [page * 400], hkv, d, page, spare=0)
    g = torch.Generator().manual_seed(5)
    c.lens = [int(n) for n in torch.randint(0, 400, (batch,), generator=g)]
    for b in (3, 100, 255, 256, 270, 299):
        c.lens[b] = width * page - b
    c.width, c.table = width, torch.randint(0, 400, (batch, width), generator=g).int()
    c.cuda()
    q = torch.randn((batch * hq, d), generator=g).bfloat16()
    qn = q.double().numpy().reshape(batch, hq, d)
    kw = dict(hq=hq, hkv=hkv, k_scales=c.ks_, v_scales=c.vs_)
    ref, tol = plain.attend(c, qn, hq, lambda b, h: np.arange(c.lens[b]), 1 / math.sqrt(d))

    def check(out):
        assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all(-1).all(-1).all()

    assert _decode_bytes(c, batch, hq, width) > 0
    order = torch.stack([torch.randperm(width, generator=g) for _ in range(batch)]).int()[:, None]
    for b, n in enumerate(c.lens):  # only the first ceil(n / page) entries of a selection count
        pages = -(-n // page)
        order[b, 0, :pages] = torch.randperm(pages, generator=g).int()
    check(fa.attention_decode_selected(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, order.cuda(), **kw))
    if kind == "int4":
        assert _decode_bytes(c, batch, hq) > 0
        check(fa.attention_decode_paged(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, **kw))
    assert fa.check_device_error() == fa.FA_OK


def test_selection_for_more_sequences_than_a_launch_holds():
    """1100 sequences with queries, tables and lengths of their own over up to 160 pages: launches of 1024, pages dealt
    evenly; the choice of every sequence and head, and the attention over it."""
    fa = _fa()
    hq, hkv, d, page, batch, width, top = 4, 2, 64, 32, 1100, 160, 6
    c = plain.Cache(1011, "int8", [page * 700], hkv, d, page, spare=0)
    g = torch.Generator().manual_seed(6)
    c.lens = [int(n) for n in torch.randint(0, width * page + 1, (batch,), generator=g)]
    c.width, c.table = width, torch.stack([torch.randperm(700, generator=g)[:width] for _ in range(batch)]).int()
    c.cuda()
    q = torch.randn((batch * hq, d), generator=g).bfloat16()
    qn = q.double().numpy().reshape(batch, hq, d)
    assert fa.lib.fa_page_select_workspace_size(batch, hkv, width) > 0
    got = fa.page_select(q.cuda(), c.bounds_, c.lens_, c.table_, hq=hq, hkv=hkv, page_size=page, top_k=top, n_recent=2)
    want = plain.select(c, qn, hq, top, 1, 2)
    assert np.array_equal(got.cpu().numpy(), want)
    out = fa.attention_decode_selected(q.cuda(), c.kp_, c.vp_, c.lens_, c.table_, got, hq=hq, hkv=hkv, k_scales=c.ks_,
                                       v_scales=c.vs_)

    def keys(b, h):
        at = [np.arange(p * page, min(c.lens[b], (p + 1) * page)) for p in want[b, h] if p >= 0]
        return np.concatenate(at) if at else np.arange(0)

    ref, tol = plain.attend(c, qn, hq, keys, 1 / math.sqrt(d))
    assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    assert fa.check_device_error() == fa.FA_OK
