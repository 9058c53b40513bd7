"""Cases of the paged serving operators: the rotated append, attention over a
4-bit cache, and attention over the pages that a cheap score selects.

Three kinds of pass over page pools [num_pages, hkv, page_size, d]:

  append   the new tokens' Q and K are rotated to their positions, K and V
           written to their slots (bf16, int8 with a scale per row, or 4 bits
           with a step and an offset per row), and each page's per-channel key
           bounds brought up to date; quantised rows are read back.
  decode4  one query per sequence and head attends to a 4-bit cache.
  sparse   one query per sequence and head scores every page by the upper
           bound that the page's key bounds give, and attends to the best.

Where `own` is true the framework's entry points make these passes, else
elementary torch operations do.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def _lens(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # the append of one chat's decode step: one token, latency only
        dict(name="append_one_bf16", kind="append", cache="bf16", hq=32, hkv=8, d=128, page=64, rot=128,
             interleaved=False, bounds=True, past="1000", new="1", width=32),
        # the append of a served batch's decode step into a 4-bit cache
        dict(name="append_step_int4", kind="append", cache="int4", hq=32, hkv=8, d=128, page=64, rot=128,
             interleaved=False, bounds=True, past=",".join(str(37 * i % 4001) for i in range(96)),
             new=",".join(["1"] * 96), width=64),
        # ragged prompts and prompt chunks, some of them single tokens, half the channels rotated in pairs
        dict(name="append_ragged_int8", kind="append", cache="int8", hq=16, hkv=4, d=64, page=128, rot=32,
             interleaved=True, bounds=False, past="0,511,64,0,7,4096,0,1,1023,0", new="4097,1,777,1024,1,33,2048,5,1,900",
             width=64),
        # one long prompt into a 4-bit cache
        dict(name="append_long_int4", kind="append", cache="int4", hq=32, hkv=8, d=128, page=64, rot=128,
             interleaved=False, bounds=True, past="0", new="16384", width=256),
        # a short chat over a 4-bit cache: latency only
        dict(name="decode4_one_short", kind="decode4", hq=32, hkv=8, d=128, page=64, window=0, lens="257", width=8),
        # a served batch with cache lengths spread over 1024 .. 32768
        dict(name="decode4_batch_ragged", kind="decode4", hq=32, hkv=8, d=128, page=256, window=0, width=128,
             lens="28673,21889,17797,9601,10753,2369,3457,1537,6593,26561,21505,29953,16897,20097,32641,24245"),
        # one long document, eight query heads to a KV head
        dict(name="decode4_long_gqa8", kind="decode4", hq=64, hkv=8, d=128, page=128, window=0, lens="131071", width=1024),
        # wide heads without sharing, a sliding window over part of the cache
        dict(name="decode4_window_d256", kind="decode4", hq=8, hkv=8, d=256, page=64, window=1024, width=80,
             lens="33,5000,1024,2047,1,4097,3333,0,512,1025,4444,4999"),
        # one chat of 32k tokens, 2048 of them attended, bf16 cache
        dict(name="sparse_one_bf16", kind="sparse", cache="bf16", hq=32, hkv=8, d=128, page=64, top=32, first=1, recent=2,
             lens="32769", width=520),
        # a served batch, small pages, 4-bit cache
        dict(name="sparse_batch_int4", kind="sparse", cache="int4", hq=32, hkv=8, d=128, page=32, top=64, first=1, recent=2,
             lens="28673,21889,17797,9601,10753,2369,3457,1537,6593,26561,21505,29953,16897,20097,32641,24245", width=1024),
        # narrow heads, int8 cache, some sequences shorter than the selection
        dict(name="sparse_ragged_int8", kind="sparse", cache="int8", hq=16, hkv=2, d=64, page=64, top=32, first=1, recent=1,
             lens="16384,1,12345,2048,2049,511,9999,15001,64,13131,7777,16001", width=256),
        # a few very long documents
        dict(name="sparse_long_bf16", kind="sparse", cache="bf16", hq=32, hkv=8, d=128, page=128, top=32, first=2, recent=2,
             lens="131071,98305,130000,65537", width=1024),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["append", "decode4", "sparse"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    page = rng.choice([32, 64, 128, 256])
    batch = spread(1, 48)
    budget = 270000 * 8 * 128 // (hkv * d)  # cached tokens of the largest listed batch, at this width
    if kind == "append":
        past = [rng.randint(0, 4000) for _ in range(batch)]
        most = max(1, 16384 * 48 * 128 // ((hq + 2 * hkv) * d) // batch)
        new = [1 if rng.random() < 0.5 else spread(1, max(1, min(4000, most))) for _ in range(batch)]
        if rng.random() < 0.4:
            new = [1] * batch
        return dict(kind=kind, cache=rng.choice(["bf16", "int8", "int4"]), hq=hq, hkv=hkv, d=d, page=page,
                    rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3, bounds=rng.random() < 0.6,
                    past=",".join(map(str, past)), new=",".join(map(str, new)),
                    width=max(-(-(p + n) // page) for p, n in zip(past, new)) + rng.randint(0, 3))
    top_len = max(1, min(131072, budget // batch))
    lens = [spread(1, top_len) for _ in range(batch)]
    width = max(-(-n // page) for n in lens) + rng.randint(0, 5)
    case = dict(kind=kind, hq=hq, hkv=hkv, d=d, page=page, lens=",".join(map(str, lens)), width=width)
    if kind == "decode4":
        return dict(case, window=rng.choice([0, 0, 0, rng.randint(1, top_len)]))
    return dict(case, cache=rng.choice(["bf16", "int8", "int4"]), top=spread(4, 64), first=rng.randint(0, 2),
                recent=rng.randint(1, 2))


def _pages_of(lens, page):
    return [-(-n // page) for n in lens]


# ---------------------------------------------------------------- the cache formats

def _quantise8(x):
    """Codes and scales of rows x [..., d] fp32: scale = max|x| / 127 (a tensor divides: a number would multiply by 1/127)."""
    s = x.abs().amax(-1)
    s = s / torch.full_like(s, 127.0)
    c = torch.round(x / torch.where(s > 0, s, 1.0)[..., None]).clamp(-127, 127)
    return c.to(torch.int8), s


def _quantise4(x):
    """Packed codes [..., d/2] (channel 2j in the low half of byte j) and (step, offset) [..., 2] of rows x [..., d] fp32:
    code = round(15 (x - min) / (max - min)), step = (max - min) / 15, offset = min."""
    lo, r = x.amin(-1), x.amax(-1) - x.amin(-1)
    c = torch.round((x - lo[..., None]) * 15.0 / torch.where(r > 0, r, 1.0)[..., None]).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([r / torch.full_like(r, 15.0), lo], -1)


def _values(rows, scales):
    """fp32 values of cached rows: [..., d] of bf16, int8 codes with scales [...], or packed 4-bit codes with [..., 2]."""
    if rows.dtype == torch.bfloat16:
        return rows.float()
    if rows.dtype == torch.int8:
        return rows.float() * scales[..., None]
    c = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float()
    return c * scales[..., 0:1] + scales[..., 1:2]


# ---------------------------------------------------------------- prepare

def _table(lens_pages, width, gen, dev):
    """A block table of distinct, shuffled pages; entries behind a sequence's pages are other sequences' pages."""
    total = sum(lens_pages) + 3
    perm = torch.randperm(total, generator=gen, device=dev)
    table = perm[torch.randint(0, total, (len(lens_pages), width), generator=gen, device=dev)]
    at = 0
    for b, n in enumerate(lens_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(torch.int32).contiguous(), total


def _pools(case, cache, total, gen, dev):
    """Keys with a centre per page and loud channels, values plain: what trained heads look like in a cache."""
    hkv, d, page = case["hkv"], case["d"], case["page"]
    shape = (total, hkv, page, d)
    k = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(0.7)
    k += torch.randn((total, hkv, 1, d), generator=gen, device=dev) * 0.7
    loud = (torch.rand((hkv, 1, d), generator=gen, device=dev) < 0.05) * torch.randn((hkv, 1, d), generator=gen, device=dev)
    k += loud * 4.0
    v = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    k, v = k.bfloat16(), v.bfloat16()
    bounds = torch.stack([k.amin(2), k.amax(2)], 2).contiguous()  # [P, hkv, 2, d]
    if cache == "bf16":
        return k, v, None, None, bounds
    quantise = _quantise8 if cache == "int8" else _quantise4
    kc, ks = quantise(k.float())
    vc, vs = quantise(v.float())
    return kc.contiguous(), vc.contiguous(), ks.contiguous(), vs.contiguous(), bounds


def _rope_table(rows, rot, dev):
    """cos | sin of position * 10000^(-2i/rot), in 64 bits, rounded to fp32: [rows, rot]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    s = dict(case=case, hq=hq, hkv=hkv, d=d, page=page)
    if case["kind"] == "append":
        past, new = _lens(case["past"]), _lens(case["new"])
        total = sum(new)
        s["table"], num = _table(_pages_of([p + n for p, n in zip(past, new)], page), case["width"], gen, dev)
        s["kp"], s["vp"], s["ks"], s["vs"], bounds = _pools(case, case["cache"], num, gen, dev)
        s["bounds"] = bounds if case["bounds"] else None
        # one projection's output, Q, K and V of a token side by side
        qkv = (torch.randn((total, (hq + 2 * hkv) * d), generator=gen, device=dev) * 1.2).bfloat16()
        s["q"] = qkv[:, :hq * d].view(total, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(total, hkv, d)
        s["cur"] = torch.tensor(past, dtype=torch.int32, device=dev)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["one"] = all(n == 1 for n in new)
        s["total"] = total
        s["lens"] = torch.zeros(len(new), dtype=torch.int32, device=dev)
        s["rope"] = _rope_table(max(p + n for p, n in zip(past, new)) + 16, case["rot"], dev)
        return s
    lens = _lens(case["lens"])
    s["table"], num = _table(_pages_of(lens, page), case["width"], gen, dev)
    cache = "int4" if case["kind"] == "decode4" else case["cache"]
    s["kp"], s["vp"], s["ks"], s["vs"], s["bounds"] = _pools(case, cache, num, gen, dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["q"] = (torch.randn((len(lens) * hq, d), generator=gen, device=dev) * 1.5).bfloat16()
    # slots behind a sequence's last key were never written: they hold NaN
    for b, n in enumerate(lens):
        if n % page:
            p = int(s["table"][b, n // page])
            for rows, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
                (rows if scales is None else scales)[p, :, n % page:] = float("nan")
    return s


# ---------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, interleaved):
    """x [total, h, d] fp32 with cos, sin [total, 1, rot/2]."""
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _plain_append(s):
    case, page = s["case"], s["page"]
    t = torch.arange(s["total"], device=s["cur"].device)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    slot = s["cur"].long()[seq] + t - s["cu"].long()[seq]
    ids = s["table"][seq, slot // page].long()
    off = slot % page
    cs = s["rope"][slot]
    cos, sin = cs[:, None, :case["rot"] // 2], cs[:, None, case["rot"] // 2:]
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"]).bfloat16()
    q_out = q.reshape(-1, s["d"]) if s["one"] else q.transpose(0, 1).contiguous()
    k, v = _rotate(s["k"].float(), cos, sin, case["interleaved"]), s["v"].float()
    s["lens"].copy_(s["cur"] + (s["cu"][1:] - s["cu"][:-1]))
    out = dict(q=q_out, lens=s["lens"])
    if s["bounds"] is not None:
        b = s["bounds"].float()
        fresh = torch.zeros(b.shape[0], dtype=torch.int32, device=b.device)
        fresh = fresh.scatter_reduce(0, ids, (off == 0).int(), "amax") > 0
        kb = k.bfloat16().float()
        lo = torch.where(fresh[:, None, None], float("inf"), b[:, :, 0]).index_reduce_(0, ids, kb, "amin")
        hi = torch.where(fresh[:, None, None], float("-inf"), b[:, :, 1]).index_reduce_(0, ids, kb, "amax")
        s["bounds"].copy_(torch.stack([lo, hi], 2))
        out["bounds"] = s["bounds"]
    if case["cache"] == "bf16":
        s["kp"][ids, :, off] = k.bfloat16()
        s["vp"][ids, :, off] = v.bfloat16()
        return dict(out, kp=s["kp"], vp=s["vp"])
    quantise = _quantise8 if case["cache"] == "int8" else _quantise4
    s["kp"][ids, :, off], s["ks"][ids, :, off] = quantise(k)
    s["vp"][ids, :, off], s["vs"][ids, :, off] = quantise(v)
    back = [_values(p[ids, :, off], c[ids, :, off]).bfloat16().transpose(0, 1).contiguous()
            for p, c in ((s["kp"], s["ks"]), (s["vp"], s["vs"]))]
    return dict(out, k=back[0], v=back[1], ks=s["ks"], vs=s["vs"])


def _attend(q, k, v, seen):
    """q [B, hkv, G, d], k and v [B, hkv, n, d], seen [B, 1 or hkv, n]: softmax attention; zeros where nothing is seen."""
    logits = q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])
    logits = torch.where(seen[:, :, None], logits, float("-inf"))
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    return p @ torch.where(seen[..., None], v, 0.0) / torch.where(total > 0, total, 1.0)


def _plain_decode4(s):
    b, width = s["table"].shape
    hkv, d, page = s["hkv"], s["d"], s["page"]
    ids = s["table"].long()
    k = _values(s["kp"][ids], s["ks"][ids]).transpose(1, 2).reshape(b, hkv, width * page, d)
    v = _values(s["vp"][ids], s["vs"][ids]).transpose(1, 2).reshape(b, hkv, width * page, d)
    at = torch.arange(width * page, device=k.device)
    n = s["lens"].long()[:, None]
    seen = at < n
    if s["case"]["window"] > 0:
        seen = seen & (at >= n - s["case"]["window"])
    q = s["q"].float().view(b, hkv, -1, d)
    return _attend(q, k, v, seen[:, None]).reshape(-1, d).bfloat16()


def _plain_sparse(s):
    case = s["case"]
    b, width = s["table"].shape
    hkv, d, page, top = s["hkv"], s["d"], s["page"], case["top"]
    ids = s["table"].long()
    # the scores in 64 bits: which of two near pages is better has to come out right
    q = s["q"].double().view(b, hkv, -1, d)
    bounds = s["bounds"][ids].permute(0, 2, 3, 4, 1).double()  # [B, hkv, 2, d, pages]
    score = (q.clamp(max=0) @ bounds[:, :, 0] + q.clamp(min=0) @ bounds[:, :, 1]).float().amax(2)  # [B, hkv, pages]
    page_no = torch.arange(width, device=q.device)
    count = (s["lens"].long() + page - 1) // page
    there = (page_no < count[:, None])[:, None]
    forced = ((page_no < case["first"]) | (page_no >= count[:, None] - case["recent"]))[:, None]
    score = torch.where(there, torch.where(forced, float("inf"), score), float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    chosen = torch.where(torch.gather(there.expand_as(score), -1, order), order, width).sort(-1).values
    chosen = torch.nn.functional.pad(chosen, (0, top - chosen.shape[-1]), value=width)
    hit = chosen < width
    chosen = torch.where(hit, chosen, 0)
    phys = torch.gather(ids[:, None].expand(b, hkv, width), -1, chosen)
    head = torch.arange(hkv, device=q.device)[None, :, None]
    scales = (None, None) if s["ks"] is None else (s["ks"][phys, head], s["vs"][phys, head])
    k = _values(s["kp"][phys, head], scales[0]).reshape(b, hkv, top * page, d)
    v = _values(s["vp"][phys, head], scales[1]).reshape(b, hkv, top * page, d)
    at = chosen[..., None] * page + torch.arange(page, device=q.device)
    seen = (hit[..., None] & (at < s["lens"].long()[:, None, None, None])).reshape(b, hkv, top * page)
    out = _attend(s["q"].float().view(b, hkv, -1, d), k, v, seen).reshape(-1, d).bfloat16()
    return dict(selected=torch.where(hit, chosen, -1).to(torch.int32), out=out)


# ---------------------------------------------------------------- the framework's calls

def _own_append(s):
    from flashattention_attention_b200 import fa
    case = s["case"]
    q = fa.kv_append_rope_paged(s["k"], s["v"], s["kp"], s["vp"], s["cur"], s["table"], q=s["q"], rope_table=s["rope"],
                                interleaved=case["interleaved"], k_scales=s["ks"], v_scales=s["vs"],
                                key_bounds=s["bounds"], cu_seqlens=None if s["one"] else s["cu"],
                                cache_seqlens=s["lens"])
    out = dict(q=q, lens=s["lens"])
    if s["bounds"] is not None:
        out["bounds"] = s["bounds"]
    if case["cache"] == "bf16":
        return dict(out, kp=s["kp"], vp=s["vp"])
    k, v = fa.kv_read_paged(s["kp"], s["vp"], s["cu"], s["table"], total=s["total"], start=s["cur"], k_scales=s["ks"],
                            v_scales=s["vs"])
    return dict(out, k=k, v=v, ks=s["ks"], vs=s["vs"])


def _own_decode4(s):
    from flashattention_attention_b200 import fa
    return fa.attention_decode_paged(s["q"], s["kp"], s["vp"], s["lens"], s["table"], hq=s["hq"], hkv=s["hkv"],
                                     k_scales=s["ks"], v_scales=s["vs"], window=s["case"]["window"])


def _own_sparse(s):
    from flashattention_attention_b200 import fa
    case = s["case"]
    selected = fa.page_select(s["q"], s["bounds"], s["lens"], s["table"], hq=s["hq"], hkv=s["hkv"], page_size=s["page"],
                              top_k=case["top"], n_first=case["first"], n_recent=case["recent"])
    out = fa.attention_decode_selected(s["q"], s["kp"], s["vp"], s["lens"], s["table"], selected, hq=s["hq"],
                                       hkv=s["hkv"], k_scales=s["ks"], v_scales=s["vs"])
    return dict(selected=selected, out=out)


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"append": _own_append, "decode4": _own_decode4, "sparse": _own_sparse}[kind](state)
    return {"append": _plain_append, "decode4": _plain_decode4, "sparse": _plain_sparse}[kind](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(cache, d):
    return {"bf16": 2 * d, "int8": d + 4, "int4": d // 2 + 8}[cache]


def work(case):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    if case["kind"] == "append":
        past, new = _lens(case["past"]), _lens(case["new"])
        total = sum(new)
        n = total * (2 * hq + 2 * hkv) * d * 2              # Q, K, V in, Q out
        n += 2 * total * hkv * _row_bytes(case["cache"], d)  # rows written
        n += total * case["rot"] * 4                         # a table row for each token
        if case["bounds"]:
            touched = sum((p + m - 1) // page - p // page + 1 for p, m in zip(past, new))
            n += touched * hkv * 4 * d
        if case["cache"] != "bf16":
            n += 2 * total * hkv * (_row_bytes(case["cache"], d) + 2 * d)  # read back
        return {"bytes": n, "flops": 3 * total * (hq + hkv) * case["rot"]}
    lens = _lens(case["lens"])
    n = 2 * 2 * len(lens) * hq * d
    if case["kind"] == "decode4":
        keys = sum(min(x, case["window"]) if case["window"] > 0 else x for x in lens)
        return {"bytes": n + 2 * keys * hkv * _row_bytes("int4", d), "flops": 4 * keys * hq * d}
    pages = _pages_of(lens, page)
    keys = sum(x if p <= case["top"] else (case["top"] - 1) * page + x - (p - 1) * page for x, p in zip(lens, pages))
    n += sum(pages) * hkv * 4 * d + 4 * len(lens) * hkv * case["top"]
    return {"bytes": n + 2 * keys * hkv * _row_bytes(case["cache"], d),
            "flops": 2 * sum(pages) * hq * d + 4 * keys * hq * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_row(codes, scales, cache):
    if cache == "bf16":
        return codes.double()
    if cache == "int8":
        return codes.double() * scales.double().unsqueeze(-1)
    both = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    both[..., 0::2] = (codes % 16).double()
    both[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    return both * scales[..., :1].double() + scales[..., 1:].double()


def _exact_append(case, s):
    hq, hkv, d, page, rot = case["hq"], case["hkv"], case["d"], case["page"], case["rot"]
    past, new = _lens(case["past"]), _lens(case["new"])
    half = rot // 2
    first = torch.arange(half, device=s["q"].device)
    a_at, b_at = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
    where, row = [], 0
    for b, n in enumerate(new):
        slots = torch.arange(past[b], past[b] + n, device=s["q"].device)
        where.append((s["table"][b].long()[slots // page], slots % page, slots))
    ids, off, slots = (torch.cat([w[i] for w in where]) for i in range(3))
    cos, sin = s["rope"].double()[slots][:, :half].unsqueeze(1), s["rope"].double()[slots][:, half:].unsqueeze(1)

    def turned(x):
        y = x.double().clone()
        y[..., a_at] = x.double()[..., a_at] * cos - x.double()[..., b_at] * sin
        y[..., b_at] = x.double()[..., b_at] * cos + x.double()[..., a_at] * sin
        return y

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
    out = dict(q=q.reshape(-1, d) if s["one"] else q.transpose(0, 1).contiguous(), lens=None)
    if case["bounds"]:
        bounds = s["bounds"].double().clone()
        for b, n in enumerate(new):
            rows = k[row:row + n]
            row += n
            at = 0
            while at < n:
                slot = past[b] + at
                take = min(n - at, page - slot % page)
                p = int(s["table"][b, slot // page])
                lo, hi = rows[at:at + take].amin(0), rows[at:at + take].amax(0)
                if slot % page:
                    lo, hi = torch.minimum(lo, bounds[p, :, 0]), torch.maximum(hi, bounds[p, :, 1])
                bounds[p, :, 0], bounds[p, :, 1] = lo, hi
                at += take
        out["bounds"] = bounds
    if case["cache"] == "bf16":
        kp, vp = s["kp"].double().clone(), s["vp"].double().clone()
        kp[ids, :, off], vp[ids, :, off] = k, v
        return dict(out, kp=kp, vp=vp)
    for name, x, pool in (("k", k, "ks"), ("v", v, "vs")):
        scales = s[pool].double().clone()
        if case["cache"] == "int8":
            step = x.abs().amax(-1) / 127
            value = torch.round(x / step.clamp(min=1e-300).unsqueeze(-1)) * step.unsqueeze(-1)
            scales[ids, :, off] = step
        else:
            low = x.amin(-1)
            span = x.amax(-1) - low
            step = span / 15
            codes = torch.round(15 * (x - low.unsqueeze(-1)) / span.clamp(min=1e-300).unsqueeze(-1))
            value = codes * step.unsqueeze(-1) + low.unsqueeze(-1)
            scales[ids, :, off, 0], scales[ids, :, off, 1] = step, low
        out[name], out[pool] = value.transpose(0, 1).contiguous(), scales
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(case, s)
    lens, page, hkv, d = _lens(case["lens"]), case["page"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    cache = "int4" if case["kind"] == "decode4" else case["cache"]
    out = torch.zeros((len(lens), case["hq"], d), dtype=torch.float64, device=s["q"].device)
    q = s["q"].double().view(len(lens), case["hq"], d)
    for b, n in enumerate(lens):
        pages = -(-n // page)
        if not n:
            continue
        ids = s["table"][b, :pages].long()
        for g in range(hkv):
            qg = q[b, g * group:(g + 1) * group]
            keys = torch.arange(n, device=q.device)
            if case["kind"] == "decode4":
                if case["window"] > 0:
                    keys = keys[max(0, n - case["window"]):]
            elif pages > case["top"]:
                bound = s["bounds"][ids, g].double()
                best = torch.maximum(qg[:, None] * bound[None, :, 0], qg[:, None] * bound[None, :, 1]).sum(-1).amax(0)
                best = best.float()  # the definition rounds a score once; ties go to the lowest page
                best[:case["first"]] = float("inf")
                best[pages - case["recent"]:] = float("inf")
                keep = torch.zeros(pages, dtype=torch.bool, device=q.device)
                keep[torch.argsort(-best, stable=True)[:case["top"]]] = True
                keys = keys[keep[keys // page]]
            p, o = ids[keys // page], keys % page
            k = _exact_row(s["kp"][p, g, o], None if s["ks"] is None else s["ks"][p, g, o], cache)
            v = _exact_row(s["vp"][p, g, o], None if s["vs"] is None else s["vs"][p, g, o], cache)
            w = torch.softmax((k @ qg.T).T / d ** 0.5, -1)
            out[b, g * group:(g + 1) * group] = w @ v
    out = out.view(-1, d)
    return out if case["kind"] == "decode4" else dict(selected=None, out=out)
