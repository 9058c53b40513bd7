"""Plain 64-bit (and, where results are bit-exact, rounded fp32) definitions
of the paged serving operators for their tests, on CPU tensors."""
import math

import numpy as np
import torch

F32 = np.float32


def f32(t) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(F32)


def to_bf16(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F32)).bfloat16()


def rope_table(rows, rot, base=10000.0):
    w = base ** (-2.0 * np.arange(rot // 2) / rot)
    a = np.arange(rows)[:, None] * w
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(F32)


def rotate(x, row, interleaved):
    """x [..., d] with the table row [rot]: products and sums rounded to x's type one by one."""
    rot = row.shape[-1]
    c, s = row[: rot // 2].astype(x.dtype), row[rot // 2:].astype(x.dtype)
    a_at = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    b_at = a_at + 1 if interleaved else a_at + rot // 2
    y = x.copy()
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at] = a * c - b * s
    y[..., b_at] = b * c + a * s
    return y


def quantise8(x):
    s = F32(np.abs(x).max()) / F32(127)
    if s == 0:
        return np.zeros(x.shape, np.int8), s
    return np.clip(np.rint(x / s), -127, 127).astype(np.int8), s


def quantise4(x):
    """Packed codes and (step, offset) of one fp32 row."""
    lo = x.min()
    r = F32(x.max() - lo)
    c = np.zeros(x.shape, np.uint8) if r == 0 else np.rint(F32(x - lo) * F32(15) / r).astype(np.uint8)
    return c[0::2] | (c[1::2] << 4), np.array([r / F32(15), lo], F32)


def unpack4(rows):
    c = np.empty(rows.shape[:-1] + (2 * rows.shape[-1],), np.uint8)
    c[..., 0::2], c[..., 1::2] = rows & 15, rows >> 4
    return c


def values(pool, scales):
    """fp64 values of pool rows."""
    if pool.dtype == torch.bfloat16:
        return pool.double().numpy()
    sc = scales.double().numpy()
    if pool.dtype == torch.int8:
        return pool.numpy().astype(np.float64) * sc[..., None]
    return unpack4(pool.numpy()).astype(np.float64) * sc[..., 0:1] + sc[..., 1:2]


class Cache:
    """Random page pools (CPU) behind a shuffled block table; slots at or past
    each length are poisoned (NaN rows or scales), and table entries behind a
    sequence's pages name no page at all."""

    def __init__(self, seed, kind, lens, hkv, d, page, width=None, poison=True, spare=2, offset=0.5):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.lens, self.hkv, self.d, self.page = kind, list(lens), hkv, d, page
        counts = [-(-n // page) for n in lens]
        self.width = width or max(1, max(counts, default=1))
        self.num = sum(counts) + spare
        perm = torch.randperm(self.num, generator=g)
        self.table = torch.full((len(lens), self.width), 2 ** 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = perm[at:at + n].int()
            at += n
        shape = (self.num, hkv, page, d)
        k = torch.randn(shape, generator=g) + offset * torch.randn((1, hkv, 1, d), generator=g)
        k = k + 0.7 * torch.randn((self.num, hkv, 1, d), generator=g)
        v = torch.randn(shape, generator=g)
        k, v = k.bfloat16(), v.bfloat16()
        self.bounds = torch.stack([k.amin(2), k.amax(2)], 2).contiguous()
        if kind == "bf16":
            self.kp, self.vp, self.ks, self.vs = k, v, None, None
        else:
            self.kp, self.ks = self._pack(k.float())
            self.vp, self.vs = self._pack(v.float())
        if poison:
            live = torch.zeros((self.num, page), dtype=torch.bool)
            for b, n in enumerate(lens):
                for i in range(counts[b]):
                    live[self.table[b, i], : min(page, n - i * page)] = True
            dead = ~live[:, None].expand(self.num, hkv, page)
            for rows, scales in ((self.kp, self.ks), (self.vp, self.vs)):
                (rows if scales is None else scales)[dead] = float("nan")

    def _pack(self, x):
        if self.kind == "int8":
            s = x.abs().amax(-1) / 127
            return torch.round(x / s[..., None]).to(torch.int8), s.contiguous()
        lo, hi = x.amin(-1), x.amax(-1)
        c = torch.round((x - lo[..., None]) * 15 / (hi - lo)[..., None]).to(torch.uint8)
        return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), torch.stack([(hi - lo) / 15, lo], -1).contiguous()

    def rows(self, b, g, keys):
        """fp64 K and V rows of KV head g at these key positions of sequence b."""
        keys = np.asarray(keys, dtype=np.int64)
        p, o = self.table[b].numpy()[keys // self.page], keys % self.page
        pick = lambda t: None if t is None else t[p, g, o]
        return values(self.kp[p, g, o], pick(self.ks)), values(self.vp[p, g, o], pick(self.vs))

    def cuda(self):
        for name in ("kp", "vp", "ks", "vs", "table", "bounds"):
            t = getattr(self, name)
            setattr(self, name + "_", None if t is None else t.cuda())
        self.lens_ = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return self


def epilogue_of(y, ops):
    for op, v in ops:
        y = y * v if op == "mul" else y + v
    return y


def attend(cache, q, hq, keys_of, scale, epilogue=()):
    """(out, tolerance) [batch, hq, d] in fp64: softmax attention of q [batch,
    hq, d] over the keys keys_of(b, g), the epilogue of 0 where there are none.

    The tolerance counts the roundings between the cached values and the bf16
    result.  (1) The result: half a bf16 step, 2^-8 |out|.  (2) The weights,
    rounded before the second product: to two bf16 terms (bf16 cache: the
    second holds what the first left, to half a step, 2^-8 2^-8) or to fp16
    (2^-11, and 2^-25 of the largest weight for each key below fp16's normal
    range) -- at most that share of the largest |v|, for 4 bits of the largest
    |code * step|, 15 steps (the offsets' part stays in fp32).  (3) The logits:
    sums of d products in fp32, whose error is at most (d + 8) 2^-23 of the sum
    of the absolute terms, for 4 bits step |q| . code + |offset| sum |q| <=
    sum |q| (15 step + |offset|), since code and offset are summed apart; an
    error e of every logit moves a weight by at most the factor exp(2e), and
    the result by twice that of the largest |v|.  (4) 2^-20 of the largest |v|
    for the exponentials, the weights' sum and merges in fp32, and the second
    product's sums: one addition per 16 keys (two for a bf16 cache's two
    terms), each losing at most 2^-22 of a partial sum, which is at most the
    largest |v|, or |code * step|, times the weights' sum."""
    B, d = q.shape[0], q.shape[-1]
    group = hq // cache.hkv
    out, tol = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    for b in range(B):
        for g in range(cache.hkv):
            keys = keys_of(b, g)
            hs = slice(g * group, (g + 1) * group)
            if len(keys) == 0:
                out[b, hs] = epilogue_of(np.zeros((group, d)), epilogue)
                tol[b, hs] = 2.0 ** -8 * np.abs(out[b, hs])
                continue
            k, v = cache.rows(b, g, keys)
            x = q[b, hs] @ k.T * scale
            w = np.exp(x - x.max(-1, keepdims=True))
            y = (w / w.sum(-1, keepdims=True)) @ v
            vmax = np.abs(v).max(0)
            terms = (np.abs(q[b, hs]) @ np.abs(k).T).max()
            wide = vmax
            weights = 2.0 ** -16 if cache.kind == "bf16" else 2.0 ** -11 + 2.0 ** -25 * len(keys)
            sums = (len(keys) / 8 + 2) * 2.0 ** -22
            if cache.kind == "int4":
                p, o = cache.table[b].numpy()[np.asarray(keys) // cache.page], np.asarray(keys) % cache.page
                step_k, off_k = (cache.ks[p, g, o].double().numpy()[:, i] for i in (0, 1))
                terms = (np.abs(q[b, hs]).sum(-1).max() * (15 * step_k + np.abs(off_k)).max())
                wide = np.full(d, 15 * cache.vs[p, g, o].double().numpy()[:, 0].max())
            logit = (d + 8) * 2.0 ** -23 * terms * scale
            gain = np.prod([v_ for op, v_ in epilogue if op == "mul"]) if epilogue else 1.0
            y = epilogue_of(y, epilogue)
            out[b, hs] = y
            tol[b, hs] = (2.0 ** -8 * np.abs(y)
                          + abs(gain) * ((weights + sums) * wide + 2 * (math.exp(2 * logit) - 1) * vmax
                                         + 2.0 ** -20 * vmax))
    return out, tol


def select(cache, q, hq, top_k, n_first, n_recent):
    """int32 [batch, hkv, top_k] by the definition, sums in fp64."""
    B = q.shape[0]
    group = hq // cache.hkv
    got = np.full((B, cache.hkv, top_k), -1, np.int32)
    bounds = cache.bounds.double().numpy()
    for b, n in enumerate(cache.lens):
        count = -(-n // cache.page)
        ids = cache.table[b, :count].numpy()
        for g in range(cache.hkv):
            qg = q[b, g * group:(g + 1) * group]
            score = np.maximum(qg[:, None] * bounds[ids, g, 0], qg[:, None] * bounds[ids, g, 1]).sum(-1).astype(F32).max(0)
            score[:n_first] = np.inf
            score[max(0, count - n_recent):] = np.inf
            best = np.sort(np.argsort(-score, kind="stable")[:top_k])
            got[b, g, : len(best)] = best
    return got


def append(cache, k, v, q, cur, new, table, interleaved, total=None):
    """The caches after appending (in place), the rotated queries as bf16 [total, hq, d] and the new lengths: every
    operation rounded to fp32 as the definition says.  k, v, q: fp32 numpy [total, heads, d]; table None: no rotation."""
    at, lens = 0, []
    q_out = None if q is None else np.zeros_like(q)
    for b, n in enumerate(new):
        for i in range(n):
            slot = cur[b] + i
            page, off = int(cache.table[b, slot // cache.page]), slot % cache.page
            kr, qr = k[at], None if q is None else q[at]
            if table is not None:
                kr = rotate(kr, table[slot], interleaved)
                qr = None if q is None else rotate(qr, table[slot], interleaved)
            if q is not None:
                q_out[at] = qr
            for g in range(cache.hkv):
                for x, pool, scales in ((kr[g], cache.kp, cache.ks), (v[at, g], cache.vp, cache.vs)):
                    if cache.kind == "bf16":
                        pool[page, g, off] = to_bf16(x)
                        continue
                    c, s = (quantise8 if cache.kind == "int8" else quantise4)(x)
                    pool[page, g, off] = torch.from_numpy(c)
                    scales[page, g, off] = torch.from_numpy(np.asarray(s))
                kb = to_bf16(kr[g])
                if off == 0:
                    cache.bounds[page, g, 0], cache.bounds[page, g, 1] = kb, kb
                else:
                    cache.bounds[page, g, 0] = torch.minimum(cache.bounds[page, g, 0], kb)
                    cache.bounds[page, g, 1] = torch.maximum(cache.bounds[page, g, 1], kb)
            at += 1
        lens.append(cur[b] + n)
    return None if q is None else to_bf16(q_out), lens
