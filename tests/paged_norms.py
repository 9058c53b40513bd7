"""Tolerances of the paged attention that follow the size of the answer: what
the roundings between the cached values and the bf16 result can move it by,
with the weights that the keys really have."""
import numpy as np

import paged_plain as plain


def attend(cache, q, hq, keys_of, scale, span=None):
    """(out, tolerance) [batch, hq, d] in fp64 of the softmax attention of q
    [batch, hq, d] over the keys keys_of(b, g) (some for every head).

    With weights p_j that sum to 1, P(x) = sum_j p_j |x_j|, n keys:
    (1) the result: half a bf16 step, 2^-8 |out|.
    (2) the weights as the second product takes them: two bf16 terms, 2^-16
    P(v); or p step in fp16, half a step of it, 2^-11, and where that is below
    fp16's smallest step, 2^-25 of the largest p step of the 16 tiles of at most
    64 keys up to it: for the 512 keys of 8 tiles 2^-16 of the largest of theirs
    and of the 8 tiles before, 2^-15 of the sum.  On the code, at most 127, or,
    for 4 bits, on code - 7.5, what the codes share being summed in fp32.
    (3) the logits: sums of d products in fp32, each within (d + 8) 2^-23 of the
    sum of the absolute terms (4 bits: |q| times 15 steps and the offset), at
    most e: every weight is within the factor exp(2 e), and so the result
    within (exp(2 e) - 1) (P(v) + |out|).
    (4) exponentials, and the merges' few products: 2^-20 of the same.
    (5) sums over keys in fp32: a thread adds every eighth key's weight (and
    offset) to a sum: one rounding each, and a few for the lanes; the second
    product adds 16 keys at a time (twice for two terms), each addition losing
    at most 2^-22 of a partial sum of |p code step|.  So over the `span` keys
    that one warp has at most (None: all); then the n / span warps' sums are
    merged, every eighth by one warp, with a rounding each (two for l)."""
    B, d = q.shape[0], q.shape[-1]
    group = hq // cache.hkv
    out, tol = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    for b in range(B):
        for g in range(cache.hkv):
            keys = np.asarray(keys_of(b, g))
            n = len(keys)
            m = min(n, span or n)
            merge = (n / m / 4 + 16) * 2.0 ** -24
            hs = slice(g * group, (g + 1) * group)
            k, v = cache.rows(b, g, keys)
            p, o = cache.table[b].numpy()[keys // cache.page], keys % cache.page
            x = q[b, hs] @ k.T * scale
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            y, pv = w @ v, w @ np.abs(v)
            qa = np.abs(q[b, hs])
            if cache.kind == "int4":
                ks, vs = cache.ks[p, g, o].double().numpy(), cache.vs[p, g, o].double().numpy()
                steps = (w @ vs[:, 0])[:, None]
                terms = (qa.sum(-1)[:, None] * (15 * ks[:, 0] + np.abs(ks[:, 1]))).max()
                weights = (2.0 ** -11 + 2.0 ** -15) * 7.5 * steps
                sums = ((m / 8 + 16) * 2.0 ** -24 * (w @ np.abs(vs[:, 1] + 7.5 * vs[:, 0]))[:, None]
                        + (m / 16 + 16) * 2.0 ** -22 * 15 * steps)
            else:
                terms = (qa @ np.abs(k).T).max()
                if cache.kind == "int8":
                    steps = (w @ cache.vs[p, g, o].double().numpy())[:, None]
                    weights = 2.0 ** -11 * pv + 2.0 ** -15 * 127 * steps
                    sums = (m / 16 + 16) * 2.0 ** -22 * pv
                else:
                    weights = 2.0 ** -16 * pv
                    sums = (m / 8 + 16) * 2.0 ** -22 * pv
            sums = sums + (m / 8 + 16) * 2.0 ** -24 * np.abs(y) + merge * (pv + np.abs(y))
            logit = (d + 8) * 2.0 ** -23 * terms * scale
            out[b, hs] = y
            tol[b, hs] = (2.0 ** -8 * np.abs(y) + weights + sums
                          + (np.exp(2 * logit) - 1 + 2.0 ** -20) * (pv + np.abs(y)))
    return out, tol


def repack(cache, k, v, b=0):
    """Sequence b's keys and values become k, v [hkv, n, d] fp32 (rounded to bf16, quantised)."""
    n = k.shape[1]
    at = np.arange(n)
    p, o = cache.table[b].numpy()[at // cache.page], at % cache.page
    for x, pool, scales in ((k, cache.kp, cache.ks), (v, cache.vp, cache.vs)):
        x = x.bfloat16()
        if cache.kind == "bf16":
            pool[p, :, o] = x.transpose(0, 1)
            continue
        x = x.float()
        if cache.kind == "int8":
            s = x.abs().amax(-1) / 127
            pool[p, :, o] = (x / s[..., None]).round().to(pool.dtype).transpose(0, 1)
            scales[p, :, o] = s.transpose(0, 1)
        else:
            lo, r = x.amin(-1), x.amax(-1) - x.amin(-1)
            c = ((x - lo[..., None]) * 15 / r.clamp(min=1e-30)[..., None]).round().to(pool.dtype)
            pool[p, :, o] = (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(0, 1)
            scales[p, :, o, 0], scales[p, :, o, 1] = (r / 15).transpose(0, 1), lo.transpose(0, 1)
    return cache
