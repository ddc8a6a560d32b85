"""Plain 64-bit forms of the decode and scoring operators, and error bounds.

Everything is computed on the CPU from the exact input bits, element by
element from the definitions.  ``HALF`` is half a step of a type relative to
the value: what one rounding to it may be off by.
"""
from __future__ import annotations

import math

import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn)}
F64 = torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def page_table(lens, page_size, num_pages, g, width=None):
    """A shuffled page table for sequences of the given lengths; entries no sequence needs hold -1."""
    need = [-(-n // page_size) for n in lens]
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1]) if width is None else width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = perm.pop()
    return table


def rotate(x, pos, base):
    """Interleaved pairs of x [..., D] turned by pos * base^(-2j/D); returns 64 bits."""
    d = x.shape[-1]
    x = x.to(F64)
    phi = pos * torch.tensor([base ** (-2.0 * j / d) for j in range(d // 2)], dtype=F64)
    c, s = torch.cos(phi), torch.sin(phi)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)


def append(Z, positions, row_seq, table, hq, hkv, d, page_size, base):
    """Per row: None where it is left out, else (q, k, v in 64 bits, page, slot)."""
    out = []
    for i, p in enumerate(positions.tolist()):
        if p < 0:
            out.append(None)
            continue
        z = Z[i].reshape(hq + 2 * hkv, d).to(F64)
        qk = rotate(z[:hq + hkv], p, base) if base else z[:hq + hkv]
        out.append((qk[:hq], qk[hq:], z[hq + hkv:], int(table[row_seq[i], p // page_size]), p % page_size))
    return out


def pages(cache, ids, head):
    """cache[ids, head], for the 8-bit type too (indexed as bytes)."""
    if cache.element_size() == 1:
        return cache.view(torch.uint8)[ids, head].view(cache.dtype)
    return cache[ids, head]


def attention(q, k_cache, v_cache, table, lengths, row_seq, scale, sk=1.0, sv=1.0):
    """(o [M, Hq, D], lse [M, Hq], slack [M, Hq, D], spread [M, Hq]) in 64 bits.  ``slack`` is sum_t p_t |v_t| and
    ``spread`` the largest sum_d |q_d k_td| scale over the keys: what relative errors of p and of s act on."""
    M, hq, d = q.shape
    hkv, page = k_cache.shape[1:3]
    o, slack = torch.zeros(M, hq, d, dtype=F64), torch.zeros(M, hq, d, dtype=F64)
    lse, spread = torch.full((M, hq), -math.inf, dtype=F64), torch.zeros(M, hq, dtype=F64)
    for i in range(M):
        n = max(int(lengths[i]), 0)
        if n == 0:
            continue
        ids = table[row_seq[i], :-(-n // page)].long()
        for h in range(hq):
            hk = h // (hq // hkv)
            k = pages(k_cache, ids, hk).reshape(-1, d)[:n].to(F64) * sk
            v = pages(v_cache, ids, hk).reshape(-1, d)[:n].to(F64) * sv
            s = (k @ q[i, h].to(F64)) * scale
            lse[i, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[i, h])
            o[i, h], slack[i, h] = p @ v, p @ v.abs()
            spread[i, h] = (k.abs() @ q[i, h].to(F64).abs()).max() * scale
    return o, lse, slack, spread


def score_bound(spread, d):
    """|error of a score|: d products summed in fp32 in any order, the scale and the log2 e of the exponent."""
    return (d + 4) * 2.0 ** -24 * spread


def attention_bounds(o, slack, spread, lse, d, n, out_dtype, p_half):
    """Element-wise bounds of o and lse.  p is off by the score's error twice (its own and the maximum's or sum's), by
    2^-21 of the exponential and by its rounding to p_half; n fp32 additions of weights and of products, in parts that
    are joined; then one rounding of the output."""
    ds = score_bound(spread, d)
    add = (n + 16) * 2.0 ** -24
    rel = 2 * ds + 2.0 ** -20 + p_half + 2 * add
    bo = slack * rel[..., None] * 1.01 + HALF[out_dtype] * o.abs() + 1e-30
    bl = ds + 2.0 ** -20 + add + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22
    return bo, bl


def logprobs(x, targets, top):
    """Row by row in 64 bits: logp, entropy, lse, top values and ids (ties by the lower index)."""
    x = x.to(F64)
    lse = torch.logsumexp(x, 1)
    lp = x - lse[:, None]
    p = torch.exp(lp)
    ent = -(torch.where(p > 0, lp, torch.zeros(())) * p).sum(1)
    t = targets.long()
    at = lp.gather(1, t.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    logp = torch.where((t >= 0) & (t < x.shape[1]), at, torch.zeros((), dtype=F64))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return {"logp": logp, "entropy": ent, "lse": lse, "top_logp": lp.gather(1, order), "top_ids": order.int()}


def logprobs_bounds(x, ref):
    """Bounds of lse (and every log probability), and of the entropy.  A thread adds at most V/256 + 64 terms one by
    one (128 threads or more a row, two sums each), the exponentials are off by 2^-21, x - lse rounds twice at the size of its parts;
    the entropy's terms carry |x - max| as well."""
    V = x.shape[1]
    rel = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
    finite = torch.where(torch.isfinite(x), x, torch.zeros((), dtype=x.dtype)).to(F64)
    size = finite.abs().amax(1) + ref["lse"].abs().nan_to_num(0, 0, 0)
    b = rel + size * 2.0 ** -22
    spread = ref["entropy"].abs() + (x.to(F64).amax(1) - ref["lse"]).abs().nan_to_num(0, 0, 0) + math.log(V) + 1
    return b, 4 * rel * spread + size * 2.0 ** -22


def logprobs_grad(x, targets, lse, ent, dlogp, dent):
    """(gradient in 64 bits, p (|dlogp| + |dent| (|logp| + |H|)): what relative errors of p act on)."""
    x, lse, ent, dlogp, dent = (t.to(F64) for t in (x, lse, ent, dlogp, dent))
    lp = x - lse[:, None]
    p = torch.where(torch.isfinite(lse)[:, None], torch.exp(lp), torch.zeros((), dtype=F64))
    lp = torch.where(p > 0, lp, torch.zeros((), dtype=F64))
    t = targets.long()
    scored = (t >= 0) & (t < x.shape[1]) & torch.isfinite(lse)
    dl = torch.where(scored, dlogp, torch.zeros((), dtype=F64))
    g = -p * (dl[:, None] + dent[:, None] * (lp + ent.nan_to_num(0)[:, None]))
    rows = torch.nonzero(scored)[:, 0]
    g[rows, t[rows]] += dl[rows]
    return g, p * (dl.abs()[:, None] + dent.abs()[:, None] * (lp.abs() + ent.abs().nan_to_num(0)[:, None])), lp
