"""The decode and scoring operators as measured cases: paged-cache append with
the position rotation, attention of one new token over the paged cache, log
probabilities of given tokens (with entropy and top alternatives) and their
gradient.

``listed()`` gives the cases, ``draw()`` more of the same ranges, ``prepare()``
a case's inputs on the GPU, ``run()`` one pass: the plain form in elementary
torch operations, or (``own = True``) the library's calls.  ``exact()`` is the
definition in 64 bits, and ``work()`` what a pass cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


def listed():
    heads8 = {"q_heads": 32, "kv_heads": 8, "head_dim": 128}   # LLaMA-3-8B
    heads70 = {"q_heads": 64, "kv_heads": 8, "head_dim": 128}  # LLaMA-3-70B
    return [
        # one user's next token: the smallest append, launch latency
        {"name": "append_one_token", "op": "append", "tokens": 1, "seqs": 1, "padded": 0, "start": 1900, **heads8,
         "page": 16, "dtype": "bf16", "cache": "bf16", "base": 500000.0},
        # one token for each of a full serving batch, FP8 cache
        {"name": "append_batch_e4m3", "op": "append", "tokens": 250, "seqs": 250, "padded": 6, "start": 9000,
         **heads70, "page": 64, "dtype": "bf16", "cache": "e4m3", "base": 500000.0},
        # a prompt batch: five prompts, some continuing far into their sequences, a padded tail of rows
        {"name": "append_prompts", "op": "append", "tokens": 16284, "seqs": 5, "padded": 100, "start": 100003,
         **heads8, "page": 16, "dtype": "bf16", "cache": "bf16", "base": 500000.0},
        # one user, a short context: latency
        {"name": "attn_one_short", "op": "attn", "seqs": 1, "shortest": 1900, "longest": 1900, **heads8, "page": 16,
         "dtype": "bf16", "cache": "bf16"},
        # one user, a long context: one sequence over the whole GPU
        {"name": "attn_one_long", "op": "attn", "seqs": 1, "shortest": 131071, "longest": 131071, **heads8,
         "page": 16, "dtype": "bf16", "cache": "bf16"},
        # an ordinary serving batch, ragged lengths
        {"name": "attn_batch_ragged", "op": "attn", "seqs": 64, "shortest": 17, "longest": 8192, **heads8,
         "page": 16, "dtype": "bf16", "cache": "bf16"},
        # a large batch on an FP8 cache
        {"name": "attn_batch_e4m3", "op": "attn", "seqs": 128, "shortest": 4000, "longest": 16000, **heads70,
         "page": 64, "dtype": "bf16", "cache": "e4m3"},
        # a small fp32 model without shared heads, from one token up, pages that end inside any tile
        {"name": "attn_f32_own_heads", "op": "attn", "seqs": 16, "shortest": 1, "longest": 2000, "q_heads": 12,
         "kv_heads": 12, "head_dim": 64, "page": 24, "dtype": "f32", "cache": "f32"},
        # the sampled token's log probability and the 20 best alternatives of one decode step
        {"name": "logprobs_one_token", "op": "logprobs", "rows": 1, "vocab": 128256, "stride": 128256, "top": 20,
         "dtype": "bf16"},
        # scoring a batch of given tokens
        {"name": "logprobs_scoring", "op": "logprobs", "rows": 2048, "vocab": 128256, "stride": 128256, "top": 8,
         "dtype": "bf16"},
        # the training step on those log probabilities, with an entropy term
        {"name": "logprobs_grad_train", "op": "logprobs_grad", "rows": 4096, "vocab": 128256, "stride": 128256,
         "dtype": "bf16"},
        # fp32 logits, odd vocabulary in padded rows
        {"name": "logprobs_grad_f32_odd", "op": "logprobs_grad", "rows": 333, "vocab": 50257, "stride": 50260,
         "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "logprobs", "logprobs_grad"])
    if op in ("append", "attn"):
        kv = rng.choice([1, 2, 4, 5, 8, 12])
        c = {"op": op, "q_heads": kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), "kv_heads": kv,
             "head_dim": rng.choice([64, 80, 96, 128, 128, 128, 192, 256]), "page": rng.choice([1, 8, 16, 24, 64, 128])}
        c["dtype"], c["cache"] = rng.choice([("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
        row = kv * c["head_dim"] * 2 * SIZE[c["cache"]]
        if op == "append":
            width = (c["q_heads"] + 2 * kv) * c["head_dim"] * SIZE[c["dtype"]]
            c["tokens"] = _log(rng, 1, max(2, min(16384, 200_000_000 // width)))
            c["seqs"] = _log(rng, 1, c["tokens"])
            c["padded"] = rng.choice([0, 0, 3])
            c["start"] = _log(rng, 1, 200000)
            c["base"] = rng.choice([10000.0, 500000.0])
        else:
            c["seqs"] = _log(rng, 1, 128)
            most = max(2, min(131072, 1_000_000_000 // (row * c["seqs"])))
            c["longest"] = _log(rng, 1, most)
            c["shortest"] = _log(rng, 1, c["longest"])
        return c
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "vocab": _log(rng, 100, 200000)}
    step = 16 // SIZE[c["dtype"]]
    c["stride"] = -(-c["vocab"] // step) * step
    c["rows"] = _log(rng, 1, max(2, min(4096, 400_000_000 // (c["stride"] * SIZE[c["dtype"]]))))
    if op == "logprobs":
        c["top"] = min(rng.choice([0, 1, 5, 20, 50]), c["vocab"])
    return c


def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi: the same ones for every seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _append_counts(case):
    """New tokens of each sequence: 1, or unequal parts of the whole."""
    n, s = case["tokens"], case["seqs"]
    cuts = [n * i * (i + 1) // (s * (s + 1)) for i in range(s + 1)]
    got = [max(1, b - a) for a, b in zip(cuts, cuts[1:])]
    over = sum(got) - n
    for i in reversed(range(s)):
        cut = min(over, got[i] - 1)
        got[i] -= cut
        over -= cut
    return got


def _pages(needed_from, needed_to, pool, gen):
    """A page table over a shuffled pool of pages: sequence b holds pages needed_from[b] .. needed_to[b] - 1 (others -1)."""
    rows, width = len(needed_to), max(max(needed_to), 1)
    lo, hi = torch.tensor(needed_from, device=DEV)[:, None], torch.tensor(needed_to, device=DEV)[:, None]
    count = hi - lo
    perm = torch.randperm(pool, generator=gen, device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    index = torch.cumsum(count, 0) - count + at - lo
    table = torch.where((at >= lo) & (at < hi), perm[index.clamp(0, pool - 1)], torch.full_like(index, -1))
    return table.to(torch.int32).reshape(rows, width)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = random.Random(seed)
    op = case["op"]
    st = {"case": case}

    def normal(*shape, dtype, scale=1.0):
        x = torch.empty(*shape, dtype=torch.float32 if dtype != torch.bfloat16 else dtype, device=DEV)
        x.normal_(0.0, scale, generator=gen)
        return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x

    if op in ("append", "attn"):
        hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
        dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
        e4m3 = case["cache"] == "e4m3"
        if e4m3:  # the cache's fixed scales: keys and values of unit size near code 50
            st["scale_k"] = torch.tensor([0.02], device=DEV)
            st["scale_v"] = torch.tensor([0.017], device=DEV)
        spread = 50.0 if e4m3 else 1.0
        if op == "append":
            counts = _append_counts(case)
            host.shuffle(counts)
            starts = [host.randrange(case["start"]) for _ in counts]
            starts[0] = case["start"]
            seq, pos = [], []
            for b, (s, n) in enumerate(zip(starts, counts)):
                seq += [b] * n
                pos += range(s, s + n)
            rows = case["tokens"] + case["padded"]
            seq += [0] * case["padded"]
            pos += [-1] * case["padded"]  # rows behind the last sequence
            st["row_seq"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
            st["positions"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
            pool = case["tokens"] // page + 2 * case["seqs"] + 3  # a few more than the new tokens can touch
            st["table"] = _pages([s // page for s in starts],
                                 [(s + n - 1) // page + 1 for s, n in zip(starts, counts)], pool, gen)
            st["Z"] = normal(rows, (hq + 2 * hkv) * d, dtype=dt)
            st["Q"] = torch.zeros(rows, hq, d, dtype=dt, device=DEV)
        else:
            lens = _spread(case["shortest"], case["longest"], case["seqs"])
            host.shuffle(lens)
            st["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
            pool = sum(-(-n // page) for n in lens) + 3
            st["table"] = _pages([0] * len(lens), [-(-n // page) for n in lens], pool, gen)
            st["Q"] = normal(len(lens), hq, d, dtype=dt)
            st["O"] = torch.empty(len(lens), hq * d, dtype=dt, device=DEV)
            st["lse"] = torch.empty(len(lens), hq, dtype=torch.float32, device=DEV)
            if own:  # the split's workspace, which a serving loop keeps
                import gemm_epilogue_fusion_gb300 as g
                st["workspace"] = g.paged_attention_workspace(hq, hkv, d, DEV)
        st["k"] = normal(pool, hkv, page, d, dtype=ct, scale=spread)
        st["v"] = normal(pool, hkv, page, d, dtype=ct, scale=spread)
        return st
    rows, vocab, stride, dt = case["rows"], case["vocab"], case["stride"], DTYPES[case["dtype"]]
    st["logits"] = normal(rows, stride, dtype=dt, scale=2.5)[:, :vocab]
    st["targets"] = torch.randint(0, vocab, (rows,), generator=gen, device=DEV, dtype=torch.int32)
    if rows > 2:
        st["targets"][rows // 2] = -1  # a token that is not scored
    if op == "logprobs":
        st["logp"], st["entropy"], st["lse"] = (torch.empty(rows, device=DEV) for _ in range(3))
        st["top_logp"] = torch.empty(rows, case["top"], device=DEV)
        st["top_ids"] = torch.empty(rows, case["top"], dtype=torch.int32, device=DEV)
    else:
        # what the forward pass left behind: its row statistics in 32 bits
        lse, ent = [], []
        for x in st["logits"].split(256):
            x = x.double()
            m = torch.logsumexp(x, 1)
            lse.append(m.float())
            ent.append((m - (torch.exp(x - m[:, None]) * x).sum(1)).float())
        st["lse"], st["entropy"] = torch.cat(lse), torch.cat(ent)
        st["dlogp"] = torch.empty(rows, device=DEV).normal_(0.0, 1.0, generator=gen)
        st["dentropy"] = torch.empty(rows, device=DEV).normal_(0.0, 0.05, generator=gen)
        st["dlogits"] = torch.empty(rows, stride, dtype=dt, device=DEV)[:, :vocab]
    return st


# ------------------------------------------------------------ plain forms ----

def _plain_append(st):
    c = st["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    x = st["Z"].float().reshape(-1, hq + 2 * hkv, d)
    freq = c["base"] ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
    phi = st["positions"].double()[:, None] * freq  # 64 bits: far positions
    cos, sin = torch.cos(phi).float()[:, None, :], torch.sin(phi).float()[:, None, :]
    a, b = x[:, : hq + hkv, 0::2], x[:, : hq + hkv, 1::2]
    turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).reshape(-1, hq + hkv, d)
    keep = torch.nonzero(st["positions"] >= 0)[:, 0]
    st["Q"][keep] = turned[keep, :hq].to(st["Q"].dtype)
    pos = st["positions"][keep].long()
    at = st["table"][st["row_seq"][keep].long(), pos // page].long()
    for cache, new, scale in ((st["k"], turned[:, hq:], "scale_k"), (st["v"], x[:, hq + hkv:], "scale_v")):
        new = new[keep]
        if c["cache"] == "e4m3":
            new = (new / st[scale]).clamp(-448, 448).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[at, :, pos % page] = new.to(cache.dtype)
    return {"q": st["Q"], "k": st["k"], "v": st["v"]}


def _plain_attention(st):
    c = st["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    q = st["Q"].float().reshape(-1, hkv, hq // hkv, d)
    table = st["table"].long().clamp(min=0)
    keys = table.shape[1] * page

    def gathered(cache, scale):  # [seqs, heads, keys, d] in 32 bits
        raw = cache.view(torch.uint8)[table].view(cache.dtype) if c["cache"] == "e4m3" else cache[table]
        x = raw.transpose(1, 2).reshape(-1, hkv, keys, d).float()
        return x * st[scale] if c["cache"] == "e4m3" else x

    s = torch.matmul(q, gathered(st["k"], "scale_k").transpose(2, 3)) * (1.0 / math.sqrt(d))
    there = torch.arange(keys, device=DEV)[None, :] < st["lengths"].long()[:, None]
    s = torch.where(there[:, None, None, :], s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where(there[:, None, :, None], gathered(st["v"], "scale_v"), torch.zeros((), device=DEV))
    o = torch.matmul(p / total, v)
    return {"o": o.reshape(-1, hq * d).to(st["Q"].dtype), "lse": (m + torch.log(total)).reshape(-1, hq)}


def _plain_logprobs(st):
    c = st["case"]
    x = st["logits"].float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    entropy = torch.log(total) - (e * (x - m)).sum(1, keepdim=True) / total
    lse = m + torch.log(total)
    t = st["targets"].long()[:, None]
    logp = torch.where(t >= 0, x.gather(1, t.clamp(min=0)) - lse, torch.zeros_like(lse))
    out = {"logp": logp[:, 0], "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if c["top"]:
        # ties go to the lowest index: one whole number orders by value, then by index
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -2147483648 - bits) * 4294967296 - torch.arange(x.shape[1], device=DEV)
        ids = (-key.topk(c["top"], 1).values) % 4294967296
        out["top_logp"], out["top_ids"] = x.gather(1, ids) - lse, ids.int()
    return out


def _plain_logprobs_grad(st):
    x = st["logits"].float()
    logp = x - st["lse"][:, None]
    p = torch.exp(logp)
    t = st["targets"].long()[:, None]
    chosen = torch.arange(x.shape[1], device=DEV)[None, :] == t
    scored = torch.where(t >= 0, st["dlogp"][:, None], torch.zeros((), device=DEV))
    g = scored * (chosen.float() - p) - st["dentropy"][:, None] * p * (logp + st["entropy"][:, None])
    return {"dlogits": g.to(st["logits"].dtype)}


def run(state):
    c = state["case"]
    if own:
        import gemm_epilogue_fusion_gb300 as g
        if c["op"] == "append":
            q = g.coda_paged_append(state["Z"], state["positions"], state["table"], state["k"], state["v"],
                                    c["q_heads"], row_seq=state["row_seq"], base=c["base"], Q=state["Q"],
                                    scale_k=state.get("scale_k"), scale_v=state.get("scale_v"))
            return {"q": q, "k": state["k"], "v": state["v"]}
        if c["op"] == "attn":
            o = g.coda_paged_attention(state["Q"], state["k"], state["v"], state["table"], state["lengths"],
                                       state["workspace"], O=state["O"], lse=state["lse"],
                                       scale_k=state.get("scale_k"), scale_v=state.get("scale_v"))
            return {"o": o, "lse": state["lse"]}
        if c["op"] == "logprobs":
            got = g.coda_logprobs(state["logits"], state["targets"], c["top"], logp=state["logp"],
                                  entropy=state["entropy"], lse=state["lse"],
                                  top_logp=state["top_logp"] if c["top"] else None,
                                  top_ids=state["top_ids"] if c["top"] else None)
            out = {"logp": got["logp"], "entropy": got["entropy"], "lse": got["lse"]}
            if c["top"]:
                out["top_logp"], out["top_ids"] = got["top_logp"], got["top_ids"]
            return out
        return {"dlogits": g.coda_logprobs_backward(state["logits"], state["targets"], state["lse"],
                                                    state["entropy"], state["dlogp"], state["dentropy"],
                                                    dlogits=state["dlogits"])}
    return {"append": _plain_append, "attn": _plain_attention, "logprobs": _plain_logprobs,
            "logprobs_grad": _plain_logprobs_grad}[c["op"]](state)


def work(case):
    op = case["op"]
    if op == "append":
        hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        e, ec, n = SIZE[case["dtype"]], SIZE[case["cache"]], case["tokens"]
        return {"bytes": n * d * ((hq + 2 * hkv) * e + hq * e + 2 * hkv * ec) + 12 * n, "flops": 3 * n * (hq + hkv) * d}
    if op == "attn":
        hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        keys = sum(_spread(case["shortest"], case["longest"], case["seqs"]))
        row = hq * d * SIZE[case["dtype"]] * 2 + 4 * hq
        return {"bytes": 2 * keys * hkv * d * SIZE[case["cache"]] + case["seqs"] * row + 4 * keys // case["page"],
                "flops": 4 * keys * hq * d}
    n = case["rows"] * case["vocab"]
    if op == "logprobs":
        return {"bytes": n * SIZE[case["dtype"]] + case["rows"] * (16 + 8 * case["top"]), "flops": 5 * n}
    return {"bytes": 2 * n * SIZE[case["dtype"]] + 20 * case["rows"], "flops": 7 * n}


# ------------------------------------------------------ the definition, 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "append":
        hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
        z = st["Z"].to(f64).view(-1, hq + 2 * hkv, d // 2, 2)
        pos = st["positions"].cpu().numpy()
        freq = np.array([case["base"] ** (-2.0 * j / d) for j in range(d // 2)])
        turn = torch.from_numpy(np.exp(1j * np.maximum(pos, 0)[:, None] * freq[None, :])).to(DEV)
        spun = torch.view_as_real(torch.view_as_complex(z[:, : hq + hkv].contiguous()) * turn[:, None, :])
        n = case["tokens"]
        q = st["Q"].to(f64)
        q[:n] = spun[:n, :hq].reshape(n, hq, d)
        table, seq = st["table"].cpu().numpy(), st["row_seq"].cpu().numpy()
        flat = torch.from_numpy(table[seq[:n], pos[:n] // page].astype(np.int64) * page + pos[:n] % page).to(DEV)
        out = {"q": q}
        for name, new, s in (("k", spun[:n, hq:], "scale_k"), ("v", z[:n, hq + hkv:], "scale_v")):
            new = new.reshape(n, hkv, d)
            rows = st[name].to(f64).transpose(1, 2).reshape(-1, hkv, d).clone()
            if case["cache"] == "e4m3":  # a code is a decision of the rounding: taken on the 64-bit quotient in 32 bits
                new = (new / st[s].to(f64)).clamp(-448, 448).float().to(torch.float8_e4m3fn).to(f64)
            rows[flat] = new
            out[name] = rows.view(-1, page, hkv, d).transpose(1, 2).contiguous()
        return out
    if op == "attn":
        hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
        group = hq // hkv
        o = torch.empty(case["seqs"], hq * d, dtype=f64, device=DEV)
        lse = torch.empty(case["seqs"], hq, dtype=f64, device=DEV)
        sk = st["scale_k"].item() if "scale_k" in st else 1.0
        sv = st["scale_v"].item() if "scale_v" in st else 1.0
        for b, n in enumerate(st["lengths"].tolist()):
            ids = st["table"][b, : -(-n // page)].long()
            for h in range(hkv):
                raw = (st[x][:, h].view(torch.uint8)[ids].view(st[x].dtype) if case["cache"] == "e4m3"
                       else st[x][ids, h] for x in ("k", "v"))
                k, v = (x.reshape(-1, d)[:n].to(f64) for x in raw)
                g = slice(h * group, (h + 1) * group)
                s = (st["Q"][b, g].to(f64) @ k.T) * (sk / math.sqrt(d))
                lse[b, g] = torch.logsumexp(s, 1)
                w = torch.softmax(s, 1)
                o[b, h * group * d:(h + 1) * group * d] = (w @ v * sv).reshape(-1)
        return {"o": o, "lse": lse}
    rows = case["rows"]
    if op == "logprobs":
        parts = []
        for x, t in zip(st["logits"].split(128), st["targets"].split(128)):
            lp = torch.log_softmax(x.to(f64), 1)
            p = lp.exp()
            lse = torch.logsumexp(x.to(f64), 1)
            at = lp[torch.arange(len(t), device=DEV), t.long().clamp(min=0)]
            part = [torch.where(t >= 0, at, torch.zeros_like(at)), -(p * lp).sum(1), lse]
            if case["top"]:
                part.append(torch.sort(lp, 1, descending=True).values[:, : case["top"]])
            parts.append(part)
        cols = [torch.cat(c) for c in zip(*parts)]
        out = dict(zip(("logp", "entropy", "lse", "top_logp"), cols))
        if case["top"]:
            out["top_ids"] = None
        return out
    got = torch.empty(rows, case["vocab"], dtype=f64, device=DEV)
    for i in range(0, rows, 128):
        s = slice(i, min(rows, i + 128))
        x = st["logits"][s].to(f64)
        lp = x - st["lse"][s].to(f64)[:, None]
        p = torch.exp(lp)
        t = st["targets"][s].long()
        live = (t >= 0).to(f64) * st["dlogp"][s].to(f64)
        de = st["dentropy"][s].to(f64)
        g = p * (-live[:, None] - de[:, None] * (lp + st["entropy"][s].to(f64)[:, None]))
        g[torch.arange(len(t), device=DEV), t.clamp(min=0)] += live
        got[s] = g
    return {"dlogits": got}
