"""The decode and scoring operators as they are used: a two-layer model
answering token by token on a paged cache (chain.decode_layer, the LM head's
log probabilities), and the head's gradient down to the residual stream."""
import math

import pytest
import torch

import decode_util as U
import oracle

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TOL = 2e-2  # of the largest value, per block of bf16 products (as in the block tests)
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


class Model:
    """hidden N, two layers, query and key/value heads of d, a vocabulary padded to whole 16-byte rows."""
    N, I, HQ, HKV, D, L, V, VPAD, PAGE = 256, 192, 4, 2, 64, 2, 301, 304, 16
    BASE = 10000.0

    def __init__(self, seed, dtype):
        g = U.gen(seed)
        self.g, self.dtype = g, dtype
        qkv = (self.HQ + 2 * self.HKV) * self.D
        shapes = {"Wq": (qkv, self.N), "Wo": (self.N, self.HQ * self.D), "Wg": (self.I, self.N), "Wu": (self.I, self.N),
                  "Wd": (self.N, self.I)}
        self.W = [{k: (torch.randn(*s, generator=g) / math.sqrt(s[1])).to(dtype) for k, s in shapes.items()}
                  for _ in range(self.L)]
        self.gq = [1 + 0.1 * torch.randn(self.N, generator=g) for _ in range(self.L)]
        self.gm = [1 + 0.1 * torch.randn(self.N, generator=g) for _ in range(self.L)]
        self.gv = 1 + 0.1 * torch.randn(self.N, generator=g)
        self.Wv = (torch.randn(self.VPAD, self.N, generator=g) * (3.0 / math.sqrt(self.N))).to(dtype)

    def fold(self):
        import gemm_epilogue_fusion_gb300 as gg
        f = lambda w, gamma: gg.coda_fold_gamma(w.cuda(), gamma.cuda())  # noqa: E731
        self.Wq = [f(w["Wq"], a) for w, a in zip(self.W, self.gq)]
        self.Wg = [f(w["Wg"], a) for w, a in zip(self.W, self.gm)]
        self.Wu = [f(w["Wu"], a) for w, a in zip(self.W, self.gm)]
        self.Wo = [w["Wo"].cuda() for w in self.W]
        self.Wd = [w["Wd"].cuda() for w in self.W]
        self.Wvf = f(self.Wv, self.gv)

    def exact_logits(self, embeddings):
        """Logits of every position of one sequence [T, N] in 64 bits, with full causal attention."""
        h = embeddings.to(U.F64)
        T = h.shape[0]
        norm = lambda x, gamma: x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * gamma.to(U.F64)  # noqa: E731
        causal = torch.ones(T, T, dtype=torch.bool).tril()
        for w, gq, gm in zip(self.W, self.gq, self.gm):
            w = {k: v.to(U.F64) for k, v in w.items()}
            z = (norm(h, gq) @ w["Wq"].T).view(T, -1, self.D)
            qk = torch.stack([U.rotate(z[t, :self.HQ + self.HKV], t, self.BASE) for t in range(T)])
            out = []
            for i in range(self.HQ):
                k, v = qk[:, self.HQ + i * self.HKV // self.HQ], z[:, self.HQ + self.HKV + i * self.HKV // self.HQ]
                s = (qk[:, i] @ k.T / math.sqrt(self.D)).masked_fill(~causal, -math.inf)
                out.append(torch.softmax(s, 1) @ v)
            h = h + torch.cat(out, 1) @ w["Wo"].T
            y = norm(h, gm)
            gate = y @ w["Wg"].T
            h = h + (gate * torch.sigmoid(gate) * (y @ w["Wu"].T)) @ w["Wd"].T
        return norm(h, self.gv) @ self.Wv.to(U.F64).T


@pytest.mark.parametrize("cache", [BF, E4], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rope_in", ["append", "gemm"])
def test_decode_token_by_token(cache, rope_in):
    import gemm_epilogue_fusion_gb300 as gg
    from gemm_epilogue_fusion_gb300 import chain
    m = Model(1, BF)
    m.fold()
    T, B = 37, 3
    emb = torch.randn(B, T, m.N, generator=m.g).to(BF)
    tokens = torch.randint(0, m.V, (B, T), generator=m.g, dtype=torch.int32)
    want = [m.exact_logits(e)[:, :m.V] for e in emb]
    lens = [T, T - 5, 20]  # the other sequences end earlier: padded rows from then on
    pages = sum(-(-n // m.PAGE) for n in lens) + 1
    table = U.page_table(lens, m.PAGE, pages, m.g).cuda()
    caches = [[torch.zeros(pages, m.HKV, m.PAGE, m.D, dtype=cache).cuda() for _ in range(2)] for _ in range(m.L)]
    ws = gg.paged_attention_workspace(m.HQ, m.HKV, m.D, "cuda")
    kw = {}
    if cache == E4:
        kw = {"scale_k": torch.tensor([0.02]).cuda(), "scale_v": torch.tensor([0.02]).cuda()}
    qk_cols = (m.HQ + m.HKV) * m.D
    base = m.BASE if rope_in == "append" else 0.0
    worst = 0.0
    for t in range(T):
        live = [t < n for n in lens]
        pos = torch.tensor([t if a else -1 for a in live], dtype=torch.int32).cuda()
        ln = torch.tensor([t + 1 if a else 0 for a in live], dtype=torch.int32).cuda()
        R = emb[:, t].contiguous().cuda()
        r = torch.rsqrt(R.float().square().mean(1) + EPS)
        at = torch.full((B,), t, dtype=torch.int32).cuda()
        if base:
            Z = gg.coda_gemm_rowscale(R, m.Wq[0], r)
        else:
            Z = gg.coda_gemm_rowscale_rope(R, m.Wq[0], m.D, qk_cols, m.BASE, positions=at, r=r)
        for layer in range(m.L):
            nxt = m.Wq[layer + 1] if layer + 1 < m.L else m.Wvf
            # the padded rows' values are whatever append left out: keep the block's inputs finite
            out = chain.decode_layer(Z, R, pos, ln, table, caches[layer][0], caches[layer][1], m.HQ, ws, m.Wo[layer],
                                     m.Wg[layer], m.Wu[layer], m.Wd[layer], nxt, EPS, base=base, **kw)
            R, Z = out["h2"], out["Z"]
            if not base and layer + 1 < m.L:
                Z = gg.coda_gemm_rowscale_rope(R, nxt, m.D, qk_cols, m.BASE, positions=at, r=out["r2"])
        got = chain.head_logprobs(R, out["P2"], m.Wvf, EPS, tokens[:, t].contiguous().cuda(), top=5, vocab=m.V)
        assert torch.equal(got["logits"], out["Z"]) if base else True
        ref = U.logprobs(got["logits"].cpu()[:, :m.V], tokens[:, t], 5)
        assert torch.equal(got["top_ids"].cpu(), ref["top_ids"])
        for b in range(B):
            if live[b]:
                x = want[b][t]
                worst = max(worst, float((got["logits"][b, :m.V].cpu().to(U.F64) - x).abs().max() / x.abs().max()))
                lp = torch.log_softmax(x, 0)[int(tokens[b, t])]
                assert abs(float(got["logp"][b]) - lp) <= 4 * TOL * float(x.abs().max())
    assert gg.coda_get_device_status() == gg.CODA_OK
    # two layers of blocks; e4m3 keys and values add their own half step (2^-4) on the attention's part of the stream
    assert worst <= (2 * TOL if cache == BF else 2 * TOL + 2.0 ** -4), worst


def test_fp32_decode_of_the_layer():
    """The same layer call in fp32 (the block's products in tf32), several new tokens of one sequence in one call."""
    import gemm_epilogue_fusion_gb300 as gg
    from gemm_epilogue_fusion_gb300 import chain
    m = Model(2, F32)
    m.fold()
    T = 24
    emb = torch.randn(T, m.N, generator=m.g)
    want = m.exact_logits(emb)
    table = U.page_table([T], m.PAGE, 4, m.g).cuda()
    caches = [[torch.zeros(4, m.HKV, m.PAGE, m.D).cuda() for _ in range(2)] for _ in range(m.L)]
    ws = gg.paged_attention_workspace(m.HQ, m.HKV, m.D, "cuda")
    pos = torch.arange(T, dtype=torch.int32).cuda()
    seq = torch.zeros(T, dtype=torch.int32).cuda()
    R = emb.cuda()
    Z = gg.coda_gemm_rowscale(R, m.Wq[0], torch.rsqrt(R.square().mean(1) + EPS))
    for layer in range(m.L):
        out = chain.decode_layer(Z, R, pos, pos + 1, table, *caches[layer], m.HQ, ws, m.Wo[layer], m.Wg[layer],
                                 m.Wu[layer], m.Wd[layer], m.Wq[1] if layer == 0 else m.Wvf, EPS, row_seq=seq,
                                 base=m.BASE)
        R, Z = out["h2"], out["Z"]
    assert oracle.rel_err(Z.cpu()[:, :m.V], want[:, :m.V].numpy()) <= 2 * TOL


@pytest.mark.parametrize("M,V,pad", [(130, 304, 0), (37, 301, 3), (1, 64, 0)])
def test_head_gradient(M, V, pad):
    """head_logprobs_backward against 64-bit autograd of the definition."""
    import gemm_epilogue_fusion_gb300 as gg
    from gemm_epilogue_fusion_gb300 import chain
    g = U.gen(M)
    N = 128
    h = torch.randn(M, N, generator=g).to(BF)
    W = (torch.randn(V + pad, N, generator=g) * (2.0 / math.sqrt(N))).to(BF)
    gamma = 1 + 0.1 * torch.randn(N, generator=g)
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    if M > 2:
        t[1] = -1
    a, b = torch.randn(M, generator=g), 0.3 * torch.randn(M, generator=g)
    P = h.float().square().sum(1, keepdim=True).cuda()  # one 128-column group
    Wf = gg.coda_fold_gamma(W.cuda(), gamma.cuda())
    fwd = chain.head_logprobs(h.cuda(), P, Wf, EPS, t.cuda(), vocab=V if pad else None)
    grad = chain.head_logprobs_backward(h.cuda(), W.cuda(), gamma.cuda(), fwd, t.cuda(), a.cuda(), b.cuda(),
                                        vocab=V if pad else None)
    hx, wx, gx = (x.to(U.F64).requires_grad_() for x in (h, W, gamma))
    y = hx * torch.rsqrt((hx * hx).mean(1, keepdim=True) + EPS) * gx
    lp = torch.log_softmax((y @ wx.T)[:, :V], 1)
    scored = (t >= 0).to(U.F64)
    logp = lp.gather(1, t.long().clamp(min=0)[:, None])[:, 0] * scored
    ent = -(lp.exp() * lp).sum(1)
    assert oracle.rel_err(fwd["logp"].cpu(), logp.detach().numpy()) <= TOL
    ((logp * a.to(U.F64)).sum() + (ent * b.to(U.F64)).sum()).backward()
    for got, ref in ((grad["dh"], hx.grad), (grad["dWvt"], wx.grad), (grad["dgamma"], gx.grad)):
        assert oracle.rel_err(got.cpu(), ref.numpy()) <= 2 * TOL
    if pad:
        assert (grad["dWvt"][V:] == 0).all()
    assert gg.coda_get_device_status() == gg.CODA_OK
