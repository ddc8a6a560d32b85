"""The paged cache on the GPU: append with the position rotation, and attention
of one new token, against plain 64-bit forms with bounds from the formats."""
import math

import pytest
import torch

import decode_util as U

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [(BF, BF), (BF, E4), (F32, F32)]
IDS = ["bf16", "e4m3", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


def randn(*shape, dtype, g, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).clamp(-448 if dtype == E4 else -1e30, 448 if dtype == E4 else 1e30).to(dtype)


# ------------------------------------------------------------------ append ----

@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("hq,hkv,d,page,base", [(32, 8, 128, 16, 500000.0), (3, 1, 64, 5, 10000.0),
                                                (2, 2, 16, 1, 10000.0), (7, 7, 80, 24, 500000.0),
                                                (10, 2, 256, 64, 1.5), (32, 8, 128, 16, 0.0), (1, 1, 48, 3, 0.0)])
def test_append_against_64_bits(types, hq, hkv, d, page, base):
    import gemm_epilogue_fusion_gb300 as gg
    dt, ct = types
    g = U.gen(hq * 1000 + d)
    starts, counts = [0, 5, 100_000, 1_000_003], [3, 1, 9, 2]
    width = (1_000_005 + page - 1) // page + 1
    num_pages = 40
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = torch.full((4, width), -1, dtype=torch.int32)
    seq, pos = [], []
    for b, (s, n) in enumerate(zip(starts, counts)):
        for t in range(s, s + n):
            if table[b, t // page] < 0:
                table[b, t // page] = perm.pop()
            seq.append(b)
            pos.append(t)
    seq += [0, 3, -7]
    pos += [-1, -1, -2147483648]  # padded rows; the last one's sequence is never looked at
    order = torch.randperm(len(pos), generator=g)
    seq, pos = torch.tensor(seq, dtype=torch.int32)[order], torch.tensor(pos, dtype=torch.int32)[order]
    M = len(pos)
    Z = randn(M, (hq + 2 * hkv) * d, dtype=dt, g=g, scale=3.0)
    k0, v0 = randn(num_pages, hkv, page, d, dtype=ct, g=g), randn(num_pages, hkv, page, d, dtype=ct, g=g)
    q0 = randn(M, hq, d, dtype=dt, g=g)
    sk, sv = (0.013, 0.02) if ct == E4 else (None, None)
    kc, vc, Q = k0.cuda(), v0.cuda(), q0.cuda()
    kw = {} if sk is None else {"scale_k": torch.tensor([sk]).cuda(), "scale_v": torch.tensor([sv]).cuda()}
    out = gg.coda_paged_append(Z.cuda(), pos.cuda(), table.cuda(), kc, vc, hq, row_seq=seq.cuda(), base=base, Q=Q, **kw)
    assert out.data_ptr() == Q.data_ptr()
    assert gg.coda_get_device_status() == gg.CODA_OK
    kc, vc, Q = kc.cpu(), vc.cpu(), Q.cpu()
    want_k, want_v, want_q = k0.to(U.F64), v0.to(U.F64), q0.to(U.F64)
    bk, bv, bq = (torch.zeros_like(t) for t in (want_k, want_v, want_q))
    # the rotation: angle and sine off by 2^-20, three fp32 roundings; each acts on |a| + |b| of the pair
    turn = 2.0 ** -19 if base else 0.0

    def pair(x):
        a = x.abs().unflatten(-1, (d // 2, 2)).sum(-1, keepdim=True).expand(*x.shape[:-1], d // 2, 2).flatten(-2)
        return a * turn

    for i, row in enumerate(U.append(Z, pos, seq.tolist(), table, hq, hkv, d, page, base)):
        if row is None:
            continue
        q, k, v, pg, slot = row
        want_q[i], bq[i] = q, U.HALF[dt] * q.abs() + pair(q)
        for want, bound, x, s, p in ((want_k, bk, k, sk, pair(k)), (want_v, bv, v, sv, torch.zeros_like(v))):
            if ct == E4:
                x, p = (x / s).clamp(-448, 448), p / s + 2.0 ** -22 * (x / s).abs()
                # below 2^-6 an e4m3 step is 2^-9, whatever the value
                want[pg, :, slot], bound[pg, :, slot] = x, (U.HALF[E4] * x.abs()).clamp(min=2.0 ** -10) + p
            else:
                want[pg, :, slot], bound[pg, :, slot] = x, U.HALF[ct] * x.abs() + p
    for got, want, bound in ((Q, want_q, bq), (kc, want_k, bk), (vc, want_v, bv)):
        assert ((got.to(U.F64) - want).abs() <= bound * 1.0001 + 1e-30).all()  # where nothing is written: the same bits


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_append_without_row_seq_and_without_q(types):
    import gemm_epilogue_fusion_gb300 as gg
    dt, ct = types
    g = U.gen(5)
    M, hq, hkv, d, page = 6, 4, 2, 64, 16
    Z = randn(M, (hq + 2 * hkv) * d, dtype=dt, g=g).cuda()
    table = U.page_table([40] * 7, page, 30, g).cuda()
    pos = torch.tensor([0, 15, 16, 39, -1, 31], dtype=torch.int32).cuda()
    caches = [torch.zeros(30, hkv, page, d, dtype=ct).cuda() for _ in range(4)]
    kw = {} if ct != E4 else {"scale_k": torch.tensor([0.02]).cuda(), "scale_v": torch.tensor([0.02]).cuda()}
    q = gg.coda_paged_append(Z, pos, table, caches[0], caches[1], hq, base=10000.0, **kw)
    seq = torch.arange(M, dtype=torch.int32).cuda()
    assert gg.coda_paged_append(Z, pos, table, caches[2], caches[3], hq, row_seq=seq, base=10000.0, want_q=False,
                                **kw) is None
    assert q.shape == (M, hq, d)
    for a, b in ((0, 2), (1, 3)):
        assert torch.equal(caches[a].view(torch.uint8), caches[b].view(torch.uint8))
        assert torch.count_nonzero(caches[a].view(torch.uint8)) > 0
    # already rotated rows are only laid out: the same bits
    gg.coda_paged_append(Z, pos, table, caches[0], caches[1], hq, want_q=False, **kw)
    if ct == dt:
        z = Z.view(M, hq + 2 * hkv, d)
        for i, p in enumerate(pos.tolist()):
            if p >= 0:
                assert torch.equal(caches[0][table[i, p // page], :, p % page], z[i, hq:hq + hkv])
                assert torch.equal(caches[1][table[i, p // page], :, p % page], z[i, hq + hkv:])


def test_append_leaves_bad_rows_out_and_says_so():
    import gemm_epilogue_fusion_gb300 as gg
    g = U.gen(6)
    hq, hkv, d, page, pages = 2, 1, 64, 4, 6
    table = torch.tensor([[0, 1], [2, pages], [-1, 3]], dtype=torch.int32)
    rows = [(0, 0), (0, 8), (1, 4), (2, 0), (3, 0), (-1, 0), (2, 5), (0, 2147483647)]  # bad: all but the first and (2, 5)
    Z = randn(len(rows), (hq + 2 * hkv) * d, dtype=BF, g=g).cuda()
    kc, vc = torch.zeros(pages, hkv, page, d, dtype=BF).cuda(), torch.zeros(pages, hkv, page, d, dtype=BF).cuda()
    Q = torch.zeros(len(rows), hq, d, dtype=BF).cuda()
    seq = torch.tensor([r[0] for r in rows], dtype=torch.int32).cuda()
    pos = torch.tensor([r[1] for r in rows], dtype=torch.int32).cuda()
    gg.coda_paged_append(Z, pos, table.cuda(), kc, vc, hq, row_seq=seq, base=10000.0, Q=Q)
    with pytest.raises(gg.CodaError, match="out of range"):
        gg.coda_get_device_status()
    assert gg.coda_get_device_status() == gg.CODA_OK
    written = [i for i in range(len(rows)) if torch.count_nonzero(Q[i])]
    assert written == [0, 6]
    slots = (kc != 0).any(-1).any(1).nonzero().tolist()
    assert slots == [[0, 0], [3, 1]]


# --------------------------------------------------------------- attention ----

def make(hq, hkv, d, page, lens, types, seed, q_scale=1.0, poison=True):
    """Inputs of an attention call on the CPU; slots behind the lengths and pages of no sequence hold NaN."""
    dt, ct = types
    g = U.gen(seed)
    num_pages = sum(-(-max(n, 0) // page) for n in lens) + 2
    table = U.page_table([max(n, 0) for n in lens], page, num_pages, g)
    spread = 40.0 if ct == E4 else 1.0
    k, v = (randn(num_pages, hkv, page, d, dtype=ct, g=g, scale=spread) for _ in range(2))
    if poison:
        live = torch.zeros(num_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(max(n, 0)):
                live[table[b, t // page], t % page] = True
        dead = (~live)[:, None, :, None].expand_as(k)
        if ct == E4:
            for t in (k, v):
                t.view(torch.uint8)[dead] = 0x7F  # e4m3 NaN
        else:
            k[dead] = math.nan
            v[dead] = math.nan
    q = randn(len(lens), hq, d, dtype=dt, g=g, scale=q_scale)
    s = (0.021, 0.017) if ct == E4 else (1.0, 1.0)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32), s


def scales(ct, s):
    return {} if ct != E4 else {"scale_k": torch.tensor([s[0]]).cuda(), "scale_v": torch.tensor([s[1]]).cuda()}


def check(q, k, v, table, lens, s, got_o, got_lse, row_seq=None, scale=None):
    dt, ct = q.dtype, k.dtype
    M, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    seq = list(range(M)) if row_seq is None else row_seq
    o, lse, slack, spread = U.attention(q, k, v, table, lens, seq, scale, *s)
    # the weights are held in 16 bits for the second product: bf16, or f16 with an e4m3 cache
    p_half = {BF: U.HALF[BF], E4: U.HALF[torch.float16], F32: 0.0}[ct]
    n = max([int(x) for x in lens] + [0])
    bo, bl = U.attention_bounds(o, slack, spread, lse, d, n, dt, p_half)
    got_o = got_o.cpu().view(M, hq, d).to(U.F64)
    assert ((got_o - o).abs() <= bo).all(), ((got_o - o).abs() / bo).max()
    if got_lse is not None:
        got_lse = got_lse.cpu().to(U.F64)
        empty = torch.isinf(lse)
        assert torch.equal(got_lse[empty], lse[empty])
        assert ((got_lse - lse).abs()[~empty] <= bl[~empty]).all()


HEADS = [(32, 8, 128, 16), (64, 8, 128, 64), (4, 4, 64, 5), (16, 1, 80, 24), (14, 2, 256, 1), (40, 2, 96, 128),
         (1, 1, 16, 3), (9, 1, 48, 7), (6, 3, 192, 16), (34, 1, 64, 16), (16, 1, 256, 16), (5, 1, 128, 2), (8, 2, 256, 8),
         (14, 2, 192, 8), (32, 2, 160, 16), (3, 1, 176, 5), (16, 1, 192, 64)]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("hq,hkv,d,page", HEADS, ids=lambda v: str(v))
def test_attention_against_64_bits(types, hq, hkv, d, page):
    import gemm_epilogue_fusion_gb300 as gg
    lens = [1, 0, 65, 128, -3, 17, 63, 300, 2, 64]
    q, k, v, table, ln, s = make(hq, hkv, d, page, lens, types, hq + d, q_scale=2.0)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    lse = torch.empty(len(lens), hq).cuda()
    kw = scales(types[1], s)
    args = (q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws)
    o = gg.coda_paged_attention(*args, lse=lse, **kw)
    assert gg.coda_get_device_status() == gg.CODA_OK
    check(q, k, v, table, ln, s, o, lse)
    again = gg.coda_paged_attention(*args, **kw)  # the workspace is ready for the next call, and the bits are the same
    assert torch.equal(o, again)


@pytest.mark.parametrize("types,d", [((BF, BF), 8), ((F32, F32), 4), ((F32, F32), 12)], ids=["bf16-8", "f32-4", "f32-12"])
def test_attention_and_append_of_the_narrowest_heads(types, d):
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, page, lens = 3, 3, 4, [1, 0, 30, 65]
    q, k, v, table, ln, s = make(hq, hkv, d, page, lens, types, d)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    lse = torch.empty(4, hq).cuda()
    kc, vc = k.cuda(), v.cuda()
    o = gg.coda_paged_attention(q.cuda(), kc, vc, table.cuda(), ln.cuda(), ws, lse=lse)
    check(q, k, v, table, ln, s, o, lse)
    Z = randn(4, 3 * hq * d, dtype=types[0], g=U.gen(1))
    pos = torch.tensor([0, -1, 29, 64], dtype=torch.int32)
    gg.coda_paged_append(Z.cuda(), pos.cuda(), table.cuda(), kc, vc, hq, want_q=False)
    for i, p in ((0, 0), (2, 29), (3, 64)):
        assert torch.equal(kc[table[i, p // page], :, p % page].cpu(), Z[i, hq * d:2 * hq * d].view(hkv, d))
        assert torch.equal(vc[table[i, p // page], :, p % page].cpu(), Z[i, 2 * hq * d:].view(hkv, d))
    assert gg.coda_get_device_status() == gg.CODA_OK


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_attention_does_not_mix_rows_in_a_long_batch(types):
    """Thousands of short rows: one key each, so every output is that key's value, and rows without keys between them."""
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page, M = 4, 2, 64, 4, 5003
    lens = [(1 if i % 7 else 0) for i in range(M)]
    q, k, v, table, ln, s = make(hq, hkv, d, page, lens, types, 77)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, **scales(types[1], s)).cpu()
    first = v.view(torch.uint8 if types[1] == E4 else types[1])[table[:, 0].clamp(min=0).long(), :, 0]
    first = (first.view(E4) if types[1] == E4 else first).to(U.F64) * s[1]
    want = first[:, :, None].expand(M, hkv, hq // hkv, d).reshape(M, hq * d) * (ln > 0).to(U.F64)[:, None]
    # a single weight of 1: the scale's product and the output's rounding are left
    assert ((o.to(U.F64) - want).abs() <= (U.HALF[types[0]] + 2.0 ** -21) * want.abs()).all()


def test_attention_workspace_serves_other_heads_and_batches():
    """One workspace, sized for the larger heads, taken in turn by calls of other shapes: every call leaves it ready."""
    import gemm_epilogue_fusion_gb300 as gg
    shapes = [(32, 8, 128, 16, [3000, 5]), (4, 2, 64, 16, [9000]), (8, 8, 128, 5, [100] * 20), (32, 8, 128, 16, [1])]
    ws = gg.paged_attention_workspace(32, 8, 128, "cuda")
    for _ in range(2):
        for hq, hkv, d, page, lens in shapes:
            q, k, v, table, ln, s = make(hq, hkv, d, page, lens, (BF, BF), hq + d)
            fresh = gg.paged_attention_workspace(hq, hkv, d, "cuda")
            args = (q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda())
            assert torch.equal(gg.coda_paged_attention(*args, ws), gg.coda_paged_attention(*args, fresh))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", [[1], [2], [5000], [4096], [20000, 1, 1, 0], [1] * 300, [37] * 700,
                                  list(range(0, 260))], ids=lambda v: f"{len(v)}x{v[0]}")
def test_attention_splits_the_length(types, lens):
    """One long sequence over many blocks, many short ones over one, and mixtures."""
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page = 4, 2, 64, 16
    q, k, v, table, ln, s = make(hq, hkv, d, page, lens, types, len(lens), q_scale=3.0)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    lse = torch.empty(len(lens), hq).cuda()
    for _ in range(2):
        o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse,
                                    **scales(types[1], s))
        check(q, k, v, table, ln, s, o, lse)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("hq", [8, 24, 48])
def test_attention_keeps_the_small_weights_beside_a_large_one(types, hq):
    """One key with 2^25 times the others' weight and no value: the output is what the others add up to."""
    import gemm_epilogue_fusion_gb300 as gg
    M, hkv, d, page, n = 24, 4, 16, 64, 16384
    q, k, v, table, _, s = make(1, hkv, d, page, [n], types, hq, poison=False)
    q = torch.ones(M, hq, d).to(types[0])
    k.view(torch.uint8).zero_()
    at = int(table[0, 0])
    k.view(torch.uint8 if types[1] == E4 else types[1])[at, :, 5] = (
        torch.tensor(208.0).to(E4).view(torch.uint8) if types[1] == E4 else 4.5)
    v = (v.float().abs() + 8).to(types[1])
    v.view(torch.uint8 if types[1] == E4 else types[1])[at, :, 5] = 0
    row_seq, ln = torch.zeros(M, dtype=torch.int32), torch.full((M,), n, dtype=torch.int32)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    lse = torch.empty(M, hq).cuda()
    o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse,
                                row_seq=row_seq.cuda(), **scales(types[1], s))
    check(q, k, v, table, ln, s, o, lse, row_seq=row_seq.tolist())


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_attention_rows_of_one_sequence_strided_queries_and_scale(types):
    """Several new tokens of one sequence, each with its own length; queries read out of a QKV product's rows."""
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page = 8, 2, 64, 16
    q, k, v, table, _, s = make(hq, hkv, d, page, [70, 33], types, 3)
    row_seq, lens = [0, 0, 0, 1, 1, 0], [70, 69, 1, 33, 32, 0]
    g = U.gen(9)
    Z = randn(6, (hq + 2 * hkv) * d, dtype=types[0], g=g)
    q = Z[:, :hq * d].reshape(6, hq, d)
    ln = torch.tensor(lens, dtype=torch.int32)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    view = Z.cuda()[:, :hq * d].unflatten(1, (hq, d))
    assert not view.is_contiguous()
    lse = torch.empty(6, hq).cuda()
    o = gg.coda_paged_attention(view, k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse, scale=0.31,
                                row_seq=torch.tensor(row_seq, dtype=torch.int32).cuda(), **scales(types[1], s))
    check(q, k, v, table, ln, s, o, lse, row_seq=row_seq, scale=0.31)


@pytest.mark.parametrize("types", [(BF, BF), (F32, F32)], ids=["bf16", "f32"])
def test_attention_infinite_and_nan_keys(types):
    """Scores of -inf have no weight (in the whole row: zeros), the type's lowest values are ordinary numbers, and NaN
    in a row's own keys reaches that row's heads only."""
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page = 4, 2, 64, 16
    lens = [40, 40, 40, 40]
    q, k, v, table, ln, s = make(hq, hkv, d, page, lens, types, 4)
    q = q.abs() + 0.1
    low = torch.finfo(types[0]).min

    def put(cache, b, t, h, e, x):
        cache[table[b, t // page], h, t % page, e] = x

    for t in range(40):
        put(k, 0, t, 0, 3, -math.inf)       # sequence 0, head 0: nothing left
        if t != 21:
            put(k, 1, t, 1, 5, -math.inf)   # sequence 1, head 1: only key 21 left
        if t % 3:
            put(k, 2, t, 0, 0, low)         # sequence 2: the lowest value in two of three keys
    put(k, 3, 7, 1, 2, math.nan)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    lse = torch.empty(4, hq).cuda()
    o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse).cpu()
    o, lse = o.view(4, hq, d), lse.cpu()
    assert (o[0, :2] == 0).all() and torch.isneginf(lse[0, :2]).all()
    assert torch.isfinite(o[0, 2:]).all() and torch.isfinite(lse[0, 2:]).all()
    assert torch.equal(o[1, 2:], v[table[1, 1], 1, 5].expand(2, d))
    assert torch.isnan(o[3, 2:]).all() and torch.isnan(lse[3, 2:]).all()
    assert torch.isfinite(o[3, :2]).all()
    ref = U.attention(q, k, v, table, ln, range(4), d ** -0.5)
    assert ((o[2].to(U.F64) - ref[0][2]).abs() <= ref[2][2] * 2.0 ** -6).all()


def test_attention_bad_indices_are_left_out_and_said():
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page = 4, 2, 64, 16
    q, k, v, table, ln, s = make(hq, hkv, d, page, [50, 50, 50], (BF, BF), 8, poison=False)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    c = lambda t: t.cuda()  # noqa: E731
    good = gg.coda_paged_attention(c(q), c(k), c(v), c(table), c(ln), ws).cpu()
    # a length beyond the table counts as the table's end (its last slots are filled here)
    ln2 = torch.tensor([50, 64, 2147483647], dtype=torch.int32)
    o = gg.coda_paged_attention(c(q), c(k), c(v), c(table), c(ln2), ws)
    with pytest.raises(gg.CodaError, match="out of range"):
        gg.coda_get_device_status()
    check(q, k, v, table, torch.tensor([50, 64, 64]), s, o, None)
    # a sequence out of range: a row without keys; the other rows are as before
    seq = torch.tensor([0, 3, -1], dtype=torch.int32)
    o = gg.coda_paged_attention(c(q), c(k), c(v), c(table), c(ln), ws, row_seq=c(seq)).cpu()
    with pytest.raises(gg.CodaError, match="out of range"):
        gg.coda_get_device_status()
    assert torch.equal(o[0], good[0]) and (o[1:] == 0).all()
    # a page out of range: its keys are left out
    for bad in (-1, k.shape[0], 2147483647, -2147483648):
        t2 = table.clone()
        t2[1, 1] = bad
        o = gg.coda_paged_attention(c(q), c(k), c(v), c(t2), c(ln), ws).cpu()
        with pytest.raises(gg.CodaError, match="out of range"):
            gg.coda_get_device_status()
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        t3 = torch.cat((table[1:2, :1], table[1:2, 2:]), 1)  # the same sequence with those 16 keys cut out
        check(q[1:2], k, v, t3, torch.tensor([34]), s, o[1:2], None)
    assert gg.coda_get_device_status() == gg.CODA_OK


@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_cache_offsets_beyond_32_bits(types):
    """Pages whose elements lie behind 2^31 of the cache, written by append and read by attention."""
    import gemm_epilogue_fusion_gb300 as gg
    dt, ct = types
    hq, hkv, d, page = 2, 1, 128, 64
    num_pages = (1 << 31) // (hkv * page * d) + 3
    kc, vc = (torch.empty(num_pages, hkv, page, d, dtype=ct, device="cuda") for _ in range(2))
    g = U.gen(2)
    table = torch.tensor([[num_pages - 1, num_pages - 2]], dtype=torch.int32)
    n = 100
    Z = randn(n, (hq + 2 * hkv) * d, dtype=dt, g=g)
    s = (0.02, 0.02) if ct == E4 else (1.0, 1.0)
    kw = scales(ct, s)
    pos = torch.arange(n, dtype=torch.int32)
    gg.coda_paged_append(Z.cuda(), pos.cuda(), table.cuda(), kc, vc, hq, want_q=False,
                         row_seq=torch.zeros(n, dtype=torch.int32).cuda(), **kw)
    q = randn(1, hq, d, dtype=dt, g=g)
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    o = gg.coda_paged_attention(q.cuda(), kc, vc, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), ws, **kw)
    tail_k, tail_v = kc[num_pages - 2:].cpu(), vc[num_pages - 2:].cpu()
    check(q, tail_k, tail_v, table - (num_pages - 2), torch.tensor([n]), s, o, None)
    if ct == dt:
        assert torch.equal(tail_k[1, 0, :64], Z.view(n, hq + 2, d)[:64, hq])
    del kc, vc
    torch.cuda.empty_cache()


def test_append_and_attention_on_another_stream_and_in_a_graph():
    """A captured decode step (append, then attention) replayed on new values in the same buffers equals eager calls,
    with an eager call on the same workspace between the replays."""
    import gemm_epilogue_fusion_gb300 as gg
    hq, hkv, d, page = 8, 2, 128, 16
    q, k, v, table, ln, s = make(hq, hkv, d, page, [500, 3, 77, 0], (BF, BF), 12, poison=False)
    g = U.gen(13)
    width = (hq + 2 * hkv) * d
    Zs = [randn(4, width, dtype=BF, g=g).cuda() for _ in range(3)]
    kc, vc, table, ln = k.cuda(), v.cuda(), table.cuda(), ln.cuda()
    pos = (ln - 1).int()
    ws = gg.paged_attention_workspace(hq, hkv, d, "cuda")
    want = []
    for z in Zs:
        qq = gg.coda_paged_append(z, pos, table, kc, vc, hq, base=10000.0)
        qq[3].zero_()  # the padded row's queries are left as they were
        want.append(gg.coda_paged_attention(qq, kc, vc, table, ln, ws).clone())
    Z, Q, O = Zs[0].clone(), torch.zeros(4, hq, d, dtype=BF).cuda(), torch.empty(4, hq * d, dtype=BF).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gg.coda_paged_append(Z, pos, table, kc, vc, hq, base=10000.0, Q=Q)
        gg.coda_paged_attention(Q, kc, vc, table, ln, ws, O=O)
    side.synchronize()
    assert torch.equal(O, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gg.coda_paged_append(Z, pos, table, kc, vc, hq, base=10000.0, Q=Q)
        gg.coda_paged_attention(Q, kc, vc, table, ln, ws, O=O)
    for z, w in list(zip(Zs, want)) * 2:
        Z.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, w)
        eager = gg.coda_paged_attention(Q, kc, vc, table, ln, ws)
        assert torch.equal(eager, w)
    assert gg.coda_get_device_status() == gg.CODA_OK
