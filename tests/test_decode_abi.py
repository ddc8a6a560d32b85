"""Refusals of the decode and scoring calls, on the host: bad arguments come
back before anything is enqueued (the addresses are never dereferenced)."""
import pytest
import torch

import gemm_epilogue_fusion_gb300 as g

A = 0x7F0000000000
MB = 1 << 20
BAD, OK = g.CODA_ERR_INVALID_ARG, g.CODA_OK


@pytest.fixture(scope="module")
def lib():
    return g.load_library()


def append(lib, Z=A, positions=A + 64 * MB, row_seq=None, table=A + 65 * MB, Q=A + 66 * MB, K=A + 128 * MB,
           V=A + 192 * MB, M=4, seqs=4, max_pages=8, hq=8, hkv=2, d=64, pages=32, page=16, base=10000.0, dt=1, ct=1,
           sk=None, sv=None):
    return lib.coda_paged_append(Z, positions, row_seq, table, Q, K, V, M, seqs, max_pages, hq, hkv, d, pages, page,
                                 base, dt, ct, sk, sv, None)


def attend(lib, Q=A, ldq=512, K=A + 128 * MB, V=A + 192 * MB, table=A + 65 * MB, lengths=A + 64 * MB, row_seq=None,
           O=A + 66 * MB, lse=None, M=4, seqs=4, max_pages=8, hq=8, hkv=2, d=64, pages=32, page=16, scale=0.125, dt=1,
           ct=1, sk=None, sv=None, ws=A + 512 * MB):
    return lib.coda_paged_attention(Q, ldq, K, V, table, lengths, row_seq, O, lse, M, seqs, max_pages, hq, hkv, d,
                                    pages, page, scale, dt, ct, sk, sv, ws, None)


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("bad", [
    dict(dt=2, ct=2), dict(dt=0, ct=1), dict(dt=1, ct=0), dict(dt=0, ct=2), dict(dt=7, ct=7),
    dict(M=-1), dict(M=1 << 31), dict(M=5),  # more rows than sequences, and no row_seq
    dict(seqs=-1), dict(max_pages=0), dict(max_pages=1 << 31), dict(pages=0), dict(pages=1 << 31), dict(page=0),
    dict(page=-4), dict(hq=0), dict(hkv=0), dict(hq=7), dict(hq=-8, hkv=-2), dict(hq=1 << 20, hkv=1),
    dict(d=0), dict(d=-64), dict(d=60), dict(d=264), dict(pages=(1 << 31) - 1, page=(1 << 31) - 1),
    dict(ct=2), dict(ct=2, sk=A + 700 * MB), dict(ct=2, sk=A + 700 * MB, sv=A + 700 * MB + 2),
    dict(ct=2, sk=A + 700 * MB, sv=A + 700 * MB + 4, d=72), dict(sk=A + 700 * MB, sv=A + 700 * MB + 4),
    dict(table=None), dict(K=None), dict(V=None), dict(K=A + 128 * MB + 8), dict(table=A + 65 * MB + 2),
    dict(row_seq=A + 63 * MB + 2), dict(K=A + 192 * MB), dict(V=A + 128 * MB + 4096)],
    ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_paged_calls_refuse(lib, call, bad):
    if call is attend and (bad == dict(K=A + 192 * MB) or bad == dict(V=A + 128 * MB + 4096)):
        bad = dict(O=A + 128 * MB)  # only read there: an output over the cache instead
    assert call(lib, **bad) == BAD
    assert lib.coda_last_error()


@pytest.mark.parametrize("bad", [dict(Z=None), dict(Z=A + 8), dict(positions=None), dict(Q=A + 66 * MB + 4),
                                 dict(base=1.0), dict(base=-2.0), dict(base=float("nan")), dict(base=float("inf")),
                                 dict(Q=A), dict(K=A), dict(Q=A + 128 * MB), dict(positions=A + 128 * MB),
                                 dict(table=A + 192 * MB)], ids=str)
def test_append_refuses(lib, bad):
    assert append(lib, **bad) == BAD


@pytest.mark.parametrize("bad", [dict(Q=None), dict(lengths=None), dict(O=None), dict(ws=None), dict(ldq=504),
                                 dict(ldq=516), dict(ldq=1 << 41), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(scale=float("nan")), dict(lse=A + 66 * MB),
                                 dict(O=A), dict(ws=A + 128 * MB), dict(ws=A + 66 * MB), dict(lse=A + 1),
                                 dict(M=1 << 29, seqs=1 << 29)], ids=str)
def test_attention_refuses(lib, bad):
    assert attend(lib, **bad) == BAD


def test_no_rows_enqueue_nothing(lib):
    assert append(lib, M=0) == OK and attend(lib, M=0) == OK
    assert lib.coda_logprobs(A, 64, A, A, None, None, None, None, 0, 64, 0, 1, None) == OK
    assert lib.coda_logprobs_backward(A, 64, A, A, None, None, None, A, 64, 0, 64, 1, None) == OK


def test_workspace_size(lib):
    size = lib.coda_paged_attention_workspace_bytes
    assert size(32, 8, 128) > 0 and size(1, 1, 8) > 0
    for bad in ((0, 1, 64), (8, 0, 64), (7, 2, 64), (8, 2, 0), (8, 2, 257)):
        assert size(*bad) == -1
    with pytest.raises(ValueError, match="out of range"):
        g.paged_attention_workspace(7, 2, 64, "cpu")


def logp(lib, x=A, ld=512, t=A + 64 * MB, logp=A + 65 * MB, ent=None, lse=None, tl=A + 66 * MB, ti=A + 67 * MB, M=4,
         V=500, top=5, dt=1):
    return lib.coda_logprobs(x, ld, t, logp, ent, lse, tl, ti, M, V, top, dt, None)


@pytest.mark.parametrize("bad", [dict(dt=2), dict(dt=9), dict(M=-1), dict(M=1 << 31), dict(V=0), dict(V=1 << 30),
                                 dict(ld=499), dict(ld=501), dict(V=513), dict(top=-1), dict(top=65),
                                 dict(V=3, top=4), dict(x=None), dict(x=A + 2), dict(t=None), dict(logp=None),
                                 dict(tl=None), dict(ti=None), dict(logp=A), dict(ent=A + 65 * MB), dict(lse=A + 2),
                                 dict(tl=A + 67 * MB), dict(M=1 << 30, ld=1 << 39)], ids=str)
def test_logprobs_refuses(lib, bad):
    assert logp(lib, **bad) == BAD


def grad(lib, x=A, ld=512, t=A + 64 * MB, lse=A + 65 * MB, ent=A + 66 * MB, dl=A + 67 * MB, dh=A + 68 * MB,
         dx=A + 128 * MB, ldd=512, M=4, V=500, dt=1):
    return lib.coda_logprobs_backward(x, ld, t, lse, ent, dl, dh, dx, ldd, M, V, dt, None)


@pytest.mark.parametrize("bad", [dict(dt=2), dict(M=-1), dict(V=0), dict(ld=499), dict(ldd=504 - 8), dict(ldd=501),
                                 dict(x=None), dict(t=None), dict(lse=None), dict(ent=None), dict(dx=None),
                                 dict(dx=A), dict(dx=A + 1024), dict(dx=A + 65 * MB), dict(dl=A + 2)], ids=str)
def test_logprobs_backward_refuses(lib, bad):
    assert grad(lib, **bad) == BAD


def test_binding_checks_before_the_library_sees_a_pointer():
    bf, i32 = torch.bfloat16, torch.int32
    M, hq, hkv, d, page, pages = 3, 4, 2, 64, 16, 5
    Z, Q = torch.zeros(M, (hq + 2 * hkv) * d, dtype=bf), torch.zeros(M, hq, d, dtype=bf)
    K = torch.zeros(pages, hkv, page, d, dtype=bf)
    pos, table, ws = torch.zeros(M, dtype=i32), torch.zeros(M, 4, dtype=i32), torch.zeros(1 << 24, dtype=i32)
    x, t, r = torch.zeros(M, 64, dtype=bf), torch.zeros(M, dtype=i32), torch.zeros(M)
    cases = [
        (lambda: g.coda_paged_append(Z[:, 8:], pos, table, K, K.clone(), hq), ValueError, "Z has shape"),
        (lambda: g.coda_paged_append(Z.half(), pos, table, K, K.clone(), hq), TypeError, "dtype"),
        (lambda: g.coda_paged_append(Z, pos.long(), table, K, K.clone(), hq), TypeError, "positions has dtype"),
        (lambda: g.coda_paged_append(Z, pos[:2], table, K, K.clone(), hq), ValueError, "positions has shape"),
        (lambda: g.coda_paged_append(Z, pos, table[0], K, K.clone(), hq), ValueError, "page_table"),
        (lambda: g.coda_paged_append(Z, pos, table, K[0], K.clone(), hq), ValueError, "k_cache has 3"),
        (lambda: g.coda_paged_append(Z, pos, table, K, K[:4].clone(), hq), ValueError, "v_cache has shape"),
        (lambda: g.coda_paged_append(Z, pos, table, K, K.float(), hq), TypeError, "v_cache has dtype"),
        (lambda: g.coda_paged_append(Z.float(), pos, table, K, K.clone(), hq), TypeError, "k_cache has dtype"),
        (lambda: g.coda_paged_append(Z, pos, table, K, K.clone(), hq, row_seq=pos[:1]), ValueError, "row_seq"),
        (lambda: g.coda_paged_append(Z, pos, table, K, K.clone(), hq, Q=Q[:, :2]), ValueError, "Q has shape"),
        (lambda: g.coda_paged_append(Z, pos, table, K, K.clone(), hq), ValueError, "CUDA tensor"),
        (lambda: g.coda_paged_attention(Q[0], K, K, table, pos, ws), ValueError, "Q has 2"),
        (lambda: g.coda_paged_attention(Q[:, :, :32], K, K, table, pos, ws), ValueError, "head_dim"),
        (lambda: g.coda_paged_attention(Q, K, K, table, pos[:2], ws), ValueError, "lengths has shape"),
        (lambda: g.coda_paged_attention(Q, K, K, table, pos, ws[:1]), ValueError, "workspace holds"),
        (lambda: g.coda_paged_attention(Q, K, K, table, pos, ws, lse=r), ValueError, "lse has shape"),
        (lambda: g.coda_paged_attention(Q, K, K, table, pos, ws, O=Q), ValueError, "O has shape"),
        (lambda: g.coda_paged_attention(Q, K, K, table, pos, ws), ValueError, "CUDA tensor"),
        (lambda: g.coda_logprobs(x[0], t), ValueError, "logits has 1"),
        (lambda: g.coda_logprobs(x.half(), t), TypeError, "logits has dtype"),
        (lambda: g.coda_logprobs(x, t.long()), TypeError, "targets has dtype"),
        (lambda: g.coda_logprobs(x, t, 2, top_ids=torch.zeros(M, 3, dtype=i32)), ValueError, "top_ids has shape"),
        (lambda: g.coda_logprobs(x, t, logp=r[:2]), ValueError, "logp has shape"),
        (lambda: g.coda_logprobs(x, t), ValueError, "CUDA tensor"),
        (lambda: g.coda_logprobs_backward(x, t, r, dlogp=r.double()), TypeError, "dlogp has dtype"),
        (lambda: g.coda_logprobs_backward(x, t, r, dlogits=x[:, :8]), ValueError, "dlogits has shape"),
        (lambda: g.coda_logprobs_backward(x, t, r), ValueError, "CUDA tensor"),
    ]
    for fn, exc, msg in cases:
        with pytest.raises(exc, match=msg):
            fn()
