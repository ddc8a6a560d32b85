"""The C marshalling of the decode and scoring calls (coda_marshal.c), on the
host with no GPU: stand-in tensors and stand-in library functions show which
arguments reach the C ABI, and that every defect of an argument is handed back
to the Python checks (None) instead of being passed on."""
import ctypes

import pytest
import torch

import gemm_epilogue_fusion_gb300 as g

BF, F32, E4, U8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.int32
NAMES = ("coda_paged_append", "coda_paged_attention", "coda_paged_attention_workspace_bytes", "coda_logprobs",
         "coda_logprobs_backward")


class Fake:
    """What the marshalling reads of a tensor."""

    def __init__(self, ptr, shape, dtype, device=0, contiguous=True, stride=None):
        self.ptr, self.shape, self.dtype, self.device_index = ptr, tuple(shape), dtype, device
        self.contiguous, self.strides = contiguous, stride
        if stride is None:
            s, n = [], 1
            for x in reversed(self.shape):
                s.insert(0, n)
                n *= x
            self.strides = tuple(s)

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.ptr

    def stride(self):
        return self.strides


@pytest.fixture()
def fast():
    """The module with stand-ins for the library's functions; `calls` collects their arguments."""
    lib = g.load_library()
    m = g._fast
    assert m is not None
    calls, keep = [], []

    def stand_in(name):
        res, args = g.SIGNATURES[name]
        proto = ctypes.CFUNCTYPE(res, *args)
        answer = (lambda *a: 4096) if name.endswith("_bytes") else (lambda *a: calls.append(a) or 7)
        keep.append(proto(answer))
        return ctypes.cast(keep[-1], ctypes.c_void_p).value

    m.init(F32, BF, E4, U8, I32, lambda: 0, lambda dev: 1000 + dev, *(stand_in(n) for n in NAMES))
    m.calls = calls
    yield m
    del m.calls
    g._load_marshal(lib)


def append_args():
    M, hq, hkv, d, page, pages = 3, 4, 2, 64, 16, 5
    return {"Z": Fake(16, (M, (hq + 2 * hkv) * d), BF), "pos": Fake(32, (M,), I32), "seq": Fake(48, (M,), I32),
            "tab": Fake(64, (2, 9), I32), "Q": Fake(80, (M, hq, d), BF), "k": Fake(96, (pages, hkv, page, d), E4),
            "v": Fake(112, (pages, hkv, page, d), E4), "sk": Fake(128, (1,), F32), "sv": Fake(144, (), F32), "hq": hq,
            "base": 1e4, "stream": None}


def attention_args():
    M, hq, hkv, d, page, pages = 3, 4, 2, 64, 16, 5
    return {"Q": Fake(16, (M, hq, d), BF, contiguous=False, stride=(512, d, 1)), "k": Fake(32, (pages, hkv, page, d), BF),
            "v": Fake(48, (pages, hkv, page, d), BF), "tab": Fake(64, (3, 9), I32), "len": Fake(80, (M,), I32),
            "ws": Fake(96, (1024,), I32), "seq": None, "scale": 0.125, "O": Fake(112, (M, hq * d), BF),
            "lse": Fake(128, (M, hq), F32), "sk": None, "sv": None, "stream": 77}


def logprobs_args():
    M, V, top = 3, 13, 2
    return {"x": Fake(16, (M, V), BF, contiguous=False, stride=(16, 1)), "t": Fake(32, (M,), I32), "top": top,
            "lp": Fake(48, (M,), F32), "ent": Fake(64, (M,), F32), "lse": Fake(80, (M,), F32),
            "tl": Fake(96, (M, top), F32), "ti": Fake(112, (M, top), I32), "stream": None}


def backward_args():
    M, V = 3, 13
    return {"x": Fake(16, (M, V), F32, contiguous=False, stride=(16, 1)), "t": Fake(32, (M,), I32),
            "lse": Fake(48, (M,), F32), "ent": Fake(64, (M,), F32), "dl": Fake(80, (M,), F32), "dh": None,
            "dx": Fake(96, (M, V), F32, contiguous=False, stride=(20, 1)), "stream": None}


ALL = {"paged_append": append_args, "paged_attention": attention_args, "logprobs": logprobs_args,
       "logprobs_backward": backward_args}


def test_arguments_reach_the_library_in_order(fast):
    assert fast.paged_append(*append_args().values()) == 7
    assert fast.calls.pop() == (16, 32, 48, 64, 80, 96, 112, 3, 2, 9, 4, 2, 64, 5, 16, 1e4, g.CODA_BF16, g.CODA_E4M3,
                                128, 144, 1000)
    assert fast.paged_attention(*attention_args().values()) == 7
    assert fast.calls.pop() == (16, 512, 32, 48, 64, 80, None, 112, 128, 3, 3, 9, 4, 2, 64, 5, 16, 0.125, g.CODA_BF16,
                                g.CODA_BF16, None, None, 96, 77)
    assert fast.logprobs(*logprobs_args().values()) == 7
    assert fast.calls.pop() == (16, 16, 32, 48, 64, 80, 96, 112, 3, 13, 2, g.CODA_BF16, 1000)
    assert fast.logprobs_backward(*backward_args().values()) == 7
    assert fast.calls.pop() == (16, 16, 32, 48, 64, 80, None, 96, 20, 3, 13, g.CODA_F32, 1000)


def test_optional_arguments_and_single_rows(fast):
    a = append_args()
    a.update(seq=None, Q=None, sk=None, sv=None, k=Fake(96, (5, 2, 16, 64), BF), v=Fake(112, (5, 2, 16, 64), BF), base=0)
    assert fast.paged_append(*a.values()) == 7
    assert fast.calls.pop()[2:6] == (None, 64, None, 96)
    a = logprobs_args()
    a.update(x=Fake(16, (1, 13), BF), t=Fake(32, (1,), I32), top=0, lp=Fake(48, (1,), F32), ent=Fake(64, (1,), F32),
             lse=Fake(80, (1,), F32), tl=None, ti=None)
    assert fast.logprobs(*a.values()) == 7
    assert fast.calls.pop()[:2] == (16, 16)  # a single row: whole 16 bytes
    a = attention_args()
    a["Q"] = Fake(16, (1, 4, 64), BF)
    a.update(tab=Fake(64, (1, 9), I32), len=Fake(80, (1,), I32), O=Fake(112, (1, 256), BF), lse=None)
    assert fast.paged_attention(*a.values()) == 7
    assert fast.calls.pop()[1] == 256


@pytest.mark.parametrize("name", ALL)
def test_every_defect_is_handed_back(fast, name):
    call, good = getattr(fast, name), ALL[name]
    for key, t in good().items():
        if not isinstance(t, Fake):
            continue
        strided = not t.contiguous
        bad = [Fake(t.ptr, t.shape, torch.float16, stride=t.strides, contiguous=t.contiguous),
               Fake(t.ptr, t.shape, torch.int64, stride=t.strides, contiguous=t.contiguous),
               Fake(t.ptr, t.shape, t.dtype, device=1, stride=t.strides, contiguous=t.contiguous),
               Fake(t.ptr, t.shape, t.dtype, device=-1, stride=t.strides, contiguous=t.contiguous),
               object(), [1, 2], "x"]
        if key not in ("sk", "sv"):
            bad.append(Fake(t.ptr, t.shape + (1,), t.dtype) if key != "ws" else Fake(t.ptr, (1023,), t.dtype))
            bad.append(Fake(t.ptr, t.shape * 3, t.dtype))
        if key not in ("tab", "ws", "sk", "sv"):
            bad.append(Fake(t.ptr, (t.shape[0] + 1,) + t.shape[1:], t.dtype, stride=t.strides))
            if (name, key) != ("logprobs", "x"):  # there the logits themselves say how wide they are
                bad.append(Fake(t.ptr, t.shape[:-1] + (t.shape[-1] + 1,), t.dtype, stride=t.strides))
        if strided:
            bad.append(Fake(t.ptr, t.shape, t.dtype, contiguous=False, stride=t.strides[:-1] + (2,)))
        else:
            bad.append(Fake(t.ptr, t.shape, t.dtype, contiguous=False))
        if key in ("sk", "sv"):
            bad.append(Fake(t.ptr, (0,), t.dtype))
        for b in bad:
            if key == "ws" and isinstance(b, Fake) and b.shape == t.shape * 3 and b.contiguous:
                continue  # a larger workspace is fine
            a = good()
            a[key] = b
            assert call(*a.values()) is None, (key, getattr(b, "shape", b), getattr(b, "dtype", None))
    assert call() is None and call(None) is None and call(*[None] * len(good())) is None
    assert not fast.calls


def test_caches_of_two_types_and_missing_tensors_are_handed_back(fast):
    for update in ({"v": Fake(112, (5, 2, 16, 64), U8)}, {"v": Fake(112, (5, 2, 16, 64), BF)}, {"k": None}, {"Z": None},
                   {"pos": None}, {"tab": None}, {"hq": "x"}, {"hq": 5}, {"base": "x"}, {"stream": "x"}):
        a = append_args()
        a.update(update)
        assert fast.paged_append(*a.values()) is None, update
    assert not fast.calls


def test_cpu_tensors_are_handed_back_to_the_checks():
    g.load_library()
    x, t = torch.zeros(2, 16, dtype=BF), torch.zeros(2, dtype=I32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        g.coda_logprobs(x, t)


@pytest.mark.gpu
def test_both_ways_give_the_same_bits(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib_ready = g.load_library()
    assert lib_ready is not None and g._fast is not None
    gen = torch.Generator(device="cuda").manual_seed(0)
    M, hq, hkv, d, page, pages = 3, 4, 2, 64, 16, 12
    Z = torch.randn(M, (hq + 2 * hkv) * d, device="cuda", generator=gen).bfloat16()
    table = torch.randperm(pages, device="cuda", generator=gen)[:9].int().view(3, 3)
    pos, ln = torch.tensor([4, 40, 17]).int().cuda(), torch.tensor([5, 41, 18]).int().cuda()
    x = torch.randn(5, 1000, device="cuda", generator=gen)
    t = torch.randint(0, 1000, (5,), device="cuda", generator=gen).int()
    ws = g.paged_attention_workspace(hq, hkv, d, "cuda")

    def everything(stream):
        k, v = (torch.zeros(pages, hkv, page, d, device="cuda").bfloat16() for _ in range(2))
        q = g.coda_paged_append(Z, pos, table, k, v, hq, base=1e4, stream=stream)
        o = g.coda_paged_attention(q, k, v, table, ln, ws, stream=stream)
        f = g.coda_logprobs(x, t, 4, stream=stream)
        return [k, v, q, o, *f.values(), g.coda_logprobs_backward(x, t, f["lse"], f["entropy"], f["logp"], f["logp"],
                                                                  stream=stream)]

    a = everything(None)
    b = everything(torch.cuda.current_stream())
    monkeypatch.setattr(g, "_fast", None)
    c = everything(None)
    for p, q, r in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, r)
    with pytest.raises(g.CodaError, match="page_size|head_dim|top"):
        g.coda_logprobs(x, t, 65)
    monkeypatch.undo()
    with pytest.raises(g.CodaError, match="top"):
        g.coda_logprobs(x, t, 65)
