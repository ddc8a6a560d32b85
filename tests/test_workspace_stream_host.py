"""Workspaces that a call makes for itself come from the pool of the stream it
launches on, on the host: a block that the caching allocator takes back when
the call returns is then given out again behind the call's kernels alone, and
what used it before has ended when they begin."""
import contextlib

import pytest
import torch

import gemm_epilogue_fusion_gb300 as g

BF, I32 = torch.bfloat16, torch.int32


class Stream:
    """Anything with the address of a stream."""
    cuda_stream = 0x5EED0


def external(address, device=None):
    return "external", address


HERE = external(Stream.cuda_stream)


@pytest.fixture
def made(monkeypatch):
    """(name, stream it was made under) of each workspace."""
    lib = g.load_library()
    under, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        under.append(stream)
        yield
        under.pop()

    def recorded(name):
        inner = getattr(g, name)

        def make(*args, **kw):
            made.append((name, under[-1]))
            return inner(*args, **kw)
        monkeypatch.setattr(g, name, make)

    class Fast:
        def __getattr__(self, name):
            return lambda *args: g.CODA_OK

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(g, "_fast", Fast())
    monkeypatch.setattr(g, "load_library", lambda: lib)
    for n in ("route_workspace", "add_rmsnorm_backward_workspace"):
        recorded(n)
    return made


def norm_backward(**kw):
    X = torch.zeros(4, 16, dtype=BF)
    g.coda_add_rmsnorm_backward(X, X, torch.ones(4), torch.ones(16), **kw)


def route(**kw):
    g.coda_route(torch.zeros(600, 16, dtype=BF), 2, **kw)


@pytest.mark.parametrize("call, name", [(route, "route_workspace"), (norm_backward, "add_rmsnorm_backward_workspace")])
def test_a_given_stream(made, call, name):
    s = Stream()
    call(stream=s)
    call()
    call(stream=s, workspace=torch.zeros(100000))
    assert made == [(name, HERE), (name, None)]


def test_the_dense_norm_gradient(made, monkeypatch):
    """coda_rmsnorm_backward, which is not marshalled in C: up to its own checks."""
    s, seen = Stream(), []
    inner = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append(made_under()) or inner(*a, **k))
    held = []

    @contextlib.contextmanager
    def on(stream):
        held.append(stream)
        yield
        held.pop()

    def made_under():
        return held[-1] if held else None

    monkeypatch.setattr(torch.cuda, "stream", on)
    X = torch.zeros(4, 16, dtype=BF)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        g.coda_rmsnorm_backward(X, X, torch.ones(4), torch.ones(16), torch.ones(4, 1), dgamma=torch.ones(16), dH=X.clone(),
                                Yt=X.clone(), stream=s)
    assert seen == [HERE]


def test_addresses_of_streams(monkeypatch):
    """A stream by its address: the default one's two addresses, and another's."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    assert g._stream_object(0, "cuda") == g._stream_object(1, "cuda") == "default"
    assert g._stream_object(0x7000, "cuda") == external(0x7000)
    assert g._stream_object(Stream(), "cuda") == HERE
