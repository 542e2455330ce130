"""Whose memory the wrappers take when the caller names a stream; no GPU is needed (torch's streams and the library are
stood in for)."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn


class FakeStream:
    device, cuda_stream = None, 77


class FakeLibrary:
    """Every function succeeds, or says 64 where it is asked for a size, and is noted with its last argument."""
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 64
        return lambda *a: self.streams.append(a[-1]) or 0


@pytest.fixture
def world(monkeypatch):
    """What is current, what was allocated while what was current, and what was recorded for which stream."""
    here, w = FakeStream(), {"made": [], "recorded": []}
    here.cuda_stream, w["here"], w["now"] = 5, here, here

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.was, w["now"] = w["now"], self.s

        def __exit__(self, *a):
            w["now"] = self.was

    def noted(make):
        def f(*a, **k):
            t = make(*a, **{**k, "device": "cpu"})
            w["made"].append((t, w["now"]))
            return t
        return f

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w["now"])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w["recorded"].append((t, s)))
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noted(torch.empty_like))
    monkeypatch.setattr(gdn, "_empty", torch.empty)
    monkeypatch.setattr(gdn, "_empty_like", torch.empty_like)
    monkeypatch.setattr(gdn, "_raw_stream", lambda device: w["now"].cuda_stream)
    monkeypatch.setattr(gdn, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(gdn, "load_library", lambda: w["lib"])
    w["lib"] = FakeLibrary()
    monkeypatch.setattr(gdn, "_lib", w["lib"])
    return w


X, V, I = torch.zeros(2, 3, 8), torch.zeros(8), torch.zeros(2, 8)
T = torch.zeros(2, dtype=torch.int32)
S = torch.zeros(2, 3)
AROUND = {
    "scan forward": lambda s: gdn.gated_scan_fwd(X, X, stream=s),
    "scan backward": lambda s: gdn.gated_scan_bwd(None, X, X, X, stream=s),
    "scan step": lambda s: gdn.gated_scan_step(I, I, I, stream=s),
    "norm forward": lambda s: gdn.layer_norm_fwd(X, V, V, stream=s),
    "norm backward": lambda s: gdn.layer_norm_bwd(X, X, S, S, V, stream=s),
    "loss": lambda s: gdn.linear_cross_entropy_fwd(I, I, T, stream=s),
    "gradient": lambda s: gdn.linear_cross_entropy_bwd(I, I, T, V[:2], V[:2], stream=s),
}
Q, G, M = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2), torch.zeros(1, 2, 8, 8)
F, P = torch.zeros(2, 8, 4), torch.zeros(2)
LAYER = {
    "chunked forward": lambda s: gdn.chunk_fwd(Q, Q, Q, G, G, stream=s),
    "chunked backward": lambda s: gdn.chunk_bwd(Q, Q, Q, G, G, Q, stream=s),
    "decode": lambda s: gdn.decode_step(M, Q[:, 0], Q[:, 0], Q[:, 0], G[:, 0], G[:, 0], stream=s),
    "tokens of decode": lambda s: gdn.decode_multi(M, Q, Q, Q, G, G, stream=s),
    "prologue": lambda s: gdn.prologue(Q, Q, Q, F, F, F, G, G, P, P, stream=s),
    "prologue and forward": lambda s: gdn.prologue_chunk_fwd(*[Q.bfloat16()] * 3, F, F, F, G, G, P, P, stream=s),
}
CALLS = {**AROUND, **LAYER}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_named_stream(world, name):
    """What a kernel on the named stream writes is taken from that stream's memory and kept until the caller's stream,
    which uses it next, has done so."""
    stream = FakeStream()
    got = CALLS[name](stream)
    got = got if isinstance(got, tuple) else (got,)
    assert world["lib"].streams == [77] and world["now"] is world["here"]
    assert world["made"] and all(s is stream for _, s in world["made"])
    for t in got:
        assert any(t is r and s is world["here"] for r, s in world["recorded"])


def test_what_the_caller_gave_is_the_callers(world):
    out, state = torch.zeros_like(X), torch.zeros_like(I)
    world["made"].clear()
    got = gdn.gated_scan_fwd(X, X, out=out, final_state=state, stream=FakeStream())
    assert got[0] is out and got[1] is state and not world["made"] and not world["recorded"]
    five = tuple(torch.zeros_like(t) for t in (Q, Q, Q, G, G))
    world["made"].clear()
    assert gdn.prologue(Q, Q, Q, F, F, F, G, G, P, P, out=five, stream=FakeStream()) is not None
    assert not world["made"] and not world["recorded"]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_name_the_current_stream_it_is(world, name):
    CALLS[name](None)
    assert world["lib"].streams == [5] and all(s is world["here"] for _, s in world["made"]) and not world["recorded"]


def test_an_empty_batch_of_the_scan_needs_no_call(world):
    """As the other operators around the layer have it: nothing to compute is no error."""
    x = torch.zeros(0, 3, 8)
    out, fin = gdn.gated_scan_fwd(x, x, init_state=torch.zeros(0, 8))
    assert out.shape == x.shape and fin.shape == (0, 8)
    dx, dg, dinit = gdn.gated_scan_bwd(x, x, out, x, input_gate=True)
    assert dx.shape == dg.shape == x.shape and dinit.shape == (0, 8)
    assert gdn.gated_scan_bwd(None, x, out, x, want_dinit=False)[2] is None
    assert not world["lib"].streams
    with pytest.raises(ValueError, match="states"):
        gdn.gated_scan_fwd(x, x, init_state=torch.zeros(1, 8))
