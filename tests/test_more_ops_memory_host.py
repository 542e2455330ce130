"""Whose memory the newer wrappers take when the caller names a stream, sizes beyond 32 bits, and refusals of the 8-bit
product's self-test; no GPU is needed."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
from gated_delta_rule_12_gb300 import build as gbuild
from test_ops_memory_host import FakeStream, world  # noqa: F401
from test_ops_sizes_host import BIG, wide

X, V, I = torch.zeros(2, 3, 8), torch.zeros(8), torch.zeros(2, 8)
T, S = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3)
E, C = torch.zeros(2, 8, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(2, 1)
CALLS = {
    "norm": lambda s: gdn.rms_norm_fwd(X, V, residual=X, stream=s),
    "norm in 8 bits": lambda s: gdn.rms_norm_fp8(X, V, residual=X, stream=s),
    "norm backward": lambda s: gdn.rms_norm_bwd(X, X, S, V, dresidual=X, stream=s),
    "quantising": lambda s: gdn.fp8_quantize(X, stream=s),
    "product": lambda s: gdn.fp8_linear(E, C, E, C[:1], stream=s),
    "log probabilities": lambda s: gdn.linear_log_probs_fwd(I, I, T, top_k=2, stream=s),
    "gradient": lambda s: gdn.linear_log_probs_bwd(I, I, T, V[:2], V[:2], V[:2], V[:2], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_named_stream(world, name):  # noqa: F811
    stream = FakeStream()
    got = CALLS[name](stream)
    got = got if isinstance(got, tuple) else (got,)
    assert world["lib"].streams == [77] and world["now"] is world["here"]
    assert world["made"] and all(s is stream for _, s in world["made"])
    for t in got:
        assert any(t is r and s is world["here"] for r, s in world["recorded"])


@pytest.mark.parametrize("name", CALLS)
def test_without_a_name_the_current_stream_it_is(world, name):  # noqa: F811
    CALLS[name](None)
    assert world["lib"].streams == [5] and all(s is world["here"] for _, s in world["made"]) and not world["recorded"]


def test_what_the_caller_gave_is_the_callers(world):  # noqa: F811
    out, total = torch.zeros_like(X), X.clone()
    world["made"].clear()
    y, s, rstd = gdn.rms_norm_fwd(X, V, residual=total, out=out, residual_out=total, stream=FakeStream())
    assert y is out and s is total and all(r is rstd for r, _ in world["recorded"])
    given = torch.zeros(2, 2, dtype=torch.bfloat16)
    world["recorded"].clear()
    assert gdn.fp8_linear(E, C, E, C[:1], out=given, stream=FakeStream()) is given and not world["recorded"]


B8 = lambda *shape: wide(*shape, dtype=torch.float8_e4m3fn)  # noqa: E731


@pytest.mark.parametrize("call", [
    lambda: gdn.rms_norm_fwd(wide(1, BIG)),
    lambda: gdn.rms_norm_fp8(wide(1, BIG)),
    lambda: gdn.rms_norm_bwd(wide(1, BIG), wide(1, BIG), wide(1)),
    lambda: gdn.fp8_quantize(wide(1, BIG)),
    lambda: gdn.fp8_linear(B8(BIG, 8), wide(BIG, 1), B8(3, 8), wide(1, 1)),
    lambda: gdn.fp8_linear(B8(3, 8), wide(3, 1), B8(BIG, 8), wide(-(-BIG // 128), 1)),
    lambda: gdn.linear_log_probs_fwd(wide(1, 8), wide(BIG, 8), wide(1, dtype=torch.int32)),
    lambda: gdn.linear_log_probs_bwd(wide(BIG, 8), wide(3, 8), wide(BIG, dtype=torch.int32), wide(BIG), None, wide(BIG)),
])
def test_sizes_beyond_32_bits_are_refused(call):
    gbuild.build()
    with pytest.raises(ValueError, match="2\\^31"):
        call()


FAKE = 1 << 20
STALL = dict(limit=1000, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, out=FAKE, M=4, N=16, K=32, work=FAKE, size=1 << 40, stream=None)


@pytest.mark.parametrize("over,code", [(dict(limit=0), 1), (dict(limit=1000001), 1), (dict(x=None), 1), (dict(M=0), 1),
                                       (dict(K=24), 2), (dict(x=FAKE + 8), 2), (dict(work=None), 3), (dict(size=64), 3)])
def test_selftest_refusals(over, code):
    gbuild.build()
    assert gdn.load_library().gdn_selftest_fp8_linear_timeout(*{**STALL, **over}.values()) == code


LOGP_STALL = dict(limit=1000, h=FAKE, w=FAKE, t=FAKE, logp=FAKE, ent=FAKE, ids=FAKE, top=FAKE, N=4, D=16, V=32, k=3,
                  work=FAKE, size=1 << 40, stream=None)


@pytest.mark.parametrize("over,code", [(dict(limit=0), 1), (dict(limit=1000001), 1), (dict(h=None), 1), (dict(N=0), 1),
                                       (dict(k=33), 1), (dict(ids=None), 1), (dict(logp=FAKE + 2), 1), (dict(D=12), 2),
                                       (dict(work=None), 3), (dict(size=256), 3)])
def test_log_probabilities_selftest_refusals(over, code):
    gbuild.build()
    assert gdn.load_library().gdn_selftest_linear_log_probs_timeout(*{**LOGP_STALL, **over}.values()) == code
