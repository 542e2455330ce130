"""Calls on a named stream while the current one still uses memory that it has given back."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_12_gb300 import build
    build.build()
    gdn.load_library()


def operators():
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy = r(2, 600, 256).bfloat16(), r(2, 600, 256).bfloat16()
    g, w = -x.abs() * 0.1, r(256)
    h, head = x.view(1200, 256), (r(1000, 256) * 0.1).bfloat16()
    t, dl = torch.arange(1200, device="cuda", dtype=torch.int32) - 100, torch.rand(1200, generator=gen, device="cuda")
    out, _ = gdn.gated_scan_fwd(x, g)
    _, mean, rstd = gdn.layer_norm_fwd(x, w, w)
    _, lse = gdn.linear_cross_entropy_fwd(h, head, t)
    state = r(1200, 256)
    q, gate = r(2, 300, 2, 128).bfloat16(), -0.1 * torch.rand(2, 300, 2, generator=gen, device="cuda")
    beta, memory = torch.rand(2, 300, 2, generator=gen, device="cuda"), r(2, 2, 128, 128)
    token = [v[:, 0].contiguous() for v in (q, q, q, gate, beta)]
    flt, par = 0.5 * r(2, 128, 4), r(2)
    return {
        "chunked forward": lambda s: gdn.chunk_fwd(q, q, q, gate, beta, stream=s),
        # all but dg, whose sums over a chunk's rows are atomic and differ in their last bits from call to call
        "chunked backward": lambda s: [gdn.chunk_bwd(q, q, q, gate, beta, q, stream=s)[i] for i in (0, 1, 2, 4, 5)],
        "decode": lambda s: (gdn.decode_step(memory.clone() if s is None else memory, *token, stream=s),),
        "prologue": lambda s: gdn.prologue(q, q, q, flt, flt, flt, gate, beta, par, par, stream=s),
        "prologue and forward": lambda s: gdn.prologue_chunk_fwd(q, q, q, flt, flt, flt, gate, beta, par, par, stream=s),
        "scan forward": lambda s: gdn.gated_scan_fwd(x, g, stream=s),
        "scan backward": lambda s: gdn.gated_scan_bwd(None, g, out, dy, stream=s),
        "scan step": lambda s: (gdn.gated_scan_step(state.clone() if s is None else state, h, g.view(1200, 256), stream=s),),
        "norm forward": lambda s: gdn.layer_norm_fwd(x, w, w, stream=s),
        "norm backward": lambda s: gdn.layer_norm_bwd(dy, x, mean, rstd, w, stream=s),
        "loss": lambda s: gdn.linear_cross_entropy_fwd(h, head, t, stream=s),
        "gradient": lambda s: gdn.linear_cross_entropy_bwd(h, head, t, lse, dl, stream=s),
    }


@pytest.mark.parametrize("name", ["scan forward", "scan backward", "scan step", "norm forward", "norm backward", "loss",
                                  "gradient", "chunked forward", "chunked backward", "decode", "prologue",
                                  "prologue and forward"])
def test_memory_still_in_use_on_the_current_stream(name):
    call = operators()[name]
    want = call(None)
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = a
    for _ in range(20):      # some 10 ms of work in front of the temporaries' use
        b = a @ b
    temps = [torch.empty_like(v) for v in want for _ in range(3)]
    for v in temps:
        v.fill_(7)
    copies = [v.clone() for v in temps]
    del temps, v             # their memory is free, their use is not over
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all((c == 7).all() for c in copies)
