"""The operators around the layer on a stream that the caller names, as a torch stream or as a raw handle."""
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


def calls(stream):
    """Every operator once, on inputs made on the current stream; what they return."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy = r(2, 600, 256).bfloat16(), r(2, 600, 256).bfloat16()
    g, w, state = -x.abs() * 0.1, r(256), r(1200, 256)
    head, t = (r(1000, 256) * 0.1).bfloat16(), torch.arange(1200, device="cuda", dtype=torch.int32) - 100
    dl = torch.rand(1200, generator=gen, device="cuda")
    if stream is not None:
        handle = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)
        handle.wait_stream(torch.cuda.current_stream())
    got = list(gdn.gated_scan_fwd(x, g, stream=stream))
    got += gdn.gated_scan_bwd(x, g, got[0], dy, stream=stream)
    got += [gdn.gated_scan_step(state, x.view(1200, 256), g.view(1200, 256), stream=stream), state]
    y, mean, rstd = gdn.layer_norm_fwd(x, w, w, stream=stream)
    got += [y, mean, rstd, *gdn.layer_norm_bwd(dy, x, mean, rstd, w, stream=stream)]
    loss, lse = gdn.linear_cross_entropy_fwd(x.view(1200, 256), head, t, stream=stream)
    got += [loss, lse, *gdn.linear_cross_entropy_bwd(x.view(1200, 256), head, t, lse, dl, stream=stream)]
    # the wrappers' own workspaces are free again here; memory of the same sizes must not reach running kernels
    trash = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20, 1 << 24)]
    torch.cuda.synchronize()
    del trash
    return got


def test_named_streams_give_the_same_bits():
    want = calls(None)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for a, b in zip(calls(stream), want):
            assert torch.equal(a, b)
