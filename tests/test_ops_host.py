"""Refusals of the gated scan, layer norm and linear cross entropy, and checks of their 64-bit test references; no GPU
is needed (the pointers below are never dereferenced: validation fails first)."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
import ops_reference as ref
from gated_delta_rule_12_gb300 import build as gbuild

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


def call(fn, args, over):
    a = dict(args)
    a.update(over)
    return fn(*a.values())


SCAN = dict(x=FAKE, g=FAKE, s0=None, cu=None, nseq=0, out=FAKE, sf=None, B=1, T=8, D=16, dt=0, gate=0, stream=None)
SCAN_BWD = dict(x=FAKE, g=FAKE, out=FAKE, dout=FAKE, s0=None, df=None, cu=None, nseq=0, dx=FAKE, dg=FAKE, di=None,
                B=1, T=8, D=16, dt=0, gate=0, stream=None)
STEP = dict(s=FAKE, x=FAKE, g=FAKE, out=FAKE, N=1, D=16, dt=0, gate=0, stream=None)
NORM = dict(x=FAKE, w=FAKE, b=FAKE, out=FAKE, mean=FAKE, rstd=FAKE, rows=4, D=16, dt=0, eps=1e-5, stream=None)
NORM_BWD = dict(dout=FAKE, x=FAKE, mean=FAKE, rstd=FAKE, w=FAKE, dx=FAKE, dw=FAKE, db=FAKE, rows=4, D=16, dt=0,
                ws=FAKE, wsb=1 << 40, stream=None)
CE = dict(h=FAKE, w=FAKE, t=FAKE, loss=FAKE, lse=FAKE, N=4, D=16, V=32, dt=0, ws=FAKE, wsb=1 << 40, stream=None)
CE_BWD = dict(h=FAKE, w=FAKE, t=FAKE, lse=FAKE, dl=FAKE, dh=FAKE, dw=FAKE, N=4, D=16, V=32, dt=0, ws=FAKE,
              wsb=1 << 40, stream=None)


@pytest.mark.parametrize("over", [dict(B=0), dict(T=-1), dict(D=0), dict(dt=7), dict(x=None), dict(g=None),
                                  dict(out=None), dict(x=FAKE + 2), dict(s0=FAKE + 2), dict(sf=FAKE + 1),
                                  dict(cu=FAKE), dict(cu=FAKE, nseq=2, B=2), dict(cu=FAKE + 2, nseq=2), dict(nseq=3),
                                  dict(dt=1, g=FAKE + 1)])
def test_scan_fwd_refusals(lib, over):
    assert call(lib.gdn_gated_scan_fwd, SCAN, over) == 1


@pytest.mark.parametrize("over", [dict(B=0), dict(D=-4), dict(dt=-1), dict(x=None, gate=1), dict(g=None),
                                  dict(out=None), dict(dout=None), dict(dx=None), dict(dg=None), dict(di=FAKE + 2),
                                  dict(df=FAKE + 2), dict(dout=FAKE + 2), dict(nseq=2)])
def test_scan_bwd_refusals(lib, over):
    assert call(lib.gdn_gated_scan_bwd, SCAN_BWD, over) == 1


@pytest.mark.parametrize("over", [dict(N=-1), dict(D=0), dict(dt=2), dict(s=None), dict(x=None), dict(g=None),
                                  dict(out=None), dict(s=FAKE + 2), dict(out=FAKE + 2)])
def test_step_refusals(lib, over):
    assert call(lib.gdn_gated_scan_step, STEP, over) == 1


@pytest.mark.parametrize("over", [dict(rows=-1), dict(D=0), dict(dt=5), dict(x=None), dict(out=None), dict(eps=-1.0),
                                  dict(eps=float("nan")), dict(x=FAKE + 2), dict(w=FAKE + 2), dict(mean=FAKE + 1),
                                  dict(rows=1 << 46)])
def test_norm_fwd_refusals(lib, over):
    assert call(lib.gdn_layer_norm_fwd, NORM, over) == 1


@pytest.mark.parametrize("over,code", [(dict(rows=-1), 1), (dict(D=0), 1), (dict(dt=5), 1), (dict(dout=None), 1),
                                       (dict(x=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
                                       (dict(dx=FAKE + 2), 1), (dict(dw=FAKE + 2), 1), (dict(ws=None), 3),
                                       (dict(ws=FAKE + 8), 3), (dict(wsb=16), 3)])
def test_norm_bwd_refusals(lib, over, code):
    assert call(lib.gdn_layer_norm_bwd, NORM_BWD, over) == code


@pytest.mark.parametrize("over,code", [(dict(N=-1), 1), (dict(D=0), 1), (dict(V=0), 1), (dict(dt=3), 1),
                                       (dict(h=None), 1), (dict(w=None), 1), (dict(t=None), 1), (dict(loss=None), 1),
                                       (dict(h=FAKE + 8), 1), (dict(w=FAKE + 4), 1), (dict(t=FAKE + 2), 1),
                                       (dict(lse=FAKE + 2), 1), (dict(ws=None), 3), (dict(ws=FAKE + 128), 3),
                                       (dict(wsb=100), 3), (dict(N=(1 << 23) + 1), 2), (dict(V=(1 << 30) + 1), 2),
                                       (dict(N=1 << 23, V=(1 << 22) + 1), 2)])
def test_ce_fwd_refusals(lib, over, code):
    assert call(lib.gdn_linear_cross_entropy_fwd, CE, over) == code


@pytest.mark.parametrize("over,code", [(dict(N=-1), 1), (dict(D=0), 1), (dict(V=0), 1), (dict(dt=3), 1),
                                       (dict(h=None), 1), (dict(w=None), 1), (dict(t=None), 1), (dict(lse=None), 1),
                                       (dict(dl=None), 1), (dict(dh=FAKE + 8), 1), (dict(dw=FAKE + 8), 1),
                                       (dict(ws=None), 3), (dict(wsb=100), 3), (dict(N=(1 << 23) + 1), 2),
                                       (dict(V=(1 << 30) + 1), 2)])
def test_ce_bwd_refusals(lib, over, code):
    assert call(lib.gdn_linear_cross_entropy_bwd, CE_BWD, over) == code


def test_nothing_to_do_is_no_error(lib):
    assert call(lib.gdn_gated_scan_fwd, SCAN, dict(T=0)) == 0
    assert call(lib.gdn_gated_scan_step, STEP, dict(N=0)) == 0
    assert call(lib.gdn_layer_norm_fwd, NORM, dict(rows=0)) == 0
    assert call(lib.gdn_linear_cross_entropy_fwd, CE, dict(N=0)) == 0
    assert call(lib.gdn_linear_cross_entropy_bwd, CE_BWD, dict(dh=None, dw=None)) == 0


def test_workspace_sizes(lib):
    assert gdn.layer_norm_bwd_workspace_size(100, 64) > 0 and gdn.layer_norm_bwd_workspace_size(-1, 64) == 0
    size = gdn.linear_cross_entropy_workspace_size
    assert size(8192, 2048, 65536) > 256 and size(8192, 0, 65536) == 0 and size(-1, 8, 8, backward=True) == 0
    # never as large as the logits would be
    assert size(8192, 2048, 65536, backward=True) < 8192 * 65536 * 4 // 4
    assert size(8192, 2048, 65536) < 8192 * 65536 * 4 // 16


def test_wrappers_check_before_any_launch(lib):
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_scan_fwd(x, x)
    with pytest.raises(TypeError, match="dtype"):
        gdn.gated_scan_fwd(x, x.bfloat16())
    with pytest.raises(TypeError, match="cu_seqlens"):
        gdn.gated_scan_fwd(x[:1], x[:1], cu_seqlens=torch.tensor([0, 3]))
    with pytest.raises(ValueError, match="states"):
        gdn.gated_scan_fwd(x, x, init_state=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="input gate"):
        gdn.gated_scan_bwd(None, x, x, x, input_gate=True)
    with pytest.raises(ValueError, match="shape"):
        gdn.gated_scan_bwd(None, x, x, x[:, :2])
    with pytest.raises(TypeError, match="state"):
        gdn.gated_scan_step(x[0].double(), x[0], x[0])
    with pytest.raises(ValueError, match=r"\[N,D\]"):
        gdn.gated_scan_step(x[0], x[0], x[0, :2])
    with pytest.raises(TypeError, match="float32"):
        gdn.layer_norm_fwd(x, torch.ones(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=r"\[D\]"):
        gdn.layer_norm_fwd(x, torch.ones(7))
    with pytest.raises(ValueError, match="row"):
        gdn.layer_norm_bwd(x, x, torch.zeros(5), torch.zeros(6))
    with pytest.raises(TypeError, match="int32"):
        gdn.linear_cross_entropy_fwd(x[0], x[0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match=r"\[V,D\]"):
        gdn.linear_cross_entropy_fwd(x[0], torch.zeros(4, 9), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="dtype"):
        gdn.linear_cross_entropy_fwd(x[0], x[0].bfloat16(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous|CUDA"):
        gdn.layer_norm_fwd(x.transpose(0, 1))


def test_references_against_autograd():
    """The 64-bit backward forms are the gradients of the 64-bit forward forms."""
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    for gate in (False, True):
        x, g, s = r(1, 9, 4).requires_grad_(), (-r(1, 9, 4).abs()).requires_grad_(), r(3, 4).requires_grad_()
        cu, dout, df = [0, 4, 4, 9], r(1, 9, 4), r(3, 4)
        outs, fins = [], []
        for n in range(3):
            h = s[n]
            for t in range(cu[n], cu[n + 1]):
                a = g[0, t].exp()
                h = a * h + ((1 - a) if gate else 1.0) * x[0, t]
                outs.append(h)
            fins.append(h)
        out, fin = torch.stack(outs)[None], torch.stack(fins)
        ro, rf, _, _ = ref.scan_fwd(x, g, s, cu, gate)
        assert torch.allclose(ro, out) and torch.allclose(rf, fin)
        want = torch.autograd.grad((out * dout).sum() + (fin * df).sum(), (x, g, s))
        got, _ = ref.scan_bwd(x, g, out, dout, s, df, cu, gate)
        assert all(torch.allclose(p, q) for p, q in zip(got, want))
    x, w, b, dy = r(5, 12).requires_grad_(), r(12).requires_grad_(), r(12).requires_grad_(), r(5, 12)
    y = torch.nn.functional.layer_norm(x, (12,), w, b, 1e-5)
    (ry, m, rs), _ = ref.norm_fwd(x, w, b, 1e-5)
    assert torch.allclose(ry, y)
    want = torch.autograd.grad((y * dy).sum(), (x, w, b))
    got, _ = ref.norm_bwd(dy, x, m, rs, w)
    assert all(torch.allclose(p, q) for p, q in zip(got, want))
    h, w, t, dl = r(7, 6).requires_grad_(), r(11, 6).requires_grad_(), torch.tensor([0, 10, -1, 3, 11, 5, 5]), r(7)
    keep = (t >= 0) & (t < 11)
    loss = torch.nn.functional.cross_entropy(h @ w.T, torch.where(keep, t, -100), reduction="none")
    (rl, lse), _ = ref.ce_fwd(h, w, t)
    assert torch.allclose(rl, loss)
    want = torch.autograd.grad((loss * dl).sum(), (h, w))
    got, _ = ref.ce_bwd(h, w, t, lse, dl, False)
    assert all(torch.allclose(p, q) for p, q in zip(got, want))
