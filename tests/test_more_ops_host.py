"""Refusals of the root-mean-square norm, the 8-bit quantising, the product of 8-bit operands and the token log
probabilities; no GPU is needed (the pointers below are never dereferenced: validation fails first)."""
import pytest
import torch

import gated_delta_rule_12_gb300 as gdn
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


RMS = dict(x=FAKE, res=FAKE, w=FAKE, out=FAKE, sum=2 * FAKE, rstd=FAKE, rows=4, D=16, dt=0, eps=1e-5, stream=None)
RMS8 = dict(x=FAKE, res=FAKE, w=FAKE, q=FAKE, c=FAKE, sum=2 * FAKE, rows=4, D=16, dt=0, eps=1e-5, stream=None)
RMS_BWD = dict(dout=FAKE, x=FAKE, rstd=FAKE, w=FAKE, dres=FAKE, dx=FAKE, dw=FAKE, rows=4, D=16, dt=0, ws=FAKE,
               wsb=1 << 40, stream=None)
QUANT = dict(x=FAKE, q=FAKE, c=FAKE, rows=4, D=16, br=1, dt=0, stream=None)
LINEAR = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, out=FAKE, M=4, N=16, K=32, work=FAKE, size=1 << 40, stream=None)
LOGP = dict(h=FAKE, w=FAKE, t=FAKE, logp=FAKE, ent=FAKE, lse=FAKE, ids=FAKE, top=FAKE, N=4, D=16, V=32, k=3, dt=0,
            work=FAKE, size=1 << 40, stream=None)
LOGP_BWD = dict(h=FAKE, w=FAKE, t=FAKE, lse=FAKE, ent=FAKE, da=FAKE, db=FAKE, dh=FAKE, dw=FAKE, N=4, D=16, V=32, dt=0,
                work=FAKE, size=1 << 40, stream=None)


@pytest.mark.parametrize("over", [dict(rows=-1), dict(D=0), dict(dt=5), dict(x=None), dict(out=None), dict(eps=-1.0),
                                  dict(eps=float("nan")), dict(x=FAKE + 2), dict(w=FAKE + 2), dict(rstd=FAKE + 1),
                                  dict(rows=1 << 46), dict(res=None), dict(sum=None), dict(res=FAKE + 2),
                                  dict(sum=FAKE + 2), dict(sum=FAKE), dict(dt=1, x=FAKE + 1)])
def test_rms_fwd_refusals(lib, over):
    assert call(lib.gdn_rms_norm_fwd, RMS, over) == 1


@pytest.mark.parametrize("over", [dict(rows=-1), dict(D=0), dict(dt=-1), dict(x=None), dict(q=None), dict(c=None),
                                  dict(c=FAKE + 2), dict(res=None), dict(sum=None), dict(eps=-0.5), dict(x=FAKE + 2)])
def test_rms_fp8_refusals(lib, over):
    assert call(lib.gdn_rms_norm_fp8, RMS8, over) == 1


@pytest.mark.parametrize("over,code", [(dict(rows=-1), 1), (dict(D=0), 1), (dict(dt=5), 1), (dict(dout=None), 1),
                                       (dict(x=None), 1), (dict(rstd=None), 1), (dict(dx=FAKE + 2), 1),
                                       (dict(dw=FAKE + 2), 1), (dict(dres=FAKE + 2), 1), (dict(rows=1 << 46), 1),
                                       (dict(ws=None), 3), (dict(ws=FAKE + 8), 3), (dict(wsb=16), 3)])
def test_rms_bwd_refusals(lib, over, code):
    assert call(lib.gdn_rms_norm_bwd, RMS_BWD, over) == code


@pytest.mark.parametrize("over,code", [(dict(rows=-1), 1), (dict(D=0), 1), (dict(dt=3), 1), (dict(br=64), 1),
                                       (dict(br=0), 1), (dict(x=None), 1), (dict(q=None), 1), (dict(c=None), 1),
                                       (dict(x=FAKE + 2), 1), (dict(c=FAKE + 1), 1), (dict(rows=1 << 46), 1),
                                       (dict(br=128, rows=1 << 40, D=8), 2)])
def test_quantize_refusals(lib, over, code):
    assert call(lib.gdn_fp8_quantize, QUANT, over) == code


@pytest.mark.parametrize("over,code", [(dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(x=None), 1),
                                       (dict(xs=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(out=None), 1),
                                       (dict(xs=FAKE + 2), 1), (dict(ws=FAKE + 1), 1), (dict(out=FAKE + 1), 1),
                                       (dict(work=None), 3), (dict(work=FAKE + 16), 3), (dict(size=100), 3),
                                       (dict(M=(1 << 23) + 1), 2), (dict(N=(1 << 23) + 1), 2), (dict(K=(1 << 20) + 1), 2),
                                       (dict(M=1 << 22, N=1 << 21), 2)])
def test_linear_refusals(lib, over, code):
    assert call(lib.gdn_fp8_linear, LINEAR, over) == code


@pytest.mark.parametrize("over,code", [(dict(N=-1), 1), (dict(D=0), 1), (dict(V=0, k=0), 1), (dict(dt=3), 1), (dict(k=-1), 1),
                                       (dict(k=21), 1), (dict(V=2), 1), (dict(h=None), 1), (dict(w=None), 1),
                                       (dict(t=None), 1), (dict(logp=None), 1), (dict(ent=None), 1), (dict(ids=None), 1),
                                       (dict(top=None), 1), (dict(ids=FAKE + 2), 1), (dict(ent=FAKE + 1), 1),
                                       (dict(h=FAKE + 8), 1), (dict(work=None), 3), (dict(work=FAKE + 64), 3),
                                       (dict(size=256), 3), (dict(N=(1 << 23) + 1), 2), (dict(V=(1 << 30) + 1), 2)])
def test_log_probs_fwd_refusals(lib, over, code):
    assert call(lib.gdn_linear_log_probs_fwd, LOGP, over) == code


@pytest.mark.parametrize("over,code", [(dict(N=-1), 1), (dict(dt=3), 1), (dict(h=None), 1), (dict(w=None), 1),
                                       (dict(t=None), 1), (dict(lse=None), 1), (dict(da=None), 1), (dict(ent=None), 1),
                                       (dict(db=FAKE + 2), 1), (dict(ent=FAKE + 2), 1), (dict(dh=FAKE + 8), 1),
                                       (dict(dw=FAKE + 8), 1), (dict(work=None), 3), (dict(size=256), 3),
                                       (dict(V=(1 << 30) + 1), 2)])
def test_log_probs_bwd_refusals(lib, over, code):
    assert call(lib.gdn_linear_log_probs_bwd, LOGP_BWD, over) == code


def test_nothing_to_do(lib):
    """No rows: nothing is enqueued, and no pointer to rows is needed."""
    assert call(lib.gdn_rms_norm_fwd, RMS, dict(rows=0, x=None, out=None, res=None, sum=None)) == 0
    assert call(lib.gdn_rms_norm_fp8, RMS8, dict(rows=0, x=None, q=None, c=None)) == 0
    assert call(lib.gdn_rms_norm_bwd, RMS_BWD, dict(dx=None, dw=None)) == 0
    assert call(lib.gdn_fp8_quantize, QUANT, dict(rows=0, x=None, q=None, c=None)) == 0
    assert call(lib.gdn_fp8_linear, LINEAR, dict(M=0, x=None, xs=None, out=None)) == 0
    assert call(lib.gdn_linear_log_probs_fwd, LOGP, dict(N=0, h=None, t=None, logp=None, ent=None, ids=None, top=None)) == 0
    assert call(lib.gdn_linear_log_probs_bwd, LOGP_BWD, dict(dh=None, dw=None)) == 0


def test_workspace_sizes(lib):
    assert gdn.rms_norm_bwd_workspace_size(8, 1 << 32) == 0 and gdn.rms_norm_bwd_workspace_size(-1, 8) == 0
    assert gdn.rms_norm_bwd_workspace_size(8, 512) >= 512 * 4
    assert gdn.fp8_linear_workspace_size(1 << 32, 8, 8) == 0 and gdn.fp8_linear_workspace_size(8, 8, 0) == 0
    assert gdn.fp8_linear_workspace_size(0, 8, 8) >= 256
    size = gdn.linear_log_probs_workspace_size
    assert size(4, 8, 4, 5) == 0 and size(4, 8, 40, 21) == 0 and size(4, 8, 40, -1) == 0 and size(1 << 33, 8, 40) == 0
    assert 0 < size(4, 8, 40) < size(4, 8, 40, 5) < size(4, 8, 40, 20)


def test_python_refusals(lib):
    x, w = torch.zeros(4, 128), torch.ones(128)
    e = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    c, cw = torch.ones(4, 1), torch.ones(1, 1)
    h, t, z = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    wrong = [
        (ValueError, lambda: gdn.linear_log_probs_fwd(h, h, t, top_k=5)),
        (ValueError, lambda: gdn.linear_log_probs_fwd(h, h, t[:3])),
        (TypeError, lambda: gdn.linear_log_probs_fwd(h, h, t.long())),
        (TypeError, lambda: gdn.linear_log_probs_fwd(h, h.bfloat16(), t)),
        (ValueError, lambda: gdn.linear_log_probs_fwd(h, h, t)),
        (ValueError, lambda: gdn.linear_log_probs_bwd(h, h, t, z, None, z, z)),
        (TypeError, lambda: gdn.linear_log_probs_bwd(h, h, t, z, z, z.double())),
        (ValueError, lambda: gdn.linear_log_probs_bwd(h, h, t, z, z, z, z[:2])),
        (ValueError, lambda: gdn.rms_norm_fwd(x, w)),                                    # not on the GPU
        (ValueError, lambda: gdn.rms_norm_fwd(torch.zeros(()), None)),
        (ValueError, lambda: gdn.rms_norm_fwd(x, w[:100])),
        (TypeError, lambda: gdn.rms_norm_fwd(x, w.double())),
        (ValueError, lambda: gdn.rms_norm_fwd(x, w, residual=x[:2])),
        (TypeError, lambda: gdn.rms_norm_fwd(x, w, residual=x.bfloat16())),
        (ValueError, lambda: gdn.rms_norm_fwd(x, w, residual_out=x)),                    # without a residual
        (ValueError, lambda: gdn.rms_norm_fp8(x, w, residual_out=x)),
        (ValueError, lambda: gdn.rms_norm_bwd(x, x, torch.ones(3), w)),
        (TypeError, lambda: gdn.rms_norm_bwd(x.half(), x, torch.ones(4), w)),
        (ValueError, lambda: gdn.rms_norm_bwd(x, x, torch.ones(4), w, dresidual=x[0])),
        (ValueError, lambda: gdn.fp8_quantize(x, block_rows=64)),
        (ValueError, lambda: gdn.fp8_quantize(x.view(2, 2, 128), block_rows=128)),
        (TypeError, lambda: gdn.fp8_quantize(x.half())),
        (ValueError, lambda: gdn.fp8_quantize(x)),
        (TypeError, lambda: gdn.fp8_linear(x, c, e, cw)),
        (TypeError, lambda: gdn.fp8_linear(e, c.double(), e, cw)),
        (ValueError, lambda: gdn.fp8_linear(e, c[:2], e, cw)),
        (ValueError, lambda: gdn.fp8_linear(e, c, e, c)),
        (ValueError, lambda: gdn.fp8_linear(e, c, e.view(8, 64), cw)),
        (TypeError, lambda: gdn.fp8_linear(e, c, e, cw, out=torch.zeros(4, 4))),
        (ValueError, lambda: gdn.fp8_linear(e, c, e, cw, out=torch.zeros(4, 5, dtype=torch.bfloat16))),
        (ValueError, lambda: gdn.fp8_linear(e, c, e, cw)),
    ]
    for kind, f in wrong:
        with pytest.raises(kind):
            f()
