"""The new calls' refusals that need no GPU: MuonSR's arguments, and the C
entry points' checks before any CUDA call."""
import ctypes

import pytest
import torch

from stochastic_rounding_gb300 import MuonSR, _lib


@pytest.fixture(scope="module")
def L():
    from stochastic_rounding_gb300 import build
    build.build()
    return _lib.lib()


def _param(*shape):
    return torch.nn.Parameter(torch.zeros(*shape))


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(weight_decay=-1.0), dict(momentum=1.0), dict(eps=0.0),
                                dict(ns_steps=0), dict(ns_coefficients=(1.0, 2.0)), dict(adjust_lr_fn="other"),
                                dict(rounding="up"), dict(seed=-1), dict(base_offset=2**64), dict(check_errors="no")])
def test_muonsr_arguments(kw):
    with pytest.raises(ValueError):
        MuonSR([_param(4, 4)], **kw)


def test_muonsr_takes_matrices_on_cuda():
    with pytest.raises(ValueError):
        MuonSR([_param(4)])
    opt = MuonSR([_param(4, 4)])
    opt.step()                                   # nothing has a gradient
    opt.param_groups[0]["params"][0].grad = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        opt.step()


P = ctypes.c_void_p(4096)


def _ns(**kw):
    d = dict(a=3.4445, b=-4.775, c=2.0315, eps=1e-7, steps=5)
    d.update(kw)
    return _lib.NsParams(d["a"], d["b"], d["c"], d["eps"], d["steps"], 0)


def _matrix(**kw):
    d = dict(x=4096, out=8192, count=1, rows=8, cols=16, x_ld=16, x_stride=128, out_ld=16, out_stride=128, x_dtype=1,
             reserved=0)
    d.update(kw)
    return (_lib.MatrixDesc * 1)(_lib.MatrixDesc(*d.values()))


def test_newton_schulz_checks(L):
    need = ctypes.c_uint64(7)
    assert L.asr_newton_schulz_workspace(_matrix(), 1, ctypes.byref(need)) == _lib.ASR_OK and need.value > 0
    call = lambda t, ns, ws=P, size=need.value: L.asr_newton_schulz(t, 1, ctypes.byref(ns), ws, size, None)  # noqa: E731
    for bad in (dict(rows=2**21), dict(x_ld=15), dict(out_ld=8), dict(x=None), dict(out=None), dict(x=4097),
                dict(out=8193), dict(count=2**25)):
        assert call(_matrix(**bad), _ns()) == _lib.ASR_ERR_INVALID_VALUE, bad
    assert call(_matrix(x_dtype=5), _ns()) == _lib.ASR_ERR_UNSUPPORTED_DTYPE
    for bad in (dict(steps=0), dict(steps=101), dict(eps=0.0), dict(eps=float("nan")), dict(a=9.0), dict(c=float("inf")),
                dict(a=2.0, b=2.0, c=2.0)):
        assert call(_matrix(), _ns(**bad)) == _lib.ASR_ERR_INVALID_VALUE, bad
    assert call(_matrix(), _ns(), None) == _lib.ASR_ERR_INVALID_VALUE
    assert call(_matrix(), _ns(), ctypes.c_void_p(4097)) == _lib.ASR_ERR_INVALID_VALUE
    assert call(_matrix(), _ns(), P, need.value - 1) == _lib.ASR_ERR_INVALID_VALUE
    assert L.asr_newton_schulz(None, 1, ctypes.byref(_ns()), P, 1 << 30, None) == _lib.ASR_ERR_INVALID_VALUE
    assert L.asr_newton_schulz(_matrix(), 1, None, P, 1 << 30, None) == _lib.ASR_ERR_INVALID_VALUE
    for empty in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert call(_matrix(**empty), _ns(), None, 0) == _lib.ASR_OK


def test_muon_checks(L):
    def desc(**kw):
        d = dict(param=4096, grad=8192, momentum=12288, count=1, rows=8, cols=16, base=0, pdt=1, gdt=1)
        d.update(kw)
        return (_lib.MuonDesc * 1)(_lib.MuonDesc(*d.values()))

    def hp(**kw):
        d = dict(lr=0.1, momentum=0.9, wd=0.1, ns=_ns(), nesterov=1, adjust=1, step=1, rounding=0, seed=0)
        d.update(kw)
        return _lib.MuonHparams(*d.values())
    call = lambda t, h: L.asr_muon_sr_multi_tensor(t, 1, ctypes.byref(h), P, 1 << 30, None)  # noqa: E731
    for bad in (dict(param=None), dict(momentum=12289), dict(base=2**64 - 5), dict(grad=8193), dict(rows=2**21)):
        assert call(desc(**bad), hp()) == _lib.ASR_ERR_INVALID_VALUE, bad
    for bad in (dict(pdt=2), dict(gdt=-1)):
        assert call(desc(**bad), hp()) == _lib.ASR_ERR_UNSUPPORTED_DTYPE, bad
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(momentum=1.0), dict(wd=-0.1), dict(step=0), dict(adjust=3),
                dict(nesterov=2), dict(ns=_ns(steps=0))):
        assert call(desc(), hp(**bad)) == _lib.ASR_ERR_INVALID_VALUE, bad
    assert call(desc(), hp(rounding=9)) == _lib.ASR_ERR_UNSUPPORTED_DTYPE
    assert L.asr_muon_sr_multi_tensor(desc(), 1, None, P, 1 << 30, None) == _lib.ASR_ERR_INVALID_VALUE


def test_int8_checks(L):
    bad, dt, ok = _lib.ASR_ERR_INVALID_VALUE, _lib.ASR_ERR_UNSUPPORTED_DTYPE, _lib.ASR_OK
    q = L.asr_quantize_int8
    assert q(P, 1, 8, 8, 7, 0, P, 8, P, 1, 0, 1, 0, None) == bad          # pitch below the columns
    assert q(P, 1, 8, 16, 16, 1, P, 7, P, 1, 0, 1, 0, None) == bad        # transposed: pitch below the rows
    assert q(None, 1, 8, 8, 8, 0, P, 8, P, 1, 0, 1, 0, None) == bad
    assert q(P, 1, 8, 8, 8, 2, P, 8, P, 1, 0, 1, 0, None) == bad
    assert q(P, 2, 8, 8, 8, 0, P, 8, P, 1, 0, 1, 0, None) == dt
    assert q(P, 1, 8, 8, 8, 0, P, 8, P, 3, 0, 1, 0, None) == dt
    assert q(P, 1, 8, 8, 8, 0, P, 8, P, 1, 2**64 - 3, 1, 0, None) == bad
    assert q(None, 1, 0, 8, 8, 0, None, 8, None, 1, 0, 1, 0, None) == ok
    g = L.asr_gemm_int8_sr
    args = dict(a=P, lda=32, b=P, ldb=32, sa=P, sb=P, c=P, ldc=8, cdt=1, m=40, n=8, k=32, r=1, step=0, seed=0, ws=P,
                size=1 << 30, stream=None)
    for kw in (dict(a=None), dict(sb=None), dict(lda=31), dict(ldc=7), dict(k=0), dict(k=131072), dict(m=2**25),
               dict(ws=None), dict(size=0), dict(c=ctypes.c_void_p(4097))):
        assert g(*{**args, **kw}.values()) == bad, kw
    assert g(*{**args, "cdt": 7}.values()) == dt and g(*{**args, "r": 7}.values()) == dt
    assert g(*{**args, "m": 0}.values()) == ok
    lin = L.asr_linear_int8
    args = dict(x=P, xdt=1, x_ld=32, w=P, ldw=32, sw=P, y=P, ldy=8, ydt=1, m=40, n=8, k=32, r=1, step=0, seed=0, ws=P,
                size=1 << 30, stream=None)
    for kw in (dict(x=None), dict(sw=None), dict(x_ld=31), dict(ldy=7), dict(k=0), dict(ws=None), dict(size=0)):
        assert lin(*{**args, **kw}.values()) == bad, kw
    assert lin(*{**args, "xdt": 9}.values()) == dt
    gr = L.asr_linear_int8_grads
    args = dict(dy=P, ddt=1, dld=8, x=P, xdt=1, xld=32, w=P, wdt=1, wld=32, dx=P, dxld=32, dw=P, dwld=32, t=4, n=8, k=32,
                step=0, seed=0, ws=P, size=1 << 30, stream=None)
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(dld=7), dict(dxld=31), dict(t=0), dict(n=131072),
               dict(ws=None), dict(size=0)):
        assert gr(*{**args, **kw}.values()) == bad, kw
    assert gr(*{**args, "wdt": 9}.values()) == dt
    assert gr(*{**args, "dx": None, "dw": None}.values()) == ok
