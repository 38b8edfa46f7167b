"""MuonSR: what it refuses leaves the model as it was (no GPU: the library's
step is replaced, its checks are not)."""
import pytest
import torch

from stochastic_rounding_gb300 import MuonSR, _lib


@pytest.fixture
def steps(monkeypatch):
    from stochastic_rounding_gb300 import build
    build.build()
    real, done = _lib.asr_muon_sr_multi_tensor, []

    def fake(entries, **kw):
        if entries:
            done.append((len(entries), kw["step"]))
        else:
            real(entries, **kw)                   # an empty table: the checks alone
    monkeypatch.setattr(_lib, "asr_muon_sr_multi_tensor", fake)
    monkeypatch.setattr(MuonSR, "_check", staticmethod(lambda p: None))
    return done


def _params(n):
    ps = [torch.nn.Parameter(torch.zeros(4, 6)) for _ in range(n)]
    for p in ps:
        p.grad = torch.ones(4, 6)
    return ps


@pytest.mark.parametrize("bad", [dict(ns_coefficients=(20.0, 0.0, 0.0)), dict(lr=float("nan")),
                                 dict(lr=float("inf")), dict(eps=1e-40), dict(weight_decay=float("nan")),
                                 dict(ns_coefficients=(float("nan"), 0.0, 0.0))])
def test_a_refused_group_stops_the_step_before_it_begins(steps, bad):
    ps = _params(2)
    opt = MuonSR([{"params": ps[:1]}, {"params": ps[1:]}], check_errors=False)
    opt.param_groups[1].update(bad)
    with pytest.raises(_lib.AsrError):
        opt.step()
    assert not steps and not opt.state
    opt.param_groups[1].update({k: opt.param_groups[0][k] for k in bad})
    opt.step()
    assert steps == [(1, 1), (1, 1)]


def test_a_group_without_gradients_is_not_checked(steps):
    ps = _params(2)
    opt = MuonSR([{"params": ps[:1]}, {"params": ps[1:]}], check_errors=False)
    opt.param_groups[1]["lr"] = float("nan")
    ps[1].grad = None
    opt.step()
    assert steps == [(1, 1)]


def test_later_groups_hold_matrices(steps):
    ps = _params(3)
    opt = MuonSR(ps[:1])
    for bad in (torch.zeros(4), torch.zeros(()), torch.zeros(2, 2, 2, 2)):
        with pytest.raises(ValueError):
            opt.add_param_group({"params": [ps[1], torch.nn.Parameter(bad)]})
        assert len(opt.param_groups) == 1
    opt.add_param_group({"params": (p for p in ps[1:])})
    assert [opt.base_index(p) for p in ps] == [0, 24, 48]
