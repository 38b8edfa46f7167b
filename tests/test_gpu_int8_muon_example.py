"""The example that trains a network on the 8-bit products with Muon and serves
it, and the optimizer's own behaviour."""
import copy
import os
import sys

import pytest

from gpu_util import assert_same_bits, host, torch_cuda

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


def test_example_trains_repeats_and_serves(asr):
    """The loss falls to less than half; a second run repeats it bit for bit;
    a token served alone gives the bits it gives in a batch (a row's product does
    not depend on the others: the integer sums are exact)."""
    import torch
    import int8_muon_mlp as ex
    losses, net = ex.train(steps=40)
    assert losses[-1] < 0.5 * losses[0]
    again, net2 = ex.train(steps=40)
    assert losses == again
    for p, q in zip(net.parameters(), net2.parameters()):
        assert_same_bits(host(p), host(q))
    for count in (3, 40, 150):
        x = torch.randn(count, 256, device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            assert torch.equal(ex.serve(net, x), net(x))


def test_muonsr_is_the_library_call_and_resumes(asr):
    import torch
    torch.manual_seed(0)
    shapes = [(64, 96), (96, 64), (3, 64, 96), (40, 40)]
    ps = [torch.nn.Parameter((torch.randn(s, device="cuda") * 0.02).to(torch.bfloat16)) for s in shapes]
    opt = asr.MuonSR([{"params": ps[:2]}, {"params": ps[2:], "lr": 0.05, "rounding": "rne"}], lr=0.02, seed=3,
                     base_offset=11)
    want = [(p.detach().clone(), torch.zeros_like(p, dtype=torch.float32)) for p in ps]
    base = [11]
    for p in ps:
        base.append(base[-1] + p.numel())

    def grads(step):
        g = torch.Generator(device="cuda")
        g.manual_seed(step)
        return [torch.randn(s, device="cuda", generator=g) * 1e-3 for s in shapes]
    saved = None
    for step in range(1, 4):
        gs = grads(step)
        for p, g in zip(ps, gs):
            p.grad = g.to(torch.bfloat16) if step == 2 else g.to(p.dtype)
        opt.step()
        for (p, m), q, b, i in zip(want, ps, base, range(4)):
            asr.asr_muon_sr_multi_tensor([(p, q.grad, m, b)], lr=0.02 if i < 2 else 0.05, weight_decay=0.1, step=step,
                                         seed=3, rounding="sr" if i < 2 else "rne")
            assert_same_bits(host(q), host(p))
            assert_same_bits(host(opt.state[q]["momentum_buffer"]), host(m))
        if step == 2:
            saved = copy.deepcopy(opt.state_dict()), [p.detach().clone() for p in ps]
    qs = [torch.nn.Parameter(p.clone()) for p in saved[1]]
    new = asr.MuonSR([{"params": qs[:2]}, {"params": qs[2:]}], base_offset=11)
    new.load_state_dict(saved[0])
    for q, g in zip(qs, grads(3)):
        q.grad = g.to(q.dtype)
    new.step(check_errors="deferred")
    new.poll_errors(wait=True)
    for p, q in zip(ps, qs):
        assert_same_bits(host(q), host(p))
