"""The norm, the activation, 8-bit checkpoints and the embedding at the ends of what they take, and where every result
is exact: sums of whole numbers, activations far from zero."""
import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asr():
    torch_cuda()
    from stochastic_rounding_gb300 import build
    build.build()
    import stochastic_rounding_gb300 as m
    yield m
    assert m.asr_take_device_error() == 0


@pytest.mark.parametrize("cols", [2 ** 23 + 32, 2 ** 23 + 17, 2 ** 24])
@pytest.mark.parametrize("rounding", ["rne", "sr"])
def test_a_gated_input_of_any_width_is_kept(asr, cols, rounding):
    """Both halves together are wider than either: 2^25 columns where the output has 2^24.  Codes are those of the
    input's parts, which end with whole groups, and a backward pass from them is that from the values they stand for."""
    import torch
    g = torch.Generator("cuda").manual_seed(cols)
    x = torch.randn(1, 2 * cols, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(1, cols, device="cuda", generator=g).to(torch.bfloat16)
    y, kept = asr.activation(x, gated=True, save="int8", rounding=rounding, step=3, seed=5)
    assert torch.equal(y, asr.activation(x, gated=True))
    n = 2 ** 23
    for at in range(0, 2 * cols, n):
        part = asr.checkpoint_int8(x[:, at:at + n], rounding=rounding, base_index=at, step=3, seed=5)
        assert torch.equal(kept.q[:, at:at + n], part.q)
        assert torch.equal(kept.power[:, at // 32:(at + n) // 32], part.power)
    back = asr.restore_int8(kept)
    assert torch.equal(asr.activation_grads(dy, kept, gated=True), asr.activation_grads(dy, back, gated=True))
