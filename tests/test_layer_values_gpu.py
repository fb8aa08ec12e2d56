"""Activations and their slopes value by value, against 64 bits and the header's bounds."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import act, slope  # noqa: E402

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def grid(part):
    """fp32 values: every one in [4, 8) (where exp(-v) and the tails meet fp32's last place), steps of 2^-18 up to 32, and
    every 2^10th from the smallest normal number to 4, of both signs."""
    i = torch.arange(1 << 23, device="cuda")
    if part == "dense":
        v = 4 + i.double() * 2.0 ** -21
    elif part == "wide":
        v = i.double() * 2.0 ** -18
    else:
        v = (0x0080_0000 + torch.arange((0x4080_0000 - 0x0080_0000) >> 10, device="cuda") * 1024).to(torch.int32).view(torch.float32).double()
    return torch.cat([v, -v]).float().view(1, -1)


@pytest.mark.parametrize("part", ["dense", "wide", "small"])
@pytest.mark.parametrize("name", ACTS[1:])
def test_values_and_slopes_are_as_near_as_stated(name, part):
    """A value within 2^-20 (|v| + 1), a slope within 2^-19, and the result's own rounding (2^-24 of it)."""
    v = grid(part).view(-1, 1 << 10)
    d = v.double()
    want = act(name, d)
    far = (binding.activation(v, activation=name).double() - want).abs() - 2.0 ** -24 * want.abs() - 2.0 ** -20 * (d.abs() + 1)
    assert float(far.max()) <= 0, (float(far.max()), float(v.flatten()[far.argmax()]))
    want = slope(name, d)
    far = (binding.activation_bwd(torch.ones_like(v), v, activation=name).double() - want).abs() - 2.0 ** -24 * want.abs() - 2.0 ** -19
    assert float(far.max()) <= 0, (float(far.max()), float(v.flatten()[far.argmax()]))
