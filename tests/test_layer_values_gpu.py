"""Activations and their slopes value by value, against 64 bits and the header's bounds."""
import math

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


def same(got, *wants):
    """Each element one of the wanted ones: NaN where that is NaN, the same signed infinity, the same number (of rounded
    values)."""
    ok = torch.zeros(got.shape, dtype=torch.bool, device=got.device)
    for w in wants:
        w = w.to(got.dtype).expand_as(got)
        ok |= (got == w) | (torch.isnan(got) & torch.isnan(w))
    return bool(ok.all())


def formula(name, v):
    """Value and slope as the header's formulas give them in fp32, and their limits."""
    e, r2 = torch.exp(-v), 2.0 ** -0.5
    inner = (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    t = torch.tanh(inner)
    s = 1 / (1 + e)
    value = {"none": v, "relu": torch.where(v < 0, torch.zeros_like(v), v), "gelu": v * (1 + torch.erf(v * r2)) / 2,
             "gelu_tanh": v * (1 + t) / 2, "silu": v / (1 + e)}[name]
    one = torch.ones_like(v)
    sl = {"none": one, "relu": torch.where(v <= 0, torch.zeros_like(v), one),
          "gelu": (1 + torch.erf(v * r2)) / 2 + v * torch.exp(-v * v / 2) / (2 * math.pi) ** 0.5,
          "gelu_tanh": (1 + t) / 2 + v * (1 - t * t) / 2 * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * v * v),
          "silu": s * (1 + v * (1 - s))}[name]
    inf = torch.isinf(v)
    limit = v if name == "none" else torch.where(inf, v.clamp(min=0.0), value)
    return value, limit, sl, sl if name == "none" else torch.where(inf, (v > 0).float(), sl)


INF = float("inf")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dt,cols", [(torch.float32, 16), (torch.bfloat16, 16), (torch.float16, 333)])
def test_infinities_and_nan(name, dt, cols):
    """v and z of both infinities and NaN: the formula's value in fp32 or its limit, alone and behind a product."""
    v = torch.tensor([INF, -INF, float("nan"), 2.0], device="cuda").repeat(84)[:cols].expand(5, cols).contiguous().to(dt)
    value, limit, sl, slim = formula(name, v.float())
    finite = torch.isfinite(v)
    y, d = binding.activation(v, activation=name), binding.activation_bwd(torch.ones_like(v), v, activation=name)
    assert same(y[~finite], value[~finite], limit[~finite]), y[0, :4]
    # (relu's slope at NaN: the comparison with 0 fails, so dy.)
    assert same(d[~finite], sl[~finite], slim[~finite]), d[0, :4]
    assert bool(torch.isfinite(y[finite]).all()) and bool(torch.isfinite(d[finite]).all())
    if dt == torch.float32:
        return
    # The same as pre-activations of a product: x w' is 0, the bias brings v; and as z of an input gradient of ones.
    for rows in (5, 300):  # few rows, tiles
        zeros, w = torch.zeros(rows, 64, dtype=dt, device="cuda"), torch.ones(cols, 64, dtype=dt, device="cuda")
        y, z = binding.linear(zeros, w, v[0].contiguous(), activation=name, keep_z=True)
        assert same(z, v[0])
        assert same(y[:, ~finite[0]], value[0][~finite[0]], limit[0][~finite[0]]), y[0, :4]
        assert bool(torch.isfinite(y[:, finite[0]]).all())
        dy = torch.zeros(rows, 64, dtype=dt, device="cuda")
        dy[:, 0] = 1
        d = binding.linear_bwd_data(dy, torch.ones(64, cols, dtype=dt, device="cuda"), v[:1].expand(rows, cols).contiguous(), activation=name)
        assert same(d[:, ~finite[0]], sl[0][~finite[0]], slim[0][~finite[0]]), d[0, :4]
        assert bool(torch.isfinite(d[:, finite[0]]).all())


@pytest.mark.parametrize("tokens,inf,out", [(3, 72, 264), (20, 2048, 40), (300, 264, 333), (300, 65, 72)])
def test_infinities_of_products(tokens, inf, out):
    """Infinite and NaN operands give each result what 64-bit sums give it: signed infinities, NaN where both meet."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randint(1, 4, s, generator=g, device="cuda").to(torch.bfloat16) for s in ((tokens, inf), (out, inf)))
    x[0, 3], x[1, 5], x[2, 1], x[2, inf - 1] = INF, -INF, INF, -INF
    w[0] = -w[0]
    w[1, 3], w[2, inf - 1], w[3, 0] = 0, INF, float("nan")
    want = x.double() @ w.double().T
    for y in (binding.linear(x, w), binding.linear_bwd_data(x, w.t().contiguous()), binding.linear_bwd_weight(w.t().contiguous(), x.t().contiguous())):
        odd = ~torch.isfinite(want)
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y[odd & ~torch.isnan(want)].double(), want[odd & ~torch.isnan(want)])
        assert bool(torch.isfinite(y[~odd]).all())
