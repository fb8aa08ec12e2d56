"""Activation with bias, dropout and residual alone, and its gradient, against the definition in 64 bits."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import DT, act, close, drop, slope  # noqa: E402

SEED, OFFSET = 0xFEDC_BA98_7654_3210, (1 << 40) + 3
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def randn(seed, *shape, size=1.0, dt="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(shape, generator=g, device="cuda")).to(DT[dt])


def value(name, v, p, residual, gain_error=2.0 ** -23):
    """y and its error before the last rounding: layer_oracle.py's."""
    a = act(name, v)
    err = 1.13 * 2.0 ** -24 * v.abs() + (2.0 ** -20 * (v.abs() + 1) if name != "none" else 0.0)
    a, gain = drop(a, p, SEED, OFFSET)
    err = err * gain + gain_error * a.abs()
    if residual is not None:
        a = a + residual.double()
        err = err + 2.0 ** -23 * a.abs()
    return a, err


@pytest.mark.parametrize("act_name", ACTS)
@pytest.mark.parametrize("rows,dim,dt,ydt", [(1, 1, "bf16", "bf16"), (3, 7, "fp32", "fp32"), (70, 64, "bf16", "bf16"),
                                             (257, 999, "fp16", "fp32"), (1030, 2056, "bf16", "fp16"), (5000, 130, "fp32", "bf16")])
def test_forward(rows, dim, dt, ydt, act_name):
    x, bias, res = randn(1, rows, dim, size=2, dt=dt), randn(2, dim), randn(3, rows, dim, dt=ydt)
    for b, r, p in ((bias, res, 0.3), (None, None, 0.0), (bias, None, 0.9), (None, res, 0.0)):
        y = torch.full((rows, dim), float("nan"), dtype=DT[ydt], device="cuda")
        binding.activation(x, b, r, act_name, p, SEED, OFFSET, out=y)
        want, err = value(act_name, x.double() + (0 if b is None else b.double()), p, r)
        close(y, want, err, ydt, (act_name, p))


@pytest.mark.parametrize("act_name", ACTS)
@pytest.mark.parametrize("rows,dim,dt,ydt", [(1, 1, "bf16", "bf16"), (3, 7, "fp32", "fp32"), (70, 64, "bf16", "bf16"),
                                             (257, 999, "fp16", "fp32"), (1030, 2056, "bf16", "fp16"), (20000, 24, "fp32", "bf16")])
def test_gradient(rows, dim, dt, ydt, act_name):
    x, bias, dy = randn(1, rows, dim, size=2, dt=dt), randn(2, dim), randn(3, rows, dim, dt=ydt)
    for b, p in ((bias, 0.3), (None, 0.0)):
        db = torch.full((dim,), float("nan"), device="cuda")
        dx = binding.activation_bwd(dy, x, b, act_name, p, SEED, OFFSET, dbias=db)
        v = x.double() + (0 if b is None else b.double())
        want = slope(act_name, v) * dy.double()
        # (A slope's slope is at most 1.6, and v is rounded to fp32.)
        err = (2.0 ** -19 + 1.6 * 2.0 ** -24 * v.abs()) * dy.double().abs() if act_name != "none" else torch.zeros_like(want)
        if act_name == "relu":
            err = torch.zeros_like(want)
        want, gain = drop(want, p, SEED, OFFSET)
        err = err * gain + 2.0 ** -23 * want.abs()
        close(dx, want, err, dt, (act_name, p))
        # dbias: fewer than 256 roundings of sums that are at most the sum of the terms' sizes.
        close(db, want.sum(0), err.sum(0) + 256 * 2.0 ** -24 * want.abs().sum(0), "fp32", "dbias")


def test_in_place_and_strides():
    for pad in (8, 3):
        buf, bias, res = randn(1, 90, 64 + pad, dt="bf16"), randn(2, 64, dt="bf16"), randn(3, 90, 64 + pad, dt="bf16")
        sp = {"tokens": 90, "dim": 64, "ld_x": 64 + pad, "ld_y": 64 + pad, "ld_residual": 64 + pad, "ld_dx": 64 + pad,
              "bias_dtype": "bf16", "activation": "gelu", "dropout": 0.2, "seed": SEED, "offset": OFFSET}
        want, err = value("gelu", buf[:, :64].double() + bias.double(), 0.2, res[:, :64])
        over = buf.clone()
        binding.wg_activation(sp, over, over, bias, res)
        close(over[:, :64], want, err, "bf16")
        assert torch.equal(over[:, 64:], buf[:, 64:])
        into = res.clone()
        binding.wg_activation(sp, buf, into, bias, into)
        assert torch.equal(into[:, :64], over[:, :64]) and torch.equal(into[:, 64:], res[:, 64:])
        one = torch.empty(90, 64 + pad, dtype=DT["bf16"], device="cuda")
        binding.wg_activation_bwd(sp, res, buf, one, bias)
        for t in (buf.clone(), res.clone()):
            binding.wg_activation_bwd(sp, t if torch.equal(t, res) else res, buf if torch.equal(t, res) else t, t, bias)
            assert torch.equal(t[:, :64], one[:, :64])


@pytest.mark.parametrize("p", [0.1, 0.5, 0.999])
def test_how_many_are_kept(p):
    """n draws of probability q: within six standard deviations; rows, columns, seeds and offsets draw apart."""
    x = torch.ones(4096, 512, device="cuda")
    masks = [binding.activation(x, dropout=p, seed=s, offset=o) != 0 for s, o in ((1, 1), (1, 2), (2, 1), (1, 1 + (1 << 32)))]
    n, thr = x.numel(), round(65536 * p)
    q = 1 - thr / 65536
    for m in masks:
        assert abs(float(m.double().mean()) - q) < 6 * (q * (1 - q) / n) ** 0.5
        assert abs(float(m[:, 0].double().mean()) - q) < 6 * (q * (1 - q) / 4096) ** 0.5
    for i in range(4):
        for j in range(i):
            both = float((masks[i] & masks[j]).double().mean())
            assert abs(both - q * q) < 6 * (q * q * (1 - q * q) / n) ** 0.5
    y = binding.activation(x, dropout=p, seed=1, offset=1)
    assert float(y[masks[0]].min()) == float(y[masks[0]].max()) == pytest.approx(65536 / (65536 - thr), rel=2.0 ** -23)


def test_dropped_infinities_are_zeros():
    x = torch.full((64, 64), float("inf"), device="cuda")
    y = binding.activation(x, dropout=0.5, seed=3)
    assert set(y.flatten().tolist()) == {0.0, float("inf")}
    dx = binding.activation_bwd(torch.full_like(x, float("nan")), dropout=0.5, seed=3)
    assert torch.equal(dx == 0, y == 0) and torch.equal(torch.isnan(dx), y != 0)
    v = torch.tensor([[1e30, -1e30, 1e20, -1e20, 3e4, -3e4, 90.0, -90.0]], device="cuda")
    for name in ACTS[1:]:
        y, d = binding.activation(v, activation=name), binding.activation_bwd(torch.ones_like(v), v, activation=name)
        assert torch.allclose(y, torch.where(v > 0, v, torch.zeros_like(v)), atol=1e-30, rtol=1e-6), (name, y)
        assert torch.allclose(d, (v > 0).float(), atol=1e-30), (name, d)


def test_nothing_to_do():
    x = torch.empty(0, 40, device="cuda")
    assert binding.activation(x, activation="gelu").shape == (0, 40)
    db = torch.ones(40, device="cuda")
    assert binding.activation_bwd(x, x, activation="gelu", dbias=db).shape == (0, 40)
    assert not db.any()


def test_many_rows_of_one_column():
    x = randn(1, 3_000_001, 1)
    db = torch.empty(1, device="cuda")
    dx = binding.activation_bwd(x, dropout=0.5, seed=SEED, offset=OFFSET, dbias=db)
    want, _ = drop(x.double(), 0.5, SEED, OFFSET)
    close(dx, want, 2.0 ** -23 * want.abs(), "fp32")
    # At most 128 + 2 * 2048 roundings along any way through the sums.
    assert abs(float(db) - float(want.sum())) < 4500 * 2.0 ** -24 * float(want.abs().sum())


@pytest.mark.parametrize("dim,pad,at", [(129, 0, (0, 0, 0)), (255, 1, (1, 2, 3)), (257, 2, (7, 0, 5)), (999, 0, (3, 3, 3)),
                                        (1000, 4, (4, 1, 6)), (2047, 1, (0, 5, 2)), (264, 0, (1, 1, 1))])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_long_rows_that_start_anywhere(dim, pad, at, dt):
    """16-bit rows at every distance from 16 bytes, in place and not; what lies around the rows stays as it is."""
    rows, ld = 83, dim + pad

    def place(t, k):
        buf = randn(9, 16 + rows * ld, dt=dt)
        view = torch.as_strided(buf, (rows, dim), (ld, 1), k)
        view.copy_(t)
        return buf, view

    def check(buf, view, want, err):
        rest = buf.clone()
        torch.as_strided(rest, (rows, dim), (ld, 1), view.storage_offset()).zero_()
        clean = randn(9, 16 + rows * ld, dt=dt)
        torch.as_strided(clean, (rows, dim), (ld, 1), view.storage_offset()).zero_()
        assert torch.equal(rest, clean)
        close(view, want, err, dt)

    x0, r0, bias = randn(1, rows, dim, size=2, dt=dt), randn(2, rows, dim, dt=dt), randn(3, dim)
    sp = {"tokens": rows, "dim": dim, "ld_x": ld, "ld_y": ld, "ld_residual": ld, "ld_dx": ld, "in_dtype": dt, "out_dtype": dt,
          "activation": "silu", "dropout": 0.2, "seed": SEED, "offset": OFFSET}
    v = x0.double() + bias.double()
    want, err = value("silu", v, 0.2, r0)
    grad = slope("silu", v) * r0.double()
    gerr = (2.0 ** -19 + 1.6 * 2.0 ** -24 * v.abs()) * r0.double().abs()
    grad, gain = drop(grad, 0.2, SEED, OFFSET)
    gerr = gerr * gain + 2.0 ** -23 * grad.abs()
    ws = torch.empty(binding.wg_activation_workspace_size(sp), dtype=torch.uint8, device="cuda")
    for over in ("", "x", "other"):
        (xb, x), (rb, r), (yb, y) = place(x0, at[0]), place(r0, at[1]), place(torch.zeros_like(x0), at[2])
        b, t = {"": (yb, y), "x": (xb, x), "other": (rb, r)}[over]
        binding.wg_activation(sp, x, t, bias, r)
        check(b, t, want, err)
        (xb, x), (rb, r) = place(x0, at[0]), place(r0, at[1])
        b, t = {"": (yb, y), "x": (xb, x), "other": (rb, r)}[over]
        db = torch.full((dim,), float("nan"), device="cuda")
        binding.wg_activation_bwd(sp, r, x, t, bias, db, ws)
        check(b, t, grad, gerr)
        # dbias: fewer than 256 roundings of sums that are at most the sum of the terms' sizes.
        close(db, grad.sum(0), gerr.sum(0) + 256 * 2.0 ** -24 * grad.abs().sum(0), "fp32", "dbias")
