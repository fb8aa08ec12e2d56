"""Layer calls whose tensors pass 2^31 elements (and 2^32 bytes): every address is one of 64 bits."""
import numpy as np
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import DT, act, close, data, drop, forward, slope, sum_error, weight  # noqa: E402

SEED, OFFSET = 0x1234_5678_9ABC_DEF0, (5 << 32) + 77


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    binding.wg_check_status()
    torch.cuda.empty_cache()


def randn(seed, *shape, size=1.0, dt="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(shape, generator=g, device="cuda")).to(DT[dt])


def far(seed, rows, cols, ld, dt, size=1.0):
    """Rows of `cols` values, ld apart, in memory of their own that nothing else touches."""
    t = torch.empty(rows * ld, dtype=DT[dt], device="cuda").as_strided((rows, cols), (ld, 1))
    t.copy_(randn(seed, rows, cols, size=size, dt=dt))
    return t


def space(sp, call):
    return torch.empty(binding.wg_linear_workspace_size(sp, call), dtype=torch.uint8, device="cuda")


# Rows so far apart that 40 of them, and the few of a decoding step, pass 2^31 elements; aligned and not.
@pytest.mark.parametrize("tokens,ld", [(40, (1 << 26) + 8), (40, (1 << 26) + 1), (5, (1 << 29) + 8), (5, (1 << 29) + 3)])
def test_rows_far_apart(tokens, ld):
    inf, out, dt = 264, 136, "bf16"
    assert (tokens - 1) * ld > 1 << 31
    kw = dict(activation="gelu", dropout=0.2, seed=SEED, offset=OFFSET)
    sp = {"tokens": tokens, "in": inf, "out": out, "ld_in": ld, "ld_out": ld, "ld_z": ld, "ld_residual": ld, **kw}
    x, res, y, z = far(1, tokens, inf, ld, dt), far(2, tokens, out, ld, dt), far(3, tokens, out, ld, dt), far(4, tokens, out, ld, dt)
    w, bias = randn(5, out, inf, size=inf ** -0.5, dt=dt), randn(6, out)
    binding.wg_linear(sp, x, w, y, bias, res, z, None, space(sp, "forward"))
    (v, verr), (want, err) = forward(x, w[None], bias[None], res, "gelu", 0.2, SEED, OFFSET)
    close(z, v, verr, dt, "z")
    close(y, want, err, dt, "y")
    dx, zin = far(7, tokens, inf, ld, dt), far(8, tokens, inf, ld, dt)
    binding.wg_linear_bwd_data(sp, y, w, dx, zin, None, None, space(sp, "bwd_data"))
    want, err = data(y, w[None], zin, None, "gelu", 0.2, SEED, OFFSET)
    close(dx, want, err, dt, "dx")
    sw = dict(sp, out_dtype="fp32", activation="none", dropout=0.0)
    dw, db = torch.empty(1, out, inf, device="cuda"), torch.empty(1, out, device="cuda")
    binding.wg_linear_bwd_weight(sw, x, y, dw, db, workspace=space(sw, "bwd_weight"))
    (wd, werr), (wb, berr) = weight(x, y)
    close(dw, wd, werr, "fp32", "dw")
    close(db, wb, berr, "fp32", "dbias")
    sa = {"tokens": tokens, "dim": out, "ld_x": ld, "ld_y": ld, "ld_residual": ld, "ld_dx": ld, **kw}
    binding.wg_activation(sa, z, y, bias, res)
    u = z.double() + bias.double()
    a, gain = drop(act("gelu", u), 0.2, SEED, OFFSET)
    close(y, a + res.double(), gain * (1.13 * 2.0 ** -24 * u.abs() + 2.0 ** -20 * (u.abs() + 1)) + 2.0 ** -22 * (a.abs() + res.double().abs()), dt)
    ws = torch.empty(binding.wg_activation_workspace_size(sa), dtype=torch.uint8, device="cuda")
    db = torch.empty(out, device="cuda")
    binding.wg_activation_bwd(sa, res, z, y, bias, db, ws)
    d, gain = drop(slope("gelu", u) * res.double(), 0.2, SEED, OFFSET)
    err = gain * (2.0 ** -19 + 1.6 * 2.0 ** -24 * u.abs()) * res.double().abs() + 2.0 ** -23 * d.abs()
    close(y, d, err, dt)
    close(db, d.sum(0), err.sum(0) + 256 * 2.0 ** -24 * d.abs().sum(0), "fp32", "dbias")


@pytest.mark.parametrize("tokens,stride,counts", [(300, (1 << 30) + 8, [100, 0, 120, 80]), (300, (1 << 30) + 1, [100, 0, 120, 80]),
                                                  (9, (1 << 30) + 8, [2, 0, 3, 4]), (9, (1 << 30) + 5, [2, 0, 3, 4])])
def test_experts_far_apart(tokens, stride, counts):
    """Experts' weights and their gradients 2^30 elements apart."""
    inf, out, n, dt = 72, 136, len(counts), "bf16"
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    wbuf = torch.empty((n - 1) * stride + out * inf, dtype=DT[dt], device="cuda")
    w = wbuf.as_strided((n, out, inf), (stride, inf, 1))
    w.copy_(randn(1, n, out, inf, size=0.1, dt=dt))
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n, "weight_stride": stride}
    x, dy = randn(2, tokens, inf, dt=dt), randn(3, tokens, out, dt=dt)
    y, dx = torch.empty(tokens, out, dtype=DT[dt], device="cuda"), torch.empty(tokens, inf, dtype=DT[dt], device="cuda")
    binding.wg_linear(sp, x, wbuf, y, offsets=off, workspace=space(sp, "forward"))
    _, (want, err) = forward(x, w, offsets=off.tolist())
    close(y, want, err, dt, "y")
    binding.wg_linear_bwd_data(sp, dy, wbuf, dx, offsets=off, workspace=space(sp, "bwd_data"))
    want, err = data(dy, w, offsets=off.tolist())
    close(dx, want, err, dt, "dx")
    start = w.double()
    binding.wg_linear_bwd_weight(sp, x, dy, wbuf, accumulate=True, offsets=off, workspace=space(sp, "bwd_weight"))
    (wd, werr), _ = weight(x, dy, off.tolist(), n)
    close(w, wd + start, werr + 2.0 ** -23 * (wd.abs() + start.abs()), dt, "dw")


def kept(rows, cols, p):
    """The mask of the given rows, wherever they are: Philox 4x32-10 as include/wgrad.h states it."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    groups = (cols + 7) // 8
    c = [np.tile(np.arange(groups, dtype=u), len(rows)), np.repeat(np.array(rows, dtype=u), groups),
         np.full(len(rows) * groups, OFFSET & 0xFFFFFFFF, dtype=u), np.full(len(rows) * groups, OFFSET >> 32, dtype=u)]
    k0, k1 = SEED & 0xFFFFFFFF, SEED >> 32
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & low, (a >> u(32)) ^ c[3] ^ u(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    h = np.stack([x for w in c for x in (w & u(0xFFFF), w >> u(16))], -1).reshape(len(rows), -1)[:, :cols]
    return torch.from_numpy(h >= u(round(65536 * p))).cuda()


@pytest.mark.parametrize("rows,dim,dt", [(17_000_001, 129, "bf16"), (280_000, 8200, "fp16"), (2100, 1 << 20, "bf16")])
def test_activations_of_many_elements(rows, dim, dt):
    """More than 2^31 elements in one call, in place: rows near both ends and the 2^31st element."""
    assert rows * dim > 1 << 31
    x, step = torch.empty(rows, dim, dtype=DT[dt], device="cuda"), max(1, (1 << 28) // dim)
    for r in range(0, rows, step):
        x[r:r + step].normal_(generator=torch.Generator(device="cuda").manual_seed(r + 1))
    mid = (1 << 31) // dim
    some = [0, 1, mid - 1, mid, mid + 1, rows - 2, rows - 1]
    v, gain = x[some].double(), 4 / 3
    binding.wg_activation({"tokens": rows, "dim": dim, "in_dtype": dt, "out_dtype": dt, "activation": "silu", "dropout": 0.25,
                           "seed": SEED, "offset": OFFSET}, x, x)
    mask = kept(some, dim, 0.25)
    a = act("silu", v) * gain * mask
    close(x[some], a, mask * gain * 2.0 ** -20 * (v.abs() + 1) + 2.0 ** -23 * a.abs(), dt)


def test_a_product_of_many_elements():
    """2^31 and more results in one call, with the mask of late rows, and the weight gradient that reads them."""
    tokens, inf, out = 270_000, 64, 8200
    x, w = randn(1, tokens, inf, dt="bf16"), randn(2, out, inf, size=inf ** -0.5, dt="bf16")
    assert tokens * out > 1 << 31
    y = binding.linear(x, w, activation="relu", dropout=0.5, seed=SEED, offset=OFFSET)
    for lo in (0, (1 << 31) // out - 40, tokens - 100):
        u = slice(lo, lo + 100)
        v, A = x[u].double() @ w.double().T, x[u].double().abs() @ w.double().abs().T
        mask = kept(range(lo, lo + 100), out, 0.5)
        want = torch.relu(v) * 2 * mask
        close(y[u], want, mask * (2.26 * sum_error(A, inf) + 2.0 ** -23 * want), "bf16")
    dw = binding.linear_bwd_weight(x, y)
    cols = torch.tensor([0, 1, 31, 4099, 8191, 8192, 8198, 8199], device="cuda")
    part = torch.zeros(8, inf, dtype=torch.float64, device="cuda")
    size = part.clone()
    for r in range(0, tokens, 30000):
        d, e = y[r:r + 30000][:, cols].double(), x[r:r + 30000].double()
        part, size = part + d.T @ e, size + d.abs().T @ e.abs()
    close(dw[cols], part, sum_error(size, tokens), "fp32")
