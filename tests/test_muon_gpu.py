"""GPU checks of the orthogonalised update against the iteration in 64 bits.

Tolerance: X's relative error in the 2-norm is at most 4e-3 (the bound include/wgrad.h states), and no element is
off by more than 40 times that against the larger of its size and the matrix's root mean square (errors are spread
over the elements like roundings, so far tails stay below some ten standard deviations); then one rounding to the
output's type.  The momentum is one or two fp32 operations: 2^-22 of the sum of its terms' sizes.
"""
import numpy as np
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
COEF = (3.4445, -4.7750, 2.0315)
BOUND = 4e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def gradient(seed, b, r, c, dt="fp32", kind="mixed", size=1e-3):
    g = rng(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    if kind == "noise":
        u = n(b, r, c)
    elif kind == "rank one":
        u = n(b, r, 1) @ n(b, 1, c)
    else:
        k = max(1, min(r, c) // 8)
        u = n(b, r, k) @ n(b, k, c) / k ** 0.5 + 0.3 * n(b, r, c)
    return (u * size).to(DT[dt])


def f32(v):
    return float(np.float32(v))


def exact_x(u, steps=5, eps=1e-7, coef=None):
    u = u.double()
    x = u / (torch.linalg.matrix_norm(u)[:, None, None] + f32(eps))
    tall = u.shape[1] > u.shape[2]
    for i in range(steps):
        a, b, c = (f32(v) for v in (coef[i] if coef else COEF))
        q = x.mT @ x if tall else x @ x.mT
        p = b * q + c * (q @ q)
        x = a * x + (x @ p if tall else p @ x)
    return x


def close(got, ref, dt, bound=BOUND, extra=0.0):
    """Per matrix: got against ref, which is off by `bound` relatively and then rounded to dt."""
    got = got.double()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    norm = torch.linalg.matrix_norm(ref)
    rms = norm[:, None, None] / (ref.shape[1] * ref.shape[2]) ** 0.5
    far = torch.linalg.matrix_norm(err)
    assert (far <= (bound + HALF[dt]) * norm + 1e-30).all(), float((far / norm).max())
    assert (err <= (40 * bound + HALF[dt]) * torch.maximum(rms, ref.abs()) + extra + 1e-30).all()


SHAPES = [(1, 1, 1), (1, 1, 9), (1, 9, 1), (3, 5, 7), (1, 2, 2), (32, 8, 72), (7, 3, 40), (2, 64, 576), (1, 96, 3456),
          (2, 65, 80), (1, 128, 128), (1, 127, 129), (1, 129, 130), (1, 1, 3000), (1, 3000, 2), (2, 200, 333),
          (3, 256, 64), (4, 72, 8), (5, 100, 31), (1, 300, 1000), (1, 1000, 300), (1, 257, 2049), (2, 512, 512),
          (1, 640, 256), (1, 1100, 1300), (1, 2050, 700)]


@pytest.mark.parametrize("b,r,c", SHAPES)
@pytest.mark.parametrize("kind", ["mixed", "noise", "rank one"])
def test_update(b, r, c, kind):
    grad = gradient(b + r + c, b, r, c, kind=kind)
    out = torch.full((b, r, c), float("nan"), dtype=torch.bfloat16, device="cuda")
    sp = {"batch": b, "rows": r, "cols": c, "scale": 1.75}
    ws = torch.full((binding.wg_muon_workspace_size(sp),), 0xFF, dtype=torch.uint8, device="cuda")
    binding.wg_muon_update(sp, grad, out=out, workspace=ws)
    close(out, 1.75 * exact_x(grad), "bf16")
    again = torch.full_like(out, float("nan"))
    binding.wg_muon_update(sp, grad, out=again, workspace=ws)
    assert torch.equal(out, again)
    binding.wg_check_status()


@pytest.mark.parametrize("gdt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("odt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("b,r,c", [(2, 48, 100), (1, 190, 140)])
def test_types(gdt, odt, b, r, c):
    grad = gradient(5, b, r, c, gdt)
    out = torch.empty((b, r, c), dtype=DT[odt], device="cuda")
    binding.muon_update({"batch": b, "rows": r, "cols": c, "grad_dtype": gdt, "out_dtype": odt}, grad, out=out)
    close(out, exact_x(grad), odt)


@pytest.mark.parametrize("b,r,c", [(1, 40, 72), (3, 16, 9), (1, 150, 220), (2, 300, 136), (1, 64, 576)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("damp", [0.0, 0.9])
@pytest.mark.parametrize("wdt", ["bf16", "fp32"])
def test_step(b, r, c, nesterov, damp, wdt):
    g = rng(r)
    mu, lr, wd, scale = 0.9, 0.05, 0.1, 0.8
    grad = gradient(1, b, r, c, "bf16")
    mom = 3 * gradient(2, b, r, c)
    w = torch.randn((b, r, c), generator=g, device="cuda").to(DT[wdt])
    m0, w0 = mom.double(), w.double()
    out = torch.empty((b, r, c), dtype=torch.bfloat16, device="cuda")
    sp = {"batch": b, "rows": r, "cols": c, "grad_dtype": "bf16", "weight_dtype": wdt, "momentum": mu, "lr": lr,
          "weight_decay": wd, "scale": scale, "dampening": damp, "nesterov": nesterov}
    binding.muon_update(sp, grad, momentum=mom, weight=w, out=out)
    gain = f32(1 - np.float32(damp))
    m1 = f32(mu) * m0 + gain * grad.double()
    assert ((mom.double() - m1).abs() <= 2.0 ** -22 * (m0.abs() + grad.double().abs())).all()
    u = gain * grad.double() + f32(mu) * m1 if nesterov else m1
    x = exact_x(u)
    close(out, scale * x, "bf16")
    keep = 1 - f32(lr) * f32(wd)
    want = keep * w0 - lr * scale * x
    norm = torch.linalg.matrix_norm(x)
    err = torch.linalg.matrix_norm(w.double() - want)
    assert (err <= lr * scale * BOUND * norm + HALF[wdt] * torch.linalg.matrix_norm(want) * 1.01
            + 2.0 ** -22 * torch.linalg.matrix_norm(w0)).all()


@pytest.mark.parametrize("r,c", [(24, 40), (40, 24), (140, 200), (200, 140)])
@pytest.mark.parametrize("gap,off", [(0, 0), (8, 8), (5, 3)])
@pytest.mark.parametrize("beside", [False, True])
def test_strides(r, c, gap, off, beside):
    """Matrices of rows apart, after one another or side by side, from any element on: between them nothing changes."""
    b = 3
    ld = b * (c + gap) if beside else c + gap
    bs = c + gap if beside else r * ld + gap
    total = off + r * b * (c + gap) + b * gap + 64
    view = lambda t: torch.as_strided(t, (b, r, c), (bs, ld, 1), off)  # noqa: E731
    grad = torch.full((total,), float("nan"), device="cuda")
    view(grad).copy_(gradient(r, b, r, c))
    mom, w, out = torch.full_like(grad, 5.0), torch.full_like(grad, 5.0), torch.full_like(grad, 5.0)
    w, out = w.bfloat16(), out.bfloat16()
    view(mom).copy_(gradient(r + 1, b, r, c))
    view(w).fill_(1.0)
    u = f32(0.95) * (f32(0.95) * view(mom).double() + view(grad).double()) + view(grad).double()
    sp = {"batch": b, "rows": r, "cols": c, "ld": ld, "batch_stride": bs, "lr": 1.0}
    ws = torch.empty(binding.wg_muon_workspace_size(sp), dtype=torch.uint8, device="cuda")
    binding.wg_muon_update(sp, grad[off:], mom[off:], w[off:], out[off:], ws)
    x = exact_x(u)
    close(view(out).contiguous(), x, "bf16")
    far = torch.linalg.matrix_norm(view(w).double() - (1 - x))
    assert (far <= BOUND * torch.linalg.matrix_norm(x) + HALF["bf16"] * torch.linalg.matrix_norm(1 - x) * 1.01).all()
    for t in (mom, w, out):
        view(t).fill_(5.0)
        assert (t == 5).all()


@pytest.mark.parametrize("r,c", [(20, 50), (50, 20), (150, 170), (170, 150)])
def test_zero_nan_and_infinite_matrices_keep_to_themselves(r, c):
    grad = gradient(9, 6, r, c)
    ref = exact_x(grad)
    grad[1] = 0
    grad[2, r // 2, c // 3] = float("nan")
    grad[4, 0, c - 1] = float("inf")
    for eps in (1e-7, 0.0):
        out = binding.muon_update({"batch": 6, "rows": r, "cols": c, "eps": eps}, grad)
        assert not out[1].any()
        assert torch.isnan(out[2]).all() and torch.isnan(out[4]).all()
        good = torch.tensor([0, 3, 5], device="cuda")
        close(out[good], ref[good], "bf16", bound=BOUND + (2e-6 if eps == 0 else 0))


@pytest.mark.parametrize("size", [1e-12, 1e-3, 1e6])
@pytest.mark.parametrize("r,c", [(30, 70), (160, 200)])
def test_sizes_of_gradients(size, r, c):
    grad = gradient(11, 1, r, c, size=size)
    out = binding.muon_update({"rows": r, "cols": c, "eps": 0.0}, grad)
    close(out, exact_x(grad, eps=0.0), "bf16")


@pytest.mark.parametrize("r,c", [(30, 70), (160, 200), (200, 160)])
@pytest.mark.parametrize("steps", [0, 1, 2, 16])
def test_steps_and_coefficients(r, c, steps):
    grad = gradient(12, 2, r, c, kind="noise")
    # Two forms of coefficients in turn; with many steps the iteration with fixed point 1 ends at an orthogonal matrix.
    coef = [(1.875, -1.25, 0.375) if i % 2 or steps == 16 else (3.4445, -4.775, 2.0315) for i in range(steps)]
    sp = {"batch": 2, "rows": r, "cols": c, "steps": steps, "coef": coef, "out_dtype": "fp32"}
    out = binding.muon_update(sp, grad)
    close(out, exact_x(grad, steps, coef=coef), "fp32", bound=BOUND if steps else 2.0 ** -20)
    if steps == 16:
        x = out.double() if r <= c else out.double().mT
        eye = torch.eye(min(r, c), dtype=torch.float64, device="cuda")
        assert float((x @ x.mT - eye).abs().max()) < 0.02


def test_wrapper_lays_its_result_out_like_the_gradient():
    b, r, c, ld = 2, 24, 40, 51
    room = torch.zeros((b, r, ld), device="cuda")
    room[..., :c] = gradient(14, b, r, c)
    out = binding.muon_update({"batch": b, "rows": r, "cols": c, "ld": ld}, room[..., :c])
    assert out.shape == (b, r, c) and out.stride() == (r * ld, ld, 1)
    close(out.contiguous(), exact_x(room[..., :c].contiguous()), "bf16")


def test_batches_past_32_bits():
    r, c, bs = 24, 40, (1 << 31) + 24
    grad = torch.zeros(bs + r * c, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(grad)
    view = lambda t: torch.as_strided(t, (2, r, c), (bs, c, 1))  # noqa: E731
    view(grad).copy_(gradient(13, 2, r, c, "bf16"))
    sp = {"batch": 2, "rows": r, "cols": c, "batch_stride": bs, "grad_dtype": "bf16"}
    ws = torch.empty(binding.wg_muon_workspace_size(sp), dtype=torch.uint8, device="cuda")
    binding.wg_muon_update(sp, grad, out=out, workspace=ws)
    close(view(out).contiguous(), exact_x(view(grad)), "bf16")


@pytest.mark.parametrize("r,c", [(64, 576), (192, 260)])
def test_other_stream_and_graph(r, c):
    grad = gradient(14, 1, r, c)
    sp = {"rows": r, "cols": c}
    want = binding.muon_update(sp, grad)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = binding.muon_update(sp, grad, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(binding.wg_muon_workspace_size(sp), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.wg_muon_update(sp, grad, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_runs_after_the_weight_gradient_that_makes_its_input():
    """Chained on one stream without synchronisation: the convolution's dW is the update's gradient."""
    g = rng(15)
    cv = {"ndim": 2, "G": 2, "N": 2, "C": 16, "K": 32, "in": [10, 12], "filt": [3, 3], "stride": [1, 1],
          "dil": [1, 1], "pad_l": [1, 1], "pad_r": [1, 1], "in_dtype": "bf16", "out_dtype": "fp32"}
    x = torch.randn((2, 10, 12, 2, 16), generator=g, device="cuda").bfloat16()
    dy = torch.randn((2, 10, 12, 2, 32), generator=g, device="cuda").bfloat16()
    sp = {"batch": 2, "rows": 32, "cols": 144}
    ws = torch.empty(binding.wg_muon_workspace_size(sp), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 32, 144), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((2, 32, 3, 3, 16), device="cuda")
    for _ in range(20):
        dw.fill_(float("nan"))
        binding.conv_bwd_weight(cv, x, dy, 1, "direct", out=dw)
        binding.wg_muon_update(sp, dw, out=out, workspace=ws)
    close(out, exact_x(dw.view(2, 32, 144)), "bf16")
