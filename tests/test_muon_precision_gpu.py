"""GPU checks of the orthogonalised update where roundings grow: few strong directions, steep spectra, many steps,
large first factors.

Tolerance: the bound that include/wgrad.h states.  X's relative error (2-norm of all elements) is at most 4e-3, or
2^-22 S where that is more, S being the largest slope of the steps' map of a singular value on [0, 1] (at 0, the
product of the factors a): a rounding of X by 2^-22 in a direction that u lacks grows by S.  Sums of n > 512 elements
by tensor cores lose bits to truncation as they grow: S n / 512.  Above 1 the bound says
nothing about X, and only its largest singular value is looked at.  Results are fp32: no rounding hides the error.
"""
import numpy as np
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.875, -1.25, 0.375)
# A schedule with a large first factor that falls from step to step.
FALLING = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518),
           (3.3184, -2.4885, 0.5100), (2.3007, -1.6690, 0.4188)]
BOUND = 4e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def gradient(seed, b, r, c, kind, size=1e-3):
    """kind: ('rank', k, noise) or ('power', q): singular values i^-q, or ('two', s): one of 1, the others s."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    m = min(r, c)
    if kind[0] == "rank":
        k = max(1, m // kind[1]) if kind[1] > 1 else 1
        u = n(b, r, k) @ n(b, k, c) / k ** 0.5 + kind[2] * n(b, r, c)
    else:
        s = torch.arange(1, m + 1, device="cuda", dtype=torch.float64)
        s = s ** -kind[1] if kind[0] == "power" else torch.where(s > 1, kind[1], 1.0)
        u = (torch.linalg.qr(n(b, r, m))[0] * s) @ torch.linalg.qr(n(b, c, m))[0].mT
    return (u * size).float()


def f32(v):
    return float(np.float32(v))


def exact_x(u, coef, eps=1e-7):
    u = u.double()
    x = u / (torch.linalg.matrix_norm(u)[:, None, None] + f32(eps))
    tall = u.shape[1] > u.shape[2]
    for step in coef:
        a, b, c = (f32(v) for v in step)
        q = x.mT @ x if tall else x @ x.mT
        p = b * q + c * (q @ q)
        x = a * x + (x @ p if tall else p @ x)
    return x


def bound(coef, n=0):
    s, slope = np.linspace(0, 1, 20001), 1.0
    for a, b, c in coef:
        slope = slope * (a + 3 * b * s ** 2 + 5 * c * s ** 4)
        s = s * (a + b * s ** 2 + c * s ** 4)
    return max(BOUND, 2.0 ** -22 * float(np.abs(slope).max()) * max(1.0, n / 512))


def check(got, ref, coef, n=0):
    assert torch.isfinite(got).all()
    tol = bound(coef, n)
    if tol < 1:
        far = torch.linalg.matrix_norm(got.double() - ref) / torch.linalg.matrix_norm(ref)
        assert (far <= tol).all(), (float(far.max()), tol)
    else:
        assert (torch.linalg.matrix_norm(got.double(), 2) < 1.3).all()


GRAM = [(64, 3, 7), (32, 8, 72), (16, 72, 8), (8, 32, 288), (2, 64, 576), (2, 65, 575), (1, 96, 3456), (3, 128, 128),
        (1, 577, 63)]
KINDS = [("rank", 1, 0.0), ("rank", 1, 1e-3), ("rank", 1, 3e-3), ("rank", 1, 1e-2), ("rank", 1, 2e-2), ("rank", 8, 1e-3),
         ("rank", 8, 2e-2), ("power", 1), ("power", 2), ("power", 3), ("two", 5e-3), ("two", 1e-3), ("two", 1e-4)]


@pytest.mark.parametrize("b,r,c", GRAM)
@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("momentum", [False, True])
def test_few_directions_and_steep_spectra(b, r, c, kind, momentum):
    """Matrices of a side of at most 128, whose products are taken on the Gram matrix: u keeps its bits."""
    grad = gradient(b + r + c, b, r, c, kind)
    u, mom = grad.double(), None
    sp = {"batch": b, "rows": r, "cols": c, "out_dtype": "fp32", "momentum": 0.9}
    if momentum:
        mom = gradient(b + r + c, b, r, c, kind, 5e-3)  # the same directions
        u = f32(0.9) * (f32(0.9) * mom.double() + u) + u
    out = torch.empty((b, r, c), device="cuda")
    binding.muon_update(sp, grad, momentum=mom, out=out)
    check(out, exact_x(u, [QUINTIC] * 5), [QUINTIC] * 5)
    binding.wg_check_status()


SCHEDULES = {"6": [QUINTIC] * 6, "7": [QUINTIC] * 7, "8": [QUINTIC] * 8, "10": [QUINTIC] * 10, "16": [QUINTIC] * 16,
             "cubic 16": [CUBIC] * 16, "8 + 2": [QUINTIC] * 8 + [CUBIC] * 2, "falling": FALLING,
             "falling 8": FALLING + [CUBIC] * 3}


@pytest.mark.parametrize("b,r,c", [(64, 3, 7), (32, 8, 72), (5, 100, 31), (2, 64, 576), (2, 128, 128), (1, 61, 1001)])
@pytest.mark.parametrize("name", SCHEDULES)
@pytest.mark.parametrize("kind", [("rank", 1, 0.0), ("rank", 8, 0.0), ("rank", 8, 1e-3), ("power", 2), ("rank", 1, 1.0)],
                         ids=str)
def test_many_steps_and_large_factors_of_small_matrices(b, r, c, name, kind):
    coef = SCHEDULES[name]
    grad = gradient(b + r + c, b, r, c, kind)
    sp = {"batch": b, "rows": r, "cols": c, "out_dtype": "fp32", "steps": len(coef), "coef": coef}
    check(binding.muon_update(sp, grad), exact_x(grad, coef), coef)
    binding.wg_check_status()


@pytest.mark.parametrize("b,r,c", [(1, 160, 200), (1, 300, 260), (2, 256, 512), (1, 131, 1100), (1, 700, 330)])
@pytest.mark.parametrize("name", ["5", *SCHEDULES])
@pytest.mark.parametrize("kind", [("rank", 1, 0.0), ("rank", 8, 0.0), ("rank", 8, 1e-3), ("power", 2), ("two", 0.3),
                                  ("two", 0.2), ("rank", 1, 1.0)], ids=str)
def test_many_steps_and_large_factors_of_larger_matrices(b, r, c, name, kind):
    coef = [QUINTIC] * 5 if name == "5" else SCHEDULES[name]
    grad = gradient(b + r + c, b, r, c, kind)
    sp = {"batch": b, "rows": r, "cols": c, "out_dtype": "fp32", "steps": len(coef), "coef": coef}
    out = torch.full((b, r, c), float("nan"), device="cuda")
    ws = torch.full((binding.wg_muon_workspace_size(sp),), 0xFF, dtype=torch.uint8, device="cuda")
    binding.wg_muon_update(sp, grad, out=out, workspace=ws)
    check(out, exact_x(grad, coef), coef, max(r, c))
    binding.wg_check_status()
