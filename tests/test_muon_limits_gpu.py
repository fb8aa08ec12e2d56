"""GPU checks of the orthogonalised update at the ends of fp32's range, and at sizes beyond those of the other tests."""
import pytest

from implicit_gemm_gb300 import binding, build
from tests.test_muon_gpu import BOUND, close, exact_x, gradient

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("r,c", [(20, 50), (50, 20), (9, 33), (150, 170)])
@pytest.mark.parametrize("big", [3.4e38, -3.3953e38, 1e37, 1.9e19])
def test_elements_whose_square_is_beyond_fp32_keep_to_their_matrix(r, c, big):
    """Several matrices share a block of the Gram kernel; 3.4e38 is finite, and infinite when rounded to bf16."""
    grad = gradient(9, 6, r, c)
    ref = exact_x(grad)
    grad[2, r // 2, c // 3] = big
    out = binding.muon_update({"batch": 6, "rows": r, "cols": c}, grad)
    assert torch.isnan(out[2]).all()
    good = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    close(out[good], ref[good], "bf16", bound=BOUND)


@pytest.mark.parametrize("r,c", [(40, 72), (150, 220)])
def test_factors_are_the_call_s_own(r, c):
    """Calls that differ in their factors alone share a plan, and nothing else."""
    grad = gradient(3, 1, r, c)
    x = exact_x(grad)
    for lr, wd, scale, mu, damp in ((0.1, 0.0, 1.0, 0.9, 0.0), (0.02, 0.5, 1.0, 0.9, 0.0), (0.02, 0.5, 3.0, 0.5, 0.25)):
        w = torch.ones((1, r, c), device="cuda")
        mom = torch.zeros_like(w)
        sp = {"rows": r, "cols": c, "lr": lr, "weight_decay": wd, "scale": scale, "momentum": mu, "dampening": damp,
              "weight_dtype": "fp32", "eps": 0.0}
        binding.muon_update(sp, grad, momentum=mom, weight=w)
        close(w.double() - (1 - lr * wd), -lr * scale * x, "fp32", extra=1e-6)
        assert torch.allclose(mom, (1 - damp) * grad, rtol=1e-6)
        close(binding.muon_update({**sp, "out_dtype": "fp32"}, grad), scale * x, "fp32")
        assert not binding.muon_update({**sp, "eps": 1e30, "out_dtype": "fp32"}, grad).abs().max() > 1e-20


@pytest.mark.parametrize("r,c", [(40, 72), (72, 40), (150, 220), (1100, 700)])
def test_norms_far_below_eps(r, c):
    """u / (|u|_F + eps) is small then, and every step multiplies it by a: X in fp16 keeps its bits down to the norm that
    the header names, 1e-7 sqrt(rows cols) eps."""
    grad = gradient(4, 1, r, c, kind="noise").double()
    grad = (grad * (2e-7 * (r * c) ** 0.5 * 1e-3 / torch.linalg.matrix_norm(grad))).float()
    out = binding.muon_update({"rows": r, "cols": c, "eps": 1e-3, "out_dtype": "fp32"}, grad)
    close(out, exact_x(grad, eps=1e-3), "fp32")


@pytest.mark.parametrize("b,r,c", [(1, 4096, 1100), (1, 1030, 5000)])
def test_larger_matrices(b, r, c):
    """Several waves of tiles, and the leftovers."""
    grad = gradient(5, b, r, c)
    ref = exact_x(grad)
    close(binding.muon_update({"batch": b, "rows": r, "cols": c, "out_dtype": "fp32"}, grad), ref, "fp32")
