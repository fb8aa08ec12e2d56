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
