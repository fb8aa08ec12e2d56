"""GPU checks of the table's gradient where its sort takes more than one wave of CTAs (above 223,744 rows on 152 SMs)."""
import pytest

from implicit_gemm_gb300 import binding, build
from tests.test_embedding_gpu import close, randn, ref_grad, rng

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("T,V,D", [(5000, 300001, 16), (40000, 262144, 24), (3000, 700003, 5), (1, 500000, 9), (1025, 1000000, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_a_table_of_many_rows(T, V, D, accumulate):
    g = rng(T + V)
    tok = torch.randint(V, (T,), generator=g, device="cuda")
    tok[:T // 3] = V - 1  # a long run in the last CTA's rows
    tok[T // 3:T // 2] = torch.randint(V - 2000, V, (T // 2 - T // 3,), generator=g, device="cuda")
    dy = randn(g, (T, D), "bf16")
    out = randn(g, (V, D), "fp32") if accumulate else torch.full((V, D), float("nan"), device="cuda")
    old = out.double() if accumulate else 0.0
    binding.embedding_bwd_weight(tok, dy, V, 0.5, out=out, accumulate=accumulate)
    ref, slack = ref_grad(tok, dy, V, 0.5)
    if accumulate:
        slack = slack + 2.0 ** -23 * (ref.abs() + old.abs())
    close(out, ref + old, slack, "fp32")
    binding.wg_check_status()
