"""GPU check of wg_check_status where two things have happened."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def status():
    try:
        binding.wg_check_status()
    except binding.WgradError as e:
        return e.status
    return 0


@pytest.mark.parametrize("first", ["token", "timeout"])
def test_a_timeout_does_not_hide_a_bad_token(first):
    """The library's self-test lets a bounded wait run out (about two seconds); both are reported, each once."""
    build.build()
    binding.load()
    table = torch.zeros((4, 8), device="cuda")
    tok = torch.tensor([1, 4], device="cuda")
    for what in ([0, 1] if first == "token" else [1, 0]):
        if what == 0:
            binding.embedding_lookup(tok, table)
        else:
            binding.wg_selftest_timeout()
    assert [status(), status(), status()] == [6, 7, 0]
    binding.embedding_lookup(tok, table)
    assert [status(), status()] == [7, 0]
