"""The convenience calls on a stream of their own, while the current stream still works on memory that it has freed.

Each call allocates its result (and its workspace) itself.  A block that torch has back from the current stream may
not be used on another one until the work pending there has ended: the calls must take their memory from the blocks of
the stream that they run on.
"""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def randn(*shape):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(len(shape)), device="cuda")


CONV = {"ndim": 2, "G": 1, "N": 4, "C": 32, "K": 32, "in": [20, 24], "filt": [3, 3], "stride": [1, 1], "dil": [1, 1],
        "pad_l": [1, 1], "pad_r": [1, 1], "in_dtype": "bf16", "out_dtype": "fp32"}


def call(name):
    """(the call, the bytes of its workspace)"""
    tok = torch.arange(3000, device="cuda") * 7 % 1000
    if name == "lookup":
        table = randn(1000, 256)
        return lambda **kw: binding.embedding_lookup(tok, table, 2.0, **kw), 0
    if name == "table gradient":
        dy = randn(3000, 256)
        spec = {"tokens": 3000, "vocab": 1000, "dim": 256, "table_dtype": "fp32", "out_dtype": "fp32"}
        return lambda **kw: binding.embedding_bwd_weight(tok, dy, 1000, **kw), binding.wg_embedding_workspace_size(spec)
    if name.startswith("update"):
        rows, cols = (64, 576) if name == "update, small" else (200, 320)
        spec, grad = {"rows": rows, "cols": cols}, randn(rows, cols)
        return lambda **kw: binding.muon_update(spec, grad, **kw), binding.wg_muon_workspace_size(spec)
    dy = randn(4, 20, 24, 1, 32).bfloat16()
    if name == "conv weight":
        x = randn(4, 20, 24, 1, 32).bfloat16()
        return (lambda **kw: binding.conv_bwd_weight(CONV, x, dy, 4, "deterministic", **kw),
                binding.wg_workspace_size(CONV, 4, "deterministic", 0))
    w = randn(1, 32, 3, 3, 32).bfloat16()
    return lambda **kw: binding.conv_bwd_data(CONV, dy, w, **kw), binding.wg_bwd_data_workspace_size(CONV)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["lookup", "table gradient", "update, small", "update, large", "conv weight", "conv data"])
def test_memory_of_a_call_is_not_what_the_current_stream_still_writes(name, raw):
    f, nbytes = call(name)
    want = f().clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    # Blocks of the sizes that the call needs, freed while their last writes are pending.
    torch.cuda._sleep(100_000_000)
    for block in [torch.empty_like(want) for _ in range(2)] + [torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")]:
        block.fill_(77)
    del block
    got = f(stream=s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
