"""GPU checks of the embedding lookup and the table's gradient against 64-bit sums.

Tolerances, per element: a lookup is one product rounded to fp32 and once more to the output's type; a gradient's
fp32 sum of n terms is off by at most (n + 1) * 2^-24 * sum |dy| before the scale, and is then rounded like a lookup.
"""
import numpy as np
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a unit in the last place, relative (at most)
TINY = {"fp32": 1e-38, "bf16": 1e-38, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda").to(DT[dt])


def close(got, ref, slack, dt):
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all()
    tol = slack + HALF[dt] * ref.abs() * 1.01 + TINY[dt]
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol).max()))


def ref_grad(token, dy, vocab, scale, padding=-1):
    """(gradient, its error bound before rounding) in 64 bits on the host."""
    tok = token.cpu().numpy().astype(np.int64).ravel()
    d = dy.double().cpu().numpy().reshape(len(tok), -1)
    g, a = np.zeros((vocab, d.shape[1])), np.zeros((vocab, d.shape[1]))
    n = np.zeros(vocab)
    ok = (tok >= 0) & (tok < vocab) & (tok != padding)
    np.add.at(g, tok[ok], d[ok])
    np.add.at(a, tok[ok], np.abs(d[ok]))
    np.add.at(n, tok[ok], 1)
    bound = (n[:, None] + 3) * 2.0 ** -24 * a * abs(scale)
    return torch.from_numpy(g * scale).cuda(), torch.from_numpy(bound).cuda()


@pytest.mark.parametrize("tdt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("odt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (3, 7, 5), (9, 100, 64), (300, 1000, 129), (257, 33, 1024)])
def test_lookup(tdt, odt, T, V, D):
    g = rng(T + V + D)
    table = randn(g, (V, D), tdt)
    for idt in (torch.int32, torch.int64):
        tok = torch.randint(V, (T,), generator=g, device="cuda").to(idt)
        out = torch.full((T, D), float("nan"), dtype=DT[odt], device="cuda")
        binding.embedding_lookup(tok, table, 3.7, out=out)
        ref = table[tok.long()].double() * float(np.float32(3.7))
        close(out, ref, 2.0 ** -23 * ref.abs(), odt)
    binding.wg_check_status()


@pytest.mark.parametrize("tdt,odt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("D", [2, 254, 258, 510, 1001])
def test_lookup_of_rows_that_start_anywhere(tdt, odt, D, off):
    g = rng(D + off)
    T, V = 77, 50
    table = randn(g, (off + V * D,), tdt)
    tok = torch.randint(V, (T,), generator=g, device="cuda").int()
    tok[5], tok[6] = -1, V
    out = torch.full((off + T * D + 3,), float("nan"), dtype=DT[odt], device="cuda")
    sp = {"tokens": T, "vocab": V, "dim": D, "table_dtype": tdt, "out_dtype": odt, "token_dtype": "i32", "scale": 3.7}
    binding.wg_embedding_lookup(sp, tok, table[off:], out[off:])
    ref = table[off:].view(V, D)[tok.long().clamp(0, V - 1)].double() * float(np.float32(3.7))
    ref[5:7] = 0
    close(out[off:off + T * D].view(T, D), ref, 2.0 ** -23 * ref.abs(), odt)
    assert torch.isnan(out[:off]).all() and torch.isnan(out[off + T * D:]).all()
    with pytest.raises(binding.WgradError) as e:
        binding.wg_check_status()
    assert e.value.status == 7


def test_lookup_strides_and_offsets():
    """Rows apart, buffers that start at any element; what lies between rows stays as it was."""
    g = rng(1)
    for ldt, ldo, off, D in ((70, 66, 0, 64), (72, 80, 8, 64), (72, 80, 1, 64), (33, 41, 3, 33)):
        table = randn(g, (50 * ldt + 16,), "bf16")
        out = torch.full((20 * ldo + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        tok = torch.randint(50, (20,), generator=g, device="cuda")
        sp = {"tokens": 20, "vocab": 50, "dim": D, "ld_table": ldt, "ld_out": ldo}
        binding.wg_embedding_lookup(sp, tok, table[off:], out[off:])
        got = out[off:off + 20 * ldo].view(20, ldo)
        assert torch.equal(got[:, :D], table[off:off + 50 * ldt].view(50, ldt)[tok][:, :D])
        assert (got[:, D:] == 7).all() and (out[:off] == 7).all() and (out[off + 20 * ldo:] == 7).all()


def test_lookup_of_no_tokens_and_of_bad_ones():
    table = randn(rng(2), (10, 48), "fp32")
    binding.embedding_lookup(torch.empty(0, dtype=torch.int64, device="cuda"), table)
    binding.wg_check_status()
    for bad in (-1, 10, 1 << 40, -(1 << 40)):
        tok = torch.tensor([1, bad, 2], dtype=torch.int64, device="cuda")
        out = binding.embedding_lookup(tok, table)
        with pytest.raises(binding.WgradError) as e:
            binding.wg_check_status()
        assert e.value.status == 7
        binding.wg_check_status()  # read once
        assert torch.equal(out[0], table[1]) and torch.equal(out[2], table[2]) and not out[1].any()


def test_lookup_passes_nan_and_inf():
    table = torch.tensor([[float("nan"), 1.0], [float("inf"), -0.0], [3e38, 1e-45]], device="cuda")
    out = binding.embedding_lookup(torch.tensor([0, 1, 2], device="cuda"), table, 2.0)
    assert torch.isnan(out[0, 0]) and torch.isinf(out[1, 0]) and torch.isinf(out[2, 0]) and out[0, 1] == 2


GRADS = [
    # T, V, D, how often the most frequent token occurs
    (1, 1, 1, 1), (5, 3, 7, 2), (64, 1, 33, 64), (65, 2, 8, 65), (100, 1000, 64, 32), (100, 1000, 64, 33),
    (1000, 300, 129, 500), (5000, 37, 72, 5000), (4099, 5000, 40, 2000), (3000, 2, 2051, 1500), (20000, 17, 16, 3),
]


@pytest.mark.parametrize("T,V,D,hot", GRADS)
@pytest.mark.parametrize("ydt,gdt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp16", "fp16"),
                                     ("fp32", "bf16")])
def test_gradient(T, V, D, hot, ydt, gdt):
    g = rng(T * 7 + D)
    tok = torch.randint(V, (T,), generator=g, device="cuda")
    tok[torch.randperm(T, generator=g, device="cuda")[:hot]] = V // 2
    dy = randn(g, (T, D), ydt)
    out = torch.full((V, D), float("nan"), dtype=DT[gdt], device="cuda")
    binding.embedding_bwd_weight(tok, dy, V, 0.37, out=out)
    ref, slack = ref_grad(tok, dy, V, float(np.float32(0.37)))
    close(out, ref, slack, gdt)
    # Bit for bit the same again, from other contents of the workspace and with 32-bit tokens.
    sp = {"tokens": T, "vocab": V, "dim": D, "table_dtype": gdt, "out_dtype": ydt, "token_dtype": "i32", "scale": 0.37}
    ws = torch.full((binding.wg_embedding_workspace_size(sp),), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        again = torch.full_like(out, float("nan"))
        binding.wg_embedding_bwd_weight(sp, tok.int(), dy, again, False, ws)
        assert torch.equal(out, again)
    binding.wg_check_status()


@pytest.mark.parametrize("gdt", ["fp32", "bf16"])
def test_gradient_accumulates_padding_and_bad_tokens(gdt):
    g = rng(3)
    T, V, D = 700, 90, 56
    tok = torch.randint(-3, 50, (T,), generator=g, device="cuda")
    tok[:200] = 5
    dy = randn(g, (T, D), "bf16")
    old = randn(g, (V, D), gdt)
    out = old.clone()
    binding.embedding_bwd_weight(tok, dy, V, 2.0, padding_token=7, out=out, accumulate=True)
    with pytest.raises(binding.WgradError) as e:
        binding.wg_check_status()
    assert e.value.status == 7
    ref, slack = ref_grad(tok, dy, V, 2.0, padding=7)
    total = ref + old.double()
    close(out, total, slack + 2.0 ** -23 * (ref.abs() + old.double().abs()), gdt)
    untouched = torch.ones(V, dtype=torch.bool, device="cuda")
    untouched[tok[(tok >= 0)]] = False
    untouched[7] = True
    assert torch.equal(out[untouched], old[untouched])
    # Written, not added to: the padding token's row is zero, like the rows without a token.
    out2 = torch.full((V, D), float("nan"), dtype=DT[gdt], device="cuda")
    binding.embedding_bwd_weight(tok, dy, V, 2.0, padding_token=7, out=out2)
    with pytest.raises(binding.WgradError):
        binding.wg_check_status()
    assert not out2[untouched].any()


def test_gradient_strides_and_offsets():
    g = rng(4)
    for ldt, ldy, off, D, gdt in ((70, 66, 0, 64, "fp32"), (72, 80, 8, 64, "bf16"), (72, 80, 1, 64, "bf16"),
                                  (33, 41, 3, 33, "fp16")):
        tok = torch.randint(50, (200,), generator=g, device="cuda")
        tok[:70] = 11
        dy = randn(g, (200 * ldy + 16,), "fp16")
        out = torch.full((50 * ldt + 16,), 7.0, dtype=DT[gdt], device="cuda")
        sp = {"tokens": 200, "vocab": 50, "dim": D, "ld_table": ldt, "ld_out": ldy, "out_dtype": "fp16",
              "table_dtype": gdt}
        ws = torch.empty(binding.wg_embedding_workspace_size(sp), dtype=torch.uint8, device="cuda")
        binding.wg_embedding_bwd_weight(sp, tok, dy[off:], out[off:], False, ws)
        got = out[off:off + 50 * ldt].view(50, ldt)
        ref, slack = ref_grad(tok, dy[off:off + 200 * ldy].view(200, ldy)[:, :D], 50, 1.0)
        close(got[:, :D], ref, slack, gdt)
        assert (got[:, D:] == 7).all() and (out[:off] == 7).all() and (out[off + 50 * ldt:] == 7).all()


def test_gradient_of_no_tokens_is_zero():
    out = torch.full((13, 24), float("nan"), device="cuda")
    dy = torch.empty((0, 24), device="cuda")
    binding.embedding_bwd_weight(torch.empty(0, dtype=torch.int64, device="cuda"), dy, 13, out=out)
    assert not out.any()


def test_gradient_is_the_adjoint_of_the_lookup():
    """The difference quotient of sum(lookup * r) along a direction of the table equals <gradient, direction>."""
    g = rng(5)
    T, V, D = 500, 60, 96
    tok = torch.randint(V, (T,), generator=g, device="cuda")
    table, way = randn(g, (V, D), "fp32"), randn(g, (V, D), "fp32")
    r = randn(g, (T, D), "fp32")
    h = 0.5  # the lookup is linear: any step does, and a large one loses nothing
    lo = (binding.embedding_lookup(tok, table - h * way, 1.5).double() * r.double()).sum()
    hi = (binding.embedding_lookup(tok, table + h * way, 1.5).double() * r.double()).sum()
    grad = binding.embedding_bwd_weight(tok, r, V, 1.5)
    inner = (grad.double() * way.double()).sum()
    size = (grad.double().abs() * way.double().abs()).sum() + (r.double().abs() * 10).sum()
    assert abs(float((hi - lo) / (2 * h) - inner)) <= 2.0 ** -20 * float(size)


def test_tables_past_32_bits():
    """2^31 elements lie before the last rows of table and gradient."""
    V, D = 70001, 32000
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    g = rng(6)
    table[-3:] = randn(g, (3, D), "bf16")
    tok = torch.tensor([V - 1, 0, V - 3, V - 2, V - 1], device="cuda")
    out = binding.embedding_lookup(tok, table)
    assert torch.equal(out, table[tok])
    dy = randn(g, (5, D), "bf16")
    table.fill_(float("nan"))
    binding.embedding_bwd_weight(tok, dy, V, out=table)
    two = (dy[0].float() + dy[4].float()).bfloat16()
    assert torch.equal(table[V - 1], two) and torch.equal(table[V - 2], dy[3]) and torch.equal(table[0], dy[1])
    assert not table[1:V - 3].any()


def test_other_stream_and_graph():
    g = rng(7)
    tok = torch.randint(100, (900,), generator=g, device="cuda")
    tok[:300] = 3
    dy = randn(g, (900, 72), "bf16")
    want = binding.embedding_bwd_weight(tok, dy, 100)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = binding.embedding_bwd_weight(tok, dy, 100, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    sp = {"tokens": 900, "vocab": 100, "dim": 72}
    ws = torch.empty(binding.wg_embedding_workspace_size(sp), dtype=torch.uint8, device="cuda")
    out, look = torch.zeros_like(want), torch.zeros_like(dy)
    table = randn(g, (100, 72), "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.wg_embedding_bwd_weight(sp, tok, dy, out, False, ws)
        binding.wg_embedding_lookup(sp, tok, table, look)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(look, table[tok])
