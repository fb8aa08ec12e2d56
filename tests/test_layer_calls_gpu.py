"""Calls of the layer operators after one another and in forms that a training step or a server meets, against 64 bits."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import DT, close, forward, weight  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    build.build()
    binding.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    binding.wg_check_status()


def randn(seed, *shape, size=1.0, dt="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(shape, generator=g, device="cuda")).to(DT[dt])


def offsets_of(counts, first=0, kind=torch.int32):
    return torch.tensor([first] + counts).cumsum(0).to(kind).cuda()


def space(sp, call):
    return torch.empty(binding.wg_linear_workspace_size(sp, call), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("last", ["offsets", "dw", "dbias", "dy"])
@pytest.mark.parametrize("tokens,inf,out,counts", [(512, 1024, 1000, None), (600, 136, 333, ([200, 0, 393], [1, 500, 77])),
                                                   (1000, 72, 2000, ([100] * 10, [1] * 9 + [900])), (1009, 1001, 130, None), (1500, 264, 520, None),
                                                   (5000, 96, 333, ([1000, 2000, 2000], [4000, 0, 999])), (4100, 64, 72, None)])
def test_weight_gradient_of_what_the_call_before_wrote(tokens, inf, out, counts, last):
    """offsets, dw, dbias and dy are all written anew right before the call that reads them (by kernels of this library,
    which let the next one start early), each in turn by the very last one: as with a pause after every call."""
    n = len(counts[0]) if counts else 1
    offs = [offsets_of(c) for c in counts] if counts else [None, None]
    off = torch.empty_like(offs[0]) if counts else None
    x = randn(1, tokens, inf, dt="bf16")
    dys, dbs = [randn(2 + i, tokens, out, dt="bf16") for i in range(2)], [randn(4 + i, n, out) for i in range(2)]
    a, b = [randn(6 + i, n * out, 64, dt="bf16") for i in range(2)], randn(8, inf, 64, dt="bf16")
    dy, dw, db = torch.empty_like(dys[0]), torch.empty(n, out, inf, device="cuda"), torch.empty(n, out, device="cuda")
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n if counts else 0, "out_dtype": "fp32"}
    sw = {"tokens": n * out, "in": 64, "out": inf, "out_dtype": "fp32"}
    ws, wy = space(sp, "bwd_weight"), space(sw, "forward")

    def copy(src, dst):  # (fp32 values as they are; offsets as the bits of such)
        src, dst = src.view(1, -1), dst.view(1, -1)
        dt = "bf16" if src.dtype == torch.bfloat16 else "fp32"
        return binding.PreparedActivation({"tokens": 1, "dim": src.numel(), "in_dtype": dt, "out_dtype": dt}, src, dst) \
            if src.numel() <= 1 << 20 else binding.PreparedActivation(
                {"tokens": tokens, "dim": out, "in_dtype": dt, "out_dtype": dt}, src, dst)
    rounds = []
    for i in range(2):
        first = {"dw": binding.PreparedLinear(sw, a[i], b, dw, workspace=wy), "dbias": copy(dbs[i], db), "dy": copy(dys[i], dy)}
        if counts:
            first["offsets"] = copy(offs[i], off)
        order = [k for k in first if k != last] + [k for k in first if k == last]
        rounds.append([first[k] for k in order] + [binding.PreparedLinearBwdWeight(sp, x, dy, dw, db, True, off, workspace=ws)])
    st, want = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for calls in rounds:
        for c in calls:
            c(st.cuda_stream)
            torch.cuda.synchronize()
        want.append((dw.clone(), db.clone()))
        assert not counts or torch.equal(off, offs[len(want) - 1])
    kept = [[(torch.empty_like(dw), torch.empty_like(db)) for _ in range(2)] for _ in range(6)]
    with torch.cuda.stream(st):
        for pair in kept:
            for calls, (w, v) in zip(rounds, pair):
                for c in calls:
                    c(st.cuda_stream)
                w.copy_(dw)
                v.copy_(db)
        for _ in range(10):  # and without anything else between
            for calls in rounds:
                for c in calls:
                    c(st.cuda_stream)
    torch.cuda.synchronize()
    for pair in kept + [[want[0], (dw, db)]]:
        for (w, v), (ww, vv) in zip(pair, want):
            assert torch.equal(w, ww) and torch.equal(v, vv)
    for i in range(2):
        (wd, werr), (wb, berr) = weight(x, dys[i], offs[i].tolist() if counts else None, n)
        start = (a[i].double() @ b.double().T).view_as(wd)
        serr = (a[i].double().abs() @ b.double().abs().T).view_as(wd) * 2.0 ** -18  # (64 terms in fp32)
        close(want[i][0], wd + start, werr + serr + 2.0 ** -23 * (wd.abs() + start.abs()), "fp32", "dw")
        close(want[i][1], wb + dbs[i].double(), berr + 2.0 ** -23 * (wb.abs() + dbs[i].double().abs()), "fp32", "dbias")


@pytest.mark.parametrize("dt,bdt", [("bf16", "fp32"), ("fp16", "fp16"), ("bf16", "bf16")])
@pytest.mark.parametrize("tokens,inf,out,counts", [(1, 64, 8, None), (1, 64, 1, None), (63, 40, 65, None), (64, 64, 64, None),
                                                   (65, 200, 72, None), (512, 64, 1001, None), (513, 64, 1001, None),
                                                   (1024, 72, 264, None), (1025, 72, 264, None), (2048, 136, 2000, None), (2049, 136, 264, None), (2048, 72, 333, [9, 0, 1900, 0]), (1002, 64, 136, [0, 1000, 0]),
                                                   (300, 64, 8200, [7, 0, 290]), (1024, 64, 40, [16] * 63), (900, 64, 24, [0, 0])])
def test_bias_sums_of_few_rows(tokens, inf, out, counts, dt, bdt):
    """Around the sizes where the sums are the product's own; experts without rows; added to what is there, which an
    expert without rows leaves as it is."""
    n = len(counts) if counts else 1
    off = offsets_of(counts, 2) if counts else None
    x, dy, start = randn(1, tokens, inf, dt=dt), randn(2, tokens, out, dt=dt), randn(3, n, out, dt=bdt)
    if counts:
        dy[:2], dy[int(off[-1]):] = float("nan"), float("inf")
        x[:2], x[int(off[-1]):] = float("nan"), float("inf")
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n if counts else 0, "in_dtype": dt, "out_dtype": "fp32", "bias_dtype": bdt}
    dw, db, ws = torch.full((n, out, inf), float("nan"), device="cuda"), torch.full_like(start, float("nan")), space(sp, "bwd_weight")
    binding.wg_linear_bwd_weight(sp, x, dy, dw, db, offsets=off, workspace=ws)
    (wd, werr), (wb, berr) = weight(x, dy, off.tolist() if counts else None, n)
    close(dw, wd, werr, "fp32", "dw")
    close(db, wb, berr, bdt, "dbias")
    acc = start.clone()
    binding.wg_linear_bwd_weight(sp, x, dy, dw, acc, True, offsets=off, workspace=ws)
    close(dw, 2 * wd, 2 * werr + 2.0 ** -22 * wd.abs(), "fp32", "dw added")
    close(acc, wb + start.double(), berr + 2.0 ** -23 * (wb.abs() + start.double().abs()), bdt, "dbias added")
    for e, c in enumerate(counts or []):
        assert c or torch.equal(acc[e], start[e])


@pytest.mark.parametrize("tokens,inf,out,pad,dt", [(5, 64, 72, 0, "bf16"), (90, 136, 72, 8, "bf16"), (700, 264, 520, 8, "fp16"),
                                                   (13, 65, 71, 1, "fp16"), (300, 129, 333, 3, "bf16")])
def test_columns_of_one_buffer(tokens, inf, out, pad, dt):
    """x | y | z | residual as columns of one buffer: each call writes its own and nothing beside them."""
    cols = {"x": inf, "y": out, "z": out, "res": out, "dx": inf}
    at, o = {}, pad
    for k, c in cols.items():
        at[k], o = slice(o, o + c), o + c + pad
    start = randn(1, tokens, o, dt=dt)
    buf, w, bias = start.clone(), randn(2, out, inf, size=inf ** -0.5, dt=dt), randn(3, out)
    v = {k: buf[:, s] for k, s in at.items()}
    kw = dict(activation="silu", dropout=0.2, seed=3, offset=4)
    sp = {"tokens": tokens, "in": inf, "out": out, "ld_in": o, "ld_out": o, "ld_z": o, "ld_residual": o, "in_dtype": dt,
          "out_dtype": dt, **kw}
    x, res = start[:, at["x"]].contiguous(), start[:, at["res"]].contiguous()
    wy, wz = binding.linear(x, w, bias, res, keep_z=True, **kw)
    binding.wg_linear(sp, v["x"], w, v["y"], bias, v["res"], v["z"], None, space(sp, "forward"))
    want = start.clone()
    want[:, at["y"]], want[:, at["z"]] = wy, wz
    assert torch.equal(buf, want)
    wdx = binding.linear_bwd_data(wy, w, x, **kw)
    binding.wg_linear_bwd_data(sp, v["y"], w, v["dx"], v["x"], None, None, space(sp, "bwd_data"))
    want[:, at["dx"]] = wdx
    assert torch.equal(buf, want)
    sa = {"tokens": tokens, "dim": out, "ld_x": o, "ld_y": o, "ld_residual": o, "ld_dx": o, "in_dtype": dt, "out_dtype": dt, **kw}
    wa = binding.activation(wz, bias, res, **kw)
    binding.wg_activation(sa, v["z"], v["y"], bias, v["res"])
    want[:, at["y"]] = wa
    assert torch.equal(buf, want)
    wd = binding.activation_bwd(res, wz, bias, **kw)
    binding.wg_activation_bwd(sa, v["res"], v["z"], v["y"], bias)
    want[:, at["y"]] = wd
    assert torch.equal(buf, want)


@pytest.mark.parametrize("counts,inf,out", [([1] * 64, 261, 40), ([9] * 7 + [0], 130, 77), ([64] + [0] * 7, 333, 600), ([0] * 1000 + [33, 0, 31], 65, 24),
                                            ([16], 264, 72), ([9, 7], 1024, 264), ([0] * 500 + [16], 72, 40), ([8, 0, 8], 4096, 72),
                                            ([17, 0, 30, 16, 0, 0, 0, 0], 2050, 99), ([0] * 9, 261, 40)])
def test_few_rows_in_passes(counts, inf, out):
    """As many passes as there may be, experts of one row more or less than a pass takes."""
    n = len(counts)
    off = offsets_of(counts, 0)
    rows = sum(counts) or 7
    x, w, bias = randn(1, rows, inf, dt="bf16"), randn(2, n, out, inf, size=inf ** -0.5, dt="bf16"), randn(3, n, out)
    sp = {"tokens": rows, "in": inf, "out": out, "experts": n}
    assert "linear_rows" in binding.wg_linear_plan_string(sp)
    y = torch.full((rows, out), 7.0, dtype=DT["bf16"], device="cuda")
    binding.linear(x, w, bias, activation="silu", dropout=0.2, seed=3, offset=4, offsets=off, out=y)
    _, (want, err) = forward(x, w, bias, None, "silu", 0.2, 3, 4, off.tolist())
    used = slice(0, sum(counts))
    close(y[used], want[used], err[used], "bf16")
    assert bool((y[used.stop:] == 7).all())
