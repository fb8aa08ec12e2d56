"""Calls of the layer operators after one another and in forms that a training step or a server meets, against 64 bits."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import DT, HALF, close, data, forward, keep_mask, weight  # noqa: E402


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


def plan_of(sp, call="forward"):
    return dict(v.split("=") for v in binding.wg_linear_plan_string(sp, call).split())


# Every shape of the few-rows kernel, with more blocks' worth of columns than the GPU holds blocks, and sums longer than the
# 64 MMAs after which a warp puts its sums away.
ROWS = [(1, 8456, 9800, "8 32 8"), (8, 8456, 5000, "8 16 8"), (13, 6400, 5000, "16 16 8"), (13, 10248, 3200, "16 16 8"), (3, 8458, 5000, "8 16 2"),
        (12, 8458, 5000, "16 16 2"), (8, 8457, 9801, "8 32 1"), (5, 8457, 4901, "8 16 1"), (2, 8457, 2500, "8 8 1"),
        (16, 8457, 5001, "16 16 1"), (9, 264, 9801, "16 16 8"), (1, 257, 9801, "8 32 1"), (2, 200, 8200, "8 32 8")]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,inf,out,shape", ROWS)
def test_every_shape_of_few_rows(tokens, inf, out, shape, dt):
    sp = {"tokens": tokens, "in": inf, "out": out, "in_dtype": dt, "out_dtype": "fp32"}
    p = plan_of(sp)
    assert p["kernel"] == "linear_rows" and " ".join((p["rows"], p["columns"], p["access"])) == shape
    x, w = randn(1, tokens, inf, dt=dt), randn(2, out, inf, size=inf ** -0.5, dt=dt)
    bias, y = randn(3, out), torch.full((tokens, out), float("nan"), device="cuda")
    binding.linear(x, w, bias, out=y)
    _, (want, err) = forward(x, w[None], bias[None])
    close(y, want, err, "fp32")


def test_the_shapes_are_all_there():
    assert {s for *_, s in ROWS} == {f"{8 * xr} {8 * fg} {v}" for v in (8, 2, 1) for xr, fg in ((1, 1), (1, 2), (1, 4), (2, 2))
                                     if not (fg == 1 and v > 1) and not (fg == 4 and v == 2)}


@pytest.mark.parametrize("counts,inf,out", [([40] * 6, 264, 2600), ([3, 0, 8, 5], 520, 8200), ([1, 2, 0, 4], 1025, 4901)])
def test_wide_results_of_experts(counts, inf, out):
    """Experts' few rows by 32 columns a block, and tiles of rows for more."""
    off, n = offsets_of(counts), len(counts)
    x, w = randn(1, sum(counts), inf, dt="fp16"), randn(2, n, out, inf, size=inf ** -0.5, dt="fp16")
    y = binding.linear(x, w, activation="gelu", offsets=off)
    _, (want, err) = forward(x, w, activation="gelu", offsets=off.tolist())
    close(y, want, err, "fp16")


LONG = [("forward", 2600, 1100, 2600, None), ("forward", 2600, 3100, 2600, None), ("bwd_data", 2600, 2600, 1100, None),
        ("bwd_data", 2570, 2600, 3130, None), ("bwd_weight", 1100, 2570, 2570, None), ("bwd_weight", 3500, 2568, 2600, None),
        ("bwd_weight", 7100, 1032, 2056, [1030, 40, 0, 2100, 1024, 1025, 1, 1800]),
        ("forward", 1800, 2100, 2056, [500, 0, 3, 257, 700, 256]), ("bwd_data", 1800, 2056, 2100, [500, 0, 3, 257, 700, 256])]


@pytest.mark.parametrize("call,tokens,inf,out,counts", LONG)
def test_sums_of_several_chunks_over_more_tiles_than_pairs(call, tokens, inf, out, counts):
    """fp32 results, whose sums are added up 1024 terms at a time: the buffers of sums and the totals in registers go on
    from one tile of a pair to the next."""
    n, off = len(counts) if counts else 1, offsets_of(counts, 4) if counts else None
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n if counts else 0, "out_dtype": "fp32"}
    p = plan_of(sp, call)
    m, rows = (out, tokens) if call == "forward" else (inf, tokens) if call == "bwd_data" else (inf, n * out)
    assert p["split"] == "1" and int(p["chunks"]) > 1
    assert -(-m // 256) * -(-rows // int(p["rows"])) > int(p["pairs"])
    offs, used = off.tolist() if counts else None, slice(4, 4 + sum(counts)) if counts else slice(0, tokens)
    x, w, dy = randn(1, tokens, inf, dt="bf16"), randn(2, n, out, inf, size=inf ** -0.5, dt="bf16"), randn(3, tokens, out, dt="bf16")
    ws = space(sp, call)
    if call == "forward":
        y = torch.full((tokens, out), 7.0, device="cuda")
        binding.wg_linear(sp, x, w, y, offsets=off, workspace=ws)
        _, (want, err) = forward(x, w, offsets=offs)
    elif call == "bwd_data":
        y = torch.full((tokens, inf), 7.0, device="cuda")
        binding.wg_linear_bwd_data(sp, dy, w, y, offsets=off, workspace=ws)
        want, err = data(dy, w, offsets=offs)
    else:
        y, db = torch.full((n, out, inf), float("nan"), device="cuda"), torch.full((n, out), float("nan"), device="cuda")
        binding.wg_linear_bwd_weight(sp, x, dy, y, db, offsets=off, workspace=ws)
        (want, err), (wb, berr) = weight(x, dy, offs, n)
        close(db, wb, berr, "fp32", "dbias")
        close(y, want, err, "fp32")
        return
    close(y[used], want[used], err[used], "fp32")
    assert bool((y[:used.start] == 7).all()) and bool((y[used.stop:] == 7).all())


@pytest.mark.parametrize("call,tokens,inf,out", [("forward", 1400, 40008, 4100), ("bwd_data", 1400, 4100, 33000),
                                                 ("bwd_weight", 70000, 2300, 2570)])
def test_16_bit_results_of_several_chunks(call, tokens, inf, out):
    """More than 32768 terms to a 16-bit result in whole sums, over more tiles than pairs."""
    sp = {"tokens": tokens, "in": inf, "out": out, "in_dtype": "fp16", "out_dtype": "fp16"}
    p = plan_of(sp, call)
    assert p["split"] == "1" and int(p["chunks"]) > 1
    ws, size = space(sp, call), {"forward": inf, "bwd_data": out, "bwd_weight": tokens}[call] ** -0.5
    if call == "bwd_weight":
        x, dy, y = randn(1, tokens, inf, size=size, dt="fp16"), randn(3, tokens, out, dt="fp16"), torch.empty(1, out, inf, dtype=DT["fp16"], device="cuda")
        binding.wg_linear_bwd_weight(sp, x, dy, y, workspace=ws)
        (want, err), _ = weight(x, dy)
    elif call == "forward":
        x, w, y = randn(1, tokens, inf, dt="fp16"), randn(2, out, inf, size=size, dt="fp16"), torch.empty(tokens, out, dtype=DT["fp16"], device="cuda")
        binding.wg_linear(sp, x, w, y, workspace=ws)
        _, (want, err) = forward(x, w[None])
    else:
        dy, w, y = randn(1, tokens, out, dt="fp16"), randn(2, out, inf, size=size, dt="fp16"), torch.empty(tokens, inf, dtype=DT["fp16"], device="cuda")
        binding.wg_linear_bwd_data(sp, dy, w, y, workspace=ws)
        want, err = data(dy, w[None])
    close(y, want, err, "fp16")


@pytest.mark.parametrize("tokens,terms,out", [(9, 32768, 264), (1400, 32768, 4100), (1400, 40008, 4100), (700, 1000, 264)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_16_bit_sums_of_equal_signs(tokens, terms, out, dt):
    """What truncation takes of a 16-bit result's sum is at most 2e-4 of it, beside its rounding."""
    a, b = 1 + 2.0 ** -5, 1 + 2.0 ** -6
    x, w = torch.full((tokens, terms), a, dtype=DT[dt], device="cuda"), torch.full((out, terms), b, dtype=DT[dt], device="cuda")
    want = a * b * terms
    assert want < 65504
    y = binding.linear(x, w)
    assert float((y.double() / want - 1).abs().max()) <= 2e-4 + HALF[dt] * (1 + 2e-4)
    y = binding.linear_bwd_data(x, w.t().contiguous())
    assert float((y.double() / want - 1).abs().max()) <= 2e-4 + HALF[dt] * (1 + 2e-4)


@pytest.mark.parametrize("xat,wat", [(0, 0), (1, 0), (0, 2), (2, 6), (4, 3)])
@pytest.mark.parametrize("tokens,inf,out,counts", [(1, 512, 72, None), (12, 264, 72, None), (11, 64, 40, [3, 0, 8])])
def test_few_rows_of_aligned_strides_and_other_bases(tokens, inf, out, counts, xat, wat):
    """Strides of whole 16 bytes from a base that is on none: taken by the few-rows kernel, as the header says."""
    n, dt = len(counts) if counts else 1, "bf16"
    xb, wb = torch.full((tokens * inf + 16,), float("nan"), dtype=DT[dt], device="cuda"), torch.full((n * out * inf + 16,), float("nan"), dtype=DT[dt], device="cuda")
    x, w = xb[xat:xat + tokens * inf].view(tokens, inf), wb[wat:wat + n * out * inf].view(n, out, inf)
    x.copy_(randn(1, tokens, inf, dt=dt))
    w.copy_(randn(2, n, out, inf, size=inf ** -0.5, dt=dt))
    off = offsets_of(counts) if counts else None
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n if counts else 0, "out_dtype": "fp32"}
    assert plan_of(sp)["kernel"] == "linear_rows"
    y = torch.empty(tokens, out, device="cuda")
    binding.wg_linear(sp, x, w, y, offsets=off, workspace=space(sp, "forward"))
    _, (want, err) = forward(x, w, offsets=off.tolist() if counts else None)
    close(y, want, err, "fp32")


@pytest.mark.parametrize("kind", ["few", "tiles", "cut", "data", "activation", "gradient"])
def test_a_mask_of_a_counter_at_every_replay(kind):
    """Captured calls whose counter lies in device memory draw the mask of offset + counter, past 2^32 too."""
    t, a, b = (5, 72, 40) if kind == "few" else (20, 4096, 264) if kind == "cut" else (300, 136, 264)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    x, w = torch.ones(t, a, dtype=DT["bf16"], device="cuda"), torch.full((b, a), 1 / a, dtype=DT["bf16"], device="cuda")
    dims = (t, a) if kind in ("data", "activation", "gradient") else (t, b)
    y = torch.empty(dims, dtype=DT["bf16"], device="cuda")
    kw = {"dropout": 0.5, "seed": 11, "offset": (1 << 32) - 3, "counter": counter}
    if kind in ("activation", "gradient"):
        sp = {"tokens": t, "dim": a, **kw}
        call = binding.PreparedActivation(sp, x, y) if kind == "activation" else binding.PreparedActivationBwd(sp, x, None, y)
    elif kind == "data":
        sp = {"tokens": t, "in": a, "out": b, **kw}
        call = binding.PreparedLinearBwdData(sp, torch.ones(t, b, dtype=DT["bf16"], device="cuda"), w, y, workspace=space(sp, "bwd_data"))
    else:
        sp = {"tokens": t, "in": a, "out": b, **kw}
        assert (plan_of(sp)["kernel"] == "linear_rows") == (kind == "few") and (plan_of(sp).get("split", "1") != "1") == (kind == "cut")
        call = binding.PreparedLinear(sp, x, w, y, workspace=space(sp, "forward"))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream().cuda_stream)
        counter += 2
    counter.zero_()
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        mask, _ = keep_mask(11, (1 << 32) - 3 + 2 * i, *dims, 0.5)
        assert torch.equal((y != 0).cpu(), mask)


@pytest.mark.parametrize("kind", ["forward", "bwd_data", "bwd_weight"])
def test_products_behind_calls_that_take_long(kind):
    """Weight gradients on one CTA each, seconds in all, that let the next kernel start early: a product that has started
    waits for them however long they take (its bounded waits are for its own copies and products only)."""
    n, width = 64, 1 << 20
    conv = {"ndim": 1, "G": 1, "N": n, "C": 8, "K": 8, "in": [width], "filt": [1]}
    assert "grid=(1,1,1)" in binding.wg_plan_string(conv, 1, "direct")
    cx, cy = (torch.ones(n * width * 8, dtype=DT["bf16"], device="cuda") for _ in range(2))
    cw = torch.empty(64, device="cuda")

    def run():
        binding.wg_conv_bwd_weight(conv, cx, cy, cw, 1, "direct")
    t, a, b = 300, 264, 136
    x, w, dy = randn(1, t, a, dt="bf16"), randn(2, b, a, size=a ** -0.5, dt="bf16"), randn(3, t, b, dt="bf16")
    sp = {"tokens": t, "in": a, "out": b, "out_dtype": "fp32"}
    shape = {"forward": (t, b), "bwd_data": (t, a), "bwd_weight": (b, a)}[kind]
    y, db, ws = torch.empty(shape, device="cuda"), torch.empty(b, device="cuda"), space(sp, kind)
    call = {"forward": lambda: binding.PreparedLinear(sp, x, w, y, workspace=ws), "bwd_data": lambda: binding.PreparedLinearBwdData(sp, dy, w, y, workspace=ws),
            "bwd_weight": lambda: binding.PreparedLinearBwdWeight(sp, x, dy, y, db, workspace=ws)}[kind]()
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    run()
    ends[0].record()
    run()
    ends[1].record()
    torch.cuda.synchronize()
    count = int(2600 / ends[0].elapsed_time(ends[1])) + 1
    ends[0].record()
    for _ in range(count):
        run()
    call(torch.cuda.current_stream().cuda_stream)
    ends[1].record()
    torch.cuda.synchronize()
    assert ends[0].elapsed_time(ends[1]) > 2200
    binding.wg_check_status()
    if kind == "forward":
        _, (want, err) = forward(x, w[None])
    elif kind == "bwd_data":
        want, err = data(dy, w[None])
    else:
        (want, err), (wb, berr) = weight(x, dy)
        want, err = want[0], err[0]
        close(db, wb[0], berr[0], "fp32", "dbias")
    close(y, want, err, "fp32")
