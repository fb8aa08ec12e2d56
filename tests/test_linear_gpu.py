"""The matrix product with bias, activation, dropout and residual, its gradients, and the same by expert, against the
definition in 64 bits (layer_oracle.py, which derives the tolerances)."""
import pytest

from implicit_gemm_gb300 import binding, build

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from layer_oracle import DT, close, data, forward, weight  # noqa: E402

SEED, OFFSET = 0x1234_5678_9ABC_DEF0, (5 << 32) + 77


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


SIZES = [(1, 64, 64), (1, 8, 8), (3, 64, 256), (8, 4096, 512), (17, 129, 65), (33, 1000, 1000), (64, 64, 1), (5, 1, 7),
         (256, 512, 256), (257, 520, 264), (300, 72, 1030), (1009, 1001, 515), (2048, 576, 1024), (700, 2050, 2050)]


@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp16")])
@pytest.mark.parametrize("tokens,inf,out", SIZES)
def test_product_alone(tokens, inf, out, dt, ydt):
    x, w = randn(1, tokens, inf, dt=dt), randn(2, out, inf, size=inf ** -0.5, dt=dt)
    y = torch.full((tokens, out), float("nan"), dtype=DT[ydt], device="cuda")
    binding.linear(x, w, out=y)
    _, (want, err) = forward(x, w[None])
    close(y, want, err, ydt)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("tokens,inf,out,dt,ydt,bdt", [(1, 256, 512, "bf16", "bf16", "fp32"), (70, 200, 333, "fp16", "fp32", "fp16"),
                                                       (300, 1024, 264, "bf16", "bf16", "bf16"), (4, 8192, 264, "bf16", "fp16", "fp32")])
def test_what_follows(tokens, inf, out, dt, ydt, bdt, act):
    x, w = randn(1, tokens, inf, dt=dt), randn(2, out, inf, size=2 * inf ** -0.5, dt=dt)
    bias, res = randn(3, out, dt=bdt), randn(4, tokens, out, size=2, dt=ydt)
    y, z = binding.linear(x, w, bias, res, act, 0.3, SEED, OFFSET, keep_z=True)
    (v, verr), (want, err) = forward(x, w[None], bias[None], res, act, 0.3, SEED, OFFSET)
    close(z, v, verr, dt, "z")
    close(y, want, err, ydt, "y")
    inplace = res.clone()
    binding.linear(x, w, bias, inplace, act, 0.3, SEED, OFFSET, out=inplace)
    assert torch.equal(inplace, y)


COUNTS = [[0], [1], [5, 0, 3], [0, 0, 64, 64, 0], [1] * 40, [300, 2, 0, 129, 31], [256, 256], [1000, 0, 1, 63, 65, 257]]


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("inf,out,dt", [(64, 64, "bf16"), (200, 264, "fp16"), (130, 77, "bf16"), (1032, 520, "bf16")])
@pytest.mark.parametrize("counts", COUNTS)
def test_experts(counts, inf, out, dt, kind):
    """Rows before the first and behind the last expert are left as they were, and their NaN reach nothing."""
    n, first, behind = len(counts), 3, 5
    off = offsets_of(counts, first, kind)
    rows = int(off[-1]) + behind
    x, w, dy = randn(1, rows, inf, dt=dt), randn(2, n, out, inf, size=inf ** -0.5, dt=dt), randn(3, rows, out, dt=dt)
    bias = randn(4, n, out)
    for t in (x, dy):
        t[:first], t[rows - behind:] = float("nan"), float("inf")
    offs = off.tolist()
    used = slice(first, rows - behind)
    y0 = randn(5, rows, out, dt=dt)
    y, z = y0.clone(), None
    binding.linear(x, w, bias, None, "silu", 0.2, SEED, OFFSET, offsets=off, out=y)
    _, (want, err) = forward(x, w, bias, None, "silu", 0.2, SEED, OFFSET, offs)
    close(y[used], want[used], err[used], dt, "y")
    y[used] = y0[used]
    assert torch.equal(y, y0)
    zin = randn(6, rows, inf, dt=dt)
    dx0 = randn(7, rows, inf, dt=dt)
    dx = dx0.clone()
    binding.linear_bwd_data(dy, w, zin, None, "gelu", 0.1, SEED, OFFSET, offsets=off, out=dx)
    want, err = data(dy, w, zin, None, "gelu", 0.1, SEED, OFFSET, offs)
    close(dx[used], want[used], err[used], dt, "dx")
    dx[used] = dx0[used]
    assert torch.equal(dx, dx0)
    db = torch.full((n, out), float("nan"), device="cuda")
    dw = binding.linear_bwd_weight(x, dy, off, dbias=db)
    (wdw, werr), (wdb, berr) = weight(x, dy, offs, n)
    close(dw, wdw, werr, "fp32", "dw")
    close(db, wdb, berr, "fp32", "dbias")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,inf,out", SIZES)
def test_gradients(tokens, inf, out, dt):
    x, w, dy = randn(1, tokens, inf, dt=dt), randn(2, out, inf, size=out ** -0.5, dt=dt), randn(3, tokens, out, dt=dt)
    dx = torch.full((tokens, inf), float("nan"), device="cuda")
    binding.linear_bwd_data(dy, w, out=dx)
    want, err = data(dy, w[None])
    close(dx, want, err, "fp32", "dx")
    db = torch.full((out,), float("nan"), dtype=DT[dt], device="cuda")
    dw = binding.linear_bwd_weight(x, dy, dbias=db)
    (wdw, werr), (wdb, berr) = weight(x, dy)
    close(dw, wdw[0], werr[0], "fp32", "dw")
    close(db, wdb[0], berr[0], dt, "dbias")
    # Added to what is there.
    start, start_b = randn(4, out, inf, dt=dt), randn(5, out, dt=dt)
    acc, acc_b = start.clone(), start_b.clone()
    binding.linear_bwd_weight(x, dy, out=acc, dbias=acc_b, accumulate=True)
    close(acc, wdw[0] + start.double(), werr[0] + 2.0 ** -23 * (wdw[0].abs() + start.double().abs()), dt, "dw added")
    close(acc_b, wdb[0] + start_b.double(), berr[0] + 2.0 ** -23 * (wdb[0].abs() + start_b.double().abs()), dt, "dbias added")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("tokens,inf,out,dt,xdt", [(5, 512, 4096, "bf16", "bf16"), (70, 333, 200, "fp16", "fp32"),
                                                   (300, 264, 1024, "bf16", "bf16")])
def test_input_gradient_through_the_layer_below(tokens, inf, out, dt, xdt, act):
    w, dy = randn(2, out, inf, size=out ** -0.5, dt=dt), randn(3, tokens, out, dt=dt)
    z, res = randn(4, tokens, inf, size=2, dt=dt), randn(5, tokens, inf, dt=xdt)
    dx = binding.linear_bwd_data(dy, w, z, res, act, 0.25, SEED, OFFSET)
    want, err = data(dy, w[None], z, res, act, 0.25, SEED, OFFSET)
    close(dx, want, err, xdt)


def test_gradients_against_differences():
    """The derivative of sum(y r) along a direction, of the call's own y in fp32: central differences of 64-bit sums."""
    g = {"activation": "silu"}
    x, w, b = randn(1, 40, 96, dt="fp16"), randn(2, 72, 96, size=0.1, dt="fp16"), randn(3, 72, dt="fp32")
    r = randn(4, 40, 72)
    y, z = binding.linear(x, w, b, None, out=torch.empty(40, 72, device="cuda"), keep_z=True, **g)
    dz = binding.activation_bwd(r.half(), z, **g)
    dx = binding.linear_bwd_data(dz, w)
    db = torch.empty(72, device="cuda")
    dw = binding.linear_bwd_weight(x, dz, dbias=db)
    # Steps that are multiples of the types' own steps: x and w move by exact 16-bit amounts.
    for which, grad in ((0, dx), (1, dw), (2, db)):
        d = torch.sign(randn(5 + which, *grad.shape)) * 2.0 ** -6
        ends = []
        for s in (1.0, -1.0):
            args = [x, w, b]
            moved = (args[which].float() + s * d)
            args[which] = moved.to(args[which].dtype)
            out = torch.empty(40, 72, device="cuda")
            binding.linear(args[0], args[1], args[2], out=out, **g)
            ends.append(((out.double() * r.half().double()).sum(), args[which].double()))
        want = float(ends[0][0] - ends[1][0])
        got = float((grad.double() * (ends[0][1] - ends[1][1])).sum())
        # The gradients hold 16-bit roundings (z, dz, dx: 2^-11 of each term, of random sign) and the differences the
        # cubic term of steps of 2^-6: both far below 2% of the sum of the terms' root mean square.
        scale = float(((grad.double() * (ends[0][1] - ends[1][1])) ** 2).sum() ** 0.5)
        assert abs(got - want) < 0.02 * scale + 0.01 * abs(want), (which, got, want, scale)


def test_strides():
    """Rows of larger buffers: aligned and not, experts' matrices apart; what lies between them is left as it was."""
    for pad, dt in ((8, "bf16"), (3, "fp16")):
        t, inf, out, n = 90, 136, 72, 3
        off = offsets_of([40, 0, 45], 2)
        big = lambda s, r, c, d=dt: randn(s, r, c + pad, dt=d)  # noqa: E731
        x, dy, res, z = big(1, t, inf), big(2, t, out), big(3, t, out, "fp32"), big(4, t, inf)
        wbuf = randn(5, n, out + 1, inf + pad, size=0.1, dt=dt)
        bias = randn(6, n, out)
        sp = {"tokens": t, "in": inf, "out": out, "experts": n, "ld_in": inf + pad, "ld_out": out + pad, "ld_weight": inf + pad,
              "weight_stride": (out + 1) * (inf + pad), "ld_z": out + pad, "ld_residual": out + pad, "in_dtype": dt,
              "out_dtype": "fp32", "activation": "gelu", "dropout": 0.15, "seed": SEED, "offset": OFFSET}
        y0, zo0 = big(7, t, out, "fp32"), big(8, t, out)
        y, zo = y0.clone(), zo0.clone()
        ws = lambda s, c: torch.empty(binding.wg_linear_workspace_size(s, c), dtype=torch.uint8, device="cuda")  # noqa: E731
        binding.wg_linear(sp, x, wbuf, y, bias, res, zo, off, ws(sp, "forward"))
        wv = wbuf[:, :out, :inf]
        (v, verr), (want, err) = forward(x[:, :inf], wv, bias, res[:, :out], "gelu", 0.15, SEED, OFFSET, off.tolist())
        u = slice(2, 87)
        close(y[u, :out], want[u], err[u], "fp32")
        close(zo[u, :out], v[u], verr[u], dt)
        y[u, :out], zo[u, :out] = y0[u, :out], zo0[u, :out]
        assert torch.equal(y, y0) and torch.equal(zo, zo0)
        sd = dict(sp, ld_z=inf + pad, ld_residual=inf + pad, out_dtype=dt)
        dx0 = big(9, t, inf)
        dx = dx0.clone()
        binding.wg_linear_bwd_data(sd, dy, wbuf, dx, z, dx, off, ws(sd, "bwd_data"))
        want, err = data(dy[:, :out], wv, z[:, :inf], dx0[:, :inf], "gelu", 0.15, SEED, OFFSET, off.tolist())
        close(dx[u, :inf], want[u], err[u], dt)
        dx[u, :inf] = dx0[u, :inf]
        assert torch.equal(dx, dx0)
        dw0 = randn(10, n, out + 1, inf + pad, dt=dt)
        dw = dw0.clone()
        binding.wg_linear_bwd_weight(sd, x, dy, dw, None, False, off, ws(sd, "bwd_weight"))
        (wdw, werr), _ = weight(x[:, :inf], dy[:, :out], off.tolist(), n)
        close(dw[:, :out, :inf], wdw, werr, dt)
        dw[:, :out, :inf] = dw0[:, :out, :inf]
        assert torch.equal(dw, dw0)


def test_bad_offsets_are_told_and_stay_in_bounds():
    x, w = randn(1, 50, 64, dt="bf16"), randn(2, 4, 72, 64, size=0.1, dt="bf16")
    dy = randn(3, 50, 72, dt="bf16")
    for offs in ([0, 30, 20, 45, 50], [-7, 10, 20, 30, 1000], [60, 61, 62, 63, 64], [5, 4, 3, 2, 1]):
        off = torch.tensor(offs, dtype=torch.int64, device="cuda")
        y = torch.zeros(50, 72, dtype=DT["bf16"], device="cuda")
        binding.linear(x, w, offsets=off, out=y)
        with pytest.raises(binding.WgradError) as e:
            binding.wg_check_status()
        assert e.value.status == 8
        _, (want, err) = forward(x, w, offsets=offs)
        done = torch.isfinite(want).all(1)
        close(y[done], want[done], err[done], "bf16")
        assert not y[~done].any()
        dw = binding.linear_bwd_weight(x, dy, off)
        with pytest.raises(binding.WgradError):
            binding.wg_check_status()
        (wdw, werr), _ = weight(x, dy, offs, 4)
        close(dw, wdw, werr, "fp32")


def test_experts_do_not_touch_one_another():
    """An infinity or a NaN in one expert's rows or weight stays in its results; a row's end inside a block of the sum is
    no way into the next expert's."""
    off = offsets_of([37, 30, 61])
    x, w, dy = randn(1, 128, 192, dt="bf16"), randn(2, 3, 136, 192, size=0.1, dt="bf16"), randn(3, 128, 136, dt="bf16")
    clean = [binding.linear(x, w, offsets=off), binding.linear_bwd_data(dy, w, offsets=off), binding.linear_bwd_weight(x, dy, off)]
    x[37:67], dy[40], w[1, 5, 7] = float("nan"), float("inf"), float("inf")
    dirty = [binding.linear(x, w, offsets=off), binding.linear_bwd_data(dy, w, offsets=off), binding.linear_bwd_weight(x, dy, off)]
    for a, b in zip(clean[:2], dirty[:2]):
        assert torch.equal(a[:37], b[:37]) and torch.equal(a[67:], b[67:]) and not torch.isfinite(b[40]).all()
    assert torch.equal(clean[2][[0, 2]], dirty[2][[0, 2]]) and not torch.isfinite(dirty[2][1]).any()


def test_nothing_to_do():
    x, w = torch.empty(0, 64, dtype=DT["bf16"], device="cuda"), randn(1, 72, 64, dt="bf16")
    assert binding.linear(x, w).shape == (0, 72)
    dy = torch.empty(0, 72, dtype=DT["bf16"], device="cuda")
    assert binding.linear_bwd_data(dy, w).shape == (0, 64)
    db = randn(2, 72)
    dw = binding.linear_bwd_weight(x, dy, dbias=db)
    assert dw.shape == (72, 64) and not dw.any() and not db.any()
    start, db = randn(3, 72, 64), randn(4, 72)
    kept, kept_b = start.clone(), db.clone()
    binding.linear_bwd_weight(x, dy, out=start, dbias=db, accumulate=True)
    assert torch.equal(start, kept) and torch.equal(db, kept_b)


def test_a_feed_forward_block_with_experts():
    """Forward, then every gradient, as a training step makes them: the calls' own intermediate results go on."""
    t, d, h, n = 200, 96, 160, 4
    off = offsets_of([60, 0, 90, 50])
    kw = dict(offsets=off)
    x, w1, w2 = randn(1, t, d, dt="bf16"), randn(2, n, h, d, size=0.1, dt="bf16"), randn(3, n, d, h, size=0.1, dt="bf16")
    b1 = randn(4, n, h)
    a, z = binding.linear(x, w1, b1, activation="gelu_tanh", dropout=0.1, seed=SEED, offset=1, keep_z=True, **kw)
    y = binding.linear(a, w2, residual=x, **kw)
    dy = randn(5, t, d, dt="bf16")
    dz = binding.linear_bwd_data(dy, w2, z, activation="gelu_tanh", dropout=0.1, seed=SEED, offset=1, **kw)
    dw2 = binding.linear_bwd_weight(a, dy, **kw)
    db1 = torch.empty(n, h, device="cuda")
    dw1 = binding.linear_bwd_weight(x, dz, dbias=db1, **kw)
    dx = binding.linear_bwd_data(dz, w1, residual=dy, **kw)
    offs = off.tolist()
    (v, _), (want, err) = forward(x, w1, b1, None, "gelu_tanh", 0.1, SEED, 1, offs)
    close(a, want, err, "bf16")
    _, (want, err) = forward(a, w2, None, x, offsets=offs)
    close(y, want, err, "bf16")
    want, err = data(dy, w2, z, None, "gelu_tanh", 0.1, SEED, 1, offs)
    close(dz, want, err, "bf16")
    (want, err), _ = weight(a, dy, offs, n)
    close(dw2, want, err, "fp32")
    (want, err), (wb, berr) = weight(x, dz, offs, n)
    close(dw1, want, err, "fp32")
    close(db1, wb, berr, "fp32")
    want, err = data(dz, w1, None, dy, offsets=offs)
    close(dx, want, err, "bf16")


def test_long_sums_keep_their_bits():
    """Sums of equal signs: the tensor cores' truncation would take 1e-7 of them per 16 terms."""
    t = 40000
    x, dy = torch.ones(t, 72, dtype=DT["bf16"], device="cuda"), torch.full((t, 64), 1.0 + 2.0 ** -7, dtype=DT["bf16"], device="cuda")
    x *= 1 + 2.0 ** -6
    dw = binding.linear_bwd_weight(x, dy)
    want = t * (1 + 2.0 ** -7) * (1 + 2.0 ** -6)
    assert float((dw.double() / want - 1).abs().max()) < 64 * 2.0 ** -23


def test_captured_calls_and_the_counter():
    """A captured call replays the same; with a counter in device memory each replay draws the mask of its number."""
    x, w = randn(1, 70, 128, dt="bf16"), randn(2, 264, 128, size=0.1, dt="bf16")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    y = torch.empty(70, 264, dtype=DT["bf16"], device="cuda")
    sp = {"tokens": 70, "in": 128, "out": 264, "dropout": 0.5, "seed": SEED, "offset": 9, "counter": counter}
    ws = torch.empty(binding.wg_linear_workspace_size(sp), dtype=torch.uint8, device="cuda")
    call = binding.PreparedLinear(sp, x, w, y, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(s.cuda_stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream().cuda_stream)
        counter += 1
    counter.zero_()
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        _, (want, err) = forward(x, w[None], dropout=0.5, seed=SEED, offset=9 + i)
        close(y, want, err, "bf16")


def test_two_calls_at_once_give_what_they_give_alone():
    x, w = randn(1, 300, 1024, dt="bf16"), randn(2, 2, 520, 1024, size=0.1, dt="bf16")
    want = [binding.linear(x, w[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(binding.linear(x, w[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.parametrize("tokens", [3, 20, 700])
def test_many_experts(tokens):
    """As many experts as there may be, most of them without rows; offsets of 64 bits."""
    n, inf, out = 1024, 64, 40
    g = torch.Generator().manual_seed(tokens)
    count = torch.bincount(torch.randint(n, (tokens,), generator=g), minlength=n)
    off = offsets_of(count.tolist(), 0, torch.int64)
    x, w, dy = randn(1, tokens, inf, dt="bf16"), randn(2, n, out, inf, size=0.1, dt="bf16"), randn(3, tokens, out, dt="bf16")
    bias, offs = randn(4, n, out), off.tolist()
    y = binding.linear(x, w, bias, activation="relu", offsets=off)
    _, (want, err) = forward(x, w, bias, activation="relu", offsets=offs)
    close(y, want, err, "bf16")
    dx = binding.linear_bwd_data(dy, w, offsets=off)
    want, err = data(dy, w, offsets=offs)
    close(dx, want, err, "bf16")
    db = torch.empty(n, out, device="cuda")
    dw = binding.linear_bwd_weight(x, dy, off, dbias=db)
    (want, err), (wb, berr) = weight(x, dy, offs, n)
    close(dw, want, err, "fp32")
    close(db, wb, berr, "fp32")


@pytest.mark.parametrize("counts,inf,out", [([30, 0, 11], 2048, 264), ([2, 90], 4096, 72), ([5000, 1, 3000], 64, 72),
                                            ([0, 6000], 200, 136), ([17], 5000, 257)])
def test_experts_with_cut_sums(counts, inf, out):
    """Few tiles and long sums: the sum is cut among the SMs, of an expert's rows too."""
    n = len(counts)
    off = offsets_of(counts, 1)
    rows = int(off[-1]) + 2
    x, w, dy = randn(1, rows, inf, dt="fp16"), randn(2, n, out, inf, size=inf ** -0.5, dt="fp16"), randn(3, rows, out, dt="fp16")
    x[0], dy[0], x[-2:], dy[-2:] = float("nan"), float("nan"), float("inf"), float("inf")
    sp = {"tokens": rows, "in": inf, "out": out, "experts": n, "in_dtype": "fp16", "out_dtype": "fp16"}
    assert any("split=1 " not in binding.wg_linear_plan_string(sp, c) for c in ("forward", "bwd_weight"))
    offs, used = off.tolist(), slice(1, rows - 2)
    res = randn(4, rows, out, dt="fp16")
    y = binding.linear(x, w, None, res, "gelu_tanh", 0.2, SEED, OFFSET, offsets=off)
    _, (want, err) = forward(x, w, None, res, "gelu_tanh", 0.2, SEED, OFFSET, offs)
    close(y[used], want[used], err[used], "fp16")
    assert not y[0].any() and not y[-2:].any()
    acc = randn(5, n, out, inf)
    start = acc.clone()
    db = torch.empty(n, out, device="cuda")
    binding.linear_bwd_weight(x, dy, off, out=acc, accumulate=True)
    binding.linear_bwd_weight(x, dy, off, out=torch.empty_like(acc), dbias=db)
    (want, err), (wb, berr) = weight(x, dy, offs, n)
    close(acc, want + start.double(), err + 2.0 ** -23 * (want.abs() + start.double().abs()), "fp32")
    close(db, wb, berr, "fp32")


@pytest.mark.parametrize("tokens", [7, 20, 300])
@pytest.mark.parametrize("ydt", ["bf16", "fp32"])
def test_very_long_sums(tokens, ydt):
    inf, out = 40008, 40
    x, w = randn(1, tokens, inf, dt="bf16"), randn(2, out, inf, size=inf ** -0.5, dt="bf16")
    y = torch.empty(tokens, out, dtype=DT[ydt], device="cuda")
    binding.linear(x, w, out=y)
    _, (want, err) = forward(x, w[None])
    close(y, want, err, ydt)
    dx = binding.linear_bwd_data(x, w.t().contiguous(), out=torch.empty(tokens, out, dtype=DT[ydt], device="cuda"))
    close(dx, want, err, ydt)


def test_results_are_the_same_again():
    """Bit for bit, cut sums and bias sums too, and in whatever workspace."""
    x, w, dy = randn(1, 500, 2048, dt="bf16"), randn(2, 264, 2048, size=0.1, dt="bf16"), randn(3, 500, 264, dt="bf16")
    db = [torch.empty(264, device="cuda") for _ in range(2)]
    first = [binding.linear(x, w), binding.linear_bwd_data(dy, w), binding.linear_bwd_weight(x, dy, dbias=db[0]), db[0]]
    torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(0xff)  # what the next workspaces may hold
    again = [binding.linear(x, w), binding.linear_bwd_data(dy, w), binding.linear_bwd_weight(x, dy, dbias=db[1]), db[1]]
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_calls_after_one_another_in_one_workspace():
    """One workspace for calls of one stream, as in a captured training step: packed operands, parts of sums and bias sums
    of each call give way to the next one's."""
    t, a, b = 260, 1001, 135
    x, w, dy = randn(1, t, a, dt="bf16"), randn(2, b, a, size=0.03, dt="bf16"), randn(3, t, b, dt="bf16")
    sp = {"tokens": t, "in": a, "out": b, "out_dtype": "fp32"}
    ws = torch.empty(max(binding.wg_linear_workspace_size(sp, c) for c in binding.LINEAR_CALLS), dtype=torch.uint8, device="cuda")
    out = {k: torch.empty(s, device="cuda") for k, s in (("y", (t, b)), ("dx", (t, a)), ("dw", (b, a)), ("db", (b,)))}
    calls = [binding.PreparedLinear(sp, x, w, out["y"], workspace=ws), binding.PreparedLinearBwdData(sp, dy, w, out["dx"], workspace=ws),
             binding.PreparedLinearBwdWeight(sp, x, dy, out["dw"], dbias=out["db"], workspace=ws)]
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for c in calls:
            c(st.cuda_stream)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for c in calls:
            c(torch.cuda.current_stream().cuda_stream)
    for v in out.values():
        v.fill_(float("nan"))
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    _, (want, err) = forward(x, w[None])
    close(out["y"], want, err, "fp32", "y")
    want, err = data(dy, w[None])
    close(out["dx"], want, err, "fp32", "dx")
    (want, err), (wb, berr) = weight(x, dy)
    close(out["dw"], want[0], err[0], "fp32", "dw")
    close(out["db"], wb[0], berr[0], "fp32", "db")


def test_memory_of_a_call_on_another_stream():
    """The convenience calls' results and workspaces come from their stream's blocks (test_wrapper_streams_gpu.py)."""
    x, w, dy = randn(1, 120, 1001, dt="bf16"), randn(2, 72, 1001, size=0.1, dt="bf16"), randn(3, 120, 72, dt="bf16")
    off = offsets_of([50, 70])
    we = randn(4, 2, 72, 1001, size=0.1, dt="bf16")
    calls = [lambda **k: binding.linear(x, w, activation="gelu", **k), lambda **k: binding.linear(x, we, offsets=off, **k),
             lambda **k: binding.linear_bwd_data(dy, w, **k), lambda **k: binding.linear_bwd_weight(x, dy, **k),
             lambda **k: binding.activation(x, activation="silu", dropout=0.1, **k),
             lambda **k: binding.activation_bwd(x, x, activation="silu", **k)]
    for f in calls:
        want = f().clone()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        s = torch.cuda.Stream()
        torch.cuda._sleep(50_000_000)
        blocks = [torch.empty_like(want) for _ in range(2)] + [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(4)]
        for block in blocks:
            block.fill_(77)
        del block, blocks
        got = f(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("xat,wat", [(0, 0), (2, 4), (1, 0), (0, 3), (5, 7)])
@pytest.mark.parametrize("tokens,inf,out,pad,counts", [(1, 1000, 130, 0, None), (1, 1002, 130, 2, None), (1, 1001, 67, 0, None),
                                                       (7, 70, 200, 1, None), (13, 515, 72, 1, None), (16, 1030, 72, 4, None),
                                                       (2, 7, 9, 1, None), (3, 1, 5, 0, None), (9, 518, 40, 0, [3, 0, 5]),
                                                       (15, 261, 33, 2, [0, 14]), (8, 264, 24, 0, [1, 1, 1, 4])])
def test_few_rows_that_start_anywhere(tokens, inf, out, pad, counts, xat, wat):
    """Rows of even and odd lengths, starts and strides, for one weight and for experts'; NaN all around them."""
    n = len(counts) if counts else 1
    ld, wstride = inf + pad, out * (inf + pad) + 3
    aligned = ld % 8 == 0 and (n == 1 or wstride % 8 == 0)
    if aligned and (xat or wat):
        xat, wat = 8 * xat, 8 * wat
    xb, wb = (torch.full((k,), float("nan"), dtype=DT["fp16"], device="cuda") for k in (64 + tokens * ld, 64 + n * wstride))
    x = torch.as_strided(xb, (tokens, inf), (ld, 1), xat)
    w = torch.as_strided(wb, (n, out, inf), (wstride, ld, 1), wat)
    x.copy_(randn(1, tokens, inf, dt="fp16"))
    w.copy_(randn(2, n, out, inf, size=inf ** -0.5, dt="fp16"))
    off = offsets_of(counts) if counts else None
    y = torch.full((tokens, out), 7.0, device="cuda")
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": n if counts else 0, "ld_in": ld, "ld_weight": ld,
          "weight_stride": wstride, "in_dtype": "fp16", "out_dtype": "fp32"}
    assert "linear_rows" in binding.wg_linear_plan_string(sp)
    binding.wg_linear(sp, x, w, y, offsets=off, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    _, (want, err) = forward(x, w, offsets=off.tolist() if counts else None)
    used = slice(0, sum(counts) if counts else tokens)
    close(y[used], want[used], err[used], "fp32")
    assert bool((y[used.stop:] == 7).all())


@pytest.mark.parametrize("counts", [[0, 40, 0, 0, 61, 0], [0, 0, 0], [17, 0, 0, 0, 0, 0, 0, 90]])
def test_weights_of_experts_without_rows_are_not_read(counts):
    """Unaligned weights go through copies, of the experts that have rows only; the others' may hold anything."""
    n, inf, out = len(counts), 333, 77
    off = offsets_of(counts, 4)
    rows = int(off[-1]) + 40
    x, dy, w = randn(1, rows, inf, dt="bf16"), randn(2, rows, out, dt="bf16"), randn(3, n, out, inf, size=0.05, dt="bf16")
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")
    offs, used = off.tolist(), slice(4, rows - 40)
    y = binding.linear(x, w, offsets=off)
    _, (want, err) = forward(x, w, offsets=offs)
    close(y[used], want[used], err[used], "bf16")
    dx = binding.linear_bwd_data(dy, w, offsets=off)
    want, err = data(dy, w, offsets=offs)
    close(dx[used], want[used], err[used], "bf16")


@pytest.mark.parametrize("tokens,inf,out,experts", [(5000, 64, 264, 0), (3000, 520, 640, 0), (5000, 96, 333, 7), (600, 136, 1000, 0),
                                                    (2500, 72, 2000, 40), (4100, 1001, 77, 0)])
def test_gradients_of_what_the_call_before_wrote(tokens, inf, out, experts):
    """dy, dw and dbias are written and read by one call after another without a pause, as in a captured step: the results
    are those of calls that wait for each other."""
    off = offsets_of([tokens // experts] * experts, 1) if experts else None
    n = max(experts, 1)
    x, w = randn(1, tokens, inf, dt="bf16"), randn(2, n, out, inf, size=0.1, dt="bf16")
    zs, gs = [randn(3 + i, tokens, out, dt="bf16") for i in range(2)], [randn(5 + i, tokens, out, dt="bf16") for i in range(2)]
    dy, dw, db = torch.empty_like(zs[0]), torch.empty(n, out, inf, device="cuda"), torch.empty(n, out, device="cuda")
    dx = torch.zeros(tokens, inf, dtype=DT["bf16"], device="cuda")
    sa = {"tokens": tokens, "dim": out, "activation": "silu"}
    sp = {"tokens": tokens, "in": inf, "out": out, "experts": experts, "out_dtype": "fp32"}
    sd = dict(sp, out_dtype="bf16")
    ws = torch.empty(max(binding.wg_linear_workspace_size(sp, "bwd_weight"), binding.wg_linear_workspace_size(sd, "bwd_data")),
                     dtype=torch.uint8, device="cuda")
    calls = []
    for i in range(2):
        calls += [binding.PreparedActivationBwd(sa, gs[i], zs[i], dy),
                  binding.PreparedLinearBwdWeight(sp, x, dy, dw, dbias=db, accumulate=i == 1, offsets=off, workspace=ws),
                  binding.PreparedLinearBwdData(sd, dy, w, dx, offsets=off, workspace=ws)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in calls:
        c(st.cuda_stream)
        torch.cuda.synchronize()
    want = [t.clone() for t in (dw, db, dx)]
    for t in (dw, db, dx, dy):
        t.fill_(float("nan") if t is not dx else 0.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            c(st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dw, db, dx), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c(torch.cuda.current_stream().cuda_stream)
    for t in (dw, db, dx, dy):
        t.fill_(float("nan") if t is not dx else 0.0)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dw, db, dx), want))
    (wdw, werr), (wdb, berr) = [0, 0], [0, 0]
    for i in range(2):
        d = binding.activation_bwd(gs[i], zs[i], activation="silu")
        (a, b), (c, e) = weight(x, d, off.tolist() if experts else None, n)
        wdw, werr, wdb, berr = wdw + a, werr + b, wdb + c, berr + e
    close(dw, wdw, werr + 2.0 ** -22 * wdw.abs() + 2.0 ** -23 * werr, "fp32", "dw")
    close(db, wdb, berr + 2.0 ** -22 * wdb.abs(), "fp32", "dbias")


@pytest.mark.parametrize("counts", [[64, 0, 0, 0, 0, 0, 0, 0], [0, 7, 9, 0, 17, 8, 0, 22], [1] * 8, [20, 0, 21]])
def test_few_rows_of_experts_with_unaligned_weights(counts):
    """Up to 64 rows, of one expert or of many, in passes of eight."""
    n, inf, out, rows = len(counts), 517, 90, sum(counts)
    off = offsets_of(counts)
    x, w, bias, res = randn(1, rows, inf, dt="bf16"), randn(2, n, out, inf, size=0.05, dt="bf16"), randn(3, n, out), randn(4, rows, out, dt="bf16")
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")
    y, z = binding.linear(x, w, bias, res, "gelu_tanh", 0.2, SEED, OFFSET, offsets=off, keep_z=True)
    (v, verr), (want, err) = forward(x, w, bias, res, "gelu_tanh", 0.2, SEED, OFFSET, off.tolist())
    close(z, v, verr, "bf16", "z")
    close(y, want, err, "bf16", "y")
