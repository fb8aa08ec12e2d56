"""Host-side checks of the layer entry points (no GPU needed): sizes, plans and refusals.  Only calls that fail
validation are made here, so nothing is launched."""
import ctypes
import math
import random

import pytest

from implicit_gemm_gb300 import binding, build

A = 1 << 24  # stands for a device address; refused before it is used
CALLS = ("forward", "bwd_data", "bwd_weight")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def lin(**kw):
    sp = {"tokens": 20, "in": 64, "out": 72, **kw}
    if "in_" in sp:
        sp["in"] = sp.pop("in_")
    return sp


def act(**kw):
    return {"tokens": 20, "dim": 64, **kw}


def refused(status, f, *a, **kw):
    with pytest.raises(binding.WgradError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value
    assert binding.wg_last_error()


def calls(sp, at=A, **kw):
    big = {"workspace": 15 * A, "ws_bytes": 1 << 40, "stream": 0, "offsets": 14 * A if sp.get("experts") else None, **kw}
    yield lambda: binding.wg_linear(sp, at, 2 * A, 3 * A, **big)
    yield lambda: binding.wg_linear_bwd_data(sp, at, 2 * A, 3 * A, z=4 * A, **big)
    yield lambda: binding.wg_linear_bwd_weight(sp, at, 2 * A, 3 * A, **big)


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=-1), 1), (dict(in_=0), 1), (dict(out=-3), 1), (dict(experts=-1), 1), (dict(tokens=(1 << 31) - 65535), 2),
    (dict(in_=(1 << 20) + 1), 2), (dict(out=(1 << 20) + 1), 2), (dict(experts=1025), 2), (dict(in_dtype="fp32"), 1),
    (dict(ld_in=63), 1), (dict(ld_out=71), 1), (dict(ld_weight=63), 1), (dict(experts=2, weight_stride=64 * 71), 1),
    (dict(dropout=1.0), 1), (dict(dropout=-0.1), 1), (dict(dropout=math.nan), 1), (dict(ld_in=1 << 45), 1),
    (dict(ld_weight=1 << 45), 1), (dict(experts=1024, weight_stride=1 << 40), 1), (dict(ld_z=3), 1), (dict(ld_residual=3), 1),
    (dict(tokens=(1 << 31) - 65536, in_=1 << 20, out=1 << 20), 1), (dict(counter=4), 3),
])
def test_linear_problem_refusals(bad, status):
    for call, run in zip(CALLS, calls(lin(**bad))):
        refused(status, binding.wg_linear_workspace_size, lin(**bad), call)
        refused(status, run)


def test_enumerations_are_checked():
    lib = binding.load()
    p, n = binding.make_linear_problem(lin()), ctypes.c_size_t(0)
    for field, value in (("activation", 5), ("activation", -1), ("in_dtype", 7), ("out_dtype", 3), ("bias_dtype", -1),
                         ("offset_bits", 16)):
        q = binding.make_linear_problem(lin())
        setattr(q, field, value)
        assert lib.wg_linear_workspace_size(ctypes.byref(q), 0, ctypes.byref(n)) == 1
    for call in (-1, 3):
        assert lib.wg_linear_workspace_size(ctypes.byref(p), call, ctypes.byref(n)) == 1
    assert lib.wg_linear_workspace_size(None, 0, ctypes.byref(n)) == 1
    assert lib.wg_linear_workspace_size(ctypes.byref(p), 0, None) == 1
    a = binding.make_activation_problem(act())
    a.activation = 9
    assert lib.wg_activation_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 1
    assert lib.wg_activation_workspace_size(None, ctypes.byref(n)) == 1


def test_linear_buffer_refusals():
    sp, big = lin(), {"workspace": 15 * A, "ws_bytes": 1 << 30, "stream": 0}
    f, d, w = binding.wg_linear, binding.wg_linear_bwd_data, binding.wg_linear_bwd_weight
    for args in ((0, 2 * A, 3 * A), (A, 0, 3 * A), (A, 2 * A, 0)):
        for call in (f, d, w):
            refused(1, call, sp, *args, **big)
    # Operands whose rows are on 16 bytes start on 16 bytes; others on their elements, as everything else.
    refused(3, f, sp, A + 2, 2 * A, 3 * A, **big)
    refused(3, f, sp, A, 2 * A + 8, 3 * A, **big)
    refused(3, d, sp, A + 2, 2 * A, 3 * A, **big)
    refused(3, w, sp, A, 2 * A + 2, 3 * A, **big)
    refused(3, f, sp, A, 2 * A, 3 * A + 1, **big)
    refused(3, f, lin(out_dtype="fp32"), A, 2 * A, 3 * A + 2, **big)
    refused(3, f, sp, A, 2 * A, 3 * A, bias=4 * A + 2, **big)
    refused(3, f, sp, A, 2 * A, 3 * A, z=4 * A + 1, **big)
    refused(3, f, sp, A, 2 * A, 3 * A, **{**big, "workspace": 15 * A + 8})
    refused(3, f, lin(experts=1), A, 2 * A, 3 * A, offsets=4 * A + 2, **big)
    refused(3, f, lin(experts=1, offset_dtype="i64"), A, 2 * A, 3 * A, offsets=4 * A + 4, **big)
    # Offsets go with experts.
    refused(1, f, lin(experts=2), A, 2 * A, 3 * A, **big)
    refused(1, f, sp, A, 2 * A, 3 * A, offsets=4 * A, **big)
    # An activation's gradient needs z.
    refused(1, d, lin(activation="gelu"), A, 2 * A, 3 * A, **big)
    # Outputs share nothing with other tensors, but for a residual that is the output.
    nx, nw, ny = 20 * 64 * 2, 72 * 64 * 2, 20 * 72 * 2
    refused(1, f, sp, A, 2 * A, A + nx - 2, **big)
    refused(1, f, sp, A, 2 * A, 2 * A + nw - 2, **big)
    refused(1, f, sp, A, 2 * A, 3 * A, residual=3 * A + 2, **big)
    refused(1, f, sp, A, 2 * A, 3 * A, z=3 * A + ny - 2, **big)
    refused(1, f, sp, A, 2 * A, 3 * A, z=A, **big)
    refused(1, f, sp, A, 2 * A, 3 * A, bias=3 * A, **big)
    refused(1, f, lin(ld_residual=80), A, 2 * A, 3 * A, residual=3 * A, **big)
    refused(1, f, lin(counter=3 * A), A, 2 * A, 3 * A, **big)
    refused(1, d, sp, A, 2 * A, A, **big)
    refused(1, d, lin(activation="relu"), A, 2 * A, 3 * A, z=3 * A, **big)
    refused(1, w, sp, A, 2 * A, A, **big)
    refused(1, w, sp, A, 2 * A, 3 * A, dbias=3 * A + 4, **big)
    refused(1, w, lin(experts=1), A, 2 * A, 3 * A, offsets=3 * A, **big)
    for call, run in (("forward", f), ("bwd_data", d), ("bwd_weight", w)):
        refused(4, run, sp, A, 2 * A, 3 * A, workspace=15 * A, ws_bytes=binding.wg_linear_workspace_size(sp, call) - 1, stream=0)
        refused(4, run, sp, A, 2 * A, 3 * A, stream=0)


def test_activation_refusals():
    big = {"workspace": 15 * A, "ws_bytes": 1 << 30, "stream": 0}
    f, b = binding.wg_activation, binding.wg_activation_bwd
    for bad, status in ((dict(tokens=-1), 1), (dict(dim=0), 1), (dict(tokens=(1 << 31) - 65535), 2), (dict(dim=(1 << 20) + 1), 2),
                        (dict(ld_x=63), 1), (dict(ld_y=63), 1), (dict(ld_dx=63), 1), (dict(ld_residual=1), 1),
                        (dict(ld_x=1 << 45), 1), (dict(dropout=1.0), 1), (dict(dropout=math.nan), 1), (dict(counter=12), 3)):
        refused(status, binding.wg_activation_workspace_size, act(**bad))
        refused(status, f, act(**bad), A, 2 * A, stream=0)
        refused(status, b, act(**bad), A, 2 * A, 3 * A, **big)
    sp = act(activation="silu")
    refused(1, f, sp, 0, A, stream=0)
    refused(1, f, sp, A, 0, stream=0)
    refused(1, b, sp, 0, A, 2 * A, **big)
    refused(1, b, sp, A, 0, 2 * A, **big)
    refused(1, b, sp, A, 2 * A, 0, **big)
    refused(3, f, sp, A + 1, 2 * A, stream=0)
    refused(3, b, sp, A, 2 * A, 3 * A, dbias=4 * A + 2, **big)
    refused(1, f, sp, A, A + 2, stream=0)
    refused(1, f, act(out_dtype="fp16"), A, A, stream=0)          # types of one size are not one type
    refused(1, f, sp, A, 2 * A, residual=2 * A + 64, stream=0)
    refused(1, f, sp, A, 2 * A, bias=2 * A, stream=0)
    refused(1, f, act(ld_y=72), A, A, stream=0)
    refused(1, b, act(out_dtype="fp16", activation="silu"), A, 2 * A, A, **big)
    refused(1, b, sp, A, 2 * A, 3 * A, dbias=3 * A, **big)
    refused(4, b, sp, A, 2 * A, 3 * A, dbias=4 * A, stream=0)
    refused(4, b, sp, A, 2 * A, 3 * A, dbias=4 * A, workspace=15 * A, ws_bytes=8, stream=0)


def test_plans_of_random_problems():
    """What the kernels rely on: tiles of 32 to 256 rows in steps of 32, a ring of at least two stages inside the shared
    memory of a CTA, and a workspace that holds the parts."""
    rng = random.Random(3)
    log = lambda hi: int(math.exp(rng.uniform(0, math.log(hi))))  # noqa: E731
    for _ in range(400):
        sp = lin(tokens=log(1 << 20), in_=log(1 << 15), out=log(1 << 15), experts=rng.choice([0, 0, log(1024)]))
        for call in CALLS:
            plan = dict(v.split("=") for v in binding.wg_linear_plan_string(sp, call).split())
            if plan["kernel"] == "linear_rows":
                copied = sp["in"] % 8 != 0 and sp["tokens"] <= min(64, 8 * sp["experts"])
                assert call == "forward" and (sp["tokens"] <= 16 or copied)
                continue
            rows, split, stages = int(plan["rows"]), int(plan["split"]), int(plan["stages"])
            assert rows % 32 == 0 and 32 <= rows <= 256 and 1 <= split <= 16 and 2 <= stages <= 12
            cols = sp["out"] if call == "forward" else sp["in"]
            held = max(sp["experts"], 1) * sp["out"] if call == "bwd_weight" else sp["tokens"]
            assert int(plan["ws"]) == binding.wg_linear_workspace_size(sp, call)
            assert split == 1 or int(plan["ws"]) >= split * held * cols * 4
    assert binding.wg_linear_workspace_size(lin(tokens=0), "bwd_weight") >= 256


def test_more_tiles_than_one_launch_covers():
    for call in ("forward", "bwd_data"):
        refused(2, binding.wg_linear_workspace_size, lin(tokens=1 << 28, in_=1 << 20, out=1 << 20), call)
    refused(2, binding.wg_linear_workspace_size, lin(in_=1 << 20, out=1 << 20, experts=128), "bwd_weight")


def test_status_string():
    assert binding.wg_status_string(8) == "WG_ERR_INVALID_OFFSET"


def test_convenience_calls_refuse_what_does_not_fit():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 64), torch.zeros(72, 64)
    with pytest.raises(ValueError):
        binding.linear(x.double(), w)
    for bad in (dict(w=torch.zeros(72, 63)), dict(w=torch.zeros(2, 72, 64)), dict(bias=torch.zeros(71)), dict(activation="tanh"),
                dict(offsets=torch.zeros(3, dtype=torch.int32))):
        kw = {"w": w.bfloat16(), **bad}
        kw["w"] = kw["w"].bfloat16()
        with pytest.raises(ValueError):
            binding.linear(x.bfloat16(), kw.pop("w"), **kw)
    with pytest.raises(ValueError):  # not on a GPU
        binding.linear(x.bfloat16(), w.bfloat16())
    with pytest.raises(ValueError):
        binding.activation(x, counter=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.linear_bwd_weight(x.bfloat16(), torch.zeros(5, 72).bfloat16())
    with pytest.raises(ValueError):
        binding.linear_bwd_weight(x.bfloat16(), torch.zeros(4, 72).bfloat16(), accumulate=True)


def no_gpu():
    """Whether no CUDA device is there: then a call that passes validation reaches the driver's refusal and nothing else."""
    torch = pytest.importorskip("torch")
    return not torch.cuda.is_available()


@pytest.mark.parametrize("sp,f", [
    (lin(in_=65), lambda sp, kw: binding.wg_linear(sp, A, 2 * A, 3 * A, **kw)),
    (lin(out=71), lambda sp, kw: binding.wg_linear_bwd_data(sp, A, 2 * A, 3 * A, **kw)),
    (lin(tokens=5000), lambda sp, kw: binding.wg_linear_bwd_weight(sp, A, 2 * A, 3 * A, dbias=4 * A, accumulate=True, **kw)),
    (lin(tokens=5000, in_=65), lambda sp, kw: binding.wg_linear_bwd_weight(sp, A, 2 * A, 3 * A, dbias=4 * A, **kw))])
def test_what_may_fail_comes_before_the_first_launch(sp, f):
    """Without a driver the tensor maps cannot be made: the call ends there, with no launch tried before."""
    if not no_gpu():
        pytest.skip("would launch with the addresses of nothing")
    refused(5, f, sp, {"workspace": 15 * A, "ws_bytes": 1 << 40, "stream": 0})
    assert "launch" not in binding.wg_last_error() and "cuTensorMapEncodeTiled" in binding.wg_last_error()


def test_columns_of_one_buffer_are_apart():
    """x, y, z and residual side by side in the rows of one buffer share no bytes; shifted by an element they do."""
    big = {"workspace": 15 * A, "ws_bytes": 1 << 40, "stream": 0}
    x, y, z, w = 64 * 2, 72 * 2, 72 * 2, 2 * A
    row = x + y + z
    for tokens in (2, 20, 300):
        sp = lin(tokens=tokens, ld_in=row // 2, ld_out=row // 2, ld_z=row // 2, ld_residual=row // 2)
        f, d, g = binding.wg_linear, binding.wg_linear_bwd_data, binding.wg_linear_bwd_weight
        apart = [lambda: f(sp, A, w, A + x, z=A + x + y, **big), lambda: f(sp, A + row - x, w, A, z=A + y, **big),
                 lambda: f(sp, A + y, w, A, residual=A + y + x, **big), lambda: d(sp, A, w, A + y, **big),
                 lambda: binding.wg_activation(act(tokens=tokens, ld_x=200, ld_y=200), A, A + 256, stream=0),
                 lambda: binding.wg_activation(act(tokens=tokens, ld_x=200, ld_y=100, out_dtype="fp32"), A, A + 144, stream=0),
                 lambda: g(lin(tokens=tokens, ld_weight=100), w, 3 * A, A, dbias=A + 128 + 72 * 200, **big)]
        if no_gpu():
            for call in apart:
                refused(5, call)  # (what a call comes to that passes validation here)
        for call in (lambda: f(sp, A, w, A + x - 2, z=A + x + y, **big), lambda: f(sp, A, w, A + x, z=A + x + y - 2, **big),
                     lambda: f(sp, A, w, A + x + 2, z=A + x + y, **big), lambda: f(sp, A, w, A + x + z + 2, **big),
                     lambda: f({**sp, "ld_out": row // 2 + 8}, A, w, A + x, **big), lambda: d(sp, A, w, A + y - 2, **big),
                     lambda: f({**sp, "ld_out": 72}, A, w, A + x, **big),
                     lambda: binding.wg_activation(act(tokens=tokens, ld_x=200, ld_y=100, out_dtype="fp32"), A, A + 148, stream=0),
                     lambda: g(lin(tokens=tokens, ld_weight=100), w, 3 * A, A, dbias=A + 128, **big)):
            refused(1, call)
