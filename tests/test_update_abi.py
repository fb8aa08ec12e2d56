"""Host-side checks of the weight-update entry points (no GPU needed): sizes, plans and refusals.  Only calls that
fail validation are made here, so nothing is launched."""
import math

import pytest

from implicit_gemm_gb300 import binding, build

A = 1 << 20  # stands for a device address; refused before it is used


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def muon(**kw):
    return {"rows": 24, "cols": 40, **kw}


def emb(**kw):
    return {"tokens": 7, "vocab": 11, "dim": 16, **kw}


def refused(status, f, *a, **kw):
    with pytest.raises(binding.WgradError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value
    assert binding.wg_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(rows=0), 1), (dict(cols=-1), 1), (dict(batch=0), 1), (dict(rows=40000), 2), (dict(batch=70000), 2),
    (dict(steps=-1), 1), (dict(steps=17), 1), (dict(momentum=1.0), 1), (dict(momentum=-0.1), 1),
    (dict(momentum=math.nan), 1), (dict(dampening=1.5), 1), (dict(eps=-1e-8), 1), (dict(eps=math.inf), 1),
    (dict(scale=math.inf), 1), (dict(lr=math.nan), 1), (dict(weight_decay=math.inf), 1), (dict(ld=39), 1),
    (dict(batch=2, batch_stride=39), 1), (dict(batch=2, ld=79, batch_stride=40), 1),
    (dict(steps=1, coef=[(8.0, 0.0, 0.0)]), 1), (dict(steps=2, coef=[(2.0, 0.0, 0.0), (math.nan, 0.0, 0.0)]), 1),
])
def test_muon_problem_refusals(bad, status):
    refused(status, binding.wg_muon_workspace_size, muon(**bad))
    refused(status, binding.wg_muon_update, muon(**bad), A, out=2 * A, workspace=3 * A, ws_bytes=1 << 40, stream=0)


def test_muon_layouts_accepted():
    assert binding.wg_muon_workspace_size(muon(batch=2, ld=80, batch_stride=40)) > 0   # side by side
    assert binding.wg_muon_workspace_size(muon(batch=2, ld=41, batch_stride=24 * 41 + 5)) > 0
    assert "muon" in binding.wg_muon_plan_string(muon())
    with pytest.raises(ValueError):
        binding.make_muon_problem(muon(steps=2, coef=[(1.0, 0.0, 0.0)]))


def test_muon_buffer_refusals():
    sp, big = muon(), 1 << 30
    refused(1, binding.wg_muon_update, sp, 0, out=A, workspace=2 * A, ws_bytes=big, stream=0)
    refused(1, binding.wg_muon_update, sp, A, workspace=2 * A, ws_bytes=big, stream=0)
    refused(1, binding.wg_muon_update, sp, A, out=A, workspace=4 * A, ws_bytes=big, stream=0)
    refused(1, binding.wg_muon_update, sp, A, momentum=A + 64, out=2 * A, workspace=4 * A, ws_bytes=big, stream=0)
    refused(3, binding.wg_muon_update, sp, A + 2, out=2 * A, workspace=4 * A, ws_bytes=big, stream=0)
    refused(3, binding.wg_muon_update, sp, A, momentum=2 * A + 2, out=4 * A, workspace=8 * A, ws_bytes=big, stream=0)
    refused(3, binding.wg_muon_update, sp, A, out=2 * A, workspace=4 * A + 8, ws_bytes=big, stream=0)
    refused(4, binding.wg_muon_update, sp, A, out=2 * A, workspace=4 * A,
            ws_bytes=binding.wg_muon_workspace_size(sp) - 1, stream=0)
    refused(4, binding.wg_muon_update, sp, A, out=2 * A, stream=0)


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=-1), 1), (dict(tokens=1 << 31), 1), (dict(vocab=0), 1), (dict(dim=0), 1), (dict(ld_table=15), 1),
    (dict(ld_out=15), 1), (dict(padding_token=11), 1), (dict(padding_token=-2), 1), (dict(scale=math.nan), 1),
    (dict(vocab=(1 << 31) - 1), 1), (dict(dim=(1 << 31) - 1), 1),
])
def test_embedding_problem_refusals(bad, status):
    refused(status, binding.wg_embedding_workspace_size, emb(**bad))
    refused(status, binding.wg_embedding_lookup, emb(**bad), A, 2 * A, 3 * A, stream=0)
    refused(status, binding.wg_embedding_bwd_weight, emb(**bad), A, 2 * A, 3 * A, workspace=4 * A, ws_bytes=1 << 40,
            stream=0)


def test_embedding_buffer_refusals():
    sp, big = emb(), 1 << 30
    for args in ((0, A, 2 * A), (A, 0, 2 * A), (A, 2 * A, 0)):
        refused(1, binding.wg_embedding_lookup, sp, *args, stream=0)
        refused(1, binding.wg_embedding_bwd_weight, sp, *args, workspace=4 * A, ws_bytes=big, stream=0)
    refused(3, binding.wg_embedding_lookup, sp, A + 4, 2 * A, 3 * A, stream=0)
    refused(3, binding.wg_embedding_lookup, sp, A, 2 * A + 1, 3 * A, stream=0)
    refused(3, binding.wg_embedding_lookup, emb(out_dtype="fp32"), A, 2 * A, 3 * A + 2, stream=0)
    refused(4, binding.wg_embedding_bwd_weight, sp, A, 2 * A, 3 * A, stream=0)
    refused(4, binding.wg_embedding_bwd_weight, sp, A, 2 * A, 3 * A, workspace=4 * A, ws_bytes=16, stream=0)
    refused(3, binding.wg_embedding_bwd_weight, sp, A, 2 * A, 3 * A, workspace=4 * A + 4, ws_bytes=big, stream=0)


def test_status_of_a_bad_token_has_a_name():
    assert binding.wg_status_string(7) == "WG_ERR_INVALID_TOKEN"


def test_embedding_overlap_refusals():
    sp, big = emb(), 1 << 30  # 56 bytes of tokens, a table of 352 bytes, out of 224
    for args in ((8 * A, A, A + 336), (8 * A, A + 208, A), (A + 208, 8 * A, A)):
        refused(1, binding.wg_embedding_lookup, sp, *args, stream=0)
    for args in ((8 * A, A + 336, A), (8 * A, A, A + 208), (A + 336, 8 * A, A)):
        refused(1, binding.wg_embedding_bwd_weight, sp, *args, workspace=4 * A, ws_bytes=big, stream=0)


def test_wrappers_refuse_tensors_that_do_not_fit():
    """Shapes, types and layouts are refused before anything is allocated; so are tensors in host memory."""
    import torch
    b16 = torch.bfloat16
    tok, table = torch.zeros((2, 3), dtype=torch.int64), torch.zeros((11, 16), dtype=b16)

    def bad(why, f, **kw):
        with pytest.raises(ValueError, match=why):
            f(**kw)

    look, lk = binding.embedding_lookup, {"token": tok, "table": table}
    bad("token", look, **{**lk, "token": tok.short()})
    bad("token", look, **{**lk, "token": tok.mT})
    bad("table must be contiguous", look, **{**lk, "table": torch.zeros((16, 11), dtype=b16).mT})
    bad("float64", look, **{**lk, "table": table.double()})
    bad("out has shape", look, **lk, out=torch.zeros((2, 3, 15), dtype=b16))
    bad("out has shape", look, **lk, out=torch.zeros((3, 2, 16), dtype=b16))
    bad("token is not a CUDA tensor", look, **lk)
    dy = torch.zeros((2, 3, 16), dtype=b16)
    grad, gk = binding.embedding_bwd_weight, {"token": tok, "dy": dy, "vocab": 11}
    bad("dy has shape", grad, **{**gk, "dy": dy[:1]})
    bad("dy must be contiguous", grad, **{**gk, "dy": torch.zeros((2, 3, 32), dtype=b16)[..., ::2]})
    bad("accumulate needs out", grad, **gk, accumulate=True)
    bad("out has shape", grad, **gk, out=torch.zeros((10, 16)))
    bad("int32", grad, **gk, out=torch.zeros((11, 16), dtype=torch.int32))
    bad("token is not a CUDA tensor", grad, **gk)
    g, up = torch.zeros((24, 40)), binding.muon_update
    bad("grad holds fewer", up, spec=muon(), grad=torch.zeros((23, 40)))
    bad("grad must be contiguous", up, spec=muon(), grad=g.mT)
    bad("grad is", up, spec=muon(), grad=g.to(b16))
    bad("grad is", up, spec=muon(grad_dtype="bf16"), grad=g)
    bad("momentum is", up, spec=muon(), grad=g, momentum=g.to(b16))
    bad("weight is", up, spec=muon(), grad=g, weight=g)
    bad("out holds fewer", up, spec=muon(), grad=g, out=torch.zeros(24 * 40 - 1, dtype=b16))
    bad("out holds fewer", up, spec=muon(ld=48), grad=torch.zeros((24, 48))[:, :40], out=torch.zeros((24, 40), dtype=b16))
    bad("grad holds fewer", up, spec=muon(batch=2, batch_stride=1000), grad=torch.zeros(1959))
    bad("grad is not a CUDA tensor", up, spec=muon(), grad=g)


@pytest.mark.parametrize("rows,cols", [(1, 1), (8, 72), (64, 576), (128, 128), (300, 400)])
def test_muon_kernels_take_an_sm_whole(rows, cols):
    """A CTA of these kernels takes tensor memory and then waits for its cluster: two that shared an SM could wait for
    each other for ever.  They ask for so much of an SM's 228 KB of shared memory (1 KB of it per CTA is the system's)
    that none fits beside another, nor beside a convolution's that is reduced over a cluster or runs on a pair."""
    plan = dict(kv.split("=") for kv in binding.wg_muon_plan_string(muon(rows=rows, cols=cols)).split())
    least = 228 * 1024 - 1024 - int(plan["smem"])  # what another CTA could have, the system's part of it included
    assert least < 1024 + int(plan["smem"])
    conv = {"ndim": 1, "G": 1, "N": 2, "C": 8, "K": 8, "in": [8], "filt": [1], "stride": [1], "dil": [1], "pad_l": [0],
            "pad_r": [0], "in_dtype": "bf16", "out_dtype": "fp32"}
    seen = 0
    for n in (2, 8, 32):
        for c, k, cluster in ((8, 8, 2), (8, 8, 4), (16, 8, 8), (8, 64, 2), (64, 64, 2)):
            for x in (1, 3):
                sp = {**conv, "N": n, "C": c, "K": k, "in": [16], "filt": [x], "pad_l": [x // 2], "pad_r": [x // 2]}
                try:
                    text = binding.wg_plan_string(sp, 2 * cluster, "deterministic", cluster=cluster)
                except binding.WgradError:
                    continue
                other = dict(kv.split("=", 1) for kv in text.split() if "=" in kv)
                seen += other.get("cluster", "1") != "1"
                assert least < 1024 + int(other["smem"]), text
    assert seen


def test_muon_steps_of_a_launch():
    """Small matrices: five default steps in one launch, without a workspace to speak of; more steps, or larger factors,
    in several, with X kept in between."""
    def plan(**kw):
        sp = muon(**kw)
        text = dict(kv.split("=") for kv in binding.wg_muon_plan_string(sp).split())
        assert int(text["ws"]) == binding.wg_muon_workspace_size(sp)
        return int(text["launches"]), int(text["ws"])

    assert plan() == (1, 256) and plan(steps=1) == (1, 256)
    assert plan(steps=16, coef=[(1.2, -0.2, 0.0)] * 16)[0] == 1
    falling = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518),
               (3.3184, -2.4885, 0.5100), (2.3007, -1.6690, 0.4188)]
    assert plan(steps=4, coef=falling[:4])[0] == 1  # factors' product 446
    for kw in (dict(steps=6), dict(steps=16), dict(steps=5, coef=falling)):
        n, ws = plan(**kw)
        assert n > 1 and ws >= 24 * 40 * 4


def test_muon_operands_of_larger_matrices():
    """Five default steps multiply matrices of one 16-bit value an element; more, or steeper ones, of two."""
    values = lambda **kw: dict(kv.split("=") for kv in binding.wg_muon_plan_string(  # noqa: E731
        {"rows": 300, "cols": 400, **kw}).split())["values"]
    assert values() == "1" and values(steps=3) == "1" and values(steps=16, coef=[(1.875, -1.25, 0.375)] * 16) == "1"
    falling = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518),
               (3.3184, -2.4885, 0.5100), (2.3007, -1.6690, 0.4188)]
    assert values(steps=6) == "2" and values(steps=16) == "2" and values(steps=5, coef=falling) == "2"
    # What follows does not mend what a steep step has spoilt.
    assert values(steps=8, coef=falling + [(1.875, -1.25, 0.375)] * 3) == "2"
    one, two = (binding.wg_muon_workspace_size({"rows": 300, "cols": 400, "steps": n}) for n in (5, 6))
    assert two >= one + 300 * 400 * 2 + 2 * 300 * 304 * 2


@pytest.mark.parametrize("big", [(1 << 63) - 1, 1 << 62, 1 << 50])
def test_strides_whose_addresses_would_overflow_are_refused(big):
    for bad in (dict(ld=big), dict(batch=2, batch_stride=big), dict(rows=30000, ld=big)):
        refused(1, binding.wg_muon_workspace_size, muon(**bad))
        refused(1, binding.wg_muon_update, muon(**bad), A, out=2 * A, workspace=3 * A, ws_bytes=1 << 40, stream=0)
    for bad in (dict(ld_table=big, vocab=1 << 30), dict(ld_out=big, tokens=1 << 30)):
        refused(1, binding.wg_embedding_workspace_size, emb(**bad))
        refused(1, binding.wg_embedding_lookup, emb(**bad), A, 2 * A, 3 * A, stream=0)
        refused(1, binding.wg_embedding_bwd_weight, emb(**bad), A, 2 * A, 3 * A, workspace=4 * A, ws_bytes=1 << 60,
                stream=0)
    refused(1, binding.wg_muon_workspace_size, muon(batch=60000, rows=30000, ld=1 << 33))
    refused(1, binding.wg_muon_workspace_size, muon(ld=-big))
    refused(1, binding.wg_muon_workspace_size, muon(batch=2, batch_stride=-big))
    # What no address is made of does not count: the distance to a second matrix that is not there.
    assert binding.wg_muon_workspace_size(muon(batch_stride=big)) > 0


def test_plans_are_found_whatever_the_record_s_padding_and_factors_hold():
    """A caller in C leaves the bytes between the record's members as they were, and a learning rate changes with every
    step: such a call finds the plan all the same, instead of making it anew (some 30 times as long)."""
    import ctypes
    import time
    lib, p, n = binding.load(), binding.make_muon_problem({"rows": 1000, "cols": 2731}), ctypes.c_size_t(0)
    raw = (ctypes.c_ubyte * ctypes.sizeof(p)).from_buffer(p)
    used = set()
    for name, kind in p._fields_:
        at = getattr(type(p), name).offset
        used |= set(range(at, at + ctypes.sizeof(kind)))
    holes = [i for i in range(ctypes.sizeof(p)) if i not in used]
    assert holes

    def best(change):
        times = []
        for k in range(400):
            if change:
                for i in holes:
                    raw[i] = (37 * best.calls + i) & 255
                p.lr, p.scale = 1e-3 / (1 + best.calls), 1 + best.calls
                best.calls += 1
            t = time.perf_counter()
            assert lib.wg_muon_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
            times.append(time.perf_counter() - t)
        return sorted(times)[200]

    best.calls = 0
    same = best(False)
    assert best(True) < 5 * same
