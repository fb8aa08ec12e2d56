"""Cases of the layer operators: the matrix product with bias, activation, dropout and residual in its epilogue, its
gradients, the same products grouped by expert with ragged numbers of rows, and the activation with dropout alone.

`own` chooses between the operators' plain form in torch (32-bit arithmetic, one rounding at the end) and the calls a
user makes of this package.  Sizes are generic: projections and feed-forward layers of some thousand features, batches
from one token to a training batch.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def _linear(name, tokens, inf, out, dtype, y="", act="none", bias=True, residual=False, keep_z=False, dropout=0.0,
            experts=0, behind=0):
    return {"name": name, "op": "linear", "tokens": tokens, "in": inf, "out": out, "dtype": dtype, "y": y or dtype,
            "act": act, "bias": bias, "residual": residual, "keep_z": keep_z, "dropout": dropout, "experts": experts,
            "behind": behind}


def _grad(name, tokens, inf, out, dtype, dw="fp32", act="none", dropout=0.0, experts=0, behind=0):
    return {"name": name, "op": "linear_grad", "tokens": tokens, "in": inf, "out": out, "dtype": dtype, "dw": dw,
            "act": act, "dropout": dropout, "experts": experts, "behind": behind}


def _activation(name, form, tokens, dim, dtype, act, bias, residual, dropout):
    return {"name": name, "op": form, "tokens": tokens, "dim": dim, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "dropout": dropout}


def listed():
    return [
        # One decoding step of one sequence through a square projection with its residual: latency.
        _linear("token 4096->4096", 1, 4096, 4096, "bf16", bias=False, residual=True),
        # A decoding step of 24 sequences through a wide feed-forward layer.
        _linear("24 tokens 4096->16384", 24, 4096, 16384, "bf16", act="silu"),
        # A training batch through the wide layer of a feed-forward block; the pre-activations are kept.
        _linear("batch 8192x4096->16384", 8192, 4096, 16384, "bf16", act="gelu_tanh", keep_z=True),
        # The way back to the residual stream, with dropout, in fp16.
        _linear("batch 8192x8192->2048 dropout", 8192, 8192, 2048, "fp16", residual=True, dropout=0.1),
        # Sizes that are no multiples of any tile, rows that start at no 16-byte boundary.
        _linear("ragged 1009x1001->1515", 1009, 1001, 1515, "bf16", y="fp32", act="gelu"),
        # Both gradients of the wide layer's successor: of its input's pre-activations, its weight and its bias.
        _grad("gradients 8192x16384->4096", 8192, 16384, 4096, "bf16", act="gelu_tanh"),
        # The same for a small layer: a short batch, dropout below it.
        _grad("gradients 512x1024->1000", 512, 1024, 1000, "fp16", act="relu", dropout=0.2),
        # A decoding step of 16 sequences, two of 64 experts each.
        _linear("experts 32 rows", 32, 2048, 1024, "bf16", act="silu", bias=False, experts=64),
        # A training batch's rows, sorted by expert, some experts with none, in a padded buffer.
        _linear("experts 16384 rows", 16384, 2048, 4096, "bf16", act="gelu_tanh", keep_z=True, experts=64, behind=100),
        # Its gradients.
        _grad("experts' gradients 16384 rows", 16384, 4096, 2048, "bf16", dw="bf16", act="gelu_tanh", experts=64,
              behind=100),
        # What follows a convolution in a residual block: bias, activation, dropout, residual.
        _activation("activation 16384x4096", "activation", 16384, 4096, "bf16", "gelu", True, True, 0.1),
        # Its gradient and the bias's, rows that start at no 16-byte boundary.
        _activation("activation gradient 5001x2047", "activation_grad", 5001, 2047, "fp16", "silu", True, False, 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _features(rng, lo, hi):
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.3 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "experts", "experts_grad", "activation", "activation_grad"])
    dtype, act = rng.choice(["bf16", "fp16"]), rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    dropout = rng.choice([0.0, 0.0, 0.1, 0.37])
    if op in ("linear", "linear_grad"):
        tokens = _log(rng, 1, 40) if op == "linear" and rng.random() < 0.4 else _log(rng, 33, 8192)
        inf, out = _features(rng, 65, 8192), _features(rng, 65, 8192)
        if op == "linear":
            c = _linear("", tokens, inf, out, dtype, rng.choice([dtype, "fp32"]), act, rng.random() < 0.6,
                        rng.random() < 0.5, rng.random() < 0.4, dropout)
        else:
            c = _grad("", tokens, inf, out, dtype, rng.choice([dtype, "fp32"]), act, dropout)
    elif op in ("experts", "experts_grad"):
        experts = _log(rng, 2, 128)
        tokens = _log(rng, 1, 64) if op == "experts" and rng.random() < 0.4 else _log(rng, 65, 16384)
        inf, out = _features(rng, 65, 4096), _features(rng, 65, 4096)
        while experts * inf * out > 1 << 28:
            experts //= 2
        behind = rng.choice([0, 0, 77])
        if op == "experts":
            c = _linear("", tokens, inf, out, dtype, rng.choice([dtype, "fp32"]), act, rng.random() < 0.6,
                        rng.random() < 0.5, rng.random() < 0.4, dropout, experts, behind)
        else:
            c = _grad("", tokens, inf, out, dtype, rng.choice([dtype, "fp32"]), act, dropout, experts, behind)
    else:
        c = _activation("", op, _log(rng, 1, 16384), _features(rng, 65, 4096), dtype, act, rng.random() < 0.6,
                        op == "activation" and rng.random() < 0.5, dropout or 0.25)
    return {k: v for k, v in c.items() if k != "name"}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    # A training loop's seed of the generator, and the number of the step and layer.
    s = {"case": case, "stream": torch.cuda.current_stream().cuda_stream, "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64),
         "offset": 7 + 1000 * seed}
    if case["op"].startswith("activation"):
        t, d = case["tokens"], case["dim"]
        s["x"] = _randn(g, t, d).to(dt)
        s["bias"] = 0.5 * _randn(g, d) if case["bias"] else None
        if case["op"] == "activation":
            s["residual"] = (2.0 * _randn(g, t, d)).to(dt) if case["residual"] else None
            s["y"] = torch.empty((t, d), dtype=dt, device="cuda")
        else:
            s["dy"] = (0.05 * _randn(g, t, d)).to(dt)
            s["dx"] = torch.empty((t, d), dtype=dt, device="cuda")
            s["dbias"] = torch.empty(d, device="cuda") if case["bias"] else None
        return s
    t, inf, out, e = case["tokens"], case["in"], case["out"], case["experts"]
    rows = t + case["behind"]
    s["w"] = (_randn(g, max(e, 1), out, inf) / math.sqrt(inf)).to(dt)
    if e:
        # How many rows chose each expert: popular ones and rare ones, one in sixteen with none.
        like = torch.exp(0.6 * _randn(g, e))
        like[torch.rand(e, generator=g, device="cuda") < 1 / 16] = 0.0
        like[0] += 1e-3
        chosen = torch.multinomial(like, t, replacement=True, generator=g)
        count = torch.bincount(chosen, minlength=e)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
        s["most"] = int(count.max())
    s["x"] = _randn(g, rows, inf).to(dt)
    if case["op"] == "linear":
        ydt = _DT[case["y"]]
        s["bias"] = 0.5 * _randn(g, max(e, 1), out) if case["bias"] else None
        s["residual"] = (2.0 * _randn(g, rows, out)).to(ydt) if case["residual"] else None
        s["y"] = torch.zeros((rows, out), dtype=ydt, device="cuda")
        s["z"] = torch.zeros((rows, out), dtype=dt, device="cuda") if case["keep_z"] else None
    else:
        s["dy"] = (0.05 * _randn(g, rows, out)).to(dt)
        s["z"] = _randn(g, rows, inf).to(dt) if case["act"] != "none" else None
        s["dx"] = torch.zeros((rows, inf), dtype=dt, device="cuda")
        s["dw"] = torch.empty((max(e, 1), out, inf), dtype=_DT[case["dw"]], device="cuda")
        s["dbias"] = torch.empty((max(e, 1), out), device="cuda")
    return s


def _threshold(p):
    return min(65535, int(round(p * 65536)))


def _mask(s, rows, cols):
    """The dropout factor of each element: 0, or 1 / (1 - p).  Philox 4x32 with ten rounds (Salmon et al., 2011), its
    products in wrapping 64-bit integers: counter (column / 8, row, offset), 16 bits of the result an element."""
    low = 0xFFFFFFFF
    c0 = torch.arange((cols + 7) // 8, device="cuda")[None, :].expand(rows, -1)
    c1 = torch.arange(rows, device="cuda")[:, None].expand_as(c0)
    c2 = torch.full_like(c0, s["offset"] & low)
    c3 = torch.full_like(c0, s["offset"] >> 32)
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & low) ^ c1 ^ k0, q & low, ((p >> 32) & low) ^ c3 ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    halves = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xFFFF, c >> 16)], -1).view(rows, -1)[:, :cols]
    thr = _threshold(s["case"]["dropout"])
    return (halves >= thr).float() * (65536.0 / (65536 - thr))


def _act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0.0)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v / (1.0 + torch.exp(-v)) if name == "silu" else v


def _slope(name, v):
    if name == "relu":
        return (v > 0).float()
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * v * v)
    if name == "silu":
        y = 1.0 / (1.0 + torch.exp(-v))
        return y * (1.0 + v * (1.0 - y))
    return torch.ones_like(v)


def _groups(s):
    """Experts' rows side by side: row numbers (expert, place), which places hold a row, and each row's expert and place."""
    off, t = s["offsets"].long(), s["case"]["tokens"]
    place = torch.arange(s["most"], device="cuda")
    row = off[:-1, None] + place
    held = row < off[1:, None]
    r = torch.arange(t, device="cuda")
    e = (r[:, None] >= off[None, 1:]).sum(1)
    return row.clamp(max=t - 1), held, e, r - off[e]


def _plain(s):
    case = s["case"]
    if case["op"].startswith("activation"):
        t, d = case["tokens"], case["dim"]
        v = s["x"].float()
        if case["bias"]:
            v = v + s["bias"]
        if case["op"] == "activation":
            a = _act(case["act"], v) * _mask(s, t, d)
            s["y"].copy_(a + s["residual"].float() if case["residual"] else a)
            return s["y"]
        dv = s["dy"].float() * _mask(s, t, d) * _slope(case["act"], v)
        s["dx"].copy_(dv)
        if not case["bias"]:
            return s["dx"]
        s["dbias"].copy_(dv.sum(0))
        return {"dx": s["dx"], "dbias": s["dbias"]}
    t, e = case["tokens"], case["experts"]
    if e:
        row, held, expert, place = _groups(s)
    if case["op"] == "linear":
        if e:
            v = torch.bmm(s["x"][row].float(), s["w"].float().mT)
            if case["bias"]:
                v = v + s["bias"][:, None]
            v = v[expert, place]
        else:
            v = s["x"].float() @ s["w"][0].float().t()
            if case["bias"]:
                v = v + s["bias"][0]
        if case["keep_z"]:
            s["z"][:t] = v.to(s["z"].dtype)
        a = _act(case["act"], v)
        if case["dropout"]:
            a = a * _mask(s, t, case["out"])
        if case["residual"]:
            a = a + s["residual"][:t].float()
        s["y"][:t] = a.to(s["y"].dtype)
        return {"y": s["y"], "z": s["z"]} if case["keep_z"] else s["y"]
    if e:
        dy = s["dy"][row].float() * held[..., None]
        x = s["x"][row].float() * held[..., None]
        dx = torch.bmm(dy, s["w"].float())[expert, place]
        s["dw"].copy_(torch.bmm(dy.mT, x))
        s["dbias"].copy_(dy.sum(1))
    else:
        dy, x = s["dy"].float(), s["x"].float()
        dx = dy @ s["w"][0].float()
        s["dw"][0] = dy.t() @ x
        s["dbias"][0] = dy.sum(0)
    if case["act"] != "none":
        dx = dx * _slope(case["act"], s["z"][:t].float())
    if case["dropout"]:
        dx = dx * _mask(s, t, case["in"])
    s["dx"][:t] = dx.to(s["dx"].dtype)
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}


def _calls(s):
    """The calls a user's program makes of these buffers again and again, their arguments laid out at the first one."""
    from implicit_gemm_gb300 import binding
    case = s["case"]
    spec = {"in_dtype": case["dtype"], "bias_dtype": "fp32", "activation": case["act"], "dropout": case["dropout"],
            "seed": s["seed"], "offset": s["offset"]}
    memory = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    if case["op"].startswith("activation"):
        spec.update(tokens=case["tokens"], dim=case["dim"], out_dtype=case["dtype"])
        if case["op"] == "activation":
            return [binding.PreparedActivation(spec, s["x"], s["y"], bias=s["bias"], residual=s["residual"])]
        return [binding.PreparedActivationBwd(spec, s["dy"], s["x"], s["dx"], bias=s["bias"], dbias=s["dbias"],
                                              workspace=memory(binding.wg_activation_workspace_size(spec)))]
    spec.update(tokens=s["x"].shape[0], out=case["out"], experts=case["experts"], offset_dtype="i32", **{"in": case["in"]})
    if case["op"] == "linear":
        spec.update(out_dtype=case["y"])
        ws = memory(binding.wg_linear_workspace_size(spec, "forward"))
        return [binding.PreparedLinear(spec, s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], z=s["z"],
                                       offsets=s.get("offsets"), workspace=ws)]
    data, weight = dict(spec, out_dtype=case["dtype"]), dict(spec, out_dtype=case["dw"])
    ws = memory(max(binding.wg_linear_workspace_size(data, "bwd_data"),
                    binding.wg_linear_workspace_size(weight, "bwd_weight")))
    return [binding.PreparedLinearBwdData(data, s["dy"], s["w"], s["dx"], z=s["z"], offsets=s.get("offsets"),
                                          workspace=ws),
            binding.PreparedLinearBwdWeight(weight, s["x"], s["dy"], s["dw"], dbias=s["dbias"],
                                            offsets=s.get("offsets"), workspace=ws)]


def run(s):
    if not own:
        return _plain(s)
    calls = s.get("calls")
    if calls is None:
        calls = s["calls"] = _calls(s)
    for call in calls:
        call(s["stream"])
    op = s["case"]["op"]
    if op == "linear":
        return s["y"] if s["z"] is None else {"y": s["y"], "z": s["z"]}
    if op == "linear_grad":
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    if op == "activation":
        return s["y"]
    return s["dx"] if s["dbias"] is None else {"dx": s["dx"], "dbias": s["dbias"]}


def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"].startswith("activation"):
        n = case["tokens"] * case["dim"]
        arrays = 2 + (case["residual"] if case["op"] == "activation" else 1)
        return {"bytes": n * b * arrays + (4 * case["dim"] if case["bias"] else 0), "flops": 8 * n}
    t, inf, out, e = case["tokens"], case["in"], case["out"], case["experts"]
    product = 2 * t * inf * out
    # Weights of experts that some row chose (as many as of equally popular ones).
    used = inf * out * (e * (1 - (1 - 1 / e) ** t) if e > 1 else 1)
    if case["op"] == "linear":
        moved = t * inf * b + used * b + t * out * _SIZE[case["y"]] * (1 + case["residual"]) + t * out * b * case["keep_z"]
        return {"bytes": int(moved), "flops": product}
    moved = t * out * b + t * inf * b + used * b + t * inf * b * (1 + (case["act"] != "none"))
    return {"bytes": int(moved + max(e, 1) * inf * out * _SIZE[case["dw"]]), "flops": 2 * product}


def _exact_keep(s, rows, cols):
    """Philox again, 32-bit products from 16-bit halves, a bit per element."""
    groups = (cols + 7) // 8
    n = torch.arange(rows * groups, device="cuda")
    word = [n % groups, n // groups, torch.full_like(n, s["offset"] % 2 ** 32), torch.full_like(n, s["offset"] // 2 ** 32)]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]

    def product(a, m):
        lo, hi, ml, mh = a % 65536, a // 65536, m % 65536, m // 65536
        mid = lo * mh + (lo * ml) // 65536
        mid2 = hi * ml + mid % 65536
        return hi * mh + mid // 65536 + mid2 // 65536, mid2 % 65536 * 65536 + (lo * ml) % 65536
    for _ in range(10):
        hi0, lo0 = product(word[0], 0xD2511F53)
        hi1, lo1 = product(word[2], 0xCD9E8D57)
        word = [hi1 ^ word[1] ^ key[0], lo1, hi0 ^ word[3] ^ key[1], lo0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = torch.empty((rows, groups, 8), dtype=torch.bool, device="cuda")
    thr = _threshold(s["case"]["dropout"])
    for i in range(4):
        bits[:, :, 2 * i] = (word[i] % 65536 >= thr).view(rows, groups)
        bits[:, :, 2 * i + 1] = (word[i] // 65536 >= thr).view(rows, groups)
    return bits.view(rows, -1)[:, :cols], 65536 / (65536 - thr)


def _exact_act(name, v):
    f = torch.nn.functional
    if name == "gelu":
        return f.gelu(v)
    if name == "gelu_tanh":
        return f.gelu(v, approximate="tanh")
    return f.relu(v) if name == "relu" else f.silu(v) if name == "silu" else v


def _exact_slope(name, v):
    v = v.detach().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(_exact_act(name, v).sum(), v)[0]


def _exact_drop(s, a):
    if not s["case"]["dropout"]:
        return a
    keep, gain = _exact_keep(s, *a.shape)
    return torch.where(keep, a * gain, torch.zeros_like(a))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("activation"):
        v = s["x"].double()
        if case["bias"]:
            v += s["bias"].double()
        if case["op"] == "activation":
            a = _exact_drop(s, _exact_act(case["act"], v))
            return a + s["residual"].double() if case["residual"] else a
        dx = _exact_drop(s, _exact_slope(case["act"], v) * s["dy"].double())
        return {"dx": dx, "dbias": dx.sum(0)} if case["bias"] else dx
    t, e = case["tokens"], max(case["experts"], 1)
    bounds = s["offsets"].tolist() if case["experts"] else [0, t]
    if case["op"] == "linear":
        y = s["y"].double()
        z = y.clone() if case["keep_z"] else None
        v = torch.empty((t, case["out"]), dtype=torch.float64, device="cuda")
        for i in range(e):
            lo, hi = bounds[i], bounds[i + 1]
            v[lo:hi] = torch.nn.functional.linear(s["x"][lo:hi].double(), s["w"][i].double(),
                                                  s["bias"][i].double() if case["bias"] else None)
        if z is not None:
            z[:t] = v
        a = _exact_drop(s, _exact_act(case["act"], v))
        y[:t] = a + s["residual"][:t].double() if case["residual"] else a
        return y if z is None else {"y": y, "z": z}
    dx = s["dx"].double()
    d = torch.empty((t, case["in"]), dtype=torch.float64, device="cuda")
    dw = torch.empty(s["dw"].shape, dtype=torch.float64, device="cuda")
    db = torch.empty(s["dbias"].shape, dtype=torch.float64, device="cuda")
    for i in range(e):
        lo, hi = bounds[i], bounds[i + 1]
        dy = s["dy"][lo:hi].double()
        torch.mm(dy, s["w"][i].double(), out=d[lo:hi])
        torch.mm(dy.mT, s["x"][lo:hi].double(), out=dw[i])
        db[i] = dy.sum(0)
    if case["act"] != "none":
        d = d * _exact_slope(case["act"], s["z"][:t].double())
    dx[:t] = _exact_drop(s, d)
    return {"dx": dx, "dw": dw, "dbias": db}
