"""Cases of the weight-update operators: the orthogonalised update (Newton-Schulz products, with momentum and the
weight step), the embedding lookup and the embedding table's gradient.

`own` chooses between the operators' plain form in torch (32-bit arithmetic, one rounding at the end) and the calls a
user makes of this package.  Sizes of the matrices follow the filters that this repository's weight gradients are
measured on (64x576, 32 groups of 8x72, 96x3456) and generic projection matrices; the tables and token counts are
generic.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_COEF = (3.4445, -4.7750, 2.0315)  # the quintic's coefficients, of every step
_STEPS = 5
_EPS = 1e-7
_MU, _LR, _DECAY = 0.95, 0.02, 0.01


def _muon(name, form, batch, rows, cols, grad, out):
    return {"name": name, "op": "muon", "form": form, "batch": batch, "rows": rows, "cols": cols, "grad": grad,
            "out": out}


def _lookup(name, tokens, vocab, dim, dtype, zipf):
    return {"name": name, "op": "lookup", "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "zipf": zipf}


def _bwd(name, tokens, vocab, dim, dtype, out, zipf):
    return {"name": name, "op": "lookup_grad", "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype,
            "out": out, "zipf": zipf}


def listed():
    return [
        # One optimiser step of a 3x3, 64 -> 64 convolution: the fp32 weight gradient, fp32 momentum, bf16 weights.
        _muon("step conv 64x576", "step", 1, 64, 576, "fp32", "bf16"),
        # The groups of a grouped 3x3 convolution, each a matrix of its own.
        _muon("update 32 groups 8x72", "update", 32, 8, 72, "fp32", "bf16"),
        # A 3-D 3x3x3 convolution, 128 -> 96, fp16 training.
        _muon("step conv3d 96x3456", "step", 1, 96, 3456, "fp16", "bf16"),
        # The square projections of eight layers, taken together.
        _muon("step 8 of 1024x1024", "step", 8, 1024, 1024, "bf16", "bf16"),
        # A projection whose sizes are no multiples of any tile, wide.
        _muon("update ragged 1000x2731", "update", 1, 1000, 2731, "bf16", "bf16"),
        # A large feed-forward matrix, more rows than columns.
        _muon("step tall 8192x4096", "step", 1, 8192, 4096, "bf16", "bf16"),
        # One decoding step of a small batch: latency.
        _lookup("lookup 8 tokens", 8, 32768, 4096, "bf16", True),
        # A training batch's lookup.
        _lookup("lookup 32768 tokens", 32768, 131072, 2048, "bf16", True),
        # The table's gradient: a small model with a small vocabulary, fp32 gradient.
        _bwd("table grad 512 tokens", 512, 8192, 512, "bf16", "fp32", True),
        # Odd sizes: rows that start at no 16-byte boundary.
        _bwd("table grad ragged", 16001, 50001, 999, "fp16", "fp32", True),
        # A training batch's gradient of a large table, words as frequent as in text.
        _bwd("table grad 65536 tokens", 65536, 131072, 2048, "bf16", "bf16", True),
        # The same with tokens that hardly repeat, and few of them for the table.
        _bwd("table grad spread tokens", 8192, 65536, 1024, "bf16", "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["muon small", "muon", "lookup", "lookup_grad"])
    if op == "muon small":
        rows = _log(rng, 1, 256)
        cols = _log(rng, 9, 4608)
        batch = max(1, min(_log(rng, 1, 64), (1 << 22) // (rows * cols)))
        if rng.random() < 0.25:
            rows, cols = cols, rows
        return {k: v for k, v in _muon("", rng.choice(["step", "update"]), batch, rows, cols,
                                       rng.choice(["fp32", "bf16", "fp16"]), "bf16").items() if k != "name"}
    if op == "muon":
        rows, cols = _log(rng, 129, 4096), _log(rng, 129, 8192)
        batch = max(1, min(_log(rng, 1, 8), (1 << 24) // (rows * cols)))
        return {k: v for k, v in _muon("", rng.choice(["step", "update"]), batch, rows, cols,
                                       rng.choice(["fp32", "bf16"]), "bf16").items() if k != "name"}
    vocab, dim = _log(rng, 256, 131072), _log(rng, 33, 2048)
    if rng.random() < 0.6:
        dim = max(64, dim // 64 * 64)
    tokens = _log(rng, 1, 65536)
    dtype, zipf = rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.7
    if op == "lookup":
        c = _lookup("", tokens, vocab, dim, dtype, zipf)
    else:
        c = _bwd("", tokens, vocab, dim, dtype, rng.choice(["fp32", "bf16"]), zipf)
    return {k: v for k, v in c.items() if k != "name"}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _tokens(g, case):
    """Token ids: as frequent as the words of a text (log-uniform ranks, in a random order of ids), or spread evenly."""
    n, v = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if not case["zipf"]:
        return (u * v).long().clamp_(max=v - 1).int()
    rank = torch.exp(u * math.log(v + 1.0)).floor().long() - 1
    return torch.randperm(v, generator=g, device="cuda")[rank.clamp_(0, v - 1)].int()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    if case["op"] == "muon":
        b, r, c = case["batch"], case["rows"], case["cols"]
        # A gradient is a few strong directions and noise; the momentum has seen more of the same directions.
        k = max(1, min(r, c) // 8)
        left, right = _randn(g, b, r, k), _randn(g, b, k, c)
        signal = torch.bmm(left, right) * (1e-3 / math.sqrt(k))
        s["grad"] = (signal + 1e-3 * _randn(g, b, r, c)).to(_DT[case["grad"]])
        if case["form"] == "step":
            s["momentum"] = 6.0 * signal + 2e-3 * _randn(g, b, r, c)
            s["weight"] = (0.02 * _randn(g, b, r, c)).to(_DT[case["out"]])
        else:
            s["out"] = torch.empty((b, r, c), dtype=_DT[case["out"]], device="cuda")
        return s
    s["tokens"] = _tokens(g, case)
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    if case["op"] == "lookup":
        s["table"] = (0.02 * _randn(g, v, d)).to(_DT[case["dtype"]])
        s["out"] = torch.empty((n, d), dtype=_DT[case["dtype"]], device="cuda")
    else:
        s["dy"] = (1e-3 * _randn(g, n, d)).to(_DT[case["dtype"]])
        s["dtable"] = torch.empty((v, d), dtype=_DT[case["out"]], device="cuda")
    return s


def _scale(case):
    """The factor on the orthogonal matrix that makes its entries' size that of an Adam step; sqrt(dim) for lookups."""
    if case["op"] == "muon":
        return math.sqrt(max(1.0, case["rows"] / case["cols"]))
    return math.sqrt(case["dim"])


def _orthogonalise(u):
    wide = u if u.shape[-2] <= u.shape[-1] else u.transpose(-1, -2)
    x = wide / (torch.sqrt((wide * wide).sum((-1, -2), keepdim=True)) + _EPS)
    a, b, c = _COEF
    for _ in range(_STEPS):
        gram = torch.bmm(x, x.transpose(-1, -2))
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x if u.shape[-2] <= u.shape[-1] else x.transpose(-1, -2)


def _plain(s):
    case = s["case"]
    if case["op"] == "lookup":
        s["out"].copy_(s["table"][s["tokens"].long()].float() * _scale(case))
        return s["out"]
    if case["op"] == "lookup_grad":
        total = torch.zeros(s["dtable"].shape, dtype=torch.float32, device="cuda")
        total.index_add_(0, s["tokens"].long(), s["dy"].float())
        s["dtable"].copy_(total * _scale(case))
        return s["dtable"]
    g = s["grad"].float()
    if case["form"] == "update":
        s["out"].copy_(_orthogonalise(g) * _scale(case))
        return s["out"]
    m = s["momentum"]
    m.mul_(_MU).add_(g)
    o = _orthogonalise(g + _MU * m) * _scale(case)
    s["weight"].copy_(s["weight"].float() * (1.0 - _LR * _DECAY) - _LR * o)
    return {"weight": s["weight"], "momentum": m}


def _call(s):
    """The call a user's program makes of these buffers again and again, its arguments laid out at the first one."""
    from implicit_gemm_gb300 import binding
    case = s["case"]
    if case["op"] == "muon":
        step = case["form"] == "step"
        spec = {"batch": case["batch"], "rows": case["rows"], "cols": case["cols"], "grad_dtype": case["grad"],
                "out_dtype": case["out"], "weight_dtype": case["out"], "steps": _STEPS, "scale": _scale(case),
                "eps": _EPS, "momentum": _MU, "nesterov": True, "lr": _LR, "weight_decay": _DECAY}
        ws = torch.empty(max(1, binding.wg_muon_workspace_size(spec)), dtype=torch.uint8, device="cuda")
        if step:
            return binding.PreparedMuonUpdate(spec, s["grad"], momentum=s["momentum"], weight=s["weight"],
                                              workspace=ws)
        return binding.PreparedMuonUpdate(spec, s["grad"], out=s["out"], workspace=ws)
    spec = {"tokens": case["tokens"], "vocab": case["vocab"], "dim": case["dim"], "scale": _scale(case),
            "token_dtype": "i32"}
    if case["op"] == "lookup":
        spec.update(table_dtype=case["dtype"], out_dtype=case["dtype"])
        return binding.PreparedEmbeddingLookup(spec, s["tokens"], s["table"], s["out"])
    spec.update(table_dtype=case["out"], out_dtype=case["dtype"])
    ws = torch.empty(max(1, binding.wg_embedding_workspace_size(spec)), dtype=torch.uint8, device="cuda")
    return binding.PreparedEmbeddingBwd(spec, s["tokens"], s["dy"], s["dtable"], workspace=ws)


def run(s):
    if not own:
        return _plain(s)
    call = s.get("call")
    if call is None:
        call = s["call"] = _call(s)
    call(s["stream"])
    if s["case"]["op"] == "muon":
        return s["out"] if "out" in s else {"weight": s["weight"], "momentum": s["momentum"]}
    return s["out"] if "out" in s else s["dtable"]


def work(case):
    if case["op"] == "muon":
        b, n = case["batch"], case["rows"] * case["cols"]
        lo, hi = sorted((case["rows"], case["cols"]))
        # Products of commuting symmetric matrices need half their elements.  Step by step: X X' and A A (half of
        # each), B X.  Or with all steps taken on the Gram matrix: X X' (half), 17 symmetric products, and Q X.
        step = _STEPS * (3 * lo * lo * hi + lo ** 3)
        gram = 3 * lo * lo * hi + (4 * _STEPS - 3) * lo ** 3
        moved = n * _SIZE[case["grad"]] + (n * (8 + 2 * _SIZE[case["out"]]) if case["form"] == "step"
                                           else n * _SIZE[case["out"]])
        return {"bytes": b * moved, "flops": b * min(step, gram)}
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    if case["op"] == "lookup":
        return {"bytes": 4 * n + (min(n, v) + n) * d * _SIZE[case["dtype"]], "flops": n * d}
    return {"bytes": 4 * n + n * d * _SIZE[case["dtype"]] + v * d * _SIZE[case["out"]], "flops": n * d}


def exact(case, seed):
    s = prepare(case, seed)
    f = _scale(case)
    if case["op"] == "lookup":
        return torch.index_select(s["table"], 0, s["tokens"]).double().mul_(f)
    if case["op"] == "lookup_grad":
        order = torch.argsort(s["tokens"])
        ids, count = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        rows = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        for lo in range(0, case["dim"], 256):  # columns at a time: the whole in 64 bits is large
            part = s["dy"][order, lo:lo + 256].double()
            rows[ids.long(), lo:lo + 256] = torch.segment_reduce(part, "sum", lengths=count, axis=0, unsafe=True)
        return rows.mul_(f)
    g = s["grad"].double()
    u = g
    if case["form"] == "step":
        m = _MU * s["momentum"].double() + g
        u = g + _MU * m
    norm = torch.linalg.matrix_norm(u)[:, None, None] + _EPS
    x = u / norm
    tall = case["rows"] > case["cols"]
    eye = torch.eye(min(case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
    a, b, c = _COEF
    for _ in range(_STEPS):
        if tall:
            q = x.mT @ x
            x = x @ (a * eye + b * q + c * (q @ q))
        else:
            q = x @ x.mT
            x = (a * eye + b * q + c * (q @ q)) @ x
    x = f * x
    if case["form"] == "update":
        return x
    return {"weight": s["weight"].double() * (1.0 - _LR * _DECAY) - _LR * x, "momentum": m}
