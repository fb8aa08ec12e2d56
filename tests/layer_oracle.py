"""The layer operators in 64 bits, from their definitions, and how far a call may be from them.

Tolerances.  Products of two 16-bit values are exact in fp32.  The tensor cores add 16 of them at a time, with
truncation, to a sum of at most 1024 terms (of an fp32 result): 64 additions, each off by at most a unit of fp32's last
place of the sum of the terms' sizes A: 64 * 2^-23 A; then a rounding 2^-24 A for each such sum (and each part of a cut
one).  A 16-bit result's sums have up to 32768 terms, so up to 2048 additions, but truncation takes what is proportional to
the sum so far, which stays near the root of the terms' number for terms of both signs, as all inputs here have: less than
the same bound.  What follows is fp32: the bias adds 2^-24 |v|, an activation's value is off
by at most 2^-20 (|v| + 1) (exponential, quotient and erf to a few last places of their own and of their arguments; |v| up
to 40 grows the exponential's argument error by as much where its value is below 2^-50) and carries v's error with a slope of at most
1.13 (its slope's slope is at most 1.6, and a slope is off by 2^-19), dropout's factor and the residual 2^-23 of their
values.  The last rounding is half a unit of the result's type (and 2^-25 below fp16's normal numbers).
"""
import numpy as np
import torch

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 1e-37, "bf16": 1e-37, "fp16": 2.0 ** -25}


def keep_mask(seed, offset, rows, cols, p):
    """(kept, factor) of dropout p: Philox 4x32-10 in numpy, as include/wgrad.h states it."""
    u = np.uint64
    groups = (cols + 7) // 8
    low = u(0xFFFFFFFF)
    c = [np.tile(np.arange(groups, dtype=u), rows), np.repeat(np.arange(rows, dtype=u), groups),
         np.full(rows * groups, offset & 0xFFFFFFFF, dtype=u), np.full(rows * groups, offset >> 32, dtype=u)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & low, (a >> u(32)) ^ c[3] ^ u(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    h = np.stack([x for w in c for x in (w & u(0xFFFF), w >> u(16))], -1).reshape(rows, -1)[:, :cols]
    thr = min(65535, int(np.floor(65536 * float(np.float32(p)) + 0.5)))
    return torch.from_numpy(h >= u(thr)), 65536.0 / (65536 - thr)


def act(name, v):
    f = torch.nn.functional
    return {"none": lambda: v, "relu": lambda: f.relu(v), "gelu": lambda: f.gelu(v),
            "gelu_tanh": lambda: f.gelu(v, approximate="tanh"), "silu": lambda: f.silu(v)}[name]()


def slope(name, v):
    if name == "none":
        return torch.ones_like(v)
    v = v.detach().clone().requires_grad_()
    return torch.autograd.grad(act(name, v).sum(), v)[0]


def drop(a, p, seed, offset):
    if not p:
        return a, 1.0
    kept, gain = keep_mask(seed, offset, a.shape[0], a.shape[1], p)
    return torch.where(kept.to(a.device), a * gain, torch.zeros_like(a)), gain


def sum_error(A, terms):
    return A * (64 * 2.0 ** -23 + (terms / 512 + 17) * 2.0 ** -24)


def spans(tokens, offsets):
    """(expert, first row, row after the last) of every expert, the offsets brought into order as the header says."""
    if offsets is None:
        return [(0, 0, tokens)]
    run, clean = 0, []
    for v in offsets:
        run = max(run, min(max(int(v), 0), tokens))
        clean.append(run)
    return [(e, clean[e], clean[e + 1]) for e in range(len(clean) - 1)]


def products(a, w, groups, transposed):
    """Rows of a times w[e] (transposed: its transpose) per expert, and the sums of the terms' sizes; NaN elsewhere."""
    out = torch.full((a.shape[0], w.shape[1] if transposed else w.shape[2]), float("nan"), dtype=torch.float64, device=a.device)
    size = out.clone()
    for e, lo, hi in groups:
        m = w[e].double().mT if transposed else w[e].double()
        out[lo:hi] = a[lo:hi].double() @ m
        size[lo:hi] = a[lo:hi].double().abs() @ m.abs()
    return out, size


def forward(x, w, bias=None, residual=None, activation="none", dropout=0.0, seed=0, offset=0, offsets=None):
    """(v, its error), (y, its error) before their last rounding; w (experts, out, in)."""
    groups = spans(x.shape[0], offsets)
    v, A = products(x, w, groups, True)
    err = sum_error(A, x.shape[1])
    if bias is not None:
        for e, lo, hi in groups:
            v[lo:hi] += bias[e].double()
        err = err + 2.0 ** -24 * (v.abs() + err)
    a = act(activation, v)
    aerr = 1.13 * err + (2.0 ** -20 * (v.abs() + 1) if activation != "none" else 0.0)
    a, gain = drop(a, dropout, seed, offset)
    aerr = aerr * gain + 2.0 ** -23 * a.abs()
    if residual is not None:
        a = a + residual.double()
        aerr = aerr + 2.0 ** -23 * a.abs()
    return (v, err), (a, aerr)


def data(dy, w, z=None, residual=None, activation="none", dropout=0.0, seed=0, offset=0, offsets=None):
    d, A = products(dy, w, spans(dy.shape[0], offsets), False)
    err = sum_error(A, dy.shape[1])
    if activation != "none":
        s = slope(activation, z.double())
        err = 1.13 * err + 2.0 ** -19 * d.abs() * (1 + 0.01 * z.double().abs())
        d = d * s
    d, gain = drop(d, dropout, seed, offset)
    err = err * gain + 2.0 ** -23 * d.abs()
    if residual is not None:
        d = d + residual.double()
        err = err + 2.0 ** -23 * d.abs()
    return d, err


def weight(x, dy, offsets=None, experts=1):
    dw = torch.zeros((experts, dy.shape[1], x.shape[1]), dtype=torch.float64, device=x.device)
    A, db, B = dw.clone(), dw.new_zeros(experts, dy.shape[1]), dw.new_zeros(experts, dy.shape[1])
    for e, lo, hi in spans(x.shape[0], offsets):
        g = dy[lo:hi].double()
        dw[e] = g.mT @ x[lo:hi].double()
        A[e] = g.abs().mT @ x[lo:hi].double().abs()
        db[e], B[e] = g.sum(0), g.abs().sum(0)
    n = x.shape[0]
    # dbias: at most 128 terms a thread, then sums of sums: fewer than 256 roundings of what is at most B.
    return (dw, sum_error(A, n)), (db, 2.0 ** -24 * 256 * B)


def close(got, want, err, dt, what=""):
    """got against want, off by at most err and then rounded to dt; non-finite values are the same."""
    got = got.double()
    assert got.shape == want.shape, (got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), what
    tol = err + HALF[dt] * (want.abs() + err) + TINY[dt]
    far = ((got - want).abs() - tol)[fine]
    assert not far.numel() or float(far.max()) <= 0, (what, float(((got - want).abs() / tol)[fine].max()))
