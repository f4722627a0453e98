"""The packed-sequence operators in 64 bits, from their formulas, with bounds on
what rounding may do to each output value.

Roundings counted, u = half a step of the output type (bf16 2^-8, fp32 2^-24):

* every output is rounded once: u |x|;
* bf16 only: the softmax weights P (forward and dv) and dS (dq, dk) are rounded
  once as operands of a product: u sum |P| |v| and so on;
* fp32 arithmetic: a logit's dot product of d terms is off by at most
  2 d 2^-24 tau |q| . |k|, its scaling and exponential (and the difference with a
  max or lse of like size) by 2^-20 relative to the weight for |S| <= 16 in these
  tests; rho bounds both together, relative to a weight.  A sum of n weighted
  terms adds n 2^-24 of the sum of their magnitudes (twice: products that
  accumulate without rounding to nearest);
* delta = dout . out is taken from the rounded out.

The bounds are sums of these terms per value, nothing is fitted.
"""
import math

import numpy as np
import torch

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, 2.0 ** -24)}


def prefix(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(lens, heads, kv_heads, dim, dtype, seed=0, fused=False, tail=0, device="cuda"):
    """q, k, v, dout (rows behind the last sequence: `tail` of them)."""
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + tail
    dt = TYPES[dtype][0]
    qkv = torch.randn(n, heads + 2 * kv_heads, dim, generator=g)
    qkv[:, :heads + kv_heads] *= 1.3
    qkv = qkv.to(dt).to(device)
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    dout = torch.randn(n, heads, dim, generator=g).to(dt).to(device)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v, dout


def reference(lens, q, k, v, dout, causal, scale=0.0, dtype="bf16"):
    """{name: (value, bound)} in 64 bits over the sequences' rows."""
    H, K, d = q.shape[1], k.shape[1], q.shape[2]
    G = H // K
    tau = scale if scale > 0 else 1 / math.sqrt(d)
    u = TYPES[dtype][1]
    uo = u if dtype == "bf16" else 0.0  # operands rounded to 16 bits
    n_all = sum(lens)
    res = {x: torch.zeros(n_all, h, d, dtype=torch.float64, device=q.device)
           for x, h in (("out", H), ("dq", H), ("dk", K), ("dv", K))}
    res["lse"] = torch.zeros(H, n_all, dtype=torch.float64, device=q.device)
    tol = {x: torch.zeros_like(t) for x, t in res.items()}
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        qs, do = (x[rows].double().transpose(0, 1) for x in (q, dout))
        ks, vs = (x[rows].double().transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))
        t = lambda x: x.transpose(1, 2)  # noqa: E731
        s = tau * qs @ t(ks)
        rho = float(2 * d * 2 ** -24 * (tau * qs.abs() @ t(ks).abs()).max() + 2 ** -20)
        if causal:
            s = s.masked_fill(torch.ones(n, n, device=q.device).triu(1).bool(), -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[..., None])
        out = p @ vs
        back = lambda x: x.transpose(0, 1)  # noqa: E731
        grow = uo + 2 * rho + 2 * n * 2 ** -24
        e_out = grow * (p @ vs.abs()) + u * out.abs()
        res["out"][rows], tol["out"][rows] = back(out), back(e_out)
        res["lse"][:, rows] = lse
        tol["lse"][:, rows] = rho + 2 * n * 2 ** -24 + 2 ** -23 * lse.abs()
        dp = do @ t(vs)
        delta = (do * out).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        e_delta = (do.abs() * (e_out + 2 * d * 2 ** -24 * out.abs())).sum(-1, keepdim=True)
        e_dp = 2 * d * 2 ** -24 * (do.abs() @ t(vs).abs())
        e_ds = uo * ds.abs() + p * (e_delta + e_dp) + 2 * rho * p * (dp - delta).abs()
        e_p = (uo + 2 * rho) * p
        more = 2 * n * G * 2 ** -24
        shared = lambda x: x.view(K, G, n, d).sum(1)  # noqa: E731
        dq, e_dq = tau * ds @ ks, tau * (e_ds + more * ds.abs()) @ ks.abs()
        dk, e_dk = shared(tau * t(ds) @ qs), shared(tau * t(e_ds + more * ds.abs()) @ qs.abs())
        dv, e_dv = shared(t(p) @ do), shared(t(e_p + more * p) @ do.abs())
        for x, y, e in (("dq", dq, e_dq), ("dk", dk, e_dk), ("dv", dv, e_dv)):
            # second order terms (an error of an error): 1/16 covers (1 + u)^2
            res[x][rows], tol[x][rows] = back(y), back(e * (1 + 1 / 16) + u * y.abs())
    return {x: (res[x], tol[x] * (1 + 1 / 16) + 1e-30) for x in res}


def within(got, value, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - value).abs() - bound
    if over.numel():
        worst = int(over.argmax())
        assert float(over.max()) <= 0, (
            f"{what}: value {worst} is {float((got - value).abs().flatten()[worst]):.3g} off, "
            f"bound {float(bound.flatten()[worst]):.3g}")


def frequencies(r, base, scaling="none", factor=1.0, length=0, low=0.0, high=0.0):
    """theta_j of a rotary scaling, and its amplitude.  The tensor carries theta_j in
    64-bit mantissas too (attribute `ld`): at position 2^31 half a step of a
    double theta is 2^-22 of a radian already, as large as the fp32 bounds."""
    ld, two_pi = np.longdouble, 2 * np.arccos(np.longdouble(-1))
    j = np.arange(r // 2)
    b = ld(base) * (ld(factor) ** (ld(r) / ld(r - 2)) if scaling == "base" and r > 2 else ld(1))
    th, amp = b ** (-2 * j.astype(ld) / ld(r)), 1.0
    if scaling == "linear":
        th = th / ld(factor)
    if scaling == "bands":
        w = np.clip((length * th / two_pi - ld(low)) / (ld(high) - ld(low)), ld(0), ld(1))
        th = w * th + (1 - w) * th / ld(factor)
    if scaling == "ramp":
        def pair(turns):
            return r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), r - 1)
        w = np.clip((j.astype(ld) - lo) / ld(max(hi - lo, 0.001)), ld(0), ld(1))
        th, amp = (1 - w) * th + w * th / ld(factor), 0.1 * math.log(factor) + 1
    out = torch.from_numpy(th.astype(np.float64))
    out.ld = th
    return out, amp


def angles(positions, th):
    """position * theta_j modulo a turn, to 2^-30 of a radian at any position."""
    two_pi = 2 * np.arccos(np.longdouble(-1))
    a = positions.cpu().numpy().astype(np.longdouble)[:, None] * th.ld
    a = a - two_pi * np.floor(a / two_pi)
    return torch.from_numpy(a.astype(np.float64)).to(positions.device)


def rotated(x, positions, th, amp, layout, sense=1.0):
    """(value, bound) of the rotation of x [rows, heads, d] in 64 bits.

    fp32: the angle's half turns (1 rounding of a float, pi 2^-25 of angle and the
    same again for the sine), the amplitude, two products and a sum: 8 half steps
    2^-24 of a (|x1| + |x2|) cover them; then the output's rounding."""
    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    r = 2 * th.numel()
    ang = angles(positions, th)[:, None]
    c, s = amp * ang.cos(), sense * amp * ang.sin()
    y = x.double()
    i1, i2 = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else \
        (slice(0, r, 2), slice(1, r, 2))
    out, bound = y.clone(), torch.zeros_like(y)
    out[..., i1] = y[..., i1] * c - y[..., i2] * s
    out[..., i2] = y[..., i1] * s + y[..., i2] * c
    size = abs(amp) * (y[..., i1].abs() + y[..., i2].abs())
    bound[..., i1] = 8 * 2.0 ** -24 * size
    bound[..., i2] = 8 * 2.0 ** -24 * size
    bound[..., :r] += u * out[..., :r].abs() + 1e-30
    return out, bound * (1 + 2.0 ** -6)
