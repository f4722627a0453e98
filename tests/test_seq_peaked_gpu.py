"""Logits that move the running maximum of the softmax after the first key tile, or never
again, at every head dim the kernels are built for; forward and backward against the
formulas in 64 bits."""
import math

import pytest
import torch

import seq_common as S
from local_global_attention_b200 import pack3d as P

pytestmark = pytest.mark.gpu


def inputs(lens, heads, kv_heads, dim, dtype, size, seed=0):
    """Logits along a sequence's keys from -size to size (even heads) and back (odd ones),
    beside a random part of about a hundredth of that."""
    q, k, v, dout = S.make(lens, heads, kv_heads, dim, dtype, seed)
    ramp = torch.cat([torch.linspace(-1, 1, n) if n > 1 else torch.zeros(n) for n in lens]).cuda()
    sign = torch.tensor([1.0, -1.0]).repeat(heads)[:heads].cuda()
    k2 = 0.05 * k.float() + (ramp * size / (4 * math.sqrt(dim)))[:, None, None]
    q2 = 0.05 * q.float() + 4 * sign[None, :, None]
    return q2.to(q.dtype), k2.to(k.dtype), v, dout


def logits(lens, q, k, causal):
    """Per sequence: S [heads, n, n] in 64 bits, -inf where masked."""
    G, at = q.shape[1] // k.shape[1], 0
    for n in lens:
        qs = q[at:at + n].double().transpose(0, 1)
        ks = k[at:at + n].double().transpose(0, 1).repeat_interleave(G, 0)
        s = qs @ ks.transpose(1, 2) / math.sqrt(q.shape[2])
        if causal:
            s = s.masked_fill(torch.ones(n, n, device=q.device).triu(1).bool(), -math.inf)
        yield at, n, s
        at += n


def rescales(lens, q, k, causal):
    """(rows whose maximum, kept until a tile of 128 keys tops it by 8 in powers of two,
    moves after the first tile; rows that see more than one tile and where it does not)"""
    moved = stayed = 0
    for _, n, s in logits(lens, q, k, causal):
        m, any_ = None, None
        for c in range(0, n, 128):
            top = s[..., c:c + 128].amax(-1) / math.log(2)
            if m is None:
                m, any_ = top, torch.zeros_like(top, dtype=torch.bool)
                continue
            up = top > m + 8
            any_ |= up
            m = torch.where(up, top, m)
        rows = torch.arange(n, device=q.device)[None].expand_as(any_)
        several = rows >= 128 if causal else torch.full_like(any_, n > 128)
        moved += int((any_ & several).sum())
        stayed += int((~any_ & several).sum())
    return moved, stayed


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 72, 96, 128])
def test_maximum_moves_after_the_first_tile(dim, causal, dtype):
    """Logits within 16: the bounds of seq_common hold as they stand."""
    lens, H, K = [700, 90, 385], 4, 2
    q, k, v, dout = inputs(lens, H, K, dim, dtype, 14, dim)
    moved, stayed = rescales(lens, q, k, causal)
    assert moved > 500 and stayed > 500
    p = P.make_seq_params(len(lens), sum(lens), H, K, dim, causal, dtype)
    ix = P.pack3d_seq_build_index(p, torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda"))
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    ref = S.reference(lens, q, k, v, dout, causal, dtype=dtype)
    assert max(float(s[s > -math.inf].abs().max()) for *_, s in logits(lens, q, k, causal)) <= 16
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        S.within(got, *ref[name], f"{name} d{dim} causal {causal} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 72, 96, 128])
def test_logits_of_several_hundred(dim, causal, dtype):
    """|S| <= A = 300.  Per value, as in seq_common, with rho for these logits: the dot
    product's 2 d 2^-24 tau |q| |k|, 2^-20 for the exponential, and for scaling, lse and
    its way back to powers of two five roundings of A log2 e: 8 A 2^-24 covers them."""
    lens, H, K = [600], 2, 1
    q, k, v, dout = inputs(lens, H, K, dim, dtype, 280, dim + 1)
    moved, stayed = rescales(lens, q, k, causal)
    assert moved > 250 and stayed > 250
    n, tau = lens[0], 1 / math.sqrt(dim)
    p = P.make_seq_params(1, n, H, K, dim, causal, dtype)
    ix = P.pack3d_seq_build_index(p, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    dq, dk, dv = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    u = S.TYPES[dtype][1]
    uo = u if dtype == "bf16" else 0.0
    qs, do = (x.double().transpose(0, 1) for x in (q, dout))
    ks, vs = (x.double().transpose(0, 1).expand(H, n, dim) for x in (k, v))
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    s = tau * qs @ t(ks)
    A = float(s.abs().max())
    assert 200 < A <= 300
    rho = float(2 * dim * 2 ** -24 * (tau * qs.abs() @ t(ks).abs()).max()) + 2 ** -20 + 8 * A * 2 ** -24
    if causal:
        s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
    z = torch.logsumexp(s, -1)
    w = torch.exp(s - z[..., None])
    o = w @ vs
    add = 2 * n * 2 ** -24
    e_o = (uo + 2 * rho + add) * (w @ vs.abs()) + u * o.abs()
    dp = do @ t(vs)
    ds = w * (dp - (do * o).sum(-1, keepdim=True))
    e_delta = (do.abs() * (e_o + 2 * dim * 2 ** -24 * o.abs())).sum(-1, keepdim=True)
    e_dp = 2 * dim * 2 ** -24 * (do.abs() @ t(vs).abs())
    e_ds = (uo + H * add) * ds.abs() + w * (e_delta + e_dp) + \
        2 * rho * w * (dp - (do * o).sum(-1, keepdim=True)).abs()
    both = lambda x: x.sum(0, keepdim=True)  # noqa: E731
    want = {"out": (o, e_o), "dq": (tau * ds @ ks, tau * e_ds @ ks.abs()),
            "dk": (both(tau * t(ds) @ qs), both(tau * t(e_ds) @ qs.abs())),
            "dv": (both(t(w) @ do), both((uo + 2 * rho + H * add) * t(w) @ do.abs()))}
    assert float((lse.double() - z).abs().max()) <= rho + add + 2 ** -23 * A
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        x, e = want[name]
        # (second order terms, as in seq_common)
        S.within(got.transpose(0, 1), x, (e + u * x.abs()) * (1 + 1 / 8) + 1e-30, f"{name} d{dim}")
