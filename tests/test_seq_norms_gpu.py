"""Packed-sequence attention against 64 bits in the 2-norm (an error that all values
share, such as a factor, passes bounds of single values that are as large as a rounding),
over longer sequences and heads that share one key/value head.

A rounding to bf16 of values spread over their binades is off by 2^-7 / sqrt(12) times
the root mean square of 1/m, m log-uniform over [1, 2): 0.00166 relative.  Independent
roundings add in squares: out and dv hold two (P and the output), dq and dk three (dS,
the output, and out inside delta, which over rows of many keys weighs no more than dS's
own).  15 % of room for the spread of a sample.

fp32: sums of n products and of d, random signs: (sqrt(n) + sqrt(d) + 8) half steps."""
import math

import pytest
import torch

import seq_common as S
from local_global_attention_b200 import pack3d as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,heads,kv_heads,dim,causal,dtype", [
    ([4096], 16, 1, 64, True, "bf16"), ([2500, 1200], 16, 2, 128, True, "bf16"),
    ([3000, 513], 8, 8, 96, False, "bf16"), ([9000], 2, 1, 96, True, "bf16"),
    ([5000, 1], 2, 2, 128, False, "bf16"), ([2048, 300], 16, 1, 48, True, "fp32"),
    ([4100], 2, 1, 128, True, "fp32"), ([1500], 4, 4, 96, False, "fp32")], ids=str)
def test_norms_of_longer_sequences(lens, heads, kv_heads, dim, causal, dtype):
    p = P.make_seq_params(len(lens), sum(lens), heads, kv_heads, dim, causal, dtype)
    ix = P.pack3d_seq_build_index(p, torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda"))
    q, k, v, dout = S.make(lens, heads, kv_heads, dim, dtype, sum(lens))
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    assert P.pack3d_seq_index_check(ix) == P.OK
    ref = S.reference(lens, q, k, v, dout, causal, dtype=dtype)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        value, bound = ref[name]
        S.within(got, value, bound, name)
        if name == "lse":
            continue
        off = float((got.double() - value).norm() / value.norm())
        if dtype == "bf16":
            room = 1.15 * 0.00166 * math.sqrt(2 if name in ("out", "dv") else 3)
        else:
            room = (math.sqrt(max(lens) * heads / kv_heads) + math.sqrt(dim) + 8) * 2.0 ** -24
        assert off <= room, f"{name}: {off:.3g} off in the 2-norm, bound {room:.3g}"
        # the factor that fits best: random errors of 0.003 over 10^5 values and more
        # leave it within 10^-4 of 1
        fit = float((got.double() * value).sum() / (value * value).sum())
        assert abs(fit - 1) <= (1e-4 if dtype == "bf16" else room), f"{name}: scaled by {fit}"
