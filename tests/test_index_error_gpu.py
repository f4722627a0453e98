"""A volume's index that holds the timeout bit: every call leaves its outputs alone."""
from types import SimpleNamespace

import pytest
import torch

from local_global_attention_b200 import pack3d as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(96, "bf16"), (48, "bf16"), (48, "fp32"), (96, "fp32")])
def test_calls_with_the_timeout_bit_write_nothing(d, dtype):
    """The bit that a kernel sets when a bounded wait gives up, written here by the host:
    the check reports it, and building the index anew clears it."""
    sh = SimpleNamespace(B=1, H=2, d=d, Z=4, Y=8, X=16, window=(3, 5, 5), block=(4, 4, 8),
                         rope_base=100.0, dtype=dtype)
    n, dt = 4 * 8 * 16, {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(0)
    q, k, v, dout = (torch.randn(1, n, 2, d, generator=g).to(dt).cuda() for _ in range(4))
    zyx = torch.cartesian_prod(torch.arange(4), torch.arange(8), torch.arange(16))
    coords = zyx.to(torch.int16)[None].cuda()
    op = P.Pack3D(sh)
    op.build_index(coords)
    out, lse = op.forward(q, k, v)
    ksum, vsum = P.pack3d_block_summaries(op.params, op.index, k, v)
    op.index.arrays()["err"][0] = 4
    assert P.pack3d_index_check(op.index) == P.ERR_TIMEOUT
    kept = [torch.full_like(x, 7) for x in (ksum, vsum, out, out, q, k, v)]
    l1, l2 = torch.full_like(lse, 7), torch.full_like(lse, 7)
    P.pack3d_block_summaries(op.params, op.index, k, v, kept[0], kept[1])
    P.pack3d_forward(op.params, op.index, q, k, v, ksum, vsum, kept[2], l1)
    P.pack3d_window_forward(op.params, op.index, q, k, v, kept[3], l2)
    P.pack3d_backward(op.params, op.index, q, k, v, out, lse, dout, *kept[4:])
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in (*kept, l1, l2))
    op.build_index(coords)
    got = op.forward(q, k, v)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
