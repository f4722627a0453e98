"""Host-side behaviour of the packed-sequence calls beside their refusals: no GPU."""
import pytest

from local_global_attention_b200 import build as B
from local_global_attention_b200 import pack3d as P

FAKE, WS = 1 << 30, 1 << 32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load()


def test_zeroing_flag_is_no_type(lib):
    """The flag stands beside either type and changes no size; alone with another
    type it is refused as that type is."""
    for dtype in ("bf16", "fp32"):
        p = P.make_seq_params(3, 1000, 8, 2, 96, dtype=dtype)
        need = lib.pack3d_seq_index_bytes(p), lib.pack3d_seq_backward_workspace_bytes(p)
        p.dtype |= P.ZERO_UNUSED_ROWS
        assert need == (lib.pack3d_seq_index_bytes(p), lib.pack3d_seq_backward_workspace_bytes(p))
        p.n_tokens = 0
        ix = P.SeqIndexStruct()
        assert lib.pack3d_seq_index_init(p, WS, 1 << 40, ix) == P.OK
        assert lib.pack3d_seq_forward(p, ix, None, *[None] * 6) == P.OK
        r = P.make_rotary_params(96, dtype=dtype)
        r.Hq, r.dtype = 8, r.dtype | P.ZERO_UNUSED_ROWS
        assert lib.pack3d_rotary(r, *[None] * 6) == P.OK
    for bad in (2 | P.ZERO_UNUSED_ROWS, P.ZERO_UNUSED_ROWS << 1):
        p.dtype = r.dtype = bad
        assert lib.pack3d_seq_index_bytes(p) == 0
        assert lib.pack3d_rotary(r, *[None] * 6) == P.ERR_ARG
