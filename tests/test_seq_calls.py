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


def test_wrapper_keeps_a_forward_with_its_index(monkeypatch):
    """SeqAttention's bookkeeping, with the calls beneath it replaced: the backward runs
    with its forward's index, and not once that has been built anew."""
    class Index:
        builds, positions = 1, None

    seen = []
    monkeypatch.setattr(P, "pack3d_seq_forward", lambda p, ix, q, k, v, stream: ("out", "lse"))
    monkeypatch.setattr(P, "pack3d_seq_backward", lambda p, ix, *a, stream: seen.append(ix) or a[:3])
    capturing = [False]
    monkeypatch.setattr(P.torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    op, own, other = P.SeqAttention(None), Index(), Index()
    op.index = own
    first = op.forward("q", "k", "v")
    second = op.forward("q", "k", "v", index=other)
    assert first[2] == ("q", "k")
    op.backward(second[2], "v", "out", "lse", "dout")
    op.backward(first[2], "v", "out", "lse", "dout")
    assert seen == [other, own]
    own.builds += 1
    with pytest.raises(ValueError):
        op.backward(first[2], "v", "out", "lse", "dout")
    with pytest.raises(ValueError):
        op.backward(second[2], "v", "out", "lse", "dout", index=own)
    op.backward(second[2], "v", "out", "lse", "dout", index=other)
    op.backward(("q", "k"), "v", "out", "lse", "dout")
    assert seen[2:] == [other, own]
    # a captured forward follows the index
    capturing[0] = True
    third = op.forward("q", "k", "v")
    own.builds += 1
    op.backward(third[2], "v", "out", "lse", "dout")
    assert seen[4:] == [own]


def rotary_status(lib, call, **kw):
    """Status of a call without rows: the checks alone."""
    r = P.make_rotary_params(96, **kw)
    r.Hq = 8
    return getattr(lib, call)(r, *[None] * 6)


@pytest.mark.parametrize("call", ["pack3d_rotary", "pack3d_rotary_backward"])
def test_rotary_bases(lib, call):
    """Bases whose fastest pair makes too many turns per position to keep its angle's
    bits are refused, and none else: the pair of base 0.01 makes 0.01^(-94/96) / (2 pi)
    = 14.5 turns, that of 0.0085 17.0."""
    for base in (1e-38, 1e-10, 1e-3, 0.0085):
        assert rotary_status(lib, call, base=base) == P.ERR_ARG, base
        assert rotary_status(lib, call, base=base, scaling="linear", factor=1.0) == P.ERR_ARG
    for base in (0.01, 0.25, 0.999, 1.0, 1.5, 100.0, 5e5, 3e38):
        assert rotary_status(lib, call, base=base) == P.OK, base
    # a scaling that slows the pairs down, and a head with one pair
    assert rotary_status(lib, call, base=1e-3, scaling="linear", factor=16.0) == P.OK
    assert rotary_status(lib, call, base=1e-38, rot_dim=2) == P.OK
    assert rotary_status(lib, call, base=1e-3, scaling="base", factor=1000.0) == P.OK


def test_views_of_an_index_whose_params_changed_since(lib):
    """The views are of the rows that the buffer was sized for, whatever the caller's
    params say by then."""
    p = P.make_seq_params(3, 1000, 8, 2, 96)
    ix = P.SeqIndex(p, device="cpu")
    p.n_tokens = 5000
    assert ix.positions.numel() == ix.sequences.numel() == 1000
    p.n_tokens = 10
    assert ix.positions.numel() == ix.sequences.numel() == 1000
