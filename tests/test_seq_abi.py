"""Host-side checks of the packed-sequence calls: they need no GPU and refuse
before anything is launched."""
import ctypes

import pytest
import torch

from local_global_attention_b200 import build as B
from local_global_attention_b200 import pack3d as P

FAKE, WS = 1 << 30, 1 << 32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load()


def params(**kw):
    base = dict(n_seqs=3, n_tokens=1000, heads=8, kv_heads=2, head_dim=96)
    base.update(kw)
    return P.make_seq_params(**base)


def index(lib, p):
    ix = P.SeqIndexStruct()
    assert lib.pack3d_seq_index_init(p, WS, 1 << 40, ix) == P.OK
    return ix


def forward(lib, p, ix, st=None, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE):
    return lib.pack3d_seq_forward(p, ix, st, q, k, v, out, lse, None)


def backward(lib, p, ix, st=None, ws=WS, nbytes=1 << 40, **kw):
    a = {n: kw.get(n, FAKE) for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv")}
    return lib.pack3d_seq_backward(p, ix, st, *a.values(), ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(n_seqs=0), dict(n_seqs=-1), dict(n_tokens=-1), dict(n_tokens=(1 << 30) + 1),
    dict(heads=0), dict(heads=8, kv_heads=3), dict(kv_heads=0), dict(head_dim=0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(heads=65536, kv_heads=1),
    dict(n_tokens=1 << 30, heads=4096, kv_heads=1)])
def test_bad_params(lib, bad):
    p = params(**bad)
    assert lib.pack3d_seq_index_bytes(p) == 0
    assert lib.pack3d_seq_backward_workspace_bytes(p) == 0
    assert lib.pack3d_seq_index_init(p, WS, 1 << 40, P.SeqIndexStruct()) == P.ERR_ARG
    assert forward(lib, p, P.SeqIndexStruct()) == P.ERR_ARG
    assert backward(lib, p, P.SeqIndexStruct()) == P.ERR_ARG


def test_bad_dtype(lib):
    p = params()
    p.dtype = 2
    assert forward(lib, p, P.SeqIndexStruct()) == P.ERR_ARG


@pytest.mark.parametrize("d", [4, 12, 100, 132, 136, 256])
def test_head_dims_not_built(lib, d):
    p = params(head_dim=d)
    assert lib.pack3d_seq_index_init(p, WS, 1 << 40, P.SeqIndexStruct()) == P.ERR_UNSUPPORTED


def test_index_sizes(lib):
    p = params()
    need = lib.pack3d_seq_index_bytes(p)
    # positions and sequence numbers, then the tile lists: at most
    # floor(rows / tile) + sequences entries of 16 bytes
    a = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert need == 2 * a(4000) + a(16 * (3 + 3)) + 2 * a(16 * (7 + 3)) + 256
    ix = P.SeqIndexStruct()
    assert lib.pack3d_seq_index_init(p, WS, need - 1, ix) == P.ERR_ARG
    assert lib.pack3d_seq_index_init(p, WS + 16, need, ix) == P.ERR_ARG
    assert lib.pack3d_seq_index_init(p, None, need, ix) == P.ERR_ARG
    assert lib.pack3d_seq_index_init(p, WS, need, ix) == P.OK
    assert (ix.n_pair, ix.n_rows) == (6, 10)
    assert lib.pack3d_seq_build_index(p, None, ix, None) == P.ERR_ARG
    assert lib.pack3d_seq_build_index(p, FAKE + 2, ix, None) == P.ERR_ARG
    assert lib.pack3d_seq_build_index(p, FAKE, P.SeqIndexStruct(), None) == P.ERR_ARG
    assert lib.pack3d_seq_index_check(None, None) == P.ERR_ARG


@pytest.mark.parametrize("built,used", [(dict(n_tokens=896), dict(n_tokens=1023)),
                                        (dict(n_tokens=1023), dict(n_tokens=896)),
                                        (dict(n_seqs=4, n_tokens=128), dict(n_seqs=5, n_tokens=0))])
def test_index_of_other_params(lib, built, used):
    """An index whose lists have the same lengths but whose rows were sized for
    other params (896 rows end where 1,023 rows would still write)."""
    ix, n0 = index(lib, params(**built)), P.pack3d_kernel_launches()
    p = params(**used)
    other = index(lib, p)
    assert (ix.n_rows == other.n_rows) and ix.n_tokens != other.n_tokens
    assert lib.pack3d_seq_build_index(p, FAKE, ix, None) == P.ERR_ARG
    assert forward(lib, p, ix) == P.ERR_ARG and backward(lib, p, ix) == P.ERR_ARG
    assert P.pack3d_kernel_launches() == n0


@pytest.mark.parametrize("what", ["q", "k", "v", "out", "lse"])
def test_forward_pointers(lib, what):
    p = params()
    ix, n0 = index(lib, p), P.pack3d_kernel_launches()
    assert forward(lib, p, ix, **{what: None}) == P.ERR_ARG
    assert forward(lib, p, ix, **{what: FAKE + 2}) == P.ERR_ARG
    # an index of another shape
    assert forward(lib, params(n_tokens=1500), ix) == P.ERR_ARG
    assert P.pack3d_kernel_launches() == n0


@pytest.mark.parametrize("what", ["q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"])
def test_backward_pointers(lib, what):
    p = params()
    ix, n0 = index(lib, p), P.pack3d_kernel_launches()
    need = lib.pack3d_seq_backward_workspace_bytes(p)
    assert need == 2 * ((4 * 8 * 1000 + 255) // 256 * 256)
    assert backward(lib, p, ix, **{what: None}) == P.ERR_ARG
    assert backward(lib, p, ix, **{what: FAKE + 2}) == P.ERR_ARG
    for ws, nbytes in ((None, need), (WS + 16, need), (WS, need - 1)):
        assert backward(lib, p, ix, ws=ws, nbytes=nbytes) == P.ERR_ARG
    assert P.pack3d_kernel_launches() == n0


@pytest.mark.parametrize("st", [dict(q=8 * 96 - 8), dict(q=8 * 96 + 4), dict(k=96), dict(v=-8),
                                dict(out=760), dict(q=1 << 37)])
def test_strides(lib, st):
    p = params()
    assert forward(lib, p, index(lib, p), P.SeqStrides(**st)) == P.ERR_ARG


def test_no_rows(lib):
    """Only empty sequences: nothing to do, nothing launched."""
    p = params(n_tokens=0)
    ix, n0 = index(lib, p), P.pack3d_kernel_launches()
    assert forward(lib, p, ix, q=None, k=None, v=None, out=None, lse=None) == P.OK
    assert backward(lib, p, ix, ws=None, nbytes=0) == P.OK
    assert P.pack3d_kernel_launches() == n0


def rotary(lib, pos=FAKE, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, call="pack3d_rotary", **kw):
    base = dict(head_dim=96, rot_dim=96)
    fields = {n: kw.pop(n) for n in list(kw) if n in dict(P.RotaryParams._fields_) and n not in
              ("base", "factor", "low", "high", "amplitude", "original_length", "head_dim",
               "rot_dim", "scaling", "layout", "dtype")}
    raw = {n: kw.pop(n) for n in list(kw) if n in ("scaling", "layout", "dtype") and
           isinstance(kw[n], int)}
    base.update(kw)
    p = P.make_rotary_params(**base)
    p.n_tokens, p.Hq, p.Hk = 10, 8, 2
    for n, x in {**fields, **raw}.items():
        setattr(p, n, x)
    return getattr(lib, call)(p, pos, q, k, qo, ko, None)


@pytest.mark.parametrize("call", ["pack3d_rotary", "pack3d_rotary_backward"])
@pytest.mark.parametrize("bad", [
    dict(pos=None), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(q=FAKE + 8),
    dict(ko=FAKE + 8), dict(pos=FAKE + 2), dict(rot_dim=0), dict(rot_dim=95), dict(rot_dim=98),
    dict(rot_dim=-2), dict(base=0.0), dict(base=float("nan")), dict(layout=2), dict(scaling=5),
    dict(dtype=2), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
    dict(scaling="bands", factor=2.0), dict(amplitude=-1.0),
    dict(scaling="bands", factor=2.0, original_length=100, low=4.0, high=4.0),
    dict(scaling="ramp", factor=2.0, original_length=100, low=1.0, high=8.0, base=1.0),
    dict(n_tokens=-1), dict(Hq=0), dict(Hk=-1), dict(stride_q=760), dict(stride_q=772),
    dict(stride_k_out=96), dict(stride_q=800), dict(base=1e-38, scaling="none", rot_dim=96,
                                                     head_dim=90)])
def test_rotary_refusals(lib, call, bad):
    n0 = P.pack3d_kernel_launches()
    st = rotary(lib, call=call, **bad)
    assert st in (P.ERR_ARG, P.ERR_UNSUPPORTED) and st != P.ERR_CUDA
    assert P.pack3d_kernel_launches() == n0


def test_rotary_no_rows_and_sizes(lib):
    assert rotary(lib, n_tokens=0, q=None, k=None, qo=None, ko=None, pos=None) == P.OK
    for d in (4, 100, 264):
        assert rotary(lib, head_dim=d, rot_dim=4) == P.ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    p = params(n_tokens=4)
    x = torch.zeros(4, 8, 96, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.pack3d_seq_build_index(p, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        P.pack3d_rotary(P.make_rotary_params(96), torch.zeros(4, dtype=torch.int32), x)
    with pytest.raises(KeyError):
        P.make_rotary_params(96, layout="other")
    with pytest.raises(KeyError):
        P.make_seq_params(1, 1, 1, dtype=torch.float16)


def test_strerror_lengths(lib):
    assert "lengths" in P.strerror(P.ERR_LENGTHS)
    assert ctypes.sizeof(P.SeqParams) == 32 and ctypes.sizeof(P.RotaryParams) == 88
