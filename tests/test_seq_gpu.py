"""Packed-sequence attention and rotary positions on the GPU against the
formulas in 64 bits, with bounds counted from the roundings (seq_common)."""
import pytest
import torch

import seq_common as S
from local_global_attention_b200 import pack3d as P

pytestmark = pytest.mark.gpu


def built(lens, heads, kv_heads, dim, causal, dtype, tail=0, scale=0.0):
    p = P.make_seq_params(len(lens), sum(lens) + tail, heads, kv_heads, dim, causal, dtype, scale)
    cu = torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda")
    ix = P.pack3d_seq_build_index(p, cu)
    assert P.pack3d_seq_index_check(ix) == P.OK
    return p, ix


def check(lens, heads, kv_heads, dim, causal, dtype, seed=0, fused=False, scale=0.0):
    p, ix = built(lens, heads, kv_heads, dim, causal, dtype, scale=scale)
    q, k, v, dout = S.make(lens, heads, kv_heads, dim, dtype, seed, fused)
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    assert P.pack3d_seq_index_check(ix) == P.OK
    ref = S.reference(lens, q, k, v, dout, causal, scale, dtype)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        S.within(got, *ref[name], f"{name} {lens} {heads}/{kv_heads} d{dim} {dtype}")


# ---- index ------------------------------------------------------------------------------


@pytest.mark.parametrize("lens,tail", [([1], 0), ([0], 5), ([0, 0, 3, 0], 0), ([128], 0), ([300], 7),
                                       ([255, 256, 257, 1, 0, 700], 3), ([5] * 400, 11),
                                       ([40000, 1, 9000], 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_index(lens, tail, causal):
    p, ix = built(lens, 2, 1, 64, causal, "bf16", tail)
    pos = [i for n in lens for i in range(n)] + [-1] * tail
    seq = [s for s, n in enumerate(lens) for _ in range(n)] + [-1] * tail
    assert ix.positions.tolist() == pos and ix.sequences.tolist() == seq
    cu = S.prefix(lens)
    for field, rows, count in (("pair", 256, ix.struct.n_pair), ("query", 128, ix.struct.n_rows),
                               ("key", 128, ix.struct.n_rows)):
        off = getattr(ix.struct, field) - ix.buffer.data_ptr()
        got = ix.buffer[off:off + 16 * count].view(torch.int32).view(count, 4).tolist()
        want = [[cu[s], n, t, 0] for s, n in enumerate(lens) for t in range(0, n, rows)]
        used = got[:len(want)]
        assert sorted(used) == sorted(want)
        assert all(t == [0, 0, 0, 0] for t in got[len(want):])
        cols = [(n if not causal else n - t if field == "key" else min(n, t + rows)) // 128
                for _, n, t, _ in used]
        assert cols == sorted(cols, reverse=True)


@pytest.mark.parametrize("cu", [[1, 5, 10], [0, 6, 5], [0, 5, 11], [0, -1, 10], [-2, 5, 10],
                                [0, 2 ** 31 - 1, 10]])
def test_bad_lengths_write_nothing(cu):
    p = P.make_seq_params(2, 10, 2, 2, 64, dtype="bf16")
    ix = P.pack3d_seq_build_index(p, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert P.pack3d_seq_index_check(ix) == P.ERR_LENGTHS
    q, k, v, dout = S.make([10], 2, 2, 64, "bf16")
    kept = [torch.full_like(q, 7) for _ in range(4)]
    lse = torch.full((2, 10), 7.0, device="cuda")
    P.pack3d_seq_forward(p, ix, q, k, v, kept[0], lse)
    P.pack3d_seq_backward(p, ix, q, k, v, q, lse, dout, *kept[1:])
    assert all((x == 7).all() for x in (*kept, lse))
    # the same buffer with good lengths
    P.pack3d_seq_build_index(p, torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda"), ix)
    assert P.pack3d_seq_index_check(ix) == P.OK


# ---- attention ----------------------------------------------------------------------------

LENS = [[1], [2], [0, 1, 0], [127], [128], [129], [64, 1, 200, 0, 33], [255, 256, 257], [513],
        [384, 385], [1, 1, 1, 1, 130]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, causal, dtype):
    check(lens, 2, 1, 96, causal, dtype, seed=sum(lens))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [8, 16, 24, 48, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128])
def test_head_dims(dim, dtype):
    check([150, 40, 300], 2, 2, dim, True, dtype, seed=dim)
    check([140], 2, 2, dim, False, dtype, seed=dim)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (6, 2), (8, 8), (16, 2)])
@pytest.mark.parametrize("fused", [False, True])
def test_heads_and_strides(heads, kv, fused, dtype):
    check([70, 333, 1, 129], heads, kv, 64, True, dtype, seed=heads, fused=fused)
    check([70, 333, 1, 129], heads, kv, 128, False, dtype, seed=heads, fused=fused)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_longer_and_scale(dtype):
    check([1500, 700], 4, 2, 96, True, dtype, seed=1)
    check([1200, 100], 2, 2, 128, False, dtype, seed=2, scale=0.2)
    check([2300], 2, 1, 64, True, dtype, seed=3, scale=0.05)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_outputs_and_tail_rows(dtype):
    """Outputs as slices of larger tensors, rows behind the last sequence: only
    the sequences' rows of the slices are written."""
    lens, tail, H, K, d = [100, 0, 190], 37, 4, 2, 48
    p, ix = built(lens, H, K, d, True, dtype, tail)
    n = sum(lens)
    q, k, v, dout = S.make(lens, H, K, d, dtype, 5, True, tail)
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    big = torch.full((n + tail, H + 2 * K + 1, d), 3.0, dtype=q.dtype, device="cuda")
    fo = torch.full((n + tail, 2 * H, d), 3.0, dtype=q.dtype, device="cuda")
    fl = torch.full((H, n + tail), 3.0, device="cuda")
    P.pack3d_seq_forward(p, ix, q, k, v, fo[:, H:], fl)
    assert torch.equal(fo[:n, H:], out[:n]) and torch.equal(fl[:, :n], lse[:, :n])
    assert (fo[:, :H] == 3).all() and (fo[n:] == 3).all() and (fl[:, n:] == 3).all()
    wide = torch.zeros(n + tail, H + 1, d, dtype=q.dtype, device="cuda")
    wide[:, 1:] = dout
    P.pack3d_seq_backward(p, ix, q, k, v, fo[:, H:], fl, wide[:, 1:], big[:, :H],
                          big[:, H:H + K], big[:, H + K:H + 2 * K])
    for got, want in zip((big[:n, :H], big[:n, H:H + K], big[:n, H + K:H + 2 * K]), grads):
        assert torch.equal(got, want[:n])
    assert (big[:, H + 2 * K:] == 3).all() and (big[n:] == 3).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
def test_other_sequences_never_reach_a_row(bad, dtype, causal):
    """A sequence beside one full of non-finite values, and before rows of no
    sequence that hold them, gives the bits it gives alone."""
    lens, tail, H, K, d = [150, 61, 300], 20, 2, 1, 96
    p, ix = built(lens, H, K, d, causal, dtype, tail)
    q, k, v, dout = S.make(lens, H, K, d, dtype, 9, False, tail)
    clean = P.pack3d_seq_forward(p, ix, q, k, v)
    cg = P.pack3d_seq_backward(p, ix, q, k, v, *clean, dout)
    for x in (q, k, v, dout):
        x[150:211] = bad
        x[511:] = bad
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    # the rows of no sequence hold the bad values in out and lse too
    o2, l2 = out.clone(), lse.clone()
    o2[511:], l2[:, 511:] = bad, bad
    grads = P.pack3d_seq_backward(p, ix, q, k, v, o2, l2, dout)
    keep = list(range(150)) + list(range(211, 511))
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
    for a, b in zip(grads, cg):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_peaked_logits(dtype):
    """Logits of several hundred, rising and falling along the keys: the running
    maximum moves at every tile, or never again after the first."""
    lens, d = [700], 64
    p, ix = built(lens, 1, 1, d, False, dtype)
    q, k, v, dout = S.make(lens, 1, 1, d, dtype, 4)
    for order in (1, -1):
        ramp = torch.linspace(-1, 1, 700, device="cuda") * order
        kk = (k.float() * 0.05 + ramp[:, None, None] * 8).to(k.dtype)
        qq = (q.float() * 0.05 + 4).to(q.dtype)
        out, lse = P.pack3d_seq_forward(p, ix, qq, kk, v)
        s = (qq[:, 0].double() @ kk[:, 0].double().T) / 8
        ref = torch.logsumexp(s, 1)
        assert float(s.max()) > 200
        # |S| <= 260 here: scaled in fp32 to 2^-23 of its size (2^-15 absolute), and
        # the dot product's 2 d 2^-24 |q| |k| / 8 below 2^-9
        tol = 2.0 ** -9 + 2.0 ** -14
        assert float((lse[0].double() - ref).abs().max()) <= tol
        pr = torch.exp(s - ref[:, None])
        u = S.TYPES[dtype][1]
        e = (u + 4 * tol) * (pr @ v[:, 0].double().abs()) + u * (pr @ v[:, 0].double()).abs()
        assert ((out[:, 0].double() - pr @ v[:, 0].double()).abs() <= e).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_against_differences(dtype):
    """The gradient's inner product with a direction against a central
    difference of the formula in 64 bits."""
    lens = [90, 140]
    p, ix = built(lens, 2, 1, 48, True, dtype)
    q, k, v, dout = S.make(lens, 2, 1, 48, dtype, 8)
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    ref = S.reference(lens, q, k, v, dout, True, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(0)
    xs = [x.double() for x in (q, k, v)]

    def loss(*x):
        r = S.reference(lens, *x, dout.double(), True, dtype=dtype)["out"][0]
        return float((r * dout.double()).sum())

    for i, name in enumerate(("dq", "dk", "dv")):
        w = torch.randn(xs[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        hi, lo = list(xs), list(xs)
        hi[i], lo[i] = xs[i] + h * w, xs[i] - h * w
        diff = (loss(*hi) - loss(*lo)) / (2 * h)
        got = float((grads[i].double() * w).sum())
        # the values' bounds, and 1e-6 of the sum's size for the difference itself
        room = float((ref[name][1] * w.abs()).sum()) + 1e-6 * float(
            (ref[name][0] * w).abs().sum())
        assert abs(got - diff) <= room


# ---- how calls are made -------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeated_streams_and_graph(dtype):
    """The same bits from call to call, on a side stream, from two streams at
    once and from a replayed graph whose inputs change."""
    lens = [300, 77, 512]
    p, ix = built(lens, 4, 2, 96, True, dtype)
    sets = [S.make(lens, 4, 2, 96, dtype, s) for s in (1, 2)]

    def both(x, **kw):
        out, lse = P.pack3d_seq_forward(p, ix, *x[:3], **kw)
        return (out, lse, *P.pack3d_seq_backward(p, ix, *x[:3], out, lse, x[3], **kw))

    want = [both(x) for x in sets]
    again = [both(x) for x in sets]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    side = [both(x, stream=s) for _ in range(3) for x, s in zip(sets, (a, b))][-2:]
    raw = both(sets[0], stream=a.cuda_stream)
    torch.cuda.synchronize()
    for got in (again, side, [raw]):
        for x, y in zip(want, got):
            assert all(torch.equal(m, n) for m, n in zip(x, y))
    static = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both(static)
    for x, y in zip(sets[::-1], want[::-1]):
        for s, t in zip(static, x):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(res, y))
    assert P.pack3d_seq_index_check(ix) == P.OK


def test_memory_of_a_given_stream():
    """Outputs of a call on a given stream never stand in memory that work queued
    on the caller's stream still reads, although its owner is gone."""
    n, H, d = 16384, 16, 128
    q = torch.ones(n, H, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    p = P.make_rotary_params(d)
    side = torch.cuda.Stream()
    total = torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda")
    P.pack3d_rotary(p, pos, q, stream=side)
    torch.cuda.synchronize()
    x = torch.ones(n, H, d, dtype=torch.bfloat16, device="cuda")
    for _ in range(200):
        total.add_(x)
    del x
    outs = [P.pack3d_rotary(p, pos, q, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert (total == 200).all()  # whole numbers up to 256 are exact in bf16
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_index_built_in_a_graph():
    """Lengths that change between replays of one captured graph."""
    p = P.make_seq_params(3, 400, 2, 1, 64, True, "bf16")
    q, k, v, dout = S.make([400], 2, 1, 64, "bf16", 3)
    cu = torch.tensor(S.prefix([100, 200, 100]), dtype=torch.int32, device="cuda")
    ix = P.pack3d_seq_build_index(p, cu)
    P.pack3d_seq_forward(p, ix, q, k, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pack3d_seq_build_index(p, cu, ix)
        out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    for lens in ([400, 0, 0], [1, 398, 1], [130, 130, 140]):
        cu.copy_(torch.tensor(S.prefix(lens), dtype=torch.int32))
        graph.replay()
        assert P.pack3d_seq_index_check(ix) == P.OK
        ref = S.reference(lens, q, k, v, dout, True)
        S.within(out, *ref["out"], f"out {lens}")
        S.within(lse, *ref["lse"], f"lse {lens}")


def test_binding_refusals():
    lens = [10, 20]
    p, ix = built(lens, 2, 1, 64, True, "bf16")
    q, k, v, dout = S.make(lens, 2, 1, 64, "bf16")
    wide = torch.zeros(30, 64, 2, dtype=q.dtype, device="cuda")
    for bad in ((q.float(), k, v), (q[:29], k, v), (q, k[:, :, :32], v), (q, k, v.cpu()),
                (wide.transpose(1, 2), k, v), (q[:1].expand(30, 2, 64), k, v)):
        with pytest.raises(ValueError):
            P.pack3d_seq_forward(p, ix, *bad)
    with pytest.raises(ValueError):
        P.pack3d_seq_forward(p, ix, q, k, v, lse=torch.empty(30, 2, device="cuda"))
    off = torch.zeros(30 * 2 * 64 + 4, dtype=q.dtype, device="cuda")[4:].view(30, 2, 64)
    with pytest.raises(P.Pack3dError):  # not on a 16-byte boundary
        P.pack3d_seq_forward(p, ix, off, k, v)
    with pytest.raises(ValueError):
        P.pack3d_seq_build_index(p, torch.zeros(4, dtype=torch.int32, device="cuda"))


def test_index_that_was_never_built():
    p = P.make_seq_params(2, 300, 2, 1, 64, True, "bf16")
    ix = P.SeqIndex(p)
    q, k, v, dout = S.make([300], 2, 1, 64, "bf16")
    kept = [torch.full_like(q, 7) for _ in range(2)]
    lse = torch.zeros(2, 300, device="cuda")
    P.pack3d_seq_forward(p, ix, q, k, v, kept[0], lse)
    P.pack3d_seq_backward(p, ix, q, k, v, q, lse, dout, dq=kept[1])
    assert all((x == 7).all() for x in kept) and not lse.any()
    with pytest.raises(P.Pack3dError):  # an index of other params
        P.pack3d_seq_forward(P.make_seq_params(2, 301, 2, 1, 64), ix, *S.make([301], 2, 1, 64,
                                                                             "bf16")[:3])


def test_empty_pack():
    p, ix = built([0, 0], 2, 1, 64, True, "bf16")
    q, k, v, dout = S.make([0], 2, 1, 64, "bf16")
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    grads = P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0) and grads[1].shape == (0, 1, 64)


# ---- rotary -------------------------------------------------------------------------------

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="bands", factor=8.0, original_length=8192, low=1.0, high=4.0),
            dict(scaling="ramp", factor=32.0, original_length=4096, low=1.0, high=32.0)]


def rotary_check(n, heads, kv, d, r, layout, dtype, base=10000.0, far=1 << 20, seed=0, amplitude=0.0,
                 **scaling):
    dt = S.TYPES[dtype][0]
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(n, heads, d, generator=g).to(dt).cuda()
    k = torch.randn(n, kv, d, generator=g).to(dt).cuda() if kv else None
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int64).to(torch.int32).cuda()
    p = P.make_rotary_params(d, r, layout, base, dtype, amplitude=amplitude, **scaling)
    th, amp = S.frequencies(r, base, scaling.get("scaling", "none"), scaling.get("factor", 1.0),
                            scaling.get("original_length", 0), scaling.get("low", 0.0),
                            scaling.get("high", 0.0))
    amp = amplitude or amp
    for call, sense in ((P.pack3d_rotary, 1.0), (P.pack3d_rotary_backward, -1.0)):
        got = call(p, pos, q, k)
        for x, y in ((q, got[0] if kv else got),) + (((k, got[1]),) if kv else ()):
            val, bound = S.rotated(x, pos, th, amp, layout, sense)
            S.within(y, val, bound, f"{call.__name__} d{d} r{r} {layout} {dtype} {scaling}")
            assert torch.equal(y[..., r:], x[..., r:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s.get("scaling", "none"))
def test_rotary_scalings(scaling, layout, dtype):
    rotary_check(37, 4, 2, 128, 128, layout, dtype, **scaling)
    rotary_check(5, 3, 1, 96, 64, layout, dtype, base=500000.0, seed=1, **scaling)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,r", [(8, 2), (8, 8), (16, 6), (24, 24), (48, 12), (72, 10), (96, 96),
                                 (96, 32), (128, 4), (256, 256), (248, 130)])
def test_rotary_widths(d, r, layout, dtype):
    rotary_check(19, 2, 1, d, r, layout, dtype)


@pytest.mark.parametrize("n,heads,kv", [(1, 1, 0), (1, 32, 8), (8, 16, 4), (1000, 3, 3), (257, 64, 1),
                                        (3000, 16, 16), (20, 300, 100)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_shapes(n, heads, kv, layout):
    rotary_check(n, heads, kv, 128, 128, layout, "bf16", seed=n)


def test_rotary_largest_positions():
    rotary_check(64, 2, 1, 64, 64, "half", "fp32", far=2 ** 31 - 1)
    rotary_check(64, 2, 1, 64, 64, "half", "fp32", far=2 ** 31 - 1, base=0.25, amplitude=1.5)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n", [23, 6000])
def test_rotary_in_place_strides_and_skipped_rows(layout, n):
    H, K, d = 6, 2, 64
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(n, H + 2 * K, d, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 5000, (n,), generator=g).to(torch.int32).cuda()
    pos[::5] = -1
    p = P.make_rotary_params(d, 48, layout)
    q, k = qkv[:, :H], qkv[:, H:H + K]
    want = P.pack3d_rotary(p, pos, q.contiguous(), k.contiguous())
    before = qkv.clone()
    qo, ko = P.pack3d_rotary(p, pos, q, k, q, k)
    keep = pos >= 0
    assert qo.data_ptr() == q.data_ptr() and ko.data_ptr() == k.data_ptr()
    assert torch.equal(q[keep], want[0][keep]) and torch.equal(k[keep], want[1][keep])
    assert torch.equal(qkv[~keep], before[~keep]) and int((~keep).sum()) > 0
    assert torch.equal(qkv[:, H + K:], before[:, H + K:])
    # there and back: the transpose of a rotation is its inverse
    P.pack3d_rotary_backward(p, pos, q, k, q, k)
    err = (q.double() - before[:, :H].double()).abs()
    size = q.double().abs() + before[:, :H].double().abs() + 8
    assert (err <= 4 * 2.0 ** -8 * size).all()


def test_rotary_is_orthogonal_to_its_backward():
    """<R x, y> = <x, R^T y>: the backward is the gradient of a linear map."""
    n, H, d = 50, 3, 96
    g = torch.Generator().manual_seed(7)
    x, y = (torch.randn(n, H, d, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 10 ** 6, (n,), generator=g).to(torch.int32).cuda()
    p = P.make_rotary_params(d, 80, "interleaved", dtype="fp32", amplitude=1.25)
    a = (P.pack3d_rotary(p, pos, x).double() * y.double())
    b = (x.double() * P.pack3d_rotary_backward(p, pos, y).double())
    # values off by 8 half steps of 1.25 (|x1| + |x2|) each, summed over n H d
    room = 16 * 2.0 ** -24 * 1.25 * float((x.double().abs().sum() * y.double().abs().max()))
    assert abs(float(a.sum() - b.sum())) <= room


# ---- together -----------------------------------------------------------------------------


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotated_attention_layer(layout):
    """Index, rotation by its positions, attention and the way back, as a layer
    runs them, against the composed formulas: shifting every position of a
    sequence changes no logit, so positions that restart per sequence and
    positions along the pack give the same result."""
    lens, H, K, d = [300, 0, 77, 150], 4, 2, 96
    n = sum(lens)
    op = P.SeqAttention(P.make_seq_params(len(lens), n, H, K, d, True, "bf16"),
                        P.make_rotary_params(d, 64, layout))
    cu = torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda")
    op.build_index(cu)
    q, k, v, dout = S.make(lens, H, K, d, "bf16", 2)
    out, lse, rot = op.forward(q, k, v)
    dq, dk, dv = op.backward(rot, v, out, lse, dout)
    th, amp = S.frequencies(64, 10000.0)
    pos = op.index.positions
    for x, y in zip((q, k), rot):
        S.within(y, *S.rotated(x, pos, th, amp, layout), "rotated")
    ref = S.reference(lens, *rot, v, dout, True)
    S.within(out, *ref["out"], "out")
    S.within(lse, *ref["lse"], "lse")
    S.within(dv, *ref["dv"], "dv")
    for got, name in ((dq, "dq"), (dk, "dk")):
        val, _ = S.rotated(ref[name][0].bfloat16(), pos, th, amp, layout, -1.0)
        exact = torch.zeros_like(ref[name][0])
        # turn the 64-bit gradient back; its bound turns with the pairs' sizes, then
        # the rounding before the turn and the one after it
        i1, i2 = (slice(0, 32), slice(32, 64)) if layout == "half" else (slice(0, 64, 2),
                                                                       slice(1, 64, 2))
        y, e = ref[name][0], ref[name][1]
        ang = pos.double()[:, None, None] * th.cuda()
        exact = y.clone()
        exact[..., i1] = y[..., i1] * ang.cos() + y[..., i2] * ang.sin()
        exact[..., i2] = -y[..., i1] * ang.sin() + y[..., i2] * ang.cos()
        room = e.clone()
        room[..., i1] = room[..., i2] = e[..., i1] + e[..., i2]
        room = room + 2.0 ** -8 * exact.abs() * (1 + 2.0 ** -4) + 2.0 ** -20 * y.abs().amax()
        S.within(got, exact, room, name)
    # the same layer without restarting the positions
    along = torch.arange(n, dtype=torch.int32, device="cuda")
    q2, k2 = P.pack3d_rotary(op.rotary, along, q, k)
    out2, _ = P.pack3d_seq_forward(op.params, op.index, q2, k2, v)
    ref2 = S.reference(lens, q2, k2, v, dout, True)
    S.within(out2, *ref2["out"], "positions along the pack")


def test_volumes_in_one_pack_beside_the_local_global_operator():
    """A volume attended densely beside the same volume's local-global output
    with a window that covers it: the two operators agree (axial rotation
    applied by the local-global call; here by hand)."""
    import numpy as np
    from types import SimpleNamespace
    sh = SimpleNamespace(B=1, H=2, d=96, Z=3, Y=5, X=9, window=(5, 9, 17), block=(3, 5, 9),
                         rope_base=100.0, dtype="bf16")
    n = 3 * 5 * 9
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(1, n, 2, 96, generator=g).bfloat16().cuda() for _ in range(3))
    zyx = np.stack(np.meshgrid(range(3), range(5), range(9), indexing="ij"), -1).reshape(-1, 3)
    coords = torch.tensor(zyx, dtype=torch.int16)[None].cuda()
    op = P.Pack3D(sh)
    op.build_index(coords)
    want, wl = op.window_forward(q, k, v)
    # each axis' 32 channels are a head of their own for the rotary call
    qs, ks = q[0].clone(), k[0].clone()
    rp = P.make_rotary_params(32, 32, "half", base=100.0)
    for a in range(3):
        pos = coords[0, :, a].to(torch.int32).contiguous()
        for x in (qs, ks):
            part = x[:, :, 32 * a:32 * a + 32].contiguous()
            x[:, :, 32 * a:32 * a + 32] = P.pack3d_rotary(rp, pos, part)
    p, ix = built([n], 2, 2, 96, False, "bf16")
    out, lse = P.pack3d_seq_forward(p, ix, qs, ks, v[0])
    ref = S.reference([n], qs, ks, v[0], v[0], False)
    S.within(out, *ref["out"], "out")
    # the local-global call rotates in fp32 and rounds to bf16 as well; both are
    # within the operator's stated bound of the same value
    assert float((out.double() - want[0].double()).abs().max()) <= 2e-2
    assert float((lse.double() - wl[0].double()).abs().max()) <= 2e-2
