"""Calls of the packed-sequence operators that a user may make beside the plain ones:
padded packs, several packs in flight, an index that holds an error, logits that move
the running maximum."""
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


# ---- rows behind the last sequence ---------------------------------------------------------


def dirty(shapes):
    """Leave NaN in memory that the next tensors of these shapes and types get."""
    kept = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    del kept


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,tail", [([100, 0, 190], 37), ([0], 5), ([128], 1), ([256, 256], 256),
                                       ([1] * 40, 900), ([700, 3], 130), ([5], 1111)], ids=str)
@pytest.mark.parametrize("dim,causal,layout", [(48, True, "half"), (96, False, "interleaved"),
                                               (128, True, "interleaved"), (72, False, "half")])
def test_new_outputs_are_zero_behind_the_last_sequence(lens, tail, dim, causal, layout, dtype):
    """Memory that held NaN before: a padded pack's weight gradients x^T dq would hold
    them too."""
    H, K, n = 4, 2, sum(lens)
    op = P.SeqAttention(P.make_seq_params(len(lens), n + tail, H, K, dim, causal, dtype),
                        P.make_rotary_params(dim, dim // 8 * 4, layout, dtype=dtype))
    op.build_index(torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda"))
    q, k, v, dout = S.make(lens, H, K, dim, dtype, 3, False, tail)
    for x in (q, k, v, dout):
        x[n:] = float("nan")
    shapes = [(q.shape, q.dtype), (k.shape, k.dtype), ((H, n + tail), torch.float32)]
    dirty(shapes)
    out, lse, rot = op.forward(q, k, v)
    dirty(shapes)
    grads = op.backward(rot, v, out, lse, dout)
    for x in (out, *rot, *grads):
        assert not x[n:].any() and torch.isfinite(x).all()
    assert not lse[:, n:].any() and torch.isfinite(lse).all()
    # the same rows as without the padding
    p, ix = built(lens, H, K, dim, causal, dtype)
    if n:
        part = [x[:n].contiguous() for x in (*rot, v, dout)]
        o, z = P.pack3d_seq_forward(p, ix, *part[:3])
        assert torch.equal(o, out[:n]) and torch.equal(z, lse[:, :n])
        g = P.pack3d_seq_backward(p, ix, *part[:3], o, z, part[3])
        assert torch.equal(g[2], grads[2][:n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_given_and_new_outputs_of_one_call(dtype):
    """Given outputs keep their rows behind the last sequence, new ones beside them are
    zero there."""
    lens, tail, H, K, d = [130, 61], 70, 2, 1, 64
    n, N = sum(lens), sum(lens) + tail
    p, ix = built(lens, H, K, d, True, dtype, tail)
    q, k, v, dout = S.make(lens, H, K, d, dtype, 4, False, tail)
    want = P.pack3d_seq_forward(p, ix, q, k, v)
    wg = P.pack3d_seq_backward(p, ix, q, k, v, *want, dout)
    shapes = [(q.shape, q.dtype), (k.shape, k.dtype), ((H, N), torch.float32)]

    def same(got, kept, want, rows):
        a, b = (got, want) if rows == 0 else (got.T, want.T)
        assert torch.equal(a[:n], b[:n])
        assert (a[n:] == (7 if kept else 0)).all()

    for given in ((True, False), (False, True), (True, True)):
        o = torch.full_like(q, 7) if given[0] else None
        z = torch.full((H, N), 7.0, device="cuda") if given[1] else None
        dirty(shapes)
        got = P.pack3d_seq_forward(p, ix, q, k, v, o, z)
        same(got[0], given[0], want[0], 0)
        same(got[1], given[1], want[1], 1)
    for one in range(3):
        outs = [torch.full_like(x, 7) if i == one else None for i, x in enumerate((q, k, v))]
        dirty(shapes)
        got = P.pack3d_seq_backward(p, ix, q, k, v, *want, dout, *outs)
        for i in range(3):
            same(got[i], i == one, wg[i], 0)
    pos = ix.positions
    r = P.make_rotary_params(d, 48, dtype=dtype)
    wq, wk = P.pack3d_rotary(r, pos, q, k)
    dirty(shapes)
    qo, ko = P.pack3d_rotary(r, pos, q, k, q_out=torch.full_like(q, 7))
    same(qo, True, wq, 0)
    same(ko, False, wk, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zeroed_rows_in_strided_outputs_and_in_place(dtype):
    """The C calls with the flag: rows of no sequence of given slices become zero, what
    stands between the slices stays."""
    lens, tail, H, K, d = [150, 9], 41, 3, 1, 40
    n, N = sum(lens), sum(lens) + tail
    p, ix = built(lens, H, K, d, False, dtype, tail)
    q, k, v, dout = S.make(lens, H, K, d, dtype, 6, True, tail)
    want = P.pack3d_seq_forward(p, ix, q, k, v)
    wg = P.pack3d_seq_backward(p, ix, q, k, v, *want, dout)
    p.dtype |= P.ZERO_UNUSED_ROWS
    wide = torch.full((N, H + 2 * K + 1, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((H, N), 7.0, device="cuda")
    P.pack3d_seq_forward(p, ix, q, k, v, wide[:, 1:1 + H], lse)
    assert torch.equal(wide[:, 1:1 + H], want[0]) and torch.equal(lse, want[1])
    assert (wide[:, 0] == 7).all() and (wide[:, 1 + H:] == 7).all()
    wide[:] = 7
    P.pack3d_seq_backward(p, ix, q, k, v, *want, dout, wide[:, 1:1 + H], wide[:, 1 + H:1 + H + K],
                          wide[:, 1 + H + K:])
    assert torch.equal(wide[:, 1:], torch.cat(wg, 1)) and (wide[:, 0] == 7).all()
    # rotary in place, part of the head
    r = P.make_rotary_params(d, 24, dtype=dtype)
    wq, wk = P.pack3d_rotary(r, ix.positions, q, k)
    r.dtype |= P.ZERO_UNUSED_ROWS
    q2, k2 = q.clone(), k.clone()
    P.pack3d_rotary(r, ix.positions, q2, k2, q2, k2)
    assert torch.equal(q2, wq) and torch.equal(k2, wk) and not q2[n:].any()


def test_rows_of_an_index_that_was_never_built():
    """It holds no sequence: every row of a new output is one of no sequence."""
    p = P.make_seq_params(2, 300, 2, 1, 64, True, "bf16")
    ix = P.SeqIndex(p)
    q, k, v, dout = S.make([300], 2, 1, 64, "bf16")
    dirty([(q.shape, q.dtype), (k.shape, k.dtype), ((2, 300), torch.float32)])
    out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
    assert not out.any() and not lse.any()
    dirty([(q.shape, q.dtype), (k.shape, k.dtype)])
    assert not any(x.any() for x in P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout))


# ---- several packs in flight ---------------------------------------------------------------


def layer(lens, dtype="bf16"):
    H, K, d = 4, 2, 64
    op = P.SeqAttention(P.make_seq_params(len(lens), sum(lens), H, K, d, True, dtype),
                        P.make_rotary_params(d, dtype=dtype))
    return op, [torch.tensor(S.prefix(x), dtype=torch.int32, device="cuda")
                for x in (lens, lens[::-1])]


def test_backward_after_another_pack_was_built():
    """The wrapper's index holds the lengths of the last pack: the backward of the pack
    before it is refused."""
    lens = [100, 300, 17]
    op, (a, b) = layer(lens)
    q, k, v, dout = S.make(lens, 4, 2, 64, "bf16", 1)
    op.build_index(a)
    out, lse, rot = op.forward(q, k, v)
    want = op.backward(rot, v, out, lse, dout)
    op.build_index(b)
    with pytest.raises(ValueError):
        op.backward(rot, v, out, lse, dout)
    with pytest.raises(ValueError):
        op.backward(rot, v, out, lse, dout, index=P.pack3d_seq_build_index(op.params, a))
    out, lse, rot = op.forward(q, k, v)  # the pack that the index holds
    op.backward(rot, v, out, lse, dout)
    # a plain pair goes with the given index
    op.build_index(a)
    out, lse, rot = op.forward(q, k, v)
    for index in (None, P.pack3d_seq_build_index(op.params, a)):
        got = op.backward(tuple(rot), v, out, lse, dout, index=index)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_packs_in_flight_with_their_own_indexes():
    """Two micro-batches: both forwards, then both backwards."""
    lens = [100, 300, 17]
    op, cus = layer(lens)
    sets = [S.make(lens, 4, 2, 64, "bf16", s) for s in (1, 2)]
    want = []
    for cu, (q, k, v, dout) in zip(cus, sets):
        op.build_index(cu)
        out, lse, rot = op.forward(q, k, v)
        want.append((out, lse, *op.backward(rot, v, out, lse, dout)))
    idx = [P.pack3d_seq_build_index(op.params, cu) for cu in cus]
    runs = [op.forward(*x[:3], index=ix) for x, ix in zip(sets, idx)]
    for (out, lse, rot), x, w in zip(runs, sets, want):
        got = (out, lse, *op.backward(rot, x[2], out, lse, x[3]))
        assert all(torch.equal(m, n) for m, n in zip(got, w))


def test_wrapper_in_a_graph_follows_the_lengths():
    """Index, forward and backward of one captured step, replayed with other lengths
    written into its prefix sums; and an index built anew outside a graph that holds the
    forward alone."""
    lens = [100, 300, 17]
    op, (a, b) = layer(lens)
    q, k, v, dout = S.make(lens, 4, 2, 64, "bf16", 1)

    def step():
        out, lse, rot = op.forward(q, k, v)
        return (out, lse, *op.backward(rot, v, out, lse, dout))

    want = []
    for cu in (a, b):
        op.build_index(cu)
        want.append(step())
    cu = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.build_index(cu, check=False)
        res = step()
    for x, w in ((b, want[1]), (a, want[0])):
        cu.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(res, w))
    alone = torch.cuda.CUDAGraph()
    with torch.cuda.graph(alone):
        res = step()
    for x, w in ((b, want[1]), (a, want[0])):
        op.build_index(x)
        alone.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(res, w))


# ---- an index that holds an error ----------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_index_with_the_timeout_bit(dim, dtype):
    """The bit that a kernel sets when a bounded wait gives up, written here by the host:
    later calls write nothing, the check reports it, building anew clears it."""
    lens, H, K = [300, 129], 4, 2
    p, ix = built(lens, H, K, dim, True, dtype, 11)
    q, k, v, dout = S.make(lens, H, K, dim, dtype, 2, False, 11)
    want = P.pack3d_seq_forward(p, ix, q, k, v)
    off = ix.struct.err - ix.buffer.data_ptr()
    err = ix.buffer[off:off + 8].view(torch.int32)
    assert err.tolist() == [0, sum(lens)]
    err[0] = 4
    assert P.pack3d_seq_index_check(ix) == P.ERR_TIMEOUT
    kept = [torch.full_like(x, 7) for x in (q, q, k, v)]
    lse = torch.full_like(want[1], 7)
    p.dtype |= P.ZERO_UNUSED_ROWS
    P.pack3d_seq_forward(p, ix, q, k, v, kept[0], lse)
    P.pack3d_seq_backward(p, ix, q, k, v, *want, dout, *kept[1:])
    assert all((x == 7).all() for x in (*kept, lse))
    assert P.pack3d_seq_index_check(ix) == P.ERR_TIMEOUT
    cu = torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda")
    P.pack3d_seq_build_index(p, cu, ix)
    assert P.pack3d_seq_index_check(ix) == P.OK
    got = P.pack3d_seq_forward(p, ix, q, k, v)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- rotary bases below 1 ------------------------------------------------------------------


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("base,r", [(0.010009765625, 96), (0.01953125, 64),
                                    (0.5, 128), (0.90625, 8)])
def test_rotary_fast_pairs_at_far_positions(base, r, layout):
    """Pairs of up to 14.4 turns per position (bases that are floats).  Beside the roundings that rotated()
    counts, the angle of position 2^31: 2^-61 relative of 14.5 x 2^31 turns is 2^-26 of
    a turn, 0.9e-7; the 64-bit mantissas of the oracle are off by as much (a power, a
    product and the reduction): 4 half steps 2^-24 of a (|x1| + |x2|) cover both."""
    d = 128
    g = torch.Generator().manual_seed(r)
    q = torch.randn(64, 2, d, generator=g).cuda()
    pos = torch.randint(0, 2 ** 31 - 1, (64,), generator=g).to(torch.int32).cuda()
    p = P.make_rotary_params(d, r, layout, base, "fp32")
    th, amp = S.frequencies(r, base)
    for call, sense in ((P.pack3d_rotary, 1.0), (P.pack3d_rotary_backward, -1.0)):
        val, bound = S.rotated(q, pos, th, amp, layout, sense)
        x = q.double()
        i1, i2 = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else \
            (slice(0, r, 2), slice(1, r, 2))
        more = 4 * 2.0 ** -24 * (x[..., i1].abs() + x[..., i2].abs())
        bound[..., i1] += more
        bound[..., i2] += more
        S.within(call(p, pos, q), val, bound, f"{call.__name__} base {base}")


# ---- non-finite values inside a causal sequence --------------------------------------------


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("dtype,tile,dim", [("bf16", 128, 64), ("bf16", 128, 96), ("bf16", 128, 128),
                                            ("fp32", 64, 48)])
def test_reach_of_a_non_finite_token(dtype, tile, dim, what, bad):
    """The formulas take q_t to out, lse and dq of t and dk and dv up to t; k_t and v_t to
    rows from t on and, by these, to every dk (k_t: and dv); dout_t to dq of t and dk and
    dv up to t.  Beyond that only what the header lists, in the token's own tile: all
    other values are the bits they are without it."""
    lens, H, K = [90, 500, 40], 4, 2
    p, ix = built(lens, H, K, dim, True, dtype)
    s0, n = 90, 500
    clean = S.make(lens, H, K, dim, dtype, 7)
    names = ("out", "lse", "dq", "dk", "dv")

    def run(q, k, v, dout):
        out, lse = P.pack3d_seq_forward(p, ix, q, k, v)
        return dict(zip(names, (out, lse.T, *P.pack3d_seq_backward(p, ix, q, k, v, out, lse, dout))))

    want = run(*clean)
    for t in (0, 30, 127, 128, 200, 383, 499):
        x = [y.clone() for y in clean]
        x[("q", "k", "v", "dout").index(what)][s0 + t] = bad
        got = run(*x)
        at, upto, since, all_, none = {t}, set(range(t + 1)), set(range(t, n)), set(range(n)), set()
        own = set(range(t // tile * tile, min(n, (t // tile + 1) * tile)))
        reach = {"q": dict(out=at, lse=at, dq=at, dk=upto | own, dv=upto),
                 "k": dict(out=since, lse=since, dq=since | own, dk=all_, dv=all_),
                 "v": dict(out=since | own, lse=none, dq=since | own, dk=all_, dv=none),
                 "dout": dict(out=none, lse=none, dq=at, dk=upto | own, dv=upto | own)}[what]
        for name in names:
            other = [s0 + i for i in range(n) if i not in reach[name]]
            rows = list(range(s0)) + other + list(range(s0 + n, sum(lens)))
            assert torch.equal(got[name][rows], want[name][rows]), (name, t)


# ---- padded packs in graphs and on given streams -------------------------------------------


def test_padded_pack_in_a_replayed_graph():
    """Index, forward and backward in one graph over tensors of fixed size: rows that a
    replay's sequences no longer hold are zero, not the replay before's."""
    H, K, d, N = 4, 2, 96, 640
    op = P.SeqAttention(P.make_seq_params(3, N, H, K, d), P.make_rotary_params(d))
    q, k, v, dout = S.make([N], H, K, d, "bf16", 3)
    cu = torch.tensor([0, 300, 500, 640], dtype=torch.int32, device="cuda")

    def step():
        out, lse, rot = op.forward(q, k, v)
        return (out, lse.T, *rot, *op.backward(rot, v, out, lse, dout))

    op.build_index(cu)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.build_index(cu, check=False)
        res = step()
    for ends in ([300, 500, 640], [100, 100, 130], [1, 2, 3], [0, 0, 0], [128, 256, 639]):
        cu.copy_(torch.tensor([0, *ends], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        assert P.pack3d_seq_index_check(op.index) == P.OK
        assert all(not x[ends[-1]:].any() for x in got)
        op.build_index(cu)
        assert all(torch.equal(x, y) for x, y in zip(got, step()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padded_packs_on_two_given_streams(dtype):
    """Two packs at once, each with its index, outputs allocated on the given streams."""
    H, K, d, lens, tail = 4, 2, 64, [200, 77], 301
    n = sum(lens)
    p, _ = built(lens, H, K, d, True, dtype, tail)
    cu = torch.tensor(S.prefix(lens), dtype=torch.int32, device="cuda")
    sets = [S.make(lens, H, K, d, dtype, s, False, tail) for s in (1, 2)]
    want = []
    for x in sets:
        ix = P.pack3d_seq_build_index(p, cu)
        out, lse = P.pack3d_seq_forward(p, ix, *x[:3])
        want.append((out, lse, *P.pack3d_seq_backward(p, ix, *x[:3], out, lse, x[3])))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    runs = []
    for _ in range(3):
        for x, s in zip(sets, streams):
            ix = P.pack3d_seq_build_index(p, cu, stream=s)
            out, lse = P.pack3d_seq_forward(p, ix, *x[:3], stream=s)
            runs.append((out, lse, *P.pack3d_seq_backward(p, ix, *x[:3], out, lse, x[3], stream=s)))
    torch.cuda.synchronize()
    for i, got in enumerate(runs):
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2]))
        assert not got[0][n:].any() and not got[2][n:].any()


def test_replayed_forward_and_eager_backward():
    """A captured forward, replayed after the index was built for other lengths, with the
    backward called outside the graph each time."""
    lens = [100, 300, 17]
    op, cus = layer(lens)
    q, k, v, dout = S.make(lens, 4, 2, 64, "bf16", 1)
    want = []
    for cu in cus:
        op.build_index(cu)
        out, lse, rot = op.forward(q, k, v)
        want.append((out, lse, *op.backward(rot, v, out, lse, dout)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, rot = op.forward(q, k, v)
    for cu, w in zip(cus, want):
        op.build_index(cu)
        graph.replay()
        got = (out, lse, *op.backward(rot, v, out, lse, dout))
        assert all(torch.equal(x, y) for x, y in zip(got, w))
