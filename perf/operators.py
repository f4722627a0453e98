"""What is measured of the packed-sequence operators: dense attention over packed sequences
(causal or not, shared key/value heads, forward and forward + backward) and rotary positions
of queries and keys (forward and backward).

``own = False`` computes them in elementary torch operations in 32 bits; ``own = True`` makes
the calls a user makes of ``local_global_attention_b200.pack3d``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# Heads and head dims 8 x 96 and 4 x 48 are the volume workloads' own; 16 query heads on 4 or 2
# key/value heads with head dims 64 and 128 are generic sequence-model shapes.


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _attention(kind, lens, heads, kv_heads, dim, causal=True, dtype="bf16", fused=False):
    return {"kind": kind, "lens": ",".join(str(x) for x in lens), "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": causal, "dtype": dtype, "fused": fused}


def _rotary(kind, tokens, heads, kv_heads, dim, rot, layout="half", dtype="bf16", scaling="none",
            factor=1.0, base=10000.0, far=0):
    return {"kind": kind, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "dtype": dtype, "scaling": scaling, "factor": factor,
            "base": base, "far": far}


def listed():
    return [
        # a handful of very short prompts, one of a single token, one empty: latency counts
        {"name": "prompts short", **_attention("forward", [17, 1, 60, 0, 33], 8, 8, 96)},
        # a serving batch: prompts of uneven lengths, key/value heads shared by four query heads,
        # q, k and v three slices of one projection's output
        {"name": "prompts ragged",
         **_attention("forward", [1311, 77, 2046, 512, 5, 903, 1024, 311, 129, 1650, 1, 724], 16, 4,
                      128, fused=True)},
        # the 16 x 32 x 32 volume as one sequence, every token on every token (not causal)
        {"name": "volume 16k dense", **_attention("forward", [16384], 8, 8, 96, causal=False)},
        # one long prompt
        {"name": "prompt 32k", **_attention("forward", [32768], 16, 2, 128)},
        # many small volumes in one pack, not causal, narrow heads
        {"name": "volumes small",
         **_attention("forward", [512, 1000, 216, 768, 343, 1331, 512, 64, 729, 1000], 8, 8, 64,
                      causal=False)},
        # a fine-tuning step's smallest layer
        {"name": "train short", **_attention("train", [129, 64, 1, 200], 8, 8, 96)},
        # a training batch of packed documents
        {"name": "train ragged",
         **_attention("train", [700, 2048, 333, 64, 1500, 9, 1201, 2337], 8, 8, 96, fused=True)},
        # the largest training step: two sequences of 8192, shared key/value heads
        {"name": "train 2 x 8k", **_attention("train", [8192, 8192], 16, 4, 128)},
        # the 32-bit mode at the tiny workload's heads
        {"name": "train fp32", **_attention("train", [512, 1000, 77, 411], 4, 4, 48, dtype="fp32")},
        # single tokens of eight running sequences at far positions, base-scaled
        {"name": "rotary tokens",
         **_rotary("rotary", 8, 16, 4, 128, 128, scaling="base", factor=4.0, far=1000000)},
        # the 65,536-token volume's queries and keys, neighbouring channels paired
        {"name": "rotary 64k",
         **_rotary("rotary", 65536, 8, 8, 96, 96, layout="interleaved", base=100.0)},
        # gradients of a training batch, half of each head rotated, long-context bands
        {"name": "rotary backward",
         **_rotary("rotary_backward", 16411, 16, 4, 128, 64, scaling="bands", factor=8.0,
                   base=500000.0, far=100000)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "train", "train", "rotary", "rotary_backward"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    while kv * group > 16:
        group = rng.choice([1, 2, 3, 4])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind in ("rotary", "rotary_backward"):
        dim = rng.choice([24, 48, 64, 80, 96, 128])
        rot = rng.choice([dim, dim, dim // 2, 8 * rng.randint(1, dim // 8)])
        scaling = rng.choice(["none", "linear", "base", "bands", "ramp"])
        return _rotary(kind, _log_int(rng, 1, 32768), kv * group, kv, dim, rot - rot % 2,
                       layout=rng.choice(["half", "interleaved"]), dtype=dtype, scaling=scaling,
                       factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                       base=rng.choice([100.0, 10000.0, 500000.0]),
                       far=rng.choice([0, 5000, 1000000]))
    dim = rng.choice([16, 48, 64, 72, 96, 96, 104, 128, 128])
    causal = rng.random() < 0.7
    fused = rng.random() < 0.4
    total = _log_int(rng, 1, 4096 if dtype == "fp32" else 16384)
    n = min(rng.choice([1, 2, 3, 5, 8, 13, 32]), total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if kind == "train" and max(lens) < 2:
        # a token alone in its sequence has no gradient of q and k: one pair of tokens at least
        lens = [max(total, 2)]
    return _attention(kind, lens, kv * group, kv, dim, causal, dtype, fused)


# ---- inputs ---------------------------------------------------------------------------


def _frequencies(case):
    """The angle per position of each rotated pair, as Python floats."""
    r, base, s, f = case["rot"], case["base"], case["scaling"], case["factor"]
    if s == "base":  # the slowest pair turns `factor` times slower, the fastest as before
        base = base * f ** (r / (r - 2)) if r > 2 else base
    th = [base ** (-2.0 * j / r) for j in range(r // 2)]
    if s == "linear":
        th = [t / f for t in th]
    if s == "bands":  # by the turns a pair makes over the original length
        turns = [LENGTH * t / (2 * math.pi) for t in th]
        mix = [min(1.0, max(0.0, (n - BANDS[0]) / (BANDS[1] - BANDS[0]))) for n in turns]
        th = [m * t + (1 - m) * t / f for m, t in zip(mix, th)]
    if s == "ramp":  # by the pair's number, between the pairs of two turn counts
        at = [r * math.log(LENGTH / (2 * math.pi * n)) / (2 * math.log(base)) for n in RAMP]
        hi, lo = min(math.ceil(at[0]), r - 1), max(math.floor(at[1]), 0)
        mix = [min(1.0, max(0.0, (j - lo) / max(hi - lo, 0.001))) for j in range(r // 2)]
        th = [(1 - m) * t + m * t / f for m, t in zip(mix, th)]
    return th


LENGTH, BANDS, RAMP = 8192, (1.0, 4.0), (1.0, 32.0)  # original length; turns, slow and fast


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, K, d, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    if case["kind"].startswith("rotary"):
        n = case["tokens"]
        st["q"], st["k"] = normal(n, H, d).to(dt), normal(n, K, d).to(dt)
        if case["far"]:  # running sequences, each at a position of its own
            st["positions"] = torch.randint(0, case["far"] + 1, (n,), generator=g, device="cuda",
                                            dtype=torch.int32)
        else:
            st["positions"] = torch.arange(n, device="cuda", dtype=torch.int32)
        st["theta"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        if own:
            from local_global_attention_b200 import pack3d as P
            band = {"bands": BANDS, "ramp": RAMP}.get(case["scaling"], (0.0, 0.0))
            st["params"] = P.make_rotary_params(
                d, rot_dim=case["rot"], layout=case["layout"], base=case["base"],
                dtype=case["dtype"], scaling=case["scaling"], factor=case["factor"],
                original_length=LENGTH, low=band[0], high=band[1])
        return st
    lens = _lens(case)
    n = sum(lens)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["lens"], st["starts"] = lens, cu[:-1]
    # peaked softmax: keys share a direction per head, logits of standard deviation about 2
    qkv = 1.4 * normal(n, H + 2 * K, d) + 0.5 * normal(1, H + 2 * K, d)
    qkv[:, H + K:] = normal(n, K, d)
    qkv = qkv.to(dt)
    parts = (qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:])
    st["q"], st["k"], st["v"] = parts if case["fused"] else [x.contiguous() for x in parts]
    if case["kind"] == "train":
        st["dout"] = normal(n, H, d).to(dt)
    if own:
        from local_global_attention_b200 import pack3d as P
        st["params"] = P.make_seq_params(n_seqs=len(lens), n_tokens=n, heads=H, kv_heads=K,
                                         head_dim=d, causal=case["causal"], dtype=case["dtype"])
        st["index"] = P.pack3d_seq_build_index(
            st["params"], torch.tensor(cu, dtype=torch.int32, device="cuda"))
    return st


# ---- one pass ---------------------------------------------------------------------------


def run(st):
    case = st["case"]
    kind = case["kind"]
    if kind.startswith("rotary"):
        if own:
            from local_global_attention_b200 import pack3d as P
            call = P.pack3d_rotary if kind == "rotary" else P.pack3d_rotary_backward
            return call(st["params"], st["positions"], st["q"], st["k"])
        return _plain_rotary(case, st["positions"], st["theta"], st["q"], st["k"],
                             -1.0 if kind == "rotary_backward" else 1.0)
    if own:
        from local_global_attention_b200 import pack3d as P
        p, ix = st["params"], st["index"]
        out, lse = P.pack3d_seq_forward(p, ix, st["q"], st["k"], st["v"])
        if kind == "forward":
            return out, lse
        return (out, lse, *P.pack3d_seq_backward(p, ix, st["q"], st["k"], st["v"], out, lse,
                                                 st["dout"]))
    return _plain_attention(st)


def _plain_rotary(case, positions, theta, q, k, sense):
    angle = positions.double()[:, None] * theta
    a = _amplitude(case)
    cos = (a * angle.cos()).float()[:, None]
    sin = (sense * a * angle.sin()).float()[:, None]
    r = case["rot"]

    def turn(x):
        y = x.float()
        out = y.clone()
        if case["layout"] == "half":
            one, two = slice(0, r // 2), slice(r // 2, r)
        else:
            one, two = slice(0, r, 2), slice(1, r, 2)
        out[..., one] = y[..., one] * cos - y[..., two] * sin
        out[..., two] = y[..., one] * sin + y[..., two] * cos
        return out.to(x.dtype)

    return turn(q), turn(k)


def _plain_attention(st):
    """Sequence by sequence, and the key/value heads in as many groups as the logits of one
    fit into 2^32 values."""
    case, q, k, v = st["case"], st["q"], st["k"], st["v"]
    H, K, d = case["heads"], case["kv_heads"], case["dim"]
    G, scale, train = H // K, case["dim"] ** -0.5, case["kind"] == "train"
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(H, q.shape[0], dtype=torch.float32, device=q.device)
    grads = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v)]
    for start, n in zip(st["starts"], st["lens"]):
        if n == 0:
            continue
        rows = slice(start, start + n)
        step = max(1, min(K, 2 ** 32 // (G * n * n)))
        for k0 in range(0, K, step):
            ks = slice(k0, min(K, k0 + step))
            hs = slice(k0 * G, min(K, k0 + step) * G)
            m = ks.stop - ks.start
            qs = q[rows, hs].float().permute(1, 0, 2).reshape(m, G * n, d)
            kt, vt = k[rows, ks].float().permute(1, 0, 2), v[rows, ks].float().permute(1, 0, 2)
            s = torch.matmul(qs, kt.transpose(1, 2)).mul_(scale).view(m, G, n, n)
            if case["causal"]:
                at = torch.arange(n, device=q.device)
                s.masked_fill_(at[None, :] > at[:, None], -math.inf)
            top = s.amax(-1, keepdim=True)
            s.sub_(top).exp_()
            total = s.sum(-1, keepdim=True)
            lse[hs, rows] = (total.log() + top).view(m * G, n)
            p = s.div_(total).view(m, G * n, n)
            o = torch.matmul(p, vt)
            out[rows, hs] = o.view(m * G, n, d).permute(1, 0, 2).to(q.dtype)
            if train:
                do = st["dout"][rows, hs].float().permute(1, 0, 2).reshape(m, G * n, d)
                dv = torch.matmul(p.transpose(1, 2), do)
                ds = torch.matmul(do, vt.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True))
                ds.mul_(p).mul_(scale)
                dq = torch.matmul(ds, kt)
                dk = torch.matmul(ds.transpose(1, 2), qs)
                grads[0][rows, hs] = dq.view(m * G, n, d).permute(1, 0, 2).to(q.dtype)
                grads[1][rows, ks] = dk.permute(1, 0, 2).to(q.dtype)
                grads[2][rows, ks] = dv.permute(1, 0, 2).to(q.dtype)
    return (out, lse, *grads) if train else (out, lse)


# ---- what a pass cannot do without --------------------------------------------------------


def work(case):
    H, K, d = case["heads"], case["kv_heads"], case["dim"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["kind"].startswith("rotary"):
        n, r = case["tokens"], case["rot"]
        return {"bytes": 2 * n * (H + K) * d * size + 4 * n, "flops": 3 * n * (H + K) * r}
    lens = _lens(case)
    n = sum(lens)
    pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in lens)
    forward = n * (2 * H + 2 * K) * d * size + 4 * n * H
    if case["kind"] == "forward":
        return {"bytes": forward, "flops": 4 * H * d * pairs}
    # q, k, v, dout read, out, lse and three gradients written; two products forward, five back
    return {"bytes": forward + n * (2 * H + 2 * K) * d * size, "flops": 14 * H * d * pairs}


# ---- the definition in 64 bits ------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    H, K, d = case["heads"], case["kv_heads"], case["dim"]
    if case["kind"].startswith("rotary"):
        # pairs as complex numbers, turned by exp(i angle)
        th = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        angle = torch.outer(st["positions"].double(), th)
        turn = torch.polar(torch.full_like(angle, _amplitude(case)), angle)
        if case["kind"] == "rotary_backward":
            turn = turn.conj()
        r, res = case["rot"], []
        for x in (st["q"], st["k"]):
            x = x.double()
            y = x[..., :r]
            if case["layout"] == "half":
                y = y.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            else:
                y = y.unflatten(-1, (r // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn[:, None])
            z = z.transpose(-1, -2) if case["layout"] == "half" else z
            res.append(torch.cat([z.flatten(-2), x[..., r:]], -1))
        return tuple(res)
    train, n_all = case["kind"] == "train", sum(_lens(case))
    out = torch.zeros(n_all, H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(H, n_all, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(out), *(torch.zeros(n_all, K, d, dtype=torch.float64,
                                                      device="cuda") for _ in range(2))
    at = 0
    for n in _lens(case):
        for h in range(H):
            kv = h * K // H
            q, k, v = (st[x][at:at + n, i].double() for x, i in (("q", h), ("k", kv), ("v", kv)))
            for r0 in range(0, n, 8192):  # query rows at a time
                r1 = min(n, r0 + 8192)
                s = q[r0:r1] @ k.T / math.sqrt(d)
                if case["causal"]:
                    s = s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(r0 + 1), -math.inf)
                lse[h, at + r0:at + r1] = z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                out[at + r0:at + r1, h] = p @ v
                if train:
                    g = st["dout"][at + r0:at + r1, h].double()
                    gp = g @ v.T
                    gs = p * (gp - (p * gp).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[at + r0:at + r1, h] = gs @ k
                    dk[at:at + n, kv] += gs.T @ q[r0:r1]
                    dv[at:at + n, kv] += p.T @ g
        at += n
    return (out, lse, dq, dk, dv) if train else (out, lse)
