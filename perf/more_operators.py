"""Cases of the operators around the attention stage: the norms of queries and
keys, head by head, with the rotary positions in the same pass, and attention of
queries to keys and values of another length (an encoder's states), with grouped
heads, packed or padded sequences; forward and backward.

`run` computes a case in elementary torch operations in 32 bits (rotary angles
and sums over tokens in 64), or, with `own`, through the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _norm(name, tokens, q_heads, k_heads, head_dim, rot_dim, centred, adjacent, axes, dtype, back, far=0):
    return {"name": name, "op": "norm_bwd" if back else "norm", "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": head_dim, "rot_dim": rot_dim, "centred": centred, "adjacent": adjacent, "axes": axes, "dtype": dtype,
            "far": far}


def _cross(name, n, sq, sk, heads, kv_heads, head_dim, packed, ragged_q, ragged_k, empty, back):
    return {"name": name, "op": "cross_bwd" if back else "cross", "n": n, "sq": sq, "sk": sk, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "packed": packed, "ragged_q": ragged_q, "ragged_k": ragged_k,
            "empty": empty, "behind": 37 if packed else 0}


def listed():
    return [
        # one token of a small model: the shortest call there is
        _norm("norm 1 token", 1, 12, 12, 64, 64, False, False, 1, "bf16", False),
        # Q and K of one layer of the 96-layer GPT
        _norm("norm 4096", 4096, 64, 64, 128, 128, False, False, 1, "bf16", False),
        # grouped heads, LayerNorm with shifts, half of each head rotated in adjacent pairs, image and text axes, odd count
        _norm("norm 8191 grouped centred", 8191, 32, 8, 128, 64, True, True, 2, "bf16", False, 100000),
        # a small model's micro-batch of odd sequences, backward
        _norm("norm backward 4x509", 2036, 12, 12, 64, 64, True, False, 1, "bf16", True),
        # the backward pass of the 96-layer GPT's Q and K
        _norm("norm backward 4096", 4096, 64, 64, 128, 128, False, False, 1, "bf16", True),
        # one new token of each of 8 sequences against encoder states of different lengths: latency
        _cross("cross 8x1 to 1000", 8, 1, 1000, 12, 12, 64, False, False, True, False, False),
        # one new token of each of 32 sequences, grouped heads, long states: all of K and V is read
        _cross("cross 32x1 to 8192", 32, 1, 8192, 64, 8, 128, False, False, True, False, False),
        # micro-batches of odd sequences attending to short prompts
        _cross("cross 4x1037 to 333", 4, 1037, 333, 64, 64, 128, False, False, True, False, False),
        # long sequences against long states: the matrix rate counts
        _cross("cross 4096 to 8192", 1, 4096, 8192, 64, 64, 128, False, False, False, False, False),
        # a small model's backward pass, states of different lengths
        _cross("cross backward 4x509 to 201", 4, 509, 201, 12, 12, 64, False, True, True, False, True),
        # packed documents, each with its own states (one has none), grouped heads
        _cross("cross backward packed", 9, 700, 900, 64, 8, 128, True, True, True, True, True),
        # the backward pass of long sequences against long states
        _cross("cross backward 4096 to 8192", 1, 4096, 8192, 16, 16, 128, False, False, False, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "cross", "cross", "cross", "cross_bwd", "cross_bwd"])
    if op.startswith("norm"):
        d = rng.choice([64, 64, 80, 96, 128, 128, 256])
        kh = _log(rng, 1, 64)
        qh = min(64, kh * rng.choice([1, 1, 2, 4, 8]))
        most = 4096 * 128 * 128 // ((qh + kh) * d)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return {"op": op, "tokens": _log(rng, 1, min(32768, most) // (2 if dtype == "fp32" else 1)), "q_heads": qh,
                "k_heads": rng.choice([kh, kh, kh, 0]), "head_dim": d, "rot_dim": rng.choice([d, d, d // 2, d // 2 - 4, 0]),
                "centred": rng.random() < 0.4, "adjacent": rng.random() < 0.4, "axes": rng.choice([1, 1, 2, 3]),
                "dtype": dtype, "far": rng.choice([0, 0, 100000, 4000000])}
    d = rng.choice([64, 128])
    kvh = rng.choice([1, 2, 5, 8, 12, 16, 32])
    heads = kvh * rng.choice([1, 1, 2, 3, 4, 8])
    n = _log(rng, 1, 32)
    back = op == "cross_bwd"
    pairs = (4096 * 8192 * (16 if back else 64)) // (n * heads)
    sq = _log(rng, 1, min(4096, 4096 * 64 * 128 // (n * heads * d)))
    sk = _log(rng, 1, min(16384, pairs // sq, 32 * 8192 * 8 * 128 // (n * kvh * d)))
    packed = n > 1 and rng.random() < 0.4
    return {"op": op, "n": n, "sq": sq, "sk": sk, "heads": heads, "kv_heads": kvh, "head_dim": d, "packed": packed,
            "ragged_q": rng.random() < 0.5, "ragged_k": rng.random() < 0.7, "empty": n > 2 and rng.random() < 0.3,
            "behind": rng.randint(0, 200) if packed else 0}


# ------------------------------------------------------------------ inputs
def _sections(case):
    """Pairs of each axis: the first axis takes what is left over."""
    pairs, axes = case["rot_dim"] // 2, case["axes"]
    rest = [pairs // (axes + 1) if axes > 1 else pairs] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _lengths(case, which, seed):
    """Real queries or keys of each sequence: a function of the case, so that its work is; the seed orders them."""
    n, s = case["n"], case["s" + which]
    rng = random.Random(n * 7919 + s * 31 + ord(which))
    lens = [s] * n
    if case["ragged_" + which]:
        lens = [s] + [rng.randint((s + 2) // 3, s) for _ in range(n - 1)]
    if case["empty"] and which == "k":
        lens[-1] = 0
    random.Random(seed * 1000003 + ord(which)).shuffle(lens)
    return lens


def _layout(case, which, seed):
    """First row of each sequence's slot (and the end of the last), real rows of each, rows in all."""
    lens = _lengths(case, which, seed)
    if case["packed"]:
        offsets = [0]
        for x in lens:
            offsets.append(offsets[-1] + x)
        return offsets, lens, offsets[-1] + case["behind"]
    s = case["s" + which]
    return [s * i for i in range(case["n"] + 1)], lens, s * case["n"]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    if case["op"].startswith("norm"):
        T, H, d = case["tokens"], case["q_heads"] + case["k_heads"], case["head_dim"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # Q and K lie beside V in each row; heads differ in size and, by a little, in mean
        x = _randn(g, T, H + case["k_heads"], d)
        x = x * (0.3 + 3.0 * torch.rand(x.shape[1], 1, generator=g, device=DEV)) + 0.1 * _randn(g, x.shape[1], 1)
        st["x"] = x.reshape(T, -1).to(dtype)
        for name in ("q", "k"):
            st[name + "_gain"] = (1.0 + 0.2 * _randn(g, d)).to(torch.bfloat16)
            st[name + "_shift"] = (0.1 * _randn(g, d)).to(torch.bfloat16) if case["centred"] else None
        st["eps"] = 1e-5
        if case["rot_dim"]:
            rng = random.Random(seed)
            step = torch.arange(T, dtype=torch.int64)
            grid = [step + rng.randint(0, 1000) + case["far"]]
            grid += [(step // (7 ** k)) % (13 + 5 * k) + rng.randint(0, 50) for k in range(1, case["axes"])]
            st["positions"] = torch.stack(grid).to(torch.int32).to(DEV)
            st["inv_freq"] = torch.tensor([1e4 ** (-2.0 * p / case["rot_dim"]) for p in range(case["rot_dim"] // 2)],
                                          dtype=torch.float64).float().to(DEV)
            st["axis"] = torch.tensor([x for x, n in enumerate(_sections(case)) for _ in range(n)], device=DEV)
        if case["op"] == "norm_bwd":
            st["dout"] = _randn(g, T, H * d).to(dtype)
        if own:
            from megatron_transformer_layer_gb300 import _lib as L
            st["out"] = torch.empty(T, H * d, dtype=dtype, device=DEV)
            st["norm"] = L.make_qk_norm(st["q_gain"], st["k_gain"], st["q_shift"], st["k_shift"], eps=st["eps"],
                                        centred=case["centred"])
            st["spec"] = L.make_rotary_spec(case["rot_dim"], _sections(case), interleaved_pairs=case["adjacent"]) \
                if case["rot_dim"] else None
            if case["op"] == "norm_bwd":
                names = [t + part for part in (("_gain", "_shift") if case["centred"] else ("_gain",))
                         for t in (("q", "k") if case["k_heads"] else ("q",))]
                st["grads"] = torch.empty(len(names), d, device=DEV)
                st["grads_c"] = L.make_qk_norm_grads(**dict(zip(names, st["grads"])))
                st["scratch"] = torch.empty(L.mc_qk_norm_scratch_floats(T, case["q_heads"], case["k_heads"], d), device=DEV)
        return st
    H, KV, d = case["heads"], case["kv_heads"], case["head_dim"]
    q_off, q_len, q_rows = _layout(case, "q", seed)
    k_off, k_len, k_rows = _layout(case, "k", seed)
    st["q"] = (1.5 * _randn(g, q_rows, H * d)).to(torch.bfloat16)
    st["kv"] = _randn(g, k_rows, 2 * KV * d).to(torch.bfloat16)  # K | V, as a projection of the states leaves them
    st["layout"] = [(q_off[i], q_len[i], k_off[i], k_len[i]) for i in range(case["n"])]
    back = case["op"] == "cross_bwd"
    if back:
        st["dout"] = _randn(g, q_rows, H * d).to(torch.bfloat16)
        st["o"], st["lse"] = _plain_cross(st)
    if own:
        from megatron_transformer_layer_gb300 import _lib as L
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        if case["packed"]:
            rows = {"q_offsets": i32(q_off), "kv_offsets": i32(k_off), "max_q": max(q_len), "max_kv": max(k_len)}
        else:
            rows = {"q_lens": i32(q_len) if case["ragged_q"] else None, "kv_lens": i32(k_len)}
        st["cross"] = L.make_cross_attention(case["n"], q_rows, k_rows, H, KV, d, ld_kv=2 * KV * d, **rows)
        # (rows behind the last sequence are not written)
        if not back:
            st["o"] = torch.zeros(q_rows, H * d, dtype=torch.bfloat16, device=DEV)
            st["lse"] = torch.zeros(H, q_rows, device=DEV)
        else:
            st["dq"], st["dkv"] = torch.zeros_like(st["q"]), torch.zeros_like(st["kv"])
            st["delta"] = torch.empty(H, q_rows, device=DEV)
            st["ws_bytes"] = L.mc_attention_backward_cross_ws_bytes(st["cross"])
            st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ the plain forms
def _turn(x, st, inverse):
    """The rotation of x [T, H, d] (32 bits), by the opposite angle if `inverse`."""
    c = st["case"]
    r = c["rot_dim"]
    if not r:
        return x
    ang = st["positions"][st["axis"]].double().t() * st["inv_freq"].double()
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if inverse:
        sin = -sin
    rot, rest = x[:, :, :r], x[:, :, r:]
    if c["adjacent"]:
        u, v = rot[:, :, 0::2], rot[:, :, 1::2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(2)
    else:
        u, v = rot[:, :, : r // 2], rot[:, :, r // 2:]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _per_head(st, part):
    """A gain or shift for every head [H, d], 32 bits."""
    c = st["case"]
    return torch.cat([st["q" + part].float().expand(c["q_heads"], -1), st["k" + part].float().expand(c["k_heads"], -1)])


def _normed(st):
    c = st["case"]
    T, H, d = c["tokens"], c["q_heads"] + c["k_heads"], c["head_dim"]
    x = st["x"][:, : H * d].view(T, H, d).float()
    if c["centred"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
    return x * r, r


def _plain_norm(st):
    c = st["case"]
    n, _ = _normed(st)
    y = n * _per_head(st, "_gain")
    if c["centred"]:
        y = y + _per_head(st, "_shift")
    return _turn(y, st, False).flatten(1).to(st["x"].dtype)


def _plain_norm_backward(st):
    c = st["case"]
    n, r = _normed(st)
    t = _turn(st["dout"].view(n.shape).float(), st, True)
    u = t * _per_head(st, "_gain")
    dx = u - n * (u * n).mean(-1, keepdim=True)
    if c["centred"]:
        dx = dx - u.mean(-1, keepdim=True)
    dx = (dx * r).flatten(1).to(st["x"].dtype)
    grads = []
    for w in [t * n] + ([t] if c["centred"] else []):
        s = w.sum(0, dtype=torch.float64)
        grads.append(s[: c["q_heads"]].sum(0))
        if c["k_heads"]:
            grads.append(s[c["q_heads"]:].sum(0))
    return [dx, torch.stack(grads).float()]


def _grouped(x, KV, d):
    """[rows, H d] as [KV, G rows, d], 32 bits: the query heads of a key head one after another."""
    rows = x.shape[0]
    return x.float().view(rows, KV, -1, d).permute(1, 2, 0, 3).reshape(KV, -1, d)


def _flat(x, rows, dtype=torch.bfloat16):
    """The way back: [KV, G rows, d] as [rows, H d]."""
    KV, _, d = x.shape
    return x.view(KV, -1, rows, d).permute(2, 0, 1, 3).reshape(rows, -1).to(dtype)


def _weights(q, k, scale):
    z = (q @ k.transpose(1, 2)) * scale
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    s = p.sum(-1, keepdim=True)
    return p / s, (m + torch.log(s)).squeeze(-1)


def _plain_cross(st):
    c = st["case"]
    KV, d = c["kv_heads"], c["head_dim"]
    o = torch.zeros_like(st["q"])
    lse = torch.zeros(c["heads"], st["q"].shape[0], device=DEV)
    for i, (q0, nq, k0, nk) in enumerate(st["layout"]):
        if not c["packed"]:
            lse[:, q0: q0 + c["sq"]] = -math.inf
        if nq and not nk:
            lse[:, q0: q0 + nq] = -math.inf
        if not nq or not nk:
            continue
        k, v = st["kv"][k0: k0 + nk].chunk(2, dim=1)
        p, l = _weights(_grouped(st["q"][q0: q0 + nq], KV, d), _grouped(k, KV, d), 1.0 / math.sqrt(d))
        o[q0: q0 + nq] = _flat(p @ _grouped(v, KV, d), nq)
        lse[:, q0: q0 + nq] = l.reshape(c["heads"], nq)
    return o, lse


def _plain_cross_backward(st):
    c = st["case"]
    KV, d = c["kv_heads"], c["head_dim"]
    scale = 1.0 / math.sqrt(d)
    dq, dkv = torch.zeros_like(st["q"]), torch.zeros_like(st["kv"])
    for q0, nq, k0, nk in st["layout"]:
        if not nq or not nk:
            continue
        k, v = (_grouped(x, KV, d) for x in st["kv"][k0: k0 + nk].chunk(2, dim=1))
        q, do = _grouped(st["q"][q0: q0 + nq], KV, d), _grouped(st["dout"][q0: q0 + nq], KV, d)
        p, _ = _weights(q, k, scale)
        dv = p.transpose(1, 2) @ do
        dz = do @ v.transpose(1, 2)
        dz = p * (dz - (p * dz).sum(-1, keepdim=True))
        dq[q0: q0 + nq] = _flat((dz @ k) * scale, nq)
        dk = (dz.transpose(1, 2) @ q) * scale
        dkv[k0: k0 + nk] = torch.cat([_flat(dk, nk), _flat(dv, nk)], dim=1)
    return [dq, dkv]


# ------------------------------------------------------------------ one pass
def _ok(rc):
    if rc != 0:
        raise RuntimeError("status %d" % rc)


def _own(st):
    from megatron_transformer_layer_gb300 import _lib as L
    c = st["case"]
    stream = torch.cuda.current_stream()
    if c["op"].startswith("norm"):
        heads = (c["tokens"], c["q_heads"], c["k_heads"], c["head_dim"])
        positions = (st["positions"], st["inv_freq"], st["spec"]) if c["rot_dim"] else (None, None, None)
        if c["op"] == "norm":
            _ok(L.mc_qk_norm_forward(st["x"], st["out"], *heads, st["x"].stride(0), st["out"].stride(0), st["norm"],
                                     *positions, stream=stream))
            return st["out"]
        _ok(L.mc_qk_norm_backward(st["x"], st["dout"], st["out"], *heads, st["x"].stride(0), st["dout"].stride(0),
                                  st["out"].stride(0), st["norm"], *positions, st["grads_c"], 0, st["scratch"],
                                  stream=stream))
        return [st["out"], st["grads"]]
    a = c["kv_heads"] * c["head_dim"]
    k, v = st["kv"][:, :a], st["kv"][:, a:]
    if c["op"] == "cross":
        _ok(L.mc_attention_forward_cross(st["q"], k, v, st["o"], st["lse"], st["cross"], stream=stream))
        return [st["o"], st["lse"]]
    _ok(L.mc_attention_backward_cross(st["q"], k, v, st["o"], st["lse"], st["dout"], st["dq"], st["dkv"][:, :a],
                                      st["dkv"][:, a:], st["delta"], st["cross"], st["ws"], st["ws_bytes"],
                                      stream=stream))
    return [st["dq"], st["dkv"]]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_backward, "cross": lambda s: list(_plain_cross(s)),
            "cross_bwd": _plain_cross_backward}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"].startswith("norm"):
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        size = 2 if case["dtype"] == "bf16" else 4
        back = case["op"] == "norm_bwd"
        small = (4 * case["tokens"] * case["axes"] + 2 * case["rot_dim"] if case["rot_dim"] else 0) + 4 * case["head_dim"]
        return {"bytes": (3 if back else 2) * n * size + small + (16 * case["head_dim"] if back else 0),
                "flops": (16 if back else 8) * n}
    H, KV, d = case["heads"], case["kv_heads"], case["head_dim"]
    # (who meets whom depends on the order of the lengths, but little: seed 0 stands for all)
    q, k = _lengths(case, "q", 0), _lengths(case, "k", 0)
    pairs = sum(a * b for a, b in zip(q, k))
    q_bytes, k_bytes = 2 * sum(q) * H * d, 2 * sum(k) * KV * d
    if case["op"] == "cross":
        return {"bytes": 2 * q_bytes + 2 * k_bytes + 4 * H * sum(q), "flops": 4 * d * H * pairs}
    return {"bytes": 4 * q_bytes + 4 * k_bytes + 4 * H * sum(q), "flops": 10 * d * H * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(case, seed):
    st = prepare(case, seed)
    qh, kh, d, r = case["q_heads"], case["k_heads"], case["head_dim"], case["rot_dim"]
    T, H = case["tokens"], qh + kh
    x = st["x"].double()[:, : H * d].unflatten(1, (H, d)).clone()
    back = case["op"] == "norm_bwd"
    mean = x.mean(2, keepdim=True) if case["centred"] else torch.zeros(T, H, 1, dtype=torch.float64, device=DEV)
    std = ((x - mean).square().mean(2, keepdim=True) + st["eps"]).sqrt()
    y = (x - mean) / std

    def turn(z, sign):
        for p in range(r // 2):
            w = sign * st["positions"][int(st["axis"][p])].double() * st["inv_freq"][p].double()
            i, j = (2 * p, 2 * p + 1) if case["adjacent"] else (p, p + r // 2)
            t = torch.complex(z[:, :, i], z[:, :, j]) * torch.polar(torch.ones_like(w), w)[:, None]
            z[:, :, i], z[:, :, j] = t.real, t.imag
        return z

    gain = torch.stack([st["q_gain"]] * qh + [st["k_gain"]] * kh).double()
    if not back:
        z = y * gain
        if case["centred"]:
            z += torch.stack([st["q_shift"]] * qh + [st["k_shift"]] * kh).double()
        return turn(z, 1.0).reshape(T, H * d)
    t = turn(st["dout"].double().reshape(T, H, d).clone(), -1.0)
    grads = []
    for w in (t * y, t) if case["centred"] else (t * y,):
        grads += [w[:, :qh].sum((0, 1))] + ([w[:, qh:].sum((0, 1))] if kh else [])
    u = t * gain
    # the derivative of (x - mean) / std as a projection: off the normed head and, centred, off the ones
    dx = (u - y * (u * y).sum(2, keepdim=True) / d - (u.mean(2, keepdim=True) if case["centred"] else 0.0)) / std
    return [dx.reshape(T, H * d), torch.stack(grads)]


def exact(case, seed):
    if case["op"].startswith("norm"):
        return _exact_norm(case, seed)
    st = prepare(case, seed)
    H, KV, d, n = case["heads"], case["kv_heads"], case["head_dim"], case["n"]
    back = case["op"] == "cross_bwd"
    q_off, q_len, q_rows = _layout(case, "q", seed)
    k_off, k_len, k_rows = _layout(case, "k", seed)
    o = torch.zeros(q_rows, H, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(H, q_rows, dtype=torch.float64, device=DEV)
    dk, dv = (torch.zeros(k_rows, KV, d, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(n):
        lse[:, q_off[i]: q_off[i + 1]] = -math.inf
        rows, keys = slice(q_off[i], q_off[i] + q_len[i]), slice(k_off[i], k_off[i] + k_len[i])
        if not q_len[i] or not k_len[i]:
            continue
        for h in range(H):
            g = h * KV // H
            q = st["q"][rows, h * d: (h + 1) * d].double()
            k = st["kv"][keys, g * d: (g + 1) * d].double()
            v = st["kv"][keys, (KV + g) * d: (KV + g + 1) * d].double()
            z = torch.mm(q, k.t()) / d ** 0.5
            total = torch.logsumexp(z, 1, keepdim=True)
            p = z.sub_(total).exp_()
            if not back:
                o[rows, h] = torch.mm(p, v)
                lse[h, rows] = total[:, 0]
                continue
            do = st["dout"][rows, h * d: (h + 1) * d].double()
            dv[keys, g] += torch.mm(p.t(), do)
            e = torch.mm(do, v.t())
            e = p * (e - (torch.mm(p, v) * do).sum(1, keepdim=True)) / d ** 0.5
            o[rows, h] = torch.mm(e, k)
            dk[keys, g] += torch.mm(e.t(), q)
    if not back:
        return [o.reshape(q_rows, H * d), lse]
    return [o.reshape(q_rows, H * d), torch.cat([dk.reshape(k_rows, -1), dv.reshape(k_rows, -1)], 1)]
