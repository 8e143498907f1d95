"""Cases of the attention stage's operators beyond plain causal attention:
rotary positions with several axes, the interval tables of document / prefix /
window masks, and attention over them (scores optionally capped by a tanh and
biased by the distance), forward and backward.

`run` computes a case in elementary torch operations in 32 bits (rotary angles
in 64), or, with `own`, through the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROWS = 128          # rows of a block in the mask tables
MAX_SORTED = 4096   # blocks up to which the tables are sorted by work


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a small model: the shortest call there is
        {"name": "rotary 1 token", "op": "rotary", "tokens": 1, "heads": 24, "head_dim": 64, "rot_dim": 64, "axes": 1,
         "interleaved": False, "mixed_axes": False, "inverse": False, "dtype": "bf16", "far": 0, "base": 10000.0},
        # Q and K of one layer of the 96-layer GPT over image and text tokens (time, height, width)
        {"name": "rotary 4096 3 axes", "op": "rotary", "tokens": 4096, "heads": 128, "head_dim": 128, "rot_dim": 128,
         "axes": 3, "interleaved": False, "mixed_axes": False, "inverse": False, "dtype": "bf16", "far": 0, "base": 1e6},
        # the gradient's way back, adjacent pairs, half of each head rotated, an odd count of far tokens
        {"name": "rotary backward partial", "op": "rotary", "tokens": 8191, "heads": 32, "head_dim": 128, "rot_dim": 64,
         "axes": 2, "interleaved": True, "mixed_axes": True, "inverse": True, "dtype": "bf16", "far": 1000000, "base": 5e5},
        # a short micro-batch's mask
        {"name": "mask 1x128", "op": "mask", "b": 1, "s": 128, "docs": 4, "pad": 5, "prefix": False, "causal": True,
         "window": 0},
        # a packed micro-batch of 8 sequences: many documents with prefixes, a sliding window, padding at the ends
        {"name": "mask 8x4096", "op": "mask", "b": 8, "s": 4096, "docs": 24, "pad": 77, "prefix": True, "causal": True,
         "window": 1024},
        # the smallest model's shortest sequence, capped scores: latency
        {"name": "forward 1x96", "op": "fwd", "b": 1, "s": 96, "heads": 12, "head_dim": 64, "docs": 1, "pad": 0,
         "prefix": False, "causal": True, "window": 0, "cap": 30.0, "bias": False, "qstd": 3.0},
        # the 96-layer GPT's sequence packed with documents
        {"name": "forward 4096 packed", "op": "fwd", "b": 1, "s": 4096, "heads": 64, "head_dim": 128, "docs": 9, "pad": 61,
         "prefix": False, "causal": True, "window": 0, "cap": 0.0, "bias": False, "qstd": 1.0},
        # a long sequence whose scores are capped
        {"name": "forward 16384 capped", "op": "fwd", "b": 1, "s": 16384, "heads": 16, "head_dim": 128, "docs": 1, "pad": 0,
         "prefix": False, "causal": True, "window": 0, "cap": 50.0, "bias": False, "qstd": 3.0},
        # micro-batches of medium odd sequences with a distance bias and prefixes that see themselves whole
        {"name": "forward 4x1037 biased", "op": "fwd", "b": 4, "s": 1037, "heads": 16, "head_dim": 128, "docs": 3, "pad": 40,
         "prefix": True, "causal": True, "window": 0, "cap": 0.0, "bias": True, "qstd": 1.0},
        # a small model's backward pass: biased, prefixes, odd length
        {"name": "backward 4x509 biased", "op": "bwd", "b": 4, "s": 509, "heads": 12, "head_dim": 64, "docs": 3, "pad": 9,
         "prefix": True, "causal": True, "window": 0, "cap": 0.0, "bias": True, "qstd": 1.0},
        # the backward pass of the packed sequence above
        {"name": "backward 4096 packed", "op": "bwd", "b": 1, "s": 4096, "heads": 64, "head_dim": 128, "docs": 9, "pad": 61,
         "prefix": False, "causal": True, "window": 0, "cap": 0.0, "bias": False, "qstd": 1.0},
        # long capped rows with a sliding window, backward
        {"name": "backward 8192 capped", "op": "bwd", "b": 1, "s": 8192, "heads": 16, "head_dim": 128, "docs": 2, "pad": 3,
         "prefix": False, "causal": True, "window": 4096, "cap": 30.0, "bias": False, "qstd": 3.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "mask", "fwd", "fwd", "bwd", "bwd"])
    if op == "rotary":
        hd = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([hd, hd // 2, hd // 2 - 4])
        heads = _log(rng, 2, 128)
        most = 4096 * 128 * 128 // (heads * hd)
        axes = rng.choice([1, 2, 3, 4])
        return {"op": op, "tokens": _log(rng, 1, min(32768, most)), "heads": heads, "head_dim": hd, "rot_dim": rot,
                "axes": axes, "interleaved": rng.random() < 0.5, "mixed_axes": rng.random() < 0.3,
                "inverse": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "far": rng.choice([0, 0, 100000, 4000000]), "base": rng.choice([1e4, 5e5, 1e6])}
    b = _log(rng, 1, 16)
    case = {"op": op, "b": b, "prefix": rng.random() < 0.4, "causal": rng.random() < 0.85}
    if op == "mask":
        case["s"] = _log(rng, 24, 32768 // b)
    else:
        case["heads"] = rng.choice([1, 2, 5, 12, 20, 32, 64])
        case["head_dim"] = rng.choice([64, 128])
        most = (4.2e9 if op == "fwd" else 1.0e9) / (b * case["heads"])
        case["s"] = _log(rng, 1, min(16384, int(math.sqrt(most))))
        case["cap"] = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
        case["bias"] = rng.random() < 0.35
        case["qstd"] = 3.0 if case["cap"] else 1.0
    s = case["s"]
    case["docs"] = rng.randint(4, 40) if op == "mask" else rng.randint(1, min(12, s))
    case["pad"] = rng.choice([0, 0, min(s // 5, _log(rng, 1, 200))])
    case["window"] = rng.choice([0, 0, _log(rng, max(1, s // 3) if op == "mask" else 1, s)])
    return case


# ------------------------------------------------------------------ inputs
def _doc_lengths(case, seed):
    """Lengths of one sequence's documents.  Attention's are a function of the case alone, so that its
    work is (the seed orders them)."""
    n, total = case["docs"], case["s"] - case["pad"]
    rng = random.Random(n * 7919 + case["s"] + (seed * 104729 if case["op"] == "mask" else 0))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [hi - lo for lo, hi in zip([0] + cuts, cuts + [total])]


def _documents(case, seed):
    """Starts and ends of the documents over all tokens, and their prefix lengths; the
    padding behind a sequence's last document belongs to none."""
    rng = random.Random(seed * 1000003 + 17)
    lens = _doc_lengths(case, seed)
    starts, ends, prefix = [], [], []
    for b in range(case["b"]):
        order = list(range(len(lens)))
        rng.shuffle(order)
        at = b * case["s"]
        for k in order:
            starts.append(at)
            at += lens[k]
            ends.append(at)
            prefix.append(lens[k] // 3 if case["prefix"] else 0)
    return starts, ends, prefix


def _intervals(case, docs):
    """Visible keys [lo, hi) of every token, as CPU int64 [b, s] (the definition, token by token, in vector form)."""
    b, s = case["b"], case["s"]
    starts, ends, prefix = docs
    first = torch.zeros(b * s, dtype=torch.int64)
    last = torch.zeros(b * s, dtype=torch.int64)
    pre = torch.zeros(b * s, dtype=torch.int64)
    for a, e, p in zip(starts, ends, prefix):
        first[a:e], last[a:e], pre[a:e] = a, e, a + p
    t = torch.arange(b * s)
    live = last > first
    hi = torch.maximum(t + 1, torch.minimum(pre, last)) if case["causal"] else last
    lo = first
    if case["window"]:
        lo = torch.maximum(lo, t + 1 - case["window"])
        hi = torch.minimum(hi, t + case["window"])
    base = t // s * s
    lo, hi = torch.where(live, lo - base, 0), torch.where(live, hi - base, 0)
    return lo.view(b, s), hi.view(b, s)


def _sections(case):
    """Pairs of each axis: the first axis takes what is left over."""
    pairs, axes = case["rot_dim"] // 2, case["axes"]
    rest = [pairs // (axes + 1) if axes > 1 else pairs] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _axis_of_pair(case):
    """The axis of each pair: sections one after another, or dealt in turn, an axis leaving when its count is used up."""
    left = _sections(case)
    if not case["mixed_axes"]:
        return [x for x, n in enumerate(left) for _ in range(n)]
    got = []
    while any(left):
        for x in range(len(left)):
            if left[x]:
                got.append(x)
                left[x] -= 1
    return got


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rotary":
        T, H, d = case["tokens"], case["heads"], case["head_dim"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # Q and K lie beside V in each row: the rotated heads are the row's first two thirds
        width = (3 * H + 1) // 2 * d
        st["x"] = _normal(g, (T, width), 1.0, dtype)
        rng = random.Random(seed)
        start = rng.randint(0, 1000) + case["far"]
        step = torch.arange(T, dtype=torch.int64)
        grid = [step + start] + [(step // (7 ** k)) % (13 + 5 * k) + rng.randint(0, 50) for k in range(1, case["axes"])]
        st["positions"] = torch.stack(grid).to(torch.int32).to(DEV)
        st["inv_freq"] = torch.tensor([case["base"] ** (-2.0 * p / case["rot_dim"]) for p in range(case["rot_dim"] // 2)],
                                      dtype=torch.float64).float().to(DEV)
        st["axis"] = torch.tensor(_axis_of_pair(case), device=DEV)
        st["out"] = torch.empty(T, H * d, dtype=dtype, device=DEV)
    else:
        b, s = case["b"], case["s"]
        docs = _documents(case, seed)
        if case["op"] == "mask":
            # offsets of all documents; the padding between two sequences is a document whose tokens see nothing
            offs, pre = [docs[0][0]], []
            for (a, e, p) in zip(*docs):
                if offs[-1] != a:
                    pre.append(-1)
                    offs.append(a)
                pre.append(p)
                offs.append(e)
            st["offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
            st["prefix"] = torch.tensor(pre, dtype=torch.int32, device=DEV)
            n = b * ((s + ROWS - 1) // ROWS)
            st["key_lo"] = torch.empty(b, s, dtype=torch.int32, device=DEV)
            st["key_hi"] = torch.empty(b, s, dtype=torch.int32, device=DEV)
            st["tables"] = torch.empty(2, n, 4, dtype=torch.int32, device=DEV)
            return st
        H, d = case["heads"], case["head_dim"]
        a = H * d
        lo, hi = _intervals(case, docs)
        st["key_lo"], st["key_hi"] = lo.to(torch.int32).to(DEV), hi.to(torch.int32).to(DEV)
        st["qkv"] = _normal(g, (b, s, 3 * a), 1.0, torch.float32)
        st["qkv"][:, :, :a] *= case["qstd"]
        st["qkv"] = st["qkv"].to(torch.bfloat16)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (k + 1) / H) for k in range(H)], device=DEV) if case["bias"] else None
        if case["op"] == "bwd":
            st["dout"] = _normal(g, (b, s, a), 1.0, torch.bfloat16)
            o, st["lse"] = _plain_forward(st)
            st["o"] = o
        st["tables"] = torch.empty(2, b * ((s + ROWS - 1) // ROWS), 4, dtype=torch.int32, device=DEV)
        if own:
            from megatron_transformer_layer_gb300 import _lib as L
            stream = torch.cuda.current_stream()
            _ok(L.mc_attention_mask_intervals(b, s, st["key_lo"], st["key_hi"], st["tables"], stream=stream))
            st["options"] = L.make_attention_options(st["key_lo"], st["key_hi"], st["tables"], slopes=st["slopes"],
                                                     softcap=case["cap"], causal=case["causal"] and not case["prefix"])
            if case["op"] == "fwd":
                st["o"] = torch.empty(b, s, a, dtype=torch.bfloat16, device=DEV)
                st["lse"] = torch.empty(b, H, s, dtype=torch.float32, device=DEV)
            else:
                st["dqkv"] = torch.empty(b, s, 3 * a, dtype=torch.bfloat16, device=DEV)
                st["delta"] = torch.empty(b, H, s, dtype=torch.float32, device=DEV)
                n = L.mc_attention_backward_opt_ws_bytes(b, s, H, d, st["options"])
                st["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
                st["ws_bytes"] = n
    return st


# ------------------------------------------------------------------ the plain forms
def _plain_rotary(st):
    c = st["case"]
    T, H, d, r = c["tokens"], c["heads"], c["head_dim"], c["rot_dim"]
    x = st["x"][:, : H * d].view(T, H, d).float()
    pos = st["positions"][st["axis"]].double().t()                       # [T, pairs]
    ang = pos * st["inv_freq"].double()
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if c["inverse"]:
        sin = -sin
    rot, rest = x[:, :, :r], x[:, :, r:]
    if c["interleaved"]:
        u, v = rot[:, :, 0::2], rot[:, :, 1::2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).reshape(T, H, r)
    else:
        u, v = rot[:, :, : r // 2], rot[:, :, r // 2:]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    return torch.cat([y, rest], dim=-1).reshape(T, H * d).to(st["x"].dtype)


def _plain_tables(lo, hi):
    """The block tables of intervals [b, s]: [2, n, 4]."""
    b, s = lo.shape
    nb = (s + ROWS - 1) // ROWS
    n = b * nb
    big = torch.iinfo(torch.int32).max
    live = lo < hi
    l = torch.full((b, nb * ROWS), big, dtype=torch.int64, device=lo.device)
    h = torch.zeros(b, nb * ROWS, dtype=torch.int64, device=lo.device)
    l[:, :s] = torch.where(live, lo.long(), big)
    h[:, :s] = torch.where(live, hi.long(), 0)
    h = h.view(b, nb, ROWS).amax(-1)
    l = torch.where(h > 0, l.view(b, nb, ROWS).amin(-1), 0)
    k0 = torch.arange(nb, device=lo.device) * ROWS
    sees = (h[:, :, None] > l[:, :, None]) & (l[:, :, None] < k0 + ROWS) & (h[:, :, None] > k0)   # [b, q, k]
    q = torch.arange(nb, device=lo.device)[None, :, None]
    end = torch.where(sees, q + 1, 0).amax(1)
    first = torch.where(end > 0, torch.where(sees, q, big).amin(1), 0)
    bi = torch.arange(b, device=lo.device)[:, None].expand(b, nb)
    blk = torch.arange(nb, device=lo.device)[None].expand(b, nb)
    qt = torch.stack([bi, blk, l, h], -1).view(n, 4)
    kt = torch.stack([bi, blk, first, end], -1).view(n, 4)
    if n <= MAX_SORTED:
        qt = qt[torch.argsort(qt[:, 3] - qt[:, 2], descending=True, stable=True)]
        kt = kt[torch.argsort(kt[:, 3] - kt[:, 2], descending=True, stable=True)]
    else:
        qt = qt.flip(0)
    return torch.stack([qt, kt]).to(torch.int32)


def _plain_mask(st):
    c = st["case"]
    b, s = c["b"], c["s"]
    off, pre = st["offsets"].long(), st["prefix"].long()
    t = torch.arange(b * s, device=off.device)
    k = (off[None, :] <= t[:, None]).sum(1) - 1                          # the last document that starts at or before t
    live = (k >= 0) & (k < off.numel() - 1)
    k = k.clamp(0, off.numel() - 2)
    live = live & (pre[k] >= 0)
    base = t // s * s
    first, last = torch.maximum(off[k], base), torch.minimum(off[k + 1], base + s)
    hi = torch.maximum(t + 1, torch.minimum(off[k] + pre[k], last)) if c["causal"] else last
    lo = first
    if c["window"]:
        lo = torch.maximum(lo, t + 1 - c["window"])
        hi = torch.minimum(hi, t + c["window"])
    lo = torch.where(live, lo - base, 0).view(b, s)
    hi = torch.where(live, hi - base, 0).view(b, s)
    return [lo.to(torch.int32), hi.to(torch.int32), _plain_tables(lo, hi)]


def _heads(x, H, d):
    b, s, _ = x.shape
    return x.float().view(b, s, H, d).transpose(1, 2)


def _scores(st):
    """Scores after cap, bias and mask [b, H, s, s], the cap's derivative (or None), and q, k, v."""
    c = st["case"]
    s, H, d = c["s"], c["heads"], c["head_dim"]
    q, k, v = (_heads(x, H, d) for x in st["qkv"].chunk(3, dim=-1))
    z = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    slope = None
    if c["cap"]:
        t = torch.tanh(z / c["cap"])
        slope = 1.0 - t * t if c["op"] == "bwd" else None
        z = c["cap"] * t
    i = torch.arange(s, device=z.device)
    if c["bias"]:
        z -= st["slopes"][:, None, None] * (i[:, None] - i[None, :]).abs().float()
    seen = (i >= st["key_lo"][:, None, :, None]) & (i < st["key_hi"][:, None, :, None])
    z = torch.where(seen, z, -math.inf)
    return z, slope, q, k, v


def _softmax(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).squeeze(-1)
    return p / torch.where(l > 0, l, 1.0), lse


def _plain_forward(st):
    c = st["case"]
    z, _, _, _, v = _scores(st)
    p, lse = _softmax(z)
    o = (p @ v).transpose(1, 2).reshape(c["b"], c["s"], -1)
    return o.to(torch.bfloat16), lse


def _plain_backward(st):
    c = st["case"]
    z, slope, q, k, v = _scores(st)
    p, _ = _softmax(z)
    del z
    do = _heads(st["dout"], c["heads"], c["head_dim"])
    dv = p.transpose(-1, -2) @ do
    dz = do @ v.transpose(-1, -2)
    dz = p * (dz - (p * dz).sum(-1, keepdim=True))
    if slope is not None:
        dz = dz * slope
    scale = 1.0 / math.sqrt(c["head_dim"])
    dq, dk = (dz @ k) * scale, (dz.transpose(-1, -2) @ q) * scale
    return torch.cat([x.transpose(1, 2).reshape(c["b"], c["s"], -1) for x in (dq, dk, dv)], dim=-1).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def _ok(rc):
    if rc != 0:
        raise RuntimeError("status %d" % rc)


def _own(st):
    from megatron_transformer_layer_gb300 import _lib as L
    c = st["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "rotary":
        call = L.mc_rotary_backward if c["inverse"] else L.mc_rotary_forward
        spec = L.make_rotary_spec(c["rot_dim"], _sections(c), interleaved_pairs=c["interleaved"],
                                  interleaved_axes=c["mixed_axes"])
        _ok(call(st["x"], st["out"], c["tokens"], c["heads"], c["head_dim"], st["x"].stride(0), st["out"].stride(0),
                 st["positions"], st["inv_freq"], spec, stream=stream))
        return st["out"]
    if c["op"] == "mask":
        _ok(L.mc_attention_mask_documents(st["offsets"], st["prefix"].numel(), st["prefix"], int(c["causal"]), c["window"],
                                          c["b"], c["s"], st["key_lo"], st["key_hi"], st["tables"], stream=stream))
        return [st["key_lo"], st["key_hi"], st["tables"]]
    if c["op"] == "fwd":
        _ok(L.mc_attention_forward_opt(st["qkv"], st["o"], st["lse"], c["b"], c["s"], c["heads"], c["head_dim"],
                                       st["options"], stream=stream))
        return [st["o"], st["lse"]]
    _ok(L.mc_attention_backward_opt(st["qkv"], st["o"], st["lse"], st["dout"], st["dqkv"], st["delta"], c["b"], c["s"],
                                    c["heads"], c["head_dim"], st["options"], st["ws"], st["ws_bytes"], stream=stream))
    return st["dqkv"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rotary":
        return _plain_rotary(state)
    if op == "mask":
        return _plain_mask(state)
    if op == "fwd":
        return list(_plain_forward(state))
    return _plain_backward(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * case["head_dim"] * size + 4 * case["tokens"] * case["axes"] + 2 * case["rot_dim"],
                "flops": 3 * n * case["rot_dim"]}
    b, s = case["b"], case["s"]
    n = b * ((s + ROWS - 1) // ROWS)
    if case["op"] == "mask":
        return {"bytes": 8 * b * s + 32 * n + 8 * case["docs"] * b, "flops": 8 * b * s}
    lo, hi = _intervals(case, _documents(case, 0))
    pairs = int((hi - lo).clamp(min=0).sum())
    H, d = case["heads"], case["head_dim"]
    tokens = b * s * H * d * 2
    if case["op"] == "fwd":
        return {"bytes": 4 * tokens + 4 * b * s * H + 8 * b * s, "flops": 4 * d * H * pairs}
    return {"bytes": 8 * tokens + 4 * b * s * H + 8 * b * s, "flops": 10 * d * H * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "mask":
        return None
    if case["op"] == "rotary":
        T, H, d, r = case["tokens"], case["heads"], case["head_dim"], case["rot_dim"]
        x = st["x"][:, : H * d].reshape(T, H, d).double()
        f = st["inv_freq"].double()
        pos = st["positions"].double()
        sign = -1.0 if case["inverse"] else 1.0
        for p, ax in enumerate(_axis_of_pair(case)):
            w = sign * (pos[ax] * f[p])
            turn = torch.polar(torch.ones_like(w), w)[:, None]
            i, j = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + r // 2)
            z = torch.complex(x[:, :, i], x[:, :, j]) * turn
            x[:, :, i], x[:, :, j] = z.real, z.imag
        return x.reshape(T, H * d)
    b, s, H, d = case["b"], case["s"], case["heads"], case["head_dim"]
    a = H * d
    # who sees whom, from the documents themselves
    starts, ends, prefix = _documents(case, seed)
    doc = torch.full((b * s,), -1, dtype=torch.int64)
    lead = torch.zeros(b * s, dtype=torch.int64)
    for k, (x0, x1, p) in enumerate(zip(starts, ends, prefix)):
        doc[x0:x1], lead[x0:x1] = k, x0 + p
    doc, lead = doc.to(DEV).view(b, s), lead.to(DEV).view(b, s)
    i = torch.arange(s, device=DEV)
    qkv = st["qkv"]
    back = case["op"] == "bwd"
    out = torch.zeros(b, s, 3 * a if back else a, dtype=torch.float64, device=DEV)
    lse = torch.zeros(b, H, s, dtype=torch.float64, device=DEV)
    for bi in range(b):
        seen = (doc[bi][:, None] == doc[bi][None, :]) & (doc[bi][:, None] >= 0)
        if case["causal"]:
            seen &= (i[None, :] <= i[:, None]) | (i[None, :] + bi * s < lead[bi][:, None])
        if case["window"]:
            seen &= (i[:, None] - i[None, :]).abs() < case["window"]
        empty = ~seen.any(1)
        for h in range(H):
            q, k, v = (qkv[bi, :, n * a + h * d: n * a + (h + 1) * d].double() for n in range(3))
            z = q @ k.t() / math.sqrt(d)
            grad = None
            if case["cap"]:
                z = torch.tanh_(z / case["cap"])
                grad = 1 - z * z if back else None
                z = z * case["cap"]
            if case["bias"]:
                z = z - st["slopes"][h].double() * (i[:, None] - i[None, :]).abs()
            z.masked_fill_(~seen, -math.inf)
            n = torch.logsumexp(z, 1)
            p = torch.exp_(z - torch.where(empty, 0.0, n)[:, None])
            if not back:
                out[bi, :, h * d:(h + 1) * d] = p @ v
                lse[bi, h] = n
                continue
            do = st["dout"][bi, :, h * d:(h + 1) * d].double()
            g = do @ v.t()
            g = p * (g - ((p @ v) * do).sum(1, keepdim=True))
            if grad is not None:
                g *= grad
            out[bi, :, h * d:(h + 1) * d] = g @ k / math.sqrt(d)
            out[bi, :, a + h * d: a + (h + 1) * d] = g.t() @ q / math.sqrt(d)
            out[bi, :, 2 * a + h * d: 2 * a + (h + 1) * d] = p.t() @ do
    return out if back else [out, lse]
