"""The operators around the quantised linears that a fine-tuning step and a serving step run, as
measurable cases: causal attention over packed sequences with its backward pass, attention of new
tokens over a key/value cache, root-mean-square norm with the residual's addition, and 8-bit
activation checkpoints with the adapted linears' backward that reads them.

With ``own`` False every operator is computed in its plain form (elementary torch operations in
float32, rounded once at the end); with ``own`` True by the framework's calls. ``exact`` gives the
same outputs from the definitions in float64.

Kinds of cases (sizes follow the layers of workloads.py where a comment says so):

* ``train``   attention over packed sequences: forward, then backward.
* ``cache``   attention of ``nq`` new tokens per sequence over a padded key/value cache.
* ``norm``    h = x + residual, y = h rsqrt(mean(h^2) + eps) w; ``act8`` also keeps y as an 8-bit
              checkpoint and restores it; ``grad`` also runs the backward pass.
* ``act8``    a bf16 activation to its 8-bit checkpoint and back.
* ``bwd8``    the backward of linears that share an input kept as an 8-bit checkpoint.
"""
import math

import torch

own = False

EPS = 1e-5          # the norm's epsilon
INV127 = 127.0      # 8-bit codes run from -127 to 127
NEG = float("-inf")

# NF4 codes (the framework's codebook), as float32 values
NF4 = (-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
       -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
       0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0)


# ------------------------------------------------------------------------- the cases
def listed():
    return [
        # the attention of one Llama-3.1-8B-shaped layer in training: one sequence of 2048 tokens
        {"name": "train 8B layer", "kind": "train", "lens": "2048", "heads": 32, "kv": 8, "d": 128,
         "causal": True, "window": 0, "fused": False},
        # a packed fine-tuning batch of 4096 tokens on the 70B-shaped block: ragged conversations
        {"name": "train 70B packed", "kind": "train", "lens": "1,700,1031,64,1500,17,783", "heads": 64,
         "kv": 8, "d": 128, "causal": True, "window": 0, "fused": False},
        # a small model's step: few short sequences, head size 64, a sliding window, q/k/v as slices
        # of one projection's output
        {"name": "train small window", "kind": "train", "lens": "333,90,1", "heads": 8, "kv": 8, "d": 64,
         "causal": True, "window": 128, "fused": True},
        # serving: 512 new prompt tokens of two sequences on top of what their caches hold
        {"name": "prefill chunk", "kind": "cache", "nq": 512, "nk": "4096,1911", "room": 4096, "heads": 32,
         "kv": 8, "d": 128, "causal": True, "window": 0},
        # serving: one token each for sixteen sequences of unequal length on the 70B shape
        {"name": "decode 16", "kind": "cache", "nq": 1, "room": 8192, "heads": 64, "kv": 8, "d": 128,
         "nk": "8191,4000,130,1,7777,2048,6001,513,8000,33,1024,5555,3333,640,7000,255",
         "causal": True, "window": 0},
        # serving: one token of one short conversation, where latency is all
        {"name": "decode 1", "kind": "cache", "nq": 1, "nk": "601", "room": 1024, "heads": 32, "kv": 8,
         "d": 128, "causal": True, "window": 0},
        # the norm before q/k/v of the 8B-shaped layer, keeping the 8-bit checkpoint of its output
        {"name": "norm 8B act8", "kind": "norm", "m": 2048, "k": 4096, "residual": True, "act8": True,
         "grad": False},
        # the norm of the 70B-shaped block, forward and backward with the weight's gradient
        {"name": "norm 70B train", "kind": "norm", "m": 4096, "k": 8192, "residual": True, "act8": False,
         "grad": True},
        # the norm of one token while serving
        {"name": "norm one token", "kind": "norm", "m": 1, "k": 4096, "residual": True, "act8": False,
         "grad": False},
        # the input of the 8B-shaped layer's down projection, kept in 8 bits and restored
        {"name": "checkpoint 8B down", "kind": "act8", "m": 2048, "k": 14336},
        # the backward of gate and up of the 8B-shaped layer from one 8-bit checkpoint
        {"name": "backward 8B gate up", "kind": "bwd8", "m": 2048, "n": "14336,14336", "k": 4096, "r": 16,
         "dx": True},
        # a short ragged batch through q, k and v of the 8B-shaped layer at rank 64; the first layer's
        # input needs no gradient
        {"name": "backward q k v short", "kind": "bwd8", "m": 77, "n": "4096,1024,1024", "k": 4096, "r": 64,
         "dx": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    while "3072" in ",".join(map(str, case.values())).split(","):   # a size that no layer here has
        case = _draw(rng)
    return case


def _draw(rng):
    kind = rng.choice(["train", "train", "cache", "cache", "norm", "norm", "act8", "bwd8"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 128])
    window = rng.choice([0, 0, 0, 0, _log(rng, 16, 1024)])
    if kind == "train":
        total = _log(rng, 16, 2500)
        cuts = sorted(rng.randrange(1, total + 1) for _ in range(rng.choice([0, 0, 1, 3, 6])))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return {"kind": kind, "lens": ",".join(map(str, lens)), "heads": heads, "kv": kv, "d": d,
                "causal": rng.random() < 0.8, "window": window, "fused": rng.random() < 0.3}
    if kind == "cache":
        batch = _log(rng, 1, 16)
        room = _log(rng, 16, 8192)
        nq = 1 if rng.random() < 0.6 else _log(rng, 2, max(2, 1024 // batch))
        nk = [_log(rng, 1, room) for _ in range(batch)]
        return {"kind": kind, "nq": nq, "nk": ",".join(map(str, nk)), "room": room, "heads": heads, "kv": kv,
                "d": d, "causal": True, "window": window}
    if kind == "norm":
        return {"kind": kind, "m": _log(rng, 1, 4096), "k": 64 * _log(rng, 1, 128), "residual": rng.random() < 0.8,
                "act8": rng.random() < 0.4, "grad": rng.random() < 0.5}
    if kind == "act8":
        return {"kind": kind, "m": _log(rng, 1, 2048), "k": 64 * _log(rng, 1, 224)}
    n = [16 * _log(rng, 4, 512) for _ in range(rng.choice([1, 2, 3]))]
    return {"kind": kind, "m": _log(rng, 1, 2048), "n": ",".join(map(str, n)), "k": 64 * _log(rng, 4, 64),
            "r": rng.choice([16, 32, 64, 128]), "dx": rng.random() < 0.7}


def _ints(text):
    return [int(v) for v in str(text).split(",")]


# ------------------------------------------------------------------------- inputs
def _rand(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=gen.device) * std).to(dtype)


def _act8_of(x):
    """8-bit codes and block maxima of a bf16 [m, k] activation, in elementary operations."""
    b = x.float().reshape(x.shape[0], -1, 64)
    a = b.abs().amax(-1, keepdim=True)
    codes = torch.round(b * INV127 / torch.where(a == 0, torch.ones_like(a), a))
    return codes.to(torch.int8).reshape(x.shape), a.to(torch.bfloat16).reshape(x.shape[0], -1)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    s = {"case": case}
    kind = case["kind"]
    if kind == "train":
        lens = _ints(case["lens"])
        t, h, kv, d = sum(lens), case["heads"], case["kv"], case["d"]
        if case["fused"]:   # one projection's output, q, k and v side by side in each token's row
            qkv = _rand(g, t, h + 2 * kv, d, std=1.2)
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        else:
            s["q"], s["k"], s["v"] = _rand(g, t, h, d, std=1.5), _rand(g, t, kv, d), _rand(g, t, kv, d)
        s["do"] = _rand(g, t, h, d)
        starts = [sum(lens[:i]) for i in range(len(lens))]
        s["seqs"] = [(a, n, a, n) for a, n in zip(starts, lens)]
        s["ends"] = torch.tensor([a + n for a, n in zip(starts, lens)], device=dev)
    elif kind == "cache":
        nk, nq, room = _ints(case["nk"]), case["nq"], case["room"]
        h, kv, d = case["heads"], case["kv"], case["d"]
        s["q"] = _rand(g, len(nk) * nq, h, d, std=1.5)
        s["k"], s["v"] = _rand(g, len(nk), room, kv, d), _rand(g, len(nk), room, kv, d)
        s["seqs"] = [(i * nq, nq, i * room, n) for i, n in enumerate(nk)]
        s["nk"] = torch.tensor(nk, device=dev)
    elif kind == "norm":
        m, k = case["m"], case["k"]
        s["x"] = _rand(g, m, k)
        s["residual"] = _rand(g, m, k, std=2.0) if case["residual"] else None
        s["w"] = (1.0 + 0.2 * torch.randn(k, generator=g, device=dev)).to(torch.bfloat16)
        if case["grad"]:
            s["dy"], s["dh"] = _rand(g, m, k), _rand(g, m, k)
    elif kind == "act8":
        s["x"] = _rand(g, case["m"], case["k"])
        s["x"][:, 5] *= 12.0   # one feature that stands out, as activations have
    else:
        n, m, k, r = _ints(case["n"]), case["m"], case["k"], case["r"]
        x = _rand(g, m, k)
        s["codes"], s["absmax"] = _act8_of(x)
        s["scale"] = 32.0 / r
        s["w"], s["A"], s["B"], s["dy"], s["u"] = [], [], [], [], []
        for rows in n:
            nb = rows * k // 64
            packed = torch.randint(0, 256, (rows * k // 2,), generator=g, device=dev, dtype=torch.uint8)
            scale_q = torch.randint(0x28, 0x39, (nb,), generator=g, device=dev, dtype=torch.uint8)   # 0.25 .. 1
            c2 = 0.04 + 0.02 * torch.rand((nb + 255) // 256, generator=g, device=dev)
            a = _rand(g, r, k, std=0.01)
            s["w"].append((packed, scale_q, c2))
            s["A"].append(a)
            s["B"].append(_rand(g, rows, r, std=0.01))
            s["dy"].append(_rand(g, m, rows))
            s["u"].append(x.float() @ a.float().t())
    return s


# ------------------------------------------------------------------------- the plain forms
def _plain_scores(q, k, mask, scale):
    """Probabilities and log-sum-exp of masked scores in float32; rows with no key give 0 and -inf."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill(~mask, NEG)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return p, lse


def _plain_train(s):
    c = s["case"]
    h, kv, d = c["heads"], c["kv"], c["d"]
    t, g = s["q"].shape[0], c["heads"] // c["kv"]
    scale = 1.0 / math.sqrt(d)
    at = torch.arange(t, device=s["q"].device)
    of = torch.searchsorted(s["ends"], at, right=True)      # the sequence of each token
    mask = of[:, None] == of[None, :]
    if c["causal"]:
        mask = mask & (at[:, None] >= at[None, :])
    if c["window"]:
        mask = mask & (at[:, None] - at[None, :] < c["window"])
    # [kv, g, t, d] queries against [kv, 1, t, d] keys: the group's query heads share a key head
    q = s["q"].float().reshape(t, kv, g, d).permute(1, 2, 0, 3).contiguous()
    do = s["do"].float().reshape(t, kv, g, d).permute(1, 2, 0, 3).contiguous()
    k = s["k"].float().permute(1, 0, 2).contiguous()[:, None]
    v = s["v"].float().permute(1, 0, 2).contiguous()[:, None]
    p, lse = _plain_scores(q, k, mask, scale)
    o = torch.matmul(p, v)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
    dv = torch.matmul(p.transpose(-1, -2), do).sum(1)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(1)
    heads = lambda x: x.permute(2, 0, 1, 3).reshape(t, h, d).to(torch.bfloat16)  # noqa: E731
    keys = lambda x: x.permute(1, 0, 2).contiguous().to(torch.bfloat16)  # noqa: E731
    return {"o": heads(o), "lse": lse.reshape(h, t), "dq": heads(dq), "dk": keys(dk), "dv": keys(dv)}


def _plain_cache(s):
    c = s["case"]
    h, kv, d, nq = c["heads"], c["kv"], c["d"], c["nq"]
    b, g, room = s["k"].shape[0], c["heads"] // c["kv"], c["room"]
    key = torch.arange(room, device=s["q"].device)
    last = s["nk"][:, None] - nq + torch.arange(nq, device=s["q"].device)      # a row's own position
    mask = (key < s["nk"][:, None, None]) & (key <= last[:, :, None])
    if c["window"]:
        mask = mask & (key > last[:, :, None] - c["window"])
    q = s["q"].float().reshape(b, nq, kv, g, d).permute(0, 2, 3, 1, 4).contiguous()
    k = s["k"].float().permute(0, 2, 1, 3).contiguous()[:, :, None]
    v = s["v"].float().permute(0, 2, 1, 3).contiguous()[:, :, None]
    p, _ = _plain_scores(q, k, mask[:, None, None], 1.0 / math.sqrt(d))
    o = torch.matmul(p, v)
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(b * nq, h, d).to(torch.bfloat16)}


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    w = s["w"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = (h * rstd * w).to(torch.bfloat16)
    hb = h.to(torch.bfloat16)
    out = {"h": hb, "y": y, "rstd": rstd.squeeze(-1)}
    if c["act8"]:
        codes, a = _act8_of(y)
        out["restored"] = _plain_restore(codes, a)
    if c["grad"]:
        xhat = hb.float() * rstd
        wdy = s["dy"].float() * w
        dx = rstd * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True)) + s["dh"].float()
        out["dx"] = dx.to(torch.bfloat16)
        out["dw"] = (s["dy"].float() * xhat).sum(0)
    return out


def _plain_restore(codes, a):
    m, k = codes.shape
    return (codes.float().reshape(m, -1, 64) * (a.float() / INV127)[:, :, None]).reshape(m, k).to(torch.bfloat16)


def _plain_weight(w, n, k):
    """The bf16 weight that packed NF4 indices and double-quantised scales stand for, in float32."""
    packed, scale_q, c2 = w
    book = torch.tensor(NF4, device=packed.device)
    idx = torch.stack([packed >> 4, packed & 15], -1).reshape(-1, 64).long()
    c1 = scale_q.view(torch.float8_e4m3fn).float() * c2.repeat_interleave(256)[:scale_q.numel()]
    return (book[idx] * c1[:, None]).to(torch.bfloat16).float().reshape(n, k)


def _plain_linear(dy, w, a, b, u, x, scale, dx):
    w = _plain_weight(w, b.shape[0], a.shape[1]) if dx else None
    dy, a, b = dy.float(), a.float(), b.float()
    v = dy @ b
    return ((dy @ w + scale * (v @ a)).to(torch.bfloat16) if dx else None, scale * (v.t() @ x), scale * (dy.t() @ u))


def _plain_bwd8(s):
    m, k = s["codes"].shape
    x = (s["codes"].float().reshape(m, -1, 64) * (s["absmax"].float() / INV127)[:, :, None]).reshape(m, k)
    got = [_plain_linear(*one, x, s["scale"], s["case"]["dx"]) for one in
           zip(s["dy"], s["w"], s["A"], s["B"], s["u"])]
    return {"dx": [o[0] for o in got], "dA": [o[1] for o in got], "dB": [o[2] for o in got]}


# ------------------------------------------------------------------------- the framework's calls
def _own_train(s):
    import bit_nf4_quantised_amd as nf4
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    seqs = nf4.AttnSeqs(s["seqs"], causal=c["causal"], window=c["window"])
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
    nf4.qlora_attn_fwd(seqs, q, k, v, o, lse)
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v))
    nf4.qlora_attn_bwd(seqs, q, k, v, o, lse, s["do"], dq, dk, dv)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _own_cache(s):
    import bit_nf4_quantised_amd as nf4
    c, q = s["case"], s["q"]
    seqs = nf4.AttnSeqs(s["seqs"], causal=c["causal"], window=c["window"])
    o = torch.empty_like(q)
    nf4.qlora_attn_fwd(seqs, q, s["k"].flatten(0, 1), s["v"].flatten(0, 1), o)
    return {"o": o}


def _own_norm(s):
    import bit_nf4_quantised_amd as nf4
    c, x = s["case"], s["x"]
    h, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    kept = nf4.empty_act8(*x.shape, device=x.device) if c["act8"] else None
    nf4.qlora_rmsnorm_fwd(x, s["w"], EPS, y, residual=s["residual"], h=h, rstd=rstd, act8=kept)
    out = {"h": h, "y": y, "rstd": rstd}
    if c["act8"]:
        out["restored"] = torch.empty_like(x)
        nf4.qlora_act8_unpack(kept, out["restored"])
    if c["grad"]:
        out["dx"] = torch.empty_like(x)
        out["dw"] = torch.empty(x.shape[1], dtype=torch.float32, device=x.device)
        nf4.qlora_rmsnorm_bwd(s["dy"], h, s["w"], rstd, out["dx"], dw=out["dw"], dh=s["dh"])
    return out


def _own_act8(s):
    import bit_nf4_quantised_amd as nf4
    x = s["x"]
    kept = nf4.empty_act8(*x.shape, device=x.device)
    nf4.qlora_act8_pack(x, kept)
    out = torch.empty_like(x)
    nf4.qlora_act8_unpack(kept, out)
    return out


def _own_bwd8(s):
    import bit_nf4_quantised_amd as nf4
    m, k = s["codes"].shape
    dev = s["codes"].device
    kept = nf4.Act8(s["codes"], s["absmax"], m, k)
    ws = [nf4.NF4Weight(*w, b.shape[0], k) for w, b in zip(s["w"], s["B"])]
    dx = [torch.empty(m, k, dtype=torch.bfloat16, device=dev) for _ in ws] if s["case"]["dx"] else None
    da = [torch.empty(a.shape, dtype=torch.float32, device=dev) for a in s["A"]]
    db = [torch.empty(b.shape, dtype=torch.float32, device=dev) for b in s["B"]]
    nf4.qlora_linear_bwd_act8(ws, kept, s["dy"], s["A"], s["B"], s["scale"], s["u"], dx, da, db)
    return {"dx": dx if dx is not None else [None] * len(ws), "dA": da, "dB": db}


def _plain_act8(s):
    return _plain_restore(*_act8_of(s["x"]))


PLAIN = {"train": _plain_train, "cache": _plain_cache, "norm": _plain_norm, "act8": _plain_act8,
         "bwd8": _plain_bwd8}
OWN = {"train": _own_train, "cache": _own_cache, "norm": _own_norm, "act8": _own_act8, "bwd8": _own_bwd8}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["kind"]](state)


# ------------------------------------------------------------------------- what a pass cannot do without
def _pairs(nq, nk, causal, window):
    """Visible (query, key) pairs of one sequence whose last query stands at its last key."""
    total = 0
    for i in range(nq):
        at = nk - nq + i
        hi = min(nk, at + 1) if causal else nk
        lo = max(0, at - window + 1) if window else 0
        total += max(0, hi - lo)
    return total


def work(case):
    kind = case["kind"]
    if kind == "train":
        lens = _ints(case["lens"])
        t, h, kv, d = sum(lens), case["heads"], case["kv"], case["d"]
        pairs = sum(_pairs(n, n, case["causal"], case["window"]) for n in lens)
        # q, do in and o, dq out; k, v in and dk, dv out; lse
        return {"bytes": 2 * t * d * (4 * h + 4 * kv) + 4 * t * h, "flops": 14 * d * h * pairs}
    if kind == "cache":
        nk, nq, h, kv, d = _ints(case["nk"]), case["nq"], case["heads"], case["kv"], case["d"]
        pairs = sum(_pairs(nq, n, True, case["window"]) for n in nk)
        keys = sum(min(n, case["window"] + nq - 1) if case["window"] else n for n in nk)
        return {"bytes": 2 * d * (2 * h * nq * len(nk) + 2 * kv * keys), "flops": 4 * d * h * pairs}
    m, k = case["m"], case["k"]
    kept = m * k + m * k // 64 * 2
    if kind == "norm":
        passes = (2 if case["residual"] else 1) + 2
        b = 2 * m * k * passes + 2 * k + 4 * m
        b += (2 * m * k) if case["act8"] else 0               # the restored activation
        b += (2 * m * k * 3 + 4 * k) if case["grad"] else 0   # dy, dh in; dx, dw out
        return {"bytes": b, "flops": m * k * (4 + 4 * bool(case["act8"]) + 10 * bool(case["grad"]))}
    if kind == "act8":
        return {"bytes": 4 * m * k, "flops": 6 * m * k}
    n, r = _ints(case["n"]), case["r"]
    b, f = kept, 0
    for rows in n:
        b += 2 * m * rows + 4 * m * r + 2 * rows * r + 4 * r * (k + rows)     # dy, u, B in; dA, dB out
        f += 2 * m * rows * r * 2 + 2 * m * r * k                             # v, dB; dA
        if case["dx"]:
            b += rows * k // 2 + rows * k // 64 + 2 * r * k + 2 * m * k       # W, A in; dx out
            f += 2 * m * rows * k + 2 * m * r * k
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------- the definitions in 64 bits
def _exact_head(q, k, v, hidden, scale, do=None):
    """One query head of one sequence from the definition: o, lse and, given do, the gradients."""
    z = (q @ k.t()) * scale
    z[hidden] = NEG
    lse = torch.logsumexp(z, 1) if z.shape[1] else torch.full((z.shape[0],), NEG, dtype=z.dtype, device=z.device)
    p = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    o = p @ v
    if do is None:
        return o, lse
    dp = do @ v.t()
    dz = p * (dp - (dp * p).sum(1, keepdim=True))
    return o, lse, scale * (dz @ k), scale * (dz.t() @ q), p.t() @ do


def _exact_hidden(nq, nk, causal, window, dev):
    i = torch.arange(nk - nq, nk, device=dev)[:, None]
    j = torch.arange(nk, device=dev)[None, :]
    hidden = (j > i) if causal else torch.zeros(nq, nk, dtype=torch.bool, device=dev)
    return (hidden | (j <= i - window)) if window else hidden


def _exact_attn(s, k_rows, v_rows):
    c = s["case"]
    g, scale = c["heads"] // c["kv"], c["d"] ** -0.5
    train = c["kind"] == "train"
    q, k, v = s["q"].double(), k_rows, v_rows
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(c["heads"], q.shape[0], dtype=torch.float64, device=q.device)
    dk = torch.zeros(k.shape, dtype=torch.float64, device=q.device) if train else None
    dv = torch.zeros_like(dk) if train else None
    for q0, nq, k0, nk in s["seqs"]:
        if nq == 0:
            continue
        hidden = _exact_hidden(nq, nk, c["causal"], c["window"], q.device)
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(c["heads"]):
            kk, vv = k[b, h // g].double(), v[b, h // g].double()
            if not train:
                o[a, h], lse[h, a] = _exact_head(q[a, h], kk, vv, hidden, scale)
                continue
            o[a, h], lse[h, a], dq[a, h], one, two = _exact_head(q[a, h], kk, vv, hidden, scale,
                                                                 s["do"][a, h].double())
            dk[b, h // g] += one
            dv[b, h // g] += two
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o}


def _exact_codes(y):
    """The checkpoint's values of bf16 numbers held in float64: nearest code, ties to the even one."""
    b = y.reshape(y.shape[0], -1, 64)
    a = b.abs().amax(-1, keepdim=True)
    codes = torch.round(b * 127.0 / torch.where(a > 0, a, torch.ones_like(a)))
    return (codes * a / 127.0).reshape(y.shape)


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    rstd = 1.0 / torch.sqrt((h ** 2).sum(1) / h.shape[1] + EPS)
    y = h * rstd[:, None] * s["w"].double()
    out = {"h": h, "y": y, "rstd": rstd}
    if c["act8"]:   # the checkpoint is of the y that the linears read, so of its rounding to bf16
        out["restored"] = _exact_codes(y.to(torch.bfloat16).double())
    if c["grad"]:   # the backward reads the stored h
        n = h.to(torch.bfloat16).double() * rstd[:, None]
        dn = s["dy"].double() * s["w"].double()
        out["dx"] = s["dh"].double() + rstd[:, None] * (dn - n * (dn * n).sum(1, keepdim=True) / h.shape[1])
        out["dw"] = torch.einsum("mk,mk->k", s["dy"].double(), n)
    return out


def _exact_bwd8(s):
    m, k = s["codes"].shape
    x = s["codes"].double() * s["absmax"].double().repeat_interleave(64, 1) / 127.0
    out = {"dx": [], "dA": [], "dB": []}
    book = torch.tensor(NF4, dtype=torch.float32, device=x.device)
    for (packed, scale_q, c2), a, b, dy, u in zip(s["w"], s["A"], s["B"], s["dy"], s["u"]):
        dy, v = dy.double(), dy.double() @ b.double()
        dx = None
        if s["case"]["dx"]:
            half = torch.empty(packed.numel(), 2, dtype=torch.int64, device=x.device)
            half[:, 0], half[:, 1] = packed // 16, packed % 16
            # the format's value is the bf16 rounding of the float32 product, so it is formed so
            c1 = scale_q.view(torch.float8_e4m3fn).float() * c2[torch.arange(scale_q.numel(), device=x.device) // 256]
            w = (book[half.reshape(-1)] * c1.repeat_interleave(64)).bfloat16().double().reshape(-1, k)
            dx = dy @ w + s["scale"] * (v @ a.double())
        out["dx"].append(dx)
        out["dA"].append(s["scale"] * (v.t() @ x))
        out["dB"].append(s["scale"] * (dy.t() @ u.double()))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "train":
        return _exact_attn(s, s["k"], s["v"])
    if kind == "cache":
        return _exact_attn(s, s["k"].flatten(0, 1), s["v"].flatten(0, 1))
    if kind == "norm":
        return _exact_norm(s)
    if kind == "act8":
        return _exact_codes(s["x"].double())
    return _exact_bwd8(s)
