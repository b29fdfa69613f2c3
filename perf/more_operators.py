"""What stands between a layer's projections and its attention, and a key/value cache in 4 bits, as
measurable cases: rotary positions with and without norms of the query and key heads, each with its
backward pass; a cache that is quantised as it is written and read back; attention over that cache.

With ``own`` False every operator is computed in its plain form (elementary torch operations in float32,
angles and nearest codes in float64, rounded once at the end); with ``own`` True by the framework's calls.
``exact`` gives the same outputs from the definitions in float64.

Kinds of cases (sizes follow the layers of workloads.py where a comment says so):

* ``rotate``  query and key heads, normed first where ``norm`` is set, rotated by their tokens' positions;
              ``grad`` also runs the backward pass.
* ``store``   ``nq`` new tokens' keys and values into a 4-bit cache, then the cache read back: the new tokens
              (``read`` new) or all that the sequences hold (``read`` all).
* ``attend``  attention of ``nq`` new tokens of every sequence over a 4-bit cache.
"""
import math

import torch

own = False

EPS = 1e-6          # the norm's epsilon
BLOCK = 32          # values of the cache that share a scale
NEG = float("-inf")

# the codes of the framework's codebooks, ascending, as float32 values
NF4 = (-1.0, -0.6961928009986877, -0.5250729322433472, -0.39491742849349976, -0.2844413220882416,
       -0.18477340042591095, -0.09104997664690018, 0.0, 0.07958031445741653, 0.16093014180660248,
       0.24611225724220276, 0.3379151225090027, 0.4407097399234772, 0.5626168847084045, 0.722956657409668, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # the values of the bit patterns 0 .. 7; 8 .. 15 negate them
INT4 = tuple(range(-7, 8))
TOP = {"nf4": 1.0, "fp4": 6.0, "int4": 7.0}         # the value that a block's largest magnitude maps to


def _book(name, dev):
    """The value of each of the 16 bit patterns, and the patterns in the order of their values."""
    if name == "nf4":
        return torch.tensor(NF4, device=dev), torch.arange(16, device=dev)
    if name == "int4":
        return torch.tensor(INT4 + (7,), dtype=torch.float32, device=dev), torch.arange(15, device=dev)
    plus = torch.tensor(E2M1, device=dev)
    return torch.cat([plus, -plus]), torch.tensor([15, 14, 13, 12, 11, 10, 9, 0, 1, 2, 3, 4, 5, 6, 7], device=dev)


# ------------------------------------------------------------------------- the cases
def listed():
    return [
        # q and k of one Llama-3.1-8B-shaped layer in training, slices of one projection's output, with
        # frequencies stretched for long contexts
        {"name": "rotate 8B layer", "kind": "rotate", "lens": "2048", "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "pairs": False, "norm": False, "base": 500000.0, "stretch": 8.0, "start": 0, "fused": True, "grad": True},
        # serving: one token far into its conversation, where latency is all
        {"name": "rotate one token", "kind": "rotate", "lens": "1", "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "pairs": False, "norm": False, "base": 500000.0, "stretch": 1.0, "start": 131071, "fused": False,
         "grad": False},
        # a packed fine-tuning batch of 4096 tokens on the 70B-shaped block, heads normed before they are rotated
        {"name": "norm rotate 70B packed", "kind": "rotate", "lens": "1,700,1031,64,1500,17,783", "heads": 64, "kv": 8,
         "d": 128, "rot": 128, "pairs": False, "norm": True, "base": 1000000.0, "stretch": 1.0, "start": 0,
         "fused": False, "grad": True},
        # a small model: heads of 80 of which 32 features are rotated in neighbouring pairs, few ragged sequences
        {"name": "norm rotate small part", "kind": "rotate", "lens": "333,90,1", "heads": 8, "kv": 8, "d": 80, "rot": 32,
         "pairs": True, "norm": True, "base": 10000.0, "stretch": 1.0, "start": 0, "fused": True, "grad": True},
        # serving: 512 new prompt tokens of two sequences into their caches, which are then read whole
        {"name": "store prompt chunk", "kind": "store", "nq": 512, "nk": "4096,1911", "room": 4096, "kv": 8, "d": 128,
         "book": "nf4", "read": "all"},
        # serving: one new token of each of sixteen sequences
        {"name": "store 16 tokens", "kind": "store", "nq": 1, "room": 8192, "kv": 8, "d": 128, "book": "nf4",
         "nk": "8191,4000,130,1,7777,2048,6001,513,8000,33,1024,5555,3333,640,7000,255", "read": "new"},
        # a long prompt in one piece
        {"name": "store long prompt fp4", "kind": "store", "nq": 8191, "nk": "8191", "room": 8192, "kv": 8, "d": 128,
         "book": "fp4", "read": "new"},
        # serving: one token each for sixteen sequences of unequal length on the 70B shape
        {"name": "attend 16 tokens", "kind": "attend", "nq": 1, "room": 8192, "heads": 64, "kv": 8, "d": 128,
         "nk": "8191,4000,130,1,7777,2048,6001,513,8000,33,1024,5555,3333,640,7000,255", "window": 0, "book": "nf4"},
        # serving: one token of one short conversation, where latency is all
        {"name": "attend one token", "kind": "attend", "nq": 1, "nk": "601", "room": 1024, "heads": 32, "kv": 8,
         "d": 128, "window": 0, "book": "nf4"},
        # serving: two very long documents, which a cache of this size is for
        {"name": "attend long fp4", "kind": "attend", "nq": 1, "nk": "131071,60001", "room": 131072, "heads": 64, "kv": 8,
         "d": 128, "window": 0, "book": "fp4"},
        # serving: 512 new prompt tokens of two sequences on top of what their caches hold
        {"name": "attend prompt chunk", "kind": "attend", "nq": 512, "nk": "4096,1911", "room": 4096, "heads": 32,
         "kv": 8, "d": 128, "window": 0, "book": "nf4"},
        # serving: five drafted tokens of each sequence checked at once, a small model with a window
        {"name": "attend drafts int4", "kind": "attend", "nq": 5, "nk": "2000,777,5,64,1301,3999,350,31", "room": 4096,
         "heads": 12, "kv": 4, "d": 80, "window": 1024, "book": "int4"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "store", "attend", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 128])
    if kind == "rotate":
        total = _log(rng, 1, 4096)
        cuts = sorted(rng.randrange(0, total + 1) for _ in range(rng.choice([0, 0, 1, 3, 6])))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        norm = rng.random() < 0.5
        return {"kind": kind, "lens": ",".join(map(str, lens)), "heads": heads, "kv": kv, "d": d,
                "rot": rng.choice([d, d, d // 16 * 8, 16]), "pairs": rng.random() < 0.4, "norm": norm,
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "stretch": rng.choice([1.0, 1.0, 4.0, 8.0]),
                "start": rng.choice([0, 0, _log(rng, 1, 1 << 20)]), "fused": rng.random() < 0.4,
                "grad": rng.random() < 0.6}
    book = rng.choice(["nf4", "nf4", "fp4", "int4"])
    batch = _log(rng, 1, 16)
    if kind == "store":
        room = _log(rng, 16, 8192)
        nq = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(room, 8192 // batch)))
        nk = [_log(rng, nq, room) for _ in range(batch)]
        return {"kind": kind, "nq": nq, "nk": ",".join(map(str, nk)), "room": room, "kv": kv, "d": d, "book": book,
                "read": "all" if room * batch <= 16384 and rng.random() < 0.5 else "new"}
    nq = 1 if rng.random() < 0.6 else _log(rng, 2, max(2, 1024 // batch))
    room = _log(rng, max(16, nq), 8192 if nq > 1 else 262144 // batch)
    nk = [_log(rng, 1, room) for _ in range(batch)]
    return {"kind": kind, "nq": nq, "nk": ",".join(map(str, nk)), "room": room, "heads": heads, "kv": kv, "d": d,
            "window": rng.choice([0, 0, 0, _log(rng, 16, 2048)]), "book": book}


def _ints(text):
    return [int(v) for v in str(text).split(",")]


# ------------------------------------------------------------------------- inputs
def _rand(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=gen.device) * std).to(dtype)


def _freqs(c):
    """Radians a position of every rotated pair. Stretched frequencies: those of more than 4 turns in 8192
    positions stay, those of less than 1 are divided, linear in the turns in between."""
    out = []
    for i in range(c["rot"] // 2):
        f = c["base"] ** (-2.0 * i / c["rot"])
        keep = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1.0) / 3.0)) if c["stretch"] != 1.0 else 1.0
        out.append(f * (keep + (1.0 - keep) / c["stretch"]))
    return out


def _encode(x, book):
    """Blocks of [..., d] values: 16 bytes of codes for 32 values (the first of two in the high half of a byte) and
    the largest magnitude, in bf16. d is filled up to whole blocks with zeros."""
    *lead, d = x.shape
    nb = (d + BLOCK - 1) // BLOCK
    value, order = _book(book, x.device)
    b = torch.zeros(*lead, nb * BLOCK, dtype=torch.float64, device=x.device)
    b[..., :d] = x
    b = b.reshape(*lead, nb, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    v = value[order].double()
    zero = int((v == 0).nonzero()[0])
    at = torch.zeros(b.shape, dtype=torch.int64, device=x.device)
    for i in range(v.numel() - 1):      # codes below the value: a tie takes the lower code
        at += b * TOP[book] > (v[i] + v[i + 1]) / 2 * a
    at = torch.where(a == 0, torch.full_like(at, zero), at)
    p = order[at].to(torch.uint8)
    return p[..., 0::2] * 16 + p[..., 1::2], a.squeeze(-1).to(torch.bfloat16)


def _decode(codes, absmax, d, book):
    """The values that blocks stand for, in float32. The format's value is the bf16 rounding of the float32 product
    of the code and the block's step, so it is formed so."""
    value, _ = _book(book, codes.device)
    step = absmax.float() * torch.tensor(1.0 / TOP[book], device=codes.device)
    p = torch.stack([codes >> 4, codes & 15], -1).long().flatten(-2)
    return (value[p] * step[..., None]).to(torch.bfloat16).float().flatten(-2)[..., :d]


def _new_cache(tokens, kv, d, dev):
    """An empty cache, as views [tokens, kv, blocks, 16] and [tokens, kv, blocks] of arrays whose heads come first."""
    nb = (d + BLOCK - 1) // BLOCK
    return (torch.zeros(kv, tokens, nb, 16, dtype=torch.uint8, device=dev).permute(1, 0, 2, 3),
            torch.zeros(kv, tokens, nb, dtype=torch.bfloat16, device=dev).permute(1, 0, 2))


def _filled_cache(gen, tokens, kv, d, book, std):
    codes, absmax = _new_cache(tokens, kv, d, gen.device)
    for at in range(0, tokens, 1 << 15):
        x = _rand(gen, min(1 << 15, tokens - at), kv, d, std=std)
        x[..., 5] *= 4.0        # one feature that stands out, as keys have
        codes[at:at + x.shape[0]], absmax[at:at + x.shape[0]] = _encode(x, book)
    return codes, absmax


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 6361 + 29)
    s = {"case": case}
    kv, d = case["kv"], case["d"]
    if case["kind"] == "rotate":
        lens, h = _ints(case["lens"]), case["heads"]
        t = sum(lens)
        if case["fused"]:   # one projection's output, q, k and v side by side in each token's row
            qkv = _rand(g, t, h + 2 * kv, d, std=1.5)
            s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + kv]
        else:
            s["q"], s["k"] = _rand(g, t, h, d, std=1.5), _rand(g, t, kv, d, std=1.5)
        s["dq"], s["dk"] = _rand(g, t, h, d), _rand(g, t, kv, d)
        s["positions"] = torch.cat([torch.arange(case["start"], case["start"] + n, device=dev) for n in lens])
        s["freqs"] = _freqs(case)
        one = lambda: (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
        s["qw"], s["kw"] = (one(), one()) if case["norm"] else (None, None)
        return s
    nk, nq, room = _ints(case["nk"]), case["nq"], case["room"]
    s["seqs"] = [(i * nq, nq, i * room, n) for i, n in enumerate(nk)]
    if case["kind"] == "store":
        s["whole"] = [(sum(nk[:i]), n, i * room, n) for i, n in enumerate(nk)]
        s["k"], s["v"] = _rand(g, len(nk) * nq, kv, d), _rand(g, len(nk) * nq, kv, d)
        s["k"][..., 5] *= 4.0
    else:
        s["q"] = _rand(g, len(nk) * nq, case["heads"], d, std=1.5)
        s["nk"] = torch.tensor(nk, device=dev)
    full = case["kind"] == "attend" or case["read"] == "all"
    make = (lambda: _filled_cache(g, len(nk) * room, kv, d, case["book"], 1.0)) if full else \
        (lambda: _new_cache(len(nk) * room, kv, d, dev))
    s["k4"], s["v4"] = make(), make()
    return s


# ------------------------------------------------------------------------- the plain forms
def _turned(x, cos, sin, rot, pairs):
    """The first rot features of [tokens, heads, d] rotated by angles [tokens, 1, rot / 2]."""
    out = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _plain_rotate(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * torch.tensor(s["freqs"], dtype=torch.float64, device=s["q"].device)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].float()
        n = x
        if w is not None:
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            n = x * rstd
            x = n * w.float()
        out[name] = _turned(x, cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
        if not c["grad"]:
            continue
        g = _turned(s["d" + name].float(), cos, -sin, c["rot"], c["pairs"])
        if w is not None:
            out["d" + name + "w"] = (g * n).sum((0, 1))
            wg = g * w.float()
            g = rstd * (wg - n * (wg * n).mean(-1, keepdim=True))
        out["d" + name] = g.to(torch.bfloat16)
    return out


def _plain_store(s):
    c = s["case"]
    out = {}
    for name in ("k", "v"):
        codes, absmax = s[name + "4"]
        new, top = _encode(s[name], c["book"])
        for q0, nq, k0, nk in s["seqs"]:
            codes[k0 + nk - nq:k0 + nk] = new[q0:q0 + nq]
            absmax[k0 + nk - nq:k0 + nk] = top[q0:q0 + nq]
        rows = torch.cat([torch.arange(k0 + nk - nq, k0 + nk, device=codes.device) for _, nq, k0, nk in
                          (s["whole"] if c["read"] == "all" else s["seqs"])])
        out[name] = _decode(codes[rows], absmax[rows], c["d"], c["book"]).to(torch.bfloat16)
    return out


def _plain_attend(s):
    c = s["case"]
    h, kv, d, nq, room = c["heads"], c["kv"], c["d"], c["nq"], c["room"]
    b, g = len(s["seqs"]), h // kv
    # [batch, kv, room, d] values of the cache
    k, v = (_decode(*s[n], d, c["book"]).reshape(b, room, kv, d).permute(0, 2, 1, 3) for n in ("k4", "v4"))
    key = torch.arange(room, device=k.device)
    last = s["nk"][:, None] - nq + torch.arange(nq, device=k.device)      # a row's own position
    mask = (key < s["nk"][:, None, None]) & (key <= last[:, :, None])
    if c["window"]:
        mask = mask & (key > last[:, :, None] - c["window"])
    q = s["q"].float().reshape(b, nq, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * nq, d)
    z = torch.matmul(q, k.transpose(-1, -2)).reshape(b, kv, g, nq, room) * (1.0 / math.sqrt(d))
    z = z.masked_fill(~mask[:, None, None], NEG)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.reshape(b, kv, g * nq, room), v).reshape(b, kv, g, nq, d).permute(0, 3, 1, 2, 4)
    lse = (top + torch.log(total)).squeeze(-1).permute(1, 2, 0, 3)
    return {"o": o.reshape(b * nq, h, d).to(torch.bfloat16), "lse": lse.reshape(h, b * nq)}


# ------------------------------------------------------------------------- the framework's calls
def _kept(s, name, make):
    """What a program makes once and keeps over its layers and steps."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own_rotate(s):
    import bit_nf4_quantised_amd as nf4
    c, q, k = s["case"], s["q"], s["k"]
    rope = _kept(s, "rope", lambda: nf4.Rope(c["rot"], interleaved=c["pairs"], inv_freq=s["freqs"]))
    out = {"q": torch.empty(q.shape, dtype=q.dtype, device=q.device),
           "k": torch.empty(k.shape, dtype=k.dtype, device=k.device)}
    nf4.qlora_rope_fwd(rope, s["positions"], q, k, out["q"], out["k"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
    if not c["grad"]:
        return out
    out["dq"], out["dk"] = torch.empty_like(out["q"]), torch.empty_like(out["k"])
    if not c["norm"]:
        nf4.qlora_rope_bwd(rope, s["positions"], s["dq"], s["dk"], out["dq"], out["dk"])
        return out
    out["dqw"], out["dkw"] = (torch.empty(c["d"], dtype=torch.float32, device=q.device) for _ in range(2))
    nf4.qlora_rope_bwd(rope, s["positions"], s["dq"], s["dk"], out["dq"], out["dk"], q=q, k=k, q_weight=s["qw"],
                       k_weight=s["kw"], dq_weight=out["dqw"], dk_weight=out["dkw"], eps=EPS)
    return out


def _cache4(s):
    import bit_nf4_quantised_amd as nf4
    c = s["case"]
    return tuple(nf4.Kv4(*s[n], c["d"], c["book"]) for n in ("k4", "v4"))


def _own_store(s):
    import bit_nf4_quantised_amd as nf4
    c, k = s["case"], s["k"]
    k4, v4 = _kept(s, "cache", lambda: _cache4(s))
    new = _kept(s, "new", lambda: nf4.AttnSeqs(s["seqs"]))
    read = _kept(s, "all", lambda: nf4.AttnSeqs(s["whole"])) if c["read"] == "all" else new
    nf4.qlora_kv4_write(new, k, s["v"], k4, v4)
    rows = sum(n for _, n, _, _ in (s["whole"] if c["read"] == "all" else s["seqs"]))
    out = {n: torch.empty(rows, c["kv"], c["d"], dtype=k.dtype, device=k.device) for n in ("k", "v")}
    nf4.qlora_kv4_read(read, k4, v4, out["k"], out["v"])
    return out


def _own_attend(s):
    import bit_nf4_quantised_amd as nf4
    c, q = s["case"], s["q"]
    k4, v4 = _kept(s, "cache", lambda: _cache4(s))
    seqs = _kept(s, "new", lambda: nf4.AttnSeqs(s["seqs"], window=c["window"]))
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
    nf4.qlora_attn_kv4_fwd(seqs, q, k4, v4, o, lse)
    return {"o": o, "lse": lse}


PLAIN = {"rotate": _plain_rotate, "store": _plain_store, "attend": _plain_attend}
OWN = {"rotate": _own_rotate, "store": _own_store, "attend": _own_attend}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["kind"]](state)


# ------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    kv, d = case["kv"], case["d"]
    if case["kind"] == "rotate":
        t, h = sum(_ints(case["lens"])), case["heads"] + kv
        values = t * h * d
        b, f = 4 * values + 8 * t, 3 * t * h * case["rot"] + (4 * values if case["norm"] else 0)
        if case["grad"]:
            b += 4 * values + (8 * d if case["norm"] else 0)    # (x is counted with the forward)
            f += 3 * t * h * case["rot"] + (10 * values if case["norm"] else 0)
        return {"bytes": b + (4 * d if case["norm"] else 0), "flops": f}
    row = 18 * ((d + BLOCK - 1) // BLOCK)       # bytes of one token and head in the cache
    nk, nq = _ints(case["nk"]), case["nq"]
    if case["kind"] == "store":
        new = 2 * len(nk) * nq * kv
        old = 2 * (sum(nk) - len(nk) * nq) * kv if case["read"] == "all" else 0
        return {"bytes": new * (2 * d + row + 2 * d) + old * (row + 2 * d), "flops": 8 * new * d + 2 * (new + old) * d}
    w, h = case["window"], case["heads"]
    seen = keys = 0
    for n in nk:
        for i in range(nq):
            p = n - nq + i
            seen += max(0, p + 1) - (max(0, p - w + 1) if w else 0)
        keys += n - max(0, n - nq - w + 1) if w else n
    return {"bytes": 4 * len(nk) * nq * h * d + 4 * h * len(nk) * nq + 2 * kv * keys * row, "flops": 4 * d * h * seen}


# ------------------------------------------------------------------------- the definitions in 64 bits
def _exact_rotate(s):
    """Every pair as a complex number times exp(i angle); the norm's gradient from its own formula."""
    c, t = s["case"], s["q"].shape[0]
    half = c["rot"] // 2
    rate = torch.tensor(s["freqs"], dtype=torch.float64, device=s["q"].device)
    spin = torch.polar(torch.ones(t, half, dtype=torch.float64, device=rate.device),
                       s["positions"].double().reshape(-1, 1) * rate.reshape(1, -1))[:, None, :]
    i = torch.arange(half, device=rate.device)
    re, im = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)

    def spun(x, by):
        z = torch.complex(x.index_select(-1, re), x.index_select(-1, im)) * by
        y = x.clone()
        y.index_copy_(-1, re, z.real.contiguous())
        y.index_copy_(-1, im, z.imag.contiguous())
        return y
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "w"]
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
        out[n] = spun(x if w is None else x / norm * w.double(), spin)
        if c["grad"]:
            dy = spun(s["d" + n].double(), spin.conj())
            if w is None:
                out["d" + n] = dy
            else:
                out["d" + n + "w"] = torch.einsum("thd,thd->d", dy, x / norm)
                e = dy * w.double()
                out["d" + n] = e / norm - x * ((e * x).sum(-1, keepdim=True) / (c["d"] * norm ** 3))
    return out


def _exact_values(codes, absmax, d, book):
    """float64 values of [rows, kv, blocks, 16] codes: bf16 roundings by the format, as in _decode."""
    at = torch.empty(*codes.shape, 2, dtype=torch.int64, device=codes.device)
    at[..., 0], at[..., 1] = codes // 16, codes % 16
    step = torch.mul(absmax.float(), torch.full((), 1.0 / TOP[book], dtype=torch.float32, device=at.device))
    value = torch.mul(_book(book, codes.device)[0][at.flatten(-2)], step.unsqueeze(-1))
    return value.bfloat16().double().flatten(-2)[..., :d]


def _exact_store(s):
    c = s["case"]
    out = {}
    code = torch.sort(_book(c["book"], s["k"].device)[0].double().unique()).values
    top = TOP[c["book"]]
    for n in ("k", "v"):
        x = torch.nn.functional.pad(s[n].double(), (0, -c["d"] % BLOCK))
        b = x.unflatten(-1, (-1, BLOCK))
        a = b.abs().max(-1, keepdim=True).values
        # the nearest of the sorted codes by distance; argmin would take either of two that tie
        at = torch.searchsorted(code, b * top / torch.where(a > 0, a, torch.ones_like(a))).clamp(1, code.numel() - 1)
        lower, upper = code[at - 1], code[at]
        near = torch.where(b * top - lower * a <= upper * a - b * top, lower, upper)
        step = a.float() * torch.full((), 1.0 / top, dtype=torch.float32, device=a.device)
        new = (near.float() * step).bfloat16().double().flatten(-2)[..., :c["d"]]     # rounded by the format
        if c["read"] == "new":
            out[n] = new
            continue
        parts = []
        for q0, nq, k0, nk in s["seqs"]:
            codes, absmax = s[n + "4"]
            parts += [_exact_values(codes[k0:k0 + nk - nq], absmax[k0:k0 + nk - nq], c["d"], c["book"]), new[q0:q0 + nq]]
        out[n] = torch.cat(parts)
    return out


def _exact_attend(s):
    c = s["case"]
    g = c["heads"] // c["kv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(c["heads"], o.shape[0], dtype=torch.float64, device=o.device)
    for q0, nq, k0, nk in s["seqs"]:
        i = torch.arange(nk - nq, nk, device=o.device)[:, None]
        j = torch.arange(nk, device=o.device)[None, :]
        hidden = j > i
        if c["window"]:
            hidden |= j <= i - c["window"]
        for n in range(c["kv"]):
            k, v = (_exact_values(*(x[k0:k0 + nk, n:n + 1] for x in s[name]), c["d"], c["book"])[:, 0] for name in ("k4", "v4"))
            for h in range(n * g, n * g + g):
                z = (s["q"][q0:q0 + nq, h].double() @ k.t()) / c["d"] ** 0.5
                z[hidden] = NEG
                l = torch.logsumexp(z, 1)
                lse[h, q0:q0 + nq] = l
                o[q0:q0 + nq, h] = torch.exp(z - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None]) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "store": _exact_store, "attend": _exact_attend}[case["kind"]](s)
