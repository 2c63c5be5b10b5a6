"""What runs around the sparse decode step: queries and keys normed and rotated on their way
into the bf16 cache, attention of a sliding window with a few first tokens (prompts, chunks
and single tokens), and decode attention of a batch over a prefix that its sequences share.

The caches are bf16 [B][hkv][n][128] (include/sd.h).  Cases (kind):
  rope    m new tokens per sequence: x -> x / sqrt(mean(x^2) + eps) * weight for each query
          and key head, its first `rot` channels rotated by position * inv_freq (channel j
          with j + rot / 2, or 2j with 2j + 1 where `pairs`); keys and values go to their
          positions of the cache (sd_qk_norm_rope)
  window  query token t of a sequence stands at p = pos + t and sees the cached tokens
          i <= p with i < sink or i > p - window (sd_window_attend)
  prefix  one query token per sequence over p shared tokens and its own (sd_prefix_attend)
Softmax attention, scale 1 / sqrt(128); out bf16, lse the log of the sum of exponentials.
"""
import math

import numpy as np
import torch

own = False

D = 128
EPS = 1e-6
BASE = 500000.0
BLOCK = 512  # query tokens that the plain window form takes at a time, at most
SCORES = 1 << 31  # ... and scores
MOST_FLOPS = 2.2e12  # of the largest window case


def listed():
    return [
        # a decode step's new tokens of 64 sequences at far positions
        {"name": "rope 64x1", "kind": "rope", "B": 64, "hkv": 8, "G": 4, "n": 4096, "m": 1,
         "rot": 128, "pairs": False, "far": 1 << 20, "ragged": True},
        # short prompts of an odd padded length, each with its own length, half rotated
        {"name": "rope 3x1021", "kind": "rope", "B": 3, "hkv": 2, "G": 4, "n": 1100, "m": 1021,
         "rot": 64, "pairs": True, "far": 0, "ragged": True},
        # the prompts of a batch of 32K-token sequences written at once
        {"name": "rope 4x32768", "kind": "rope", "B": 4, "hkv": 8, "G": 4, "n": 32768,
         "m": 32768, "rot": 128, "pairs": False, "far": 0, "ragged": False},
        # the smallest decode call: one sequence, a 1,024-token window and 128 first tokens
        {"name": "window 1x1", "kind": "window", "B": 1, "hkv": 8, "G": 4, "n": 32768, "m": 1,
         "window": 1024, "sink": 128, "ragged": False},
        # a decode step of 64 sequences of up to 16,384 tokens, 4,096-token window
        {"name": "window 64x1", "kind": "window", "B": 64, "hkv": 8, "G": 4, "n": 16384, "m": 1,
         "window": 4096, "sink": 128, "ragged": True},
        # chunks of an odd length in the midst of three sequences, odd window
        {"name": "window 3x257", "kind": "window", "B": 3, "hkv": 2, "G": 8, "n": 5003, "m": 257,
         "window": 501, "sink": 3, "ragged": True},
        # prompts under plain causal attention (the window holds all)
        {"name": "window 4x4096 all", "kind": "window", "B": 4, "hkv": 8, "G": 4, "n": 4096,
         "m": 4096, "window": 4096, "sink": 0, "ragged": False},
        # a 32K-token prompt with a 4,096-token window
        {"name": "window 1x32768", "kind": "window", "B": 1, "hkv": 8, "G": 4, "n": 32768,
         "m": 32768, "window": 4096, "sink": 128, "ragged": False},
        # two sequences that share a short prompt
        {"name": "prefix 2x1024", "kind": "prefix", "B": 2, "hkv": 8, "G": 4, "p": 1024, "n": 64,
         "ragged": False},
        # odd sizes: 17 answers over one document
        {"name": "prefix 17x5003", "kind": "prefix", "B": 17, "hkv": 4, "G": 8, "p": 5003,
         "n": 333, "ragged": True},
        # 64 answers of up to 1,024 tokens over one 32K-token document
        {"name": "prefix 64x32768", "kind": "prefix", "B": 64, "hkv": 8, "G": 4, "p": 32768,
         "n": 1024, "ragged": True},
        # 128 requests over a 128K-token document
        {"name": "prefix 128x131072", "kind": "prefix", "B": 128, "hkv": 8, "G": 4, "p": 131072,
         "n": 512, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    kind = rng.choice(["rope", "window", "window", "prefix"])
    hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    ragged = rng.random() < 0.5
    if kind == "rope":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, min(32768, (1 << 22) // (B * hkv * (G + 2))))
        m = rng.choice([1, n, _log(rng, 1, n)])
        return {"kind": kind, "B": B, "hkv": hkv, "G": G, "n": n, "m": m,
                "rot": rng.choice([32, 64, 128, 128]), "pairs": rng.random() < 0.5,
                "far": rng.choice([0, 1 << 20]), "ragged": ragged}
    if kind == "prefix":
        B = _log(rng, 1, 128)
        return {"kind": kind, "B": B, "hkv": hkv, "G": G,
                "p": _log(rng, 1, min(131072, (1 << 26) // (B * G))), "n": _log(rng, 1, 1024),
                "ragged": ragged}
    B = _log(rng, 1, 64)
    n = _log(rng, 1, min(32768, (1 << 23) // (B * hkv)))
    m = 1 if rng.random() < 0.4 else _log(rng, 1, n)
    c = {"kind": kind, "B": B, "hkv": hkv, "G": G, "n": n, "m": m,
         "window": n if rng.random() < 0.25 else _log(rng, 1, 8192),
         "sink": rng.choice([0, 1, 4, 128]), "ragged": ragged}
    while work(c)["flops"] > MOST_FLOPS:
        c["m"] = max(1, c["m"] // 2)
    return c


def _lengths(case, most):
    """Each sequence's length: `most`, or spread over [1, most]; the same for every seed, so
    that the work of a case is known."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    return [1 + int((most - 1) * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(B)]


def _first(case):
    """Position of each sequence's first query token: its chunk ends with what it holds (for
    a single token, its own length)."""
    if case["m"] == 1:
        return [l - 1 for l in _lengths(case, case["n"])]
    return [case["n"] - l for l in _lengths(case, case["m"])]


def _queries(case):
    return [1] * case["B"] if case["m"] == 1 else _lengths(case, case["m"])


def _normal(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen)


def _tokens(B, hkv, m, gen):
    """bf16 [B][hkv][m][128] with channels of different spread (0.25 to 2)."""
    sd = torch.exp2(torch.rand((hkv, 1, D), device="cuda", generator=gen) * 3 - 2)
    x = torch.empty((B, hkv, m, D), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        x[b] = (_normal((hkv, m, D), gen) * sd).bfloat16()
    return x


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, h, G, n = case["B"], case["hkv"], case["G"], case["n"]
    st = {"case": dict(case), "softmax_scale": 1.0 / math.sqrt(D)}
    if case["kind"] == "rope":
        m, heads = case["m"], h * (G + 2)
        # what the projection of m tokens gives: [B][m][hq + 2 hkv][128]
        st["qkv"] = torch.empty((B, m, heads, D), dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            st["qkv"][b] = (_normal((m, heads, D), gen) * 2.0).bfloat16()
        st["q_weight"] = 1.0 + 0.2 * _normal((D,), gen)
        st["k_weight"] = 1.0 + 0.2 * _normal((D,), gen)
        j = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        st["inv_freq"] = BASE ** (-2.0 * j / case["rot"])
        st["pos"] = _int32(_first(case))
        st["len"] = _int32(_queries(case))
        # positions are those of the cache; for far ones the cache is a piece of a longer one
        st["rotary"] = st["pos"] + case["far"]
        st["q"] = torch.zeros((B, m, h * G, D), dtype=torch.bfloat16, device="cuda")
        st["K"] = torch.zeros((B, h, n, D), dtype=torch.bfloat16, device="cuda")
        st["V"] = torch.zeros_like(st["K"])
        return st
    if case["kind"] == "prefix":
        st["q"] = _normal((B, h * G, D), gen).bfloat16()
        st["Kp"], st["Vp"] = _tokens(1, h, case["p"], gen)[0], _tokens(1, h, case["p"], gen)[0]
        st["K"], st["V"] = _tokens(B, h, n, gen), _tokens(B, h, n, gen)
        st["end"] = _int32(_lengths(case, n))
        return st
    m = case["m"]
    st["q"] = _normal((B, m, h * G, D), gen).bfloat16()
    st["K"], st["V"] = _tokens(B, h, n, gen), _tokens(B, h, n, gen)
    st["pos"] = _int32(_first(case))
    st["len"] = _int32(_queries(case))
    st["out"] = torch.zeros((B, m, h * G, D), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros((B, h * G, m), dtype=torch.float32, device="cuda")
    return st


def _run_own(st):
    import top_sparse_decode_gb300 as sd
    c = st["case"]
    B, h, G, n = c["B"], c["hkv"], c["G"], c["n"]
    if "shape" not in st:  # the handles and buffers that a decode loop keeps
        st["shape"] = sd.make_shape(B, h * G, h, n)
        if c["kind"] == "rope":
            st["rope"] = sd.make_rope(st["inv_freq"], q_weight=st["q_weight"],
                                      k_weight=st["k_weight"], eps=EPS, pairs=c["pairs"])
        elif c["kind"] == "window":
            need = sd.sd_window_attend_workspace_size(st["shape"], c["m"], c["window"], c["sink"])
            st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        else:
            need = sd.sd_prefix_attend_workspace_size(st["shape"], c["p"])
            st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
            st["out"] = torch.empty((B, h * G, D), dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty((B, h * G), dtype=torch.float32, device="cuda")
    if c["kind"] == "rope":
        q, k, v = st["qkv"].transpose(1, 2).split([h * G, h, h], dim=1)
        sd.sd_qk_norm_rope(st["shape"], st["rope"], q, st["q"].transpose(1, 2), k, v, st["K"],
                           st["V"], c["m"], pos=st["pos"], length=st["len"],
                           rotary=st["rotary"])
        return {"q": st["q"], "K": st["K"], "V": st["V"]}
    if c["kind"] == "window":
        sd.sd_window_attend(st["shape"], st["q"].transpose(1, 2), st["K"], st["V"], c["m"],
                            c["window"], c["sink"], st["softmax_scale"],
                            st["out"].transpose(1, 2), st["lse"], st["ws"], pos=st["pos"],
                            length=st["len"])
    else:
        sd.sd_prefix_attend(st["shape"], st["q"], st["Kp"], st["Vp"], c["p"], st["K"], st["V"],
                            st["softmax_scale"], st["out"], st["lse"], st["ws"], end=st["end"])
    return {"out": st["out"], "lse": st["lse"]}


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _rotate(x, cos, sin, pairs):
    """x [B][m][heads][128]; cos, sin [B][m][1][rot / 2]."""
    rot = 2 * cos.shape[-1]
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _rope(st):
    c = st["case"]
    B, h, G, m = c["B"], c["hkv"], c["G"], c["m"]
    t = torch.arange(m, device="cuda")
    valid = t < st["len"][:, None]  # [B][m]
    ang = (st["rotary"][:, None] + t).double()[..., None] * st["inv_freq"]
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    q, k, v = st["qkv"].split([h * G, h, h], dim=2)
    q = _rotate(_norm(q.float(), st["q_weight"]), cos, sin, c["pairs"]).bfloat16()
    k = _rotate(_norm(k.float(), st["k_weight"]), cos, sin, c["pairs"]).bfloat16()
    st["q"].copy_(torch.where(valid[:, :, None, None], q, st["q"]))
    b, i = valid.nonzero(as_tuple=True)
    at = st["pos"].long()[b] + i
    st["K"][b, :, at] = k[b, i]
    st["V"][b, :, at] = v[b, i]
    return {"q": st["q"], "K": st["K"], "V": st["V"]}


def _softmax_parts(z):
    """exp(z - max), its sum and the max (0 in a row that is all -inf)."""
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    return p, p.sum(-1, keepdim=True), top


def _window(st):
    """The window attention, a block of query tokens of every sequence at a time, over the
    keys that the block sees."""
    c = st["case"]
    B, h, G, n, m = c["B"], c["hkv"], c["G"], c["n"], c["m"]
    w, s = min(c["window"], n), min(c["sink"], n)
    b = torch.arange(B, device="cuda")[:, None]
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    block = max(1, min(BLOCK, SCORES // (B * h * G * (w + s))))
    for t0 in range(0, m, block):
        t1 = min(m, t0 + block)
        p = st["pos"].long()[:, None] + torch.arange(t0, t1, device="cuda")  # [B][t]
        near = p[:, :1] - (w - 1) + torch.arange(w + t1 - t0 - 1, device="cuda")
        key = torch.cat((torch.arange(s, device="cuda").expand(B, s), near), 1)  # [B][keys]
        last = torch.arange(key.shape[1], device="cuda") >= s  # the window's part
        old = key[:, None] <= p[..., None] - c["window"]
        see = (key >= 0)[:, None] & (key < n)[:, None] & (key[:, None] <= p[..., None])
        see = see & (old ^ last)  # a first token inside the window counts once
        at = key.clamp(0, n - 1)
        K, V = st["K"][b, :, at].float(), st["V"][b, :, at].float()  # [B][keys][h][128]
        q = st["q"][:, t0:t1].float().unflatten(2, (h, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
        z = (q @ K.permute(0, 2, 3, 1)) * st["softmax_scale"]  # [B][h][G t][keys]
        z = z.unflatten(2, (G, t1 - t0)).masked_fill(~see[:, None, None], -math.inf)
        e, total, top = _softmax_parts(z)
        o = e.flatten(2, 3) @ V.permute(0, 2, 1, 3)
        o = o.unflatten(2, (G, t1 - t0)) / torch.where(total > 0, total, torch.ones_like(total))
        out[:, t0:t1] = o.permute(0, 3, 1, 2, 4).flatten(2, 3).bfloat16()
        lse[..., t0:t1] = (torch.log(total) + top)[..., 0].flatten(1, 2)
    valid = torch.arange(m, device="cuda") < st["len"][:, None]
    return {"out": torch.where(valid[:, :, None, None], out, st["out"]),
            "lse": torch.where(valid[:, None], lse, st["lse"])}


def _prefix(st):
    c = st["case"]
    B, h, G = c["B"], c["hkv"], c["G"]
    q = st["q"].float().unflatten(1, (h, G))  # [B][h][G][128]
    qs = q.transpose(0, 1).flatten(1, 2)  # [h][B G][128]
    zp = (qs @ st["Kp"].float().transpose(-1, -2)) * st["softmax_scale"]
    zo = (q @ st["K"].float().transpose(-1, -2)) * st["softmax_scale"]
    have = torch.arange(c["n"], device="cuda") < st["end"][:, None]
    zo = zo.masked_fill(~have[:, None, None], -math.inf)
    z = torch.cat((zp.unflatten(1, (B, G)).transpose(0, 1), zo), -1)
    e, total, top = _softmax_parts(z)
    op = e[..., :c["p"]].transpose(0, 1).flatten(1, 2) @ st["Vp"].float()
    o = op.unflatten(1, (B, G)).transpose(0, 1) + e[..., c["p"]:] @ st["V"].float()
    return {"out": (o / total).flatten(1, 2).bfloat16(),
            "lse": (torch.log(total) + top)[..., 0].flatten(1, 2)}


def run(st):
    if own:
        return _run_own(st)
    return {"rope": _rope, "window": _window, "prefix": _prefix}[st["case"]["kind"]](st)


def _seen(case):
    """(tokens that any query of each sequence sees, summed; (query, token) pairs, summed)."""
    n, w, s = case["n"], case["window"], case["sink"]
    tokens = pairs = 0
    for first, l in zip(_first(case), _queries(case)):
        p = np.arange(first, first + l, dtype=np.int64)
        hi = np.minimum(p + 1, n)
        lo = np.maximum(p - w + 1, 0)
        pairs += int((np.maximum(hi - lo, 0) + np.minimum(lo, s)).sum())
        tokens += int(hi[-1] - lo[0]) + min(int(lo[0]), s)
    return tokens, pairs


def work(case):
    B, h, G = case["B"], case["hkv"], case["G"]
    if case["kind"] == "rope":
        tokens = sum(_queries(case))
        return {"bytes": tokens * h * (G + 2) * 2 * 2 * D + 2 * 4 * D + 4 * case["rot"],
                "flops": tokens * h * (G + 1) * (4 * D + 3 * case["rot"])}
    if case["kind"] == "prefix":
        owned = sum(_lengths(case, case["n"]))
        return {"bytes": (case["p"] + owned) * h * 4 * D + B * h * G * (4 * D + 4),
                "flops": 4 * D * h * G * (B * case["p"] + owned)}
    tokens, pairs = _seen(case)
    return {"bytes": tokens * h * 4 * D + sum(_queries(case)) * h * G * (4 * D + 4),
            "flops": 4 * D * h * G * pairs}


def _exact_attention(q, K, V, see, scale):
    """out, lse in 64 bits of q [rows][128] over K, V [keys][128]; see [rows][keys] or None."""
    z = (q @ K.T) * scale
    if see is not None:
        z = torch.where(see, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, -1)
    safe = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    return torch.exp(z - safe[:, None]) @ V, lse


def _exact_rope(st, c):
    B, h, G, m, rot = c["B"], c["hkv"], c["G"], c["m"], c["rot"]
    q = torch.zeros((B, m, h * G, D), dtype=torch.float64, device="cuda")
    K = torch.zeros((B, h, c["n"], D), dtype=torch.float64, device="cuda")
    V = torch.zeros_like(K)
    half = rot // 2
    one = [2 * j if c["pairs"] else j for j in range(half)]
    two = [2 * j + 1 if c["pairs"] else j + half for j in range(half)]
    for b, (pos, far, l) in enumerate(zip(st["pos"].tolist(), st["rotary"].tolist(),
                                          st["len"].tolist())):
        where = torch.arange(far, far + l, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones((l, half), dtype=torch.float64, device="cuda"),
                           where[:, None] * st["inv_freq"])
        for head in range(h * (G + 1)):
            x = st["qkv"][b, :l, head].double()
            weight = st["q_weight"] if head < h * G else st["k_weight"]
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * weight.double()
            z = torch.complex(x[:, one], x[:, two]) * turn
            x[:, one], x[:, two] = z.real, z.imag
            if head < h * G:
                q[b, :l, head] = x
            else:
                K[b, head - h * G, pos:pos + l] = x
        V[b, :, pos:pos + l] = st["qkv"][b, :l, h * (G + 1):].transpose(0, 1).double()
    return {"q": q, "K": K, "V": V}


def exact(case, seed):
    st = prepare(case, seed)
    B, h, G, n = case["B"], case["hkv"], case["G"], case["n"]
    scale = st["softmax_scale"]
    if case["kind"] == "rope":
        return _exact_rope(st, case)
    if case["kind"] == "prefix":
        out = torch.empty((B, h * G, D), dtype=torch.float64, device="cuda")
        lse = torch.empty((B, h * G), dtype=torch.float64, device="cuda")
        for j in range(h):
            heads = slice(j * G, (j + 1) * G)
            q = st["q"][:, heads].double()
            po, pl = _exact_attention(q.flatten(0, 1), st["Kp"][j].double(), st["Vp"][j].double(),
                                      None, scale)
            for b, e in enumerate(st["end"].tolist()):
                oo, ol = _exact_attention(q[b], st["K"][b, j, :e].double(),
                                          st["V"][b, j, :e].double(), None, scale)
                a, o = pl[b * G:(b + 1) * G], po[b * G:(b + 1) * G]
                lse[b, heads] = torch.logaddexp(a, ol)
                out[b, heads] = (o * torch.exp(a - lse[b, heads])[:, None]
                                 + oo * torch.exp(ol - lse[b, heads])[:, None])
        return {"out": out, "lse": lse}
    m = case["m"]
    out = torch.zeros((B, m, h * G, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, h * G, m), dtype=torch.float64, device="cuda")
    for b, (pos, l) in enumerate(zip(_first(case), _queries(case))):
        for j in range(h):
            K, V = st["K"][b, j].double(), st["V"][b, j].double()
            for t0 in range(0, l, 1024):
                t1 = min(l, t0 + 1024)
                lo = max(0, pos + t0 - case["window"] + 1)
                key = torch.arange(n, device="cuda")
                key = key[(key < case["sink"]) | ((key >= lo) & (key < pos + t1))]
                p = torch.arange(pos + t0, pos + t1, device="cuda")[:, None]
                see = (key <= p) & ((key < case["sink"]) | (p - key < case["window"]))
                for g in range(j * G, (j + 1) * G):
                    o, e = _exact_attention(st["q"][b, t0:t1, g].double(), K[key], V[key], see,
                                            scale)
                    out[b, t0:t1, g], lse[b, g, t0:t1] = o, e
    return {"out": out, "lse": lse}
