"""The 4-bit K/V cache: quantising tokens as they are written, reading them back, decode
attention over the whole cache and over selected tokens of it.

Format (include/sd.h, sd_kv4): per token and KV head, K and V each hold 128 channels as two
groups of 64.  A group stores its minimum m (bf16, exact) and a step s = bf16((max - m) / 15),
and per channel a code c = clamp(rint((x - m) / s), 0, 15); it stands for c s + m.  The 64
code bytes are 16 little-endian 32-bit words; word w holds channels 64 (w % 2) + 8 (w // 2) + i
at bits 4 i.  scale holds [K: s0, m0, s1, m1, V: s0, m0, s1, m1] in bf16.

Cases (kind):
  store   tokens written to the cache (sd_kv4_write) and read back from it (sd_kv4_read)
  read    a range of the cache as bf16 K and V (to build a key index or move a sequence)
  attend  one query token per sequence over its whole cache (layers that are kept dense)
  gather  one query token per sequence over the tokens a top-k selected (the sparse step)
"""
import math

import torch

own = False

D = 128
LARGEST = 1 << 23  # (sequence, KV head, token) triples of the largest cache


def listed():
    return [
        # a decode step of 64 sequences of different lengths: one new token each
        {"name": "store 64x1", "kind": "store", "B": 64, "hkv": 8, "n": 16384, "m": 1,
         "ragged": True},
        # a batch of short prompts of an odd padded length, each with its own length
        {"name": "store 3x1021", "kind": "store", "B": 3, "hkv": 2, "n": 1100, "m": 1021,
         "ragged": True},
        # the prompt of the 128K-token workload's batch written at once
        {"name": "store 4x131072", "kind": "store", "B": 4, "hkv": 8, "n": 131072, "m": 131072,
         "ragged": False},
        # a 32K-token sequence read back to build its key index
        {"name": "read 1x32768", "kind": "read", "B": 1, "hkv": 8, "n": 32768, "m": 32768,
         "ragged": False},
        # ranges of odd length from sequences of different lengths
        {"name": "read 16x4095", "kind": "read", "B": 16, "hkv": 4, "n": 5000, "m": 4095,
         "ragged": True},
        # the smallest decode call: one sequence of one KV head
        {"name": "attend 1x4096 g4", "kind": "attend", "B": 1, "hkv": 1, "G": 4, "n": 4096,
         "ragged": False},
        # one 32K-token sequence, 8 KV heads
        {"name": "attend 1x32768 g4", "kind": "attend", "B": 1, "hkv": 8, "G": 4, "n": 32768,
         "ragged": False},
        # a batch of 64 sequences of 1 to 16,384 tokens
        {"name": "attend 64x16384 g8", "kind": "attend", "B": 64, "hkv": 8, "G": 8, "n": 16384,
         "ragged": True},
        # the 1M-token context
        {"name": "attend 1x1048576 g4", "kind": "attend", "B": 1, "hkv": 8, "G": 4,
         "n": 1 << 20, "ragged": False},
        # the 32K-token workload's selection: 512 tokens and two forced windows
        {"name": "gather 1x1152 g4", "kind": "gather", "B": 1, "hkv": 8, "G": 4, "n": 32768,
         "count": 1152, "block": 1, "ragged": False},
        # 512 single tokens of each 128K-token sequence
        {"name": "gather 4x512 g4", "kind": "gather", "B": 4, "hkv": 8, "G": 4, "n": 131072,
         "count": 512, "block": 1, "ragged": False},
        # 129 blocks of 16 tokens for 64 sequences
        {"name": "gather 64x2064 g4", "kind": "gather", "B": 64, "hkv": 8, "G": 4, "n": 16384,
         "count": 2064, "block": 16, "ragged": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    kind = rng.choice(["store", "read", "attend", "attend", "gather", "gather"])
    B, hkv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
    ragged = rng.random() < 0.5
    most = LARGEST // (B * hkv)
    if kind in ("store", "read"):
        n = _log(rng, 1, min(131072, most // 2))
        m = n if rng.random() < 0.5 else _log(rng, 1, n)
        return {"kind": kind, "B": B, "hkv": hkv, "n": n, "m": m, "ragged": ragged}
    G = rng.choice([1, 2, 4, 8])
    n = _log(rng, 1, min(1 << 20, most))
    c = {"kind": kind, "B": B, "hkv": hkv, "G": G, "n": n, "ragged": ragged}
    if kind == "gather":
        c["block"] = rng.choice([1, 1, 8, 16])
        c["count"] = _log(rng, 1, min(4096, n))
    return c


def _lengths(case, most):
    """Each sequence's (or row's) length: `most`, or spread over [1, most]; the same for
    every seed, so that the work of a case is known."""
    rows = case["B"] * case["hkv"] if case["kind"] == "gather" else case["B"]
    if not case["ragged"]:
        return [most] * rows
    return [1 + int((most - 1) * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(rows)]


def _normal(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen)


def _tokens(case, m, gen):
    """bf16 [B][hkv][m][128] with channels of different spread (0.1 to 4)."""
    lo, hi = math.log(0.1), math.log(4.0)
    sd = torch.exp(torch.rand((case["hkv"], 1, D), device="cuda", generator=gen) * (hi - lo) + lo)
    return (_normal((case["B"], case["hkv"], m, D), gen) * sd).bfloat16()


def _quantise(x):
    """Codes (fp32 whole numbers, [..., 2, 64]), steps and minima ([..., 2, 1]) of bf16 x."""
    g = x.float().unflatten(-1, (2, 64))
    m = g.amin(-1, keepdim=True)
    fifteen = torch.full((), 15.0, device=x.device)
    s = ((g.amax(-1, keepdim=True) - m) / fifteen).bfloat16().float()
    c = ((g - m) / torch.where(s > 0, s, torch.ones_like(s))).round().clamp(0, 15)
    return torch.where(s > 0, c, torch.zeros_like(c)), s, m


def _pack(c):
    """Code bytes [..., 64] of codes [..., 2, 64]."""
    n = c.to(torch.uint8).unflatten(-1, (8, 4, 2)).transpose(-4, -3)  # [..., 8, 2, 4, 2]
    return (n[..., 0] | (n[..., 1] << 4)).flatten(-3)


def _cache(case, gen):
    """A cache of case["n"] tokens, quantised a sequence at a time."""
    B, h, n = case["B"], case["hkv"], case["n"]
    k = torch.empty((B, h, n, 64), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    scale = torch.empty((B, h, n, 8), dtype=torch.bfloat16, device="cuda")
    one = dict(case, B=1)
    for b in range(B):
        for at, codes in ((0, k), (4, v)):
            c, s, m = _quantise(_tokens(one, n, gen)[0])
            codes[b] = _pack(c)
            scale[b, ..., at:at + 4] = torch.cat((s, m), -1).flatten(-2).bfloat16()
    return k, v, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, h, n = case["B"], case["hkv"], case["n"]
    st = {"case": dict(case)}
    if case["kind"] in ("store", "read"):
        m = case["m"]
        lens = _lengths(case, m)
        first = [n - l if case["ragged"] else 0 for l in lens]
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["pos"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        t = torch.arange(m, device="cuda")
        st["valid"] = (t < st["len"][:, None])[:, None, :, None]
        st["at"] = (st["pos"][:, None] + t).clamp(max=n - 1).long()  # [B][m]
        if case["kind"] == "store":
            st["K"], st["V"] = _tokens(case, m, gen), _tokens(case, m, gen)
            st["k"] = torch.zeros((B, h, n, 64), dtype=torch.uint8, device="cuda")
            st["v"] = torch.zeros_like(st["k"])
            st["scale"] = torch.zeros((B, h, n, 8), dtype=torch.bfloat16, device="cuda")
        else:
            st["k"], st["v"], st["scale"] = _cache(case, gen)
        st["Kr"] = torch.zeros((B, h, m, D), dtype=torch.bfloat16, device="cuda")
        st["Vr"] = torch.zeros_like(st["Kr"])
        return st
    st["k"], st["v"], st["scale"] = _cache(case, gen)
    st["q"] = _normal((B, h * case["G"], D), gen).bfloat16()
    st["softmax_scale"] = 1.0 / math.sqrt(D)
    if case["kind"] == "attend":
        st["end"] = torch.tensor(_lengths(case, n), dtype=torch.int32, device="cuda")
        return st
    # ascending token indices, as a top-k gives them: distinct blocks, cut at the count
    blk, count = case["block"], case["count"]
    units = -(-n // blk)
    take = min(units, -(-count // blk) + 1)
    order = torch.rand((B * h, units), device="cuda", generator=gen)
    u = order.topk(take, dim=-1).indices.sort(dim=-1).values
    tok = (u[..., None] * blk + torch.arange(blk, device="cuda")).flatten(-2)
    tok = torch.where(tok < n, tok, n).sort(dim=-1).values  # what lies behind n, last
    have = (tok < n).sum(-1)
    st["idx"] = tok[:, :count].clamp(max=n - 1).int().contiguous()
    lens = torch.tensor(_lengths(case, count), dtype=torch.int64, device="cuda")
    st["count"] = torch.minimum(lens, have).int()
    return st


def _decode(codes, scale):
    """fp32 values [..., 128] of code bytes [..., 64] and scale [..., 4]."""
    c = torch.stack((codes & 15, codes >> 4), -1).unflatten(-2, (8, 2, 4))
    c = c.transpose(-4, -3).flatten(-3).float()  # [..., 2, 64]
    sm = scale.float().unflatten(-1, (2, 2))
    return (c * sm[..., :1] + sm[..., 1:]).flatten(-2)


def _attention(q, K, V, mask, scale, hkv):
    """Softmax attention of q [B][hq][128] over fp32 K, V [B][hkv][n][128]; mask
    [B][hkv][n] of the tokens that count.  A row without tokens gives 0 and -inf."""
    g = q.float().unflatten(1, (hkv, -1))  # [B][hkv][G][128]
    z = (g @ K.transpose(-1, -2)) * scale
    z = z.masked_fill(~mask[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - safe)
    total = p.sum(-1, keepdim=True)
    out = (p @ V) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.log(total) + safe
    return out.flatten(1, 2), lse.flatten(1)


def _run_own(st):
    import top_sparse_decode_gb300 as sd
    c = st["case"]
    if "shape" not in st:  # the handles and buffers that a decode loop keeps
        st["shape"] = sd.make_shape(c["B"], c["hkv"] * c.get("G", 1), c["hkv"], c["n"])
        st["cache"] = sd.Kv4Cache(c["B"], c["hkv"], c["n"], k=st["k"], v=st["v"],
                                  scale=st["scale"])
        if c["kind"] in ("attend", "gather"):
            st["out"] = torch.empty(st["q"].shape, dtype=torch.float32, device="cuda")
            st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
            need = (sd.sd_kv4_attend_workspace_size(st["shape"]) if c["kind"] == "attend" else
                    sd.sd_kv4_gather_attend_workspace_size(st["shape"], c["count"]))
            st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    if c["kind"] in ("store", "read"):
        if c["kind"] == "store":
            sd.sd_kv4_write(st["shape"], st["cache"], st["K"], st["V"], c["m"], pos=st["pos"],
                            length=st["len"])
        sd.sd_kv4_read(st["shape"], st["cache"], st["Kr"], st["Vr"], c["m"], pos=st["pos"],
                       length=st["len"])
        return {"K": st["Kr"], "V": st["Vr"]}
    if c["kind"] == "attend":
        sd.sd_kv4_attend(st["shape"], st["q"], st["cache"], st["softmax_scale"], st["out"],
                         st["lse"], st["ws"], end=st["end"])
    else:
        sd.sd_kv4_gather_attend(st["shape"], st["q"], st["cache"], st["idx"], c["count"],
                                st["count"], c["count"], st["softmax_scale"], st["out"],
                                st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    B, h, n = c["B"], c["hkv"], c["n"]
    if c["kind"] == "store":
        kc, ks, km = _quantise(st["K"])
        vc, vs, vm = _quantise(st["V"])
        K, V = (kc * ks + km).flatten(-2), (vc * vs + vm).flatten(-2)
    elif c["kind"] == "read":
        b = torch.arange(B, device="cuda")[:, None, None]
        i = torch.arange(h, device="cuda")[None, :, None]
        at = st["at"][:, None, :]
        sm = st["scale"][b, i, at]
        K, V = _decode(st["k"][b, i, at], sm[..., :4]), _decode(st["v"][b, i, at], sm[..., 4:])
    if c["kind"] in ("store", "read"):
        return {"K": torch.where(st["valid"], K, st["Kr"].float()).bfloat16(),
                "V": torch.where(st["valid"], V, st["Vr"].float()).bfloat16()}
    if c["kind"] == "attend":
        mask = (torch.arange(n, device="cuda") < st["end"][:, None])[:, None].expand(B, h, n)
        k, v, sm = st["k"], st["v"], st["scale"]
    else:
        idx = st["idx"].long().view(B, h, -1)
        mask = (torch.arange(c["count"], device="cuda") < st["count"][:, None]).view(B, h, -1)
        b = torch.arange(B, device="cuda")[:, None, None]
        i = torch.arange(h, device="cuda")[None, :, None]
        k, v, sm = st["k"][b, i, idx], st["v"][b, i, idx], st["scale"][b, i, idx]
    out, lse = _attention(st["q"], _decode(k, sm[..., :4]), _decode(v, sm[..., 4:]), mask,
                          st["softmax_scale"], h)
    return {"out": out, "lse": lse}


def work(case):
    B, h, rec = case["B"], case["hkv"], 144  # 64 + 64 code bytes, 16 of scales
    if case["kind"] in ("store", "read"):
        rows = sum(_lengths(case, case["m"])) * h
        return {"bytes": rows * (rec + 512) + (rows * 512 if case["kind"] == "store" else 0),
                "flops": rows * 2 * D * (6 if case["kind"] == "store" else 2)}
    G = case["G"]
    if case["kind"] == "attend":
        rows = sum(_lengths(case, case["n"])) * h
        more = 0
    else:
        rows = sum(_lengths(case, case["count"]))
        more = 4 * rows
    return {"bytes": rows * rec + more + B * h * G * (D * 6 + 4), "flops": rows * 4 * G * D}


def _exact_values(codes, scale):
    """Values in 64 bits of [rows][64] code bytes and [rows][4] of scale."""
    words = codes.contiguous().view(torch.int32)
    nib = (words[..., None] >> torch.arange(0, 32, 4, device=codes.device)) & 15
    chan = torch.tensor([64 * (w % 2) + 8 * (w // 2) + i for w in range(16) for i in range(8)],
                        device=codes.device)
    c = torch.empty((codes.shape[0], D), dtype=torch.float64, device=codes.device)
    c[:, chan] = nib.flatten(-2).double()
    s = scale.double()
    return torch.cat((c[:, :64] * s[:, 0:1] + s[:, 1:2], c[:, 64:] * s[:, 2:3] + s[:, 3:4]), -1)


def _exact_stored(x):
    """What the cache holds of bf16 rows x [rows][128], in 64 bits."""
    parts = []
    for g in (x[:, :64].double(), x[:, 64:].double()):
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        s = ((hi - lo) / 15.0).bfloat16().double()
        c = torch.where(s > 0, torch.round((g - lo) / s.clamp(min=1e-300)), 0.0 * g)
        parts.append(c.clamp(0, 15) * s + lo)
    return torch.cat(parts, -1)


def exact(case, seed):
    st = prepare(case, seed)
    B, h, n = case["B"], case["hkv"], case["n"]
    if case["kind"] in ("store", "read"):
        K = torch.zeros((B, h, case["m"], D), dtype=torch.float64, device="cuda")
        V = torch.zeros_like(K)
        lens, pos = st["len"].tolist(), st["pos"].tolist()
        for b in range(B):
            for j in range(h):
                for to, src, codes, at in ((K, st.get("K"), st["k"], 0),
                                           (V, st.get("V"), st["v"], 4)):
                    if case["kind"] == "store":
                        to[b, j, :lens[b]] = _exact_stored(src[b, j, :lens[b]])
                    else:
                        rows = slice(pos[b], pos[b] + lens[b])
                        to[b, j, :lens[b]] = _exact_values(
                            codes[b, j, rows], st["scale"][b, j, rows, at:at + 4])
        return {"K": K, "V": V}
    G = case["G"]
    out = torch.zeros((B, h * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, h * G), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for j in range(h):
            if case["kind"] == "attend":
                rows = slice(0, int(st["end"][b]))
            else:
                rows = st["idx"][b * h + j, :int(st["count"][b * h + j])].long()
            sm = st["scale"][b, j][rows]
            if sm.shape[0] == 0:
                continue
            K = _exact_values(st["k"][b, j][rows], sm[:, :4])
            V = _exact_values(st["v"][b, j][rows], sm[:, 4:])
            heads = slice(j * G, (j + 1) * G)
            z = (st["q"][b, heads].double() @ K.T) * st["softmax_scale"]
            lse[b, heads] = torch.logsumexp(z, -1)
            out[b, heads] = torch.exp(z - lse[b, heads, None]) @ V
    return {"out": out, "lse": lse}
