"""Plain implementation of the 4-bit K/V cache (include/sd.h, sd_kv4) in numpy, for its
tests: the format in fp32 exactly as the header defines it, attention in 64 bits, and
worst-case bounds for an fp32 attention over the same cache.

Bounds (u = 2^-24, a rounding to nearest fp32; a tensor-core or other accumulation may
truncate, so an addition counts 2 u):
  z: <q, k> has 128 code products in two groups, two scale products and two minima: at
     most 140 roundings or truncations of terms whose magnitudes sum to
     zmass = scale sum_j |q_j| (c_j s + |m|); |dz| <= 280 u zmass.
  e^(z - max): relative error e^(2 |dz|max) - 1 for the two arguments, and 2^-20 for the
     exponential, the split of p into two 11-bit parts and the scales (each < 2^-21.5).
  sums over `count` tokens: at most count / 8 + 64 additions in a chain, 2 u each.
  out: these over vmass = sum_i p_i (c s + |m|) (normalised p), twice: numerator and l.
"""
import numpy as np

U = 2.0 ** -24


def bf16_bits(x):
    """fp32 -> bf16 bits, nearest even (NaN -> 0x7FC0)."""
    x = np.asarray(x, np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_val(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantise(xb):
    """Codes uint8 [..., 2, 64], step and minimum (fp32 [..., 2]) of bf16 bits [..., 128]."""
    x = bf16_val(xb).reshape(*xb.shape[:-1], 2, 64)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        s = bf16_val(bf16_bits((hi - lo) / np.float32(15)))
        bad = ~np.isfinite(s) | ~np.isfinite(x).all(-1)
        s = np.where(s < np.float32(2.0 ** -100), np.float32(0), s)
        q = np.rint((x - lo[..., None]) / np.where(s > 0, s, np.float32(1))[..., None])
        c = np.where((s > 0)[..., None] & ~bad[..., None], np.clip(q, 0, 15), 0).astype(np.uint8)
    nan = np.float32(np.nan)
    return c, np.where(bad, nan, s).astype(np.float32), np.where(bad, nan, lo).astype(np.float32)


def pack(c):
    """Code bytes [..., 64] of codes [..., 2, 64]: word 2 o + g holds octet o of group g."""
    o = c.reshape(*c.shape[:-1], 8, 8)                       # [..., g, octet, i]
    o = np.swapaxes(o, -3, -2).reshape(*c.shape[:-2], 16, 4, 2)
    return (o[..., 0] | (o[..., 1] << 4)).reshape(*c.shape[:-2], 64).astype(np.uint8)


def unpack(b):
    o = np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], 8, 2, 8)
    return np.swapaxes(o, -3, -2).reshape(*b.shape[:-1], 2, 64)


def encode(Kb, Vb):
    """(k, v, scale bits) of bf16 bits [..., 128]."""
    out = []
    rec = np.empty((*Kb.shape[:-1], 8), np.uint16)
    for at, x in ((0, Kb), (4, Vb)):
        c, s, m = quantise(x)
        out.append(pack(c))
        rec[..., at:at + 4:2] = bf16_bits(s)
        rec[..., at + 1:at + 4:2] = bf16_bits(m)
    return out[0], out[1], rec


def parts(codes, rec):
    """(c s, m) in 64 bits, each [..., 128], of code bytes and a record half [..., 4]."""
    c = unpack(codes).astype(np.float64)
    s = bf16_val(rec[..., 0::2]).astype(np.float64)[..., None]
    m = np.broadcast_to(bf16_val(rec[..., 1::2]).astype(np.float64)[..., None], c.shape)
    shape = (*codes.shape[:-1], 128)
    with np.errstate(invalid="ignore"):
        return (c * s).reshape(shape), m.reshape(shape)


def read(codes, rec):
    """bf16 bits that sd_kv4_read gives."""
    cs, m = parts(codes, rec)
    return bf16_bits((cs + m).astype(np.float32))


def attend_row(qb, k, v, rec, tok, scale):
    """One KV head: q bits [G][128], cache rows k, v [n][64], rec [n][8]; tokens tok.
    Returns out, lse (64 bits) and their bounds."""
    G = qb.shape[0]
    if len(tok) == 0:
        return (np.zeros((G, 128)), np.full(G, -np.inf), np.zeros((G, 128)), np.zeros(G))
    q = bf16_val(qb).astype(np.float64)
    kc, km = parts(k[tok], rec[tok, :4])
    vc, vm = parts(v[tok], rec[tok, 4:])
    scale = float(np.float32(scale))
    with np.errstate(all="ignore"):
        z = q @ (kc + km).T * scale
        zmass = np.abs(q) @ (kc + np.abs(km)).T * abs(scale)
        top = z.max(-1, keepdims=True)
        p = np.exp(z - top)
        l = p.sum(-1, keepdims=True)
        p = p / l
        out = p @ (vc + vm)
        lse = (top + np.log(l))[:, 0]
        vmass = p @ (vc + np.abs(vm))
        dz = 280 * U * zmass.max(-1)
        rel = np.expm1(2 * dz) + 2.0 ** -20 + 2 * U * (len(tok) / 8 + 64)
        return out, lse, 2 * rel[:, None] * vmass, rel + 4 * U * np.abs(lse)


def attend(qb, k, v, rec, toks, scale):
    """All rows: qb [B][hq][128], cache [B][hkv][ncap][..]; toks[b * hkv + h] indices."""
    B, hq = qb.shape[:2]
    hkv = k.shape[1]
    G = hq // hkv
    res = [np.zeros((B, hq, 128)), np.zeros((B, hq)), np.zeros((B, hq, 128)), np.zeros((B, hq))]
    for b in range(B):
        for h in range(hkv):
            r = attend_row(qb[b, h * G:(h + 1) * G], k[b, h], v[b, h], rec[b, h],
                           np.asarray(toks[b * hkv + h], np.int64), scale)
            for to, x in zip(res, r):
                to[b, h * G:(h + 1) * G] = x
    return res


def check(out, lse, ref):
    ro, rl, bo, bl = ref
    nan = np.isnan(ro)
    assert np.array_equal(np.isnan(out), nan)
    over = np.abs(out - ro)[~nan] - bo[~nan]
    assert over.size == 0 or over.max() <= 0, (over.max(), np.abs(out - ro)[~nan].max())
    if lse is not None:
        assert np.array_equal(np.isnan(lse), np.isnan(rl))
        fin = np.isfinite(rl)
        assert np.array_equal(lse[~fin & ~np.isnan(rl)], rl[~fin & ~np.isnan(rl)])
        assert np.all(np.abs(lse[fin] - rl[fin]) <= bl[fin])


def tokens(rng, shape, spread=True):
    """bf16 bits of normal values whose channels have spreads of 0.1 to 4."""
    x = rng.standard_normal((*shape, 128))
    if spread:
        x = x * np.exp(rng.uniform(np.log(0.1), np.log(4.0), 128))
    return bf16_bits(x.astype(np.float32))
