"""Plain float64 definitions of the serving operators, on the CPU: per-head norm and rotation, the code quantiser and
its page layout, attention of drafted nodes over dense K and V.  Shares no code with the library."""
import math

import torch

F64 = torch.float64


def norm_rope(x, w, eps, pos, theta):
    """x [n, heads, d], w [d] or None, pos [n] or None (no rotation) -> float64."""
    x = x.to(F64)
    d = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    if pos is None:
        return x
    a = pos.to(F64)[:, None, None] * torch.tensor([theta ** (-2.0 * p / d) for p in range(d // 2)], dtype=F64)
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1)


def quantise(x, bits):
    """x [..., 32 m] float64 (first rounded to fp32) -> (scales fp16 [..., m], codes int64 [..., m, 32])."""
    q = 2 ** (bits - 1) - 1
    g = x.to(torch.float32).reshape(*x.shape[:-1], -1, 32)
    s32 = g.abs().amax(-1) * (torch.tensor(1.0) / torch.tensor(float(q)))
    s = s32.to(torch.float16)
    up = (s.view(torch.int16) + 1).view(torch.float16)
    s = torch.where(s.to(torch.float32) < s32, up, s)
    sf = s.to(torch.float32)[..., None]
    c = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g)).clamp(-q, q)
    return s, c.to(torch.int64) + 2 ** (bits - 1)


def dequantise(s, c, bits):
    return ((c - 2 ** (bits - 1)).to(F64) * s.to(F64)[..., None]).flatten(-2)


def token_bytes(s, c, bits):
    """Bytes of every group's codes [..., m, 4 bits] (uint8), LSB first."""
    if bits == 8:
        return c.to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def page_bytes(hkv, d, bits, es):
    if bits == 0:
        return -(-(2 * hkv * 16 * d * es) // 128) * 128
    blk = d // 32 * (32 + 16 * 4 * bits)
    return -(-(2 * hkv * blk) // 128) * 128


def put(pages, page, slot, K, V, bits, dtype):
    """Write tokens K, V [n, hkv, d] (float64) into slots (page[i], slot[i]) of uint8 pages [n_pages, page_bytes]."""
    n, hkv, d = K.shape
    G, per = d // 32, 4 * bits
    if bits == 0:
        es = dtype.itemsize
        k = K.to(torch.float32).to(dtype).contiguous().view(torch.uint8).reshape(n, hkv, d * es)
        v = V.to(torch.float32).to(dtype).contiguous().view(torch.uint8).reshape(n, hkv * d * es)
    else:
        sk, ck = quantise(K, bits)
        sv, cv = quantise(V.reshape(n, -1), bits)
        bk, bv = token_bytes(sk, ck, bits), token_bytes(sv, cv, bits)
        blk = G * (32 + 16 * per)
    for s in range(16):
        at = torch.nonzero(slot == s).flatten()
        if len(at) == 0:
            continue
        pg = page[at].long()
        if bits == 0:
            for h in range(hkv):
                o = (h * 16 + s) * d * es
                pages[pg, o:o + d * es] = k[at, h]
            o = (hkv * 16 * d + s * hkv * d) * es
            pages[pg, o:o + hkv * d * es] = v[at]
            continue

        def group(base, n_groups, g, sc, by):
            o = base + (g * 16 + s) * 2
            pages[pg, o:o + 2] = sc.contiguous().view(torch.uint8).reshape(-1, 2)
            o = base + n_groups * 32 + (g * 16 + s) * per
            pages[pg, o:o + per] = by

        for h in range(hkv):
            for g in range(G):
                group(h * blk, G, g, sk[at, h, g], bk[at, h, g])
        for g in range(hkv * G):
            group(hkv * blk, hkv * G, g, sv[at, g], bv[at, g])


def stored(x, bits, dtype):
    """The values that the cache holds for rows x [..., d] (float64)."""
    if bits == 0:
        return x.to(torch.float32).to(dtype).to(F64)
    s, c = quantise(x, bits)
    return dequantise(s, c, bits)


def attention(q, K, V, see, scale):
    """q [n, H, d], K / V [T, hkv, d], see [n, T] bool -> [n, H * d]; a row that sees nothing is zero."""
    n, H, d = q.shape
    hkv = K.shape[1]
    qg = q.view(n, hkv, H // hkv, d)
    s = torch.einsum("nghd,tgd->nght", qg, K) * scale
    s = s.masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(see[:, None, None].expand_as(s), torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m)),
                    torch.zeros_like(s))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, torch.zeros_like(p))
    return torch.einsum("nght,tgd->nghd", p, V).reshape(n, H * d)


def random_tree(rng, n):
    """Ancestor sets (with the node itself) of a random tree of n nodes, and the nodes' depths."""
    sees, depth = [], []
    for i in range(n):
        p = rng.randrange(-1, i) if i else -1
        sees.append({i} | (sees[p] if p >= 0 else set()))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return sees, depth


def mask_words(sees, words):
    rows = []
    for s in sees:
        v = sum(1 << j for j in s)
        w = [(v >> (32 * k)) & 0xFFFFFFFF for k in range(words)]
        rows.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
    return torch.tensor(rows, dtype=torch.int32).reshape(len(sees), words)
