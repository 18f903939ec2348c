"""The operators of speculative serving over the paged cache, as cases that can be timed and compared.

Five operators of an uncompressed layer (K after RoPE and V in 16-token pages, in the layer's type or as 8 / 4-bit
codes with an fp16 scale per 32 channels):

  norm_rope   per-head RMS norm of queries and keys and their rotation, from the rows of a fused QKV projection
  append      the same, with the keys and values quantised into the cache's pages
  read        cached tokens back as dense rows
  tree        attention of drafted tokens (a tree, a chain, or one token) over the cache, out through W_o
  accept      the accepted path of a tree moved to the front of its slots, the other drafts' slots cleared

`run` computes them in elementary torch operations, or with the library's own entry points where `own` is true.
"""
import math
import random

import torch

own = False

PAGE = 16
D = 4096          # hidden size of the layers of this repository's workloads
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's projections: 16 sequences, the GQA layer (32 query heads, 8 KV heads)
        dict(name="norm_rope_decode", op="norm_rope", n=16, H=32, Hkv=8, dtype="bf16", theta=500000.0, norm=True,
             max_pos=8192),
        # a whole prompt's projections on the 32-head layer
        dict(name="norm_rope_prefill", op="norm_rope", n=4096, H=32, Hkv=32, dtype="bf16", theta=10000.0, norm=True,
             max_pos=32768),
        # 16 sequences' trees of 16 drafts written for verification, 8-bit cache, 32 heads
        dict(name="append_verify_q8", op="append", batch=16, n=16, hist=4001, H=32, Hkv=32, bits=8, dtype="bf16",
             theta=10000.0, norm=True),
        # a long prompt written into the 4-bit cache of the GQA layer
        dict(name="append_prefill_q4", op="append", batch=3, n=2731, hist=0, H=32, Hkv=8, bits=4, dtype="bf16",
             theta=500000.0, norm=True),
        # one short prefix read back (8-bit, 32 heads)
        dict(name="read_prefix_q8", op="read", batch=1, n=301, H=32, Hkv=32, bits=8, dtype="bf16"),
        # the prefixes of a batch read back (4-bit, GQA)
        dict(name="read_batch_q4", op="read", batch=16, n=2048, H=32, Hkv=8, bits=4, dtype="bf16"),
        # a single user's small tree over a short bf16 cache: latency
        dict(name="tree_small_bf16", op="tree", batch=1, n=7, hist=333, H=32, Hkv=32, bits=0, raw=True, norm=False,
             theta=10000.0, mask="tree"),
        # one token for each of 16 sequences over the 8-bit cache (plain decode)
        dict(name="decode_q8", op="tree", batch=16, n=1, hist=4095, H=32, Hkv=32, bits=8, raw=True, norm=True,
             theta=10000.0, mask="chain"),
        # trees of 16 drafts for 16 sequences, 8-bit cache, 32 heads
        dict(name="tree_q8", op="tree", batch=16, n=16, hist=4001, H=32, Hkv=32, bits=8, raw=False, norm=True,
             theta=10000.0, mask="tree"),
        # trees of 24 drafts for 64 sequences at 8K context, 4-bit cache of the GQA layer
        dict(name="tree_q4_gqa", op="tree", batch=64, n=24, hist=8101, H=32, Hkv=8, bits=4, raw=False, norm=True,
             theta=500000.0, mask="tree"),
        # a single user's accepted path
        dict(name="accept_small_q8", op="accept", batch=1, n=7, hist=333, H=32, Hkv=32, bits=8),
        # a large batch's accepted paths
        dict(name="accept_batch_q8", op="accept", batch=64, n=64, hist=501, H=32, Hkv=32, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read", "tree", "tree", "accept"])
    H, Hkv = rng.choice([(32, 32), (32, 8), (16, 16), (8, 2), (32, 4)])
    theta = rng.choice([10000.0, 500000.0])
    if op == "norm_rope":
        return dict(op=op, n=_log_int(rng, 1, 4096), H=H, Hkv=Hkv, dtype=rng.choice(["bf16", "f32"]), theta=theta,
                    norm=rng.random() < 0.7, max_pos=_log_int(rng, 64, 131072))
    if op == "append":
        b = rng.randint(1, 16)
        return dict(op=op, batch=b, n=_log_int(rng, 1, 8192 // b), hist=_log_int(rng, 1, 9000) - 1, H=H, Hkv=Hkv,
                    bits=rng.choice([0, 4, 8]), dtype=rng.choice(["bf16", "f32"]), theta=theta,
                    norm=rng.random() < 0.7)
    if op == "read":
        b = rng.randint(1, 16)
        return dict(op=op, batch=b, n=_log_int(rng, 1, 2048), H=H, Hkv=Hkv, bits=rng.choice([0, 4, 8]),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "tree":
        b = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, 64)
        n = min(n, max(1, 1536 // b))
        hist = min(_log_int(rng, 1, 16384) - 1, 4000000 // (b * Hkv))
        return dict(op=op, batch=b, n=n, hist=hist, H=H, Hkv=Hkv, bits=rng.choice([0, 4, 8]),
                    raw=rng.random() < 0.5, norm=rng.random() < 0.7, theta=theta,
                    mask=rng.choice(["tree", "tree", "chain"]))
    return dict(op=op, batch=_log_int(rng, 1, 64), n=_log_int(rng, 1, 64), hist=_log_int(rng, 1, 2000) - 1, H=H,
                Hkv=Hkv, bits=rng.choice([0, 4, 8]))


# ---------------------------------------------------------------- the cache's page format

def _page_geom(Hkv, bits, es):
    """Byte sizes: one KV head's key block, its codes' offset, the value block's codes' offset, the page."""
    if bits == 0:
        kb = PAGE * 128 * es
        return kb, 0, 0, -(-(Hkv * kb * 2) // 128) * 128
    code = 4 * PAGE * 32 * bits // 8
    kb = 4 * PAGE * 2 + code
    return kb, 4 * PAGE * 2, Hkv * 4 * PAGE * 2, -(-(Hkv * kb * 2) // 128) * 128


def _token_bytes(Hkv, bits, es):
    return 2 * Hkv * 128 * es if bits == 0 else 2 * Hkv * (128 * bits // 8 + 8)


def _quantise(x, bits):
    """Rows [..., 128 m] float32 -> (scales fp16 [..., 4 m], codes uint8 [..., 4 m, 32] before packing)."""
    qmax = 2 ** (bits - 1) - 1
    g = x.reshape(*x.shape[:-1], -1, 32)
    s32 = g.abs().amax(-1) / qmax
    s16 = s32.half()
    low = s16.float() < s32                                      # rounded towards +infinity
    s16 = torch.where(low, (s16.view(torch.int16) + 1).view(torch.float16), s16)
    sf = s16.float()[..., None]
    q = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g)).clamp(-qmax, qmax)
    return s16, (q + 2 ** (bits - 1)).to(torch.uint8)


def _pack(u, bits):
    """uint8 codes [..., 32] -> bytes [..., 32 bits / 8] (the even channel in the low half of a 4-bit byte)."""
    return u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)


def _unpack(b, bits):
    if bits == 8:
        return b.float() - 128.0
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float() - 8.0


def _dtype(c):
    return torch.float32 if c.get("dtype", "bf16") == "f32" else torch.bfloat16


def _views(pool, c):
    """Typed views of the pool's pages: (K, V) [pages, 16, Hkv, 128], or scales and codes
    (Ks [pages, Hkv, 4, 16], Kc [pages, Hkv, 4, 16, bytes], Vs [pages, 4 Hkv, 16], Vc [pages, 4 Hkv, 16, bytes])."""
    Hkv, bits, dt = c["Hkv"], c["bits"], _dtype(c)
    es = dt.itemsize
    kb, kc, vc, pb = _page_geom(Hkv, bits, es)
    pages = pool.view(-1, pb)
    n = pages.shape[0]
    k, v = pages[:, :Hkv * kb], pages[:, Hkv * kb:2 * Hkv * kb]
    if bits == 0:
        e = pool.view(dt)
        pe = pb // es
        K = e.as_strided((n, PAGE, Hkv, 128), (pe, 128, PAGE * 128, 1))
        V = e.as_strided((n, PAGE, Hkv, 128), (pe, Hkv * 128, 128, 1), Hkv * kb // es)
        return K, V
    nb = 32 * bits // 8
    h = pool.view(torch.float16)
    Ks = h.as_strided((n, Hkv, 4, PAGE), (pb // 2, kb // 2, PAGE, 1))
    Kc = pool.as_strided((n, Hkv, 4, PAGE, nb), (pb, kb, PAGE * nb, nb, 1), kc)
    Vs = h.as_strided((n, 4 * Hkv, PAGE), (pb // 2, PAGE, 1), Hkv * kb // 2)
    Vc = pool.as_strided((n, 4 * Hkv, PAGE, nb), (pb, PAGE * nb, nb, 1), Hkv * kb + vc)
    return Ks, Kc, Vs, Vc


def _store(pool, c, page, slot, K, V):
    """Rows K, V [n, Hkv, 128] (float32) into slots (page, slot) [n]."""
    if c["bits"] == 0:
        Kp, Vp = _views(pool, c)
        Kp[page, slot] = K.to(Kp.dtype)
        Vp[page, slot] = V.to(Vp.dtype)
        return
    Ks, Kc, Vs, Vc = _views(pool, c)
    n, Hkv = K.shape[:2]
    s, u = _quantise(K, c["bits"])                              # [n, Hkv, 4], [n, Hkv, 4, 32]
    Ks[page, :, :, slot] = s
    Kc[page, :, :, slot] = _pack(u, c["bits"])
    s, u = _quantise(V.reshape(n, Hkv * 128), c["bits"])
    Vs[page, :, slot] = s
    Vc[page, :, slot] = _pack(u, c["bits"])


def _load(pool, c, page, slot):
    """K, V [..., Hkv, 128] float32 of slots (page, slot) of any shape."""
    if c["bits"] == 0:
        Kp, Vp = _views(pool, c)
        return Kp[page, slot].float(), Vp[page, slot].float()
    Ks, Kc, Vs, Vc = _views(pool, c)
    Hkv, sh = c["Hkv"], tuple(page.shape)
    p, t = page.reshape(-1), slot.reshape(-1)
    K = _unpack(Kc[p, :, :, t], c["bits"]) * Ks[p, :, :, t].float()[..., None]
    V = _unpack(Vc[p, :, t], c["bits"]) * Vs[p, :, t].float()[..., None]
    return K.reshape(*sh, Hkv, 128), V.reshape(*sh, Hkv, 128)


# ---------------------------------------------------------------- inputs

def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _cache(c, g, ctx):
    """An allocated cache: page table int32 [batch, max_pages] over a permuted pool, three pages spare."""
    mp = -(-ctx // PAGE)
    n_pages = c["batch"] * mp + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda")[:c["batch"] * mp]
    pb = _page_geom(c["Hkv"], c["bits"], _dtype(c).itemsize)[3]
    pool = torch.zeros(n_pages * pb, dtype=torch.uint8, device="cuda")
    return pool, n_pages, perm.view(c["batch"], mp).to(torch.int32)


def _fill(c, g, pool, pt, lens):
    """Tokens 0 .. lens[b] - 1 of every sequence: N(0, 1) keys with a few large channels, N(0, 1) values."""
    Hkv = c["Hkv"]
    gain = 1.0 + 3.0 * (torch.rand(Hkv, 128, generator=g, device="cuda") < 0.03).float()
    for b in range(pt.shape[0]):
        for t0 in range(0, int(lens[b]), 4096):
            t = torch.arange(t0, min(t0 + 4096, int(lens[b])), device="cuda")
            K = torch.randn(len(t), Hkv, 128, generator=g, device="cuda") * gain
            V = torch.randn(len(t), Hkv, 128, generator=g, device="cuda")
            _store(pool, c, pt[b, t // PAGE].long(), t % PAGE, K, V)


def _norms(c, g):
    if not c.get("norm"):
        return None, None
    dt = _dtype(c)
    return tuple((1.0 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(dt) for _ in range(2))


def _tree_masks(g, counts, words, kind):
    """Ancestor masks (the node itself among them) of random trees, as int32 words; None for a chain."""
    if kind == "chain":
        return None
    rows = []
    for n in counts:
        u = torch.rand(n, generator=g, device="cuda").tolist()
        m = []
        for i in range(n):
            parent = int(u[i] * i) if i else -1
            m.append((m[parent] if parent >= 0 else 0) | (1 << i))
        rows += [[x - (1 << 32) if x >= 1 << 31 else x for x in ((v >> (32 * w)) & 0xFFFFFFFF for w in range(words))]
                 for v in m]
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def _layer(c, s):
    """The layer handle that a program keeps (its own append projections are not used here)."""
    from decode_attention_rank_b200 import starkv as sk
    dt = _dtype(c)
    wide = c["op"] == "tree"
    hidden = D if wide else 64
    cfg = sk.LayerConfig(hidden=hidden, n_heads=c["H"], n_kv_heads=c["Hkv"], head_dim=128,
                         dtype="f32" if dt == torch.float32 else "bf16", rope=c.get("theta") is not None,
                         rope_theta=c.get("theta") or 10000.0, plain=True)
    Wkv = torch.zeros(hidden, c["Hkv"] * 128, dtype=dt, device="cuda")
    Wo = s["W_o"] if wide else torch.zeros(c["H"] * 128, hidden, dtype=dt, device="cuda")
    return sk.load_plain(cfg, Wkv, Wkv, Wo, kv_bits=c.get("bits", 0), q_norm=s.get("q_norm"), k_norm=s.get("k_norm"),
                         norm_eps=EPS)


def _ragged(c):
    """Histories and node counts of a batch: the first sequence at the case's own sizes, the others ragged below them
    (the case alone says how, so that every seed gives outputs of one shape)."""
    r = random.Random(c["batch"] * 1000003 + c["hist"] * 101 + c["n"])
    return ([c["hist"] - (int(r.random() * 0.3 * c["hist"]) if b else 0) for b in range(c["batch"])],
            [c["n"] - (int(r.random() * 0.5 * c["n"]) if b else 0) for b in range(c["batch"])])


def _inputs(c, seed):
    g = _rand(seed)
    s = {"case": c}
    H, Hkv, op, dt = c["H"], c["Hkv"], c["op"], _dtype(c)
    if op in ("norm_rope", "append"):
        # rows of a fused QKV projection: a few channels are large, as projections' outputs are
        n = c["n"] if op == "norm_rope" else c["n"] * c["batch"]
        gain = 1.0 + 4.0 * (torch.rand((H + 2 * Hkv) * 128, generator=g, device="cuda") < 0.02).float()
        s["qkv"] = (torch.randn(n, (H + 2 * Hkv) * 128, generator=g, device="cuda") * gain).to(dt)
        s["q_norm"], s["k_norm"] = _norms(c, g)
    if op == "norm_rope":
        s["pos"] = torch.randint(0, c["max_pos"], (c["n"],), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty(c["n"], H * 128, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(c["n"], Hkv * 128, dtype=dt, device="cuda")
    elif op == "append":
        s["pool"], s["n_pages"], s["pt"] = _cache(c, g, c["hist"] + c["n"])
        i = torch.arange(c["n"] * c["batch"], device="cuda")
        s["seq"] = (i // c["n"]).to(torch.int32)
        s["slots"] = (c["hist"] + i % c["n"]).to(torch.int32)
        # drafts of a tree share depths: positions lag behind slots
        lag = (torch.rand(len(i), generator=g, device="cuda") * (i % c["n"]).float() * 0.5).to(torch.int32)
        s["pos"] = s["slots"] - lag
        s["q_out"] = torch.empty(len(i), H * 128, dtype=dt, device="cuda")
    elif op == "read":
        s["pool"], s["n_pages"], s["pt"] = _cache(c, g, c["n"])
        _fill(c, g, s["pool"], s["pt"], [c["n"]] * c["batch"])
        i = torch.arange(c["n"] * c["batch"], device="cuda")
        s["seq"], s["slots"] = (i // c["n"]).to(torch.int32), (i % c["n"]).to(torch.int32)
        s["out"] = torch.empty(len(i), 2 * Hkv * 128, dtype=dt, device="cuda")
    else:
        hist, cnt = _ragged(c)
        off = [0]
        for x in cnt:
            off.append(off[-1] + x)
        s["hist"] = torch.tensor(hist, dtype=torch.int32, device="cuda")
        s["node_off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        s["n_nodes"], s["max_nodes"] = off[-1], c["n"]
        s["pool"], s["n_pages"], s["pt"] = _cache(c, g, c["hist"] + c["n"])
        _fill(c, g, s["pool"], s["pt"], [a + b for a, b in zip(hist, cnt)])
        if op == "tree":
            s["mask"] = _tree_masks(g, cnt, -(-c["n"] // 32), c["mask"])
            s["q"] = torch.randn(off[-1], H, 128, generator=g, device="cuda").to(dt)
            depth = torch.cat([torch.arange(x) for x in cnt]) // 2
            s["pos"] = (torch.repeat_interleave(s["hist"].cpu(), torch.tensor(cnt)) + depth).to(torch.int32).cuda()
            s["q_norm"], s["k_norm"] = _norms(c, g)
            s["W_o"] = (torch.randn(H * 128, D, generator=g, device="cuda") / math.sqrt(D)).to(dt)
            s["out"] = torch.empty(off[-1], D, dtype=dt, device="cuda")
        else:
            # the accepted path: increasing node numbers, about half of the nodes
            acc, n_acc = [], []
            for x in cnt:
                keep = [j for j, r in enumerate(torch.rand(x, generator=g, device="cuda").tolist()) if r < 0.5]
                n_acc.append(len(keep))
                acc += keep + [-1] * (x - len(keep))
            s["acc"] = torch.tensor(acc, dtype=torch.int32, device="cuda")
            s["n_acc"] = torch.tensor(n_acc, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s["layer"] = _layer(case, s)
        if case["op"] == "tree":
            ws = s["layer"].tree_workspace_bytes(case["batch"], s["pt"].shape[1] * PAGE, s["n_nodes"], s["max_nodes"])
            s["ws"] = torch.empty(ws, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- the operators

def _norm_rope(x, w, pos, theta, wide=False):
    """x [n, heads, 128] -> float32. The angles in 64 bits (far positions); all of it where a quantiser rounds the
    result next (`wide`: values next to a border)."""
    ty = torch.float64 if wide else torch.float32
    y = x.to(ty)
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.to(ty)
    p = torch.arange(64, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * torch.exp2(p * (-2.0 / 128 * math.log2(theta)))
    cs, sn = ang.cos()[:, None].to(ty), ang.sin()[:, None].to(ty)
    a, b = y[..., :64], y[..., 64:]
    return torch.cat((a * cs - b * sn, b * cs + a * sn), -1).float()


def _split(s):
    c, x = s["case"], s["qkv"]
    H, Hkv = c["H"], c["Hkv"]
    return x[:, :H * 128], x[:, H * 128:(H + Hkv) * 128], x[:, (H + Hkv) * 128:]


def _run_norm_rope(s):
    c = s["case"]
    q, k, _ = _split(s)
    if own:
        s["layer"].qk_norm_rope(q, k, s["pos"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    n, dt = q.shape[0], q.dtype
    return (_norm_rope(q.reshape(n, -1, 128), s["q_norm"], s["pos"], c["theta"]).to(dt).reshape(n, -1),
            _norm_rope(k.reshape(n, -1, 128), s["k_norm"], s["pos"], c["theta"]).to(dt).reshape(n, -1))


def _run_append(s):
    """The rotated queries, and the cache's new tokens as the values that their codes stand for."""
    c = s["case"]
    q, k, v = _split(s)
    if own:
        L = s["layer"]
        L.append_qkv(s["pool"], s["n_pages"], s["pt"], s["seq"], s["slots"], q, k, v, q_out=s["q_out"],
                     positions=s["pos"])
        if "kv" not in s:
            s["kv"] = torch.empty(q.shape[0], 2 * c["Hkv"] * 128, dtype=q.dtype, device=q.device)
        L.cache_read(s["pool"], s["n_pages"], s["pt"], s["seq"], s["slots"], s["kv"])
        return s["q_out"], s["kv"]
    n, dt = q.shape[0], q.dtype
    qo = _norm_rope(q.reshape(n, -1, 128), s["q_norm"], s["pos"], c["theta"]).to(dt).reshape(n, -1)
    K = _norm_rope(k.reshape(n, -1, 128), s["k_norm"], s["pos"], c["theta"], wide=True)
    page, slot = s["pt"][s["seq"], s["slots"] // PAGE].long(), s["slots"].long() % PAGE
    _store(s["pool"], c, page, slot, K, v.float().reshape(n, -1, 128))
    K, V = _load(s["pool"], c, page, slot)
    return qo, torch.cat((K.reshape(n, -1), V.reshape(n, -1)), -1).to(dt)


def _run_read(s):
    c = s["case"]
    if own:
        s["layer"].cache_read(s["pool"], s["n_pages"], s["pt"], s["seq"], s["slots"], s["out"])
        return s["out"]
    n = s["seq"].shape[0]
    page, slot = s["pt"][s["seq"], s["slots"] // PAGE].long(), s["slots"].long() % PAGE
    K, V = _load(s["pool"], c, page, slot)
    return torch.cat((K.reshape(n, -1), V.reshape(n, -1)), -1).to(_dtype(c))


def _run_tree(s):
    c = s["case"]
    if own:
        s["layer"].tree_attn(s["pool"], s["n_pages"], s["pt"], s["hist"], s["node_off"], s["q"], s["out"], s["ws"],
                             max_nodes=s["max_nodes"], mask=s["mask"], q_pos=s["pos"] if c["raw"] else None)
        return s["out"]
    B, N, H, Hkv = c["batch"], s["max_nodes"], c["H"], c["Hkv"]
    dev = s["q"].device
    q = _norm_rope(s["q"], s["q_norm"], s["pos"], c["theta"]) if c["raw"] else s["q"].float()
    # nodes padded to [B, N]; a padded node's row is dropped at the end
    off = s["node_off"].long()
    cnt = off[1:] - off[:-1]
    i = torch.arange(N, device=dev)
    real = i[None] < cnt[:, None]
    row = torch.where(real, off[:-1, None] + i[None], 0)
    T = s["pt"].shape[1] * PAGE
    t = torch.arange(T, device=dev)
    K, V = _load(s["pool"], c, s["pt"].long()[:, t // PAGE], (t % PAGE).expand(B, T))   # [B, T, Hkv, 128]
    j = t[None] - s["hist"].long()[:, None]                      # node number of a slot (negative: history)
    if s["mask"] is None:
        sees = j[:, None, :] <= i[None, :, None]
    else:
        m = s["mask"].long()[row]                                # [B, N, words]
        jj = j.clamp(0, 32 * m.shape[2] - 1)[:, None, :].expand(B, N, T)
        sees = ((torch.gather(m, 2, jj // 32) >> (jj % 32)) & 1).bool() | (j < 0)[:, None, :]
    sees = sees & (j < cnt[:, None])[:, None, :]
    qg = q[row].view(B, N, Hkv, H // Hkv, 128).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, 128)   # rows (head, node)
    S = torch.matmul(qg, K.permute(0, 2, 3, 1)).view(B, Hkv, H // Hkv, N, T) / math.sqrt(128)
    S = S.masked_fill(~sees[:, None, None], float("-inf"))
    top = S.amax(-1, keepdim=True).clamp_min(-1e30)
    P = torch.exp(S - top)
    P = P / P.sum(-1, keepdim=True).clamp_min(1e-30)
    y = torch.matmul(P.view(B, Hkv, -1, T), V.permute(0, 2, 1, 3)).view(B, H, N, 128)
    y = y.permute(0, 2, 1, 3).reshape(B * N, H * 128)[real.reshape(-1)]
    return torch.matmul(y, s["W_o"].float()).to(_dtype(c))


def _run_accept(s):
    """The whole pool after the move (a further pass moves what the one before it left)."""
    c = s["case"]
    if own:
        s["layer"].tree_accept(s["pool"], s["n_pages"], s["pt"], s["hist"], s["node_off"], s["acc"], s["n_acc"],
                               max_nodes=s["max_nodes"])
        return s["pool"]
    off, n_acc = s["node_off"].long(), s["n_acc"].long()
    cnt = off[1:] - off[:-1]
    i = torch.arange(s["n_nodes"], device=off.device)
    b = torch.searchsorted(off[1:], i, right=True)
    k = i - off[b]
    kept = k < n_acc[b]
    src = s["hist"].long()[b] + torch.where(kept, s["acc"].long(), 0)
    dst = s["hist"].long()[b] + k
    sp, ss = s["pt"][b, src // PAGE].long(), src % PAGE
    dp, ds = s["pt"][b, dst // PAGE].long(), dst % PAGE
    for v, lead in zip(_views(s["pool"], c), (1, 1) if c["bits"] == 0 else (3, 3, 2, 2)):
        at = (slice(None),) * (lead - 1)
        rows = v[(sp, *at, ss)]
        v[(dp, *at, ds)] = torch.where(kept.view(-1, *[1] * (rows.dim() - 1)), rows, torch.zeros_like(rows))
    return s["pool"]


def run(state):
    return {"norm_rope": _run_norm_rope, "append": _run_append, "read": _run_read, "tree": _run_tree,
            "accept": _run_accept}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    H, Hkv, op = c["H"], c["Hkv"], c["op"]
    es = _dtype(c).itemsize
    tb = _token_bytes(Hkv, c.get("bits", 0), es)
    if op == "norm_rope":
        el = c["n"] * (H + Hkv) * 128
        return {"bytes": 2.0 * el * es + 4 * c["n"], "flops": 7.0 * el}
    if op == "append":       # q, k, v in, q out, the tokens into the cache, and read back as rows
        n = c["n"] * c["batch"]
        return {"bytes": n * ((2 * H + 2 * Hkv) * 128.0 * es + 2 * tb + 2 * Hkv * 128 * es + 12),
                "flops": n * 128.0 * (7 * (H + Hkv) + 6 * Hkv)}
    if op == "read":
        n = c["n"] * c["batch"]
        return {"bytes": n * (tb + 2.0 * Hkv * 128 * es + 8), "flops": 2.0 * n * Hkv * 128}
    hist, cnt = _ragged(c)
    toks, nodes = sum(hist) + sum(cnt), sum(cnt)
    if op == "tree":
        return {"bytes": toks * float(tb) + nodes * (H * 128 + D) * es + H * 128.0 * D * es,
                "flops": sum(4.0 * n * H * 128 * (h + n) for h, n in zip(hist, cnt)) + 2.0 * nodes * H * 128 * D}
    # accept: about half of the nodes are read, and every node's slot is written (moved to, or cleared)
    return {"bytes": nodes * 1.5 * tb, "flops": 0.0}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits

def _rot64(x, w, pos, theta):
    x = x.to(torch.float64)
    n, h, d = x.shape
    if w is not None:
        ms = (x * x).sum(2) / d
        x = x / torch.sqrt(ms + EPS).unsqueeze(2) * w.to(torch.float64)
    freq = torch.tensor([theta ** (-2.0 * p / d) for p in range(d // 2)], dtype=torch.float64, device=x.device)
    z = torch.polar(torch.ones(n, 1, d // 2, dtype=torch.float64, device=x.device),
                    (pos.to(torch.float64).view(n, 1) * freq).view(n, 1, d // 2))
    r = torch.complex(x[:, :, :d // 2].contiguous(), x[:, :, d // 2:].contiguous()) * z
    return torch.cat((r.real, r.imag), 2)


def _codes64(x, bits):
    """x [n, m] float64 rounded to float32 -> the stored values, float64."""
    top = float(2 ** (bits - 1) - 1)
    x = x.to(torch.float32).to(torch.float64)
    parts = x.view(x.shape[0], x.shape[1] // 32, 32)
    want = (parts.abs().max(2).values.to(torch.float32) / top).to(torch.float64)
    half = want.to(torch.float16)
    up = torch.nextafter(half, torch.full_like(half, float("inf")))
    half = torch.where(half.to(torch.float64) >= want, half, up).to(torch.float64).unsqueeze(2)
    code = torch.where(half > 0, parts / half, torch.zeros_like(parts))
    code = torch.round(code.to(torch.float32)).to(torch.float64).clamp(-top, top)
    return (code * half).reshape(x.shape)


def _stored64(pool, c, page, slot):
    """K, V [n, Hkv, 128] float64 of slots, from the byte offsets of the page format."""
    Hkv, bits, dev = c["Hkv"], c["bits"], pool.device
    kb, kc, vc, pb = _page_geom(Hkv, bits, _dtype(c).itemsize)
    h = torch.arange(Hkv, device=dev).view(1, -1, 1)
    ch = torch.arange(128, device=dev).view(1, 1, -1)
    p, t = page.view(-1, 1, 1) * pb, slot.view(-1, 1, 1)
    if bits == 0:
        el, es = pool.view(_dtype(c)), _dtype(c).itemsize
        return (el[(p + h * kb + t * 128 * es) // es + ch].to(torch.float64),
                el[(p + Hkv * kb + t * Hkv * 128 * es) // es + h * 128 + ch].to(torch.float64))
    half = pool.view(torch.float16)
    per = 32 * bits // 8                                         # bytes of one slot in a group of 32 channels

    def group(scales, codes, g):
        byte = pool[codes + g * PAGE * per + t * per + (ch % 32) * bits // 8].to(torch.int32)
        code = byte if bits == 8 else torch.where(ch % 2 == 1, byte // 16, byte % 16)
        return (code - 2 ** (bits - 1)).to(torch.float64) * half[scales // 2 + g * PAGE + t].to(torch.float64)

    return (group(p + h * kb, p + h * kb + kc, ch // 32),
            group(p + Hkv * kb, p + Hkv * kb + vc, h * 4 + ch // 32))


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    H, Hkv, op = c["H"], c["Hkv"], c["op"]
    if op == "norm_rope":
        n, x = c["n"], s["qkv"]
        return (_rot64(x[:, :H * 128].reshape(n, H, 128), s["q_norm"], s["pos"], c["theta"]).reshape(n, -1),
                _rot64(x[:, H * 128:(H + Hkv) * 128].reshape(n, Hkv, 128), s["k_norm"], s["pos"],
                       c["theta"]).reshape(n, -1))
    if op == "append":
        x = s["qkv"]
        n = x.shape[0]
        q = _rot64(x[:, :H * 128].reshape(n, H, 128), s["q_norm"], s["pos"], c["theta"]).reshape(n, -1)
        k = _rot64(x[:, H * 128:(H + Hkv) * 128].reshape(n, Hkv, 128), s["k_norm"], s["pos"], c["theta"])
        kv = torch.cat((k.reshape(n, -1), x[:, (H + Hkv) * 128:].to(torch.float64)), 1)
        return q, (_codes64(kv, c["bits"]) if c["bits"] else kv)
    if op in ("read", "accept"):
        return None                                              # values that are moved, not computed
    rows = []
    off, hist = s["node_off"].tolist(), s["hist"].tolist()
    q = _rot64(s["q"], s["q_norm"], s["pos"], c["theta"]) if c["raw"] else s["q"].to(torch.float64)
    Wo = s["W_o"].to(torch.float64)
    for b in range(c["batch"]):
        n, T = off[b + 1] - off[b], hist[b] + off[b + 1] - off[b]
        t = torch.arange(T, device="cuda")
        K, V = _stored64(s["pool"], c, s["pt"][b, t // PAGE].long(), t % PAGE)
        see = torch.ones(n, T, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            see[:, hist[b]:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            bits = (s["mask"][off[b]:off[b + 1]].unsqueeze(2) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
            see[:, hist[b]:] = bits.reshape(n, -1)[:, :n] == 1
        qb = q[off[b]:off[b + 1]].view(n, Hkv, H // Hkv, 128)
        sc = torch.einsum("nghd,tgd->ghnt", qb, K) * 128 ** -0.5
        sc = torch.where(see, sc, torch.full_like(sc, -float("inf")))
        y = torch.einsum("ghnt,tgd->nghd", torch.softmax(sc, -1), V)
        rows.append(y.reshape(n, H * 128) @ Wo)
    return torch.cat(rows)
