"""The serving operators (per-head norm and rotation, quantised append, cache read, tree attention, tree accept)
against their float64 definitions.

Tolerances.  A value rounded to bf16 is off by at most 2^-8 of itself, to fp32 by 2^-24.  The norm and rotation work in
fp32 from there: the sum of d squares, its root and the three products of a pair are each off by a few 2^-24 of the
pair's length, together below 32 * 2^-24 of it.  Packed pages are equal to the byte.  Attention outputs of bf16 layers:
the output's rounding alone is 2^-8 / sqrt(3) / 1.4 = 1.6e-3 in relative L2, and the roundings of q, P and y to
fp16 (2^-11 each, of random sign) add below 4e-4 each: 3e-3, and 1e-2 of the largest output for single values.  fp32
layers: scores of size 20 are off by about 20 * 8 * 2^-24 = 1e-5, which is the relative error of a weight: 4e-5.
"""
import random

import numpy as np
import pytest
import torch

import serving_ref as R
from harness import Case, GpuCache, check_close
from synth import gen

pytestmark = pytest.mark.gpu

EPS = 1e-6


def sk():
    from decode_attention_rank_b200 import starkv
    return starkv


def dt_of(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


class Plain:
    """One uncompressed layer with random weights."""

    def __init__(self, H=4, hkv=2, d=128, bits=0, dtype="bf16", norm=True, rope=True, theta=10000.0, hidden=96, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.hkv, self.d, self.bits, self.dtype, self.dt = H, hkv, d, bits, dtype, dt_of(dtype)
        self.theta, self.rope, self.hidden = theta, rope, hidden
        self.W_k, self.W_v = (self.r(torch.randn(hidden, hkv * d, generator=g) / hidden ** 0.5) for _ in range(2))
        self.W_o = self.r(torch.randn(H * d, hidden, generator=g) / (H * d) ** 0.5)
        self.wq, self.wk = ((self.r(1 + 0.3 * torch.randn(d, generator=g)) if norm else None) for _ in range(2))
        cfg = sk().LayerConfig(hidden=hidden, n_heads=H, n_kv_heads=hkv, head_dim=d, dtype=dtype, rope=rope,
                               rope_theta=theta, plain=True)

        def cu(t):
            return None if t is None else t.to(self.dt).cuda()
        self.L = sk().load_plain(cfg, cu(self.W_k), cu(self.W_v), cu(self.W_o), kv_bits=bits, q_norm=cu(self.wq),
                                 k_norm=cu(self.wk), norm_eps=EPS)
        assert self.L.page_bytes == R.page_bytes(hkv, d, bits, self.dt.itemsize)

    def r(self, t):
        """float64 values of t in the layer's type."""
        return t.to(self.dt).to(torch.float64)

    def norm_rope(self, x, w, pos):
        return R.norm_rope(x, w, EPS, pos if self.rope else None, self.theta)

    def cache(self, lens, seed=0, spare=3):
        return PlainCache(self, lens, seed, spare)


class PlainCache:
    """Pages on the CPU (the definition's) and on the device, over a shuffled pool."""

    def __init__(self, p, caps, seed=0, spare=3):
        g = torch.Generator().manual_seed(100 + seed)
        mp = max(1, max(-(-c // 16) for c in caps))
        self.p, self.n_pages = p, len(caps) * mp + spare
        self.pt = torch.randperm(self.n_pages, generator=g)[:len(caps) * mp].reshape(len(caps), mp)
        self.pages = torch.zeros(self.n_pages, p.L.page_bytes, dtype=torch.uint8)
        self.pt_d = self.pt.to(torch.int32).cuda()
        self.K = [torch.zeros(0, p.hkv, p.d, dtype=torch.float64) for _ in caps]
        self.V = [k.clone() for k in self.K]
        self.g = g

    def fill(self, b, n):
        """n random tokens at the end of sequence b, by the definition's packer."""
        p = self.p
        K = torch.randn(n, p.hkv, p.d, generator=self.g, dtype=torch.float64)
        V = torch.randn(n, p.hkv, p.d, generator=self.g, dtype=torch.float64)
        t = torch.arange(len(self.K[b]), len(self.K[b]) + n)
        R.put(self.pages, self.pt[b, t // 16], t % 16, K, V, p.bits, p.dt)
        self.K[b] = torch.cat((self.K[b], R.stored(K, p.bits, p.dt)))
        self.V[b] = torch.cat((self.V[b], R.stored(V.reshape(n, -1), p.bits, p.dt).reshape(n, p.hkv, p.d)))

    def upload(self):
        self.pool = self.pages.reshape(-1).cuda()
        return self.pool

    def download(self):
        return self.pool.cpu().reshape(self.n_pages, -1)


def i32(x, dev="cuda"):
    return torch.as_tensor(x, dtype=torch.int32).to(dev)


def close_rows(got, want, size, dt):
    """Element by element: the output type's rounding of the value, and 32 * 2^-24 of the pair's length."""
    got = got.to(torch.float64).cpu()
    tol = want.abs() * (torch.finfo(dt).eps / 2) * 1.001 + size * 32 * 2.0 ** -24
    assert torch.all((got - want).abs() <= tol), ((got - want).abs() - tol).max()


def pair_size(y):
    h = y.shape[-1] // 2
    return torch.sqrt(y[..., :h] ** 2 + y[..., h:] ** 2).repeat(1, 1, 2)


# ------------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("dtype,H,hkv,d,n,norm,rope", [
    ("bf16", 4, 2, 128, 1, True, True), ("bf16", 32, 8, 128, 37, True, True), ("bf16", 4, 4, 64, 700, True, True),
    ("bf16", 3, 1, 256, 5, True, True), ("f32", 4, 2, 128, 33, True, True), ("f32", 2, 2, 64, 601, False, True),
    ("f32", 2, 1, 256, 9, True, False), ("bf16", 4, 2, 80, 19, True, True), ("f32", 2, 2, 6, 3, True, True),
    ("bf16", 5, 5, 128, 17, False, False), ("bf16", 2, 1, 2, 4, True, True)])
def test_qk_norm_rope(dtype, H, hkv, d, n, norm, rope):
    p = Plain(H, hkv, d, 0, dtype, norm, rope, theta=500000.0)
    g = torch.Generator().manual_seed(n)
    x = p.r(torch.randn(n, (H + 2 * hkv) * d, generator=g) * 3)
    x[0, :d] = 0                                              # a head of zeros
    pos = torch.randint(0, 131072, (n,), generator=g)
    fused = x.to(p.dt).cuda()
    q, k = fused[:, :H * d], fused[:, H * d:(H + hkv) * d]
    qo = torch.full((n, H * d + 8), 7.0, dtype=p.dt, device="cuda")
    ko = torch.empty(n, hkv, d, dtype=p.dt, device="cuda")
    p.L.qk_norm_rope(q, k, i32(pos), qo[:, :H * d], ko)
    wq = p.norm_rope(x[:, :H * d].reshape(n, H, d), p.wq, pos)
    wk = p.norm_rope(x[:, H * d:(H + hkv) * d].reshape(n, hkv, d), p.wk, pos)
    close_rows(qo[:, :H * d].reshape(n, H, d), wq, pair_size(wq), p.dt)
    close_rows(ko, wk, pair_size(wk), p.dt)
    assert torch.all(qo[:, H * d:] == 7)                      # between the rows
    # one side alone, in place
    p.L.qk_norm_rope(None, k, i32(pos), None, k)
    assert torch.equal(k.reshape(n, hkv, d), ko)
    assert torch.equal(q, x[:, :H * d].to(p.dt).cuda())
    assert p.L.sync_status() == 0


def test_qk_norm_rope_rows_off_16_bytes():
    """Rows that start on 4 bytes only give the same values as aligned ones."""
    p = Plain(4, 2, 128)
    x = torch.randn(9, 4 * 128 + 2, dtype=torch.float32).to(torch.bfloat16).cuda()
    pos = i32(range(9))
    a, b = torch.empty(9, 512, dtype=p.dt, device="cuda"), torch.empty(9, 512, dtype=p.dt, device="cuda")
    p.L.qk_norm_rope(x[:, 2:], None, pos, a, None)
    p.L.qk_norm_rope(x[:, 2:].contiguous(), None, pos, b, None)
    w = p.norm_rope(x[:, 2:].cpu().to(torch.float64).reshape(9, 4, 128), p.wq, torch.arange(9))
    close_rows(a.reshape(9, 4, 128), w, pair_size(w), p.dt)
    close_rows(b.reshape(9, 4, 128), w, pair_size(w), p.dt)


# ------------------------------------------------------------------ quantised append and reading back

@pytest.mark.parametrize("bits,dtype,H,hkv,d,n", [
    (8, "bf16", 4, 2, 128, 37), (4, "bf16", 4, 2, 128, 37), (0, "bf16", 4, 2, 128, 37), (8, "f32", 2, 2, 64, 1),
    (4, "f32", 2, 1, 256, 20), (0, "f32", 2, 1, 128, 20), (4, "bf16", 8, 8, 64, 700), (8, "bf16", 2, 1, 256, 650),
    (0, "bf16", 3, 3, 80, 18)])
def test_append_qkv_pages_and_read(bits, dtype, H, hkv, d, n):
    p = Plain(H, hkv, d, bits, dtype)
    c = p.cache([n + 5, n + 21])
    g = torch.Generator().manual_seed(3)
    x = p.r(torch.randn(2 * n, (H + 2 * hkv) * d, generator=g) * (1 + 5 * (torch.rand((H + 2 * hkv) * d, generator=g) < 0.05)))
    x[1] = 0
    x[0, -d:] = x[0, -d:] * 1e-7                                # scales below the smallest normal fp16
    seq = torch.arange(2 * n) // n
    slots = torch.arange(2 * n) % n + 5 + 16 * seq
    pos = slots - torch.randint(0, 4, (2 * n,), generator=g)
    fused = x.to(p.dt).cuda()
    parts = [fused[:, a * d:b * d] for a, b in ((0, H), (H, H + hkv), (H + hkv, H + 2 * hkv))]
    qo = torch.empty(2 * n, H * d, dtype=p.dt, device="cuda")
    pool = c.upload()
    pool.random_(0, 255)                                        # slots hold something already: all of it is overwritten
    p.L.append_qkv(pool, c.n_pages, c.pt_d, i32(seq), i32(slots), *parts, q_out=qo, positions=i32(pos))
    K = p.norm_rope(x[:, H * d:(H + hkv) * d].reshape(-1, hkv, d), p.wk, pos)
    V = x[:, (H + hkv) * d:].reshape(-1, hkv, d)
    wq = p.norm_rope(x[:, :H * d].reshape(-1, H, d), p.wq, pos)
    close_rows(qo.reshape(-1, H, d), wq, pair_size(wq), p.dt)
    out = torch.empty(2 * n, 2 * hkv * d, dtype=p.dt, device="cuda")
    p.L.cache_read(pool, c.n_pages, c.pt_d, i32(seq), i32(slots), out)
    if bits:
        # the definition's bytes; untouched slots as they were
        want = torch.zeros_like(c.pages)
        R.put(want, c.pt[seq, slots // 16], slots % 16, K, V, bits, p.dt)
        mark = torch.zeros_like(c.pages)
        R.put(mark, c.pt[seq, slots // 16], slots % 16, torch.full_like(K, 1.0), torch.full_like(V, -1.0), bits, p.dt)
        touched = mark != 0
        got = c.download()
        assert torch.equal(got[touched], want[touched])
        kv = torch.cat((R.stored(K, bits, p.dt).reshape(2 * n, -1),
                        R.stored(V.reshape(2 * n, -1), bits, p.dt)), -1)
        assert torch.equal(out.cpu(), kv.to(torch.float32).to(p.dt))
    else:
        close_rows(out[:, :hkv * d].reshape(-1, hkv, d), K, pair_size(K), p.dt)
        assert torch.equal(out[:, hkv * d:].cpu(), x[:, (H + hkv) * d:].to(p.dt))
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [0, 4, 8])
def test_append_leaves_other_slots(bits):
    p = Plain(2, 2, 128, bits)
    c = p.cache([40])
    pool = c.upload()
    pool.random_(0, 255)
    before = c.download().clone()
    x = torch.randn(1, 3 * 256).to(p.dt).cuda()
    p.L.append_qkv(pool, c.n_pages, c.pt_d, i32([0]), i32([21]), None, x[:, 256:512], x[:, 512:])
    after = c.download()
    diff = (after != before).any(1).nonzero().flatten().tolist()
    assert diff == [int(c.pt[0, 1])]
    mark = torch.zeros_like(before)
    ones = torch.ones(1, 2, 128, dtype=torch.float64)
    R.put(mark, c.pt[0, 1:2], torch.tensor([5]), ones, -ones, bits, p.dt)
    # (codes of +1 and -1 are never byte 0 in either half, but a 4-bit -1 has low nibbles 1: every byte is marked)
    assert not torch.any((after != before) & (mark == 0))


def test_append_refuses_what_does_not_fit():
    p = Plain(2, 1, 128, 8)
    c = p.cache([33])
    bad_pt = c.pt_d.clone()
    bad_pt[0, 1] = c.n_pages
    pool = c.upload()
    x = torch.randn(4, 4 * 128).to(p.dt).cuda()
    k, v = x[:, 256:384], x[:, 384:]
    q, qo = x[:, :256], torch.zeros(4, 256, dtype=p.dt, device="cuda")
    p.L.append_qkv(pool, c.n_pages, bad_pt, i32([0, 0, 1, 0]), i32([48, 17, 0, -1]), q, k, v, q_out=qo)
    assert p.L.sync_status() == 3                              # bad position and bad page
    assert torch.all(pool == 0)
    w = p.norm_rope(q.cpu().to(torch.float64).reshape(4, 2, 128), p.wq, torch.tensor([48, 17, 0, -1]))
    close_rows(qo.reshape(4, 2, 128), w, pair_size(w), p.dt)  # the queries do not need a slot
    out = torch.full((2, 256), 5.0, dtype=p.dt, device="cuda")
    p.L.cache_read(pool, c.n_pages, bad_pt, i32([0, 0]), i32([17, 100]), out)
    assert torch.all(out == 0) and p.L.sync_status() == 3


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 40000.0])
def test_append_values_without_a_code(bits, bad):
    """A group that holds a NaN, an infinity or a value beyond 32768 is stored as zeros, and flagged."""
    p = Plain(2, 1, 128, bits, norm=False, rope=False)
    c = p.cache([16])
    pool = c.upload()
    k, v = torch.ones(1, 128), torch.ones(1, 128)
    v[0, 37] = bad
    p.L.append_qkv(pool, c.n_pages, c.pt_d, i32([0]), i32([3]), None, k.to(p.dt).cuda(), v.to(p.dt).cuda())
    out = torch.empty(1, 256, dtype=p.dt, device="cuda")
    p.L.cache_read(pool, c.n_pages, c.pt_d, i32([0]), i32([3]), out)
    want = torch.ones(1, 256)
    want[0, 128 + 32:128 + 64] = 0
    R_ = R.stored(want.to(torch.float64), bits, p.dt).to(torch.float32).to(p.dt)
    assert torch.equal(out.cpu(), R_) and p.L.sync_status() == 4


@pytest.mark.parametrize("bits", [4, 8])
def test_append_of_latents_packs_the_same(bits):
    """starkv_append of K and V rows writes the bytes of starkv_append_qkv, scales at the fp16 borders among them."""
    p = Plain(2, 1, 128, bits, "f32", norm=False, rope=False)
    n = 200
    a, b = p.cache([n]), p.cache([n])
    x = torch.randn(n, 256)
    x[:, 5] = torch.arange(n) * (2 ** (bits - 1) - 1) / 16.0           # amax / qmax is an fp16 number
    x[7, 200] = float("nan")
    x = x.cuda()
    slots = i32(torch.arange(n))
    p.L.append_qkv(a.upload(), a.n_pages, a.pt_d, i32([0] * n), slots, None, x[:, :128], x[:, 128:])
    p.L.append(b.upload(), b.n_pages, b.pt_d, i32([0] * n), slots, x, True)
    assert p.L.sync_status() == 4
    assert torch.equal(a.download(), b.download())
    K, V = x[:, :128].cpu().to(torch.float64), x[:, 128:].cpu().to(torch.float64)
    V[7, 64:96] = 0
    R.put(a.pages, a.pt[0, torch.arange(n) // 16], torch.arange(n) % 16, K.reshape(n, 1, 128), V.reshape(n, 1, 128),
          bits, p.dt)
    assert torch.equal(a.download(), a.pages)


@pytest.mark.parametrize("quantized", [False, True])
def test_cache_read_latent_layer(quantized):
    spec = gen.config_spec(3, quantized=quantized)
    c = Case(spec, 3)
    L = c.load()
    cache = GpuCache(L, [37, 5])
    Z = [c.latents_direct(b, T) for b, T in ((0, 37), (1, 5))]
    for b in range(2):
        cache.append_latents(b, Z[b])
    seq, slots = [0] * 37 + [1] * 5, list(range(37)) + list(range(5))
    out = torch.empty(42, L.latent_total, dtype=torch.bfloat16, device="cuda")
    L.cache_read(cache.pool, cache.n_pages, cache.page_table, i32(seq), i32(slots), out)
    want = np.concatenate([np.concatenate(c.stored(z), axis=1) for z in Z])
    assert torch.equal(out.cpu(), torch.from_numpy(want).to(torch.float32).to(torch.bfloat16))
    assert L.sync_status() == 0


# ------------------------------------------------------------------ tree attention

def run_tree(p, hist, counts, masks, raw=True, tail=0, seed=0, q_gain=1.0):
    """Library and definition on one batch: returns (out, want, cache, call arguments)."""
    g = torch.Generator().manual_seed(seed)
    n = sum(counts)
    c = p.cache([h + k for h, k in zip(hist, counts)], seed)
    off = [0]
    for k in counts:
        off.append(off[-1] + k)
    for b, (h, k) in enumerate(zip(hist, counts)):
        c.fill(b, h + k)
    pos = torch.cat([torch.arange(k) // 2 + h for h, k in zip(hist, counts)] or [torch.zeros(0)]).long()
    pos = torch.cat((pos, torch.zeros(tail, dtype=torch.long)))
    q = p.r(torch.randn(n + tail, p.H, p.d, generator=g) * q_gain)
    qx = p.norm_rope(q, p.wq, pos) if raw else q
    want, rows = [], []
    words = max(1, -(-max(counts + [1]) // 32))
    for b, (h, k) in enumerate(zip(hist, counts)):
        see = torch.ones(k, h + k, dtype=torch.bool)
        sets = masks[b] if masks else [set(range(i + 1)) for i in range(k)]
        for i in range(k):
            for j in range(k):
                see[i, h + j] = j in sets[i]
        rows += sets
        y = R.attention(qx[off[b]:off[b] + k], c.K[b], c.V[b], see, p.d ** -0.5)
        want.append(y @ p.W_o)
    c.upload()
    q_d, out = q.to(p.dt).cuda(), torch.full((n + tail, p.hidden), 9.0, dtype=p.dt, device="cuda")
    max_nodes = max(counts + [1])
    ws = torch.empty(p.L.tree_workspace_bytes(len(hist), c.pt.shape[1] * 16, n + tail, max_nodes), dtype=torch.uint8,
                     device="cuda").random_(0, 255)
    m = None
    if masks:
        m = torch.cat((R.mask_words(rows, words), torch.zeros(tail, words, dtype=torch.int32))).cuda()
    args = dict(pool=c.pool, n_pages=c.n_pages, page_table=c.pt_d, hist=i32(hist), node_off=i32(off), q=q_d, out=out,
                workspace=ws, max_nodes=max_nodes, mask=m, q_pos=i32(pos) if raw else None)
    p.L.tree_attn(**args)
    torch.cuda.synchronize()
    if tail:
        assert torch.all(out[n:] == 9)
    return out[:n].to(torch.float64).cpu(), torch.cat(want) if n else torch.zeros(0, p.hidden), c, args


def check_tree(got, want, dtype):
    if dtype == "bf16":
        check_close(got.numpy(), want.numpy())
        return
    assert torch.linalg.norm(got - want) <= 4e-5 * torch.linalg.norm(want)
    assert (got - want).abs().max() <= 4e-5 * want.abs().max()


TREES = [
    # H, hkv, hist, counts
    (4, 4, [0], [1]), (4, 4, [1], [1]), (4, 2, [15, 0, 16], [1, 1, 1]), (8, 1, [333], [7]),
    (4, 4, [31, 700, 0, 5], [16, 3, 9, 0]), (4, 1, [130, 1025], [33, 64]), (16, 2, [40, 250], [24, 13]),
    (2, 2, [257], [100]), (8, 1, [100, 3000, 0], [64, 40, 33]), (32, 2, [5, 640], [3, 20]), (4, 1, [1000] * 9, [9] * 9), (4, 2, [9, 9, 9] * 23, [1, 2, 0] * 23), (32, 8, [77, 5], [24, 31]), (8, 8, [2000, 1999], [5, 8])]


@pytest.mark.parametrize("bits", [0, 8, 4])
@pytest.mark.parametrize("H,hkv,hist,counts", TREES)
def test_tree(bits, H, hkv, hist, counts):
    rng = random.Random(len(hist) * 100 + bits)
    p = Plain(H, hkv, 128, bits)
    for k, kind in enumerate(("tree", "chain")):
        masks = [R.random_tree(rng, n)[0] for n in counts] if kind == "tree" else None
        got, want, _, _ = run_tree(p, hist, counts, masks, raw=k == 0, tail=k * 3, seed=k)
        check_tree(got, want, "bf16")
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("dtype,d,H,hkv,bits", [("f32", 128, 4, 2, 0), ("f32", 64, 4, 4, 8), ("f32", 256, 2, 1, 4),
                                                ("bf16", 64, 4, 2, 4), ("bf16", 256, 4, 2, 8), ("bf16", 80, 3, 3, 0),
                                                ("bf16", 128, 12, 4, 8), ("bf16", 128, 32, 1, 4)])
def test_tree_shapes(dtype, d, H, hkv, bits):
    rng = random.Random(d)
    p = Plain(H, hkv, d, bits, dtype, hidden=200)
    hist, counts = [50, 0, 161], [9, 17, 4]
    got, want, _, _ = run_tree(p, hist, counts, [R.random_tree(rng, n)[0] for n in counts], tail=2)
    check_tree(got, want, dtype)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [0, 8, 4])
def test_tree_peaky_scores(bits):
    """Scores of size 50 and far apart: the running maximum moves often."""
    p = Plain(4, 2, 128, bits, norm=False)
    got, want, _, _ = run_tree(p, [900, 33], [6, 20], None, q_gain=5.0)
    check_tree(got, want, "bf16")


@pytest.mark.parametrize("bits", [0, 8])
def test_tree_rows_that_see_nothing(bits):
    p = Plain(4, 2, 128, bits)
    masks = [[set(), {1}, {0, 2}], [set(), set()], [{0}, set()]]
    got, want, _, _ = run_tree(p, [0, 0, 20], [3, 2, 2], masks)
    assert torch.all(got[0] == 0) and torch.all(got[3:5] == 0)
    check_tree(got, want, "bf16")
    assert p.L.sync_status() == 0


def test_tree_masked_nodes_hold_nan():
    """What a node may not see does not reach it, whatever the slot holds; nor do slots past the nodes."""
    p = Plain(4, 2, 128, 0)
    rng = random.Random(1)
    sees = R.random_tree(rng, 12)[0]
    hidden = {i for i in range(12) if i and rng.random() < 0.3}
    sees = [s - hidden for s in sees]
    got, want, c, args = run_tree(p, [37], [12], [sees])
    nan = torch.full((len(hidden) + 5, 2, 128), float("nan"), dtype=torch.float64)
    t = torch.tensor([37 + j for j in sorted(hidden)] + list(range(49, 54)))
    t = t[t < c.pt.shape[1] * 16]
    R.put(c.pages, c.pt[0, t // 16], t % 16, nan[:len(t)], nan[:len(t)], 0, p.dt)
    args["pool"] = c.upload()
    p.L.tree_attn(**args)
    check_tree(args["out"].to(torch.float64).cpu(), want, "bf16")


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_tree_nan_reaches_only_the_nodes_that_see_it(what):
    p = Plain(4, 2, 128, 0)
    sees = [{0}, {0, 1}, {0, 2}, {0, 2, 3}, {0, 1, 4}]
    for side in (0, 1):
        got, want, c, args = run_tree(p, [21], [5], [sees])
        K, V = c.K[0][21 + 2:21 + 3].clone(), c.V[0][21 + 2:21 + 3].clone()
        (K if side == 0 else V)[0, :, 7] = what
        R.put(c.pages, c.pt[0, 1:2], torch.tensor([7]), K, V, 0, p.dt)
        p.L.tree_attn(**dict(args, pool=c.upload()))
        out = args["out"].to(torch.float64).cpu()
        check_tree(out[[0, 1, 4]], want[[0, 1, 4]], "bf16")
        if not (side == 0 and what == float("inf")):           # (q times an infinite key may be minus infinity: weight 0)
            assert torch.all(torch.isnan(out[[2, 3]]))


@pytest.mark.parametrize("group,n,hist", [(2, 20, 37), (4, 33, 300), (8, 64, 128)])
def test_tree_of_many_rows_and_values_that_are_not_finite(group, n, hist):
    """As the two tests above, with more rows per KV head, nodes over several tiles, and rows that see nothing."""
    p = Plain(2 * group, 2, 128, 0)
    sees = R.random_tree(random.Random(n), n)[0]
    hidden = {5, n - 2}
    sees = [s - hidden for s in sees]
    got, want, c, args = run_tree(p, [hist, 0], [n, n], [sees, [set() if i % 3 == 0 else s for i, s in enumerate(sees)]])
    check_tree(got, want, "bf16")
    assert torch.all(got[n::3][:n // 3] == 0)
    nan = torch.full((1, 2, 128), float("nan"), dtype=torch.float64)
    for b, h in enumerate((hist, 0)):
        for j in [*sorted(hidden), *range(n, n + 9)]:                 # and slots past the nodes
            if (h + j) // 16 < c.pt.shape[1]:
                R.put(c.pages, c.pt[b, (h + j) // 16:(h + j) // 16 + 1], torch.tensor([(h + j) % 16]), nan, nan, 0, p.dt)
    clean = c.upload().clone()
    p.L.tree_attn(**dict(args, pool=clean))
    check_tree(args["out"].to(torch.float64).cpu(), want, "bf16")
    for what, side in ((float("nan"), 0), (float("nan"), 1), (float("inf"), 1)):
        K, V = c.K[0][hist + 2:hist + 3].clone(), c.V[0][hist + 2:hist + 3].clone()
        (V if side else K)[0, :, 7] = what
        at = c.pt[0, (hist + 2) // 16:(hist + 2) // 16 + 1], torch.tensor([(hist + 2) % 16])
        R.put(c.pages, *at, K, V, 0, p.dt)
        p.L.tree_attn(**dict(args, pool=c.upload()))
        R.put(c.pages, *at, c.K[0][hist + 2:hist + 3], c.V[0][hist + 2:hist + 3], 0, p.dt)
        out = args["out"].to(torch.float64).cpu()
        see = torch.tensor([2 in s for s in sees] + [False] * n)
        assert see.any() and torch.all(torch.isnan(out[see]))
        check_tree(out[~see], want[~see], "bf16")
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_tree_plain_layer_of_load_factors(dtype, d):
    """Uncompressed layers without serving options: a chain of nodes is the decode of each prefix."""
    g = torch.Generator().manual_seed(0)
    H, hkv, D, dt = 8, 2, 96, dt_of(dtype)
    W = [(torch.randn(*s, generator=g) / s[0] ** 0.5).to(dt).cuda() for s in ((D, hkv * d), (D, hkv * d), (H * d, D))]
    cfg = sk().LayerConfig(hidden=D, n_heads=H, n_kv_heads=hkv, head_dim=d, dtype=dtype, rope=True, plain=True)
    L = sk().load_factors(cfg, W[0], None, W[1], None, W[2])
    n, T = 5, 40
    c = GpuCache(L, [T + n] * n)
    x = torch.randn(T + n, 2 * hkv * d, generator=g).numpy()
    for b in range(n):
        c.append_latents(b, [x[:, :d], x[:, d:2 * d], x[:, 2 * d:]])
    q = torch.randn(n, H, d, generator=g).to(dt).cuda()
    out, want = (torch.empty(n, D, dtype=dt, device="cuda") for _ in range(2))
    mp = c.page_table.shape[1]
    ws = torch.empty(max(L.tree_workspace_bytes(1, mp * 16, n, n), L.workspace_bytes(n, mp * 16)), dtype=torch.uint8,
                     device="cuda")
    L.tree_attn(c.pool, c.n_pages, c.page_table[:1], i32([T]), i32([0, n]), q, out, ws, max_nodes=n,
                q_pos=i32(range(T, T + n)))
    L.decode(c.pool, c.n_pages, c.page_table, i32(range(T + 1, T + n + 1)), q, want, ws)
    assert L.sync_status() == 0
    a, b = out.to(torch.float64).cpu(), want.to(torch.float64).cpu()
    # each side within its own bound of the definition: sqrt(2) * 1.7e-3 in bf16, two times 4e-5 in fp32
    lim = 3e-3 if dtype == "bf16" else 8e-5
    assert torch.linalg.norm(a - b) <= lim * torch.linalg.norm(b)


@pytest.mark.parametrize("bits", [0, 4])
def test_tree_bad_counts_and_pages(bits):
    """A sequence that does not fit its slots or max_nodes gives zero rows and a flag; the others are right."""
    p = Plain(4, 2, 128, bits)
    got, want, c, args = run_tree(p, [20, 30, 10], [4, 5, 3], None)
    args = dict(args)
    hist = args["hist"].clone()
    hist[1] = 44                                               # 44 + 5 > 48 slots
    args["hist"] = hist
    p.L.tree_attn(**args)
    out = args["out"].to(torch.float64).cpu()
    assert p.L.sync_status() == 2
    assert torch.all(out[4:9] == 0)
    check_tree(torch.cat((out[:4], out[9:])), torch.cat((want[:4], want[9:])), "bf16")
    args["hist"], args["max_nodes"] = i32([20, 30, 10]), 4
    p.L.tree_attn(**args)
    out = args["out"].to(torch.float64).cpu()
    assert p.L.sync_status() == 2 and torch.all(out[4:9] == 0)
    check_tree(torch.cat((out[:4], out[9:])), torch.cat((want[:4], want[9:])), "bf16")
    args["max_nodes"] = 5
    pt = c.pt_d.clone()
    pt[1, 0], pt[1, 1] = -1, c.n_pages
    p.L.tree_attn(**dict(args, page_table=pt))
    out = args["out"].to(torch.float64).cpu()
    assert p.L.sync_status() == 1
    check_tree(torch.cat((out[:4], out[9:])), torch.cat((want[:4], want[9:])), "bf16")


@pytest.mark.parametrize("bits", [0, 8])
def test_tree_node_offsets_that_go_back(bits):
    """Offsets that decrease are flagged and every row is zero; a sequence outside the call's rows leaves the others."""
    p = Plain(4, 2, 128, bits)
    got, want, c, args = run_tree(p, [20, 20, 20], [4, 5, 3], None)
    for off in ([0, 4, 0, 3], [0, 12, 4, 12], [0, 4, 4, 40], [-5, 4, 9, 12], [0, 4, 2 ** 31 - 1, -2 ** 31]):
        args["node_off"] = i32(off)
        args["max_nodes"] = 12
        ws = torch.empty(p.L.tree_workspace_bytes(3, c.pt.shape[1] * 16, 12, 12), dtype=torch.uint8, device="cuda")
        p.L.tree_attn(**dict(args, workspace=ws))
        assert p.L.sync_status() == 2, off
        if off == [0, 4, 4, 40]:
            check_tree(args["out"][:4].to(torch.float64).cpu(), want[:4], "bf16")
        elif any(b < a for a, b in zip(off, off[1:])):
            assert torch.all(args["out"][:max(off[-1], 0)] == 0)


@pytest.mark.parametrize("bits,H,hkv", [(8, 4, 4), (4, 8, 2), (8, 16, 1), (4, 40, 2)])
def test_decode_quantised(bits, H, hkv):
    """starkv_decode_attn over codes: lengths from none to long, query positions given or not."""
    p = Plain(H, hkv, 128, bits)
    lens = [0, 1, 16, 17, 700, 33, 2500]
    c = p.cache(lens)
    for b, n in enumerate(lens):
        if n:
            c.fill(b, n)
    q = p.r(torch.randn(7, H, 128, generator=torch.Generator().manual_seed(1)))
    ws = torch.empty(p.L.workspace_bytes(7, c.pt.shape[1] * 16), dtype=torch.uint8, device="cuda").random_(0, 255)
    for pos, path in ((None, 0), ([3, 5, 9, 16, 10000, 1, 2499], 0), (None, 1)):
        p.L.set_decode_path(path)
        out = torch.empty(7, p.hidden, dtype=p.dt, device="cuda")
        p.L.decode(c.upload(), c.n_pages, c.pt_d, i32(lens), q.to(p.dt).cuda(), out, ws,
                   q_pos=None if pos is None else i32(pos))
        qx = p.norm_rope(q, p.wq, torch.tensor(pos if pos else [n - 1 for n in lens]))
        want = torch.cat([R.attention(qx[b:b + 1], c.K[b], c.V[b], torch.ones(1, n, dtype=torch.bool), 128 ** -0.5)
                          @ p.W_o if n else torch.zeros(1, p.hidden, dtype=torch.float64) for b, n in enumerate(lens)])
        check_tree(out.to(torch.float64).cpu(), want, "bf16")
        assert torch.all(out[0] == 0)
    assert p.L.sync_status() == 0
    p.L.set_decode_path(0)
    p.L.decode(c.pool, c.n_pages, c.pt_d, i32([-1] + lens[1:6] + [5000]), q.to(p.dt).cuda(), out, ws)
    assert p.L.sync_status() == 2


@pytest.mark.parametrize("cfg,quantized", [(1, False), (2, True), (3, True)])
def test_tree_latent_layer(cfg, quantized):
    """Latent layers: a node's output is the decode of a sequence that ends with its path, at the same positions."""
    spec = gen.config_spec(cfg, quantized=quantized)
    c = Case(spec, 7)
    L = c.load()
    hist, n = 70, 9
    sees, depth = R.random_tree(random.Random(5), n)
    Z = c.latents_direct(0, hist + n)
    paths = [sorted(s) for s in sees]
    cache = GpuCache(L, [hist + n] + [hist + len(x) for x in paths])
    cache.append_latents(0, Z)
    for i, x in enumerate(paths):
        cache.append_latents(1 + i, [np.concatenate((z[:hist], z[hist:][x])) for z in Z])
    g = torch.Generator().manual_seed(2)
    q = (torch.randn(n, spec.n_heads, spec.head_dim, generator=g) / spec.head_dim ** 0.5 * 3).to(torch.bfloat16).cuda()
    out, want = (torch.empty(n, spec.hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mp = cache.page_table.shape[1]
    ws = torch.empty(max(L.tree_workspace_bytes(1, mp * 16, n, n), L.workspace_bytes(n, mp * 16)), dtype=torch.uint8,
                     device="cuda")
    pos = i32([hist + d for d in depth])
    L.tree_attn(cache.pool, cache.n_pages, cache.page_table[:1], i32([hist]), i32([0, n]), q, out, ws, max_nodes=n,
                mask=R.mask_words(sees, 1).cuda(), q_pos=pos)
    L.set_decode_path(1)
    L.decode(cache.pool, cache.n_pages, cache.page_table[1:].contiguous(), i32([hist + len(x) for x in paths]), q, want,
             ws)
    assert L.sync_status() == 0
    a, b = out.to(torch.float64).cpu().numpy(), want.to(torch.float64).cpu().numpy()
    # both are rounded to bf16: sqrt(2) * 1.6e-3, and single values by a step of 2^-7
    assert np.linalg.norm(a - b) <= 3e-3 * np.linalg.norm(b)
    assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max()


# ------------------------------------------------------------------ keeping the accepted path

@pytest.mark.parametrize("layer", ["q8", "q4", "bf16", "f32", "latent_43", "latent_bf16", "latent_gqa"])
def test_accept_leaves_the_pool_of_a_linear_append(layer):
    """After accept, the pool is byte for byte one into which only the accepted tokens were appended."""
    hist, counts = [37, 0, 250, 15], [9, 20, 64, 0]
    rng = random.Random(11)
    accs = [sorted(rng.sample(range(n), k)) for n, k in zip(counts, (4, 20, 31, 0))]
    accs[0][0] = 0
    if layer.startswith("latent"):
        cfg, quant = {"latent_43": (2, True), "latent_bf16": (1, False), "latent_gqa": (3, True)}[layer]
        c = Case(gen.config_spec(cfg, quantized=quant), 5)
        L, Z = c.load(), [c.latents_direct(b, h + n) for b, (h, n) in enumerate(zip(hist, counts))]
    else:
        bits = {"q8": 8, "q4": 4}.get(layer, 0)
        L = Plain(4, 2, 128, bits, "f32" if layer == "f32" else "bf16").L
        gg = np.random.default_rng(0)
        Z = [[gg.standard_normal((h + n, w)).astype(np.float32) for w in (128, 128, 256)] for h, n in zip(hist, counts)]
    full, lin = (GpuCache(L, [h + n for h, n in zip(hist, counts)], seed=3) for _ in range(2))
    for b in range(4):
        full.append_latents(b, Z[b])
        keep = list(range(hist[b])) + [hist[b] + j for j in accs[b]]
        lin.append_latents(b, [z[keep] for z in Z[b]])
    acc = sum([a + [-1] * (n - len(a)) for a, n in zip(accs, counts)], [])
    off = np.cumsum([0] + counts)
    L.tree_accept(full.pool, full.n_pages, full.page_table, i32(hist), i32(off), i32(acc),
                  i32([len(a) for a in accs]), max_nodes=64)
    assert L.sync_status() == 0
    np.testing.assert_array_equal(full.pool_pages(), lin.pool_pages())


def test_accept_refuses_a_path_that_is_none():
    p = Plain(2, 2, 128, 8)
    c = p.cache([40, 40, 40, 40, 40])
    for b in range(5):
        c.fill(b, 30)
    c.upload()
    before = c.download().clone()
    acc = [2, 2, -1] + [1, 0, -1] + [0, 3, -1] + [0, 1, 2] + [0, 1, 2]
    p.L.tree_accept(c.pool, c.n_pages, c.pt_d, i32([27] * 4 + [46]), i32([0, 3, 6, 9, 12, 15]), i32(acc),
                    i32([2, 2, 2, 4, 3]), max_nodes=3)
    assert p.L.sync_status() == 2
    assert torch.equal(c.download(), before)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("bits,dtype", [(8, "bf16"), (4, "bf16"), (0, "bf16"), (8, "f32")])
def test_speculative_rounds(bits, dtype):
    """Prompt by append_qkv and prefill, then rounds of drafts: append, verify, accept; at every step the cache and the
    outputs are those of the sequence decoded token by token."""
    p = Plain(4, 2, 128, bits, dtype)
    rng = random.Random(4)
    g = torch.Generator().manual_seed(4)
    H, hkv, d, B = 4, 2, 128, 2
    c = p.cache([150] * B)
    pool = c.upload()
    mp = c.pt.shape[1]
    Ks, Vs = [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(B)], [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(B)]
    lens = [33, 20]

    def make(n):
        return p.r(torch.randn(n, (H + 2 * hkv) * d, generator=g))

    def split(x):
        t = x.to(p.dt).cuda()
        return t[:, :H * d], t[:, H * d:(H + hkv) * d], t[:, (H + hkv) * d:]

    def kv(x, pos):
        K = p.norm_rope(x[:, H * d:(H + hkv) * d].reshape(-1, hkv, d), p.wk, pos)
        V = x[:, (H + hkv) * d:].reshape(-1, hkv, d)
        return R.stored(K, bits, p.dt), R.stored(V.reshape(len(x), -1), bits, p.dt).reshape(V.shape)

    x = [make(n) for n in lens]
    xs = torch.cat(x)
    seq, slots = torch.tensor([0] * 33 + [1] * 20), torch.cat([torch.arange(n) for n in lens])
    p.L.append_qkv(pool, c.n_pages, c.pt_d, i32(seq), i32(slots), None, *split(xs)[1:])
    out = torch.empty(53, p.hidden, dtype=p.dt, device="cuda")
    ws = torch.empty(max(p.L.workspace_bytes(B, mp * 16, 33), p.L.tree_workspace_bytes(B, mp * 16, 64, 32)),
                     dtype=torch.uint8, device="cuda")
    p.L.prefill(pool, c.n_pages, c.pt_d, [0, 0], lens, split(xs)[0].contiguous(), out, ws)
    want = []
    for b in range(B):
        Ks[b], Vs[b] = kv(x[b], torch.arange(lens[b]))
        qx = p.norm_rope(x[b][:, :H * d].reshape(-1, H, d), p.wq, torch.arange(lens[b]))
        see = torch.ones(lens[b], lens[b], dtype=torch.bool).tril()
        want.append(R.attention(qx, Ks[b], Vs[b], see, d ** -0.5) @ p.W_o)
    check_tree(out.to(torch.float64).cpu(), torch.cat(want), dtype)
    for step in range(4):
        counts = [rng.randint(1, 20) for _ in range(B)]
        trees = [R.random_tree(rng, n) for n in counts]
        off = [0, counts[0], sum(counts)]
        x = [make(n) for n in counts]
        pos = [torch.tensor([lens[b] + k for k in trees[b][1]]) for b in range(B)]
        seq = torch.tensor([0] * counts[0] + [1] * counts[1])
        slots = torch.cat([lens[b] + torch.arange(counts[b]) for b in range(B)])
        q, k, v = split(torch.cat(x))
        qo = torch.empty(off[-1], H * d, dtype=p.dt, device="cuda")
        p.L.append_qkv(pool, c.n_pages, c.pt_d, i32(seq), i32(slots), q, k, v, q_out=qo, positions=i32(torch.cat(pos)))
        out = torch.empty(off[-1], p.hidden, dtype=p.dt, device="cuda")
        p.L.tree_attn(pool, c.n_pages, c.pt_d, i32(lens), i32(off), qo, out, ws, max_nodes=32,
                      mask=R.mask_words(trees[0][0] + trees[1][0], 1).cuda())
        want, accs = [], []
        for b in range(B):
            Kn, Vn = kv(x[b], pos[b])
            see = torch.ones(counts[b], lens[b] + counts[b], dtype=torch.bool)
            for i in range(counts[b]):
                for j in range(counts[b]):
                    see[i, lens[b] + j] = j in trees[b][0][i]
            qx = p.r(p.norm_rope(x[b][:, :H * d].reshape(-1, H, d), p.wq, pos[b]).to(torch.float32))
            want.append(R.attention(qx, torch.cat((Ks[b], Kn)), torch.cat((Vs[b], Vn)), see, d ** -0.5) @ p.W_o)
            path = sorted(trees[b][0][rng.randrange(counts[b])])[:rng.randint(0, 4)]
            accs.append(path)
            Ks[b], Vs[b] = torch.cat((Ks[b], Kn[path])), torch.cat((Vs[b], Vn[path]))
        check_tree(out.to(torch.float64).cpu(), torch.cat(want), dtype)
        acc = sum([a + [0] * (n - len(a)) for a, n in zip(accs, counts)], [])
        p.L.tree_accept(pool, c.n_pages, c.pt_d, i32(lens), i32(off), i32(acc), i32([len(a) for a in accs]), max_nodes=32)
        lens = [n + len(a) for n, a in zip(lens, accs)]
    # the next token of each, by the decode call, after an append from hidden states
    h = p.r(torch.randn(B, p.hidden, generator=g))
    ws2 = torch.empty(max(256, p.L.append_workspace_bytes(B)), dtype=torch.uint8, device="cuda")
    p.L.append(pool, c.n_pages, c.pt_d, i32([0, 1]), i32(lens), h.to(p.dt).cuda(), False, workspace=ws2)
    row = torch.empty(B, 2 * hkv * d, dtype=p.dt, device="cuda")
    p.L.cache_read(pool, c.n_pages, c.pt_d, i32([0, 1]), i32(lens), row)
    q = p.r(torch.randn(B, H, d, generator=g))
    out = torch.empty(B, p.hidden, dtype=p.dt, device="cuda")
    p.L.decode(pool, c.n_pages, c.pt_d, i32([n + 1 for n in lens]), q.to(p.dt).cuda(), out, ws)
    r = row.to(torch.float64).cpu()
    for b in range(B):
        K1 = p.norm_rope((h[b:b + 1] @ p.W_k).reshape(1, hkv, d), p.wk, torch.tensor([lens[b]]))
        # a stored key is off by half a step of its group, the cache's rounding and the projection's fp16 operands
        step = K1.reshape(1, hkv * d).abs().max() / ((2 ** (bits - 1) - 1) if bits else 128)
        assert (r[b, :hkv * d] - K1.reshape(-1)).abs().max() <= 0.5 * step + 0.02 * K1.abs().max()
        K = torch.cat((Ks[b], r[b:b + 1, :hkv * d].reshape(1, hkv, d)))
        V = torch.cat((Vs[b], r[b:b + 1, hkv * d:].reshape(1, hkv, d)))
        qx = p.norm_rope(q[b:b + 1], p.wq, torch.tensor([lens[b]]))
        see = torch.ones(1, lens[b] + 1, dtype=torch.bool)
        check_tree(out[b:b + 1].to(torch.float64).cpu(), R.attention(qx, K, V, see, d ** -0.5) @ p.W_o, dtype)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [0, 8])
def test_pages_beyond_4_gib(bits):
    """Append, read, attention and accept on pages whose byte offsets pass 32 bits."""
    H = hkv = 32
    p = Plain(H, hkv, 128, bits)
    n_pages = (9 << 29) // p.L.page_bytes + 8                   # 4.5 GiB
    pool = torch.empty(n_pages * p.L.page_bytes, dtype=torch.uint8, device="cuda")
    pt = i32([[n_pages - 1, n_pages - 4, n_pages - 3], [n_pages - 6, 0, n_pages - 2]])
    g = torch.Generator().manual_seed(0)
    n = 48
    x = p.r(torch.randn(2 * n, 3 * H * 128, generator=g))
    seq, slots = i32([0] * n + [1] * n), i32(list(range(n)) * 2)
    xd = x.to(p.dt).cuda()
    parts = [xd[:, i * H * 128:(i + 1) * H * 128] for i in range(3)]
    p.L.append_qkv(pool, n_pages, pt, seq, slots, None, *parts[1:])
    out = torch.empty(2 * n, 2 * H * 128, dtype=p.dt, device="cuda")
    p.L.cache_read(pool, n_pages, pt, seq, slots, out)
    K = p.norm_rope(x[:, H * 128:2 * H * 128].reshape(-1, H, 128), p.wk, torch.arange(n).repeat(2))
    V = R.stored(x[:, 2 * H * 128:], bits, p.dt).reshape(-1, H, 128)
    if bits:
        K = R.stored(K, bits, p.dt)
        assert torch.equal(out[:, :H * 128].cpu(), K.reshape(2 * n, -1).to(torch.float32).to(p.dt))
    else:
        close_rows(out[:, :H * 128].reshape(-1, H, 128), K, pair_size(K), p.dt)
    assert torch.equal(out[:, H * 128:].cpu(), V.reshape(2 * n, -1).to(torch.float32).to(p.dt))
    k, hist = 7, n - 7
    q = p.r(torch.randn(2 * k, H, 128, generator=g))
    y = torch.empty(2 * k, p.hidden, dtype=p.dt, device="cuda")
    ws = torch.empty(p.L.tree_workspace_bytes(2, 48, 2 * k, k), dtype=torch.uint8, device="cuda")
    p.L.tree_attn(pool, n_pages, pt, i32([hist, hist]), i32([0, k, 2 * k]), q.to(p.dt).cuda(), y, ws, max_nodes=k)
    kd = out[:, :H * 128].to(torch.float64).cpu().reshape(-1, H, 128)
    see = torch.arange(n)[None] <= torch.arange(k)[:, None] + hist
    want = torch.cat([R.attention(q[b * k:(b + 1) * k], (K if bits else kd)[b * n:(b + 1) * n], V[b * n:(b + 1) * n], see,
                                  128 ** -0.5) @ p.W_o for b in range(2)])
    check_tree(y.to(torch.float64).cpu(), want, "bf16")
    p.L.tree_accept(pool, n_pages, pt, i32([hist, hist]), i32([0, k, 2 * k]), i32([1, 3, 6, 0, 0, 0, 0] * 2), i32([3, 3]),
                    max_nodes=k)
    after = torch.empty_like(out)
    p.L.cache_read(pool, n_pages, pt, seq, slots, after)
    for b in range(2):
        o = b * n
        assert torch.equal(after[o:o + hist], out[o:o + hist])
        assert torch.equal(after[o + hist:o + hist + 3], out[[o + hist + 1, o + hist + 3, o + hist + 6]])
        assert torch.all(after[o + hist + 3:o + n] == 0)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [0, 8, 4])
def test_append_and_read_captured(bits):
    """One graph of append_qkv and cache_read, replayed with other rows and slots."""
    p = Plain(4, 2, 128, bits)
    c = p.cache([64, 64])
    pool = c.upload()
    n = 9
    x = torch.zeros(n, 8 * 128, dtype=p.dt, device="cuda")
    seq, slots = i32([0] * n), i32(range(n))
    qo, out = torch.empty(n, 512, dtype=p.dt, device="cuda"), torch.empty(n, 512, dtype=p.dt, device="cuda")

    def calls():
        p.L.append_qkv(pool, c.n_pages, c.pt_d, seq, slots, x[:, :512], x[:, 512:768], x[:, 768:], q_out=qo)
        p.L.cache_read(pool, c.n_pages, c.pt_d, seq, slots, out)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        xv = p.r(torch.randn(n, 1024, generator=torch.Generator().manual_seed(k)))
        sl = torch.randperm(64, generator=torch.Generator().manual_seed(k))[:n]
        x.copy_(xv.to(p.dt))
        slots.copy_(i32(sl))
        seq.copy_(i32([k % 2] * n))
        graph.replay()
        torch.cuda.synchronize()
        K = p.norm_rope(xv[:, 512:768].reshape(n, 2, 128), p.wk, sl)
        w = p.norm_rope(xv[:, :512].reshape(n, 4, 128), p.wq, sl)
        close_rows(qo.reshape(n, 4, 128), w, pair_size(w), p.dt)
        if bits:
            kv = torch.cat((R.stored(K, bits, p.dt).reshape(n, -1), R.stored(xv[:, 768:], bits, p.dt)), -1)
            assert torch.equal(out.cpu(), kv.to(torch.float32).to(p.dt))
        else:
            close_rows(out[:, :256].reshape(n, 2, 128), K, pair_size(K), p.dt)
    assert p.L.sync_status() == 0
    del graph


@pytest.mark.parametrize("bits", [0, 8, 4])
def test_calls_on_two_streams(bits):
    """Two calls at once on one layer, each with its own cache and workspace."""
    p = Plain(4, 2, 128, bits)
    runs = [run_tree(p, [700 + 40 * k, 33], [9, 20 + k], None, seed=k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (_, _, _, args), s in zip(runs, streams):
            args["out"].zero_()
        torch.cuda.synchronize()
        for (_, _, _, args), s in zip(runs, streams):
            p.L.tree_attn(**args, stream=s)
        torch.cuda.synchronize()
        for got, want, _, args in runs:
            assert torch.equal(args["out"].to(torch.float64).cpu(), got)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits,n,hist", [(8, 40, 3000), (4, 300, 1000), (0, 33, 500)])
def test_prefill_quantised(bits, n, hist):
    """starkv_prefill_attn after a history: the definition's causal attention over the stored values."""
    p = Plain(4, 2, 128, bits)
    c = p.cache([hist + n])
    c.fill(0, hist + n)
    q = p.r(torch.randn(n, 4, 128, generator=torch.Generator().manual_seed(3)))
    out = torch.empty(n, p.hidden, dtype=p.dt, device="cuda")
    ws = torch.empty(p.L.workspace_bytes(1, c.pt.shape[1] * 16, n), dtype=torch.uint8, device="cuda")
    p.L.prefill(c.upload(), c.n_pages, c.pt_d, [hist], [n], q.to(p.dt).cuda(), out, ws)
    qx = p.norm_rope(q, p.wq, torch.arange(n) + hist)
    see = torch.arange(hist + n)[None] <= torch.arange(n)[:, None] + hist
    check_tree(out.to(torch.float64).cpu(), R.attention(qx, c.K[0], c.V[0], see, 128 ** -0.5) @ p.W_o, "bf16")
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [0, 8, 4])
def test_tree_and_accept_captured(bits):
    """One graph, replayed with other lengths, masks and paths in the same buffers; on a stream of its own."""
    p = Plain(4, 2, 128, bits)
    rng = random.Random(9)
    c = p.cache([200, 200])
    s = torch.cuda.Stream()
    hist, off = i32([0, 0]), i32([0, 0, 0])
    n = 24
    mask, pos = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    q, out = torch.zeros(n, 4, 128, dtype=p.dt, device="cuda"), torch.zeros(n, p.hidden, dtype=p.dt, device="cuda")
    acc, n_acc = torch.zeros(n, dtype=torch.int32, device="cuda"), i32([0, 0])
    ws = torch.empty(p.L.tree_workspace_bytes(2, 13 * 16, n, 16), dtype=torch.uint8, device="cuda")
    for b in range(2):
        c.fill(b, 150)
    c.upload()
    with torch.cuda.stream(s):
        p.L.tree_attn(c.pool, c.n_pages, c.pt_d, hist, off, q, out, ws, max_nodes=16, mask=mask, q_pos=pos)
        p.L.tree_accept(c.pool, c.n_pages, c.pt_d, hist, off, acc, n_acc, max_nodes=16)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            p.L.tree_attn(c.pool, c.n_pages, c.pt_d, hist, off, q, out, ws, max_nodes=16, mask=mask, q_pos=pos)
            p.L.tree_accept(c.pool, c.n_pages, c.pt_d, hist, off, acc, n_acc, max_nodes=16)
    for lens, counts in (([100, 140], [8, 9]), ([17, 0], [16, 8]), ([134, 140], [1, 0])):
        c.pool.copy_(c.pages.reshape(-1))
        trees = [R.random_tree(rng, k) for k in counts]
        m = R.mask_words(trees[0][0] + trees[1][0], 1)
        qv = p.r(torch.randn(n, 4, 128))
        hist.copy_(i32(lens))
        off.copy_(i32([0, counts[0], sum(counts)]))
        mask[:len(m)].copy_(m)
        po = torch.cat([lens[b] + torch.tensor(trees[b][1], dtype=torch.long) for b in range(2)])
        pos[:len(po)].copy_(po)
        q.copy_(qv.to(p.dt))
        paths = [sorted(t[0][-1]) if t[0] else [] for t in trees]
        acc[:sum(counts)].copy_(i32(sum([a + [0] * (k - len(a)) for a, k in zip(paths, counts)], [])))
        n_acc.copy_(i32([len(a) for a in paths]))
        out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        o = 0
        for b in range(2):
            k = counts[b]
            see = torch.ones(k, lens[b] + k, dtype=torch.bool)
            for i in range(k):
                for j in range(k):
                    see[i, lens[b] + j] = j in trees[b][0][i]
            if k:
                qx = p.norm_rope(qv[o:o + k], p.wq, po[o:o + k])
                w = R.attention(qx, c.K[b][:lens[b] + k], c.V[b][:lens[b] + k], see, 128 ** -0.5) @ p.W_o
                check_tree(out[o:o + k].to(torch.float64).cpu(), w, "bf16")
            o += k
        assert torch.all(out[o:] == 5.0)
        got = torch.empty(len(paths[0]), 512, dtype=p.dt, device="cuda")
        t = torch.arange(len(paths[0])) + lens[0]
        p.L.cache_read(c.pool, c.n_pages, c.pt_d, i32([0] * len(t)), i32(t), got)
        kv = torch.cat((c.K[0].reshape(150, -1), c.V[0].reshape(150, -1)), -1)[[lens[0] + j for j in paths[0]]]
        assert torch.equal(got.cpu(), kv.to(torch.float32).to(p.dt))
    assert p.L.sync_status() == 0
    del graph
