"""The serving operators over their whole range: values at both ends of what the codes hold, what a row sees of values
that are not finite on every kernel, rows that see nothing, blocks of three row tiles, prefills of many
tiles, and workspaces of the largest call.

Tolerances of bf16 layers (check_tree): 3e-3 in relative L2, 1e-2 of the largest output.  The output's rounding is 1.6e-3;
q, a weight, a dequantised value (|error| <= 2^-11 of itself, and none for scales below the smallest normal fp16, whose
products are multiples of 2^-24) and y are each rounded to fp16: below 4e-4 each.  Scaling all values by one number
scales y and the output with it, so these bounds do not depend on it as long as y stays a normal fp16 number (6.1e-5 to
65504); below that y is off by up to 2^-25, which the tests of small values add up themselves.
"""
import math
import random

import numpy as np
import pytest
import torch

import serving_ref as R
from harness import Case, GpuCache
from synth import gen
from test_serving_gpu import Plain, check_tree, i32

pytestmark = pytest.mark.gpu


def put(c, b, K, V):
    """Tokens K, V [n, hkv, d] (float64) at the end of sequence b, by the definition's packer."""
    p, n = c.p, len(K)
    t = torch.arange(len(c.K[b]), len(c.K[b]) + n)
    R.put(c.pages, c.pt[b, t // 16], t % 16, K, V, p.bits, p.dt)
    c.K[b] = torch.cat((c.K[b], R.stored(K, p.bits, p.dt)))
    c.V[b] = torch.cat((c.V[b], R.stored(V.reshape(n, -1), p.bits, p.dt).reshape(n, p.hkv, p.d)))


def seen(hist, n, sets):
    see = torch.ones(n, hist + n, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            see[i, hist + j] = j in sets[i] if sets is not None else j <= i
    return see


def tree(p, c, hist, counts, masks, q):
    """One tree call of queries q [n, H, d] that need no rotation, and the definition: (out, want, call arguments)."""
    off = np.cumsum([0] + counts).tolist()
    want = []
    for b, (h, k) in enumerate(zip(hist, counts)):
        y = R.attention(q[off[b]:off[b + 1]], c.K[b], c.V[b], seen(h, k, masks[b] if masks else None), p.d ** -0.5)
        want.append(y @ p.W_o)
    words = max(1, -(-max(counts) // 32))
    out = torch.full((off[-1], p.hidden), 9.0, dtype=p.dt, device="cuda")
    ws = torch.empty(p.L.tree_workspace_bytes(len(hist), c.pt.shape[1] * 16, off[-1], max(counts)), dtype=torch.uint8,
                     device="cuda").random_(0, 255)
    args = dict(pool=c.upload(), n_pages=c.n_pages, page_table=c.pt_d, hist=i32(hist), node_off=i32(off), q=q.to(p.dt).cuda(),
                out=out, workspace=ws, max_nodes=max(counts),
                mask=R.mask_words(sum(masks, []), words).cuda() if masks else None)
    p.L.tree_attn(**args)
    return out.to(torch.float64).cpu(), torch.cat(want), args


# rows per KV head: 1, 8, 16, 24 (blocks of 8, 16 and 24 rows), 32 (blocks of 128)
ROWS = [(1, 1), (4, 2), (4, 4), (4, 6), (4, 8)]


# ------------------------------------------------------------------ values at the ends of the codes' range

@pytest.mark.parametrize("kind", ["random", "rising"])
@pytest.mark.parametrize("group,n", ROWS)
@pytest.mark.parametrize("bits", [8, 4])
def test_tree_of_the_largest_values(bits, group, n, kind):
    """Values up to 32000 (the codes hold 32768): every weight times its scale stays finite.  rising: scores that go up by
    0.04 (log2) a token, so that the running maximum lags behind them."""
    p = Plain(2 * group, 2, 128, bits, norm=False, rope=False)
    hist, counts = [700, 333], [n, max(1, n - 1)]
    c = p.cache([h + k for h, k in zip(hist, counts)])
    g = torch.Generator().manual_seed(bits + n)
    base = torch.where(torch.rand(128, generator=g) < 0.5, -1.0, 1.0).to(torch.float64)
    q = p.r(torch.randn(sum(counts), p.H, 128, generator=g) * (0.3 if kind == "rising" else 1) + (base if kind == "rising" else 0))
    for b in range(2):
        T = hist[b] + counts[b]
        K = torch.randn(T, 2, 128, generator=g, dtype=torch.float64)
        if kind == "rising":
            # a step of base * x in K moves a score by 128 x log2(e) / sqrt(128) = 16.3 x
            K = 0.1 * K + base * (torch.arange(T) * (0.04 / 16.3))[:, None, None]
        V = torch.randn(T, 2, 128, generator=g, dtype=torch.float64)
        put(c, b, K, V * (32000.0 / V.abs().max()))
    rng = random.Random(n)
    for masks in ([R.random_tree(rng, k)[0] for k in counts], None):
        got, want, _ = tree(p, c, hist, counts, masks, q)
        check_tree(got, want, "bf16")
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("H,hkv", [(2, 2), (8, 1), (16, 1), (24, 1), (40, 1)])
@pytest.mark.parametrize("bits", [8, 4])
def test_decode_of_the_largest_values(bits, H, hkv):
    p = Plain(H, hkv, 128, bits, norm=False)
    lens = [1, 17, 900]
    c = p.cache(lens)
    g = torch.Generator().manual_seed(H)
    for b, T in enumerate(lens):
        K, V = (torch.randn(T, hkv, 128, generator=g, dtype=torch.float64) for _ in range(2))
        put(c, b, K, V * (32000.0 / V.abs().max()))
    q = p.r(torch.randn(3, H, 128, generator=g))
    ws = torch.empty(p.L.workspace_bytes(3, c.pt.shape[1] * 16), dtype=torch.uint8, device="cuda").random_(0, 255)
    out = torch.empty(3, p.hidden, dtype=p.dt, device="cuda")
    p.L.decode(c.upload(), c.n_pages, c.pt_d, i32(lens), q.to(p.dt).cuda(), out, ws)
    qx = p.norm_rope(q, None, torch.tensor(lens) - 1)
    want = torch.cat([R.attention(qx[b:b + 1], c.K[b], c.V[b], torch.ones(1, T, dtype=torch.bool), 128 ** -0.5) @ p.W_o
                      for b, T in enumerate(lens)])
    check_tree(out.to(torch.float64).cpu(), want, "bf16")
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("size,gap", [(1e-2, 15.5), (1e-3, 12.0)])
@pytest.mark.parametrize("group,n", ROWS)
@pytest.mark.parametrize("bits", [8, 4])
def test_tree_of_small_values_beside_a_dominant_token(bits, group, n, size, gap):
    """Every 128th token has nearly all of the weight and the value 0; the others, 2^-gap of its weight each, make up y:
    about 127 2^-gap size = 2.7e-5 or 3.1e-5, whose fp16 rounding of at most 2^-25 is 1.1e-3 of it (7e-4 rms).

    Blocks of 128 rows hold code * scale of the keys in fp16.  The dominant token's key has one magnitude in every
    channel (base * gap / 16.3: one code and one scale), so its roundings, up to 2^-11 of the value, all have one sign and
    move its score, gap above the others in log2 units, by up to gap * 2^-11: gap * ln 2 * 2^-11 of every other weight
    (5.2e-3 and 4.1e-3), and of y.  Blocks of up to 24 rows score with the codes themselves."""
    p = Plain(2 * group, 2, 128, bits, norm=False, rope=False)
    hist, counts = [4096 - n, 4096 - n], [n, n]
    c = p.cache([4096, 4096])
    g = torch.Generator().manual_seed(n)
    base = torch.where(torch.rand(128, generator=g) < 0.5, -1.0, 1.0).to(torch.float64)
    q = p.r(torch.randn(2 * n, p.H, 128, generator=g) * 0.1 + base)
    for b in range(2):
        K = 0.3 * torch.randn(4096, 2, 128, generator=g, dtype=torch.float64)
        V = size * (1 + 0.3 * torch.randn(4096, 2, 128, generator=g, dtype=torch.float64))
        K[::128] = base * (gap / 16.3)
        V[::128] = 0
        put(c, b, K, V)
    got, want, _ = tree(p, c, hist, counts, None, q)
    key = gap * math.log(2) * 2.0 ** -11 if group * n >= 25 else 0.0
    assert torch.linalg.norm(got - want) <= (3e-3 + key) * torch.linalg.norm(want)
    assert (got - want).abs().max() <= (1e-2 + key) * want.abs().max()
    assert p.L.sync_status() == 0


# ------------------------------------------------------------------ values that are not finite, rows that see nothing

# bf16 with head_dim 128 has kernels of its own (5 and 33 nodes of 4 heads a KV head: one of them each); the other layers
# take the row kernels
PLAIN = [("f32", 128, 2, 5), ("f32", 64, 2, 5), ("bf16", 64, 2, 5), ("bf16", 256, 1, 5), ("bf16", 80, 3, 5), ("bf16", 128, 1, 5),
         ("bf16", 128, 4, 33)]


def not_finite(call, plant, T, hist, sees):
    """call() -> out after plant(token, side, value, low) wrote `value` into one channel of a token's key (side 0) or value
    (side 1); low: its key makes the token's weight underflow.  Rows that see the token are infinite or NaN, the others
    are as they were."""
    clean = call()
    assert torch.isfinite(clean).all()
    n = len(sees)
    for tok in (3, hist - 1, hist + 2):
        rows = torch.tensor([tok < hist or tok - hist in s for s in sees])
        assert rows.any()
        for side, value, low in ((0, float("nan"), False), (1, float("nan"), False), (1, float("inf"), False),
                                 (1, -float("inf"), False), (1, float("nan"), True)):
            restore = plant(tok, side, value, low)
            got = call()
            restore()
            bad = ~torch.isfinite(got).all(1)
            assert torch.equal(bad, rows), (tok, side, value, low)
            assert torch.equal(got[~rows], clean[~rows])
    assert torch.equal(call(), clean)


@pytest.mark.parametrize("dtype,d,group,n", PLAIN)
def test_tree_rows_that_see_a_value_that_is_not_finite(dtype, d, group, n):
    """Over 1300 tokens: the row kernels split them, and the other splits are finite."""
    hkv, hist = 2, 1300
    p = Plain(hkv * group, hkv, d, 0, dtype, norm=False, rope=False)
    c = p.cache([hist + n])
    g = torch.Generator().manual_seed(d)
    base = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0).to(torch.float64)
    q = p.r(0.3 * torch.randn(n, p.H, d, generator=g) + base)
    K, V = (torch.randn(hist + n, hkv, d, generator=g, dtype=torch.float64) for _ in range(2))
    put(c, 0, K, V)
    rng = random.Random(d)
    sees = R.random_tree(rng, n)[0]
    sees[1], sees[2], sees[3] = {0, 1}, {0, 2}, {1, 3}
    _, want, args = tree(p, c, [hist], [n], [sees], q)

    def call():
        p.L.tree_attn(**dict(args, pool=c.upload()))
        return args["out"].to(torch.float64).cpu()

    def plant(tok, side, value, low):
        k, v = c.K[0][tok:tok + 1].clone(), c.V[0][tok:tok + 1].clone()
        if low:   # a score of -1.44 d 300 / (16 sqrt(d)) = -27 sqrt(d) or less: its weight is below the smallest fp32
            k = (-300.0 / 16 * base).expand_as(k).clone()
        (v if side else k)[0, :, d // 2] = value
        at = c.pt[0, tok // 16:tok // 16 + 1], torch.tensor([tok % 16])
        before = c.pages.clone()
        R.put(c.pages, *at, k, v, 0, p.dt)

        def restore():
            c.pages.copy_(before)
        return restore

    check_tree(call(), want, dtype)
    not_finite(call, plant, hist + n, hist, sees)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("cfg", [1, 3])
def test_tree_of_a_latent_layer_and_values_that_are_not_finite(cfg):
    spec = gen.config_spec(cfg, quantized=False)
    case = Case(spec, 11)
    L = case.load()
    hist, n = 1100, 5
    Z = case.latents_direct(0, hist + n)
    sees = [{0}, {0, 1}, {0, 2}, {1, 3}, {0, 2, 4}]
    cache = GpuCache(L, [hist + n])
    cache.append_latents(0, Z)
    g = torch.Generator().manual_seed(2)
    q = (torch.randn(n, spec.n_heads, spec.head_dim, generator=g) / spec.head_dim ** 0.5 * 3).to(torch.bfloat16).cuda()
    out = torch.empty(n, spec.hidden, dtype=torch.bfloat16, device="cuda")
    mp = cache.page_table.shape[1]
    ws = torch.empty(L.tree_workspace_bytes(1, mp * 16, n, n), dtype=torch.uint8, device="cuda")

    def call():
        L.tree_attn(cache.pool, cache.n_pages, cache.page_table[:1], i32([hist]), i32([0, n]), q, out, ws, max_nodes=n,
                    mask=R.mask_words(sees, 1).cuda(), q_pos=i32(range(hist, hist + n)))
        return out.to(torch.float64).cpu()

    def write(z, tok):
        # clear the slot (a path of no nodes), then write it again
        L.tree_accept(cache.pool, cache.n_pages, cache.page_table[:1], i32([tok]), i32([0, 1]), i32([0]), i32([0]), max_nodes=1)
        cache.append_latents(0, z, start=tok)

    clean = call()
    assert torch.isfinite(clean).all()
    for tok in (3, hist - 1, hist + 2):
        rows = torch.tensor([tok < hist or tok - hist in s for s in sees])
        for side, value in ((0, float("nan")), (1, float("nan")), (1, float("inf"))):
            z = [x[tok:tok + 1].copy() for x in Z]
            for x in (z[-1:] if side else z[:-1]):
                x[0, 1] = value
            write(z, tok)
            got = call()
            write([x[tok:tok + 1] for x in Z], tok)
            assert torch.equal(~torch.isfinite(got).all(1), rows), (tok, side, value)
            assert torch.equal(got[~rows], clean[~rows])
    assert torch.equal(call(), clean)
    assert L.sync_status() == 0


@pytest.mark.parametrize("dtype,d,bits", [("f32", 128, 0), ("bf16", 64, 8), ("bf16", 256, 4), ("bf16", 80, 0), ("bf16", 128, 4)])
def test_tree_rows_that_see_nothing_on_every_kernel(dtype, d, bits):
    p = Plain(4, 2, d, bits, dtype)
    hist, counts = [0, 0, 20], [3, 2, 2]
    masks = [[set(), {1}, {0, 2}], [set(), set()], [{0}, set()]]
    c = p.cache([h + k for h, k in zip(hist, counts)])
    g = torch.Generator().manual_seed(d)
    for b in range(3):
        put(c, b, *(torch.randn(hist[b] + counts[b], 2, d, generator=g, dtype=torch.float64) for _ in range(2)))
    got, want, _ = tree(p, c, hist, counts, masks, p.r(torch.randn(7, 4, d, generator=g)))
    assert torch.all(got[0] == 0) and torch.all(got[3:5] == 0)
    check_tree(got, want, dtype)
    assert p.L.sync_status() == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,hkv,counts", [(8, 2, [5, 6, 4]), (2, 1, [12, 9, 0]), (6, 2, [8, 7, 6]), (24, 1, [1, 1, 1])])
def test_tree_of_17_to_24_rows(bits, H, hkv, counts):
    """Three tiles of 8 rows, full and not, with masks, over odd lengths."""
    p = Plain(H, hkv, 128, bits, norm=False, rope=False)
    hist = [515, 0, 33]
    c = p.cache([h + k for h, k in zip(hist, counts)])
    g = torch.Generator().manual_seed(H)
    for b in range(3):
        put(c, b, *(torch.randn(hist[b] + counts[b], hkv, 128, generator=g, dtype=torch.float64) for _ in range(2)))
    rng = random.Random(H)
    q = p.r(torch.randn(sum(counts), H, 128, generator=g))
    for masks in ([R.random_tree(rng, k)[0] for k in counts], None):
        got, want, _ = tree(p, c, hist, counts, masks, q)
        check_tree(got, want, "bf16")
    assert p.L.sync_status() == 0


# ------------------------------------------------------------------ prefill of many query tiles

@pytest.mark.parametrize("bits,H,hkv,hist,n", [(8, 32, 8, 700, 1024), (0, 32, 8, 129, 700), (4, 40, 40, 1, 640)])
def test_prefill_of_more_tiles_than_blocks(bits, H, hkv, hist, n):
    """Several (query tile, head) items per block, so that a block's warps meet the next item's tiles while others still
    write the last one's output: calls repeat to the bit, and rows at the tiles' edges and between are the definition's."""
    p = Plain(H, hkv, 128, bits, norm=False)
    c = p.cache([hist + n])
    g = torch.Generator().manual_seed(n)
    put(c, 0, *(torch.randn(hist + n, hkv, 128, generator=g, dtype=torch.float64) for _ in range(2)))
    ws = torch.empty(p.L.workspace_bytes(1, c.pt.shape[1] * 16, n), dtype=torch.uint8, device="cuda").random_(0, 255)
    out = torch.empty(n, p.hidden, dtype=p.dt, device="cuda")
    c.upload()
    for gain in (1.0, 6.0):                                      # 6: the running maximum moves by more than 8, O is rescaled
        q = p.r(torch.randn(n, H, 128, generator=g) * gain)
        qd = q.to(p.dt).cuda()
        first = None
        for _ in range(20):
            out.fill_(7)
            p.L.prefill(c.pool, c.n_pages, c.pt_d, [hist], [n], qd, out, ws)
            first = out.clone() if first is None else first
            assert torch.equal(out, first)
        rows = sorted({0, 1, 127, 128, n // 2, n - 129, n - 2, n - 1} | set(range(5, n, 61)))
        qx = p.norm_rope(q[rows], p.wq, torch.tensor(rows) + hist)
        see = torch.arange(hist + n)[None] <= torch.tensor(rows)[:, None] + hist
        want = R.attention(qx, c.K[0], c.V[0], see, 128 ** -0.5) @ p.W_o
        check_tree(first[rows].to(torch.float64).cpu(), want, "bf16")
    assert p.L.sync_status() == 0


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("bits,dtype,H,hkv", [(8, "bf16", 32, 8), (0, "bf16", 32, 8), (4, "bf16", 8, 8), (0, "f32", 4, 1)])
def test_workspace_of_the_largest_call_serves_smaller_ones(bits, dtype, H, hkv):
    p = Plain(H, hkv, 128, bits, dtype, hidden=512)
    L = p.L
    sizes = dict(batch=[1, 3, 16], ctx=[16, 640, 4096], nodes=[1, 5, 16, 17, 63, 64, 65, 255, 256, 257, 512],
                 most=[1, 2, 4, 5, 6, 7, 16, 32])
    need = {(b, t, n, m): L.tree_workspace_bytes(b, t, n, m) for b in sizes["batch"] for t in sizes["ctx"]
            for n in sizes["nodes"] for m in sizes["most"]}
    for (b, t, n, m), x in need.items():
        for (b2, t2, n2, m2), y in need.items():
            if b2 <= b and t2 <= t and n2 <= n and m2 <= m:
                assert y <= x, ((b, t, n, m), x, (b2, t2, n2, m2), y)
    dec = [L.workspace_bytes(b, 640) for b in (1, 16, 64, 255, 256, 257, 300)]
    assert dec == sorted(dec)
    # the buffer of 512 nodes in trees of up to 32, for rounds of fewer
    ws = torch.empty(L.tree_workspace_bytes(16, 48, 512, 32), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(0)
    for counts in ([16] * 16, [5] * 16, [1] * 16, [1, 0] * 8):
        hist = [48 - 16] * 16
        c = p.cache([48] * 16)
        for b in range(16):
            put(c, b, *(torch.randn(32 + counts[b], hkv, 128, generator=g, dtype=torch.float64) for _ in range(2)))
        q = p.r(torch.randn(sum(counts), H, 128, generator=g))
        _, want, args = tree(p, c, hist, counts, None, q)
        args["out"].fill_(3)
        L.tree_attn(**dict(args, workspace=ws))
        check_tree(args["out"].to(torch.float64).cpu(), want, dtype)
    assert L.sync_status() == 0


@pytest.mark.parametrize("bits,dtype,d", [(8, "bf16", 128), (4, "bf16", 64), (0, "bf16", 128), (0, "f32", 128)])
def test_prefill_of_one_query_each_in_its_workspace(bits, dtype, d):
    """Workspace sizes of max_q = 1 serve a prefill of one query per sequence, over short tables too."""
    p = Plain(4, 2, d, bits, dtype, norm=False)
    for lens in ([1], [9, 30, 16], [40]):
        B = len(lens)
        c = p.cache(lens)
        g = torch.Generator().manual_seed(B)
        for b, T in enumerate(lens):
            put(c, b, *(torch.randn(T, 2, d, generator=g, dtype=torch.float64) for _ in range(2)))
        q = p.r(torch.randn(B, 4, d, generator=g))
        out = torch.empty(B, p.hidden, dtype=p.dt, device="cuda")
        ws = torch.empty(p.L.workspace_bytes(B, c.pt.shape[1] * 16, 1), dtype=torch.uint8, device="cuda")
        p.L.prefill(c.upload(), c.n_pages, c.pt_d, [T - 1 for T in lens], [1] * B, q.to(p.dt).cuda(), out, ws)
        qx = p.norm_rope(q, None, torch.tensor(lens) - 1)
        want = torch.cat([R.attention(qx[b:b + 1], c.K[b], c.V[b], torch.ones(1, T, dtype=torch.bool), d ** -0.5) @ p.W_o
                          for b, T in enumerate(lens)])
        check_tree(out.to(torch.float64).cpu(), want, dtype)
    assert p.L.sync_status() == 0
