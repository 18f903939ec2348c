"""The serving entry points on a machine without a GPU: refusals that come before any CUDA call, and pins of the
definitions that the GPU tests compare with."""
import ctypes

import pytest
import torch

import serving_ref as R


def raw():
    from decode_attention_rank_b200 import starkv
    return starkv.raw_lib()


def buf():
    b = ctypes.create_string_buffer(4096 + 64)
    return b, (ctypes.cast(b, ctypes.c_void_p).value + 15) // 16 * 16


def err():
    return raw().starkv_last_error().decode()


BIG = (2 ** 31 - 1) // 16 + 1


def test_load_plain_refusals():
    from decode_attention_rank_b200 import starkv as sk
    ok = dict(hidden=64, n_heads=2, n_kv_heads=2, head_dim=128, plain=True)
    for cfg, kw, text in [
            (dict(ok, plain=False, key_ranks=[4, 4], value_rank=8), {}, "uncompressed"),
            (ok, dict(kv_bits=3), "kv_bits"), (ok, dict(kv_bits=16), "kv_bits"), (ok, dict(kv_bits=-4), "kv_bits"),
            (dict(ok, head_dim=80), dict(kv_bits=8), "head_dim"), (dict(ok, head_dim=32), dict(kv_bits=4), "head_dim"),
            (ok, dict(norm_eps=-1e-6), "norm_eps"), (ok, dict(norm_eps=float("nan")), "norm_eps"),
            (dict(ok, n_heads=3), {}, "multiple"), (dict(ok, page_size=8), {}, "page_size"), (ok, {}, "non-NULL")]:
        with pytest.raises(sk.StarKVError) as e:
            sk.load_plain(sk.LayerConfig(**cfg), None, None, None, stream=0, **kw)
        assert e.value.status == 1 and text in str(e.value), (cfg, kw, str(e.value))
    with pytest.raises(ValueError):
        sk.load_plain(sk.LayerConfig(**ok), None, None, None, q_norm=torch.ones(64, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        sk.load_plain(sk.LayerConfig(**ok), None, None, None, k_norm=torch.ones(128), stream=0)


def test_null_layer_and_empty_calls():
    r, (b, p) = raw(), buf()
    assert r.starkv_qk_norm_rope(None, 1, p, p, 1, p, 1, p, 1, p, 1, None) == 1
    assert r.starkv_append_qkv(None, p, 1, p, 1, 1, 1, p, p, p, p, 1, p, 1, p, 1, p, 1, None) == 1
    assert r.starkv_cache_read(None, p, 1, p, 1, 1, 1, p, p, p, None) == 1
    assert r.starkv_tree_attn(None, p, 1, p, 1, 1, p, p, 1, 1, None, 0, p, None, p, p, 1, None) == 1
    assert r.starkv_tree_accept(None, p, 1, p, 1, 1, p, p, 1, 1, p, p, None) == 1
    assert r.starkv_tree_workspace_bytes(None, 1, 16, 1, 1) == 0
    # nothing to do
    assert r.starkv_qk_norm_rope(p, 0, None, None, 0, None, 0, None, 0, None, 0, None) == 0
    assert r.starkv_append_qkv(p, None, 0, None, 0, 0, 0, None, None, None, None, 0, None, 0, None, 0, None, 0, None) == 0
    assert r.starkv_cache_read(p, None, 0, None, 0, 0, 0, None, None, None, None) == 0
    assert r.starkv_tree_attn(p, None, 0, None, 0, 0, None, None, 0, 1, None, 0, None, None, None, None, 0, None) == 0
    assert r.starkv_tree_accept(p, None, 0, None, 0, 0, None, None, 0, 1, None, None, None) == 0


def test_sizes_and_nulls_refused():
    r, (b, p) = raw(), buf()
    assert r.starkv_qk_norm_rope(p, -1, p, p, 1, None, 0, p, 1, None, 0, None) == 1
    assert r.starkv_qk_norm_rope(p, 1, p, p, 1, None, 0, None, 0, None, 0, None) == 1 and "together" in err()
    assert r.starkv_qk_norm_rope(p, 1, p, p, -8, None, 0, p, 8, None, 0, None) == 1 and "strides" in err()
    for a in ([p, None, 1, p, 1, 1, 1, p, p, p, p, 1, p, 1, p, 1, p, 1], [p, p, 1, p, 1, 1, 1, p, p, p, p, 1, None, 1, p, 1, p, 1],
              [p, p, 1, p, 1, 1, 1, None, p, p, None, 1, p, 1, p, 1, None, 1]):
        assert r.starkv_append_qkv(*a, None) == 1 and "NULL" in err()
    assert r.starkv_append_qkv(p, p, 1, p, 1, 1, 1, p, p, p, p, 1, p, 1, p, 1, None, 1, None) == 1 and "together" in err()
    assert r.starkv_append_qkv(p, p, 1, p, 1, BIG, 1, p, p, p, p, 1, p, 1, p, 1, p, 1, None) == 1 and "overflows" in err()
    assert r.starkv_append_qkv(p, p, 0, p, 1, 1, 1, p, p, p, p, 1, p, 1, p, 1, p, 1, None) == 1 and "empty" in err()
    assert r.starkv_cache_read(p, p, 1, p, 1, BIG, 1, p, p, p, None) == 1 and "overflows" in err()
    assert r.starkv_cache_read(p, p, 1, p, 0, 1, 1, p, p, p, None) == 1 and "empty" in err()
    assert r.starkv_tree_attn(p, p, 1, p, 1, 1, p, p, 1, 0, None, 0, p, None, p, p, 1, None) == 1 and "max_nodes" in err()
    assert r.starkv_tree_attn(p, p, 1, p, 1, 1, p, p, 1, 1025, None, 0, p, None, p, p, 1, None) == 1
    assert r.starkv_tree_attn(p, p, 1, p, 1, 1, p, p, 1, 33, p, 1, p, None, p, p, 1, None) == 1 and "mask_words" in err()
    assert r.starkv_tree_attn(p, p, 1, p, 1, 1, p, p, 1, 1, p, 0, p, None, p, p, 1, None) == 1 and "mask_words" in err()
    assert r.starkv_tree_attn(p, p, 1, p, BIG, 1, p, p, 1, 1, None, 0, p, None, p, p, 1, None) == 1 and "overflows" in err()
    assert r.starkv_tree_attn(p, p, 1, p, 1, -1, p, p, 1, 1, None, 0, p, None, p, p, 1, None) == 1
    assert r.starkv_tree_accept(p, p, 1, p, BIG, 1, p, p, 1, 1, p, p, None) == 1 and "overflows" in err()
    assert r.starkv_tree_accept(p, p, 1, p, 1, 1, p, p, 1, 0, p, p, None) == 1 and "max_nodes" in err()
    assert r.starkv_tree_accept(p, p, 1, p, 1, 1, p, p, 1, 1, None, p, None) == 1 and "NULL" in err()


def test_misaligned_buffers_refused():
    r, (b, p) = raw(), buf()
    for m in (p + 2, p + 8):
        assert r.starkv_append_qkv(p, m, 1, p, 1, 1, 1, p, p, p, p, 1, p, 1, p, 1, p, 1, None) == 1 and "aligned" in err()
        assert r.starkv_cache_read(p, p, 1, p, 1, 1, 1, p, p, m, None) == 1 and "aligned" in err()
        for k in (1, 12, 14, 15):                              # pool, q, out, workspace
            a = [p, p, 1, p, 1, 1, p, p, 1, 1, None, 0, p, None, p, p, 1, None]
            a[k] = m
            assert r.starkv_tree_attn(*a) == 1 and "aligned" in err()
        assert r.starkv_tree_accept(p, m, 1, p, 1, 1, p, p, 1, 1, p, p, None) == 1 and "aligned" in err()
    m = p + 2
    assert r.starkv_qk_norm_rope(p, 1, m, p, 1, None, 0, p, 1, None, 0, None) == 1
    assert r.starkv_qk_norm_rope(p, 1, p, m, 1, None, 0, p, 1, None, 0, None) == 1
    assert r.starkv_append_qkv(p, p, 1, p, 1, 1, 1, m, p, p, p, 1, p, 1, p, 1, p, 1, None) == 1
    assert r.starkv_append_qkv(p, p, 1, p, 1, 1, 1, p, p, m, p, 1, p, 1, p, 1, p, 1, None) == 1
    for k in (3, 6, 7, 10, 13):
        a = [p, p, 1, p, 1, 1, p, p, 1, 1, p, 1, p, p, p, p, 1, None]
        a[k] = m
        assert r.starkv_tree_attn(*a) == 1 and "4-byte" in err()
    for k in (3, 6, 7, 10, 11):
        a = [p, p, 1, p, 1, 1, p, p, 1, 1, p, p, None]
        a[k] = m
        assert r.starkv_tree_accept(*a) == 1 and "4-byte" in err()


def test_binding_checks_tensors():
    from decode_attention_rank_b200 import starkv as sk
    L = sk.Layer.__new__(sk.Layer)
    L._h, L.cfg, L.latent_total = None, sk.LayerConfig(hidden=64, n_heads=2, n_kv_heads=1, head_dim=16, plain=True), 32
    q, k = torch.zeros(3, 32, dtype=torch.bfloat16), torch.zeros(3, 16, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[:, :31]), dict(k=k[:2]), dict(positions=pos.long()),
                dict(positions=pos[:2]), dict(q_out=torch.zeros(32, 3, dtype=torch.bfloat16).t())):
        with pytest.raises(ValueError):
            L.qk_norm_rope(**dict(dict(q=q, k=k, positions=pos, q_out=q, k_out=k, stream=0), **bad))
    pt, pool, ws = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.append_qkv(pool, 1, pt, pos, pos[:2], None, k, k, stream=0)
    with pytest.raises(ValueError):
        L.cache_read(pool, 1, pt, pos, pos, torch.zeros(3, 40, dtype=torch.bfloat16)[:, :32], stream=0)
    args = dict(pool=pool, n_pages=1, page_table=pt, hist=pos[:2], node_off=pos, q=q, out=torch.zeros(3, 64, dtype=torch.bfloat16),
                workspace=ws, max_nodes=2, stream=0)
    for bad in (dict(node_off=pos[:2]), dict(hist=pos, node_off=torch.zeros(4, dtype=torch.int32)),
                dict(mask=torch.zeros(2, 1, dtype=torch.int32)), dict(mask=torch.zeros(3, 1, dtype=torch.int64)),
                dict(q_pos=pos[:1]), dict(out=torch.zeros(3, 63, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            L.tree_attn(**dict(args, **bad))
    with pytest.raises(ValueError):
        L.tree_accept(pool, 1, pt, pos[:2], pos, pos, pos, max_nodes=2, stream=0)


def test_definition_of_codes():
    """Hand-worked group: amax 12.7 in 8 bits gives scale 0.1 rounded up to fp16 (0.1000366), code = round(x / scale)."""
    x = torch.zeros(32, dtype=torch.float64)
    x[0], x[1], x[2] = 12.7, -12.7, 0.05
    s, c = R.quantise(x, 8)
    assert float(s[0]) == 0.10003662109375
    assert c[0, :4].tolist() == [255, 1, 128, 128]
    s, c = R.quantise(x, 4)
    assert c[0, :4].tolist() == [15, 1, 8, 8] and float(s[0]) >= 12.7 / 7
    assert R.token_bytes(s, c, 4)[0, :2].tolist() == [0x1F, 0x88]
    page = torch.zeros(1, R.page_bytes(1, 64, 4, 2), dtype=torch.uint8)
    K = torch.cat((x, torch.ones(32, dtype=torch.float64))).reshape(1, 1, 64)
    R.put(page, torch.tensor([0]), torch.tensor([3]), K, -K, 4, torch.bfloat16)
    assert page[0, 64 + 3 * 16:64 + 3 * 16 + 2].tolist() == [0x1F, 0x88]         # after two groups' scales of 32 bytes
    assert page[0, 576 + 64 + 3 * 16:576 + 64 + 3 * 16 + 2].tolist() == [0xF1, 0x88]


def test_definition_of_attention_and_rotation():
    x = torch.tensor([[[3.0, 0.0, 4.0, 0.0]]])
    y = R.norm_rope(x, torch.tensor([1.0, 1.0, 2.0, 1.0]), 0.0, torch.tensor([0]), 100.0)
    assert torch.allclose(y, torch.tensor([[[1.2, 0.0, 3.2, 0.0]]], dtype=torch.float64))
    y = R.norm_rope(x, None, 0.0, torch.tensor([1]), 100.0)[0, 0]
    assert torch.allclose(y[[0, 2]], torch.tensor([3 * 0.5403023 - 4 * 0.8414710, 4 * 0.5403023 + 3 * 0.8414710],
                                                  dtype=torch.float64), atol=1e-6)
    K = V = torch.eye(2, dtype=torch.float64).reshape(2, 1, 2)
    q = torch.tensor([[[0.0, 0.0]], [[0.0, 0.0]], [[0.0, 0.0]]])
    see = torch.tensor([[True, True], [False, True], [False, False]])
    out = R.attention(q.to(torch.float64), K, V, see, 1.0)
    assert out.tolist() == [[0.5, 0.5], [0.0, 1.0], [0.0, 0.0]]


def fake_layer(sk, hkv=1, H=2, d=16):
    """A layer without a handle: the library would answer that the layer is NULL."""
    L = sk.Layer.__new__(sk.Layer)
    L._h, L.page_bytes, L.latent_total = None, 64, 2 * hkv * d
    L.cfg = sk.LayerConfig(hidden=64, n_heads=H, n_kv_heads=hkv, head_dim=d, plain=True)
    return L


def test_binding_refuses_host_tensors():
    """Host memory of the right shapes and types is refused before any call of the library."""
    from decode_attention_rank_b200 import starkv as sk
    L = fake_layer(sk)
    q, k = torch.zeros(3, 32, dtype=torch.bfloat16), torch.zeros(3, 16, dtype=torch.bfloat16)
    i3, i2 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pt, pool = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    out = torch.zeros(3, 64, dtype=torch.bfloat16)
    for call in (lambda: L.qk_norm_rope(q, k, i3, q, k, stream=0),
                 lambda: L.append_qkv(pool, 1, pt, i3, i3, q, k, k, q_out=q, stream=0),
                 lambda: L.cache_read(pool, 1, pt, i3, i3, torch.zeros(3, 32, dtype=torch.bfloat16), stream=0),
                 lambda: L.tree_attn(pool, 1, pt, i2, i3, q, out, pool, max_nodes=2, stream=0),
                 lambda: L.tree_accept(pool, 1, pt, i2, i3, i3, i2, max_nodes=2, stream=0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    W = torch.zeros(64, 128, dtype=torch.bfloat16)
    cfg = sk.LayerConfig(hidden=64, n_heads=1, n_kv_heads=1, head_dim=128, plain=True)
    with pytest.raises(ValueError, match="CUDA device"):
        sk.load_plain(cfg, W, W, W, stream=0)
    for bad in (W[:63], W.float(), W.t()):
        with pytest.raises(ValueError, match="W_v must hold"):
            sk.load_plain(cfg, W, bad, W, stream=0)


class OnDevice:
    """A tensor that says that it is on a device."""

    def __init__(self, t, dev):
        self.t, self.dev = t, dev

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev


def test_binding_refuses_another_device_and_a_short_pool(monkeypatch):
    from decode_attention_rank_b200 import starkv as sk
    L = fake_layer(sk)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    i3, i2 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pt, pool = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)

    def accept(dev, n_pages=1, pool_dev=1):
        a = [OnDevice(x, 1) for x in (pt, i2, i3, i3, i2)]
        a[3] = OnDevice(i3, dev)
        L.tree_accept(OnDevice(pool, pool_dev), n_pages, *a, max_nodes=2, stream=0)

    for dev, pool_dev in ((0, 1), (2, 1), (-1, 1), (1, 0), (0, 0)):
        with pytest.raises(ValueError, match="CUDA device"):
            accept(dev, 1, pool_dev)
    with pytest.raises(ValueError, match="pool must hold 2 pages"):
        accept(1, 2)
    with pytest.raises(sk.StarKVError, match="layer is NULL"):   # all as it should be: the library is asked
        accept(1)


def test_tree_page_tables_whose_tiles_would_pass_the_largest_int():
    """A length is rounded up to a tile of 128 tokens: tables within 128 of 2^31 slots are refused, below they are not."""
    r, (b, p) = raw(), buf()
    most = (2 ** 31 - 1 - 128) // 16
    for pages in (most + 1, (2 ** 31 - 1) // 16):
        assert r.starkv_tree_attn(p, p, 1, p, pages, 1, p, p, 1, 1, None, 0, p, None, p, p, 1, None) == 1 and "overflows" in err()
    # (the next check of the call is the alignment of q)
    assert r.starkv_tree_attn(p, p, 1, p, most, 1, p, p, 1, 1, None, 0, p + 8, None, p, p, 1, None) == 1 and "aligned" in err()
