"""Thin Python binding of the libstarkv C ABI (argument marshalling only).

Every step of the attention path runs in the library's CUDA kernels; this
module converts torch tensors to raw pointers and sizes, calls the C entry
points declared in include/starkv.h, and raises on a non-OK status.  torch is
used only to hold device memory and to name the current CUDA stream.

Importing succeeds on machines without a GPU (the shared library loads without
one); calling into it then fails with the CUDA error the runtime reports.  If
libstarkv.so is missing, the import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstarkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m decode_attention_rank_b200.build` "
                      "(there is no fallback path)")
_lib = ctypes.CDLL(LIB_PATH)

STARKV_F32, STARKV_BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "out of device memory", 4: "CUDA error",
          5: "device status word set", 6: "device wait timed out", 7: "workspace too small"}
DEV_BAD_PAGE, DEV_BAD_POSITION, DEV_SCALE_OVF, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8

EXPORTED = ["starkv_load_factors", "starkv_free_layer", "starkv_layer_get_info", "starkv_page_bytes",
            "starkv_cache_init", "starkv_append", "starkv_append_workspace_bytes", "starkv_decode_attn",
            "starkv_prefill_attn", "starkv_workspace_bytes", "starkv_sync_status", "starkv_status_string",
            "starkv_last_error", "starkv_version", "starkv_decode_attn_noalloc", "starkv_set_decode_path",
            "starkv_check_wait_timeout", "starkv_load_plain", "starkv_qk_norm_rope", "starkv_append_qkv",
            "starkv_cache_read", "starkv_tree_attn", "starkv_tree_workspace_bytes", "starkv_tree_accept"]
NOALLOC_SCRATCH_BYTES = 32 << 20


class _Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("key_ranks", ctypes.POINTER(ctypes.c_int)),
                ("value_rank", ctypes.c_int), ("dtype", ctypes.c_int), ("quantized", ctypes.c_int),
                ("top_fraction", ctypes.c_float), ("top_bits", ctypes.c_int), ("bottom_bits", ctypes.c_int),
                ("group_size", ctypes.c_int), ("hadamard_block", ctypes.c_int), ("rope", ctypes.c_int),
                ("rope_theta", ctypes.c_double), ("softmax_scale", ctypes.c_float), ("page_size", ctypes.c_int),
                ("plain", ctypes.c_int), ("max_positions", ctypes.c_int), ("unfused_output", ctypes.c_int)]


class _Info(ctypes.Structure):
    _fields_ = [("n_latents", ctypes.c_int), ("latent_total", ctypes.c_int), ("key_rank_total", ctypes.c_int),
                ("page_bytes", ctypes.c_size_t), ("bytes_per_token", ctypes.c_double),
                ("factor_bytes", ctypes.c_size_t)]


_vp, _i32p, _sz, _i64 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
_lib.starkv_load_factors.argtypes = [ctypes.POINTER(_Config), _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)]
_lib.starkv_free_layer.argtypes = [_vp]
_lib.starkv_free_layer.restype = None
_lib.starkv_layer_get_info.argtypes = [_vp, ctypes.POINTER(_Info)]
_lib.starkv_page_bytes.argtypes = [_vp]
_lib.starkv_page_bytes.restype = _sz
_lib.starkv_cache_init.argtypes = [_vp, _vp, _i64, _vp]
_lib.starkv_append.argtypes = [_vp, _vp, _i64, _i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i32p, _i32p, _vp,
                               ctypes.c_int, _vp, _sz, _vp]
_lib.starkv_append_workspace_bytes.argtypes = [_vp, ctypes.c_int]
_lib.starkv_append_workspace_bytes.restype = _sz
_lib.starkv_decode_attn.argtypes = [_vp, _vp, _i64, _i32p, ctypes.c_int, ctypes.c_int, _i32p, _i32p, _vp, _vp, _vp,
                                    _sz, _vp]
_lib.starkv_prefill_attn.argtypes = [_vp, _vp, _i64, _i32p, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]
_lib.starkv_decode_attn_noalloc.argtypes = [_vp, _vp, _i64, _i32p, ctypes.c_int, ctypes.c_int, _i32p, _i32p, _vp,
                                            _vp, _vp]
_lib.starkv_workspace_bytes.argtypes = [_vp, ctypes.c_int, ctypes.c_int, ctypes.c_int]
_lib.starkv_workspace_bytes.restype = _sz
_lib.starkv_sync_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
_lib.starkv_status_string.argtypes = [ctypes.c_int]
_lib.starkv_status_string.restype = ctypes.c_char_p
_lib.starkv_last_error.argtypes = []
_lib.starkv_last_error.restype = ctypes.c_char_p
_lib.starkv_set_decode_path.argtypes = [_vp, ctypes.c_int]
_lib.starkv_check_wait_timeout.argtypes = [_vp, ctypes.c_uint32, _vp]
_lib.starkv_profile_decode.argtypes = [_vp, ctypes.c_int]
_lib.starkv_decode_phase_ms.argtypes = [_vp, ctypes.POINTER(ctypes.c_float), ctypes.c_int]
_int = ctypes.c_int
_lib.starkv_load_plain.argtypes = [ctypes.POINTER(_Config), _int, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp,
                                   ctypes.POINTER(_vp)]
_lib.starkv_qk_norm_rope.argtypes = [_vp, _int, _i32p, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
_lib.starkv_append_qkv.argtypes = [_vp, _vp, _i64, _i32p, _int, _int, _int, _i32p, _i32p, _i32p, _vp, _i64, _vp, _i64,
                                   _vp, _i64, _vp, _i64, _vp]
_lib.starkv_cache_read.argtypes = [_vp, _vp, _i64, _i32p, _int, _int, _int, _i32p, _i32p, _vp, _vp]
_lib.starkv_tree_attn.argtypes = [_vp, _vp, _i64, _i32p, _int, _int, _i32p, _i32p, _int, _int, _vp, _int, _vp, _i32p,
                                  _vp, _vp, _sz, _vp]
_lib.starkv_tree_workspace_bytes.argtypes = [_vp, _int, _int, _int, _int]
_lib.starkv_tree_workspace_bytes.restype = _sz
_lib.starkv_tree_accept.argtypes = [_vp, _vp, _i64, _i32p, _int, _int, _i32p, _i32p, _int, _int, _i32p, _i32p, _vp]
N_PHASES = 4   # query preparation + scores, joint values, run merge, output projection
_lib.starkv_version.argtypes = []
_lib.starkv_version.restype = ctypes.c_char_p


class StarKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.starkv_last_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)}" + (f" ({msg})" if msg else ""))


def _check(st: int, where: str) -> None:
    if st != 0:
        raise StarKVError(st, where)


def version() -> str:
    return _lib.starkv_version().decode()


def _ptr(t) -> int:
    if t is None:
        return None
    return t.data_ptr()


_torch_module = None


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _rows(t, n: int, width: int, name: str, dtype, dense: bool = False):
    """Pointer and row stride of n rows of `width` elements ([n, width] or [n, heads, d]; rows may be strided)."""
    if t is None:
        return None, 0
    shape, stride = t.shape, t.stride()
    last = shape[-1] if len(shape) else 0
    if len(shape) == 3 and (shape[1] == 1 or stride[1] == last):
        last *= shape[1]
    elif len(shape) != 2:
        last = -1
    if last != width or shape[0] != n or stride[-1] != 1:
        raise ValueError(f"{name} must be [{n}, {width}] with contiguous rows, got {list(shape)}, strides {list(stride)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have the layer's dtype ({dtype}), got {t.dtype}")
    ld = stride[0] if n > 1 else width
    if dense and ld != width:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), ld


def _ints(t, n: int, name: str):
    """Pointer of a contiguous int32 array of n elements."""
    if t is None:
        return None
    if t.dtype is not _torch_module.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 array of {n} elements")
    return t.data_ptr()


def _on_device(*tensors):
    """Refuse tensors that are not on the current CUDA device: a kernel would follow their pointers all the same."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()                                 # -1: not on a CUDA device
            if dev is None and d >= 0:
                dev = _torch()._C._cuda_getDevice()
            if d != dev:
                raise ValueError(f"tensor {list(t.shape)} is on {t.device}, not on the current CUDA device")


def _table(page_table, batch: int = 0):
    """Pointer, rows and columns of an int32 page table."""
    rows, cols = page_table.shape
    if rows < batch:
        raise ValueError(f"page_table must have at least {batch} rows")
    return _ints(page_table, rows * cols, "page_table"), rows, cols


def _stream(stream) -> int:
    """Handle of the given stream, or of torch's current one."""
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # without building a Stream object, which takes as long as a launch (3 us)
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


@dataclass
class LayerConfig:
    """Python mirror of starkv_layer_config (see include/starkv.h)."""
    hidden: int
    n_heads: int
    n_kv_heads: int
    head_dim: int
    key_ranks: list = field(default_factory=list)
    value_rank: int = 0
    dtype: str = "bf16"
    quantized: bool = False
    top_fraction: float = 0.25
    top_bits: int = 4
    bottom_bits: int = 3
    group_size: int = 32
    hadamard_block: int = 0
    rope: bool = False
    rope_theta: float = 10000.0
    softmax_scale: float = 0.0
    page_size: int = 16
    plain: bool = False
    max_positions: int = 0
    unfused_output: bool = False

    @classmethod
    def from_spec(cls, spec) -> "LayerConfig":
        return cls(hidden=spec.hidden, n_heads=spec.n_heads, n_kv_heads=spec.n_kv_heads, head_dim=spec.head_dim,
                   key_ranks=list(spec.key_ranks), value_rank=spec.value_rank, dtype=spec.dtype,
                   quantized=spec.quantized, top_fraction=spec.top_fraction, top_bits=spec.top_bits,
                   bottom_bits=spec.bottom_bits, group_size=spec.group_size, hadamard_block=spec.hadamard_block,
                   rope=spec.rope, rope_theta=spec.rope_theta, page_size=spec.page_size, plain=spec.plain)

    def _c(self):
        ranks = (ctypes.c_int * max(1, len(self.key_ranks)))(*self.key_ranks)
        c = _Config(self.hidden, self.n_heads, self.n_kv_heads, self.head_dim,
                    ctypes.cast(ranks, ctypes.POINTER(ctypes.c_int)) if self.key_ranks else None, self.value_rank,
                    STARKV_F32 if self.dtype == "f32" else STARKV_BF16, int(self.quantized), self.top_fraction,
                    self.top_bits, self.bottom_bits, self.group_size, self.hadamard_block, int(self.rope),
                    self.rope_theta, self.softmax_scale, self.page_size, int(self.plain), self.max_positions,
                    int(self.unfused_output))
        return c, ranks


class Layer:
    """One loaded layer (owns its folded factors on the device)."""

    _dims = None

    def __init__(self, handle: int, cfg: LayerConfig):
        self._h = handle
        self.cfg = cfg
        info = _Info()
        _check(_lib.starkv_layer_get_info(self._h, ctypes.byref(info)), "starkv_layer_get_info")
        self.n_latents = info.n_latents
        self.latent_total = info.latent_total
        self.key_rank_total = info.key_rank_total
        self.page_bytes = info.page_bytes
        self.bytes_per_token = info.bytes_per_token
        self.factor_bytes = info.factor_bytes

    def __del__(self):
        self.free()

    def free(self) -> None:
        if getattr(self, "_h", None) and _lib is not None:   # (gone at interpreter exit)
            _lib.starkv_free_layer(self._h)
            self._h = None

    @property
    def handle(self) -> int:
        return self._h

    def cache_init(self, pool, n_pages: int, stream=None) -> None:
        _check(_lib.starkv_cache_init(self._h, _ptr(pool), n_pages, _stream(stream)), "starkv_cache_init")

    def append_workspace_bytes(self, n_tokens: int) -> int:
        return _lib.starkv_append_workspace_bytes(self._h, n_tokens)

    def append(self, pool, n_pages: int, page_table, seq_idx, positions, inputs, input_is_latent: bool,
               workspace=None, stream=None) -> None:
        n = int(seq_idx.numel())
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(_lib.starkv_append(self._h, _ptr(pool), n_pages, _ptr(page_table), int(page_table.shape[0]),
                                  int(page_table.shape[1]), n,
                                  _ptr(seq_idx), _ptr(positions), _ptr(inputs), int(input_is_latent),
                                  _ptr(workspace), ws_bytes, _stream(stream)), "starkv_append")

    def workspace_bytes(self, batch: int, max_ctx: int, max_q: int = 1) -> int:
        return _lib.starkv_workspace_bytes(self._h, batch, max_ctx, max_q)

    def decode(self, pool, n_pages: int, page_table, seq_lens, q, out, workspace, q_pos=None, stream=None) -> None:
        _check(_lib.starkv_decode_attn(self._h, _ptr(pool), n_pages, _ptr(page_table), int(page_table.shape[1]),
                                       int(seq_lens.numel()), _ptr(seq_lens), _ptr(q_pos), _ptr(q), _ptr(out),
                                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream(stream)), "starkv_decode_attn")

    def decode_noalloc(self, pool, n_pages: int, page_table, seq_lens, q, out, q_pos=None, stream=None) -> None:
        """Decode without a workspace (scratch in the library's fixed device array)."""
        _check(_lib.starkv_decode_attn_noalloc(self._h, _ptr(pool), n_pages, _ptr(page_table),
                                               int(page_table.shape[1]), int(seq_lens.numel()), _ptr(seq_lens),
                                               _ptr(q_pos), _ptr(q), _ptr(out), _stream(stream)),
               "starkv_decode_attn_noalloc")

    def prefill(self, pool, n_pages: int, page_table, q_start: list, q_len: list, q, out, workspace,
                stream=None) -> None:
        B = len(q_start)
        qs = (ctypes.c_int32 * B)(*q_start)
        ql = (ctypes.c_int32 * B)(*q_len)
        _check(_lib.starkv_prefill_attn(self._h, _ptr(pool), n_pages, _ptr(page_table), int(page_table.shape[1]), B,
                                        ctypes.cast(qs, _vp), ctypes.cast(ql, _vp), _ptr(q), _ptr(out),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "starkv_prefill_attn")

    # ---- serving an uncompressed layer, and speculative decoding (see include/starkv.h)

    def _shape(self):
        """Layer dtype, channels of a token's queries and of its keys."""
        if self._dims is None:
            c, torch = self.cfg, _torch()
            self._dims = (torch.float32 if c.dtype == "f32" else torch.bfloat16, c.n_heads * c.head_dim,
                          c.n_kv_heads * c.head_dim)
        return self._dims

    def _pool(self, pool, n_pages: int) -> int:
        """Pointer of a pool of n_pages pages."""
        if not pool.is_contiguous() or pool.nbytes < n_pages * self.page_bytes:
            raise ValueError(f"pool must hold {n_pages} pages of {self.page_bytes} bytes, contiguous")
        return pool.data_ptr()

    def qk_norm_rope(self, q, k, positions, q_out, k_out, stream=None) -> None:
        """Per-head norm and rotation of queries and keys (either pair may be None)."""
        dt, wq, wk = self._shape()
        some = q if q is not None else k
        n = int(some.shape[0]) if some is not None else 0
        (qp, ql), (kp, kl) = _rows(q, n, wq, "q", dt), _rows(k, n, wk, "k", dt)
        (qo, qol), (ko, kol) = _rows(q_out, n, wq, "q_out", dt), _rows(k_out, n, wk, "k_out", dt)
        pos = _ints(positions, n, "positions")
        _on_device(q, k, positions, q_out, k_out)
        _check(_lib.starkv_qk_norm_rope(self._h, n, pos, qp, ql, kp, kl, qo, qol, ko, kol, _stream(stream)),
               "starkv_qk_norm_rope")

    def append_qkv(self, pool, n_pages: int, page_table, seq_idx, slots, q, k, v, q_out=None, positions=None,
                   stream=None) -> None:
        """Norm, rotation and storing (or quantising) of new tokens' projections in one pass."""
        dt, wq, wk = self._shape()
        n = seq_idx.numel()
        (qp, ql), (kp, kl), (vp, vl) = _rows(q, n, wq, "q", dt), _rows(k, n, wk, "k", dt), _rows(v, n, wk, "v", dt)
        qo, qol = _rows(q_out, n, wq, "q_out", dt)
        pt, seqs, mp = _table(page_table)
        si, sl, pos = _ints(seq_idx, n, "seq_idx"), _ints(slots, n, "slots"), _ints(positions, n, "positions")
        _on_device(pool, page_table, seq_idx, slots, q, k, v, q_out, positions)
        _check(_lib.starkv_append_qkv(self._h, self._pool(pool, n_pages), n_pages, pt, seqs, mp, n, si, sl, pos, qp, ql, kp,
                                      kl, vp, vl, qo, qol, _stream(stream)), "starkv_append_qkv")

    def cache_read(self, pool, n_pages: int, page_table, seq_idx, slots, out, stream=None) -> None:
        """Cached tokens as dense rows [n, latent_total]."""
        dt, n = self._shape()[0], seq_idx.numel()
        op, _ = _rows(out, n, self.latent_total, "out", dt, dense=True)
        pt, seqs, mp = _table(page_table)
        si, sl = _ints(seq_idx, n, "seq_idx"), _ints(slots, n, "slots")
        _on_device(pool, page_table, seq_idx, slots, out)
        _check(_lib.starkv_cache_read(self._h, self._pool(pool, n_pages), n_pages, pt, seqs, mp, n, si, sl, op,
                                      _stream(stream)), "starkv_cache_read")

    def tree_workspace_bytes(self, batch: int, max_ctx: int, n_nodes: int, max_nodes: int) -> int:
        return _lib.starkv_tree_workspace_bytes(self._h, batch, max_ctx, n_nodes, max_nodes)

    def tree_attn(self, pool, n_pages: int, page_table, hist, node_off, q, out, workspace, max_nodes: int, mask=None,
                  q_pos=None, stream=None) -> None:
        """Attention of drafted nodes over the cache: mask int32 [n_nodes, words] (bits), None = a chain."""
        dt, wq, _ = self._shape()
        batch, n = hist.numel(), int(q.shape[0])
        words = 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[0] != n:
                raise ValueError(f"mask must be [{n}, words]")
            words = int(mask.shape[1])
        qp, _ = _rows(q, n, wq, "q", dt, dense=True)
        op, _ = _rows(out, n, self.cfg.hidden, "out", dt, dense=True)
        pt, _, mp = _table(page_table, batch)
        hp, no = _ints(hist, batch, "hist"), _ints(node_off, batch + 1, "node_off")
        mk, pos = _ints(mask, n * words, "mask"), _ints(q_pos, n, "q_pos")
        _on_device(pool, page_table, hist, node_off, q, out, workspace, mask, q_pos)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        _check(_lib.starkv_tree_attn(self._h, self._pool(pool, n_pages), n_pages, pt, mp, batch, hp, no, n, max_nodes, mk,
                                     words, qp, pos, op, workspace.data_ptr(), workspace.nbytes, _stream(stream)),
               "starkv_tree_attn")

    def tree_accept(self, pool, n_pages: int, page_table, hist, node_off, acc, n_acc, max_nodes: int,
                    stream=None) -> None:
        """Move the accepted nodes' slots to the front and clear the other nodes' slots."""
        self._shape()
        batch, n = hist.numel(), acc.numel()
        pt, _, mp = _table(page_table, batch)
        hp, no = _ints(hist, batch, "hist"), _ints(node_off, batch + 1, "node_off")
        ac, na = _ints(acc, n, "acc"), _ints(n_acc, batch, "n_acc")
        _on_device(pool, page_table, hist, node_off, acc, n_acc)
        _check(_lib.starkv_tree_accept(self._h, self._pool(pool, n_pages), n_pages, pt, mp, batch, hp, no, n, max_nodes, ac,
                                       na, _stream(stream)), "starkv_tree_accept")

    def set_decode_path(self, path: int) -> None:
        """0 automatic, 1 CUDA-core kernels, 2 tensor-core scores + CUDA-core values (diagnostics)."""
        _check(_lib.starkv_set_decode_path(self._h, path), "starkv_set_decode_path")

    def profile_decode(self, n_calls: int) -> None:
        """Keep CUDA-event timings of the next n_calls tensor-core decodes (0 = off)."""
        _check(_lib.starkv_profile_decode(self._h, n_calls), "starkv_profile_decode")

    def decode_phase_ms(self, n_calls: int) -> list:
        """Per-call lists of the phase times (ms) recorded since profile_decode."""
        buf = (ctypes.c_float * (n_calls * N_PHASES))()
        _check(_lib.starkv_decode_phase_ms(self._h, buf, n_calls), "starkv_decode_phase_ms")
        return [list(buf[c * N_PHASES:(c + 1) * N_PHASES]) for c in range(n_calls)]

    def check_wait_timeout(self, limit_us: int, stream=None) -> None:
        """Run the bounded-wait diagnostic kernel (see starkv_check_wait_timeout)."""
        _check(_lib.starkv_check_wait_timeout(self._h, limit_us, _stream(stream)), "starkv_check_wait_timeout")

    def sync_status_code(self, stream=None) -> tuple:
        """(status code of starkv_sync_status, status bits)."""
        bits = ctypes.c_uint32(0)
        st = _lib.starkv_sync_status(self._h, _stream(stream), ctypes.byref(bits))
        return st, bits.value

    def sync_status(self, stream=None) -> int:
        bits = ctypes.c_uint32(0)
        st = _lib.starkv_sync_status(self._h, _stream(stream), ctypes.byref(bits))
        if st not in (0, 5, 6):
            _check(st, "starkv_sync_status")
        return bits.value


def load_factors(cfg: LayerConfig, A_k, B_k, A_v, B_v, W_o, stream=None) -> Layer:
    """Fold and upload one layer's factors (device tensors in cfg.dtype, unrotated)."""
    c, keep = cfg._c()
    h = _vp()
    _check(_lib.starkv_load_factors(ctypes.byref(c), _ptr(A_k), _ptr(B_k), _ptr(A_v), _ptr(B_v), _ptr(W_o),
                                    _stream(stream), ctypes.byref(h)), "starkv_load_factors")
    del keep
    return Layer(h.value, cfg)


def load_plain(cfg: LayerConfig, W_k, W_v, W_o, kv_bits: int = 0, q_norm=None, k_norm=None, norm_eps: float = 1e-6,
               stream=None) -> Layer:
    """Load an uncompressed layer with a quantised cache (kv_bits 8 or 4) and per-head query / key norms."""
    want = "torch.float32" if cfg.dtype == "f32" else "torch.bfloat16"
    kv, qd = cfg.n_kv_heads * cfg.head_dim, cfg.n_heads * cfg.head_dim
    given = (("W_k", W_k, cfg.hidden * kv), ("W_v", W_v, cfg.hidden * kv), ("W_o", W_o, qd * cfg.hidden),
             ("q_norm", q_norm, cfg.head_dim), ("k_norm", k_norm, cfg.head_dim))
    for name, t, n in given:
        if t is not None and (str(t.dtype) != want or t.numel() != n or not t.is_contiguous()):
            raise ValueError(f"{name} must hold {n} elements of the layer's dtype ({want}), contiguous")
    _on_device(*(t for _, t, _ in given))
    c, keep = cfg._c()
    h = _vp()
    _check(_lib.starkv_load_plain(ctypes.byref(c), kv_bits, _ptr(q_norm), _ptr(k_norm), norm_eps, _ptr(W_k), _ptr(W_v),
                                  _ptr(W_o), _stream(stream), ctypes.byref(h)), "starkv_load_plain")
    del keep
    return Layer(h.value, cfg)


def raw_lib():
    """The ctypes handle of libstarkv.so (for tests of the C ABI itself)."""
    return _lib
