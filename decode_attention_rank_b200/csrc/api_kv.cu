// Host side of the serving calls of uncompressed layers and of speculative
// decoding: argument checks and dispatch (kernels in k_kv.cu, k_tree.cu and
// k_decode_generic.cu).
#include <limits.h>

#include <string>

#include "starkv_internal.cuh"

using namespace starkv;

#define CHECK_ARG(cond, msg)            \
  do {                                  \
    if (!(cond)) {                      \
      set_error(msg);                   \
      return STARKV_ERR_ARG;            \
    }                                   \
  } while (0)

#define CUDA_TRY(expr)                                                          \
  do {                                                                          \
    cudaError_t e_ = (expr);                                                    \
    if (e_ != cudaSuccess) {                                                    \
      set_error(std::string(#expr) + ": " + cudaGetErrorString(e_));           \
      return STARKV_ERR_CUDA;                                                   \
    }                                                                           \
  } while (0)

namespace {

bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int kMaxNodes = 1024;   // nodes of one sequence: their mask rows stay within 128 bytes

// The layer's tables live on its own device: a call with another device current would read them across devices.
bool on_device(const starkv_layer* L) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == L->device;
}

// Rows of `es`-byte elements that start on 16-byte boundaries.
bool rows16(const void* p, int64_t ld, int es) { return p == nullptr || (aligned_to(p, 16) && (ld * es) % 16 == 0); }

}  // namespace

#define CHECK_LAYER(L)                                                                        \
  do {                                                                                        \
    CHECK_ARG(on_device(L), "the layer was loaded on another device than the current one");   \
  } while (0)

extern "C" {

starkv_status starkv_qk_norm_rope(const starkv_layer* L, int n_tokens, const int32_t* positions, const void* q,
                                  int64_t q_ld, const void* k, int64_t k_ld, void* q_out, int64_t q_out_ld, void* k_out,
                                  int64_t k_out_ld, starkv_stream_t stream) {
  set_error("");
  CHECK_ARG(L != nullptr, "layer is NULL");
  CHECK_ARG(n_tokens >= 0, "negative n_tokens");
  if (n_tokens == 0 || (!q && !k)) return STARKV_OK;
  CHECK_ARG((q == nullptr) == (q_out == nullptr) && (k == nullptr) == (k_out == nullptr),
            "q and q_out, k and k_out are given together");
  CHECK_ARG(aligned_to(positions, 4), "positions must be 4-byte aligned");
  CHECK_ARG(aligned_to(q, 4) && aligned_to(k, 4) && aligned_to(q_out, 4) && aligned_to(k_out, 4) && q_ld >= 0 &&
                k_ld >= 0 && q_out_ld >= 0 && k_out_ld >= 0,
            "rows must be 4-byte aligned and their strides non-negative");
  const ServeView& v = L->view;
  if (!v.opt) {
    set_error("only layers of starkv_load_plain");
    return STARKV_ERR_UNSUPPORTED;
  }
  CHECK_LAYER(L);
  CHECK_ARG(!v.rope || positions, "positions is NULL");
  CHECK_ARG(n_tokens == 1 || ((!q || (q_ld >= v.H * v.d && q_out_ld >= v.H * v.d)) &&
                              (!k || (k_ld >= v.Hkv * v.d && k_out_ld >= v.Hkv * v.d))),
            "row strides are shorter than the rows");
  KvArgs a{};
  a.v = v;
  a.n = n_tokens;
  a.positions = positions;
  a.turn = v.turn;
  a.q = q;
  a.k = k;
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_out_ld = q_out_ld;
  a.k_out_ld = k_out_ld;
  a.rotate = v.rope;
  a.vec = rows16(q, q_ld, v.es) && rows16(k, k_ld, v.es) && rows16(q_out, q_out_ld, v.es) && rows16(k_out, k_out_ld, v.es);
  CUDA_TRY(launch_qkv(a, v.dtype == STARKV_F32, (cudaStream_t)stream));
  return STARKV_OK;
}

starkv_status starkv_append_qkv(const starkv_layer* L, void* pool, int64_t n_pages, const int32_t* page_table,
                                int n_seqs, int max_pages, int n_tokens, const int32_t* seq_idx, const int32_t* slots,
                                const int32_t* positions, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                const void* vv, int64_t v_ld, void* q_out, int64_t q_out_ld, starkv_stream_t stream) {
  set_error("");
  CHECK_ARG(L != nullptr, "layer is NULL");
  CHECK_ARG(n_tokens >= 0, "negative n_tokens");
  if (n_tokens == 0) return STARKV_OK;
  CHECK_ARG(pool && page_table && seq_idx && slots && k && vv, "NULL buffer");
  CHECK_ARG((q == nullptr) == (q_out == nullptr), "q and q_out are given together");
  CHECK_ARG(n_pages > 0 && max_pages > 0 && n_seqs > 0, "empty pool or page table");
  CHECK_ARG(max_pages <= INT_MAX / kPage, "max_pages * 16 overflows int");
  CHECK_ARG(aligned_to(pool, 16), "pool must be 16-byte aligned");
  CHECK_ARG(aligned_to(page_table, 4) && aligned_to(seq_idx, 4) && aligned_to(slots, 4) && aligned_to(positions, 4),
            "page_table, seq_idx, slots and positions must be 4-byte aligned");
  CHECK_ARG(aligned_to(q, 4) && aligned_to(k, 4) && aligned_to(vv, 4) && aligned_to(q_out, 4) && q_ld >= 0 &&
                k_ld >= 0 && v_ld >= 0 && q_out_ld >= 0,
            "rows must be 4-byte aligned and their strides non-negative");
  const ServeView& v = L->view;
  if (!v.opt) {
    set_error("only layers of starkv_load_plain");
    return STARKV_ERR_UNSUPPORTED;
  }
  CHECK_LAYER(L);
  CHECK_ARG(n_tokens == 1 || ((!q || (q_ld >= v.H * v.d && q_out_ld >= v.H * v.d)) && k_ld >= v.Hkv * v.d &&
                              v_ld >= v.Hkv * v.d),
            "row strides are shorter than the rows");
  KvArgs a{};
  a.vec = rows16(q, q_ld, v.es) && rows16(k, k_ld, v.es) && rows16(vv, v_ld, v.es) && rows16(q_out, q_out_ld, v.es);
  CHECK_ARG(!v.kv_bits || a.vec, "with a quantised cache the rows of q, k, v and q_out must be 16-byte aligned");
  a.v = v;
  a.pool = (uint8_t*)pool;
  a.n_pages = n_pages;
  a.pt = page_table;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.n = n_tokens;
  a.seq_idx = seq_idx;
  a.slots = slots;
  a.positions = positions ? positions : slots;
  a.turn = v.turn;
  a.q = q;
  a.k = k;
  a.vv = vv;
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.q_out = q_out;
  a.q_out_ld = q_out_ld;
  a.rotate = v.rope;
  CUDA_TRY(launch_qkv(a, v.dtype == STARKV_F32, (cudaStream_t)stream));
  return STARKV_OK;
}

starkv_status starkv_cache_read(const starkv_layer* L, const void* pool, int64_t n_pages, const int32_t* page_table,
                                int n_seqs, int max_pages, int n_tokens, const int32_t* seq_idx, const int32_t* slots,
                                void* out, starkv_stream_t stream) {
  set_error("");
  CHECK_ARG(L != nullptr, "layer is NULL");
  CHECK_ARG(n_tokens >= 0, "negative n_tokens");
  if (n_tokens == 0) return STARKV_OK;
  CHECK_ARG(pool && page_table && seq_idx && slots && out, "NULL buffer");
  CHECK_ARG(n_pages > 0 && max_pages > 0 && n_seqs > 0, "empty pool or page table");
  CHECK_ARG(max_pages <= INT_MAX / kPage, "max_pages * 16 overflows int");
  CHECK_ARG(aligned_to(pool, 16) && aligned_to(out, 16), "pool and out must be 16-byte aligned");
  CHECK_ARG(aligned_to(page_table, 4) && aligned_to(seq_idx, 4) && aligned_to(slots, 4),
            "page_table, seq_idx and slots must be 4-byte aligned");
  CHECK_LAYER(L);
  KvArgs a{};
  a.v = L->view;
  a.pool = (uint8_t*)pool;
  a.n_pages = n_pages;
  a.pt = page_table;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.n = n_tokens;
  a.seq_idx = seq_idx;
  a.slots = slots;
  CUDA_TRY(launch_cache_read(a, out, (cudaStream_t)stream));
  return STARKV_OK;
}

size_t starkv_tree_workspace_bytes(const starkv_layer* L, int batch, int max_ctx, int n_nodes, int max_nodes) {
  if (!L || batch <= 0 || n_nodes <= 0 || max_nodes <= 0 || max_nodes > kMaxNodes) return 0;
  if (tree_mma_supported(L->view)) return tree_mma_ws_bytes(L, batch, n_nodes, max_nodes);
  return tree_generic_ws_bytes(L, std::max(max_ctx, 1), n_nodes);
}

starkv_status starkv_tree_attn(const starkv_layer* L, const void* pool, int64_t n_pages, const int32_t* page_table,
                               int max_pages, int batch, const int32_t* hist, const int32_t* node_off, int n_nodes,
                               int max_nodes, const uint32_t* mask, int mask_words, const void* q, const int32_t* q_pos,
                               void* out, void* workspace, size_t ws_bytes, starkv_stream_t stream) {
  set_error("");
  CHECK_ARG(L != nullptr, "layer is NULL");
  CHECK_ARG(batch >= 0 && n_nodes >= 0, "negative batch or n_nodes");
  CHECK_ARG(max_nodes >= 1 && max_nodes <= kMaxNodes, "max_nodes must be in [1, 1024]");
  if (batch == 0 || n_nodes == 0) return STARKV_OK;
  CHECK_ARG(pool && page_table && hist && node_off && q && out, "NULL buffer");
  CHECK_ARG(n_pages > 0 && max_pages > 0, "empty pool or page table");
  CHECK_ARG(max_pages <= kTreeMaxPages, "max_pages * 16 + 128 overflows int");
  CHECK_ARG(!mask || (mask_words >= 1 && mask_words <= kMaxNodes / 32 && mask_words * 32 >= max_nodes),
            "mask_words * 32 must cover max_nodes");
  CHECK_ARG(aligned_to(pool, 16) && aligned_to(q, 16) && aligned_to(out, 16) && aligned_to(workspace, 16),
            "pool, q, out and workspace must be 16-byte aligned");
  CHECK_ARG(aligned_to(page_table, 4) && aligned_to(hist, 4) && aligned_to(node_off, 4) && aligned_to(mask, 4) &&
                aligned_to(q_pos, 4),
            "page_table, hist, node_off, mask and q_pos must be 4-byte aligned");
  CHECK_LAYER(L);
  const ServeView& v = L->view;
  CHECK_ARG(q_pos || v.plain || !v.rope, "a latent layer with RoPE needs q_pos");
  const size_t need = tree_mma_supported(v) ? tree_mma_need(L, batch, n_nodes, max_nodes)
                                            : tree_generic_need(L, max_pages * kPage, n_nodes);
  if (workspace == nullptr || ws_bytes < need) {
    set_error("tree workspace too small: need " + std::to_string(need) + " bytes");
    return STARKV_ERR_WORKSPACE;
  }
  TreeArgs t{(const uint8_t*)pool, n_pages, page_table, max_pages, batch, hist, node_off, n_nodes, max_nodes,
             mask, mask_words, q, q_pos, out, q_pos != nullptr, nullptr};
  if (tree_mma_supported(v))
    CUDA_TRY(launch_tree_mma(L, t, workspace, ws_bytes, (cudaStream_t)stream));
  else
    CUDA_TRY(launch_tree_generic(L, t, workspace, ws_bytes, (cudaStream_t)stream));
  return STARKV_OK;
}

starkv_status starkv_tree_accept(const starkv_layer* L, void* pool, int64_t n_pages, const int32_t* page_table,
                                 int max_pages, int batch, const int32_t* hist, const int32_t* node_off, int n_nodes,
                                 int max_nodes, const int32_t* acc, const int32_t* n_acc, starkv_stream_t stream) {
  set_error("");
  CHECK_ARG(L != nullptr, "layer is NULL");
  CHECK_ARG(batch >= 0 && n_nodes >= 0, "negative batch or n_nodes");
  CHECK_ARG(max_nodes >= 1 && max_nodes <= kMaxNodes, "max_nodes must be in [1, 1024]");
  if (batch == 0 || n_nodes == 0) return STARKV_OK;
  CHECK_ARG(pool && page_table && hist && node_off && acc && n_acc, "NULL buffer");
  CHECK_ARG(n_pages > 0 && max_pages > 0, "empty pool or page table");
  CHECK_ARG(max_pages <= INT_MAX / kPage, "max_pages * 16 overflows int");
  CHECK_ARG(aligned_to(pool, 16), "pool must be 16-byte aligned");
  CHECK_ARG(aligned_to(page_table, 4) && aligned_to(hist, 4) && aligned_to(node_off, 4) && aligned_to(acc, 4) &&
                aligned_to(n_acc, 4),
            "page_table, hist, node_off, acc and n_acc must be 4-byte aligned");
  CHECK_LAYER(L);
  CUDA_TRY(launch_accept(L, (uint8_t*)pool, n_pages, page_table, max_pages, batch, hist, node_off, n_nodes, max_nodes,
                         acc, n_acc, (cudaStream_t)stream));
  return STARKV_OK;
}

}  // extern "C"
