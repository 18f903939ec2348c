// Generic decode/prefill attention over the paged latent cache, on CUDA cores.
//
// It covers every layer shape and storage option (f32/bf16/quantized, RoPE on
// or off, MHA/GQA, plain layers) and serves as the path for shapes the fused
// kernels do not take.  Steps ("STAR-KV 阅读笔记" Algorithm 2):
//   qprep   RoPE(q) * softmax scale * log2(e)
//   scores  per (row, KV head, 64-token tile): read + dequantize the key
//           latents, reconstruct K = Zhat B' on chip, apply RoPE at each
//           slot's position, score every query head of the group (step 4)
//   value   per (row, token split, 128 value channels): exp2(s - m) over the
//           split, stacked-head accumulation Y_h += p_h(t) zhat_v(t) on the
//           shared joint value latent (steps 5-6)
//   combine merge split partials (m, l, Y) -> y = Y / l
//   out     out = sum_h y_h M_h with the fused factors (steps 7-8)
#include <float.h>

#include <type_traits>

#include "starkv_internal.cuh"

namespace starkv {

namespace {

constexpr int kTile = 64;
constexpr int kVBlock = 128;

__device__ __forceinline__ int row_seq_of(const RowInfo& ri, int row) { return ri.row_seq ? ri.row_seq[row] : row; }
__device__ __forceinline__ int row_pos_of(const RowInfo& ri, int row) {
  return ri.row_pos ? ri.row_pos[row] : ri.row_len[row] - 1;
}
// Visible length of a row, clamped to the page table's capacity (flagged when above it).
__device__ __forceinline__ int row_len_of(const RowInfo& ri, int row, int cap, uint32_t* status, bool flag) {
  int len = ri.row_len[row];
  if (len > cap || len < 0) {
    if (flag) atomicOr(status, kBadPos);
    len = len < 0 ? 0 : cap;
  }
  return len;
}


__device__ __forceinline__ double rope_freq(int p, int d, float log2_theta) {
  return exp2(-(2.0 * p / d) * (double)log2_theta);
}

template <typename T>
__device__ __forceinline__ float ldf(const T* p, size_t i);
template <>
__device__ __forceinline__ float ldf<float>(const float* p, size_t i) { return p[i]; }
template <>
__device__ __forceinline__ float ldf<__nv_bfloat16>(const __nv_bfloat16* p, size_t i) {
  return __bfloat162float(p[i]);
}

// Rows R: RowInfo, or TreeRows for the nodes of drafted trees.
template <typename R>
constexpr bool kTree = std::is_same_v<R, TreeRows>;

// qrot[row][h][p] = RoPE(q, pos)[p] * scale * log2(e); V = ServeView: layers of starkv_load_plain, and nodes
template <typename T, typename V, typename R>
__global__ void k_qprep(V v, const T* __restrict__ q, R ri, float* __restrict__ qrot) {
  constexpr bool kServe = std::is_same_v<V, ServeView>;
  const int row = blockIdx.x, h = blockIdx.y, d = v.d, half = d / 2;
  const T* qh = q + ((size_t)row * v.H + h) * d;
  float* o = qrot + ((size_t)row * v.H + h) * d;
  if constexpr (kTree<R>) {
    if (!ri.node_pos) {   // queries are normed and rotated already
      for (int p = threadIdx.x; p < d; p += blockDim.x) o[p] = ldf(qh, p) * v.scale_log2;
      return;
    }
  }
  const int pos = row_pos_of(ri, row);
  const float* w = nullptr;   // norm weights
  float inv = 1.f;
  if constexpr (kServe) {
    w = v.q_norm;
    if (w) {
      __shared__ float red[2];
      float s = 0.f;
      for (int p = threadIdx.x; p < d; p += blockDim.x) {
        const float x = ldf(qh, p);
        s += x * x;
      }
      for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
      __syncthreads();
      inv = 1.f / sqrtf((red[0] + red[1]) / (float)d + v.norm_eps);
    }
  }
  for (int p = threadIdx.x; p < half; p += blockDim.x) {
    float a = ldf(qh, p), b = ldf(qh, p + half);
    if (w) {
      a *= inv * w[p];
      b *= inv * w[p + half];
    }
    if (v.rope) {
      double sn, cs;
      bool turns = false;
      if constexpr (kServe) {
        turns = v.opt;
        if (turns) {
          const double t = (double)pos * v.turn[p];
          sincospi(2.0 * (t - rint(t)), &sn, &cs);
        }
      }
      if (!turns) sincos((double)pos * rope_freq(p, d, v.rope_log2_theta), &sn, &cs);
      const float a2 = (float)(a * cs - b * sn), b2 = (float)(b * cs + a * sn);
      a = a2;
      b = b2;
    }
    o[p] = a * v.scale_log2;
    o[p + half] = b * v.scale_log2;
  }
}

// Scores (log2 units) S[row][h][t] for one KV head and one 64-token tile.
template <typename R>
__global__ void k_scores(LayerView v, const uint8_t* __restrict__ pool, long long n_pages,
                         const int32_t* __restrict__ pt, int max_pages, R ri, const float* __restrict__ Bk,
                         const int* __restrict__ key_off, const float* __restrict__ qrot, float* __restrict__ S,
                         int S_ld) {
  extern __shared__ float smem[];
  const int row = blockIdx.z, g = blockIdx.y, t0 = blockIdx.x * kTile;
  const int len = row_len_of(ri, row, max_pages * kPage, v.status, threadIdx.x == 0 && t0 == 0 && g == 0);
  if (t0 >= len) return;
  const int nt = min(kTile, len - t0);
  const int b = row_seq_of(ri, row);
  const LatentDesc ld = v.lat[g];
  const int r = ld.width, d = v.d, half = d / 2;
  float* zt = smem;                 // [kTile][r]
  float* Kt = zt + kTile * r;       // [kTile][d]
  for (int idx = threadIdx.x; idx < nt * r; idx += blockDim.x) {
    const int t = idx / r, j = idx % r, tok = t0 + t;
    const int page = pt[(size_t)b * max_pages + tok / kPage];
    float val = 0.f;
    if (page >= 0 && page < n_pages)
      val = latent_value(v, pool + (size_t)page * v.page_bytes + ld.block_off, ld, tok % kPage, j);
    else if (j == 0)
      atomicOr(v.status, kBadPage);
    zt[idx] = val;
  }
  __syncthreads();
  if (v.plain) {
    for (int idx = threadIdx.x; idx < nt * d; idx += blockDim.x) Kt[idx] = zt[idx];
  } else {
    const float* B = Bk + (size_t)key_off[g] * d;
    for (int idx = threadIdx.x; idx < nt * d; idx += blockDim.x) {
      const int t = idx / d, p = idx % d;
      float acc = 0.f;
      for (int j = 0; j < r; ++j) acc += zt[t * r + j] * B[(size_t)j * d + p];
      Kt[idx] = acc;
    }
    if (v.rope) {
      __syncthreads();
      for (int idx = threadIdx.x; idx < nt * half; idx += blockDim.x) {
        const int t = idx / half, p = idx % half;
        // a drafted node's key stands at the node's position, not at its slot
        int kpos = t0 + t;
        if constexpr (kTree<R>) {
          const int j = kpos - ri.row_hist[row];
          if (ri.node_pos && j >= 0) kpos = ri.node_pos[ri.node_off[b] + j];
        }
        double sn, cs;
        sincos((double)kpos * rope_freq(p, d, v.rope_log2_theta), &sn, &cs);
        const float a = Kt[t * d + p], bb = Kt[t * d + p + half];
        Kt[t * d + p] = (float)(a * cs - bb * sn);
        Kt[t * d + p + half] = (float)(bb * cs + a * sn);
      }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nt * v.group_q; idx += blockDim.x) {
    const int t = idx % nt, k = idx / nt, h = g * v.group_q + k;
    const float* qh = qrot + ((size_t)row * v.H + h) * d;
    float acc = 0.f;
    for (int p = 0; p < d; ++p) acc += qh[p] * Kt[t * d + p];
    if constexpr (kTree<R>) {
      const int j = t0 + t - ri.row_hist[row];
      if (j >= 0 && !tree_sees(ri.mask, ri.mask_words, row, ri.row_node[row], j)) acc = -FLT_MAX;
    }
    S[((size_t)row * v.H + h) * S_ld + t0 + t] = acc;
  }
}

// Value partials for one (row, split, block of value channels).  Joint
// latents: every query head reads every channel (stacked-head contraction on
// the shared latent).  Plain layers: a block lies inside one KV head's d
// channels and serves that head's query group.  Nodes have the tokens that
// they do not see at -FLT_MAX in every head; those are left out, whatever their values hold.  (A test in every product,
// for decodes and prefills too, made a decode of 4 x 1000 tokens 1.3 to 2.3 times as long.)
template <typename R>
__global__ void k_value(LayerView v, const uint8_t* __restrict__ pool, long long n_pages,
                        const int32_t* __restrict__ pt, int max_pages, R ri, const float* __restrict__ S,
                        int S_ld, int n_splits, int chunk, int vb, float* __restrict__ pY, float* __restrict__ pm,
                        float* __restrict__ pl) {
  __shared__ float m_s[32];
  __shared__ float p_s[32][33];
  __shared__ float red[kVBlock / 32];
  const int row = blockIdx.z, split = blockIdx.y, cb = blockIdx.x;
  const int len = row_len_of(ri, row, max_pages * kPage, v.status, false);
  const int ts = split * chunk, te = min(len, ts + chunk);
  const int b = row_seq_of(ri, row);
  const LatentDesc ld = v.lat[v.L - 1];
  const int c0 = cb * vb;
  const int c = c0 + threadIdx.x;
  const bool cvalid = threadIdx.x < vb && c < ld.width;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int nh = v.plain ? v.group_q : v.H;
  const int hbase = v.plain ? (c0 / v.d) * v.group_q : 0;
  const int jcol = v.plain ? c - (c0 / v.d) * v.d : c;
  const bool first_block = v.plain ? (c0 % v.d == 0) : (cb == 0);
  for (int h0 = 0; h0 < nh; h0 += 32) {
    const int nhc = min(32, nh - h0);
    float acc[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[k] = 0.f;
    float lsum = 0.f;
    for (int k = 0; k < nhc; ++k) {
      const int h = hbase + h0 + k;
      float m = -FLT_MAX;
      for (int t = ts + threadIdx.x; t < te; t += blockDim.x) m = fmaxf(m, S[((size_t)row * v.H + h) * S_ld + t]);
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) red[wid] = m;
      __syncthreads();
      if (threadIdx.x == 0) {
        float mm = red[0];
        for (int w = 1; w < (int)(blockDim.x / 32); ++w) mm = fmaxf(mm, red[w]);
        m_s[k] = mm;
      }
      __syncthreads();
    }
    for (int tt = ts; tt < te; tt += 32) {
      const int ntk = min(32, te - tt);
      for (int idx = threadIdx.x; idx < 32 * nhc; idx += blockDim.x) {
        const int t = idx % 32, k = idx / 32;
        float p = 0.f;
        if constexpr (kTree<R>) {
          if (t < ntk) {
            const float s = S[((size_t)row * v.H + hbase + h0 + k) * S_ld + tt + t];
            p = s == -FLT_MAX ? -1.f : exp2f(s - m_s[k]);   // -1: a node that the row does not see
          }
        } else if (t < ntk) {
          p = exp2f(S[((size_t)row * v.H + hbase + h0 + k) * S_ld + tt + t] - m_s[k]);
        }
        p_s[t][k] = p;
      }
      __syncthreads();
      if (threadIdx.x < nhc)
        for (int t = 0; t < ntk; ++t) lsum += kTree<R> && p_s[t][threadIdx.x] < 0.f ? 0.f : p_s[t][threadIdx.x];
      if (cvalid) {
        for (int t = 0; t < ntk; ++t) {
          if (kTree<R> && p_s[t][0] < 0.f) continue;   // (a visible value counts whatever its weight: 0 times NaN is NaN)
          const int tok = tt + t;
          const int page = pt[(size_t)b * max_pages + tok / kPage];
          float z = 0.f;
          if (page >= 0 && page < n_pages)
            z = latent_value(v, pool + (size_t)page * v.page_bytes + ld.block_off, ld, tok % kPage, c);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k < nhc) acc[k] += p_s[t][k] * z;
        }
      }
      __syncthreads();
    }
    const size_t base = ((size_t)row * n_splits + split) * v.H;
    if (cvalid)
      for (int k = 0; k < nhc; ++k) pY[(base + hbase + h0 + k) * v.wv + jcol] = acc[k];
    if (first_block && threadIdx.x < nhc) {
      pm[base + hbase + h0 + threadIdx.x] = ts < te ? m_s[threadIdx.x] : -FLT_MAX;
      pl[base + hbase + h0 + threadIdx.x] = lsum;
    }
    __syncthreads();
  }
}

template <typename TY>
__global__ void k_combine(LayerView v, RowInfo ri, int n_splits, const float* __restrict__ pY,
                          const float* __restrict__ pm, const float* __restrict__ pl, TY* __restrict__ y) {
  const int row = blockIdx.x, h = blockIdx.y;
  float m = -FLT_MAX;
  for (int s = 0; s < n_splits; ++s) m = fmaxf(m, pm[((size_t)row * n_splits + s) * v.H + h]);
  float den = 0.f;
  for (int s = 0; s < n_splits; ++s) {
    const size_t i = ((size_t)row * n_splits + s) * v.H + h;
    if (pl[i] != 0.f) den += exp2f(pm[i] - m) * pl[i];   // (NaN passes)
  }
  for (int j = threadIdx.x; j < v.wv; j += blockDim.x) {
    float acc = 0.f;
    for (int s = 0; s < n_splits; ++s) {
      const size_t i = ((size_t)row * n_splits + s) * v.H + h;
      if (pl[i] != 0.f) acc += exp2f(pm[i] - m) * pY[i * v.wv + j];
    }
    y[((size_t)row * v.H + h) * v.wv + j] = (TY)(den != 0.f ? acc / den : 0.f);
  }
}

// Same merge, written as fp16 into the swizzled B-operand tiles of the output kernel:
// row r, column k = h*wv + j lives in tile (r / NB, k / 64), row r % NB, column k % 64.
__global__ void k_combine_tiled(LayerView v, int n_splits, const float* __restrict__ pY, const float* __restrict__ pm,
                                const float* __restrict__ pl, int NB, int KT, uint8_t* __restrict__ ytiles) {
  const int row = blockIdx.x, h = blockIdx.y;
  float m = -FLT_MAX;
  for (int s = 0; s < n_splits; ++s) m = fmaxf(m, pm[((size_t)row * n_splits + s) * v.H + h]);
  float den = 0.f;
  for (int s = 0; s < n_splits; ++s) {
    const size_t i = ((size_t)row * n_splits + s) * v.H + h;
    if (pl[i] != 0.f) den += exp2f(pm[i] - m) * pl[i];   // (NaN passes)
  }
  const int nt = row / NB, r = row % NB;
  for (int j = threadIdx.x; j < v.wv; j += blockDim.x) {
    float acc = 0.f;
    for (int s = 0; s < n_splits; ++s) {
      const size_t i = ((size_t)row * n_splits + s) * v.H + h;
      if (pl[i] != 0.f) acc += exp2f(pm[i] - m) * pY[i * v.wv + j];
    }
    const uint32_t k = (uint32_t)(h * v.wv + j);
    const uint32_t c = k & 63u;
    uint8_t* tile = ytiles + ((size_t)nt * KT + (k >> 6)) * (size_t)NB * 128;
    const uint32_t off = (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u + (((c >> 3) ^ (uint32_t)(r & 7)) << 4) +
                         (c & 7u) * 2u;
    *reinterpret_cast<__half*>(tile + off) = __float2half_rn(den != 0.f ? acc / den : 0.f);
  }
}

// out[row][n] = sum_k y[row][k] * M_T[n][k]; one warp per output column, eight rows per pass.
template <typename TY, typename TO>
__global__ void k_out(const TY* __restrict__ y, const TY* __restrict__ MT, int rows, int K, int D,
                      const int32_t* __restrict__ n_rows, TO* __restrict__ out) {
  if (n_rows) rows = min(rows, *n_rows);
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (warp >= D) return;
  const TY* m = MT + (size_t)warp * K;
  for (int r0 = 0; r0 < rows; r0 += 8) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int k = lane; k < K; k += 32) {
      const float mv = ldf(m, k);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r0 + i < rows) acc[i] += mv * ldf(y, (size_t)(r0 + i) * K + k);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = acc[i];
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0 && r0 + i < rows) out[(size_t)(r0 + i) * D + warp] = (TO)s;
    }
  }
}

// Value channels per block: 128 for joint latents; inside one KV head for plain layers.
int value_block(const LayerView& v) { return v.plain ? (v.d <= kVBlock ? v.d : v.d / 2) : kVBlock; }

struct WsPlan {
  size_t qrot, S, pm, pl, pY, y, part, total;
  size_t y_bytes;
  int n_splits, chunk, S_ld;
};

size_t ru256(size_t x) { return (x + 255) / 256 * 256; }

// Token splits: enough (row, split, channel-block) blocks to fill the SMs
// twice over for decode; one split per row for prefill (rows are plenty).
WsPlan plan_ws(const starkv_layer* L, int rows, int max_len, bool prefill) {
  const LayerView& v = L->view;
  WsPlan p{};
  const int cblocks = (v.rv + value_block(v) - 1) / value_block(v);
  int ns = (int)((2 * 148 * 2 + (long long)rows * cblocks - 1) / ((long long)rows * cblocks));
  ns = std::max(1, std::min(ns, (max_len + 511) / 512));
  if (plain_decode_supported(v)) {
    // streaming plain-layer kernel: (row, KV head, split) CTAs, four or more per SM, >= 256 tokens each
    const long long per = (long long)rows * v.Hkv;
    ns = (int)std::max(1LL, std::min((4LL * num_sms() + per - 1) / per, (long long)(max_len + 255) / 256));
  }
  if (prefill) ns = 1;
  p.n_splits = ns;
  p.chunk = (max_len + ns - 1) / ns;
  p.S_ld = max_len;
  const size_t ys = v.dtype == STARKV_F32 ? 4 : 2;
  size_t o = 0;
  p.qrot = o; o += ru256(sizeof(float) * (size_t)rows * v.H * v.d);
  p.S = o;    o += ru256(sizeof(float) * (size_t)rows * v.H * max_len);
  p.pm = o;   o += ru256(sizeof(float) * (size_t)rows * ns * v.H);
  p.pl = o;   o += ru256(sizeof(float) * (size_t)rows * ns * v.H);
  p.pY = o;   o += ru256(sizeof(float) * (size_t)rows * ns * v.H * v.wv);
  if (v.dtype == STARKV_F32) {
    p.y_bytes = ys * (size_t)rows * v.H * v.wv;
    p.y = o;    o += ru256(p.y_bytes);
    p.part = o;
  } else {
    // fp16 tiles [rows / NB][Kp / 64][NB][64] (swizzled) for the tensor-core output kernel
    const int NB = outproj_nb(rows);
    const size_t ntiles = (rows + NB - 1) / NB;
    p.y_bytes = ntiles * (L->Kp / 64) * (size_t)NB * 128;
    p.y = o;    o += ru256(p.y_bytes);
    p.part = o; o += ru256(outproj_part_bytes(L, rows));
  }
  p.total = o;
  return p;
}

// The row kernels up to the merge.
template <typename R>
cudaError_t launch_rows(const starkv_layer* L, const uint8_t* pool, long long n_pages, const int32_t* page_table,
                               int max_pages, int rows, const R& ri, int max_len, const void* q, const WsPlan& p, char* w,
                               cudaStream_t s, bool tc_scores) {
  const LayerView& v = L->view;
  float* qrot = (float*)(w + p.qrot);
  float* S = (float*)(w + p.S);
  float* pm = (float*)(w + p.pm);
  float* pl = (float*)(w + p.pl);
  float* pY = (float*)(w + p.pY);
  const dim3 qgrid(rows, v.H);
  auto qprep = [&](const auto& view) {
    using V = std::decay_t<decltype(view)>;
    if (v.dtype == STARKV_F32)
      k_qprep<float, V, R><<<qgrid, 64, 0, s>>>(view, (const float*)q, ri, qrot);
    else
      k_qprep<__nv_bfloat16, V, R><<<qgrid, 64, 0, s>>>(view, (const __nv_bfloat16*)q, ri, qrot);
  };
  if constexpr (kTree<R>)
    qprep(L->view);
  else if (L->view.opt)
    qprep(L->view);
  else
    qprep(v);
  int rmax = 0;
  for (int g = 0; g < v.Hkv; ++g) rmax = std::max(rmax, L->lat[g].width);
  const size_t smem = sizeof(float) * kTile * (size_t)(rmax + v.d);
  cudaError_t e = set_smem_limit((const void*)k_scores<R>, smem);
  if (e != cudaSuccess) return e;
  const bool plain = plain_decode_supported(v) && !tc_scores && !kTree<R>;
  if (plain) {
    // uncompressed bf16 layer: one streaming pass over K and V, partials for the merge below
    e = launch_plain_decode(L, pool, n_pages, page_table, max_pages, rows, ri, qrot, p.n_splits, p.chunk, pY, pm, pl,
                            s);
    if (e != cudaSuccess) return e;
  } else if (tc_scores) {
    // scores (log2 units) from the tensor-core kernel, written into S
    ScoreOut so;
    e = launch_scores_tc(L, pool, n_pages, page_table, max_pages, rows, ri.row_len, ri.row_pos, q, w + p.total, &so,
                         S, p.S_ld, s);
    if (e != cudaSuccess) return e;
  } else {
    k_scores<R><<<dim3((max_len + kTile - 1) / kTile, v.Hkv, rows), 256, smem, s>>>(
        v, pool, n_pages, page_table, max_pages, ri, L->Bk, L->d_key_off, qrot, S, p.S_ld);
  }
  if (!plain) {
    const int vb = value_block(v);
    const int cblocks = (v.rv + vb - 1) / vb;
    k_value<R><<<dim3(cblocks, p.n_splits, rows), kVBlock, 0, s>>>(v, pool, n_pages, page_table, max_pages, ri, S, p.S_ld,
                                                                   p.n_splits, p.chunk, vb, pY, pm, pl);
  }
  return cudaGetLastError();
}

}  // namespace

size_t decode_generic_ws_bytes(const starkv_layer* L, int rows, int max_len, bool prefill) {
  return plan_ws(L, rows, max_len, prefill).total;
}

cudaError_t launch_decode_generic(const starkv_layer* L, const uint8_t* pool, long long n_pages,
                                  const int32_t* page_table, int max_pages, int rows, RowInfo ri, int max_len,
                                  const void* q, void* out, void* ws, size_t ws_bytes, bool prefill,
                                  cudaStream_t s, bool tc_scores, const TreeRows* tree) {
  const LayerView& v = L->view;
  const WsPlan p = plan_ws(L, rows, max_len, prefill);
  if (ws_bytes < p.total) return cudaErrorInvalidValue;
  char* w = (char*)ws;
  float* pm = (float*)(w + p.pm);
  float* pl = (float*)(w + p.pl);
  float* pY = (float*)(w + p.pY);
  void* y = w + p.y;
  const int32_t* n_rows = tree ? tree->n_rows : nullptr;
  cudaError_t e = tree ? launch_rows(L, pool, n_pages, page_table, max_pages, rows, *tree, max_len, q, p, w, s, tc_scores)
                       : launch_rows(L, pool, n_pages, page_table, max_pages, rows, ri, max_len, q, p, w, s, tc_scores);
  if (e != cudaSuccess) return e;
  if (v.dtype == STARKV_F32) {
    k_combine<float><<<dim3(rows, v.H), 128, 0, s>>>(v, ri, p.n_splits, pY, pm, pl, (float*)y);
    k_out<float, float><<<(v.D * 32 + 255) / 256, 256, 0, s>>>((const float*)y, (const float*)L->M_T, rows,
                                                                v.H * v.wv, v.D, n_rows, (float*)out);
    return cudaGetLastError();
  }
  const int NB = outproj_nb(rows);
  const int KT = L->Kp / 64;
  // padding rows and columns of the y tiles must be zero
  if (rows % NB != 0 || L->Kp != v.H * v.wv) {
    e = cudaMemsetAsync(y, 0, p.y_bytes, s);
    if (e != cudaSuccess) return e;
  }
  k_combine_tiled<<<dim3(rows, v.H), 128, 0, s>>>(v, p.n_splits, pY, pm, pl, NB, KT, (uint8_t*)y);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_outproj_tc(L, y, rows, out, (float*)(w + p.part), s, n_rows);
}

namespace {

// A tree call's rows go through the row kernels in batches of at most this many, so that their score buffer (one fp32
// per row, head and slot) stays bounded.
constexpr int kTreeRows = 64;

// Row tables of a tree call: row -> sequence, visible length, position, history, node.  One thread per row; rows that
// belong to no sequence get length 0.  n_rows[c]: rows in use of batch c.
__global__ void k_tree_rows(LayerView v, const int32_t* __restrict__ hist, const int32_t* __restrict__ node_off,
                            int batch, int n_nodes, int max_nodes, int cap, const int32_t* __restrict__ q_pos,
                            int32_t* __restrict__ row_seq, int32_t* __restrict__ row_len, int32_t* __restrict__ row_pos,
                            int32_t* __restrict__ row_hist, int32_t* __restrict__ row_node,
                            int32_t* __restrict__ n_rows) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= n_nodes) return;
  if (r % kTreeRows == 0)
    n_rows[r / kTreeRows] = min(max(min(node_off[batch], n_nodes) - r, 0), kTreeRows);
  int32_t seq = 0, len = 0, h = 0, node = 0;
  bool back = false;   // a node_off that decreases: every row is zero
  for (int b = 0; b < batch; ++b) back = back || node_off[b + 1] < node_off[b];
  if (back && r == 0) atomicOr(v.status, kBadPos);
  for (int b = 0; b < batch && !back; ++b) {
    if (r < node_off[b] || r >= node_off[b + 1]) continue;
    const TreeSeq q = tree_seq(hist, node_off, b, n_nodes, max_nodes, cap, v.status, r == node_off[b]);
    seq = b;
    len = q.cnt ? q.hist + q.cnt : 0;
    h = q.hist;
    node = r - q.off;
    break;
  }
  row_seq[r] = seq;
  row_len[r] = len;
  row_pos[r] = q_pos ? q_pos[r] : 0;
  row_hist[r] = h;
  row_node[r] = node;
}

size_t tree_tab_bytes(int n_nodes) {
  return ru256(sizeof(int32_t) * (5 * (size_t)n_nodes + (size_t)(n_nodes + kTreeRows - 1) / kTreeRows));
}

}  // namespace

size_t tree_generic_need(const starkv_layer* L, int max_ctx, int n_nodes) {
  size_t most = 0;   // of the full batches and the last one, whose fewer rows may take more splits
  if (n_nodes >= kTreeRows) most = decode_generic_ws_bytes(L, kTreeRows, max_ctx, false);
  if (n_nodes % kTreeRows) most = std::max(most, decode_generic_ws_bytes(L, n_nodes % kTreeRows, max_ctx, false));
  return tree_tab_bytes(n_nodes) + most;
}

size_t tree_generic_ws_bytes(const starkv_layer* L, int max_ctx, int n_nodes) {
  size_t most = 0;
  for (int r = 1; r <= std::min(n_nodes, kTreeRows); ++r) most = std::max(most, decode_generic_ws_bytes(L, r, max_ctx, false));
  return tree_tab_bytes(n_nodes) + most;
}

// Every node as one row of the CUDA-core kernels, with its mask.
cudaError_t launch_tree_generic(const starkv_layer* L, const TreeArgs& t, void* ws, size_t ws_bytes, cudaStream_t s) {
  const int n = t.n_nodes, max_len = t.max_pages * kPage;
  int32_t* tab = (int32_t*)ws;
  const size_t tab_bytes = tree_tab_bytes(n);
  if (ws_bytes < tree_generic_need(L, max_len, n)) return cudaErrorInvalidValue;
  k_tree_rows<<<(n + 127) / 128, 128, 0, s>>>(L->view, t.hist, t.node_off, t.batch, n, t.max_nodes, max_len, t.q_pos,
                                              tab, tab + n, tab + 2 * n, tab + 3 * n, tab + 4 * n, tab + 5 * n);
  cudaError_t e = cudaGetLastError();
  const size_t es = L->view.dtype == STARKV_F32 ? 4 : 2;
  for (int r0 = 0; r0 < n && e == cudaSuccess; r0 += kTreeRows) {
    TreeRows ri{{tab + r0, tab + n + r0, tab + 2 * n + r0}};
    ri.row_hist = tab + 3 * n + r0;
    ri.row_node = tab + 4 * n + r0;
    ri.n_rows = tab + 5 * n + r0 / kTreeRows;
    ri.mask = t.mask ? t.mask + (size_t)r0 * t.mask_words : nullptr;
    ri.mask_words = t.mask_words;
    ri.node_off = t.node_off;
    ri.node_pos = t.q_pos;
    e = launch_decode_generic(L, t.pool, t.n_pages, t.pt, t.max_pages, std::min(kTreeRows, n - r0), ri, max_len,
                              (const char*)t.q + (size_t)r0 * L->view.H * L->view.d * es,
                              (char*)t.out + (size_t)r0 * L->view.D * es, (char*)ws + tab_bytes, ws_bytes - tab_bytes,
                              false, s, false, &ri);
  }
  return e;
}

}  // namespace starkv
