// The cache of uncompressed layers as a serving loop writes and reads it:
// per-head RMS norms of queries and keys with the position rotation in the
// same pass, K and V stored (or quantised) into their pages in that pass too,
// tokens read back as dense rows, and the accepted path of a drafted tree
// moved to the front of its slots.
//
// Norm and rotation of one head's d channels x (half = d / 2, p < half):
//   x'  = x * rsqrt(mean(x^2) + eps) * w                       (only where the layer has weights)
//   y[p] = x'[p] cos a - x'[p + half] sin a,  y[p + half] = x'[p + half] cos a + x'[p] sin a,
//   a = position * theta^(-2p/d), reduced in 64 bits (as turns: the fraction of position * f / 2 pi)
// Quantiser (kv_bits b, groups of 32 channels, qmax = 2^(b-1) - 1): scale = amax * fl(1 / qmax) in fp32, rounded
// up to fp16; code = rne(x / scale) + 2^(b-1), the fp32 division.
#include <float.h>

#include "starkv_internal.cuh"

namespace starkv {

namespace {

constexpr int kKvThreads = 256;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;   // elements of a 16-byte load
  static __device__ __forceinline__ void load(const float* p, float* f) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float f) { *p = f; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }
};

// Where a token's K and V go: its page, or null (flagged) when the slot does not exist.
__device__ __forceinline__ uint8_t* slot_page(const KvArgs& a, int i, int* slot, bool flag) {
  const int b = a.seq_idx[i], t = a.slots[i];
  if (b < 0 || b >= a.n_seqs || t < 0 || t >= a.max_pages * kPage) {
    if (flag) atomicOr(a.v.status, kBadPos);
    return nullptr;
  }
  const int page = a.pt[(size_t)b * a.max_pages + t / kPage];
  if (page < 0 || page >= a.n_pages) {
    if (flag) atomicOr(a.v.status, kBadPage);
    return nullptr;
  }
  *slot = t % kPage;
  return a.pool + (size_t)page * a.v.page_bytes;
}

// cos and sin of position * f_p, f_p in turns per position.
__device__ __forceinline__ void angle(double turns, double* sn, double* cs) {
  sincospi(2.0 * (turns - rint(turns)), sn, cs);
}

// Norm and rotation of a row held as lo[V], hi[V] (channels V c .., half + V c ..) by a group of LPR lanes, in the
// arithmetic F: float for what is rounded to 16 bits or compared in fp32, double for keys that a quantiser rounds
// next, so that codes and scales do not depend on the order of a sum (packed pages equal the definition's bit for bit).
template <typename F, int V, int LPR>
__device__ __forceinline__ void norm_rotate(float* lo, float* hi, const float* w, float eps, int half, int c,
                                            const double2* cs, bool rope) {
  F x[V], y[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    x[k] = (F)lo[k];
    y[k] = (F)hi[k];
  }
  if (w) {
    F s = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) s += x[k] * x[k] + y[k] * y[k];
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const F inv = F(1) / sqrt(s / F(2 * half) + (F)eps);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[k] *= inv * (F)w[c * V + k];
      y[k] *= inv * (F)w[half + c * V + k];
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (rope) {
      const double2 t = cs[c * V + k];
      const F cc = (F)t.x, ss = (F)t.y;
      lo[k] = (float)(x[k] * cc - y[k] * ss);
      hi[k] = (float)(y[k] * cc + x[k] * ss);
    } else {
      lo[k] = (float)x[k];
      hi[k] = (float)y[k];
    }
  }
}

// V consecutive channels (starting at channel ch of a latent block `blk` with its groups at codes + g * stride),
// quantised: the group of 32 channels is spread over GL = 32 / V lanes.  BITS 8 or 4.
template <int BITS, int V>
__device__ __forceinline__ void quant_store(const float* x, uint8_t* blk, int scale_bytes, int group, int ch, int slot,
                                            bool live, uint32_t* status) {
  constexpr int GL = 32 / V, QM = (1 << (BITS - 1)) - 1, GB = kPage * 32 * BITS / 8;
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    amax = fmaxf(amax, fabsf(x[k]));
    nan = nan || (x[k] != x[k]);
  }
  if (nan) amax = INFINITY;   // fmaxf drops NaN
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!live) return;
  const bool fits = amax <= kKvMax;
  const float s32 = fits ? __fmul_rn(amax, 1.f / (float)QM) : 0.f;
  const __half s16 = __float2half_ru(s32);
  const float sf = __half2float(s16);
  uint32_t u[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    int q = 0;
    if (sf != 0.f) q = min(max(__float2int_rn(__fdiv_rn(x[k], sf)), -QM), QM);
    u[k] = (uint32_t)(q + QM + 1);
  }
  uint8_t* dst = blk + scale_bytes + (size_t)group * GB + (size_t)slot * (32 * BITS / 8) + ch * BITS / 8;
  if constexpr (BITS == 8) {
    uint32_t w[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) w[k] = u[4 * k] | u[4 * k + 1] << 8 | u[4 * k + 2] << 16 | u[4 * k + 3] << 24;
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) w |= u[k] << (4 * k);
    if constexpr (V == 8)
      *reinterpret_cast<uint32_t*>(dst) = w;
    else
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w;
  }
  if (ch == 0) {
    reinterpret_cast<__half*>(blk)[group * kPage + slot] = s16;
    if (!fits) atomicOr(status, kScaleOvf);
  }
}

// One row (head) per group of LPR lanes; a CTA takes TOK consecutive tokens and the heads blockIdx.y, + gridDim.y ...
// of its row groups.  The tokens' cos / sin (64-bit) are made once per CTA and shared by all heads.
// Bound: bytes (2 loads of 16 B and their stores a lane).
template <typename T, int D, int BITS, int TOK>
__global__ void __launch_bounds__(kKvThreads) k_qkv(KvArgs a) {
  constexpr int V = Vec<T>::N, HALF = D / 2, LPR = HALF / V, GROUPS = kKvThreads / LPR;
  __shared__ double2 cs[TOK][HALF];
  const LayerView& v = a.v;
  const int i0 = blockIdx.x * TOK;
  if (a.rotate) {
    for (int e = threadIdx.x; e < TOK * HALF; e += kKvThreads) {
      const int i = i0 + e / HALF, p = e % HALF;
      if (i < a.n) {
        double sn, c;
        angle((double)a.positions[i] * a.turn[p], &sn, &c);
        cs[e / HALF][p] = make_double2(c, sn);
      }
    }
    __syncthreads();
  }
  const int c = threadIdx.x % LPR, row0 = blockIdx.y * GROUPS + threadIdx.x / LPR;
  const int nq = a.q ? v.H : 0, nk = a.k ? v.Hkv : 0, nv = a.vv ? v.Hkv : 0, rows = nq + nk + nv;
  // every lane of a warp makes the same number of trips (the shuffles inside are warp-wide)
  for (int r0 = row0; r0 - threadIdx.x / LPR < rows * TOK; r0 += gridDim.y * GROUPS) {
    const int tok = r0 / rows, hr = r0 % rows, i = i0 + tok;
    const bool live = r0 < rows * TOK && i < a.n;
    const int kind = hr < nq ? 0 : (hr < nq + nk ? 1 : 2);
    const int h = hr - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
    const T* src = kind == 0 ? (const T*)a.q + (size_t)i * a.q_ld
                             : kind == 1 ? (const T*)a.k + (size_t)i * a.k_ld : (const T*)a.vv + (size_t)i * a.v_ld;
    float lo[V], hi[V];
    if (live) {
      Vec<T>::load(src + (size_t)h * D + c * V, lo);
      Vec<T>::load(src + (size_t)h * D + HALF + c * V, hi);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) lo[k] = hi[k] = 0.f;
    }
    if (BITS != 0) {
      // keys that are quantised next go through 64-bit arithmetic; the warp takes both branches only where its rows
      // hold keys and others
      const bool wide = kind == 1 && a.pool != nullptr;
      const unsigned any = __ballot_sync(0xffffffffu, wide), all = 0xffffffffu;
      if (any) {
        float l2[V], h2[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          l2[k] = lo[k];
          h2[k] = hi[k];
        }
        norm_rotate<double, V, LPR>(l2, h2, v.k_norm, v.norm_eps, HALF, c, cs[live ? tok : 0],
                                    a.rotate);
        if (wide) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            lo[k] = l2[k];
            hi[k] = h2[k];
          }
        }
      }
      if (any != all) {
        float l2[V], h2[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          l2[k] = lo[k];
          h2[k] = hi[k];
        }
        norm_rotate<float, V, LPR>(l2, h2, kind == 0 ? v.q_norm : v.k_norm, v.norm_eps, HALF, c,
                                   cs[live ? tok : 0], a.rotate);
        if (kind == 0 || (kind == 1 && !wide)) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            lo[k] = l2[k];
            hi[k] = h2[k];
          }
        }
      }
    } else {
      float l2[V], h2[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        l2[k] = lo[k];
        h2[k] = hi[k];
      }
      norm_rotate<float, V, LPR>(l2, h2, kind == 0 ? v.q_norm : v.k_norm, v.norm_eps, HALF, c,
                                 cs[live ? tok : 0], a.rotate);
      if (kind != 2) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          lo[k] = l2[k];
          hi[k] = h2[k];
        }
      }
    }
    if (kind == 0) {
      if (live) {
        T* o = (T*)a.q_out + (size_t)i * a.q_out_ld + (size_t)h * D;
        Vec<T>::store(o + c * V, lo);
        Vec<T>::store(o + HALF + c * V, hi);
      }
    } else if (a.pool == nullptr) {
      if (live) {
        T* o = (T*)a.k_out + (size_t)i * a.k_out_ld + (size_t)h * D;
        Vec<T>::store(o + c * V, lo);
        Vec<T>::store(o + HALF + c * V, hi);
      }
    }
    if (a.pool != nullptr) {
      int slot = 0;
      uint8_t* page = live && kind ? slot_page(a, i, &slot, c == 0 && h == 0) : nullptr;
      const LatentDesc& ld = v.lat[kind == 2 ? v.L - 1 : h];
      if constexpr (BITS != 0) {
        uint8_t* blk = page ? page + ld.block_off : nullptr;
        const int g0 = (kind == 2 ? h * (D / 32) : 0), ch = c * V;
        quant_store<BITS, V>(lo, blk, ld.scale_bytes, g0 + ch / 32, ch % 32, slot, page != nullptr, v.status);
        quant_store<BITS, V>(hi, blk, ld.scale_bytes, g0 + (HALF + ch) / 32, (HALF + ch) % 32, slot, page != nullptr,
                             v.status);
      } else if (page) {
        const size_t o = (size_t)slot * ld.width + (kind == 2 ? (size_t)h * D : 0) + c * V;
        if (v.es == 4) {
          float* d = reinterpret_cast<float*>(page + ld.block_off) + o;
#pragma unroll
          for (int k = 0; k < V; k += 4) {
            Vec<float>::store(d + k, lo + k);
            Vec<float>::store(d + HALF + k, hi + k);
          }
        } else {
          __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(page + ld.block_off) + o;
#pragma unroll
          for (int k = 0; k < V; k += 2) {
            *reinterpret_cast<__nv_bfloat162*>(d + k) = __floats2bfloat162_rn(lo[k], lo[k + 1]);
            *reinterpret_cast<__nv_bfloat162*>(d + HALF + k) = __floats2bfloat162_rn(hi[k], hi[k + 1]);
          }
        }
      }
    }
  }
}

// Any even head_dim up to 256, unquantised pages: one warp per row, a lane per pair.
template <typename T>
__global__ void __launch_bounds__(kKvThreads) k_qkv_any(KvArgs a) {
  const LayerView& v = a.v;
  const int half = v.d / 2, lane = threadIdx.x & 31;
  const int nq = a.q ? v.H : 0, nk = a.k ? v.Hkv : 0, nv = a.vv ? v.Hkv : 0, rows = nq + nk + nv;
  const long long w = ((long long)blockIdx.x * kKvThreads + threadIdx.x) >> 5;
  if (w >= (long long)rows * a.n) return;
  const int i = (int)(w / rows), hr = (int)(w % rows);
  const int kind = hr < nq ? 0 : (hr < nq + nk ? 1 : 2);
  const int h = hr - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
  const T* src = kind == 0 ? (const T*)a.q + (size_t)i * a.q_ld
                           : kind == 1 ? (const T*)a.k + (size_t)i * a.k_ld : (const T*)a.vv + (size_t)i * a.v_ld;
  src += (size_t)h * v.d;
  const float* nw = kind == 0 ? v.q_norm : kind == 1 ? v.k_norm : nullptr;
  float inv = 1.f;
  if (nw) {
    float s = 0.f;
    for (int p = lane; p < v.d; p += 32) {
      const float x = Vec<T>::get(src + p);
      s += x * x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    inv = 1.f / sqrtf(s / (float)v.d + v.norm_eps);
  }
  int slot = 0;
  uint8_t* page = a.pool && kind ? slot_page(a, i, &slot, lane == 0 && h == 0) : nullptr;
  if (a.pool && kind && !page) return;
  for (int p = lane; p < half; p += 32) {
    float x = Vec<T>::get(src + p), y = Vec<T>::get(src + p + half);
    if (nw) {
      x *= inv * nw[p];
      y *= inv * nw[p + half];
    }
    if (a.rotate && kind != 2) {
      double sn, c;
      angle((double)a.positions[i] * a.turn[p], &sn, &c);
      const float cc = (float)c, ss = (float)sn, x2 = x * cc - y * ss;
      y = y * cc + x * ss;
      x = x2;
    }
    if (page) {
      const LatentDesc& ld = v.lat[kind == 2 ? v.L - 1 : h];
      const size_t o = (size_t)slot * ld.width + (kind == 2 ? (size_t)h * v.d : 0);
      if (v.es == 4) {
        float* d = reinterpret_cast<float*>(page + ld.block_off) + o;
        d[p] = x;
        d[p + half] = y;
      } else {
        __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(page + ld.block_off) + o;
        d[p] = __float2bfloat16_rn(x);
        d[p + half] = __float2bfloat16_rn(y);
      }
    } else {
      T* o = kind == 0 ? (T*)a.q_out + (size_t)i * a.q_out_ld : (T*)a.k_out + (size_t)i * a.k_out_ld;
      Vec<T>::put(o + (size_t)h * v.d + p, x);
      Vec<T>::put(o + (size_t)h * v.d + p + half, y);
    }
  }
}

template <typename T, int D, int BITS>
cudaError_t launch_qkv_d(const KvArgs& a, cudaStream_t s) {
  constexpr int GROUPS = kKvThreads / (D / 2 / Vec<T>::N);
  const int rows = (a.q ? a.v.H : 0) + (a.k ? a.v.Hkv : 0) + (a.vv ? a.v.Hkv : 0);
  // Few tokens: a token per CTA and its heads over several CTAs, for latency; many: four tokens share a CTA, whose
  // rows then hide each other's loads.
  if (a.n < 4 * num_sms()) {
    const dim3 grid((unsigned)a.n, (unsigned)((rows + GROUPS - 1) / GROUPS));
    k_qkv<T, D, BITS, 1><<<grid, kKvThreads, 0, s>>>(a);
  } else {
    k_qkv<T, D, BITS, 4><<<(unsigned)((a.n + 3) / 4), kKvThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_qkv_t(const KvArgs& a, cudaStream_t s) {
  const int d = a.v.d, bits = a.pool ? a.v.kv_bits : 0;
#define STARKV_QKV(DD)                                         \
  if (d == DD) {                                               \
    if (bits == 8) return launch_qkv_d<T, DD, 8>(a, s);        \
    if (bits == 4) return launch_qkv_d<T, DD, 4>(a, s);        \
    if (a.vec) return launch_qkv_d<T, DD, 0>(a, s);            \
  }
  STARKV_QKV(64)
  STARKV_QKV(128)
  STARKV_QKV(256)
#undef STARKV_QKV
  const long long rows = (long long)a.n * ((a.q ? a.v.H : 0) + (a.k ? a.v.Hkv : 0) + (a.vv ? a.v.Hkv : 0));
  k_qkv_any<T><<<(unsigned)((rows * 32 + kKvThreads - 1) / kKvThreads), kKvThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ reading back
// Rows [n][latent_total] of cached tokens in TO.  One thread per 8 channels of a token where the page's bytes allow it
// (uncompressed layers: 8 codes are 8 or 4 bytes, 8 values 16 or 32), so consecutive threads write one row in order;
// other layers an element at a time.
template <typename TO, int BITS>   // BITS 0: stored in the layer dtype TO
__global__ void __launch_bounds__(256) k_read8(KvArgs a, TO* __restrict__ out) {
  const LayerView& v = a.v;
  const int chunks = v.Ltot / 8;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= (long long)a.n * chunks) return;
  const int i = (int)(e / chunks), ch = (int)(e % chunks) * 8;
  int slot = 0;
  const uint8_t* page = slot_page(a, i, &slot, ch == 0);
  float f[8];
  if (!page) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.f;
  } else {
    const bool val = ch >= v.Rk;
    const LatentDesc& ld = v.lat[val ? v.L - 1 : ch / v.d];
    const int j = val ? ch - v.Rk : ch % v.d;
    const uint8_t* blk = page + ld.block_off;
    if constexpr (BITS == 0) {
      const TO* p = reinterpret_cast<const TO*>(blk) + (size_t)slot * ld.width + j;
#pragma unroll
      for (int k = 0; k < 8; k += Vec<TO>::N) Vec<TO>::load(p + k, f + k);
    } else {
      constexpr int GB = kPage * 32 * BITS / 8;
      const int g = j / 32;
      const float s = __half2float(reinterpret_cast<const __half*>(blk)[g * kPage + slot]);
      const uint8_t* c = blk + ld.scale_bytes + (size_t)g * GB + (size_t)slot * (32 * BITS / 8) + (j % 32) * BITS / 8;
      uint32_t w[2];
      if constexpr (BITS == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(c);
        w[0] = u.x;
        w[1] = u.y;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = (float)((int)((w[k / 4] >> (8 * (k % 4))) & 255u) - 128) * s;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(c);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = (float)((int)((w[0] >> (4 * k)) & 15u) - 8) * s;
      }
    }
  }
  TO* o = out + (size_t)i * v.Ltot + ch;
#pragma unroll
  for (int k = 0; k < 8; k += Vec<TO>::N) Vec<TO>::store(o + k, f + k);
}

template <typename TO>
__global__ void __launch_bounds__(256) k_read_any(KvArgs a, TO* __restrict__ out) {
  const LayerView& v = a.v;
  const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;   // a warp per (token, latent)
  if (w >= (long long)a.n * v.L) return;
  const int i = (int)(w / v.L), li = (int)(w % v.L), lane = threadIdx.x & 31;
  int slot = 0;
  const uint8_t* page = slot_page(a, i, &slot, lane == 0 && li == 0);
  const LatentDesc ld = v.lat[li];
  for (int j = lane; j < ld.width; j += 32)
    Vec<TO>::put(out + (size_t)i * v.Ltot + ld.ch_off + j, page ? latent_value(v, page + ld.block_off, ld, slot, j) : 0.f);
}

// ------------------------------------------------------------------ accepting a path
// Sequence b's nodes lie in slots hist .. hist + cnt - 1.  Slot hist + acc[k] moves to hist + k for k < n_acc; the
// slots hist + n_acc .. hist + cnt - 1 are cleared (appends OR codes into compressed layers' slots).  acc is strictly
// increasing, so acc[k] >= k, and taking k in order never overwrites a slot that is still to be read.  What moves is
// the slot's column of one group, always by the same lanes, so the order of k needs no wait between warps.
struct AcceptArgs {
  LayerView v;
  uint8_t* pool;
  long long n_pages;
  const int32_t* pt;
  int max_pages, batch, n_nodes, max_nodes;
  const int32_t *hist, *node_off, *acc, *n_acc;
  const int* grp_lat;
  int n_grp;
};

// One warp per (sequence, group).
__global__ void __launch_bounds__(256) k_accept(AcceptArgs a) {
  const LayerView& v = a.v;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  if (w >= (long long)a.batch * a.n_grp) return;
  const int b = (int)(w / a.n_grp), fg = (int)(w % a.n_grp);
  const TreeSeq q = tree_seq(a.hist, a.node_off, b, a.n_nodes, a.max_nodes, a.max_pages * kPage, v.status,
                             fg == 0 && lane == 0);
  if (q.cnt <= 0) return;
  const int n_acc = a.n_acc[b];
  // the path must be increasing node numbers of this sequence; a sequence whose path is not is left as it was
  bool ok = n_acc >= 0 && n_acc <= q.cnt;
  for (int k = lane; ok && k < n_acc; k += 32) {
    const int x = a.acc[q.off + k], prev = k ? a.acc[q.off + k - 1] : -1;
    if (x <= prev || x >= q.cnt) ok = false;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    if (lane == 0 && fg == 0) atomicOr(v.status, kBadPos);
    return;
  }
  const LatentDesc ld = v.lat[a.grp_lat[fg]];
  const GroupDesc gd = v.grp[fg];
  const int g = fg - ld.group0;
  // bytes of one slot of this group when they are whole and in one run
  const int run = ld.cmajor ? 0 : (v.quantized ? (gd.n * gd.bits % 8 ? 0 : gd.n * gd.bits / 8) : gd.n * v.es);
  for (int k = 0; k < q.cnt; ++k) {
    const bool kept = k < n_acc;
    const int src_t = q.hist + (kept ? a.acc[q.off + k] : k), dst_t = q.hist + k;
    if (kept && src_t == dst_t) continue;
    const int sp = a.pt[(size_t)b * a.max_pages + src_t / kPage], dp = a.pt[(size_t)b * a.max_pages + dst_t / kPage];
    if (sp < 0 || sp >= a.n_pages || dp < 0 || dp >= a.n_pages) {
      if (lane == 0 && fg == 0) atomicOr(v.status, kBadPage);
      continue;
    }
    const uint8_t* sb = a.pool + (size_t)sp * v.page_bytes + ld.block_off;
    uint8_t* db = a.pool + (size_t)dp * v.page_bytes + ld.block_off;
    const int ss = src_t % kPage, ds = dst_t % kPage;
    if (v.quantized && lane == 0) {
      const __half* sh = reinterpret_cast<const __half*>(sb) + g * kPage + ss;
      reinterpret_cast<__half*>(db)[g * kPage + ds] = kept ? *sh : __float2half_rn(0.f);
    }
    if (run) {
      const uint8_t* s8 = sb + gd.code_off + (size_t)ss * run;
      uint8_t* d8 = db + gd.code_off + (size_t)ds * run;
      if ((run & 1) == 0) {
        for (int x = lane; x < run / 2; x += 32)
          reinterpret_cast<uint16_t*>(d8)[x] = kept ? reinterpret_cast<const uint16_t*>(s8)[x] : (uint16_t)0;
      } else {
        for (int x = lane; x < run; x += 32) d8[x] = kept ? s8[x] : (uint8_t)0;
      }
    } else if (!v.quantized) {
      // channel-major values of an unquantised latent
      for (int j = lane; j < gd.n; j += 32) {
        const size_t so = elem_index(ss, gd.start + j, ld.width, ld.cmajor), dn = elem_index(ds, gd.start + j, ld.width, ld.cmajor);
        if (v.es == 4)
          reinterpret_cast<uint32_t*>(db)[dn] = kept ? reinterpret_cast<const uint32_t*>(sb)[so] : 0u;
        else
          reinterpret_cast<uint16_t*>(db)[dn] = kept ? reinterpret_cast<const uint16_t*>(sb)[so] : (uint16_t)0;
      }
    } else {
      // codes that share 32-bit words with other channels or slots: read past L1, clear and set the field's bits
      uint32_t u = 0;
      const uint32_t msk = (1u << gd.bits) - 1u;
      if (lane < gd.n && kept) {
        const uint32_t bit = code_bit(ss, lane, gd.n, gd.bits, ld.cmajor);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(sb + gd.code_off) + (bit >> 5);
        const uint32_t sh = bit & 31;
        u = __ldcg(p) >> sh;
        if (sh + gd.bits > 32) u |= __ldcg(p + 1) << (32 - sh);
        u &= msk;
      }
      __syncwarp();
      if (lane < gd.n) {
        const uint32_t bit = code_bit(ds, lane, gd.n, gd.bits, ld.cmajor);
        uint32_t* p = reinterpret_cast<uint32_t*>(db + gd.code_off) + (bit >> 5);
        const uint32_t sh = bit & 31;
        atomicAnd(p, ~(msk << sh));
        if (u << sh) atomicOr(p, u << sh);
        if (sh + gd.bits > 32) {
          atomicAnd(p + 1, ~(msk >> (32 - sh)));
          if (u >> (32 - sh)) atomicOr(p + 1, u >> (32 - sh));
        }
      }
      __threadfence();
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_qkv(const KvArgs& a, bool f32, cudaStream_t s) {
  return f32 ? launch_qkv_t<float>(a, s) : launch_qkv_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_cache_read(const KvArgs& a, void* out, cudaStream_t s) {
  const LayerView& v = a.v;
  const bool f32 = v.dtype == STARKV_F32;
  const long long threads = (long long)a.n * (v.Ltot / 8);
  const unsigned grid = (unsigned)((threads + 255) / 256);
  // eight channels a thread: rows of whole 8-channel chunks whose codes are 8 or 4 bits wide, or stored values
  if (v.plain && v.d % 8 == 0 && (v.kv_bits || !v.quantized)) {
    if (f32) {
      if (v.kv_bits == 8) k_read8<float, 8><<<grid, 256, 0, s>>>(a, (float*)out);
      else if (v.kv_bits == 4) k_read8<float, 4><<<grid, 256, 0, s>>>(a, (float*)out);
      else k_read8<float, 0><<<grid, 256, 0, s>>>(a, (float*)out);
    } else {
      if (v.kv_bits == 8) k_read8<__nv_bfloat16, 8><<<grid, 256, 0, s>>>(a, (__nv_bfloat16*)out);
      else if (v.kv_bits == 4) k_read8<__nv_bfloat16, 4><<<grid, 256, 0, s>>>(a, (__nv_bfloat16*)out);
      else k_read8<__nv_bfloat16, 0><<<grid, 256, 0, s>>>(a, (__nv_bfloat16*)out);
    }
  } else {
    const unsigned gw = (unsigned)(((long long)a.n * v.L * 32 + 255) / 256);
    if (f32) k_read_any<float><<<gw, 256, 0, s>>>(a, (float*)out);
    else k_read_any<__nv_bfloat16><<<gw, 256, 0, s>>>(a, (__nv_bfloat16*)out);
  }
  return cudaGetLastError();
}

cudaError_t launch_accept(const starkv_layer* L, uint8_t* pool, long long n_pages, const int32_t* pt, int max_pages,
                          int batch, const int32_t* hist, const int32_t* node_off, int n_nodes, int max_nodes,
                          const int32_t* acc, const int32_t* n_acc, cudaStream_t s) {
  AcceptArgs a{L->view, pool, n_pages, pt, max_pages, batch, n_nodes, max_nodes, hist, node_off, acc, n_acc,
               L->d_grp_lat, (int)L->grp.size()};
  const long long warps = (long long)batch * a.n_grp;
  k_accept<<<(unsigned)((warps * 32 + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace starkv
