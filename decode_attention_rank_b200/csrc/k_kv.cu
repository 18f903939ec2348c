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

#include <type_traits>

#include "tc_common.cuh"

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

// Packed pairs of fp32 numbers (one register pair, one instruction for two products).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk(f32x2 x, float* a) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a[0]), "=f"(a[1]) : "l"(x)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A lane's factors for one kind of row: w cos and w sin of its channels' two halves (1 for no weights, no rotation), so that
// a row costs two products an element and one by its norm.
template <int V>
struct Factors {
  f32x2 lc[V / 2], hs[V / 2], hc[V / 2], ls[V / 2];   // w_lo cos, -w_hi sin, w_hi cos, w_lo sin
};

// 1 / sqrt(mean square + eps) of a row spread over LPR lanes.
template <int V, int LPR>
__device__ __forceinline__ float inv_rms(const float* lo, const float* hi, float eps, float rd) {
  f32x2 a = pk(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    const f32x2 x = pk(lo[k], lo[k + 1]), y = pk(hi[k], hi[k + 1]);
    a = fma2(x, x, a);
    a = fma2(y, y, a);
  }
  float s[2];
  upk(a, s);
  float t = s[0] + s[1];
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return rsqrtf(fmaf(t, rd, eps));
}

// lo, hi -> the normed and rotated row.
template <int V>
__device__ __forceinline__ void rotate_row(float* lo, float* hi, const Factors<V>& f, float inv) {
  const f32x2 i2 = pk(inv, inv);
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const f32x2 x = pk(lo[2 * k], lo[2 * k + 1]), y = pk(hi[2 * k], hi[2 * k + 1]);
    upk(mul2(fma2(x, f.lc[k], mul2(y, f.hs[k])), i2), lo + 2 * k);
    upk(mul2(fma2(y, f.hc[k], mul2(x, f.ls[k])), i2), hi + 2 * k);
  }
}

// The same in 64 bits, for keys that a quantiser rounds next, so that codes and scales do not depend on the order of a sum
// (packed pages equal the definition's bit for bit).  EXACT: x * w is exact in fp32 (bf16 rows and weights).
template <int V, int LPR, bool EXACT>
__device__ __forceinline__ void norm_rotate64(float* lo, float* hi, const float* wl, const float* wh, bool norm, double eps,
                                              int d, const double2* cs, bool rope) {
  double inv = 1;
  if (norm) {
    double s = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (EXACT) {   // squares of bf16 numbers are exact in fp32
        s += (double)(lo[k] * lo[k]);
        s += (double)(hi[k] * hi[k]);
      } else {
        s += (double)lo[k] * (double)lo[k];
        s += (double)hi[k] * (double)hi[k];
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    inv = rsqrt(s * (1.0 / d) + eps);   // d is a power of two
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    double x = EXACT ? (double)(lo[k] * wl[k]) : (double)lo[k] * (double)wl[k];
    double y = EXACT ? (double)(hi[k] * wh[k]) : (double)hi[k] * (double)wh[k];
    if (rope) {
      const double2 t = cs[k * LPR];
      const double z = x * t.x - y * t.y;
      y = y * t.x + x * t.y;
      x = z;
    }
    lo[k] = (float)(x * inv);
    hi[k] = (float)(y * inv);
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
  // code = rne(x / s): the product with 1 / s is within 2^-21 of the quotient's size (<= 127 and a rounding), so only a
  // product that close to a border needs the division itself.  Adding 1.5 * 2^23 (and the even offset 2^(b-1)) rounds to an integer, to even
  // at ties, and leaves it in the low bits; |x| <= amax keeps it inside the code's range.
  const float rs = sf != 0.f ? __fdiv_rn(1.f, sf) : 0.f;
  constexpr float magic = 12582912.f + (float)(QM + 1);
  uint32_t u[V];
  float near = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float y = x[k] * rs, z = y + magic;
    near = fmaxf(near, fabsf(y - (z - magic)));
    u[k] = __float_as_uint(z);
  }
  if (!fits) {
#pragma unroll
    for (int k = 0; k < V; ++k) u[k] = QM + 1;
  } else if (near > 0.4999f) {
#pragma unroll
    for (int k = 0; k < V; ++k) u[k] = __float_as_uint(__fdiv_rn(x[k], sf) + magic);
  }
  uint8_t* dst = blk + scale_bytes + (size_t)group * GB + (size_t)slot * (32 * BITS / 8) + ch * BITS / 8;
  if constexpr (BITS == 8) {
    uint32_t w[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k)
      w[k] = __byte_perm(__byte_perm(u[4 * k], u[4 * k + 1], 0x0040), __byte_perm(u[4 * k + 2], u[4 * k + 3], 0x0040), 0x5410);
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) w |= (u[k] & 15u) << (4 * k);
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

// Channels c V .. of a row's two halves: norm weights of the lane, fp32.
template <int V>
__device__ __forceinline__ void load_w(const float* w, int half, int c, float* wl, float* wh) {
#pragma unroll
  for (int k = 0; k < V; k += 4) {
    const float4 a = *reinterpret_cast<const float4*>(w + c * V + k), b = *reinterpret_cast<const float4*>(w + half + c * V + k);
    wl[k] = a.x; wl[k + 1] = a.y; wl[k + 2] = a.z; wl[k + 3] = a.w;
    wh[k] = b.x; wh[k + 1] = b.y; wh[k + 2] = b.z; wh[k + 3] = b.w;
  }
}

// A CTA takes a token and up to blockDim / 32 * per of its row groups (32 / LPR heads each, LPR lanes to a row; first the
// queries' groups, then the keys', then the values'); its warps take them in turn, the next group's rows loaded before this
// one's are worked on.  The token's cos / sin are made once per CTA; a lane's channels are the same in every head, so it
// keeps its factors in registers.  Angles: the fraction of the turn in 64 bits, then an fp32 sincos; in 64 bits
// throughout for keys that are quantised next.  Measured: 4096 tokens of 32 + 32 heads in 28.6 us (4.7 TB/s; waits for loads, with
// 21 warps an SM, by registers; issue in 43 % of the cycles);
// 8193 tokens of 32 + 8 heads into 4 bits in 56 us (issue: 4,170 instructions a token).
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kKvThreads, 3) k_qkv(KvArgs a, int groups, int per) {
  constexpr int V = Vec<T>::N, HALF = D / 2, LPR = HALF / V, RPW = 32 / LPR;
  __shared__ double2 cs_d[BITS ? HALF : 1];
  __shared__ __align__(16) float cs_c[HALF], cs_s[HALF];
  const ServeView& v = a.v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x, nw = blockDim.x >> 5, b0 = blockIdx.y * nw * per, b1 = min(groups, b0 + nw * per);
  const int nq = a.q ? (v.H + RPW - 1) / RPW : 0, nk = a.k ? (v.Hkv + RPW - 1) / RPW : 0;
  const int c = lane % LPR, rr = lane / LPR;
  tc::grid_wait_prev();
  // the rows of this warp's next group, asked for ahead
  uint4 rl, rh;
  auto fetch = [&](int g) {
    const int kind = g < nq ? 0 : g < nq + nk ? 1 : 2;
    const int h = (g - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * RPW + rr;
    const T* s = kind == 0 ? (const T*)a.q + (size_t)i * a.q_ld
                           : kind == 1 ? (const T*)a.k + (size_t)i * a.k_ld : (const T*)a.vv + (size_t)i * a.v_ld;
    const uint4* p = reinterpret_cast<const uint4*>(s + (size_t)h * D + c * V);
    const bool live = h < (kind == 0 ? v.H : v.Hkv);
    rl = live ? p[0] : make_uint4(0, 0, 0, 0);
    rh = live ? p[HALF * sizeof(T) / 16] : make_uint4(0, 0, 0, 0);
  };
  int g = b0 + warp;
  if (g < b1) fetch(g);
  int slot = 0;
  uint8_t* page = a.pool ? slot_page(a, i, &slot, threadIdx.x == 0 && b0 == 0) : nullptr;
  if (a.rotate && b0 < nq + nk) {
    const double pos = (double)a.positions[i];
    for (int e = threadIdx.x; e < 2 * HALF; e += blockDim.x) {
      const int p = e % HALF;
      if (e < HALF) {
        const double t = pos * a.turn[p];
        sincospif((float)(2.0 * (t - rint(t))), &cs_s[p], &cs_c[p]);
      } else if (BITS && b1 > nq) {
        double sn, cs;
        angle(pos * a.turn[p], &sn, &cs);
        cs_d[p % V * LPR + p / V] = make_double2(cs, sn);   // (lanes read neighbours: no bank conflicts)
      }
    }
    __syncthreads();
  }
  // this warp's groups of one kind: rows of `heads` heads
  auto run = [&](auto kind_c, int first, int count, int heads, const float* w, T* out) {
    constexpr int KIND = decltype(kind_c)::value;
    constexpr bool WIDE = KIND == 1 && BITS != 0;
    const int end = min(b1, first + count);
    if (g >= end) return;
    Factors<V> f;
    float wl[V], wh[V];
    if constexpr (KIND != 2) {
#pragma unroll
      for (int k = 0; k < V; ++k) wl[k] = wh[k] = 1.f;
      if (w) load_w<V>(w, HALF, c, wl, wh);
      if constexpr (!WIDE) {
        float cl[V], sl[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          cl[k] = a.rotate ? cs_c[c * V + k] : 1.f;
          sl[k] = a.rotate ? cs_s[c * V + k] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const f32x2 cc = pk(cl[2 * k], cl[2 * k + 1]), ss = pk(sl[2 * k], sl[2 * k + 1]), ns = pk(-sl[2 * k], -sl[2 * k + 1]);
          const f32x2 a2 = pk(wl[2 * k], wl[2 * k + 1]), b2 = pk(wh[2 * k], wh[2 * k + 1]);
          f.lc[k] = mul2(a2, cc);
          f.hs[k] = mul2(b2, ns);
          f.hc[k] = mul2(b2, cc);
          f.ls[k] = mul2(a2, ss);
        }
      }
    }
    for (; g < end; g += nw) {
      const int h = (g - first) * RPW + rr;
      const bool live = h < heads;
      float lo[V], hi[V];
      Vec<T>::load(reinterpret_cast<const T*>(&rl), lo);
      Vec<T>::load(reinterpret_cast<const T*>(&rh), hi);
      if (g + nw < b1) fetch(g + nw);
      if constexpr (WIDE) {
        norm_rotate64<V, LPR, sizeof(T) == 2>(lo, hi, wl, wh, w != nullptr, (double)v.norm_eps, D, cs_d + c, a.rotate);
      } else if constexpr (KIND != 2) {
        const float inv = w ? inv_rms<V, LPR>(lo, hi, v.norm_eps, 1.f / D) : 1.f;
        rotate_row<V>(lo, hi, f, inv);
      }
      if (KIND == 0 || a.pool == nullptr) {
        if (live) {
          T* o = out + (size_t)h * D + c * V;
          Vec<T>::store(o, lo);
          Vec<T>::store(o + HALF, hi);
        }
        continue;
      }
      // block of KV head h's keys, or of all values, as the page lays them out
      if constexpr (BITS != 0) {
        constexpr int KB = D / 32 * (32 + 64 * BITS);
        uint8_t* blk = page ? page + (size_t)(KIND == 2 ? v.Hkv : h) * KB : nullptr;
        const int sb = KIND == 2 ? v.Hkv * D : D;   // bytes of the block's scales: one per 32 channels and slot, 2 bytes
        const int gr = KIND == 2 ? h * (D / 32) : 0, ch = c * V;
        quant_store<BITS, V>(lo, blk, sb, gr + ch / 32, ch % 32, slot, live && page, v.status);
        quant_store<BITS, V>(hi, blk, sb, gr + (HALF + ch) / 32, (HALF + ch) % 32, slot, live && page, v.status);
      } else if (live && page) {
        const size_t row = KIND == 2 ? ((size_t)v.Hkv * kPage + (size_t)slot * v.Hkv + h) * D
                                     : ((size_t)h * kPage + slot) * D;
        if (v.es == 4) {
          float* d = reinterpret_cast<float*>(page) + row + c * V;
#pragma unroll
          for (int k = 0; k < V; k += 4) {
            Vec<float>::store(d + k, lo + k);
            Vec<float>::store(d + HALF + k, hi + k);
          }
        } else {
          __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(page) + row + c * V;
          if constexpr (V == 8) {
            Vec<__nv_bfloat16>::store(d, lo);
            Vec<__nv_bfloat16>::store(d + HALF, hi);
          } else {
#pragma unroll
            for (int k = 0; k < V; k += 2) {
              *reinterpret_cast<__nv_bfloat162*>(d + k) = __floats2bfloat162_rn(lo[k], lo[k + 1]);
              *reinterpret_cast<__nv_bfloat162*>(d + HALF + k) = __floats2bfloat162_rn(hi[k], hi[k + 1]);
            }
          }
        }
      }
    }
  };
  if (a.q)
    run(std::integral_constant<int, 0>{}, 0, nq, v.H, v.q_norm, (T*)a.q_out + (size_t)i * a.q_out_ld);
  if (a.k)
    run(std::integral_constant<int, 1>{}, nq, nk, v.Hkv, v.k_norm, a.pool ? nullptr : (T*)a.k_out + (size_t)i * a.k_out_ld);
  if (a.vv)
    run(std::integral_constant<int, 2>{}, nq + nk, groups - nq - nk, v.Hkv, nullptr, nullptr);
}

// Any even head_dim up to 256, unquantised pages: one warp per row, a lane per pair.
template <typename T>
__global__ void __launch_bounds__(kKvThreads) k_qkv_any(KvArgs a) {
  const ServeView& v = a.v;
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
  constexpr int RPW = 32 / (D / 2 / Vec<T>::N), NW = kKvThreads / 32;
  const int gq = (a.v.H + RPW - 1) / RPW, gk = (a.v.Hkv + RPW - 1) / RPW;
  const int groups = (a.q ? gq : 0) + (a.k ? gk : 0) + (a.vv ? gk : 0);
  // Many tokens: one CTA for a whole token, four warps (they share the angles and keep their factors over several groups).
  // Few: a row group per warp, the token over several CTAs, for latency.  Few / many, us: norm and rotation of 32 + 8 heads, bf16,
  // 192 tokens 3.0 / 3.5, 256 3.9 / 3.5, 384 4.5 / 3.7, 768 7.6 / 4.8; 16 + 16 heads 256 2.9 / 3.3, 512 4.8 / 3.9; fp32 192 4.0 / 3.9, 384
  // 5.6 / 4.3; append of 32 heads over 8 bits 256 9.6 / 10.6, 384 12.6 / 12.1.  The sides meet at 190 to 410 tokens.
  const bool many = a.n > 2 * num_sms();
  const int nw = std::min(many ? 4 : NW, groups), per = many ? (groups + nw - 1) / nw : 1;
  return launch_k(k_qkv<T, D, BITS>, dim3((unsigned)a.n, (unsigned)((groups + nw * per - 1) / (nw * per))), 32 * nw, 0, s, true,
                  a, groups, per);
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
// Rows [n][latent_total] of cached tokens in TO, uncompressed layers: a warp per (token, part of the row), a lane 8
// channels at a time (8 codes are 8 or 4 bytes, 8 values 16 or 32), so that the warp's stores are one run.  The 16 warps
// of a CTA take consecutive tokens of the same part: tokens of one page then share the 32-byte sectors of its
// codes and scales in L1 (a slot's codes are runs of 16 or 32 bytes, its scales 2).  CPH = chunks of a head (d / 8; 0: any).
// Measured: 32768 tokens of 8 KV heads from 4 bits in 33 us (5.2 TB/s with the rows written; bytes and the integer pipe).
constexpr int kReadWarps = 16;
constexpr int kReadUnroll = 4;

template <typename TO, int BITS, int CPH>   // BITS 0: stored in the layer dtype TO
__global__ void __launch_bounds__(32 * kReadWarps) k_read8(KvArgs a, int chunks_per_warp, TO* __restrict__ out) {
  const ServeView& v = a.v;
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  if (i >= a.n) return;
  const int cph = CPH ? CPH : v.d / 8, d = CPH ? CPH * 8 : v.d;
  tc::grid_wait_prev();
  const int keys = v.Hkv * cph, chunks = 2 * keys;
  const int e0 = blockIdx.y * chunks_per_warp, e1 = min(chunks, e0 + chunks_per_warp);
  int slot = 0;
  const uint8_t* page = slot_page(a, (int)i, &slot, lane == 0 && e0 == 0);
  TO* row = out + (size_t)i * (chunks * 8);
  constexpr int GB = kPage * 32 * (BITS ? BITS : 8) / 8;            // bytes of a group's codes
  const int kb = BITS ? d / 32 * (32 + GB) : d * kPage * (int)sizeof(TO);   // bytes of a head's key block
  // chunks eb .. of one side (keys, or values): chunk e's codes at c + steps * cstep, its scale at s + steps * sstep
  auto run = [&](int eb, int end, const uint8_t* c, int cstep, const uint8_t* s, int sstep) {
    // kReadUnroll chunks' bytes are asked for before the first is used
    for (; eb < end; eb += 32 * kReadUnroll) {
      uint4 raw[kReadUnroll][BITS == 0 && sizeof(TO) == 4 ? 2 : 1];
      __half sc[kReadUnroll];
#pragma unroll
      for (int x = 0; x < kReadUnroll; ++x) {
        raw[x][0] = make_uint4(0, 0, 0, 0);
        if constexpr (BITS == 0 && sizeof(TO) == 4) raw[x][1] = raw[x][0];
        sc[x] = __float2half_rn(0.f);
        if (eb + 32 * x < end && page) {
          if constexpr (BITS == 0) {
            raw[x][0] = reinterpret_cast<const uint4*>(c)[0];
            if constexpr (sizeof(TO) == 4) raw[x][1] = reinterpret_cast<const uint4*>(c)[1];
          } else {
            sc[x] = *reinterpret_cast<const __half*>(s);
            if constexpr (BITS == 8) {
              const uint2 u = *reinterpret_cast<const uint2*>(c);
              raw[x][0].x = u.x;
              raw[x][0].y = u.y;
            } else {
              raw[x][0].x = *reinterpret_cast<const uint32_t*>(c);
            }
          }
        }
        c += cstep;
        s += sstep;
      }
#pragma unroll
      for (int x = 0; x < kReadUnroll; ++x) {
        if (eb + 32 * x >= end) break;
        TO* o = row + (eb + 32 * x) * 8;
        if constexpr (BITS == 0) {
          reinterpret_cast<uint4*>(o)[0] = raw[x][0];
          if constexpr (sizeof(TO) == 4) reinterpret_cast<uint4*>(o)[1] = raw[x][1];
        } else {
          float f[8];
          const float sf = __half2float(sc[x]);
          const f32x2 s2 = pk(sf, sf);
          if constexpr (BITS == 8) {
            // a code in the low byte of 2^23 is the number 2^23 + u (an integer conversion has a sixteenth of the rate)
            const f32x2 off = pk(-8388736.f, -8388736.f);
            auto code = [&](int k) {
              return __uint_as_float(__byte_perm(k < 4 ? raw[x][0].x : raw[x][0].y, 0x4B000000u, 0x7440 + k % 4));
            };
#pragma unroll
            for (int k = 0; k < 8; k += 2) upk(mul2(add2(pk(code(k), code(k + 1)), off), s2), f + k);
          } else {
            // codes k, k + 4 under the exponent of 1024 (fp16), exact integers after one subtraction
            const uint32_t w = raw[x][0].x, w8 = w >> 8;
            const __half2 off = __floats2half2_rn(-1032.f, -1032.f), o16 = __floats2half2_rn(-72.f, -72.f),
                          s16 = __floats2half2_rn(0.0625f, 0.0625f);
            auto h = [](uint32_t y) { return *reinterpret_cast<const __half2*>(&y); };
            const float2 a0 = __half22float2(__hadd2(h((w & 0x000F000Fu) | 0x64006400u), off));
            const float2 a1 = __half22float2(__hfma2(h((w & 0x00F000F0u) | 0x64006400u), s16, o16));
            const float2 a2 = __half22float2(__hadd2(h((w8 & 0x000F000Fu) | 0x64006400u), off));
            const float2 a3 = __half22float2(__hfma2(h((w8 & 0x00F000F0u) | 0x64006400u), s16, o16));
            upk(mul2(pk(a0.x, a1.x), s2), f);
            upk(mul2(pk(a2.x, a3.x), s2), f + 2);
            upk(mul2(pk(a0.y, a1.y), s2), f + 4);
            upk(mul2(pk(a2.y, a3.y), s2), f + 6);
          }
#pragma unroll
          for (int k = 0; k < 8; k += Vec<TO>::N) Vec<TO>::store(o + k, f + k);
        }
      }
    }
  };
  // 32 chunks on: for keys 32 / cph heads, for values 8 groups
  if (e0 < keys) {
    const int e = e0 + lane;
    if constexpr (CPH != 0) {   // (8, 16 or 32 chunks: they divide 32)
      const int h = e / CPH, j = e % CPH;
      const uint8_t* blk = page + (size_t)h * kb;
      if constexpr (BITS != 0)
        run(e, min(e1, keys), blk + d + (j >> 2) * GB + slot * (4 * BITS) + (j & 3) * BITS, 32 / CPH * kb,
            blk + (j >> 2) * 32 + slot * 2, 32 / CPH * kb);
      else
        run(e, min(e1, keys), blk + (slot * d + j * 8) * sizeof(TO), 32 / CPH * kb, nullptr, 0);
    } else {
      // rows of any number of chunks: one step at a time
      for (int x = e; x < min(e1, keys); x += 32)
        run(x, min(x + 1, keys), page + (size_t)(x / cph) * kb + (size_t)slot * d * sizeof(TO) + (x % cph) * 8 * sizeof(TO), 0,
            nullptr, 0);
    }
  }
  if (e1 > keys) {
    const int e = max(e0, keys) + lane;
    const int x = e - keys;
    const uint8_t* blk = page + (size_t)v.Hkv * kb;
    if constexpr (BITS != 0)
      run(e, e1, blk + v.Hkv * d + (x >> 2) * GB + slot * (4 * BITS) + (x & 3) * BITS, 8 * GB, blk + (x >> 2) * 32 + slot * 2, 256);
    else
      run(e, e1, blk + ((size_t)slot * v.Hkv * d + x * 8) * sizeof(TO), 256 * (int)sizeof(TO), nullptr, 0);
  }
}

template <typename TO>
__global__ void __launch_bounds__(256) k_read_any(KvArgs a, TO* __restrict__ out) {
  const ServeView& v = a.v;
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

// A sequence's path, checked (flagged when it is not increasing node numbers of the sequence; the sequence is then left
// as it was).  By the whole block; every thread gets the answer.
__device__ __forceinline__ bool path_ok(const AcceptArgs& a, const TreeSeq& q, int n_acc, bool flag) {
  bool ok = n_acc >= 0 && n_acc <= q.cnt;
  for (int k = threadIdx.x; ok && k < n_acc; k += blockDim.x) {
    const int x = a.acc[q.off + k], prev = k ? a.acc[q.off + k - 1] : -1;
    if (x <= prev || x >= q.cnt) ok = false;
  }
  ok = __syncthreads_and(ok);
  if (!ok && flag && threadIdx.x == 0) atomicOr(a.v.status, kBadPos);
  return ok;
}

// Uncompressed layers: every group of a slot is one run of 16-byte pieces (kv_bits: 32 channels and their scale; else a
// head's keys, and all heads' values).  A CTA takes one sequence and kAccPieces pieces of every slot, kAccNodes nodes at
// a time: all of them into registers, then all of them out, so nothing waits for a neighbour's node.  (A later batch
// reads slots acc[k] >= k, which earlier batches have not written.)  Measured: 64 sequences of 64 nodes, 8 bits, 32 heads in 12 us
// (latency: one wave of loads and one of stores per batch; 39 MB at most).
constexpr int kAccNodes = 32;
constexpr int kAccPieces = 32;      // 16-byte pieces of a slot per CTA
constexpr int kAccThreads = 256;

template <int BITS>
__global__ void __launch_bounds__(kAccThreads) k_accept_plain(AcceptArgs a, int pieces) {
  constexpr int PER = BITS ? BITS / 4 : 1;                                     // pieces of one group (kv_bits)
  constexpr int IT = kAccNodes * kAccPieces / kAccThreads, STEP = kAccPieces / IT;
  __shared__ long long src[kAccNodes], dst[kAccNodes];   // byte offset of the page (-1: nothing to move), per node
  __shared__ int ss[kAccNodes], ds[kAccNodes];           // slots; ss -1: cleared
  const LayerView& v = a.v;
  const int b = blockIdx.y;
  const bool first = blockIdx.x == 0;
  tc::grid_wait_prev();
  const TreeSeq q = tree_seq(a.hist, a.node_off, b, a.n_nodes, a.max_nodes, a.max_pages * kPage, v.status,
                             first && threadIdx.x == 0);
  if (q.cnt <= 0) return;
  const int n_acc = a.n_acc[b];
  if (!path_ok(a, q, n_acc, first)) return;
  for (int k0 = 0; k0 < q.cnt; k0 += kAccNodes) {
    if (threadIdx.x < kAccNodes) {
      const int k = k0 + threadIdx.x;
      long long so = -1, dn = -1;
      int s = -1, t = 0;
      if (k < q.cnt) {
        const bool kept = k < n_acc;
        const int from = q.hist + (kept ? a.acc[q.off + k] : k), to = q.hist + k;
        if (!kept || from != to) {
          const int32_t* pt = a.pt + (size_t)b * a.max_pages;
          const int sp = pt[from / kPage], dp = pt[to / kPage];
          if (sp < 0 || sp >= a.n_pages || dp < 0 || dp >= a.n_pages) {
            if (first) atomicOr(v.status, kBadPage);
          } else {
            so = sp * v.page_bytes;
            dn = dp * v.page_bytes;
            s = kept ? from % kPage : -1;
            t = to % kPage;
          }
        }
      }
      src[threadIdx.x] = so;
      dst[threadIdx.x] = dn;
      ss[threadIdx.x] = s;
      ds[threadIdx.x] = t;
    }
    __syncthreads();
    // a thread keeps its node and takes every STEP-th piece
    const int k = threadIdx.x / PER % kAccNodes;
    const int pc0 = blockIdx.x * kAccPieces + threadIdx.x / (PER * kAccNodes) * PER + threadIdx.x % PER;
    const bool move = dst[k] >= 0, keep = move && ss[k] >= 0;
    const uint8_t* sp = a.pool + (keep ? src[k] : 0);
    uint8_t* dp = a.pool + (move ? dst[k] : 0);
    const int st = ss[k], dt = ds[k];
    uint4 x[IT];
    uint16_t sc[IT];
    int at[IT], scale[IT];   // the piece's offset in the page for slot 0, and its group's scale's (-1: none)
    const int row = v.d * v.es, keys = v.Hkv * row;
    constexpr int GB = kPage * 4 * BITS;
    const int gd = v.d / 32, kb = gd * (32 + GB), hk = v.Hkv * gd;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int pc = pc0 + it * STEP;
      x[it] = make_uint4(0, 0, 0, 0);
      sc[it] = 0;
      int step = 4 * BITS;
      if constexpr (BITS != 0) {
        const int g = pc / PER;   // group of the token: keys by head, then values
        const bool val = g >= hk;
        const int gl = val ? g - hk : g % gd, blk = (val ? v.Hkv : g / gd) * kb;
        scale[it] = pc % PER == 0 ? blk + gl * 32 : -1;
        at[it] = blk + (val ? v.Hkv * v.d : v.d) + gl * GB + (pc % PER) * 16;
      } else {
        const int c = pc * 16;    // byte of the slot: the heads' key rows, then the value row
        const bool val = c >= keys;
        scale[it] = -1;
        step = val ? keys : row;
        at[it] = val ? kPage * keys + (c - keys) : c / row * kPage * row + c % row;
      }
      if (keep && pc < pieces) {
        x[it] = *reinterpret_cast<const uint4*>(sp + at[it] + st * step);
        if (scale[it] >= 0) sc[it] = reinterpret_cast<const uint16_t*>(sp + scale[it])[st];
      }
      at[it] += dt * step;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (!move || pc0 + it * STEP >= pieces) continue;
      *reinterpret_cast<uint4*>(dp + at[it]) = x[it];
      if (scale[it] >= 0) reinterpret_cast<uint16_t*>(dp + scale[it])[dt] = sc[it];
    }
    __syncthreads();
  }
}

// Any layer: one warp per (sequence, group).
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

namespace {

template <typename TO, int BITS>
cudaError_t read_plain(const KvArgs& a, void* out, cudaStream_t s) {
  const int chunks = 2 * a.v.Hkv * (a.v.d / 8);
  // few tokens: a row is spread over several warps, down to one round of a warp's unrolled loads
  const long long rows = ((long long)a.n + kReadWarps - 1) / kReadWarps;
  const int least = 32 * kReadUnroll;
  const int parts = (int)std::max(1LL, std::min((long long)(chunks + least - 1) / least, 8LL * num_sms() / rows));
  const int per = ((chunks + parts - 1) / parts + 31) / 32 * 32;
  const dim3 grid((unsigned)rows, (unsigned)((chunks + per - 1) / per));
  auto* kernel = a.v.d == 128 ? k_read8<TO, BITS, 16>
                 : a.v.d == 64 ? k_read8<TO, BITS, 8> : a.v.d == 256 ? k_read8<TO, BITS, 32> : k_read8<TO, 0, 0>;
  return launch_k(kernel, grid, 32 * kReadWarps, 0, s, true, a, per, (TO*)out);
}

}  // namespace

cudaError_t launch_cache_read(const KvArgs& a, void* out, cudaStream_t s) {
  const ServeView& v = a.v;
  const bool f32 = v.dtype == STARKV_F32;
  // eight channels a lane: rows of whole 8-channel chunks
  if (v.plain && v.d % 8 == 0) {
    if (f32)
      return v.kv_bits == 8 ? read_plain<float, 8>(a, out, s) : v.kv_bits == 4 ? read_plain<float, 4>(a, out, s)
                                                                        : read_plain<float, 0>(a, out, s);
    return v.kv_bits == 8 ? read_plain<__nv_bfloat16, 8>(a, out, s) : v.kv_bits == 4 ? read_plain<__nv_bfloat16, 4>(a, out, s)
                                                                                     : read_plain<__nv_bfloat16, 0>(a, out, s);
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
  const ServeView& v = L->view;
  const int slot_bytes = v.kv_bits ? 2 * v.Hkv * v.d * v.kv_bits / 8 : 2 * v.Hkv * v.d * v.es;
  if (v.plain && (v.d * v.es) % 16 == 0) {
    const int pieces = slot_bytes / 16;
    const dim3 grid((pieces + kAccPieces - 1) / kAccPieces, batch);
    if (batch <= 65535) {
      return launch_k(v.kv_bits == 8 ? k_accept_plain<8> : v.kv_bits == 4 ? k_accept_plain<4> : k_accept_plain<0>, grid,
                      kAccThreads, 0, s, true, a, pieces);
    }
  }
  const long long warps = (long long)batch * a.n_grp;
  k_accept<<<(unsigned)((warps * 32 + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace starkv
