// Attention of drafted tokens (nodes of a tree, a chain, or one token) over an
// uncompressed layer's cache: bf16 K and V, or their 8 / 4-bit codes.
//
// Every KV head's R = nodes * group rows of a sequence share its K and V, so a
// page (16 tokens) is read once for up to 16 rows, the M side of the warp-level
// matrix instruction m16n8k16.  The codes go from shared memory into MMA
// operands without being scaled first:
//   scores   a code byte u under the fp16 exponent of 1024 is the number 1024 + u (one PRMT per two codes; 4-bit codes
//            in a word's high nibbles come out as 1024 + 16 u, their q is 1/16).  A group's accumulator starts at
//            -sum_c q_c (1024 + 2^(b-1)), so it ends at sum_c q_c (u - 2^(b-1)); then S += scale[token][group] * it.
//            |offset| is below 40 times the sum, whose fp32 rounding stays below 2^-17 of q's length times a code.
//   values   the scale belongs to (token, group): the probabilities are multiplied by it (fp16, per group of 32
//            channels) and the codes enter as exact integers (the offset taken off by one packed subtraction; it cannot
//            be folded into the accumulator here, whose sum over thousands of tokens would cancel).
// Channels within a group and tokens within a page may enter a contraction in any order, so each lane reads runs of
// bytes: eight channels of a token for the scores, four channels of four tokens for the values, the tokens rotated by
// the lane (tok()) so that a warp's reads touch every shared-memory bank once.
//
// Running maximum and sum are per row in registers.  m is the row's maximum less 3 (log2 units) and moves only when a
// score passes m + 7: p = 2^(s - m) <= 2^7, times a scale <= 258 stays inside fp16 (65504), while the largest weight
// seen is at least 8, so that weights down to 2^-11 of it keep full precision even under small scales.
//
// Work split: the units (sequence, KV head, block of 16 rows, page) of the whole call, in this order, are dealt to the
// resident warps in equal runs; a warp writes one partial (m, l, Y) per row block that its run touches, and
// k_tree_combine merges them.  Warps never wait for one another; each keeps its own ring of pages in flight with
// 16-byte asynchronous copies.
#include <float.h>

#include "tc_common.cuh"

namespace starkv {

namespace {

constexpr int kTreeWarps = 4;          // warps per CTA
constexpr int kMinUnits = 2;           // pages of a warp's run, at least (short calls use fewer warps)
constexpr int kTcRows = 128;           // rows of a row block of k_tree_tc
constexpr int kTcTok = 128;            // tokens of its tiles

template <int BITS>
struct PageFmt {
  static constexpr int KB = BITS == 0 ? 4096 : 128 + 64 * 4 * BITS;   // key block of one head: scales, codes
  static constexpr int VS = BITS == 0 ? 0 : 128;                      // one head's value scales
  static constexpr int VB = BITS == 0 ? 4096 : 64 * 4 * BITS;         // one head's value codes
  static constexpr int STAGE = KB + VS + VB;                          // 8192, 4352 or 2304 bytes
  // warps per SM: registers (two sets of query fragments for bf16) and 220 KB of shared memory
  static constexpr int CTAS = BITS == 0 ? 2 : 3;
  static constexpr int NS = BITS == 0 ? 3 : BITS == 8 ? 4 : 6;        // pages of a warp's ring
};

struct TreeWs {
  long long* unit_off;   // [batch + 1] units before a sequence
  long long* item_off;   // [batch + 1] row blocks before a sequence
  void* q;               // [n_nodes][H][128] fp16 in the kernels' channel order; bf16 layers: the high, then the low parts
  float *pm, *pl;        // [partials][rb]
  float* pY;             // [partials][rb][128]
  void* y;               // output tiles
  void* part;            // output product
};

struct TreeMma {
  LayerView v;
  TreeArgs t;
  TreeWs w;
  int workers;           // warps (k_tree_mma) or CTAs (k_tree_tc) that share the units
  int rb;                // rows of a row block: 16, or 128
  int unit;              // tokens of a unit: a page, or a tile of 128
  int min_units;
};

// How a call's units are dealt: worker w takes units [w U / We, (w + 1) U / We).
__device__ __forceinline__ long long workers_used(const TreeMma& a, long long U) {
  return min((long long)a.workers, max(1ll, U / a.min_units));
}

__device__ __forceinline__ TreeSeq seq_of(const TreeArgs& t, int b, uint32_t* status, bool flag) {
  const int cap = t.max_pages * kPage;
  if (t.lens) {   // decode: one query per sequence over lens[b] tokens
    int len = t.lens[b];
    if (len > cap || len < 0) {
      if (flag) atomicOr(status, kBadPos);
      len = len < 0 ? 0 : cap;
    }
    return TreeSeq{len - 1, len > 0 ? 1 : 0, b, 1};
  }
  return tree_seq(t.hist, t.node_off, b, t.n_nodes, t.max_nodes, cap, status, flag);
}

// Largest b with off[b] <= x, for a non-decreasing off[0 .. n] with off[0] <= x < off[n], by the whole warp.
template <typename T>
__device__ __forceinline__ int warp_find(const T* off, int n, long long x, int lane) {
  int lo = 0, len = n;   // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, lane * step < len && (long long)off[i] <= x);
    const int k = 31 - __clz(le);          // lane 0 always holds
    const int end = lo + len;
    lo += k * step;
    len = min(step, end - lo);
  }
  return lo;
}

// ------------------------------------------------------------------ queries and the work list
// Blocks (row, head group): norm, rotation, softmax scale * log2(e) of one query row per warp, rounded to fp16 (to a
// bf16 pair high + low for bf16 caches, whose products then carry 16 bits).  The last block row: prefix sums.
// ORDER (4-bit codes): 0 = channels in order; 1, 2 = every eight in the order 0 4 1 5 2 6 3 7 in which the nibble masks give
// them, with 1/16 for the odd ones (1: k_tree_mma, which meets 16 u there) or without (2: k_tree_tc).
template <int BITS, int ORDER>
__global__ void __launch_bounds__(128) k_tree_prep(TreeMma a) {
  const LayerView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y != 0) return;
    // one warp walks the batch 32 sequences at a time
    if (warp != 0) return;
    long long units = 0, items = 0;
    // a node_off that decreases would let sequences claim the same rows, and more row blocks than there is room for
    bool back = false;
    if (!t.lens)
      for (int b = lane; b < t.batch; b += 32) back = back || t.node_off[b + 1] < t.node_off[b];
    back = __any_sync(0xffffffffu, back);
    if (back && lane == 0) atomicOr(v.status, kBadPos);
    for (int b0 = 0; b0 < t.batch; b0 += 32) {
      const int b = b0 + lane;
      long long nu = 0, ni = 0;
      if (b < t.batch) {
        TreeSeq q = seq_of(t, b, v.status, true);
        if (back) q.cnt = 0;
        ni = (long long)v.Hkv * ((q.cnt * v.group_q + a.rb - 1) / a.rb);
        nu = q.cnt ? ni * ((q.hist + q.cnt + a.unit - 1) / a.unit) : 0;
      }
      long long su = nu, si = ni;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long xu = __shfl_up_sync(0xffffffffu, su, o), xi = __shfl_up_sync(0xffffffffu, si, o);
        if (lane >= o) {
          su += xu;
          si += xi;
        }
      }
      if (b < t.batch) {
        a.w.unit_off[b] = units + su - nu;
        a.w.item_off[b] = items + si - ni;
      }
      units += __shfl_sync(0xffffffffu, su, 31);
      items += __shfl_sync(0xffffffffu, si, 31);
    }
    if (lane == 0) {
      a.w.unit_off[t.batch] = units;
      a.w.item_off[t.batch] = items;
    }
    return;
  }
  const int row = blockIdx.x, h = blockIdx.y * kTreeWarps + warp;
  if (h >= v.H) return;
  // lane: pairs p = 2 lane, 2 lane + 1 (channels p and p + 64)
  const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>((const __nv_bfloat16*)t.q + ((size_t)row * v.H + h) * 128);
  const float2 lo = __bfloat1622float2(q[lane]), hi = __bfloat1622float2(q[32 + lane]);
  float x[2] = {lo.x, lo.y}, y[2] = {hi.x, hi.y};
  if (t.raw) {
    if (v.q_norm) {
      float s = x[0] * x[0] + x[1] * x[1] + y[0] * y[0] + y[1] * y[1];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float inv = 1.f / sqrtf(s / 128.f + v.norm_eps);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[k] *= inv * v.q_norm[2 * lane + k];
        y[k] *= inv * v.q_norm[64 + 2 * lane + k];
      }
    }
    if (v.rope) {
      const int pos = t.q_pos ? t.q_pos[row] : max(min(t.lens[row], t.max_pages * kPage), 0) - 1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int p = 2 * lane + k;
        const double turns = v.turn ? (double)pos * v.turn[p]
                                    : (double)pos * exp2(-(2.0 * p / 128.0) * (double)v.rope_log2_theta) / 6.283185307179586476925286766559;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        const float x2 = x[k] * cs - y[k] * sn;
        y[k] = y[k] * cs + x[k] * sn;
        x[k] = x2;
      }
    }
  }
  if constexpr (BITS == 0) {
    __nv_bfloat16* o = (__nv_bfloat16*)a.w.q + ((size_t)row * v.H + h) * 128;
    const size_t low = (size_t)t.n_nodes * v.H * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = (k < 2 ? x[k] : y[k - 2]) * v.scale_log2;
      const int c = (k < 2 ? 0 : 64) + 2 * lane + (k & 1);
      const __nv_bfloat16 b = __float2bfloat16_rn(f);
      o[c] = b;
      o[low + c] = __float2bfloat16_rn(f - __bfloat162float(b));
    }
  } else {
    __half* o = (__half*)a.w.q + ((size_t)row * v.H + h) * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f = (k < 2 ? x[k] : y[k - 2]) * v.scale_log2;
      int c = (k < 2 ? 0 : 64) + 2 * lane + (k & 1);
      if (ORDER != 0) {
        const int j = c & 7;
        if (ORDER == 1 && (j & 1)) f *= 0.0625f;
        c = (c & ~7) | ((j & 3) * 2 + (j >> 2));
      }
      o[c] = __float2half_rn(f);
    }
  }
}

// ------------------------------------------------------------------ pieces of the main kernel
__device__ __forceinline__ void mma_h(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t b2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 16 bytes global -> shared, or zeros
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Token of a page behind lane column j (0 .. 3), place i (0 .. 3).
__device__ __forceinline__ int tok(int j, int i) { return 4 * j + ((i + j) & 3); }
// bf16 pages: 16-byte chunk c of token t's 256-byte row is kept at chunk c ^ swz(t), so that the reads of both
// contractions touch every bank once (row stride = two rounds of the banks).
__device__ __forceinline__ int swz(int t) { return ((t & 1) << 2) | (t & 2); }

// The four scales of tokens 4 j .. 4 j + 3 (8 bytes at p) in the order tok(j, 0 .. 3).
__device__ __forceinline__ void scales4(const uint8_t* p, uint32_t sel0, uint32_t sel1, float* s) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const uint32_t r0 = __byte_perm(w.x, w.y, sel0), r1 = __byte_perm(w.x, w.y, sel1);
  const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&r0));
  const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&r1));
  s[0] = f0.x;
  s[1] = f0.y;
  s[2] = f1.x;
  s[3] = f1.y;
}

// Copies of one page of KV head g into a stage.
template <int BITS>
__device__ __forceinline__ void issue_page(const TreeMma& a, int page, int g, uint32_t dst, int lane) {
  using F = PageFmt<BITS>;
  const bool live = page >= 0 && page < a.t.n_pages;
  if (!live && lane == 0) atomicOr(a.v.status, kBadPage);
  const uint8_t* base = a.t.pool + (size_t)(live ? page : 0) * a.v.page_bytes;
  const uint8_t* ks = base + (size_t)g * F::KB;
  if constexpr (BITS == 0) {
    const uint8_t* vs = base + (size_t)a.v.Hkv * F::KB + g * 256;
    const size_t ld = (size_t)a.v.Hkv * 256;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = k * 32 + lane, t = e >> 4, c = e & 15;
      const uint32_t o = (uint32_t)(t * 256 + ((c ^ swz(t)) << 4));
      cp16(dst + o, ks + e * 16, live);
      cp16(dst + F::KB + o, vs + (size_t)t * ld + c * 16, live);
    }
  } else {
    const uint8_t* vsc = base + (size_t)a.v.Hkv * F::KB + (size_t)g * F::VS;
    const uint8_t* vcd = base + (size_t)a.v.Hkv * (F::KB + F::VS) + (size_t)g * F::VB;
    constexpr int KC = F::KB / 16, VC = F::VB / 16;
#pragma unroll
    for (int k = 0; k < KC / 32; ++k) cp16(dst + (k * 32 + lane) * 16, ks + (k * 32 + lane) * 16, live);
    // the key block's last 8 chunks, and the value scales
    if (lane < 8)
      cp16(dst + (KC - 8 + lane) * 16, ks + (KC - 8 + lane) * 16, live);
    else if (lane < 16)
      cp16(dst + F::KB + (lane - 8) * 16, vsc + (lane - 8) * 16, live);
#pragma unroll
    for (int k = 0; k < VC / 32; ++k)
      cp16(dst + F::KB + F::VS + (k * 32 + lane) * 16, vcd + (k * 32 + lane) * 16, live);
  }
}

template <int BITS>
__global__ void __launch_bounds__(32 * kTreeWarps, PageFmt<BITS>::CTAS) k_tree_mma(TreeMma a) {
  using F = PageFmt<BITS>;
  extern __shared__ __align__(128) uint8_t ring_all[];
  const LayerView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, j = lane & 3;
  uint8_t* ring = ring_all + (size_t)warp * F::NS * F::STAGE;
  const uint32_t ring_s = tc::smem_u32(ring);
  const int GQ = v.group_q;
  const long long U = a.w.unit_off[t.batch];
  const int w = warp * gridDim.x + blockIdx.x;   // neighbouring runs on different SMs
  const long long We = workers_used(a, U);
  if (w >= We) return;
  long long u = (long long)w * U / We;
  const long long u1 = (long long)(w + 1) * U / We;
  // selectors that rotate four fp16 numbers by j places
  uint32_t sel0, sel1;
  {
    const uint32_t c0 = 2 * j, c1 = 2 * ((j + 1) & 3), c2 = 2 * ((j + 2) & 3), c3 = 2 * ((j + 3) & 3);
    sel0 = c0 | (c0 + 1) << 4 | c1 << 8 | (c1 + 1) << 12;
    sel1 = c2 | (c2 + 1) << 4 | c3 << 8 | (c3 + 1) << 12;
  }
  while (u < u1) {
    // ---- the row block of unit u
    const int b = warp_find(a.w.unit_off, t.batch, u, lane);
    const TreeSeq sq = seq_of(t, b, v.status, false);
    const int R = sq.cnt * GQ, nrb = (R + 15) / 16, len = sq.hist + sq.cnt, pages = (len + kPage - 1) / kPage;
    const long long rem = u - a.w.unit_off[b];
    const int blk = (int)(rem / pages), p0 = (int)(rem % pages);
    const int g = blk / nrb, rb = blk % nrb;
    const int p1 = (int)min((long long)pages, p0 + (u1 - u));
    const int32_t* pt = t.pt + (size_t)b * t.max_pages;
    // ---- query fragments: rows r and r + 8 of the block, channels 32 g' + 8 j ..
    uint32_t qa[BITS == 0 ? 16 : 8][4];
    const int row0 = rb * 16 + r, row1 = row0 + 8;
    const int node0 = row0 / GQ, node1 = row1 / GQ;
    {
      const uint4* q0 = reinterpret_cast<const uint4*>((const uint16_t*)a.w.q +
                                                       ((size_t)(sq.off + node0) * v.H + g * GQ + row0 % GQ) * 128);
      const uint4* q1 = reinterpret_cast<const uint4*>((const uint16_t*)a.w.q +
                                                       ((size_t)(sq.off + node1) * v.H + g * GQ + row1 % GQ) * 128);
#pragma unroll
      for (int part = 0; part < (BITS == 0 ? 2 : 1); ++part) {
        const size_t o = (size_t)part * t.n_nodes * v.H * 16;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = row0 < R ? q0[o + 4 * c + j] : make_uint4(0, 0, 0, 0);
          const uint4 y = row1 < R ? q1[o + 4 * c + j] : make_uint4(0, 0, 0, 0);
          uint32_t* f0 = qa[part * 8 + 2 * c];
          uint32_t* f1 = qa[part * 8 + 2 * c + 1];
          f0[0] = x.x; f0[1] = y.x; f0[2] = x.y; f0[3] = y.y;
          f1[0] = x.z; f1[1] = y.z; f1[2] = x.w; f1[3] = y.w;
        }
      }
    }
    // a group's accumulator starts at minus the part of the sum that the codes' offset makes
    float bias0[4], bias1[4];
    if constexpr (BITS != 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qa[2 * c + k][e]));
            // 4-bit: elements 2, 3 of a fragment (high nibbles) meet 1024 + 16 u
            const float z = BITS == 8 ? 1152.f : (e & 2) ? 1152.f : 1032.f;
            ((e & 1) ? s1 : s0) -= (f.x + f.y) * z;
          }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          s0 += __shfl_xor_sync(0xffffffffu, s0, o);
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        }
        bias0[c] = s0;
        bias1[c] = s1;
      }
    }
    float Y[16][4];
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[k][e] = 0.f;
    float m0 = -1e30f, m1 = -1e30f, l0 = 0.f, l1 = 0.f;
    // ---- pages p0 .. p1, NS - 1 ahead
    int ids = p0 + lane < p1 ? pt[p0 + lane] : 0, ids0 = p0;
    int next = p0;
    auto issue = [&]() {
      if (next < p1) {
        if (next - ids0 == 32) {
          ids0 = next;
          ids = ids0 + lane < p1 ? pt[ids0 + lane] : 0;
        }
        const int page = __shfl_sync(0xffffffffu, ids, next - ids0);
        issue_page<BITS>(a, page, g, ring_s + (uint32_t)((next - p0) % F::NS) * F::STAGE, lane);
        ++next;
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < F::NS - 1; ++k) issue();
    for (int p = p0; p < p1; ++p) {
      cp_wait<F::NS - 2>();
      __syncwarp();   // this page's bytes from every lane; every lane is done with the stage that is filled next
      issue();
      const uint8_t* st = ring + (size_t)((p - p0) % F::NS) * F::STAGE;
      // ---- scores of 16 tokens: S[tl] columns 2 j, 2 j + 1 = tokens tok(j, 2 tl), tok(j, 2 tl + 1)
      float S[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) S[0][e] = S[1][e] = 0.f;
      const int kn = r >> 1, ki = r & 1;   // operand column r of tile tl is token tok(r / 2, r % 2 + 2 tl)
      if constexpr (BITS == 0) {
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
          const int kt = tok(kn, ki + 2 * tl);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(st + kt * 256 + (((4 * c + j) ^ swz(kt)) << 4));
            mma_b(S[tl], qa[2 * c], x.x, x.y);
            mma_b(S[tl], qa[2 * c + 1], x.z, x.w);
            mma_b(S[tl], qa[8 + 2 * c], x.x, x.y);
            mma_b(S[tl], qa[8 + 2 * c + 1], x.z, x.w);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float sc[4];
          scales4(st + c * 32 + j * 8, sel0, sel1, sc);
#pragma unroll
          for (int tl = 0; tl < 2; ++tl) {
            const int kt = tok(kn, ki + 2 * tl);
            float acc[4] = {bias0[c], bias0[c], bias1[c], bias1[c]};
            if constexpr (BITS == 8) {
              const uint2 x = *reinterpret_cast<const uint2*>(st + 128 + c * 512 + kt * 32 + j * 8);
              mma_h(acc, qa[2 * c], __byte_perm(x.x, 0x64646464u, 0x4140), __byte_perm(x.x, 0x64646464u, 0x4342));
              mma_h(acc, qa[2 * c + 1], __byte_perm(x.y, 0x64646464u, 0x4140), __byte_perm(x.y, 0x64646464u, 0x4342));
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(st + 128 + c * 256 + kt * 16 + j * 4);
              const uint32_t x8 = x >> 8;
              mma_h(acc, qa[2 * c], (x & 0x000F000Fu) | 0x64006400u, (x & 0x00F000F0u) | 0x64006400u);
              mma_h(acc, qa[2 * c + 1], (x8 & 0x000F000Fu) | 0x64006400u, (x8 & 0x00F000F0u) | 0x64006400u);
            }
            S[tl][0] += sc[2 * tl] * acc[0];
            S[tl][1] += sc[2 * tl + 1] * acc[1];
            S[tl][2] += sc[2 * tl] * acc[2];
            S[tl][3] += sc[2 * tl + 1] * acc[3];
          }
        }
      }
      const bool tail = p * kPage + kPage > sq.hist;   // the page holds drafted nodes or unused slots
      if (tail) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = p * kPage + tok(j, i) - sq.hist;   // node of this slot (negative: history)
          bool s0 = x < 0, s1 = s0;
          if (x >= 0 && x < sq.cnt) {
            if (row0 < R) s0 = tree_sees(t.mask, t.mask_words, sq.off + node0, node0, x);
            if (row1 < R) s1 = tree_sees(t.mask, t.mask_words, sq.off + node1, node1, x);
          }
          if (!s0) S[i >> 1][i & 1] = -INFINITY;
          if (!s1) S[i >> 1][2 + (i & 1)] = -INFINITY;
        }
      }
      // ---- running maximum
      const float x0 = fmaxf(fmaxf(S[0][0], S[0][1]), fmaxf(S[1][0], S[1][1]));
      const float x1 = fmaxf(fmaxf(S[0][2], S[0][3]), fmaxf(S[1][2], S[1][3]));
      if (__any_sync(0xffffffffu, x0 > m0 + 7.f || x1 > m1 + 7.f)) {
        float y0 = x0, y1 = x1;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, o));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, o));
        }
        const float n0 = fmaxf(m0, y0 - 3.f), n1 = fmaxf(m1, y1 - 3.f);
        const float f0 = ex2(m0 - n0), f1 = ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          Y[k][0] *= f0;
          Y[k][1] *= f0;
          Y[k][2] *= f1;
          Y[k][3] *= f1;
        }
      }
      float P[4][2];   // [token place i][row]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        P[i][0] = ex2(S[i >> 1][i & 1] - m0);
        P[i][1] = ex2(S[i >> 1][2 + (i & 1)] - m1);
      }
      // ---- values
      if constexpr (BITS == 0) {
        const uint8_t* sv = st + F::KB;
        uint32_t pa[4] = {b2(P[0][0], P[1][0]), b2(P[0][1], P[1][1]), b2(P[2][0], P[3][0]), b2(P[2][1], P[3][1])};
        // the sum is over the rounded weights, so that they add up to one
        auto lo16 = [](uint32_t x) { return __uint_as_float(x << 16); };
        auto hi16 = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
        l0 += (lo16(pa[0]) + hi16(pa[0])) + (lo16(pa[2]) + hi16(pa[2]));
        l1 += (lo16(pa[1]) + hi16(pa[1])) + (lo16(pa[3]) + hi16(pa[3]));
        unsigned bad = 0;   // place i of this lane's tokens holds an infinity or a NaN
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint2 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int vt = tok(j, i);
            x[i] = *reinterpret_cast<const uint2*>(sv + vt * 256 + (((4 * c + (r >> 1)) ^ swz(vt)) << 4) + (r & 1) * 8);
            if (tail) {
              // a slot that some rows do not see must not reach them through 0 * NaN: it enters as zero, and the rows
              // that do see it become NaN below
              auto odd = [](uint32_t y) { return (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u; };
              if (odd(x[i].x) || odd(x[i].y)) {
                bad |= 1u << i;
                x[i] = make_uint2(0u, 0u);
              }
            }
          }
          mma_b(Y[4 * c + 0], pa, __byte_perm(x[0].x, x[1].x, 0x5410), __byte_perm(x[2].x, x[3].x, 0x5410));
          mma_b(Y[4 * c + 1], pa, __byte_perm(x[0].x, x[1].x, 0x7632), __byte_perm(x[2].x, x[3].x, 0x7632));
          mma_b(Y[4 * c + 2], pa, __byte_perm(x[0].y, x[1].y, 0x5410), __byte_perm(x[2].y, x[3].y, 0x5410));
          mma_b(Y[4 * c + 3], pa, __byte_perm(x[0].y, x[1].y, 0x7632), __byte_perm(x[2].y, x[3].y, 0x7632));
        }
        if (tail) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (bad >> i & 1) {
              if (S[i >> 1][i & 1] != -INFINITY) l0 = NAN;
              if (S[i >> 1][2 + (i & 1)] != -INFINITY) l1 = NAN;
            }
        }
      } else {
        l0 += (P[0][0] + P[1][0]) + (P[2][0] + P[3][0]);
        l1 += (P[0][1] + P[1][1]) + (P[2][1] + P[3][1]);
        const uint8_t* sv = st + F::KB;
        const uint8_t* cv = sv + F::VS;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float sc[4];
          scales4(sv + c * 32 + j * 8, sel0, sel1, sc);
          if (tail) {
            // unused slots may hold any bytes: no scale that is not a number meets a weight of zero
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (p * kPage + tok(j, i) >= len) sc[i] = 0.f;
          }
          const uint32_t pa[4] = {h2(P[0][0] * sc[0], P[1][0] * sc[1]), h2(P[0][1] * sc[0], P[1][1] * sc[1]),
                                  h2(P[2][0] * sc[2], P[3][0] * sc[3]), h2(P[2][1] * sc[2], P[3][1] * sc[3])};
          if constexpr (BITS == 8) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = *reinterpret_cast<const uint32_t*>(cv + c * 512 + tok(j, i) * 32 + r * 4);
            const uint32_t a01 = __byte_perm(x[0], x[1], 0x5140), b01 = __byte_perm(x[0], x[1], 0x7362);
            const uint32_t a23 = __byte_perm(x[2], x[3], 0x5140), b23 = __byte_perm(x[2], x[3], 0x7362);
            constexpr uint32_t off = 0x64806480u, ex = 0x64646464u;   // 1152, 1152
            mma_h(Y[4 * c + 0], pa, hsub2(__byte_perm(a01, ex, 0x4140), off), hsub2(__byte_perm(a23, ex, 0x4140), off));
            mma_h(Y[4 * c + 1], pa, hsub2(__byte_perm(a01, ex, 0x4342), off), hsub2(__byte_perm(a23, ex, 0x4342), off));
            mma_h(Y[4 * c + 2], pa, hsub2(__byte_perm(b01, ex, 0x4140), off), hsub2(__byte_perm(b23, ex, 0x4140), off));
            mma_h(Y[4 * c + 3], pa, hsub2(__byte_perm(b01, ex, 0x4342), off), hsub2(__byte_perm(b23, ex, 0x4342), off));
          } else {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = *reinterpret_cast<const uint16_t*>(cv + c * 256 + tok(j, i) * 16 + r * 2);
            const uint32_t w01 = __byte_perm(x[0], x[1], 0x5410), w23 = __byte_perm(x[2], x[3], 0x5410);
            constexpr uint32_t lm = 0x000F000Fu, hm = 0x00F000F0u, ex = 0x64006400u;
            constexpr uint32_t off = 0x64086408u;                       // 1032
            constexpr uint32_t s16 = 0x2C002C00u, o16 = 0xD480D480u;    // 1/16, -72
            mma_h(Y[4 * c + 0], pa, hsub2((w01 & lm) | ex, off), hsub2((w23 & lm) | ex, off));
            mma_h(Y[4 * c + 1], pa, hfma2((w01 & hm) | ex, s16, o16), hfma2((w23 & hm) | ex, s16, o16));
            const uint32_t h01 = w01 >> 8, h23 = w23 >> 8;
            mma_h(Y[4 * c + 2], pa, hsub2((h01 & lm) | ex, off), hsub2((h23 & lm) | ex, off));
            mma_h(Y[4 * c + 3], pa, hfma2((h01 & hm) | ex, s16, o16), hfma2((h23 & hm) | ex, s16, o16));
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();
    // ---- the partial of this row block
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const long long part = a.w.item_off[b] + blk + w;
    if (j == 0) {
      a.w.pm[part * 16 + r] = m0;
      a.w.pm[part * 16 + r + 8] = m1;
      a.w.pl[part * 16 + r] = l0;
      a.w.pl[part * 16 + r + 8] = l1;
    }
    float* y0 = a.w.pY + (part * 16 + r) * 128 + 8 * j;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // tile 4 c + i: columns 2 j, 2 j + 1 = channels 32 c + 8 j + i, + 4
      if (row0 < R) {
        *reinterpret_cast<float4*>(y0 + 32 * c) = make_float4(Y[4 * c][0], Y[4 * c + 1][0], Y[4 * c + 2][0], Y[4 * c + 3][0]);
        *reinterpret_cast<float4*>(y0 + 32 * c + 4) = make_float4(Y[4 * c][1], Y[4 * c + 1][1], Y[4 * c + 2][1], Y[4 * c + 3][1]);
      }
      if (row1 < R) {
        *reinterpret_cast<float4*>(y0 + 1024 + 32 * c) = make_float4(Y[4 * c][2], Y[4 * c + 1][2], Y[4 * c + 2][2], Y[4 * c + 3][2]);
        *reinterpret_cast<float4*>(y0 + 1024 + 32 * c + 4) = make_float4(Y[4 * c][3], Y[4 * c + 1][3], Y[4 * c + 2][3], Y[4 * c + 3][3]);
      }
    }
    u += p1 - p0;
  }
}

// ------------------------------------------------------------------ many rows: tcgen05
// With more rows than a few warp tiles the scores and the weighted sum are products of 128-row tiles on the tensor
// cores: S = Q K^T and O += P V over tiles of 128 tokens, Q (fp16) and P as A operands in TMEM, the codes turned into
// fp16 tiles in shared memory once for all rows of the KV head.  K and V tiles have the same layout ([token][64
// channels] atoms, 128-byte swizzle); K is read as a K-major operand, V as an MN-major one (its contraction runs over the
// tokens).
//   warps 0 - 7   dequantisation: each owns one page of every tile, with its own ring of 16-byte asynchronous copies (one
//                 copying warp with bulk copies of 128 to 2176 bytes took 2400 cycles a tile to issue them); a lane
//                 takes a slot's group of 32 channels, a warp 8 slots x 4 groups, so that its 16-byte stores do not conflict
//   warp 8        MMA issue: S(0), S(1), then O += P(k) V(k) and S(k + 2)
//   warps 9 ..    softmax, 8 warps, one row per thread: four take the even tiles, four the odd ones, so that one set's
//                 exponentials run beside the other's loads and maxima.  The row's running maximum is handed from tile to
//                 tile through shared memory as soon as it is known; rows past the block's are skipped by the warp.  P
//                 overwrites S in TMEM; O is rescaled when the maximum grew by more than 2^8.
// TMEM: S in two 128-column buffers, O in 256 .. 383, Q in 384 .. 447.  Units of work: tiles, dealt to the CTAs as above.
constexpr int kTcDeq = 8, kTcSoft = 8;
constexpr int kTcThreads = 32 * (1 + kTcDeq + kTcSoft);
constexpr int kTcTile = 32768, kTcAtom = 16384;

template <int BITS>
struct TcFmt {
  static constexpr int KB = PageFmt<BITS>::KB, VS = PageFmt<BITS>::VS;
  static constexpr int RAW = 8 * PageFmt<BITS>::STAGE;           // 34816 or 18432 bytes: the pages of a tile
  static constexpr int RS = BITS == 8 ? 2 : 4;                   // tiles in flight
  static constexpr size_t SMEM = 4 * (size_t)kTcTile + (size_t)RS * RAW + 1024;
};

// One CTA's run of units, a row block's tiles at a time; by a whole warp.
struct TcWalk {
  long long u, u1;
  int b, g, rb, p0, p1, len, R;
  TreeSeq sq;
  long long part;   // index of the partial of this row block
};
__device__ __forceinline__ bool tc_next(const TreeMma& a, TcWalk& s, int w, int lane) {
  if (s.u >= s.u1) return false;
  s.b = warp_find(a.w.unit_off, a.t.batch, s.u, lane);
  s.sq = seq_of(a.t, s.b, a.v.status, false);
  s.R = s.sq.cnt * a.v.group_q;
  s.len = s.sq.hist + s.sq.cnt;
  const int nrb = (s.R + kTcRows - 1) / kTcRows, tiles = (s.len + kTcTok - 1) / kTcTok;
  const long long rem = s.u - a.w.unit_off[s.b];
  const int blk = (int)(rem / tiles);
  s.p0 = (int)(rem % tiles);
  s.g = blk / nrb;
  s.rb = blk % nrb;
  s.p1 = (int)min((long long)tiles, s.p0 + (s.u1 - s.u));
  s.part = a.w.item_off[s.b] + blk + w;
  s.u += s.p1 - s.p0;
  return true;
}

// Visible slots among hist + j0 .. hist + j0 + 31 for node i (row `row` of the mask), as bits: the history (j < 0), and
// the nodes that the mask names.
__device__ __forceinline__ uint32_t vis32(const TreeArgs& t, int row, int i, int cnt, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  auto word = [&](int w) -> uint32_t {
    uint32_t x;
    if (t.mask)
      x = w < t.mask_words ? t.mask[(size_t)row * t.mask_words + w] : 0u;
    else
      x = i >= 32 * w + 31 ? 0xffffffffu : i < 32 * w ? 0u : (2u << (i - 32 * w)) - 1u;
    const int n = cnt - 32 * w;   // nodes from this word on
    return n >= 32 ? x : n <= 0 ? 0u : x & ((1u << n) - 1u);
  };
  if (j0 < 0) return ((1u << -j0) - 1u) | (word(0) << -j0);
  const int w = j0 >> 5, sh = j0 & 31;
  return sh == 0 ? word(w) : __funnelshift_r(word(w), word(w + 1), sh);
}

__device__ __forceinline__ void tmem_ld32x(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// One lane of the converged warp, always the same.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// tc::mma_f16_ts and tc::mma_commit by the lane whose `leader` is set.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 bd;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// Two fp32 numbers in one register pair, and their packed sum.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Wait for this thread's TMEM loads; the registers pass through, so no use of them moves before it.
__device__ __forceinline__ void tmem_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_st16x(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32x(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// Eight codes times their scale, fp16: 8-bit ones in channel order, 4-bit ones in the order 0 4 1 5 2 6 3 7 of the masks (Q has
// it too; the output is put in order where it leaves TMEM).
template <int BITS>
__device__ __forceinline__ uint4 deq8(uint2 w, uint32_t s2) {
  auto hmul = [](uint32_t x, uint32_t y) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  uint32_t o[4];
  if constexpr (BITS == 8) {
    constexpr uint32_t off = 0x64806480u, ex = 0x64646464u;
    o[0] = hmul(hsub2(__byte_perm(w.x, ex, 0x4140), off), s2);
    o[1] = hmul(hsub2(__byte_perm(w.x, ex, 0x4342), off), s2);
    o[2] = hmul(hsub2(__byte_perm(w.y, ex, 0x4140), off), s2);
    o[3] = hmul(hsub2(__byte_perm(w.y, ex, 0x4342), off), s2);
  } else {
    const uint32_t x = w.x, x8 = w.x >> 8;
    constexpr uint32_t lm = 0x000F000Fu, hm = 0x00F000F0u, ex = 0x64006400u, off = 0x64086408u;
    constexpr uint32_t s16 = 0x2C002C00u, o16 = 0xD480D480u;
    o[0] = hmul(hsub2((x & lm) | ex, off), s2);
    o[1] = hmul(hfma2((x & hm) | ex, s16, o16), s2);
    o[2] = hmul(hsub2((x8 & lm) | ex, off), s2);
    o[3] = hmul(hfma2((x8 & hm) | ex, s16, o16), s2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int BITS>
__global__ void __launch_bounds__(kTcThreads, 1) k_tree_tc(TreeMma a) {
  using F = TcFmt<BITS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], q_full,
      o_free, fin;
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;
  __shared__ float xch[2][kTcRows], xl[2][kTcRows];   // by tile parity: row maxima handed on, and sums
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* K_s = smem;                      // two stages
  uint8_t* V_s = smem + 2 * kTcTile;        // two stages
  uint8_t* R_s = smem + 4 * kTcTile;        // raw pages
  const LayerView& v = a.v;
  const TreeArgs& t = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long U = a.w.unit_off[t.batch];
  const long long We = workers_used(a, U);
  const int w = blockIdx.x;
  if (w >= We || U == 0) return;
  TcWalk wk;
  wk.u = (long long)w * U / We;
  wk.u1 = (long long)(w + 1) * U / We;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&k_full[s], kTcDeq);
      tc::mbar_init(&k_empty[s], 1);
      tc::mbar_init(&v_full[s], kTcDeq);
      tc::mbar_init(&v_empty[s], 1);
      tc::mbar_init(&s_full[s], 1);
      // one barrier per tile parity, whose tiles belong to one half of the softmax warps
      tc::mbar_init(&p_full[s], kTcSoft / 2);
      tc::mbar_init(&o_done[s], 1);
    }
    tc::mbar_init(&q_full, kTcSoft);
    tc::mbar_init(&o_free, kTcSoft);
    tc::mbar_init(&fin, 1);
    abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == kTcDeq) tc::tmem_alloc(&tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_base;
  constexpr uint32_t o_col = 256, q_col = 384;

  if (warp == kTcDeq) {
    // ------------------------------------------------ MMA issue
    const uint32_t idesc_s = tc::idesc_f16(128, 128, false, false, false);
    const uint32_t idesc_o = tc::idesc_f16(128, 128, false, false, true);   // V: tokens are the contraction
    const uint64_t dk = tc::sdesc_sw128(tc::smem_u32(K_s), 0, 1024);
    const uint64_t dv = tc::sdesc_sw128(tc::smem_u32(V_s), kTcAtom, 1024);  // 64 channels to the next, 8 tokens to the next
    const uint32_t k_lo = tc::desc_lo(dk), k_hi = tc::desc_hi(dk), v_lo = tc::desc_lo(dv), v_hi = tc::desc_hi(dv);
    // The whole warp walks the loop and one elected lane issues, by a predicate on the instruction: the control flow stays
    // uniform, so descriptors and addresses stay in uniform registers (issued from a branch of one lane, an MMA took about 100
    // cycles to issue, more than its execution).
    const uint32_t leader = elect_one();
    bool ok = true;
    int jg = 0, n = 0;   // tiles and row blocks so far
    auto issue_s = [&](int j) -> bool {
      const int s = j & 1;
      if (!tc::mbar_wait_ab(&k_full[s], ((uint32_t)(j >> 1)) & 1u, v.status, &abort_flag)) return false;
      tc::tc_fence_after();
      // S buffer j & 1 is free: P(j - 2) V(j - 2), issued before, has read it by the time these run (a block's first two
      // tiles: the last block's products have completed, its softmax warps have said so by q_full)
      const uint32_t d = tmem + (uint32_t)(s * 128), b = k_lo + (uint32_t)(s * kTcTile >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts(leader, d, tmem + q_col + 8u * kk, b + (uint32_t)(kk >> 2) * (kTcAtom >> 4) + 2u * (kk & 3), k_hi, idesc_s,
               kk ? 1u : 0u);
      commit(leader, &s_full[s]);
      commit(leader, &k_empty[s]);
      return true;
    };
    while (ok && tc_next(a, wk, w, lane)) {
      const int nt = __shfl_sync(0xffffffffu, wk.p1 - wk.p0, 0);
      ok = tc::mbar_wait_ab(&q_full, (uint32_t)n & 1u, v.status, &abort_flag);
      tc::tc_fence_after();
      ok = ok && issue_s(jg) && (nt == 1 || issue_s(jg + 1));
      for (int k = 0; ok && k < nt; ++k) {
        const int j = jg + k, s = j & 1;
        if (k == 0 && !(ok = tc::mbar_wait_ab(&o_free, ((uint32_t)n & 1u) ^ 1u, v.status, &abort_flag))) break;
        if (!(ok = tc::mbar_wait_ab(&v_full[s], ((uint32_t)(j >> 1)) & 1u, v.status, &abort_flag))) break;
        if (!(ok = tc::mbar_wait_ab(&p_full[s], ((uint32_t)(j >> 1)) & 1u, v.status, &abort_flag))) break;
        tc::tc_fence_after();
        const uint32_t p = tmem + (uint32_t)(s * 128), b = v_lo + (uint32_t)(s * kTcTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(leader, tmem + o_col, p + 8u * kk, b + (uint32_t)(kk * 2048 >> 4), v_hi, idesc_o, (k | kk) ? 1u : 0u);
        commit(leader, &o_done[s]);
        commit(leader, &v_empty[s]);
        if (k + 2 < nt && !(ok = issue_s(j + 2))) break;
      }
      jg += nt;
      ++n;
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) abort_flag = 1;
    commit(leader, &fin);
    tc::mbar_wait(&fin, 0, v.status);   // every MMA has completed before the CTA may exit
    __syncwarp();
  } else if (warp < kTcDeq) {
    // ------------------------------------------------ dequantisation: page `warp` of every tile
    const int sl = lane & 7, gr = lane >> 3;   // slot of a half page, group of 32 channels
    // this lane's stores: chunk c of its group is 16-byte chunk 4 (gr % 2) + c of atom gr / 2, at that ^ (row % 8 = slot)
    const uint32_t st0 = (uint32_t)(gr >> 1) * kTcAtom + (uint32_t)warp * 2048u + (uint32_t)sl * 128u;
    const uint32_t st1 = (uint32_t)((4 * (gr & 1)) ^ sl) << 4;
    uint8_t* ring = R_s + (size_t)warp * F::RS * PageFmt<BITS>::STAGE;
    const uint32_t ring_s = tc::smem_u32(ring);
    bool ok = true;
    int n = 0;
    while (ok && tc_next(a, wk, w, lane)) {
      const int32_t* pt = t.pt + (size_t)wk.b * t.max_pages;
      const int pages = (wk.len + kPage - 1) / kPage;
      int ids0 = wk.p0, next = wk.p0;
      auto fetch_ids = [&]() {   // this warp's page of 32 tiles; -2: past the sequence's pages
        const int p = (ids0 + lane) * 8 + warp;
        return ids0 + lane < wk.p1 ? (p < pages ? max(pt[p], -1) : -2) : -2;
      };
      int ids = fetch_ids();
      auto issue = [&]() {
        if (next < wk.p1) {
          if (next - ids0 == 32) {
            ids0 = next;
            ids = fetch_ids();
          }
          const int page = __shfl_sync(0xffffffffu, ids, next - ids0);
          // past the sequence's pages the stage keeps what it held: those tokens' scales are set to zero
          if (page != -2)
            issue_page<BITS>(a, page, wk.g, ring_s + (uint32_t)((next - wk.p0) % F::RS) * PageFmt<BITS>::STAGE, lane);
          ++next;
        }
        cp_commit();
      };
#pragma unroll
      for (int k = 0; k < F::RS - 1; ++k) issue();
      for (int k = wk.p0; k < wk.p1 && ok; ++k, ++n) {
        const int s = n & 1;
        cp_wait<F::RS - 2>();
        __syncwarp();   // this page's bytes from every lane; every lane is done with the stage that is filled next
        issue();
        const uint8_t* raw = ring + (size_t)((k - wk.p0) % F::RS) * PageFmt<BITS>::STAGE;
        const int tokens = wk.len - (k * kTcTok + warp * 16);   // of this page
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const uint8_t* sc = (side ? raw + F::KB : raw) + 32 * gr + 2 * sl;
          const uint8_t* cd = (side ? raw + F::KB + F::VS : raw + 128) + gr * (64 * BITS) + sl * (4 * BITS);
          // all loads first: the compiler keeps a load behind a store that may alias it
          uint4 code[2][BITS / 4];
          uint32_t scale[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i = 0; i < BITS / 4; ++i) code[half][i] = *reinterpret_cast<const uint4*>(cd + half * (32 * BITS) + i * 16);
            scale[half] = *reinterpret_cast<const uint16_t*>(sc + half * 16);
          }
          ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_ab(side ? &v_empty[s] : &k_empty[s], (((uint32_t)(n >> 1)) & 1u) ^ 1u, v.status, &abort_flag));
          if (ok) {
            uint8_t* tile = (side ? V_s : K_s) + (size_t)s * kTcTile + st0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // slots without a token may hold any bytes: their scale is zero
              const uint32_t h = half * 8 + sl < tokens ? scale[half] : 0u, s2 = __byte_perm(h, 0u, 0x1010);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint4& w4 = code[half][BITS == 8 ? c >> 1 : 0];
                uint2 x;
                if constexpr (BITS == 8)
                  x = c & 1 ? make_uint2(w4.z, w4.w) : make_uint2(w4.x, w4.y);
                else
                  x = make_uint2(c == 0 ? w4.x : c == 1 ? w4.y : c == 2 ? w4.z : w4.w, 0u);
                *reinterpret_cast<uint4*>(tile + half * 1024 + (((uint32_t)c << 4) ^ st1)) = deq8<BITS>(x, s2);
              }
            }
            tc::fence_proxy_async();
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(side ? &v_full[s] : &k_full[s]);
        }
      }
      cp_wait<0>();
      __syncwarp();
    }
  } else {
    // ------------------------------------------------ softmax and output
    const int qq = warp & 3, x = (warp - 1 - kTcDeq) >> 2;   // TMEM lane quarter; tiles of this parity
    const int r = qq * 32 + lane;
    const uint32_t lane_base = (uint32_t)(qq * 32) << 16;
    const uint32_t s_at = tmem + lane_base + 128u * x, o_at = tmem + lane_base + o_col;
    // named barriers of the two warps of a quarter: 1 + 2 qq + parity hands on the maximum after a tile of that
    // parity, 9 + qq joins the sums
    const int bar_out = 1 + 2 * qq + x, bar_in = 1 + 2 * qq + (x ^ 1), bar_l = 9 + qq;
    bool ok = true;
    int jg = 0;
    while (tc_next(a, wk, w, lane)) {
      const int row = wk.rb * kTcRows + r;                       // row of the sequence and KV head
      const bool warp_live = wk.rb * kTcRows + qq * 32 < wk.R;   // some row of this warp is real
      const int node = row / v.group_q;
      // ---- this row's Q: 64 of its channels (32 columns) into TMEM.  The last block's MMAs have completed (o_done).
      {
        uint32_t qv[32];
        const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)a.w.q +
                                                          ((size_t)(wk.sq.off + node) * v.H + wk.g * v.group_q + row % v.group_q) * 128 + 64 * x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 z = row < wk.R ? src[c] : make_uint4(0, 0, 0, 0);
          qv[4 * c] = z.x;
          qv[4 * c + 1] = z.y;
          qv[4 * c + 2] = z.z;
          qv[4 * c + 3] = z.w;
        }
        tmem_st32x(tmem + lane_base + q_col + 32u * x, qv);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_full);
      }
      float m_used = -1e30f, l = 0.f;   // l is the sum of this parity's tiles, in units of 2^m_used
      const int nt = wk.p1 - wk.p0;
      for (int k = (jg & 1) == x ? 0 : 1; k < nt; k += 2) {
        const int j = jg + k;
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_ab(&s_full[x], ((uint32_t)(j >> 1)) & 1u, v.status, &abort_flag));
        tc::tc_fence_after();
        if (warp_live) {   // (also after an abort: the two warps of a quarter meet at their barriers, over old columns)
          const int t0 = (wk.p0 + k) * kTcTok;
          const bool tail = t0 + kTcTok > wk.sq.hist;   // the tile holds drafted nodes or unused slots
          if (tail) {   // what a row does not see becomes -infinity in TMEM
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              float s[32];
              const uint32_t see = row < wk.R ? vis32(t, wk.sq.off + node, node, wk.sq.cnt, t0 + 32 * h - wk.sq.hist) : 0u;
              tmem_ld32x(s_at + 32u * h, s);
              tmem_wait32(s);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(see >> c & 1u)) s[c] = -INFINITY;
              tmem_st32x(s_at + 32u * h, reinterpret_cast<const uint32_t*>(s));
            }
            tc::tmem_st_wait();
          }
          // S in four pieces of 32 columns, twice: for the maximum, and for the exponentials; each piece is asked for while
          // the one before is worked on
          float s0[32], s1[32];
          auto top = [](const float* s) {
            float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 32; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          };
          tmem_ld32x(s_at, s0);
          tmem_wait32(s0);
          tmem_ld32x(s_at + 32u, s1);
          float mx = top(s0);
          tmem_wait32(s1);
          tmem_ld32x(s_at + 64u, s0);
          mx = fmaxf(mx, top(s1));
          tmem_wait32(s0);
          tmem_ld32x(s_at + 96u, s1);
          mx = fmaxf(mx, top(s0));
          tmem_wait32(s1);
          tmem_ld32x(s_at, s0);
          mx = fmaxf(mx, top(s1));
          float m_prev = m_used;
          if (k > 0) {   // the maximum as the other parity's tile left it
            asm volatile("bar.sync %0, 64;" ::"r"(bar_in) : "memory");
            m_prev = xch[x ^ 1][r];
          }
          const float m_new = mx > m_prev + 8.f ? mx : m_prev;
          xch[x][r] = m_new;
          asm volatile("bar.arrive %0, 64;" ::"r"(bar_out) : "memory");
          l *= ex2(m_used - m_new);
          m_used = m_new;
          // O is in units of 2^m_prev until here
          if (k > 0 && __any_sync(0xffffffffu, m_new != m_prev)) {
            // (S(j) is complete, so O += P(j - 2) V(j - 2), issued before it, is too: the wait is for the phase meant)
            ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_ab(&o_done[x ^ 1], ((uint32_t)((j - 1) >> 1)) & 1u, v.status, &abort_flag));
            tc::tc_fence_after();
            if (ok) {
              const float f = ex2(m_prev - m_new);
#pragma unroll 1
              for (int c = 0; c < 128; c += 16) {
                float o[16];
                uint32_t ou[16];
                tc::tmem_ld16_sync(o_at + (uint32_t)c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) ou[i] = __float_as_uint(o[i] * f);
                tc::tmem_st8(o_at + (uint32_t)c, ou);
                tc::tmem_st8(o_at + (uint32_t)c + 8, ou + 8);
              }
              tc::tmem_st_wait();
            }
          }
          // P over columns of S that have been read: 16 columns of pairs for 32 of scores
          unsigned long long l2[4] = {0ull, 0ull, 0ull, 0ull};   // packed pairs of sums
          const unsigned long long nm = pack2(-m_used, -m_used);
          auto put = [&](uint32_t at, const float* s) {
            uint32_t p2[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 d = unpack2(add2(pack2(s[c], s[c + 1]), nm));
              const float e0 = ex2(d.x), e1 = ex2(d.y);
              l2[(c >> 1) & 3] = add2(l2[(c >> 1) & 3], pack2(e0, e1));
              p2[c / 2] = h2(e0, e1);
            }
            tmem_st16x(at, p2);
          };
          tmem_wait32(s0);
          tmem_ld32x(s_at + 32u, s1);
          put(s_at, s0);
          tmem_wait32(s1);
          tmem_ld32x(s_at + 64u, s0);
          put(s_at + 16u, s1);
          tmem_wait32(s0);
          tmem_ld32x(s_at + 96u, s1);
          put(s_at + 32u, s0);
          tmem_wait32(s1);
          put(s_at + 48u, s1);
          const float2 ls = unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
          l += ls.x + ls.y;
          tc::tmem_st_wait();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[x]);
      }
      jg += nt;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_ab(&o_done[(jg - 1) & 1], ((uint32_t)((jg - 1) >> 1)) & 1u, v.status, &abort_flag));
      tc::tc_fence_after();
      if (warp_live) {
        // the final maximum: the last tile's warp has it, the other takes its last hand-over
        float m_end = m_used;
        if (((jg - 1) & 1) != x) {
          asm volatile("bar.sync %0, 64;" ::"r"(bar_in) : "memory");
          m_end = xch[x ^ 1][r];
        }
        xl[x][r] = l * ex2(m_used - m_end);
        asm volatile("bar.sync %0, 64;" ::"r"(bar_l) : "memory");
        l = xl[0][r] + xl[1][r];
        if (x == 0 && row < wk.R) {
          a.w.pm[wk.part * kTcRows + r] = m_end;
          a.w.pl[wk.part * kTcRows + r] = ok ? l : 0.f;
        }
        float* y = a.w.pY + (wk.part * kTcRows + r) * 128 + 64 * x;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          float o[16];
          if (ok)
            tc::tmem_ld16_sync(o_at + 64u * x + (uint32_t)c, o);
          else
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0.f;
          if (row < wk.R) {
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
              float4* d = reinterpret_cast<float4*>(y + c + i);
              if constexpr (BITS == 4) {
                d[0] = make_float4(o[i], o[i + 2], o[i + 4], o[i + 6]);
                d[1] = make_float4(o[i + 1], o[i + 3], o[i + 5], o[i + 7]);
              } else {
                d[0] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                d[1] = make_float4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
              }
            }
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&o_free);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kTcDeq) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merging the partials
// One warp per (output row, query head), lane: four channels.  Writes y as fp16 into the output product's B tiles;
// rows of no sequence and the tiles' padding rows are zero.
__global__ void __launch_bounds__(256) k_tree_combine(TreeMma a, int rows_pad, int NB, int KT) {
  const LayerView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31;
  const long long id = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  if (id >= (long long)rows_pad * v.H) return;
  const int row = (int)(id / v.H), h = (int)(id % v.H);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  int b = -1;
  if (t.lens)
    b = row < t.batch ? row : -1;
  else if (row >= t.node_off[0] && row < t.node_off[t.batch])
    b = warp_find(t.node_off, t.batch, row, lane);
  if (b >= 0) {
    const TreeSeq sq = seq_of(t, b, v.status, false);
    if (sq.cnt > 0 && row >= sq.off && row - sq.off < sq.cnt && a.w.item_off[b + 1] > a.w.item_off[b]) {
      const int g = h / v.group_q, rr = (row - sq.off) * v.group_q + h % v.group_q;
      const int nrb = (sq.cnt * v.group_q + a.rb - 1) / a.rb, units = (sq.hist + sq.cnt + a.unit - 1) / a.unit;
      const int blk = g * nrb + rr / a.rb, r = rr % a.rb;
      const long long U = a.w.unit_off[t.batch];
      const long long We = workers_used(a, U);
      const long long lo = a.w.unit_off[b] + (long long)blk * units, hi = lo + units - 1;
      const long long w0 = ((lo + 1) * We - 1) / U, w1 = ((hi + 1) * We - 1) / U;   // the warps of the first, last unit
      const long long base = a.w.item_off[b] + blk;
      float m = -FLT_MAX, l = 0.f;
      for (long long w = w0 + lane; w <= w1; w += 32) m = fmaxf(m, a.w.pm[(base + w) * a.rb + r]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
      for (long long w = w0; w <= w1; ++w) {
        const long long p = (base + w) * a.rb + r;
        const float f = ex2(a.w.pm[p] - m);
        const float4 x = *reinterpret_cast<const float4*>(a.w.pY + p * 128 + lane * 4);
        l += f * a.w.pl[p];
        y.x += f * x.x;
        y.y += f * x.y;
        y.z += f * x.z;
        y.w += f * x.w;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees nothing: zero; NaN stays
      y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    }
  }
  const int nt = row / NB, br = row % NB;
  const uint32_t k = (uint32_t)(h * 128 + lane * 4), c = k & 63u;
  uint8_t* tile = (uint8_t*)a.w.y + ((size_t)nt * KT + (k >> 6)) * (size_t)NB * 128;
  *reinterpret_cast<uint2*>(tile + tc::sw128((uint32_t)br, c >> 3) + (c & 7u) * 2u) = make_uint2(h2(y.x, y.y), h2(y.z, y.w));
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

int tree_workers(int kv_bits) {
  const int per_sm = (kv_bits == 0 ? PageFmt<0>::CTAS : PageFmt<8>::CTAS) * kTreeWarps;
  return per_sm * num_sms();
}

struct TreePlan {
  size_t unit_off, item_off, q, pm, pl, pY, y, part, total;
  int NB, rows_pad;
  bool tc;               // k_tree_tc
  int workers, rb;
};

// Rows per sequence and KV head from which the 128-row kernel is taken.
constexpr int kTcFrom = 33;

TreePlan tree_plan(const starkv_layer* L, int batch, int n_nodes, int max_nodes) {
  const LayerView& v = L->view;
  TreePlan p;
  p.NB = outproj_nb(n_nodes);
  p.rows_pad = (n_nodes + p.NB - 1) / p.NB * p.NB;
  // row blocks of 16 or 128 rows, one more per sequence for what its last block leaves empty
  p.tc = v.kv_bits != 0 && max_nodes * v.group_q >= kTcFrom;
  p.workers = p.tc ? num_sms() : tree_workers(v.kv_bits);
  p.rb = p.tc ? kTcRows : 16;
  const size_t items = (size_t)v.Hkv * std::min((size_t)batch * ((max_nodes * v.group_q + p.rb - 1) / p.rb),
                                                (size_t)batch + (size_t)n_nodes * v.group_q / p.rb);
  const size_t parts = items + p.workers;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += al256(bytes);
    return at;
  };
  p.unit_off = take(8 * ((size_t)batch + 1));
  p.item_off = take(8 * ((size_t)batch + 1));
  p.q = take((size_t)n_nodes * v.H * 256 * (v.kv_bits == 0 ? 2 : 1));
  p.pm = take(parts * p.rb * 4);
  p.pl = take(parts * p.rb * 4);
  p.pY = take(parts * p.rb * 512);
  p.y = take((size_t)p.rows_pad / p.NB * (L->Kp / 64) * p.NB * 128);
  p.part = take(outproj_part_bytes(L, n_nodes));
  p.total = o;
  return p;
}

template <int BITS>
cudaError_t launch_bits(const starkv_layer* L, TreeMma& a, const TreePlan& p, cudaStream_t s) {
  using F = PageFmt<BITS>;
  const LayerView& v = L->view;
  const dim3 pgrid(a.t.n_nodes + 1, (v.H + kTreeWarps - 1) / kTreeWarps);
  if (BITS == 4 && !p.tc)
    k_tree_prep<BITS, 1><<<pgrid, 32 * kTreeWarps, 0, s>>>(a);
  else if (BITS == 4)
    k_tree_prep<BITS, 2><<<pgrid, 32 * kTreeWarps, 0, s>>>(a);
  else
    k_tree_prep<BITS, 0><<<pgrid, 32 * kTreeWarps, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (BITS != 0 && p.tc) {
    constexpr int B = BITS == 0 ? 8 : BITS;
    if ((e = set_smem_limit((const void*)k_tree_tc<B>, TcFmt<B>::SMEM)) != cudaSuccess) return e;
    k_tree_tc<B><<<a.workers, kTcThreads, TcFmt<B>::SMEM, s>>>(a);
    return cudaGetLastError();
  }
  const size_t smem = (size_t)kTreeWarps * F::NS * F::STAGE;
  if ((e = set_smem_limit((const void*)k_tree_mma<BITS>, smem)) != cudaSuccess) return e;
  k_tree_mma<BITS><<<a.workers / kTreeWarps, 32 * kTreeWarps, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool tree_mma_supported(const LayerView& v) { return v.plain && v.dtype == STARKV_BF16 && v.d == 128; }

size_t tree_mma_ws_bytes(const starkv_layer* L, int batch, int n_nodes, int max_nodes) {
  return tree_plan(L, batch, n_nodes, max_nodes).total;
}

cudaError_t launch_tree_mma(const starkv_layer* L, const TreeArgs& t, void* ws, size_t ws_bytes, cudaStream_t s) {
  const LayerView& v = L->view;
  const TreePlan p = tree_plan(L, t.batch, t.n_nodes, t.max_nodes);
  if (ws_bytes < p.total) return cudaErrorInvalidValue;
  uint8_t* w = (uint8_t*)ws;
  TreeMma a;
  a.v = v;
  a.t = t;
  a.w.unit_off = (long long*)(w + p.unit_off);
  a.w.item_off = (long long*)(w + p.item_off);
  a.w.q = w + p.q;
  a.w.pm = (float*)(w + p.pm);
  a.w.pl = (float*)(w + p.pl);
  a.w.pY = (float*)(w + p.pY);
  a.w.y = w + p.y;
  a.w.part = w + p.part;
  a.workers = p.workers;
  a.rb = p.rb;
  a.unit = p.tc ? kTcTok : kPage;
  a.min_units = p.tc ? 1 : kMinUnits;
  cudaError_t e = v.kv_bits == 8 ? launch_bits<8>(L, a, p, s) : v.kv_bits == 4 ? launch_bits<4>(L, a, p, s)
                                                                               : launch_bits<0>(L, a, p, s);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)p.rows_pad * v.H;
  k_tree_combine<<<(unsigned)((warps * 32 + 255) / 256), 256, 0, s>>>(a, p.rows_pad, p.NB, L->Kp / 64);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_outproj_tc(L, a.w.y, t.n_nodes, t.out, (float*)a.w.part, s, t.lens ? nullptr : t.node_off + t.batch);
}

}  // namespace starkv
