// Attention of drafted tokens (nodes of a tree, a chain, or one token) over an
// uncompressed layer's cache: bf16 K and V, or their 8 / 4-bit codes.
//
// Every KV head's R = nodes * group rows of a sequence share its K and V, so a page (16 tokens) is read once for all of a
// block's rows.  Two kernels: k_tree_mma, up to 24 rows a block, on warp-level matrix instructions (m16n8k16: 16 tokens
// or 16 channels by 8 rows, so that a single row wastes an N of 8, not an M of 16 or 128), fed from registers; and
// k_tree_tc, 128 rows a block, on tcgen05.
//
// k_tree_mma turns codes into operands without scaling them first:
//   scores   S^T = K Q^T.  A code byte u under the fp16 exponent of 1024 is the number 1024 + u (one PRMT per two codes;
//            4-bit codes in a word's high nibbles come out as 1024 + 16 u, their q is 1/16).  A group's accumulator starts
//            at -sum_c q_c (1024 + 2^(b-1)), so it ends at sum_c q_c (u - 2^(b-1)); then S += scale[token][group] * it.
//            What cancels is far larger than what is left, so its rounding counts: the sums on the way are at most 1279 sum|q_c|
//            over a group of 8 bits (1039 over 4), and each fp32 rounding of one is off by 2^-24 of that, 7.6e-5 (6.2e-5)
//            sum|q_c| <= 4.3e-4 (3.5e-4) |q| codes.  A group's key is at least 126 (7) codes long, which makes it 3.4e-6 (5e-5)
//            of |q||k| at most; with codes spread evenly 1.0e-6 (1.5e-5).  (q's own rounding to fp16: 2^-11 of a channel.)
//   values   Y^T = V^T P^T.  P is transposed by one movmatrix per 8 tokens.  The codes become exact integers (the offset taken
//            off by one packed subtraction; it cannot be folded into the accumulator here, whose sum over thousands of tokens
//            would cancel) and are multiplied by their token's scale in fp16.  |code * scale| stays below 32800, and as every scale
//            is a multiple of 2^-24 so is every product: the rounding is 2^-11 of it at most, however small the scale.  (P * scale
//            instead, with 2 NT products a group for 8, leaves fp16 at both ends: 2^7 * 4681, the largest scale of 4 bits, is
//            infinite, and a weight 2^-12 of the largest is lost beside values of 1e-3.  It took 97.4 us for one token each of 16
//            sequences of 4K over 4 bits and 32 heads against 98.4, 133.3 against 131.9 for 16, and over 8 bits 101.0 against
//            100.7 and 129.9 against 129.5.)
// Channels may be dealt to a contraction in any order, so each lane reads runs of bytes: eight channels of a token for the
// scores, 8 bytes of each of four tokens for the values (bf16: four channels).
//
// Running maximum and sum are per row in registers.  m is the row's maximum less 3 (log2 units) and moves only when a
// score passes m + 7: p = 2^(s - m) <= 2^7, while the largest weight seen is at least 8, so that weights down to 2^-17 of it
// keep full precision in fp16.
//
// Work split: the units (sequence, KV head, row block, page) of the whole call, in this order, are dealt to the resident
// warps in equal runs; a warp writes one partial (m, l, Y) per row block that its run touches, and k_tree_combine
// merges them.  Warps never wait for one another; each keeps its own ring of pages in flight with 16-byte
// asynchronous copies.  Measured, 16 sequences of 4K (less a ragged 15 %) over 8 bits and 32 heads: one token each 82 us, 5.95 TB/s,
// 0.92 of a copy's rate (with 16 query rows as the M side a page took 670 instructions, and the call 129 us); trees of 16
// 105 us, bound by the fixed latencies of two warps a scheduler.
#include <float.h>

#include "tc_common.cuh"

namespace starkv {

namespace {

constexpr int kTreeWarps = 4;          // warps per CTA
// Pages of a warp's run, at least (short calls use fewer warps).  Runs of 1 / 2 / 4, a whole call over 8 bits, us: one token over 100 15.3 /
// 16.6 / 17.9 (8 KV heads), 7 nodes over 333 18.3 / 18.3 / 19.7 (32), 4 x 7 over 200 25.7 / 25.2 / 25.0 (32), 4 over 1000 22.2 / 22.2 /
// 24.3 (8), 16 x 1 over 500 24.5 / 24.5 / 22.6 (8).
constexpr int kMinUnits = 2;
constexpr int kTcRows = 128;           // rows of a row block of k_tree_tc
constexpr int kTcTok = 128;            // tokens of its tiles

template <int BITS>
struct PageFmt {
  static constexpr int KB = BITS == 0 ? 4096 : 128 + 64 * 4 * BITS;   // key block of one head: scales, codes
  static constexpr int VS = BITS == 0 ? 0 : 128;                      // one head's value scales
  static constexpr int VB = BITS == 0 ? 4096 : 64 * 4 * BITS;         // one head's value codes
  static constexpr int STAGE = KB + VS + VB;                          // 8192, 4352 or 2304 bytes
};

// Row blocks of 8 NT rows.  CTAs per SM by registers (16 NT + 32 NT of query fragments and sums; bf16 holds the queries as
// two parts), ring stages by shared memory.
template <int BITS, int NT>
struct MmaFmt {
  static constexpr int CTAS = BITS == 0 ? 2 : NT == 1 ? 4 : 2;
  static constexpr int NS = (int)(212 * 1024 / (CTAS * kTreeWarps) / PageFmt<BITS>::STAGE) < 8
                                ? (int)(212 * 1024 / (CTAS * kTreeWarps) / PageFmt<BITS>::STAGE) : 8;
};

struct TreeWs {
  long long* unit_off;   // [batch + 1] units before a sequence
  long long* item_off;   // [batch + 1] row blocks before a sequence
  void* q;               // [n_nodes][H][128] fp16 in the kernels' channel order; bf16 layers: the high, then the low parts
  int* row_b;            // [n_nodes] sequence of a row, -1: none
  float *pm, *pl;        // [partials][rb]
  float* pY;             // [partials][rb][128]
  void* y;               // output tiles
  void* part;            // output product
};

struct TreeMma {
  ServeView v;
  TreeArgs t;
  TreeWs w;
  int workers;           // warps (k_tree_mma) or CTAs (k_tree_tc) that share the units
  int rb;                // rows of a row block: 16, or 128
  int unit;              // tokens of a unit: a page, or a tile of 128
  int min_units;         // least units of a worker's run
  float run_scale;       // and sqrt(run_scale * units of an average row block)
};

// How a call's units are dealt: worker w takes units [w U / We, (w + 1) U / We).  Short calls use fewer workers than there are:
// a run costs its units, the merge a row block's partials, so long row blocks are cut into the fewer the longer they are.  One
// sequence, 4 drafts, 8 KV heads, 8 bits: of 8000 tokens 63 us with runs of 2 pages and 47 with this rule, of 333 tokens 25 either way.
__device__ __forceinline__ long long workers_used(const TreeMma& a, long long U) {
  const long long items = max(1ll, a.w.item_off[a.t.batch]);
  const int run = max(a.min_units, (int)__fsqrt_rn((float)(U / items) * a.run_scale));
  return min((long long)a.workers, max(1ll, U / run));
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
// bf16 pair high + low for bf16 caches, whose products then carry 16 bits, like the weights: one bf16 weight alone made the
// outputs' error 2.2e-3 instead of 1.7e-3).  The last block row: prefix sums.
// ORDER (4-bit codes): 0 = channels in order; 1, 2 = every eight in the order 0 4 1 5 2 6 3 7 in which the nibble masks give
// them, with 1/16 for the odd ones (1: k_tree_mma, which meets 16 u there) or without (2: k_tree_tc).
template <int BITS, int ORDER>
__global__ void __launch_bounds__(128) k_tree_prep(TreeMma a) {
  const ServeView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  tc::grid_wait_prev();
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
  if (h == 0) {
    int b = t.lens ? row : -1;
    if (!t.lens && row >= t.node_off[0] && row < t.node_off[t.batch]) b = warp_find(t.node_off, t.batch, row, lane);
    if (lane == 0) a.w.row_b[row] = b;
  }
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
__device__ __forceinline__ void mma_h(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const float* c) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_b(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const float* c) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
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

// bf16 pages: 16-byte chunk c of token t's 256-byte row is kept at chunk c ^ swz(t): the rows of the eight lanes that read
// together then start at different banks (row stride = two rounds of the banks).
__device__ __forceinline__ int swz(int t) { return ((t & 1) << 2) | (t & 2) | ((t >> 2) & 1); }

// The 8 x 8 matrix of 16-bit elements whose rows r = lane / 4 hold columns 2 (lane % 4), + 1: transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

template <int BITS, int NT>
__global__ void __launch_bounds__(32 * kTreeWarps, MmaFmt<BITS, NT>::CTAS) k_tree_mma(TreeMma a) {
  using F = PageFmt<BITS>;
  constexpr int NS = MmaFmt<BITS, NT>::NS, RB = 8 * NT, QP = BITS == 0 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t ring_all[];
  const ServeView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, j = lane & 3;
  uint8_t* ring = ring_all + (size_t)warp * NS * F::STAGE;
  const uint32_t ring_s = tc::smem_u32(ring);
  const int GQ = v.group_q;
  tc::grid_wait_prev();
  tc::grid_launch_next();
  const long long U = a.w.unit_off[t.batch];
  const int w = warp * gridDim.x + blockIdx.x;   // neighbouring runs on different SMs
  const long long We = workers_used(a, U);
  if (w >= We) return;
  long long u = (long long)w * U / We;
  const long long u1 = (long long)(w + 1) * U / We;
  while (u < u1) {
    // ---- the row block of unit u
    const int b = warp_find(a.w.unit_off, t.batch, u, lane);
    const TreeSeq sq = seq_of(t, b, v.status, false);
    const int R = sq.cnt * GQ, nrb = (R + RB - 1) / RB, len = sq.hist + sq.cnt, pages = (len + kPage - 1) / kPage;
    const long long rem = u - a.w.unit_off[b];
    const int blk = (int)(rem / pages), p0 = (int)(rem % pages);
    const int g = blk / nrb, rb = blk % nrb;
    const int p1 = (int)min((long long)pages, p0 + (u1 - u));
    const int32_t* pt = t.pt + (size_t)b * t.max_pages;
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
        issue_page<BITS>(a, page, g, ring_s + (uint32_t)((next - p0) % NS) * F::STAGE, lane);
        ++next;
      }
      cp_commit();
    };
#pragma unroll 1
    for (int k = 0; k < NS - 1; ++k) issue();
    // ---- query fragments (the N side): row 8 n + r, channels 32 c + 8 j ..
    uint32_t qf[QP][NT][8][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = rb * RB + 8 * n + r;
      const uint4* q = reinterpret_cast<const uint4*>((const uint16_t*)a.w.q +
                                                      ((size_t)(sq.off + row / GQ) * v.H + g * GQ + row % GQ) * 128);
#pragma unroll
      for (int part = 0; part < QP; ++part) {
        const size_t o = (size_t)part * t.n_nodes * v.H * 16;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = row < R ? q[o + 4 * c + j] : make_uint4(0, 0, 0, 0);
          qf[part][n][2 * c][0] = x.x;
          qf[part][n][2 * c][1] = x.y;
          qf[part][n][2 * c + 1][0] = x.z;
          qf[part][n][2 * c + 1][1] = x.w;
        }
      }
    }
    // a group's accumulator starts at minus the part of the sum that the codes' offset makes (rows 8 n + 2 j, + 1)
    float bias[NT][4][2];
    if constexpr (BITS != 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[0][n][2 * c + k][e]));
              // 4-bit: the second register of a step (high nibbles) meets 1024 + 16 u
              s -= (f.x + f.y) * (BITS == 8 || e == 1 ? 1152.f : 1032.f);
            }
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          bias[n][c][0] = __shfl_sync(0xffffffffu, s, 8 * j);
          bias[n][c][1] = __shfl_sync(0xffffffffu, s, 8 * j + 4);
        }
    }
    // columns: query rows 2 j, + 1.  Rows r, r + 8 of an m-tile are channels: of 2 c + i, 32 c + 4 r + 2 i and + 1 (bf16); of 4 c + i,
    // 64 c + 8 r + 2 i and + 1 (8 bits); of i, 16 r + 2 i and + 1 (4 bits)
    float Y[NT][8][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) Y[n][k][e] = 0.f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -1e30f;
      l[n][0] = l[n][1] = 0.f;
    }
    int slot = 0;
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
      cp_wait<NS - 2>();
      __syncwarp();   // this page's bytes from every lane; every lane is done with the stage that is filled next
      issue();
      const uint8_t* st = ring + slot * F::STAGE;
      slot = slot + 1 == NS ? 0 : slot + 1;
      // ---- scores of 16 tokens: S[n] rows r, r + 8 = tokens, columns = query rows 8 n + 2 j, + 1
      float S[NT][4];
      if constexpr (BITS == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][e] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + r * 256 + (((4 * c + j) ^ swz(r)) << 4));
          const uint4 y = *reinterpret_cast<const uint4*>(st + (r + 8) * 256 + (((4 * c + j) ^ swz(r + 8)) << 4));
          const uint32_t k0[4] = {x.x, y.x, x.y, y.y}, k1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
          for (int part = 0; part < QP; ++part)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_b(S[n], k0, qf[part][n][2 * c][0], qf[part][n][2 * c][1], S[n]);
              mma_b(S[n], k1, qf[part][n][2 * c + 1][0], qf[part][n][2 * c + 1][1], S[n]);
            }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float s0 = __half2float(*reinterpret_cast<const __half*>(st + c * 32 + r * 2));
          const float s1 = __half2float(*reinterpret_cast<const __half*>(st + c * 32 + 16 + r * 2));
          uint32_t k0[4], k1[4];
          if constexpr (BITS == 8) {
            constexpr uint32_t ex = 0x64646464u;
            const uint2 x = *reinterpret_cast<const uint2*>(st + 128 + c * 512 + r * 32 + j * 8);
            const uint2 y = *reinterpret_cast<const uint2*>(st + 128 + c * 512 + 256 + r * 32 + j * 8);
            k0[0] = __byte_perm(x.x, ex, 0x4140);
            k0[1] = __byte_perm(y.x, ex, 0x4140);
            k0[2] = __byte_perm(x.x, ex, 0x4342);
            k0[3] = __byte_perm(y.x, ex, 0x4342);
            k1[0] = __byte_perm(x.y, ex, 0x4140);
            k1[1] = __byte_perm(y.y, ex, 0x4140);
            k1[2] = __byte_perm(x.y, ex, 0x4342);
            k1[3] = __byte_perm(y.y, ex, 0x4342);
          } else {
            constexpr uint32_t lm = 0x000F000Fu, hm = 0x00F000F0u, ex = 0x64006400u;
            const uint32_t x = *reinterpret_cast<const uint32_t*>(st + 128 + c * 256 + r * 16 + j * 4);
            const uint32_t y = *reinterpret_cast<const uint32_t*>(st + 128 + c * 256 + 128 + r * 16 + j * 4);
            k0[0] = (x & lm) | ex;
            k0[1] = (y & lm) | ex;
            k0[2] = (x & hm) | ex;
            k0[3] = (y & hm) | ex;
            k1[0] = ((x >> 8) & lm) | ex;
            k1[1] = ((y >> 8) & lm) | ex;
            k1[2] = ((x >> 8) & hm) | ex;
            k1[3] = ((y >> 8) & hm) | ex;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float start[4] = {bias[n][c][0], bias[n][c][1], bias[n][c][0], bias[n][c][1]};
            float acc[4];
            mma_h(acc, k0, qf[0][n][2 * c][0], qf[0][n][2 * c][1], start);
            mma_h(acc, k1, qf[0][n][2 * c + 1][0], qf[0][n][2 * c + 1][1], acc);
            if (c == 0) {
              S[n][0] = s0 * acc[0];
              S[n][1] = s0 * acc[1];
              S[n][2] = s1 * acc[2];
              S[n][3] = s1 * acc[3];
            } else {
              S[n][0] += s0 * acc[0];
              S[n][1] += s0 * acc[1];
              S[n][2] += s1 * acc[2];
              S[n][3] += s1 * acc[3];
            }
          }
        }
      }
      const bool tail = p * kPage + kPage > sq.hist;   // the page holds drafted nodes or unused slots
      if (tail) {
#pragma unroll 1
        for (int x = 0; x < 2 * NT; ++x) {   // query row 8 (x / 2) + 2 j + x % 2, tokens r and r + 8
          const int row = rb * RB + 8 * (x >> 1) + 2 * j + (x & 1), node = row / GQ;
          const int k0 = p * kPage + r - sq.hist, k1 = k0 + 8;   // nodes of the slots (negative: history)
          bool v0 = k0 < 0, v1 = k1 < 0;
          if (row < R) {
            if (k0 >= 0 && k0 < sq.cnt) v0 = tree_sees(t.mask, t.mask_words, sq.off + node, node, k0);
            if (k1 >= 0 && k1 < sq.cnt) v1 = tree_sees(t.mask, t.mask_words, sq.off + node, node, k1);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (x == 2 * n + e) {
                if (!v0) S[n][e] = -INFINITY;
                if (!v1) S[n][2 + e] = -INFINITY;
              }
        }
      }
      // ---- running maximum
      bool up = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        up = up || fmaxf(S[n][0], S[n][2]) > m[n][0] + 7.f || fmaxf(S[n][1], S[n][3]) > m[n][1] + 7.f;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = fmaxf(S[n][e], S[n][2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            const float mn = fmaxf(m[n][e], y - 3.f), f = ex2(m[n][e] - mn);
            m[n][e] = mn;
            l[n][e] *= f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              Y[n][k][e] *= f;
              Y[n][k][2 + e] *= f;
            }
          }
      }
      // ---- P (tokens r, r + 8 by query rows 2 j, + 1), transposed into the operand of the values: tokens 2 j .., row r
      uint32_t pb[NT][QP][2];   // bf16: a high and a low part, like the queries
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float e0 = ex2(S[n][0] - m[n][0]), e1 = ex2(S[n][1] - m[n][1]);
        const float e2 = ex2(S[n][2] - m[n][0]), e3 = ex2(S[n][3] - m[n][1]);
        if constexpr (BITS == 0) {
          const uint32_t x = b2(e0, e1), y = b2(e2, e3);
          auto lo16 = [](uint32_t z) { return __uint_as_float(z << 16); };
          auto hi16 = [](uint32_t z) { return __uint_as_float(z & 0xFFFF0000u); };
          pb[n][0][0] = transpose8(x);
          pb[n][0][1] = transpose8(y);
          pb[n][1][0] = transpose8(b2(e0 - lo16(x), e1 - hi16(x)));
          pb[n][1][1] = transpose8(b2(e2 - lo16(y), e3 - hi16(y)));
        } else {
          pb[n][0][0] = transpose8(h2(e0, e1));
          pb[n][0][1] = transpose8(h2(e2, e3));
        }
        l[n][0] += e0 + e2;
        l[n][1] += e1 + e3;
      }
      // ---- values: tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9, channels 32 c + 4 r .. + 3
      if constexpr (BITS == 0) {
        const uint8_t* sv = st + F::KB;
        unsigned bad = 0;   // bit t: token t holds an infinity or a NaN (among this lane's bytes)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint2 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int vt = 2 * j + (i & 1) + 8 * (i >> 1);
            x[i] = *reinterpret_cast<const uint2*>(sv + vt * 256 + (((4 * c + (r >> 1)) ^ swz(vt)) << 4) + (r & 1) * 8);
            if (tail) {
              // a slot that some rows do not see must not reach them through 0 * NaN: it enters as zero, and the rows
              // that do see it become NaN below
              auto odd = [](uint32_t y) { return (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u; };
              if (odd(x[i].x) || odd(x[i].y)) {
                bad |= 1u << vt;
                x[i] = make_uint2(0u, 0u);
              }
            }
          }
          const uint32_t v0[4] = {__byte_perm(x[0].x, x[1].x, 0x5410), __byte_perm(x[0].x, x[1].x, 0x7632),
                                  __byte_perm(x[2].x, x[3].x, 0x5410), __byte_perm(x[2].x, x[3].x, 0x7632)};
          const uint32_t v1[4] = {__byte_perm(x[0].y, x[1].y, 0x5410), __byte_perm(x[0].y, x[1].y, 0x7632),
                                  __byte_perm(x[2].y, x[3].y, 0x5410), __byte_perm(x[2].y, x[3].y, 0x7632)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int part = 0; part < QP; ++part) {
              mma_b(Y[n][2 * c], v0, pb[n][part][0], pb[n][part][1], Y[n][2 * c]);
              mma_b(Y[n][2 * c + 1], v1, pb[n][part][0], pb[n][part][1], Y[n][2 * c + 1]);
            }
        }
        if (tail) {
          bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if ((bad >> r & 1u) && S[n][e] != -INFINITY) l[n][e] = NAN;
              if ((bad >> (r + 8) & 1u) && S[n][2 + e] != -INFINITY) l[n][e] = NAN;
            }
        }
      } else {
        const uint8_t* sv = st + F::KB;
        const uint8_t* cv = sv + F::VS;
        // A lane reads 8 bytes of a token: 8 channels of group 2 c + r / 4, or 16 of group r / 2.  Half of the lanes take the tokens
        // of a pair in the other order, so that the warp's reads do not meet in a bank.
        constexpr int LPG = BITS == 8 ? 4 : 2;   // lanes r to a group
        const int swap = BITS == 8 ? j >> 1 : (r >> 1) & 1;
#pragma unroll
        for (int c = 0; c < LPG / 2; ++c) {
          const int gr = 8 / LPG * c + r / LPG;
          uint32_t sc0 = *reinterpret_cast<const uint32_t*>(sv + gr * 32 + j * 4);        // scales of tokens 2 j, 2 j + 1
          uint32_t sc1 = *reinterpret_cast<const uint32_t*>(sv + gr * 32 + 16 + j * 4);   // and 8 on
          if (tail) {
            // unused slots may hold any bytes: no scale that is not a number meets a weight of zero
            const int n0 = len - p * kPage - 2 * j, n1 = n0 - 8;   // tokens of the pair on
            sc0 = n0 >= 2 ? sc0 : n0 == 1 ? sc0 & 0xFFFFu : 0u;
            sc1 = n1 >= 2 ? sc1 : n1 == 1 ? sc1 & 0xFFFFu : 0u;
          }
          uint2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint2*>(cv + gr * (64 * BITS) + (2 * j + ((i & 1) ^ swap) + 8 * (i >> 1)) * (4 * BITS) +
                                                   r % LPG * 8);
#pragma unroll
          for (int h = 0; h < 16 / BITS; ++h) {   // four of the channels
            auto word = [&](int i) { return (BITS == 8 ? h : h >> 1) ? w[i].y : w[i].x; };
            uint32_t v0[4], v1[4];
            if constexpr (BITS == 8) {
              const uint32_t lo = swap ? 0x1504u : 0x5140u, hi = swap ? 0x3726u : 0x7362u;
              const uint32_t a01 = __byte_perm(word(0), word(1), lo), b01 = __byte_perm(word(0), word(1), hi);
              const uint32_t a23 = __byte_perm(word(2), word(3), lo), b23 = __byte_perm(word(2), word(3), hi);
              constexpr uint32_t off = 0x64806480u, ex = 0x64646464u;   // 1152, 1152
              v0[0] = hsub2(__byte_perm(a01, ex, 0x4140), off);
              v0[1] = hsub2(__byte_perm(a01, ex, 0x4342), off);
              v0[2] = hsub2(__byte_perm(a23, ex, 0x4140), off);
              v0[3] = hsub2(__byte_perm(a23, ex, 0x4342), off);
              v1[0] = hsub2(__byte_perm(b01, ex, 0x4140), off);
              v1[1] = hsub2(__byte_perm(b01, ex, 0x4342), off);
              v1[2] = hsub2(__byte_perm(b23, ex, 0x4140), off);
              v1[3] = hsub2(__byte_perm(b23, ex, 0x4342), off);
            } else {
              const uint32_t sel = h & 1 ? (swap ? 0x3276u : 0x7632u) : (swap ? 0x1054u : 0x5410u);
              const uint32_t w01 = __byte_perm(word(0), word(1), sel), w23 = __byte_perm(word(2), word(3), sel);
              const uint32_t h01 = w01 >> 8, h23 = w23 >> 8;
              constexpr uint32_t lm = 0x000F000Fu, hm = 0x00F000F0u, ex = 0x64006400u;
              constexpr uint32_t off = 0x64086408u;                       // 1032
              constexpr uint32_t s16 = 0x2C002C00u, o16 = 0xD480D480u;    // 1/16, -72
              v0[0] = hsub2((w01 & lm) | ex, off);
              v0[1] = hfma2((w01 & hm) | ex, s16, o16);
              v0[2] = hsub2((w23 & lm) | ex, off);
              v0[3] = hfma2((w23 & hm) | ex, s16, o16);
              v1[0] = hsub2((h01 & lm) | ex, off);
              v1[1] = hfma2((h01 & hm) | ex, s16, o16);
              v1[2] = hsub2((h23 & lm) | ex, off);
              v1[3] = hfma2((h23 & hm) | ex, s16, o16);
            }
            // the codes times their tokens' scales (registers 0, 1: tokens 2 j, 2 j + 1; 2, 3: and 8 on)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v0[i] = hmul2(v0[i], i < 2 ? sc0 : sc1);
              v1[i] = hmul2(v1[i], i < 2 ? sc0 : sc1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_h(Y[n][4 * c + 2 * h], v0, pb[n][0][0], pb[n][0][1], Y[n][4 * c + 2 * h]);
              mma_h(Y[n][4 * c + 2 * h + 1], v1, pb[n][0][0], pb[n][0][1], Y[n][4 * c + 2 * h + 1]);
            }
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();
    // ---- the partial of this row block
    const long long part = a.w.item_off[b] + blk + w;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[n][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int q = 8 * n + 2 * j + e;
        if (r == 0) {
          a.w.pm[part * RB + q] = m[n][e];
          a.w.pl[part * RB + q] = s;
        }
        if (rb * RB + q < R) {
          float* y = a.w.pY + (part * RB + q) * 128 + (BITS == 0 ? 4 * r : BITS == 8 ? 8 * r : 16 * r);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float4*>(y + (BITS == 0 ? 32 * c : BITS == 8 ? 64 * (c >> 1) + 4 * (c & 1) : 4 * c)) =
                make_float4(Y[n][2 * c][e], Y[n][2 * c][2 + e], Y[n][2 * c + 1][e], Y[n][2 * c + 1][2 + e]);
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
//   warp 19       MMA issue: S(0), S(1), then O += P(k) V(k) and S(k + 2)
//   warps 8 - 15  softmax, one row per thread: four take the even tiles, four the odd ones, so that one set's
//                 exponentials run beside the other's loads and maxima.  The row's running maximum is handed from tile to
//                 tile through shared memory as soon as it is known; rows past the block's are skipped by the warp.  P
//                 overwrites S in TMEM; O is rescaled when the maximum grew by more than 2^8.
// Measured: 64 trees of 24 over 8K, 4 bits, 32 heads on 8 KV heads in 354 us (blocks of 16 rows in k_tree_mma's way: 1,213 us).  About
// 1,800 issue slots a scheduler and tile, 55 % of the cycles; the products alone would take 1,300 cycles a tile.  The softmax warps read S
// twice, since 20 warps leave a thread 96 registers (over codes 124 bytes of spills as it is).
// TMEM: S in two 128-column buffers, O in 256 .. 383, Q in 384 .. 447.  Units of work: tiles, dealt to the CTAs as above.
// bf16 caches: K and V are operands as they lie, so warps 0 - 7 copy them straight into three stages of tiles.  Q and P enter as
// a high and a low bf16 part (one rounding of P to bf16 would show in the output), in TMEM columns 384 .. 511 and in place, 16
// columns of each part per 32 tokens: twice the products, some 2,600 of 3,800 cycles a tile.  16 sequences of 4K, 64 rows on each
// of 8 KV heads: 95 us (k_tree_mma: 156); 24 of 10000, 512 rows on 4: 441 (1,589).  The scores of the next block during a block's
// output (its Q asked for early) spilt registers and took 7 % longer.
constexpr int kTcDeq = 8, kTcSoft = 8;
constexpr int kTcMma = 19;             // (the scheduler of lane quarter 3, whose rows are used least; warps 16 - 18 only wait)
constexpr int kTcThreads = 32 * (kTcMma + 1);
constexpr int kTcTile = 32768, kTcAtom = 16384;

template <int BITS>
struct TcFmt {
  static constexpr int KB = PageFmt<BITS>::KB, VS = PageFmt<BITS>::VS;
  static constexpr int ST = BITS == 0 ? 3 : 2;                                   // stages of K and V tiles
  static constexpr int RAW = BITS == 0 ? 0 : 8 * PageFmt<BITS>::STAGE;           // 34816 or 18432 bytes: the pages of a tile
  static constexpr int RS = BITS == 8 ? 2 : 4;                                   // tiles of codes in flight
  static constexpr size_t SMEM = 2 * ST * (size_t)kTcTile + (size_t)RS * RAW + 1024;
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
  uint32_t o[4];
  if constexpr (BITS == 8) {
    constexpr uint32_t off = 0x64806480u, ex = 0x64646464u;
    o[0] = hmul2(hsub2(__byte_perm(w.x, ex, 0x4140), off), s2);
    o[1] = hmul2(hsub2(__byte_perm(w.x, ex, 0x4342), off), s2);
    o[2] = hmul2(hsub2(__byte_perm(w.y, ex, 0x4140), off), s2);
    o[3] = hmul2(hsub2(__byte_perm(w.y, ex, 0x4342), off), s2);
  } else {
    const uint32_t x = w.x, x8 = w.x >> 8;
    constexpr uint32_t lm = 0x000F000Fu, hm = 0x00F000F0u, ex = 0x64006400u, off = 0x64086408u;
    constexpr uint32_t s16 = 0x2C002C00u, o16 = 0xD480D480u;
    o[0] = hmul2(hsub2((x & lm) | ex, off), s2);
    o[1] = hmul2(hfma2((x & hm) | ex, s16, o16), s2);
    o[2] = hmul2(hsub2((x8 & lm) | ex, off), s2);
    o[3] = hmul2(hfma2((x8 & hm) | ex, s16, o16), s2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int BITS>
__global__ void __launch_bounds__(kTcThreads, 1) k_tree_tc(TreeMma a) {
  using F = TcFmt<BITS>;
  extern __shared__ uint8_t smem_raw[];
  constexpr int ST = F::ST;
  __shared__ __align__(8) uint64_t k_full[ST], k_empty[ST], v_full[ST], v_empty[ST], s_full[2], p_full[2], o_done[2], q_full,
      o_free, fin;
  __shared__ uint16_t bad[ST][8];   // bf16: per page of a tile with drafted nodes, the tokens whose values are not finite
  __shared__ uint32_t tmem_base;
  __shared__ volatile int abort_flag;
  __shared__ float xch[2][kTcRows], xl[2][kTcRows];   // by tile parity: row maxima handed on, and sums
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* K_s = smem;
  uint8_t* V_s = smem + ST * kTcTile;
  uint8_t* R_s = smem + 2 * ST * kTcTile;   // codes
  const ServeView& v = a.v;
  const TreeArgs& t = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tc::grid_wait_prev();
  const long long U = a.w.unit_off[t.batch];
  const long long We = workers_used(a, U);
  const int w = blockIdx.x;
  if (w >= We || U == 0) return;
  TcWalk wk;
  wk.u = (long long)w * U / We;
  wk.u1 = (long long)(w + 1) * U / We;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&k_full[s], kTcDeq);
      tc::mbar_init(&k_empty[s], 1);
      tc::mbar_init(&v_full[s], kTcDeq);
      tc::mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
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
  if (warp == kTcMma) tc::tmem_alloc(&tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_base;
  constexpr uint32_t o_col = 256, q_col = 384;
  // Only now: a block of the output product that took TMEM of this SM first would keep it until the merge is done, and the
  // merge waits for this kernel.
  tc::grid_launch_next();

  if (warp == kTcMma) {
    // ------------------------------------------------ MMA issue
    const uint32_t idesc_s = tc::idesc_f16(128, 128, BITS == 0, false, false);
    const uint32_t idesc_o = tc::idesc_f16(128, 128, BITS == 0, false, true);   // V: tokens are the contraction
    constexpr int QP = BITS == 0 ? 2 : 1;   // bf16: Q and P as a high and a low part
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
      const int s = j & 1, st = j % ST;
      if (!tc::mbar_wait_ab(&k_full[st], ((uint32_t)(j / ST)) & 1u, v.status, &abort_flag)) return false;
      tc::tc_fence_after();
      // S buffer j & 1 is free: P(j - 2) V(j - 2), issued before, has read it by the time these run (a block's first two
      // tiles: the last block's products have completed, its softmax warps have said so by q_full)
      const uint32_t d = tmem + (uint32_t)(s * 128), b = k_lo + (uint32_t)(st * kTcTile >> 4);
#pragma unroll
      for (int part = 0; part < QP; ++part)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(leader, d, tmem + q_col + 64u * part + 8u * kk, b + (uint32_t)(kk >> 2) * (kTcAtom >> 4) + 2u * (kk & 3), k_hi,
                 idesc_s, (part | kk) ? 1u : 0u);
      commit(leader, &s_full[s]);
      commit(leader, &k_empty[st]);
      return true;
    };
    while (ok && tc_next(a, wk, w, lane)) {
      const int nt = __shfl_sync(0xffffffffu, wk.p1 - wk.p0, 0);
      ok = tc::mbar_wait_ab(&q_full, (uint32_t)n & 1u, v.status, &abort_flag);
      tc::tc_fence_after();
      ok = ok && issue_s(jg) && (nt == 1 || issue_s(jg + 1));
      for (int k = 0; ok && k < nt; ++k) {
        const int j = jg + k, s = j & 1, st = j % ST;
        if (k == 0 && !(ok = tc::mbar_wait_ab(&o_free, ((uint32_t)n & 1u) ^ 1u, v.status, &abort_flag))) break;
        if (!(ok = tc::mbar_wait_ab(&v_full[st], ((uint32_t)(j / ST)) & 1u, v.status, &abort_flag))) break;
        if (!(ok = tc::mbar_wait_ab(&p_full[s], ((uint32_t)(j >> 1)) & 1u, v.status, &abort_flag))) break;
        tc::tc_fence_after();
        const uint32_t p = tmem + (uint32_t)(s * 128), b = v_lo + (uint32_t)(st * kTcTile >> 4);
        // P: 8 columns per 16 tokens; in two parts, 16 columns of the high, then 16 of the low one, per 32 tokens
#pragma unroll
        for (int part = 0; part < QP; ++part)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(leader, tmem + o_col, p + (BITS == 0 ? 32u * (kk >> 1) + 8u * (kk & 1) + 16u * part : 8u * kk),
                   b + (uint32_t)(kk * 2048 >> 4), v_hi, idesc_o, (k | part | kk) ? 1u : 0u);
        commit(leader, &o_done[s]);
        commit(leader, &v_empty[st]);
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
  } else if (BITS == 0 && warp < kTcDeq) {
    // ------------------------------------------------ bf16: page `warp` of every tile, copied to its place in the tiles.  A tile
    // is handed over after the copies of the next one, of whichever block, have been asked for.  (That waits for a stage whose
    // products need no later tile than the one handed over last.)
    bool ok = true;
    int n = 0;
    const int row0 = warp * 16;
    auto at = [&](int e) { return (uint32_t)((e & 15) >> 3) * kTcAtom + tc::sw128((uint32_t)(row0 + (e >> 4)), (uint32_t)(e & 7)); };
    int tokens = kTcTok;   // of this page of tile n - 1, which is to be handed over; beyond 16: all, before the drafted nodes
    auto hand_over = [&]() {
      const int st = (n - 1) % ST;
      if (tokens < kTcTok) {
        // a slot that some rows do not see must not reach them through 0 * NaN: values that are not finite, and slots without
        // a token, enter as zero; the rows that see such a token become NaN in the softmax
        unsigned odd = 0;
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          const int e = x * 32 + lane;
          uint4* z = reinterpret_cast<uint4*>(V_s + (size_t)st * kTcTile + at(e));
          const uint4 u = *z;
          auto bad2 = [](uint32_t y) { return (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u; };
          const bool out = (e >> 4) >= tokens, nan = bad2(u.x) || bad2(u.y) || bad2(u.z) || bad2(u.w);
          if (out || nan) *z = make_uint4(0u, 0u, 0u, 0u);
          if (!out && nan) odd |= 1u << (e >> 4);
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
        if (lane == 0) bad[st][warp] = (uint16_t)odd;
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&k_full[st]);
        tc::mbar_arrive(&v_full[st]);
      }
    };
    while (ok && tc_next(a, wk, w, lane)) {
      const int32_t* pt = t.pt + (size_t)wk.b * t.max_pages;
      const int pages = (wk.len + kPage - 1) / kPage;
#pragma unroll 1
      for (int k = wk.p0; k < wk.p1 && ok; ++k) {
        const int st = n % ST, p = k * 8 + warp;
        const uint32_t ph = (((uint32_t)(n / ST)) & 1u) ^ 1u;
        const bool some = p < pages;   // past the sequence's pages the stage keeps what it held: those slots hold no token
        const int page = some ? pt[p] : 0;
        const bool live = some && page >= 0 && page < t.n_pages;
        if (some && !live && lane == 0) atomicOr(v.status, kBadPage);
        const uint8_t* base = t.pool + (size_t)(live ? page : 0) * v.page_bytes;
        const uint8_t* ks = base + (size_t)wk.g * F::KB;
        const uint8_t* vs = base + (size_t)v.Hkv * F::KB + (size_t)wk.g * 256;
        const uint32_t kd = tc::smem_u32(K_s + (size_t)st * kTcTile), vd = tc::smem_u32(V_s + (size_t)st * kTcTile);
        ok = __all_sync(0xffffffffu, tc::mbar_wait_ab(&k_empty[st], ph, v.status, &abort_flag));
        if (ok && some) {
#pragma unroll
          for (int x = 0; x < 8; ++x) cp16(kd + at(x * 32 + lane), ks + (x * 32 + lane) * 16, live);
        }
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_ab(&v_empty[st], ph, v.status, &abort_flag));
        if (ok && some) {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int e = x * 32 + lane;
            cp16(vd + at(e), vs + (size_t)(e >> 4) * v.Hkv * 256 + (e & 15) * 16, live);
          }
        }
        cp_commit();
        if (n > 0) {
          cp_wait<1>();
          hand_over();
        }
        ++n;
        tokens = (k + 1) * kTcTok > wk.sq.hist ? min(wk.len - (k * kTcTok + row0), 16) : kTcTok;
      }
    }
    cp_wait<0>();
    if (ok && n > 0) hand_over();
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
          uint4 code[2][BITS ? BITS / 4 : 1];
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
  } else if (warp < kTcDeq + kTcSoft) {
    // ------------------------------------------------ softmax and output
    const int qq = warp & 3, x = (warp - kTcDeq) >> 2;   // TMEM lane quarter; tiles of this parity
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
#pragma unroll 1
        for (int part = 0; part < (BITS == 0 ? 2 : 1); ++part) {
          uint32_t qv[32];
          const uint4* src = reinterpret_cast<const uint4*>(
              (const uint16_t*)a.w.q + (((size_t)part * t.n_nodes + wk.sq.off + node) * v.H + wk.g * v.group_q + row % v.group_q) * 128 + 64 * x);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 z = row < wk.R ? src[c] : make_uint4(0, 0, 0, 0);
            qv[4 * c] = z.x;
            qv[4 * c + 1] = z.y;
            qv[4 * c + 2] = z.z;
            qv[4 * c + 3] = z.w;
          }
          tmem_st32x(tmem + lane_base + q_col + 64u * part + 32u * x, qv);
        }
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
          bool odd = false;   // bf16: the row sees a value that is not finite
          if (tail) {   // what a row does not see becomes -infinity in TMEM
            // (long complete: the wait is for what the copying warps wrote to bad)
            if constexpr (BITS == 0) tc::mbar_wait_ab(&k_full[j % ST], ((uint32_t)(j / ST)) & 1u, v.status, &abort_flag);
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              float s[32];
              const uint32_t see = row < wk.R ? vis32(t, wk.sq.off + node, node, wk.sq.cnt, t0 + 32 * h - wk.sq.hist) : 0u;
              if constexpr (BITS == 0) odd = odd || (see & ((uint32_t)bad[j % ST][2 * h] | (uint32_t)bad[j % ST][2 * h + 1] << 16)) != 0u;
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
          // P over columns of S that have been read: 16 columns of pairs for 32 of scores (bf16: 16 and 16)
          unsigned long long l2[4] = {0ull, 0ull, 0ull, 0ull};   // packed pairs of sums
          const unsigned long long nm = pack2(-m_used, -m_used);
          auto put = [&](int h, const float* s) {   // piece h
#pragma unroll
            for (int c0 = 0; c0 < 32; c0 += 16) {
              uint32_t p2[8], q2[8];
#pragma unroll
              for (int c = c0; c < c0 + 16; c += 2) {
                const float2 d = unpack2(add2(pack2(s[c], s[c + 1]), nm));
                const float e0 = ex2(d.x), e1 = ex2(d.y);
                l2[(c >> 1) & 3] = add2(l2[(c >> 1) & 3], pack2(e0, e1));
                if constexpr (BITS == 0) {
                  const uint32_t z = b2(e0, e1);
                  p2[(c - c0) / 2] = z;
                  q2[(c - c0) / 2] = b2(e0 - __uint_as_float(z << 16), e1 - __uint_as_float(z & 0xFFFF0000u));
                } else {
                  p2[(c - c0) / 2] = h2(e0, e1);
                }
              }
              tc::tmem_st8(s_at + (BITS == 0 ? 32u : 16u) * h + c0 / 2, p2);
              if constexpr (BITS == 0) tc::tmem_st8(s_at + 32u * h + 16u + c0 / 2, q2);
            }
          };
          tmem_wait32(s0);
          tmem_ld32x(s_at + 32u, s1);
          put(0, s0);
          tmem_wait32(s1);
          tmem_ld32x(s_at + 64u, s0);
          put(1, s1);
          tmem_wait32(s0);
          tmem_ld32x(s_at + 96u, s1);
          put(2, s0);
          tmem_wait32(s1);
          put(3, s1);
          const float2 ls = unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
          l += ls.x + ls.y;
          if (BITS == 0 && odd) l = NAN;
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
  if (warp == kTcMma) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merging the partials
// One warp per output row and HPW query heads of it, lane: four channels; the first partials of all its heads are asked for
// together.  Writes y as fp16 into the output product's B tiles; rows of no sequence and the tiles' padding rows are zero.
template <int HPW>
__global__ void __launch_bounds__(256, HPW == 1 ? 6 : 4) k_tree_combine(TreeMma a, int rows_pad, int NB, int KT) {
  const ServeView& v = a.v;
  const TreeArgs& t = a.t;
  const int lane = threadIdx.x & 31;
  const long long id = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int parts = (v.H + HPW - 1) / HPW;
  if (id >= (long long)rows_pad * parts) return;
  const int row = (int)(id / parts), h0 = (int)(id % parts) * HPW;
  // (what the query kernel wrote is complete: the attention kernel lets this one start only after its own wait for it)
  tc::grid_launch_next();
  const int b = row < t.n_nodes ? a.w.row_b[row] : -1;
  TreeSeq sq{0, 0, 0, 0};
  if (b >= 0) sq = seq_of(t, b, v.status, false);
  const bool live = sq.cnt > 0 && row >= sq.off && row - sq.off < sq.cnt && a.w.item_off[b + 1] > a.w.item_off[b];
  const int nrb = (sq.cnt * v.group_q + a.rb - 1) / a.rb, units = (sq.hist + sq.cnt + a.unit - 1) / a.unit;
  const long long U = a.w.unit_off[t.batch], We = workers_used(a, U);
  const long long u0 = live ? a.w.unit_off[b] : 0, i0 = live ? a.w.item_off[b] : 0;
  const bool small = U * We < (1ll << 32);
  long long at[HPW];   // the head's first partial
  int n[HPW];          // and how many
#pragma unroll
  for (int i = 0; i < HPW; ++i) {
    at[i] = n[i] = 0;
    const int h = h0 + i;
    if (!live || h >= v.H) continue;
    const int g = h / v.group_q, rr = (row - sq.off) * v.group_q + h % v.group_q;
    const int blk = g * nrb + rr / a.rb;
    const long long lo = u0 + (long long)blk * units, hi = lo + units - 1;
    // the warps of the first and the last unit (divisions in 32 bits where they fit: a quarter of the instructions)
    long long w0, w1;
    if (small) {
      w0 = ((uint32_t)(lo + 1) * (uint32_t)We - 1u) / (uint32_t)U;
      w1 = ((uint32_t)(hi + 1) * (uint32_t)We - 1u) / (uint32_t)U;
    } else {
      w0 = ((lo + 1) * We - 1) / U;
      w1 = ((hi + 1) * We - 1) / U;
    }
    at[i] = (i0 + blk + w0) * a.rb + rr % a.rb;
    n[i] = (int)(w1 - w0) + 1;
  }
  tc::grid_wait_prev();
  float m[HPW], l[HPW];
  float4 y[HPW];
#pragma unroll
  for (int i = 0; i < HPW; ++i) {
    m[i] = n[i] ? a.w.pm[at[i]] : 0.f;
    l[i] = n[i] ? a.w.pl[at[i]] : 0.f;
    y[i] = n[i] ? *reinterpret_cast<const float4*>(a.w.pY + at[i] * 128 + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < HPW; ++i) {
    const int h = h0 + i;
    if (h >= v.H) break;
#pragma unroll 4
    for (int k = 1; k < n[i]; ++k) {
      const long long p = at[i] + (long long)k * a.rb;
      const float4 x = *reinterpret_cast<const float4*>(a.w.pY + p * 128 + lane * 4);
      const float mk = a.w.pm[p], lk = a.w.pl[p];
      const float mn = fmaxf(m[i], mk), f0 = ex2(m[i] - mn), f = ex2(mk - mn);
      m[i] = mn;
      l[i] = l[i] * f0 + lk * f;
      y[i] = make_float4(y[i].x * f0 + x.x * f, y[i].y * f0 + x.y * f, y[i].z * f0 + x.z * f, y[i].w * f0 + x.w * f);
    }
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];   // a row that sees nothing: zero; NaN stays
    const uint32_t k = (uint32_t)(h * 128 + lane * 4), c = k & 63u;
    uint8_t* tile = (uint8_t*)a.w.y + ((size_t)(row / NB) * KT + (k >> 6)) * (size_t)NB * 128;
    *reinterpret_cast<uint2*>(tile + tc::sw128((uint32_t)(row % NB), c >> 3) + (c & 7u) * 2u) =
        make_uint2(h2(y[i].x * inv, y[i].y * inv), h2(y[i].z * inv, y[i].w * inv));
  }
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

template <int BITS, int NT>
int mma_workers() { return MmaFmt<BITS, NT>::CTAS * kTreeWarps * num_sms(); }

struct TreePlan {
  size_t parts;          // partials
  size_t unit_off, item_off, q, row_b, pm, pl, pY, y, part, total;
  int NB, rows_pad;
  bool tc;               // k_tree_tc
  bool full;             // output product by 128 x 128 tiles, not stream-K
  int workers, rb, nt;   // nt: 8-row tiles of a row block of k_tree_mma
};

// Rows per sequence and KV head from which the 128-row kernel is taken.  16 sequences of 4K: 24 rows, 8 bits, 8 KV heads 72 us by
// k_tree_mma, 73 by k_tree_tc, 32 KV heads 188 and 225; 28 rows 82 and 74; 32 rows, 32 KV heads 244 and 219.
// bf16: 20 rows 85 and 85, 32 KV heads 282 and 267; 24 rows 95 and 84, 297 and 264; 28 rows 97 and 85; 64 rows 153 and 92; but 64
// short sequences of 500 tokens 86 and 115 at 20 rows, 93 and 117 at 28, 137 and 132 at 64 (8 bits, 28 rows, by k_tree_tc: 104).
// Lengths are known on the device only, so one number serves both.
constexpr int kTcFrom = 25;

size_t part_bytes(size_t parts, int rb) { return 2 * al256(parts * rb * 4) + al256(parts * rb * 512); }

TreePlan tree_plan(const starkv_layer* L, int batch, int n_nodes, int max_nodes) {
  const ServeView& v = L->view;
  TreePlan p;
  // Up to 256 rows the output product reads W_o once in an even split over the SMs; beyond, 128 x 128 tiles fill them (a whole call
  // over a short cache: 242 rows 41 us against 54, 400 rows 68 against 66, 820 rows 131 against 90).
  p.full = n_nodes > 256;
  p.NB = p.full ? 128 : outproj_nb(n_nodes);
  p.rows_pad = (n_nodes + p.NB - 1) / p.NB * p.NB;
  // row blocks, one more per sequence for what its last block leaves empty
  p.tc = max_nodes * v.group_q >= kTcFrom;
  // the fewest 8-row tiles that hold the rows, up to three (registers; bf16: two, and as many blocks as it takes)
  const int rows = max_nodes * v.group_q;
  p.nt = rows <= 8 ? 1 : rows <= 16 || v.kv_bits == 0 ? 2 : 3;
  p.workers = p.tc ? num_sms()
              : v.kv_bits == 0 ? mma_workers<0, 1>()
              : p.nt == 1 ? mma_workers<8, 1>() : p.nt == 2 ? mma_workers<8, 2>() : mma_workers<8, 3>();
  p.rb = p.tc ? kTcRows : 8 * p.nt;
  const size_t items = (size_t)v.Hkv * std::min((size_t)batch * ((max_nodes * v.group_q + p.rb - 1) / p.rb),
                                                (size_t)batch + (size_t)n_nodes * v.group_q / p.rb);
  const size_t parts = p.parts = items + p.workers;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += al256(bytes);
    return at;
  };
  p.unit_off = take(8 * ((size_t)batch + 1));
  p.item_off = take(8 * ((size_t)batch + 1));
  p.q = take((size_t)n_nodes * v.H * 256 * (v.kv_bits == 0 ? 2 : 1));
  p.row_b = take(4 * (size_t)n_nodes);
  p.pm = take(parts * p.rb * 4);
  p.pl = take(parts * p.rb * 4);
  p.pY = take(parts * p.rb * 512);
  p.y = take((size_t)p.rows_pad / p.NB * (L->Kp / 64) * p.NB * 128);
  p.part = take(p.full ? 0 : outproj_part_bytes(L, n_nodes));
  p.total = o;
  return p;
}

template <int BITS, int NT>
cudaError_t launch_mma(const TreeMma& a, cudaStream_t s) {
  const size_t smem = (size_t)kTreeWarps * MmaFmt<BITS, NT>::NS * PageFmt<BITS>::STAGE;
  const cudaError_t e = set_smem_limit((const void*)k_tree_mma<BITS, NT>, smem);
  if (e != cudaSuccess) return e;
  return launch_k(k_tree_mma<BITS, NT>, a.workers / kTreeWarps, 32 * kTreeWarps, smem, s, true, a);
}

template <int BITS>
cudaError_t launch_bits(const starkv_layer* L, TreeMma& a, const TreePlan& p, cudaStream_t s) {
  const ServeView& v = L->view;
  cudaError_t e;
  const dim3 pgrid(a.t.n_nodes + 1, (v.H + kTreeWarps - 1) / kTreeWarps);
  if constexpr (BITS == 4) {
    e = launch_k(p.tc ? k_tree_prep<BITS, 2> : k_tree_prep<BITS, 1>, pgrid, 32 * kTreeWarps, 0, s, true, a);
  } else {
    e = launch_k(k_tree_prep<BITS, 0>, pgrid, 32 * kTreeWarps, 0, s, true, a);
  }
  if (e != cudaSuccess) return e;
  if (p.tc) {
    if ((e = set_smem_limit((const void*)k_tree_tc<BITS>, TcFmt<BITS>::SMEM)) != cudaSuccess) return e;
    return launch_k(k_tree_tc<BITS>, a.workers, kTcThreads, TcFmt<BITS>::SMEM, s, true, a);
  }
  if (p.nt == 1) return launch_mma<BITS, 1>(a, s);
  if constexpr (BITS != 0)
    if (p.nt == 3) return launch_mma<BITS, 3>(a, s);
  return launch_mma<BITS, 2>(a, s);
}

}  // namespace

bool tree_mma_supported(const LayerView& v) { return v.plain && v.dtype == STARKV_BF16 && v.d == 128; }

size_t tree_mma_need(const starkv_layer* L, int batch, int n_nodes, int max_nodes) {
  return tree_plan(L, batch, n_nodes, max_nodes).total;
}

size_t tree_mma_ws_bytes(const starkv_layer* L, int batch, int n_nodes, int max_nodes) {
  const ServeView& v = L->view;
  const TreePlan p = tree_plan(L, batch, n_nodes, max_nodes);
  const size_t own = part_bytes(p.parts, p.rb);
  // Trees of fewer nodes may take blocks of other rows, with more partials in all; each kind of block needs the most with the
  // most nodes that take it.  The other buffers grow with the batch and the nodes, but for the output product's partial
  // sums, which only calls of up to 256 nodes have.
  size_t most = own;
  for (const int rows : {8, 16, kTcFrom - 1}) {
    const int m = std::min(max_nodes, rows / v.group_q);
    if (m < 1) continue;
    const TreePlan q = tree_plan(L, batch, n_nodes, m);
    most = std::max(most, part_bytes(q.parts, q.rb));
  }
  const size_t sums = p.full ? al256(outproj_part_bytes(L, 256)) : 0;
  return p.total - own + most + sums;
}

cudaError_t launch_tree_mma(const starkv_layer* L, const TreeArgs& t, void* ws, size_t ws_bytes, cudaStream_t s) {
  const ServeView& v = L->view;
  const TreePlan p = tree_plan(L, t.batch, t.n_nodes, t.max_nodes);
  if (ws_bytes < p.total) return cudaErrorInvalidValue;
  uint8_t* w = (uint8_t*)ws;
  TreeMma a;
  a.v = v;
  a.t = t;
  a.w.unit_off = (long long*)(w + p.unit_off);
  a.w.item_off = (long long*)(w + p.item_off);
  a.w.q = w + p.q;
  a.w.row_b = (int*)(w + p.row_b);
  a.w.pm = (float*)(w + p.pm);
  a.w.pl = (float*)(w + p.pl);
  a.w.pY = (float*)(w + p.pY);
  a.w.y = w + p.y;
  a.w.part = w + p.part;
  a.workers = p.workers;
  a.rb = p.rb;
  a.unit = p.tc ? kTcTok : kPage;
  a.min_units = p.tc ? 1 : kMinUnits;
  a.run_scale = p.tc ? 0.f : 0.25f;   // (a tile of k_tree_tc costs as much as merging a dozen partials)
  cudaError_t e = v.kv_bits == 8 ? launch_bits<8>(L, a, p, s) : v.kv_bits == 4 ? launch_bits<4>(L, a, p, s)
                                                                               : launch_bits<0>(L, a, p, s);
  if (e != cudaSuccess) return e;
  // A warp per head while that fills the SMs at most twice; else a row's heads share their row's lookups.  A warp per head / per four, a
  // whole call with 32 heads over 31 tokens, us: 16 rows 16.4 / 17.1, 128 30.5 / 33.0, 512 74.6 / 76.5, 592 79.7 / 77.6, 1024 116 / 113; over
  // 500 tokens 16 rows 24.7 / 37.6, 512 146 / 144.
  const bool few = (long long)p.rows_pad * v.H <= 128LL * num_sms();
  const long long warps = (long long)p.rows_pad * (few ? v.H : (v.H + 3) / 4);
  e = launch_k(few ? k_tree_combine<1> : k_tree_combine<4>, (unsigned)((warps * 32 + 255) / 256), 256, 0, s, true, a, p.rows_pad,
               p.NB, L->Kp / 64);
  if (e != cudaSuccess) return e;
  const int32_t* n_rows = t.lens ? nullptr : t.node_off + t.batch;
  if (t.n_nodes <= kOutSmallRows) return launch_out_small(L, a.w.y, t.n_nodes, t.out, n_rows, s);
  if (p.full) return launch_out_full(L, a.w.y, t.n_nodes, t.out, n_rows, s, true);
  return launch_outproj_tc(L, a.w.y, t.n_nodes, t.out, (float*)a.w.part, s, n_rows, true);
}

}  // namespace starkv
