// Tensor-core attention over the paged cache for many query rows: prompt chunks, and calls
// with more rows to a request than the decode kernel takes (bf16 queries, head_dim 64 or 128).
//
// A unit is a (request, KV head) and up to 256 query rows (tokens x heads of the group, two
// tiles A and B of 128), which share every K and V they read.  Per 128 cached tokens:
//   S = Q K^T        two pieces of Q (E4M3, the remainder E5M2) as one contraction of 2 D,
//                    K as it is stored (E4M3)
//   t = S kscale c_r + log2 vscale,  m_r: the t of some token that the row has seen
//   x = 2^(t - m_r) rounded to bf16,  l_r += x / vscale,  O += X V      bf16 x bf16
// and o = O / l.  The scales are powers of two, so V's rides in x's exponent and V's codes
// are exact in bf16.  x is rounded to 8 bits as the output is, and l sums the rounded x, so that a
// row of one strong token has no error from it (with l of the exact x the whole error was up to
// 1.43 times that of rounding the output alone, so 1.19, in the same time).  bf16 has
// float32's exponents, so m need not follow the maximum: it moves, and O is rescaled, only where x would pass
// 2^63 or l leave float32.  With x in f16, whose 2^16 strong tokens passed in four of ten tiles of
// the 8192-token prompt, the exponentials taken again and O rescaled cost it a fifth.
// Queries: a bf16 element has 8 significant bits, its first piece 4, and the remainder then at most 3, which E5M2
// holds down to steps of 2^-16: exact down to 2^-13 of the row's largest element, off by 2^-21 of the largest at most
// below that.  (With E4M3 for both pieces, whose steps end at 2^-9, it was 2^-10 and 2^-17.)
//
// How: work is cut as in the decode kernel: the 128-token tiles of all units laid end to
// end and split evenly over one CTA per SM, partials of split units added by a join
// kernel.  That also balances causal rows, whose units differ in length, and feeds all
// SMs when rows are few and the context is long.  A unit's start counts as three tiles (with two
// the CTA of the 8192-token prompt's shortest units ends last, 12 % later; four are 1 % slower).
// A split kernel first writes the queries' pieces in operand layout (a few percent of the
// time; two warps of each CTA that did it took 15 to 27 thousand clocks a unit).
// Per CTA: one warp copies K pages into a ring, one the queries, four convert V's codes to
// bf16 operand rows (a page's rows are its operand rows, so it is load, convert, store), one
// issues the matrix instructions, and two groups of four warps do the softmax of A and B, a
// thread to a row, so that no row statistic crosses threads.  The matrix warp works on
// one tile while the other's softmax runs: O(A) += X(A, j) V and S(A, j+1) while B's
// exponentials are computed, then the reverse.  X goes to TMEM, over S, as the product's
// first operand: from shared memory the two operands of both products, X's stores and V's
// would be 368 KB a step, 2900 clocks at 128 bytes, against the tensor core's 2048.
//
// Bound by the chain of one tile (exponentials, X's store, its product and the next S), which only
// the other tile's overlaps: 2950 clocks a step of 128 tokens, against 2048 of matrix work, 61 % of the
// tensor core's time.  Measured on 32/4 heads of 128: an 8192-token prompt 437 us (1.26 PFLOP/s,
// 66 % of the measured bf16 rate), five chunks of 100 to 2048 tokens behind up to 8192 314 us (1.20 PFLOP/s).
#include "paged_cut.h"
#include "paged_mma.cuh"

namespace kvs {
namespace {

using namespace pmma;

using cut::kSetup;
using cut::kTileBlocks;
using cut::Unit;
constexpr int kTile = kTileBlocks * kBlock;
static_assert(kTile == 128 && kBlock == cut::kTokens, "tiles");
constexpr int kThreads = 512;            // 8 softmax warps, K copies, matrix, query copies, a spare, 4 V warps
constexpr int kCopyWarp = 8, kMmaWarp = 9, kQWarp = 10, kVWarp = 12, kVThreads = 128;
// Registers of a softmax thread and of the others: 256 (168 + 88) = the block's 65536.
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;
constexpr int kKStages = 3, kVStages = 2, kQStages = 1;
constexpr int kSlots = 4;                // scales of this many tiles, row factors of this many segments
constexpr int kRows = 128;               // rows of a tile of queries
constexpr int kChunk = 512;              // requests of one round of the search
constexpr float kLog2e = 1.4426950408889634f;
// A row's reference moves where x would pass 2^kFarX or a part of l 2^kFarL.  What passes kLimit shows it: a tile's
// part of l, and a block's sum of x times kSumShare.  Sums of 2^26 tokens then stay within float32.
constexpr float kFarX = 63.f, kFarL = 99.f;
constexpr float kLimit = 0x1p107f, kSumShare = 0x1p39f;

// Units of request r: groups of `per` query tokens, all KV heads alike.
struct Req {
  int first, n, p0;      // first packed row; tokens handled (0: none); position of the first
};
__device__ __forceinline__ Req req_of(const PagedAttend& a, int r) {
  Req x;
  x.first = r;
  x.n = 1;
  int n = 1;
  if (a.row_start) {
    x.first = __ldg(a.row_start + r);
    n = __ldg(a.row_start + r + 1) - x.first;
    x.n = x.first < 0 ? 0 : min(min(n, a.max_q_len), a.total_q - x.first);
  }
  x.p0 = min(max(__ldg(a.kv_len + r), 0), a.table_stride * kBlock) - n;
  return x;
}
__device__ __forceinline__ Unit unit_of(const PagedAttend& a, const Req& x, int qg, int per) {
  return cut::unit_of(x.p0, x.n, a.window, qg, per);
}

struct Search {
  long long sums[32];
  long long total, before;
  long long tiles[kChunk];
  int r, qg, h, t;
};

// Cost of request r per KV head, by a warp: tiles and units' starts.
__device__ long long request_tiles(const PagedAttend& a, int r, int per) {
  const Req x = req_of(a, r);
  long long sum = cut::lane_cost(x.p0, x.n, a.window, per, threadIdx.x & 31, 32);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Total cost of the call, by a block of `warps` warps.
__device__ long long total_tiles(const PagedAttend& a, int per, int warps, Search& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long sum = 0;
  for (int r = warp; r < a.n_reqs; r += warps) {
    const long long t = request_tiles(a, r, per);
    if (lane == 0 && r < kChunk) s.tiles[r] = t;
    sum += t;
  }
  if (lane == 0) s.sums[warp] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < warps; ++w) sum += s.sums[w];
  return sum * a.d.Hkv;
}

// Where `target` of the call's cost is: s.r, s.qg, s.h, s.t (within the unit: its start, then
// its tiles), for all threads.  After total_tiles, which left the first kChunk requests' counts.
__device__ void locate(const PagedAttend& a, int per, int warps, long long target, Search& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hkv = a.d.Hkv;
  long long base = 0;
  for (int r0 = 0; r0 < a.n_reqs; r0 += kChunk) {
    const int m = min(kChunk, a.n_reqs - r0);
    if (r0 > 0) {
      __syncthreads();
      for (int i = warp; i < m; i += warps) {
        const long long t = request_tiles(a, r0 + i, per);
        if (lane == 0) s.tiles[i] = t;
      }
    }
    if (threadIdx.x == 0) s.r = -1;
    __syncthreads();
    if (warp == 0) {
      long long at = base;
      for (int i = 0; i < m; i += 32) {
        const long long mine = i + lane < m ? s.tiles[i + lane] * hkv : 0;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        upto += at;
        if (target >= upto - mine && target < upto) {
          s.r = r0 + i + lane;
          s.before = upto - mine;
        }
        at = __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) s.total = at;
    }
    __syncthreads();
    base = s.total;
    if (s.r >= 0) break;
  }
  if (warp == 0) {
    const Req x = req_of(a, s.r);
    long long at = s.before;
    for (int q0 = 0; q0 * per < x.n; q0 += 32) {
      const int qg = q0 + lane;
      const int tiles = qg * per < x.n ? unit_of(a, x, qg, per).cost() : 0;
      const long long mine = (long long)tiles * hkv;
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      upto += at;
      if (target >= upto - mine && target < upto) {
        const int off = (int)(target - (upto - mine));
        s.qg = qg;
        s.h = off / tiles;
        s.t = off % tiles;
      }
      at = __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  __syncthreads();
}

// A CTA's walk over its share of the cost, segment by segment (a segment: tiles of one unit).
// A share that ends within a unit's start leaves the unit to the next CTA.
struct Walk {
  int r, qg, h, v0, left, per, seg;        // v0: where the share enters the unit's cost; left: from there on
  int t0, nt;                              // the segment's tiles of the unit: [t0, t0 + nt); 0: no more
  int done;                                // tiles of the CTA before it
  Req q;
  Unit u;
  bool first, whole;
  __device__ void start(const PagedAttend& a, const Search& s, int cost, int per_) {
    r = s.r; qg = s.qg; h = s.h; v0 = s.t;
    left = cost;
    per = per_;
    first = true;
    seg = done = 0;
    q = req_of(a, r);
    u = unit_of(a, q, qg, per);
    clip();
  }
  __device__ void clip() {
    const int v1 = min(u.cost(), v0 + left);
    t0 = max(v0 - kSetup, 0);
    nt = max(v1 - kSetup - t0, 0);
    whole = nt == u.tiles;
  }
  __device__ void next(const PagedAttend& a) {
    left -= u.cost() - v0;
    done += nt;
    first = false;
    nt = 0;
    v0 = 0;
    ++seg;
    if (left <= 0) return;
    if (++h == a.d.Hkv) {
      h = 0;
      ++qg;
      while (qg * per >= q.n) {
        qg = 0;
        q = req_of(a, ++r);
      }
      u = unit_of(a, q, qg, per);
    }
    clip();
  }
};

struct Misc {
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], drain;
  uint64_t s_ready[2], p_ready[2], o_done[2];
  uint64_t q_ready[kSlots], q_empty[kQStages], sc_ready[kSlots];
  uint32_t tmem;
  alignas(16) float ks[kSlots][kTileBlocks], vs[kSlots][kTileBlocks];
  int bad[kSlots];                         // blocks of the tile that are not a page, as bits
  alignas(16) float qc[kSlots][2 * kRows]; // of each row: its query's scale, log2(e) / sqrt(D)
  Walk walk[8][2];                         // the softmax warps' segments, this one and the next (they would cost
                                           // the tile loop 20 registers)
};

template <int D>
struct Cfg {
  static constexpr int PAGE = 16 * D;
  static constexpr int Q = kRows * 2 * D;                 // one tile of queries, both pieces
  static constexpr int K = kTileBlocks * PAGE;            // a stage of K
  static constexpr int V = kTile * D * 2;                 // V as bf16
  static constexpr int BODY = kQStages * 2 * Q + kKStages * K + kVStages * V;
  static constexpr int SMEM = BODY + (int)sizeof(Misc) + 1024;
  static_assert(SMEM + (int)sizeof(Search) <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float scale_log2(float s) { return (float)((__float_as_int(s) >> 23) - 127); }
__device__ __forceinline__ float scale_inverse(float s) { return __int_as_float((254 << 23) - __float_as_int(s)); }
// The scales of a tile in registers: the operands' traffic starves shared-memory loads.
struct Scales {
  float ks[kTileBlocks], vs[kTileBlocks];
  __device__ __forceinline__ float ev(int b) const { return scale_log2(vs[b]); }
  __device__ __forceinline__ float iv(int b) const { return scale_inverse(vs[b]); }
};

// lo and hi plus the two elements of v.
__device__ __forceinline__ void add_bf16x2(float& lo, float& hi, uint32_t v) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n add.rn.f32.bf16 %0, l, %0;\n add.rn.f32.bf16 %1, h, %1;\n}"
      : "+f"(lo), "+f"(hi) : "r"(v));
}

// x = 2^(t - ref) of the row's tokens of a tile, as bf16 pairs; the largest sum of a block to `most`.
// Returns the row's part of l.
__device__ __forceinline__ float row_exp(uint32_t t_s, const Scales& y, float c, float ref, uint32_t (&h)[64], float& most) {
  float l = 0.f;
  most = 0.f;
  uint32_t r[2][16];
  ld16_start(t_s, r[0]);
#pragma unroll
  for (int b = 0; b < kTileBlocks; ++b) {
    ld16_wait(r[b & 1]);
    if (b + 1 < kTileBlocks) ld16_start(t_s + 16 * (b + 1), r[(b + 1) & 1]);
    uint32_t* v = r[b & 1];
    const float m1 = y.ks[b] * c, s1 = y.ev(b) - ref;
    const uint64_t mul = pack2(m1, m1), sub = pack2(s1, s1);
    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 t = unpack2(fma2(pack2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), mul, sub));
      const float x0 = ex2(t.x), x1 = ex2(t.y);
      const __nv_bfloat162 p = __floats2bfloat162_rn(x0, x1);
      const uint32_t q = h[8 * b + k] = *reinterpret_cast<const uint32_t*>(&p);
      add_bf16x2(sum0, sum1, q);
    }
    const float s = sum0 + sum1;
    most = fmaxf(most, s);
    l = fmaf(s, y.iv(b), l);
  }
  return l;
}

// The tokens of a block of 16 at position `pos` that a row sees, as bits.
__device__ __forceinline__ uint32_t seen_of(int pos, int lo, int hi) {
  const int up = min(max(hi - pos, 0), kBlock), down = min(max(lo - pos, 0), kBlock);
  return (1u << up) - (1u << min(up, down));
}

// A tile in general: rows that do not see all of it, that have seen nothing yet, or whose x is out of range.
// Looks at the maxima first and moves a reference where it has to.  Writes x to TMEM over S, whose columns it has read
// by then.  A loop, apart from row_exp: few tiles come here, and one loop with both forms cost the others 13 % in
// registers and moves.
struct Row {
  float m, f, add;
};
__device__ __forceinline__ void tile_general(Row& w, uint32_t t_s, const float* ks, const float* vs, float c, int pos,
                                             int lo, int hi, uint32_t gone) {
  float top = -INFINITY, top_l = -INFINITY;  // of x's and of l's logarithms
#pragma unroll 1
  for (int b = 0; b < kTileBlocks; b += 2) {
    float s[32];
    umma::ld32(t_s + 16 * b, s);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t seen = gone >> (b + e) & 1 ? 0u : seen_of(pos + 16 * (b + e), lo, hi);
      float v = -INFINITY;
#pragma unroll
      for (int k = 0; k < 16; ++k) v = fmaxf(v, seen >> k & 1 ? s[16 * e + k] : -INFINITY);
      if (v > -INFINITY) {
        top = fmaxf(top, fmaf(v, ks[b + e] * c, scale_log2(vs[b + e])));
        top_l = fmaxf(top_l, v * (ks[b + e] * c));
      }
    }
  }
  w.f = 1.f;                                 // what O and l so far are to be scaled by
  if (top > w.m + kFarX || top_l > w.m + kFarL || (w.m == -INFINITY && top > -INFINITY)) {
    w.f = w.m == -INFINITY ? 0.f : ex2(w.m - top);
    w.m = top;
  }
  const float ref = w.m == -INFINITY ? 0.f : w.m;
  w.add = 0.f;
#pragma unroll 1
  for (int b = 0; b < kTileBlocks; b += 2) {
    float s[32];
    uint32_t h[16];
    umma::ld32(t_s + 16 * b, s);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t seen = gone >> (b + e) & 1 ? 0u : seen_of(pos + 16 * (b + e), lo, hi);
      const float m1 = ks[b + e] * c, s1 = scale_log2(vs[b + e]) - ref;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 16 * e + 2 * k;
        float x0 = ex2(fmaf(s[i], m1, s1)), x1 = ex2(fmaf(s[i + 1], m1, s1));
        if (!(seen >> (2 * k) & 1)) x0 = 0.f;
        if (!(seen >> (2 * k + 1) & 1)) x1 = 0.f;
        const __nv_bfloat162 p = __floats2bfloat162_rn(x0, x1);
        sum += __low2float(p) + __high2float(p);
        h[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
      }
      w.add = fmaf(sum, scale_inverse(vs[b + e]), w.add);
    }
    st16(t_s + 8 * b, reinterpret_cast<const float*>(h));
    wait_st();                               // before the next load
  }
}

// Exact: 4 significant bits.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t c) {
  const float2 f = __half22float2(e4m3x2_to_half2(c));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Place of a tile of queries among the split ones, from its first packed row: a request's tiles are
// neighbours, and no two requests' meet.
__device__ __forceinline__ int query_tile(int row, int r, int qpt) { return row / qpt + r; }

// Splits the queries once: for each (tile, KV head) [16-byte chunk][128 rows][16 bytes], the first pieces' D / 16
// chunks and then the second's, and each row's factor.  Grid: tiles, KV heads; a thread to a row.
template <int D>
__global__ void __launch_bounds__(kRows) split_kernel(const PagedAttend a, const int qpt) {
  launch_dependents();
  const PagedDev& d = a.d;
  const int row = threadIdx.x, h = blockIdx.y, id = blockIdx.x;
  // the last request whose first tile is at or before this one
  int lo = 0, hi = a.n_reqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    const int first = a.row_start ? __ldg(a.row_start + mid) : mid;
    if (query_tile(first, mid, qpt) <= id) lo = mid; else hi = mid - 1;
  }
  const Req q = req_of(a, lo);
  const int i0 = (id - query_tile(q.first, lo, qpt)) * qpt;
  if (i0 < 0 || i0 >= q.n || !KVS_DCHECK(d, q.first >= 0 && q.first + q.n <= a.total_q)) return;
  const int i = i0 + row / d.G;
  const bool live = row / d.G < qpt && i < q.n;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
      (live ? ((size_t)(q.first + i) * d.Hq + h * d.G + row % d.G) * D : 0));
  uint4 raw[D / 8];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) raw[j] = live ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
  __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int u = 0; u < 4; ++u) top2 = __hmax2(top2, __habs2(reinterpret_cast<const __nv_bfloat162*>(&raw[j])[u]));
  const float amax = fmaxf(__low2float(top2), __high2float(top2));
  const int e = scale_exp(amax);
  const uint64_t up = pack2(exp2_int(-e), exp2_int(-e));
  const size_t at = (size_t)id * d.Hkv + h;
  a.q_factors[at * kRows + row] = amax <= kFloatMax ? exp2_int(live ? e : 0) * (kLog2e * rsqrtf((float)D)) : NAN;
  uint8_t* out = a.q_pieces + at * (kRows * 2 * D) + row * 16;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    uint32_t hi4[4], lo4[4];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      // scaled, an element is at most 448 and has 8 bits: f16 holds it and its first piece's remainder exactly
      const uint32_t two = reinterpret_cast<const uint32_t*>(&raw[2 * j + u / 4])[u % 4];
      const float2 f = unpack2(mul2(pack2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u)), up));
      const __half2 v = __floats2half2_rn(f.x, f.y);
      const uint32_t c1 = f16x2_to_e4m3x2(v);
      const uint32_t c2 = f16x2_to_e5m2x2(__hsub2(v, e4m3x2_to_half2(c1)));
      hi4[u / 2] = u & 1 ? hi4[u / 2] | c1 << 16 : c1;
      lo4[u / 2] = u & 1 ? lo4[u / 2] | c2 << 16 : c2;
    }
    *reinterpret_cast<uint4*>(out + (size_t)j * (kRows * 16)) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
    *reinterpret_cast<uint4*>(out + (size_t)(j + D / 16) * (kRows * 16)) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const PagedAttend a, const int qpt) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Search search;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;
  uint8_t* sk = sq + kQStages * 2 * C::Q;
  uint8_t* sv = sk + kKStages * C::K;
  Misc& ms = *reinterpret_cast<Misc*>(sv + kVStages * C::V);
  const PagedDev& d = a.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per = 2 * qpt;                                // query tokens of a unit

  launch_dependents();
  if (blockIdx.x == 0) report_rows(a, kThreads);
  const long long total = total_tiles(a, per, kThreads / 32, search);
  const long long ctas = min((long long)gridDim.x, total);
  if (blockIdx.x >= ctas) {
    if (tid == 0) a.cuts[blockIdx.x * 8 + 3] = 0;
    wait_previous();                         // nothing that follows runs before the split queries are done with
    return;
  }
  const long long begin = total * blockIdx.x / ctas, end = total * (blockIdx.x + 1) / ctas;
  locate(a, per, kThreads / 32, begin, search);
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_u32(&ms.k_full[i]), 1);
      mbar_init(smem_u32(&ms.k_empty[i]), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_u32(&ms.v_full[i]), kVThreads / 32);
      mbar_init(smem_u32(&ms.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&ms.drain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms.s_ready[i]), 1);
      mbar_init(smem_u32(&ms.p_ready[i]), 4);
      mbar_init(smem_u32(&ms.o_done[i]), 1);
      mbar_init(smem_u32(&ms.q_empty[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ms.q_ready[i]), 1);
      mbar_init(smem_u32(&ms.sc_ready[i]), 1);
    }
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    umma::alloc(smem_u32(&ms.tmem), 512);
    umma::relinquish();
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = ms.tmem;                          // S of A, S of B, O of A, O of B
  Walk w;
  w.start(a, search, (int)(end - begin), per);

  if (warp == kCopyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    // ---- K pages and the blocks' scales: lane j < 8 has block j of the tile
    const uint8_t* kbase = d.k + a.layer * d.layer_bytes;
    const float2* sbase = d.scales + a.layer * d.layer_scales;
    int count = 0;
    bool ok = true;
    while (w.nt > 0 && ok) {
      const int32_t* row = a.table + (size_t)w.r * a.table_stride;
      auto fetch = [&](int t, int& nb, int& page, float2& sc) {
        const int b = w.u.b0 + t * kTileBlocks;
        nb = max(0, min(kTileBlocks, w.u.b0 + w.u.nb - b));
        page = -1;
        sc = make_float2(1.f, 1.f);
        if (lane < nb) {
          page = __ldg(row + b + lane);
          if (page < 0 || page >= d.num_pages) {
            paged_error(d, kErrState);
            page = -1;
          } else {
            sc = __ldg(sbase + (size_t)page * d.Hkv + w.h);
            sc.x = fmaxf(sc.x, exp2_int(kScaleMinExp));
            sc.y = fmaxf(sc.y, exp2_int(kScaleMinExp));
          }
        }
      };
      int nb, page;
      float2 sc;
      fetch(w.t0, nb, page, sc);
      for (int t = w.t0; t < w.t0 + w.nt && ok; ++t, ++count) {
        const int st = count % kKStages, slot = count % kSlots;
        if (count >= kKStages) ok = mbar_wait(smem_u32(&ms.k_empty[st]), (count / kKStages - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t full = smem_u32(&ms.k_full[st]), dst = smem_u32(sk + st * C::K);
        const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) mbar_expect(full, __popc(good) * C::PAGE);
        __syncwarp();
        if (page >= 0) bulk_load(dst + lane * C::PAGE, kbase + ((size_t)page * d.Hkv + w.h) * C::PAGE, C::PAGE, full);
        if (lane < kTileBlocks) {
          ms.ks[slot][lane] = sc.x;
          ms.vs[slot][lane] = sc.y;
        }
        if (lane == 0) ms.bad[slot] = (int)(~good & 0xffu);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ms.sc_ready[slot]));
          mbar_arrive(full);
        }
        if (t + 1 < w.t0 + w.nt) fetch(t + 1, nb, page, sc);
      }
      if (ok) w.next(a);
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
    for (int i = max(0, count - kKStages); i < count; ++i) mbar_wait(smem_u32(&ms.k_full[i % kKStages]), (i / kKStages) & 1);
  } else if (warp == kQWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    // ---- the next segment's queries and row factors, as the split kernel left them
    bool ok = true;
    wait_previous();
    while (w.nt > 0 && ok) {
      const int buf = w.seg % kQStages, slot = w.seg % kSlots, tiles = w.u.cnt > qpt ? 2 : 1;
      if (w.seg >= kQStages) ok = warp_wait(smem_u32(&ms.q_empty[buf]), (w.seg / kQStages - 1) & 1);
      if (!ok) break;
      const uint32_t full = smem_u32(&ms.q_ready[slot]);
      if (lane == 0) mbar_expect(full, tiles * (C::Q + kRows * 4));
      __syncwarp();
      if (lane < tiles) {
        int id = query_tile(w.q.first + w.u.i0 + lane * qpt, w.r, qpt);
        if (!KVS_DCHECK(d, id >= 0 && id < a.total_q / qpt + a.n_reqs && w.h < d.Hkv)) id = 0;
        const size_t at = (size_t)id * d.Hkv + w.h;
        bulk_load(smem_u32(sq + (buf * 2 + lane) * C::Q), a.q_pieces + at * C::Q, C::Q, full);
        bulk_load(smem_u32(&ms.qc[slot][lane * kRows]), a.q_factors + at * kRows, kRows * 4, full);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      w.next(a);
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
    // copies still in flight land before the CTA ends
    for (int i = max(0, w.seg - kQStages); i < w.seg; ++i) mbar_wait(smem_u32(&ms.q_ready[i % kSlots]), (i / kSlots) & 1);
  } else if (warp == kQWarp + 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    // ---- for the join kernel: the unit that this share enters in its middle, if that is the unit's first cut, and
    // the CTAs that have a part of it: [blockIdx.x - 1, last], the first in its slot 1 unless the unit is its first
    if (lane == 0) {
      const long long before = total * (blockIdx.x - 1ll) / ctas, off = begin - w.v0;     // the unit's start
      const bool first = w.v0 > kSetup && before <= off + kSetup;
      int* at = a.cuts + blockIdx.x * 8;
      at[0] = w.r;
      at[1] = w.qg;
      at[2] = w.h;
      at[3] = first ? cta_of(off + w.u.cost() - 1, total, (int)ctas) : 0;
      at[4] = off > before;
    }
  } else if (warp >= kVWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    // ---- V: a page's row d (16 tokens of a dimension) becomes two 16-byte operand rows
    constexpr int PPI = kVThreads / D;                    // pages of one pass of the threads
    constexpr int NI = kTileBlocks / PPI;
    const int vt = tid - kVWarp * 32, dim = vt % D, pp = vt / D;
    const uint8_t* vbase = d.v + a.layer * d.layer_bytes;
    int count = 0;
    bool ok = true;
    uint4 raw[NI];
    auto fetch = [&](int t) {
      const int b = w.u.b0 + t * kTileBlocks;
      const int32_t* row = a.table + (size_t)w.r * a.table_stride;
      int page[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int j = i * PPI + pp;
        page[i] = b + j < w.u.b0 + w.u.nb ? __ldg(row + b + j) : -1;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
        raw[i] = page[i] >= 0 && page[i] < d.num_pages
                     ? __ldg(reinterpret_cast<const uint4*>(vbase + ((size_t)page[i] * d.Hkv + w.h) * C::PAGE + dim * 16))
                     : make_uint4(0, 0, 0, 0);
    };
    fetch(w.t0);
    while (w.nt > 0 && ok) {
      for (int t = w.t0; t < w.t0 + w.nt && ok; ++t, ++count) {
        const int st = count % kVStages;
        if (count >= kVStages) ok = warp_wait(smem_u32(&ms.v_empty[st]), (count / kVStages - 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t* c = &raw[i].x;
          uint32_t h[8];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            h[2 * u] = e4m3x2_to_bf16x2(c[u] & 0xffffu);
            h[2 * u + 1] = e4m3x2_to_bf16x2(c[u] >> 16);
          }
          uint4* dst = reinterpret_cast<uint4*>(sv + st * C::V + (size_t)(2 * (i * PPI + pp)) * (D * 16) + dim * 16);
          dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
          dst[D] = make_uint4(h[4], h[5], h[6], h[7]);    // the next 8 tokens
        }
        umma::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.v_full[st]));
        if (t + 1 < w.t0 + w.nt) fetch(t + 1);
      }
      if (ok) {
        w.next(a);
        if (w.nt > 0) fetch(w.t0);
      }
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
    // ---- matrix instructions
    constexpr uint32_t id_hi = idesc_f8(128, 128), id_lo = idesc_f8(128, 128, kE5M2), id_pv = umma::idesc_f16(true, 128, D);
    const uint32_t on = elect();
    int count = 0, count_b = 0;
    bool ok = true;
    auto qk = [&](int x, int n) {                         // S of tile x from K number n
      const uint32_t aq = desc_lo(smem_u32(sq + (w.seg % kQStages * 2 + x) * C::Q), kRows * 16);
      const uint32_t bk = desc_lo(smem_u32(sk + (n % kKStages) * C::K), 128);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)                    // the pieces hi, then lo, over the same K
        mma_f8(on, tmem + x * 128, aq + k * (2 * kRows), desc_hi(128), bk + (k % (D / 32)) * 16, desc_hi(8 * D),
                 k < D / 32 ? id_hi : id_lo, k > 0);
      commit(on, smem_u32(&ms.s_ready[x]));
    };
    auto products = [&](int x, int n, uint32_t parity, bool first, bool last) {    // O, and the next S, of tile x
      ok = ok && warp_wait(smem_u32(&ms.p_ready[x]), parity);
      if (!ok) return;
      umma::fence_after();
      const uint32_t bv = desc_lo(smem_u32(sv + (n % kVStages) * C::V), D * 16);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_f16_ts(on, tmem + 256 + x * 128, tmem + x * 128 + k * 8, bv + k * (2 * D), desc_hi(128), id_pv,
                   !(first && k == 0));
      if (last) commit(on, smem_u32(&ms.o_done[x]));
      else qk(x, n + 1);                                  // behind the product, whose P it overwrites
    };
    while (w.nt > 0 && ok) {
      const bool two = w.u.cnt > qpt;
      ok = warp_wait(smem_u32(&ms.q_ready[w.seg % kSlots]), (w.seg / kSlots) & 1);
      ok = ok && warp_wait(smem_u32(&ms.k_full[count % kKStages]), (count / kKStages) & 1);
      if (!ok) break;
      umma::fence_after();
      qk(0, count);
      if (two) qk(1, count);
      commit(on, smem_u32(&ms.k_empty[count % kKStages]));
      if (w.nt == 1) commit(on, smem_u32(&ms.q_empty[w.seg % kQStages]));
      for (int t = 0; t < w.nt && ok; ++t, ++count) {
        const bool more = t + 1 < w.nt;
        const int n = count + 1;
        ok = warp_wait(smem_u32(&ms.v_full[count % kVStages]), (count / kVStages) & 1);
        if (more) ok = ok && warp_wait(smem_u32(&ms.k_full[n % kKStages]), (n / kKStages) & 1);
        products(0, count, count & 1, t == 0, !more);
        if (two) products(1, count, count_b++ & 1, t == 0, !more);
        if (!ok) break;
        commit(on, smem_u32(&ms.v_empty[count % kVStages]));
        if (more) commit(on, smem_u32(&ms.k_empty[n % kKStages]));
        if (t + 2 == w.nt) commit(on, smem_u32(&ms.q_empty[w.seg % kQStages]));
      }
      if (!ok) break;
      w.next(a);
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
    commit(on, smem_u32(&ms.drain));
    mbar_wait(smem_u32(&ms.drain), 0);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    // ---- softmax of tile x: a thread to a row
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + x * 128 + lanes, t_o = tmem + 256 + x * 128 + lanes;
    const int token = row / d.G, head = row % d.G;        // of the tile
    int count = 0, seg = 0;                               // tiles and segments that have this tile of queries
    bool ok = true;
    // the next segment that has this tile (B may have none)
    Walk* const walks = ms.walk[warp];
    auto advance = [&](Walk& to, const Walk& from, bool step) {
      if (lane == 0) {
        to = from;
        if (step) to.next(a);
        while (to.nt > 0 && x == 1 && to.u.cnt <= qpt) to.next(a);
      }
      __syncwarp();
    };
    advance(walks[0], w, false);
    for (; walks[seg & 1].nt > 0 && ok;) {
      const Walk& w = walks[seg & 1];
      float c = 0.f;
      float m = -INFINITY, l = 0.f;
      const int i = x * qpt + token;                      // the row's token of the unit
      const int hi = w.q.p0 + w.u.i0 + i + 1, lo = a.window > 0 ? hi - a.window : 0;
      // positions that all live rows of the tile see
      const int all_hi = w.q.p0 + w.u.i0 + x * qpt + 1;
      const int last = w.q.p0 + w.u.i0 + min(w.u.cnt, (x + 1) * qpt);
      const int all_lo = a.window > 0 ? max(last - a.window, 0) : 0;
      int base = (w.u.b0 + w.t0 * kTileBlocks) * kBlock;
      const int nt = w.nt, tile = w.done;
      for (int t = 0; t < nt && ok; ++t, ++count, base += kTile) {
        const int slot = (tile + t) % kSlots;
        // The scales come ahead of S.  Not at a segment's start: B may skip segments, and is only sure of the
        // barrier's phase once S is there; that is also where the row's factor is read.
        if (t == 0) {
          ok = warp_wait(smem_u32(&ms.s_ready[x]), count & 1);
          c = ms.qc[w.seg % kSlots][x * kRows + row];
        }
        ok = ok && warp_wait(smem_u32(&ms.sc_ready[slot]), ((tile + t) / kSlots) & 1);
        const uint32_t bad = ms.bad[slot];
        if (t > 0) ok = ok && warp_wait(smem_u32(&ms.s_ready[x]), count & 1);
        if (!ok) break;
        umma::fence_after();
        // Mostly all rows see all of the tile and the reference serves, so the exponentials are taken at once.  The
        // first reference is any token's t: bf16 has float32's range.
        bool general = base < all_lo || base + kTile > all_hi || bad;
        if (t == 0 && !general) m = fmaf(ld1(t_s), ms.ks[slot][0] * c, scale_log2(ms.vs[slot][0]));
        general = general || __any_sync(0xffffffffu, !(fabsf(m) < 1e30f));
        float f = 1.f, add;
        if (!general) {
          Scales y;
          *reinterpret_cast<float4*>(y.ks) = *reinterpret_cast<const float4*>(ms.ks[slot]);
          *reinterpret_cast<float4*>(y.ks + 4) = *reinterpret_cast<const float4*>(ms.ks[slot] + 4);
          *reinterpret_cast<float4*>(y.vs) = *reinterpret_cast<const float4*>(ms.vs[slot]);
          *reinterpret_cast<float4*>(y.vs + 4) = *reinterpret_cast<const float4*>(ms.vs[slot] + 4);
          uint32_t h[64];
          float most;
          add = row_exp(t_s, y, c, m, h, most);
          general = __any_sync(0xffffffffu, !(fmaxf(most * kSumShare, add) <= kLimit));
          if (!general) {
            st32(t_s, h);                                   // P over S, two tokens to a column
            st32(t_s + 32, h + 32);
          }
        }
        if (general) {
          Row r{m};
          tile_general(r, t_s, ms.ks[slot], ms.vs[slot], c, base, lo, hi, bad);
          m = r.m;
          f = r.f;
          add = r.add;
        }
        l = fmaf(l, f, add);
        // S was issued behind the previous product, so that is done with O
        if (t > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
          for (int j = 0; j < D; j += 16) {
            float o[16];
            ld16(t_o + j, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= f;
            st16(t_o + j, o);
          }
        }
        wait_st();
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.p_ready[x]));
      }
      if (!ok) break;
      advance(walks[(seg + 1) & 1], w, true);
      ok = warp_wait(smem_u32(&ms.o_done[x]), seg & 1);
      if (!ok) break;
      umma::fence_after();
      const bool live = token < qpt && i < w.u.cnt && KVS_DCHECK(d, w.q.first >= 0 && w.q.first + w.u.i0 + i < a.total_q);
      if (w.whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
            (live ? ((size_t)(w.q.first + w.u.i0 + i) * d.Hq + w.h * d.G + head) * D : 0);
#pragma unroll
        for (int j = 0; j < D; j += 16) {
          float o[16];
          ld16(t_o + j, o);
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
            h[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (live) {
            reinterpret_cast<uint4*>(out + j)[0] = make_uint4(h[0], h[1], h[2], h[3]);
            reinterpret_cast<uint4*>(out + j)[1] = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
      } else {
        const size_t rec = ((size_t)(2 * blockIdx.x + (w.first ? 0 : 1)) * 2 + x) * kRows + row;
#pragma unroll
        for (int j = 0; j < D; j += 16) {
          float o[16];
          ld16(t_o + j, o);
          if (live) {
            float4* dst = reinterpret_cast<float4*>(a.part_o) + (rec - row) * (D / 4) + (j / 4) * kRows + row;
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[k * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (live) a.part_ml[rec] = make_float2(m, l);
      }
      umma::fence_before();
      ++seg;
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
  }
  __syncwarp();
  __syncthreads();
  if (warp == kMmaWarp) {
    umma::fence_after();
    umma::dealloc(tmem, 512);
  }
}

// Adds the partials of the unit that CTA blockIdx.x + 1 left in its cut.
constexpr int kJoinThreads = 256, kJoinRows = 16, kMostParts = 256;   // a part per CTA at most
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const PagedAttend a, const int qpt) {
  wait_previous();
  const PagedDev& d = a.d;
  const int* at = a.cuts + (blockIdx.x + 1) * 8;
  const int c0 = blockIdx.x, c1 = at[3], r = at[0], qg = at[1], h = at[2], slot = at[4];
  if (c1 == 0) return;
  if (!KVS_DCHECK(d, r >= 0 && r < a.n_reqs && h >= 0 && h < d.Hkv && c1 > c0 && c1 <= (int)gridDim.x && slot >> 1 == 0)) return;
  const Req q = req_of(a, r);
  if (!KVS_DCHECK(d, qg >= 0 && qg * 2 * qpt < q.n && q.first >= 0 && q.first + q.n <= a.total_q)) return;
  const Unit u = unit_of(a, q, qg, 2 * qpt);
  __shared__ float weight[kMostParts][kJoinRows + 1], total[kJoinRows];
  const int n = c1 - c0 + 1;
  auto rec_of = [&](int x, int i) { return ((size_t)(2 * (c0 + i) + (i == 0 ? slot : 0)) * 2 + x) * kRows; };
  // 16 threads to a row find its parts' weights and its sum
  {
    const int mine = threadIdx.x / 16, idx = threadIdx.x % 16, pr = blockIdx.y * kJoinRows + mine;
    const int x = pr / kRows, row = pr % kRows;
    const int parts = row / d.G < qpt && x * qpt + row / d.G < u.cnt ? n : 0;    // a warp has two rows: the
    float top = -INFINITY, sum = 0.f;                                            // shuffles are for both
    for (int i = idx; i < parts; i += 16) top = fmaxf(top, a.part_ml[rec_of(x, i) + row].x);
    __syncwarp();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, 16));
    const float ref = top > -INFINITY ? top : 0.f;
    for (int i = idx; i < parts; i += 16) {
      const float2 ml = a.part_ml[rec_of(x, i) + row];
      const float f = ex2(ml.x - ref);
      sum = fmaf(ml.y, f, sum);
      weight[i][mine] = f;
    }
    __syncwarp();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, 16);
    if (idx == 0) total[mine] = sum;
  }
  __syncthreads();
  // a thread has four dimensions of a row; partials are [tile][D / 4][128 rows][4]
  const int pr = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, x = pr / kRows, row = pr % kRows;
  const int i = x * qpt + row / d.G;
  if (row / d.G >= qpt || i >= u.cnt) return;
  const float sum = total[threadIdx.x % kJoinRows];
  float4 acc[D / 64];
#pragma unroll
  for (int q4 = 0; q4 < D / 64; ++q4) acc[q4] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int e = 0; e < n; ++e) {
    const size_t rec = rec_of(x, e);
    const float f = weight[e][threadIdx.x % kJoinRows];
#pragma unroll
    for (int q4 = 0; q4 < D / 64; ++q4) {
      const float4 v = reinterpret_cast<const float4*>(a.part_o)[rec * (D / 4) + (threadIdx.x / kJoinRows + 16 * q4) * kRows + row];
      acc[q4].x = fmaf(v.x, f, acc[q4].x);
      acc[q4].y = fmaf(v.y, f, acc[q4].y);
      acc[q4].z = fmaf(v.z, f, acc[q4].z);
      acc[q4].w = fmaf(v.w, f, acc[q4].w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       ((size_t)(q.first + u.i0 + i) * d.Hq + h * d.G + row % d.G) * D;
#pragma unroll
  for (int q4 = 0; q4 < D / 64; ++q4) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[q4].x * inv, acc[q4].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[q4].z * inv, acc[q4].w * inv);
    uint2 raw;
    raw.x = *reinterpret_cast<const uint32_t*>(&lo);
    raw.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(out + (threadIdx.x / kJoinRows + 16 * q4) * 4) = raw;
  }
}

template <int D>
cudaError_t launch_d(const PagedAttend& a, int grid, cudaStream_t st) {
  using C = Cfg<D>;
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_optin_once(opted, prompt_kernel<D>, C::SMEM);
  if (e != cudaSuccess) return e;
  if (grid > kMostParts) return cudaErrorInvalidConfiguration;
  const int qpt = kRows / a.d.G;
  split_kernel<D><<<dim3(paged_prompt_tiles(a.d.G, a.n_reqs, a.total_q), a.d.Hkv), kRows, 0, st>>>(a, qpt);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // each kernel starts while the one before ends, and waits for its results where it needs them
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  e = cudaLaunchKernelEx(&cfg, prompt_kernel<D>, a, qpt);
  if (e != cudaSuccess || grid == 1) return e;
  cfg.gridDim = dim3(grid - 1, 2 * kRows / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel<D>, a, qpt);
}

}  // namespace

int paged_prompt_rows() { return 2 * kRows; }
// Tiles of split queries that a call may have.
int paged_prompt_tiles(int G, int n_reqs, int total_q) { return total_q / (kRows / G) + n_reqs; }
size_t paged_prompt_tile_bytes(int D) { return (size_t)kRows * 2 * D; }

cudaError_t launch_paged_prompt(const PagedAttend& a, int grid, cudaStream_t st) {
  return a.d.D == 64 ? launch_d<64>(a, grid, st) : launch_d<128>(a, grid, st);
}

}  // namespace kvs
