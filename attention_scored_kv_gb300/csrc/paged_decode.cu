// Tensor-core attention over the paged cache for few query rows: single tokens and the
// few tokens of a speculative step (bf16 queries, head_dim 64 or 128).
//
// For a unit (request, KV head) with R query rows (tokens x heads of the group) and a
// tile of 128 cached tokens j:
//   S^T = K Q^T        [128 tokens x rows]   E4M3 x E4M3 matrix instructions
//   t_jr = S_jr kscale_j c_r + log2 vscale_j,  top_r = the tile's maximum of t
//   x_jr = 2^(t_jr - top_r + 15),  P^T = V^T X   [D x rows]   E4M3 x E5M2
//   M_r = running maximum of top, w_r = 2^(top_r - M_r - 15)
//   l_r += w_r sum_j x_jr / vscale_j,  O_r += w_r P_r    (both moved when M moves)
// and o_r = O_r / l_r.  x carries V's scale in its exponent (the scales are powers of two),
// so x <= 2^15 whatever the scales are, and K and V enter the tensor core as they are stored.
//
// Precision: E4M3 holds 4 significant bits.  A bf16 query (8 bits) is split in two pieces
// of 4, hi = rn(q), lo = rn(16 (q - hi)) after a power of two brings the row's largest to
// (224, 448]: exact for elements within 2^13 of it, off by 2^-21 of it at most below.  A
// probability is three E5M2 pieces, each of 8 times the remainder of the one before: off by
// at most 2^-11 of itself down to 2^-29 of the tile's heaviest and by 2^-38 of the heaviest
// below that.  The range is what matters: a head whose sink takes nearly all the weight has a
// value near 0 there, and its output is the sum of very many small weights.  Two E4M3
// pieces against the row's maximum lost a quarter of such an output at 131072 tokens.  For the same reason
// every tile has its own reference, and its product is added in registers.  The pieces are
// separate columns of the same instructions; accumulation is float32.
//
// How: the 128-token tiles of all units are laid end to end and cut evenly over a
// persistent grid, two CTAs to an SM (each CTA finds its range from the device lengths by
// itself); a unit that a cut splits leaves float32 partials which the join kernel adds.
// Per CTA one warp issues the pages' bulk copies into a ring, one the matrix instructions,
// four warps the softmax (a thread is a token, so scales and masks are one per thread and
// the probabilities go to shared memory as bytes; the thread of token i also sums dimension i of the
// products).  S is double buffered: the next tile's S is computed under this one's softmax.  So is the
// product up to 16 rows: the last one is added while the next is computed.
//
// Bound by the pages' bytes.  Measured on 32/4 heads of 128: 16 contexts of 32768 tokens
// 89 us (5.95 TB/s, 89 % of the measured copy rate), 64 of 1024 to 32768 with masses 190 us;
// one of 131072 on 64/8 heads 53 us (5.1 TB/s), where about 4 us before the first copy
// and the join weigh more; one of 700 tokens 10 us, the call included.
#include "paged_cut.h"
#include "paged_mma.cuh"

namespace kvs {
namespace {

using namespace pmma;

using cut::kTileBlocks;
constexpr int kTile = kTileBlocks * kBlock;      // tokens of a tile
constexpr int kThreads = 192;            // 4 softmax warps, copies, matrix instructions
constexpr int kCtasPerSm = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 15.f;             // the largest x is 2^15, E5M2's largest power of two
// Factor of a query's second piece, the largest that keeps it in range: the first is at most 448, where half
// a step is 16.  Of a probability's second and third against the one before: half a step of 3 bits.
constexpr float kLoQ = 16.f, kLoP = 8.f;

// Tiles of request r's units (all KV heads alike) and their ranges.
struct Unit {
  int first, n;          // first packed row, query tokens handled
  int hi0, lo0;          // the first query sees [lo0, hi0); the i-th [lo_i, hi0 + i)
  int b0, nb, tiles;     // visible blocks of any of them
};

__device__ __forceinline__ Unit unit_of(const PagedAttend& a, int r) {
  Unit u;
  u.first = r;
  u.n = 1;
  int n = 1;
  if (a.row_start) {
    u.first = __ldg(a.row_start + r);
    n = __ldg(a.row_start + r + 1) - u.first;
    u.n = u.first < 0 ? 0 : min(min(n, a.max_q_len), a.total_q - u.first);
  }
  const int len = min(max(__ldg(a.kv_len + r), 0), a.table_stride * kBlock);
  const int p0 = len - n;                  // position of the first query; may be negative
  u.hi0 = p0 + 1;
  u.lo0 = a.window > 0 ? p0 + 1 - a.window : 0;
  const int hi = max(p0 + u.n, 0);
  u.b0 = max(u.lo0, 0) / kBlock;
  u.nb = max((hi + kBlock - 1) / kBlock - u.b0, 0);
  u.tiles = u.n > 0 ? max((u.nb + kTileBlocks - 1) / kTileBlocks, 1) : 0;
  return u;
}

// A CTA's walk over its tiles, segment by segment (a segment: tiles of one unit).
struct Walk {
  int r, h;              // request, KV head
  int t0, nt;            // the segment's tiles of the unit: [t0, t0 + nt)
  int left;              // tiles of the CTA from here on
  Unit u;
  bool first, whole;
  __device__ void clip() {
    nt = min(u.tiles - t0, left);
    whole = nt == u.tiles;
  }
  __device__ void next(const PagedAttend& a) {
    left -= nt;
    first = false;
    t0 = 0;
    if (left <= 0) return;
    if (++h == a.d.Hkv) {
      h = 0;
      do {
        u = unit_of(a, ++r);
      } while (u.tiles == 0);
    }
    clip();
  }
};

// Tiles of the call, by every thread of the block.
__device__ long long total_tiles(const PagedAttend& a, long long* s_sum) {
  long long all = 0;
  for (int r = threadIdx.x; r < a.n_reqs; r += kThreads) all += unit_of(a, r).tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = all;
  __syncthreads();
  all = 0;
  for (int w = 0; w < kThreads / 32; ++w) all += s_sum[w];
  __syncthreads();
  return all * a.d.Hkv;
}

template <int D, int RT>
struct Cfg {
  static constexpr int N = 2 * RT;                       // columns of S: both pieces of the queries
  static constexpr int NP = RT == 8 ? 32 : 3 * RT;       // of the product: three of the probabilities (a multiple of 16)
  static constexpr int NO = RT == 32 ? 1 : 2;            // products in TMEM
  static constexpr int PAGE = 16 * D;                    // bytes of a page of K or V of one head
  static constexpr int HALF = kTileBlocks * PAGE;        // K (or V) of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int Q = N * D, P = NP * kTile;
  static constexpr int MISC = RT == 32 ? 5120 : 4096;
  static constexpr int ROOM = 227 * 1024 / kCtasPerSm - 1024 - Q - P - MISC;
  static constexpr int NS = ROOM / STAGE < 6 ? ROOM / STAGE : 6;
  // an M of 128 reads a further 1 KB behind the last page of V for D = 64: Q is there
  static constexpr int SMEM = NS * STAGE + Q + P + MISC + 1024;
  static constexpr int COLS = 2 * N + NO * NP, TMEM = COLS <= 128 ? 128 : 256;
  static_assert(NS >= 2 && COLS <= TMEM && TMEM * kCtasPerSm <= 512 && (SMEM + 1024) * kCtasPerSm <= 228 * 1024,
                "ring, TMEM, shared memory");
};

// What a tile does to a row: x is 2^(t - ref); the sums so far are multiplied by `keep`, the tile's part of l by
// `weight`; the product before it by `last`, that is its own weight times `keep`.
struct RowStep {
  float ref, keep, weight, last;
};

template <int RT>
struct Misc {
  uint64_t full[6], empty[6], s_ready[2], p_ready, o_done, q_ready, drain;
  uint32_t tmem;
  int token[RT];         // query token of a row
  int start_r, start_h, start_t;
  long long sums[kThreads / 32];
  float ks[6][kTileBlocks], ev[6][kTileBlocks], iv[6][kTileBlocks];   // of each stage's blocks
  float qc[2][RT];
  float wmax[2][4][RT];
  float wsum[4][RT];
  alignas(16) RowStep step[4][RT];       // of each softmax warp, alike
};

template <int D, int RT, bool MASS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const PagedAttend a) {
  using C = Cfg<D, RT>;
  constexpr int N = C::N, NP = C::NP;
  static_assert(sizeof(Misc<RT>) <= C::MISC, "Misc");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem;
  uint8_t* sq = ring + C::NS * C::STAGE;
  uint8_t* sp = sq + C::Q;
  Misc<RT>& ms = *reinterpret_cast<Misc<RT>*>(sp + C::P);
  const PagedDev& d = a.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  launch_dependents();
  if (blockIdx.x == 0) report_rows(a, kThreads);
  // barriers and TMEM while the lengths load
  Unit mine_u = unit_of(a, min(tid, a.n_reqs - 1));
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(&ms.full[i]), 1);
      mbar_init(smem_u32(&ms.empty[i]), 1);
    }
    mbar_init(smem_u32(&ms.s_ready[0]), 1);
    mbar_init(smem_u32(&ms.s_ready[1]), 1);
    mbar_init(smem_u32(&ms.p_ready), 4);
    mbar_init(smem_u32(&ms.o_done), 1);
    mbar_init(smem_u32(&ms.q_ready), 4);
    mbar_init(smem_u32(&ms.drain), 1);
    mbar_fence_init();
  }
  if (tid < RT) ms.token[tid] = tid / d.G;
  if (warp == 5) {
    umma::alloc(smem_u32(&ms.tmem), C::TMEM);
    umma::relinquish();
  }
  // this CTA's range: kThreads requests at a time (a call of more has their tiles counted first)
  long long total = 0, base = 0;
  if (a.n_reqs > kThreads) total = total_tiles(a, ms.sums);
  long long begin = 0, end = 0;
  for (int r0 = 0; r0 < a.n_reqs; r0 += kThreads) {
    const int r = r0 + tid;
    if (r0 > 0) mine_u = unit_of(a, min(r, a.n_reqs - 1));
    const int tiles = r < a.n_reqs ? mine_u.tiles : 0;
    const long long mine = (long long)tiles * d.Hkv;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) ms.sums[warp] = upto;
    __syncthreads();
    long long all = base;
    upto += base;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) upto += ms.sums[i];
      all += ms.sums[i];
    }
    if (a.n_reqs <= kThreads) total = all;
    const long long ctas = min((long long)gridDim.x, total);      // every one of them has a tile
    begin = ctas > blockIdx.x ? total * blockIdx.x / ctas : total;
    end = ctas > blockIdx.x ? total * (blockIdx.x + 1) / ctas : total;
    if (begin >= upto - mine && begin < upto) {
      const int off = (int)(begin - (upto - mine));
      ms.start_r = r;
      ms.start_h = off / tiles;
      ms.start_t = off % tiles;
    }
    __syncthreads();
    base = all;
    if (all > begin) break;
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  if (begin >= end) {                        // more CTAs than tiles
    if (tid == 0) a.cuts[blockIdx.x * 8 + 2] = 0;
    if (warp == 5) umma::dealloc(ms.tmem, C::TMEM);
    return;
  }
  const uint32_t tmem = ms.tmem, t_o = tmem + 2 * N;
  Walk w;
  w.r = ms.start_r;
  w.h = ms.start_h;
  w.t0 = ms.start_t;
  w.left = (int)(end - begin);
  w.first = true;
  w.u = unit_of(a, w.r);
  w.clip();

  if (warp == 4) {
    // ---- copies.  The table entries and scales of four tiles are loaded at once, a lane to a block, and
    // those of the next four while these are copied: their two latencies in a row took longer than a tile.
    const uint64_t policy = evict_first_policy();
    const uint8_t* kbase = d.k + a.layer * d.layer_bytes;
    const uint8_t* vbase = d.v + a.layer * d.layer_bytes;
    const float2* sbase = d.scales + a.layer * d.layer_scales;
    int count = 0;
    bool ok = true;
    while (w.left > 0 && ok) {
      const int32_t* row = a.table + (size_t)w.r * a.table_stride;
      const int stop = w.u.b0 + w.u.nb;
      auto load_page = [&](int t) {                         // of the lane's block from tile t on
        const int b = w.u.b0 + t * kTileBlocks + lane;
        return t < w.t0 + w.nt && b < stop ? __ldg(row + b) : -1;
      };
      auto load_scale = [&](int page) {
        return page >= 0 && page < d.num_pages ? __ldg(sbase + (size_t)page * d.Hkv + w.h) : make_float2(0.f, 1.f);
      };
      int page = load_page(w.t0), page_next = load_page(w.t0 + 4);
      float2 sc = load_scale(page), sc_next = make_float2(0.f, 1.f);
      for (int t = w.t0; t < w.t0 + w.nt && ok; ++t, ++count) {
        const int four = (t - w.t0) & 3, nb = max(0, min(kTileBlocks, w.u.nb - t * kTileBlocks));
        if (four == 0 && t > w.t0) {
          page = page_next;
          sc = sc_next;
          page_next = load_page(t + 4);
        }
        const int st = count % C::NS;
        if (count >= C::NS) ok = warp_wait(smem_u32(&ms.empty[st]), (count / C::NS - 1) & 1);
        if (!ok) break;
        const uint32_t full = smem_u32(&ms.full[st]);
        const uint32_t dst = smem_u32(ring + st * C::STAGE);
        // the last odd block's neighbour in V is read by the matrix instruction (with
        // probability 0): it gets the first block's values, which are finite
        const int odd = nb & 1;
        if (lane == 0) mbar_expect(full, (2 * nb + odd) * C::PAGE);
        __syncwarp();
        const int of = four * kTileBlocks + (lane < nb ? lane : 0);
        const int mine = __shfl_sync(0xffffffffu, page, of);
        const bool good = mine >= 0 && mine < d.num_pages;
        const size_t at = ((size_t)(good ? mine : 0) * d.Hkv + w.h) * C::PAGE;
        if (lane < nb) bulk_load(dst + lane * C::PAGE, kbase + at, C::PAGE, full, policy);
        if (lane < nb + odd) bulk_load(dst + C::HALF + lane * C::PAGE, vbase + at, C::PAGE, full, policy);
        const float ks = __shfl_sync(0xffffffffu, sc.x, of), vs = __shfl_sync(0xffffffffu, sc.y, of);
        if (lane < kTileBlocks) {
          const bool seen = lane < nb && good;
          if (lane < nb && !good) paged_error(d, kErrState);
          const float v = seen ? fmaxf(vs, exp2_int(kScaleMinExp)) : 1.f;      // a page that nothing was stored in has 0
          const float ev = (float)((__float_as_int(v) >> 23) - 127);
          ms.ks[st][lane] = seen ? fmaxf(ks, exp2_int(kScaleMinExp)) : 0.f;    // 0: nothing of this block is visible
          ms.ev[st][lane] = ev;
          ms.iv[st][lane] = exp2_int(-(int)ev);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
        if (four == 0) sc_next = load_scale(page_next);
      }
      if (ok) w.next(a);
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
    // copies still in flight land before the CTA ends
    for (int i = max(0, count - C::NS); i < count; ++i) mbar_wait(smem_u32(&ms.full[i % C::NS]), (i / C::NS) & 1);
  } else if (warp == 5) {
    // ---- matrix instructions
    constexpr uint32_t id_qk = idesc_f8(128, N), id_pv = idesc_f8(128, NP, kE4M3, kE5M2);
    const uint32_t on = elect();
    int count = 0, seg = 0;
    bool ok = true;
    auto pv = [&](int i, int nb) {                          // tile number i of the CTA
      const int st = i % C::NS, steps = (nb + 1) / 2;
      umma::fence_after();
      const uint32_t av = desc_lo(smem_u32(ring + st * C::STAGE + C::HALF), C::PAGE), bp = desc_lo(smem_u32(sp), NP * 16);
#pragma unroll
      for (int k = 0; k < kTileBlocks / 2; ++k)
        if (k < steps)
          mma_f8(on, t_o + (i % C::NO) * NP, av + k * (2 * C::PAGE / 16), desc_hi(128), bp + k * (2 * NP), desc_hi(128),
                 id_pv, k > 0);
      commit(on, smem_u32(&ms.empty[st]));
      commit(on, smem_u32(&ms.o_done));
    };
    while (w.left > 0 && ok) {
      ok = warp_wait(smem_u32(&ms.q_ready), seg & 1);
      const uint32_t bq = desc_lo(smem_u32(sq), 128);
      int nb_before = 0;
      for (int t = w.t0; t < w.t0 + w.nt && ok; ++t, ++count) {
        const int st = count % C::NS, nb = max(0, min(kTileBlocks, w.u.nb - t * kTileBlocks));
        ok = warp_wait(smem_u32(&ms.full[st]), (count / C::NS) & 1);
        if (!ok) break;
        umma::fence_after();
        const uint32_t ak = desc_lo(smem_u32(ring + st * C::STAGE), 128);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          mma_f8(on, tmem + (count & 1) * N, ak + k * 16, desc_hi(8 * D), bq + k * 16, desc_hi(8 * D), id_qk, k > 0);
        commit(on, smem_u32(&ms.s_ready[count & 1]));
        if (t > w.t0) {
          ok = warp_wait(smem_u32(&ms.p_ready), (count - 1) & 1);
          if (!ok) break;
          pv(count - 1, nb_before);
        }
        nb_before = nb;
      }
      if (ok) ok = warp_wait(smem_u32(&ms.p_ready), (count - 1) & 1);
      if (!ok) break;
      pv(count - 1, nb_before);
      ++seg;
      w.next(a);
    }
    if (!ok && lane == 0) paged_error(d, kErrTimeout);
    commit(on, smem_u32(&ms.drain));
    mbar_wait(smem_u32(&ms.drain), 0);
  } else {
    // ---- softmax: thread = token of the tile, then = dimension of the output
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float qk = kLog2e * rsqrtf((float)D);
    // the rows' queries as two E4M3 pieces; TPR threads to a row
    auto load_q = [&](const Walk& x, int buf) {
      constexpr int TPR = 128 / RT, E = D / TPR;
      const int row = tid / TPR, part = tid % TPR;
      float v[E];
      float amax = 0.f;
      const bool live = row < x.u.n * d.G;
      if (live) {
        const size_t at = ((size_t)(x.u.first + row / d.G) * d.Hq + x.h * d.G + row % d.G) * D + part * E;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + at;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const uint2 raw = __ldg(reinterpret_cast<const uint2*>(src + i));
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
          const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
          v[i] = f.x; v[i + 1] = f.y; v[i + 2] = g.x; v[i + 3] = g.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = scale_exp(amax);
      const float up = exp2_int(-e);
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f = v[i + 2 * u] * up, g = v[i + 2 * u + 1] * up;
          hi[u] = float2_to_e4m3x2(f, g);
          const float2 back = e4m3x2_to_float2(hi[u]);
          lo[u] = float2_to_e4m3x2((f - back.x) * kLoQ, (g - back.y) * kLoQ);
        }
        const int dim = part * E + i;
        *reinterpret_cast<uint32_t*>(sq + k_code(D, row, dim)) = hi[0] | hi[1] << 16;
        *reinterpret_cast<uint32_t*>(sq + k_code(D, row + RT, dim)) = lo[0] | lo[1] << 16;
      }
      if (part == 0) ms.qc[buf][row] = !live ? 0.f : amax <= kFloatMax ? exp2_int(e) * qk : NAN;
      umma::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms.q_ready));
    };
    load_q(w, 0);
    if (tid == 127) {
      // the unit that this share enters in its middle, if that is the unit's first cut, and the CTAs that have a
      // part of it: [blockIdx.x - 1, last], the first of them in its slot 1 unless the unit is its first
      const long long ctas = min((long long)gridDim.x, total), before = total * (blockIdx.x - 1ll) / ctas;
      const long long off = begin - w.t0;
      const bool first = w.t0 > 0 && before <= off;
      const int last = first ? cta_of(off + w.u.tiles - 1, total, (int)ctas) : 0;
      *reinterpret_cast<int4*>(a.cuts + blockIdx.x * 8) = make_int4(w.r, w.h, last, off > before);
    }
    named_sync(1, 128);                                    // qc of all rows
    // `ok`: this thread's waits; `go`: all threads' up to the last barrier, by which they leave the loops alike (none
    // is left waiting at a barrier)
    int count = 0, seg = 0;
    bool ok = true, go = true;
    while (w.left > 0) {
      float l[RT], o[RT];                                  // of the thread's token and of its dimension
#pragma unroll
      for (int r = 0; r < RT; ++r) l[r] = o[r] = 0.f;
      // lane r has row r's maximum so far and the weight of the last tile's product
      float most = -INFINITY, weight = 0.f;
      const float* qc = ms.qc[seg & 1];
      RowStep* step = ms.step[warp];
      const int rows = w.u.n * d.G;
      // adds the product of tile number i; `keep` and `part` of a step: the sums so far and the product times these
      auto add_product = [&](int i, auto keep, auto part) {
        const uint32_t to = t_o + (i % C::NO) * NP + lanes;
#pragma unroll
        for (int r = 0; r < RT; ++r) o[r] *= keep(step[r]);
        if constexpr (RT == 8) {
          float s[32];
          umma::ld32(to, s);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            o[r] = fmaf(fmaf(fmaf(s[r + 2 * RT], 1.f / kLoP, s[r + RT]), 1.f / kLoP, s[r]), part(step[r]), o[r]);
        } else {
#pragma unroll
          for (int r0 = 0; r0 < RT; r0 += 16) {
            float s[3][16];
#pragma unroll
            for (int i = 0; i < 3; ++i) ld16(to + i * RT + r0, s[i]);
#pragma unroll
            for (int r = 0; r < 16; ++r)
              o[r0 + r] = fmaf(fmaf(fmaf(s[2][r], 1.f / kLoP, s[1][r]), 1.f / kLoP, s[0][r]), part(step[r0 + r]), o[r0 + r]);
          }
        }
      };
      auto add_last = [&](int t) {
        if (t > w.t0)
          add_product(count - 1, [](const RowStep& y) { return y.keep; }, [](const RowStep& y) { return y.last; });
      };
      for (int t = w.t0; t < w.t0 + w.nt; ++t, ++count) {
        const int st = count % C::NS;
        ok = ok && mbar_wait(smem_u32(&ms.s_ready[count & 1]), (count >> 1) & 1);
        // the scales came with the stage: its barrier has completed, this orders the reads
        ok = ok && mbar_wait(smem_u32(&ms.full[st]), (count / C::NS) & 1);
        umma::fence_after();
        const int blk = tid >> 4, b = w.u.b0 + t * kTileBlocks;
        const float ks = ms.ks[st][blk], ev = ms.ev[st][blk], iv = ms.iv[st][blk];
        const int pos = b * kBlock + tid;
        float x[RT];
        {
          float s[N];
          const uint32_t ts = tmem + (count & 1) * N + lanes;
#pragma unroll
          for (int c = 0; c < N; c += 16) ld16(ts + c, s + c);
#pragma unroll
          for (int r = 0; r < RT; ++r) x[r] = fmaf(fmaf(s[r + RT], 1.f / kLoQ, s[r]), ks * qc[r], ev);
        }
        if (w.u.n == 1) {
          const bool seen = ks > 0.f && pos < w.u.hi0 && pos >= w.u.lo0;
#pragma unroll
          for (int r = 0; r < RT; ++r) x[r] = seen ? x[r] : -INFINITY;
        } else {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int i = ms.token[r];
            const bool seen = ks > 0.f && pos < w.u.hi0 + i && (a.window == 0 || pos >= w.u.lo0 + i);
            x[r] = seen ? x[r] : -INFINITY;
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float top = x[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (lane == (r & 31)) ms.wmax[count & 1][warp][r] = top;
        }
        go = named_and(1, 128, ok);
        if (!go) break;
        if (lane < RT) {
          const auto& wm = ms.wmax[count & 1];
          const float top = fmaxf(fmaxf(wm[0][lane], wm[1][lane]), fmaxf(wm[2][lane], wm[3][lane]));
          const float now = fmaxf(most, top);
          RowStep y;
          y.ref = top > -INFINITY ? top - kTop : 0.f;      // hidden: 2^-inf; a NaN stays one
          y.keep = now > -INFINITY ? ex2(most - now) : 1.f;
          y.last = weight * y.keep;
          y.weight = weight = top > -INFINITY ? ex2(top - now) * 0x1p-15f : 0.f;
          most = now;
          step[lane] = y;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const RowStep y = step[r];
          x[r] = ex2(x[r] - y.ref);
          l[r] = fmaf(l[r], y.keep, x[r] * iv * y.weight);
        }
        if (MASS) {
          // The blocks' sums, as log2, for the rows of one token.  Each exchange halves the rows of a lane and
          // doubles the tokens that they are summed over, so that 16 lanes sum RT rows in RT shuffles, not 4 RT.
          float y[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) y[r] = x[r] * iv;
          int row = 0;
#pragma unroll
          for (int o = 8, n = RT / 2; o > 0; o >>= 1, n >>= 1) {
            if (n > 0) {
              const bool up = lane & o;
              row = 2 * row + up;
#pragma unroll
              for (int r = 0; r < n; ++r)
                y[r] = (up ? y[r + n] : y[r]) + __shfl_xor_sync(0xffffffffu, up ? y[r] : y[r + n], o);
            } else {
              y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
            }
          }
          constexpr int EACH = RT < 16 ? 1 : RT / 16;      // rows of a lane, neighbours; of RT = 8 two lanes have one
#pragma unroll
          for (int i = 0; i < EACH; ++i) {
            const int r = row * EACH + i;
            if ((RT >= 16 || !(lane & 1)) && r < rows && b + blk < w.u.b0 + w.u.nb &&
                KVS_DCHECK(d, w.r < a.n_reqs && b >= 0 && b + blk < a.table_stride && w.h * d.G + r < d.Hq))
              a.blk[((size_t)w.r * a.table_stride + b + blk) * d.Hq + w.h * d.G + r] = __log2f(y[i]) + step[r].ref;
          }
        }
        // the previous product is done with the probabilities' buffer
        if (count > 0) ok = ok && mbar_wait(smem_u32(&ms.o_done), (count - 1) & 1);
        umma::fence_after();
        if constexpr (C::NO == 1) add_last(t);             // the next product takes its place
        uint8_t* p = sp + (tid >> 4) * (NP * 16) + (tid & 15);
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          float f = x[r], g = x[r + 1];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint32_t code = float2_to_e5m2x2(f, g);
            p[(r + i * RT) * 16] = (uint8_t)code;
            p[(r + i * RT + 1) * 16] = (uint8_t)(code >> 8);
            const float2 back = e5m2x2_to_float2(code);
            f = (f - back.x) * kLoP;
            g = (g - back.y) * kLoP;
          }
        }
        umma::fence_async_smem();
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.p_ready));
        if constexpr (C::NO > 1) add_last(t);              // under the next product
      }
      if (!go) break;
      // the sums over the tokens; the next segment's queries while the last product runs
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane == (r & 31)) ms.wsum[warp][r] = l[r];
      }
      Walk x = w;
      x.next(a);
      if (x.left > 0) load_q(x, (seg + 1) & 1);
      ok = ok && mbar_wait(smem_u32(&ms.o_done), (count - 1) & 1);
      go = named_and(1, 128, ok);
      umma::fence_after();
      if (!go) break;
      add_product(count - 1, [](const RowStep&) { return 1.f; }, [](const RowStep& y) { return y.weight; });
#pragma unroll
      for (int r = 0; r < RT; ++r) l[r] = ms.wsum[0][r] + ms.wsum[1][r] + ms.wsum[2][r] + ms.wsum[3][r];
      if (!KVS_DCHECK(d, w.u.first >= 0 && w.u.first + w.u.n <= a.total_q && w.h < d.Hkv)) {
      } else if (w.whole) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (r < rows && tid < D)
            out[((size_t)(w.u.first + r / d.G) * d.Hq + w.h * d.G + r % d.G) * D + tid] =
                __float2bfloat16_rn(l[r] == 0.f ? 0.f : o[r] / l[r]);
          if (MASS && r < rows && tid == r) a.lse[(size_t)w.r * d.Hq + w.h * d.G + r] = most + log2f(l[r]);
        }
      } else {
        const size_t rec = (size_t)(2 * blockIdx.x + (w.first ? 0 : 1)) * RT;
#pragma unroll
        for (int r = 0; r < RT; ++r)
          if (r < rows) {
            if (tid < D) a.part_o[(rec + r) * D + tid] = o[r];
            if (tid == r) a.part_ml[rec + r] = make_float2(most, l[r]);
          }
      }
      umma::fence_before();
      ++seg;
      w = x;
    }
    if (!go) paged_error(d, kErrTimeout);
  }
  __syncwarp();
  __syncthreads();
  if (warp == 5) {
    umma::fence_after();
    umma::dealloc(tmem, C::TMEM);
  }
}

// Adds the partials of the unit that CTA blockIdx.x + 1 left in its cut (most CTAs cut none, and their
// blocks here end at once).  Two rows to a block; a warp has a row and every fourth part, a lane four dimensions.
constexpr int kJoinRows = 2, kJoinGroups = 4, kJoinThreads = kJoinRows * kJoinGroups * 32;
template <int D, int RT, bool MASS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const PagedAttend a) {
  __shared__ float4 sums[kJoinGroups - 1][kJoinRows][D / 4];
  launch_dependents();
  wait_previous();
  const PagedDev& d = a.d;
  const int4 cut = *reinterpret_cast<const int4*>(a.cuts + (blockIdx.x + 1) * 8);
  const int r = cut.x, h = cut.y, c0 = blockIdx.x, n = cut.z - c0 + 1;
  if (cut.z == 0) return;
  if (!KVS_DCHECK(d, r >= 0 && r < a.n_reqs && h >= 0 && h < d.Hkv && cut.z > c0 && cut.z <= (int)gridDim.x && cut.w >> 1 == 0)) return;
  const Unit u = unit_of(a, r);
  if (!KVS_DCHECK(d, u.first >= 0 && u.n > 0 && u.first + u.n <= a.total_q)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % kJoinRows, group = warp / kJoinRows;
  const int row = blockIdx.y * kJoinRows + mine;
  const bool live = row < u.n * d.G;
  auto rec_of = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0 ? cut.w : 0)) * RT + row; };
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    for (int i = lane; i < n; i += 32) top = fmaxf(top, a.part_ml[rec_of(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top > -INFINITY ? top : 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      float f = 0.f;                         // the weight of part i0 + lane
      if (i0 + lane < n) {
        const float2 ml = a.part_ml[rec_of(i0 + lane)];
        f = ex2(ml.x - ref);
        sum = fmaf(ml.y, f, sum);
      }
      const int most = min(32, n - i0);
#pragma unroll 8
      for (int i = group; i < most; i += kJoinGroups) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        if (lane < D / 4) {
          const float4 v = reinterpret_cast<const float4*>(a.part_o + rec_of(i0 + i) * D)[lane];
          acc.x = fmaf(v.x, w, acc.x);
          acc.y = fmaf(v.y, w, acc.y);
          acc.z = fmaf(v.z, w, acc.z);
          acc.w = fmaf(v.w, w, acc.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (group > 0 && lane < D / 4) sums[group - 1][mine][lane] = acc;
  }
  __syncthreads();
  if (!live || group > 0) return;
  const int hq = h * d.G + row % d.G;
  if (lane < D / 4) {
#pragma unroll
    for (int g = 1; g < kJoinGroups; ++g) {
      const float4 v = sums[g - 1][mine][lane];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    uint2 raw;
    raw.x = *reinterpret_cast<const uint32_t*>(&lo);
    raw.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + ((size_t)(u.first + row / d.G) * d.Hq + hq) * D + lane * 4) = raw;
  }
  if (MASS && lane == 0) a.lse[(size_t)r * d.Hq + hq] = top + log2f(sum);
}

template <int D, int RT, bool MASS>
cudaError_t launch(const PagedAttend& a, int grid, cudaStream_t st) {
  using C = Cfg<D, RT>;
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_optin_once(opted, decode_kernel<D, RT, MASS>, C::SMEM);
  if (e != cudaSuccess) return e;
  decode_kernel<D, RT, MASS><<<grid, kThreads, C::SMEM, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid - 1, (a.max_q_len * a.d.G + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, RT, MASS>, a);
}

template <int D>
cudaError_t launch_d(const PagedAttend& a, int rows, int grid, cudaStream_t st) {
  const bool mass = a.mass != nullptr;
  switch (rows) {
    case 8: return mass ? launch<D, 8, true>(a, grid, st) : launch<D, 8, false>(a, grid, st);
    case 16: return mass ? launch<D, 16, true>(a, grid, st) : launch<D, 16, false>(a, grid, st);
    case 32: return mass ? launch<D, 32, true>(a, grid, st) : cudaErrorInvalidValue;      // 17 to 32 heads a group
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int paged_decode_ctas_per_sm() { return kCtasPerSm; }

// rows: 8, 16 or (with block masses) 32, at least max_q_len * G.
cudaError_t launch_paged_decode(const PagedAttend& a, int rows, int grid, cudaStream_t st) {
  if ((long long)a.max_q_len * a.d.G > rows || (a.mass && (!a.blk || !a.lse))) return cudaErrorInvalidValue;
  return a.d.D == 64 ? launch_d<64>(a, rows, grid, st) : launch_d<128>(a, rows, grid, st);
}

}  // namespace kvs
