// Append and gather of the paged cache: tokens to and from the codes at their slots.
//
// Append: for each page, KV head and cache (K or V), with x the run of new tokens of that
// page: scale s = max(old scale, 2^e), 2^e the smallest power of two with max|x| <= 448 2^e
// (old scale dropped when the run starts the page); codes = rn(x / s); the page's other
// codes c become rn(c * old / s) if s grew, 0 if the page starts.  x / s and c * old / s
// are products with powers of two, so each value is rounded once, to its code.
//
// How: a warp owns one (run, KV head, cache): it reads the run's rows once, keeps them as
// they came over the maximum and the conversion, and writes whole 16-byte pieces.  K
// pieces are 16 dimensions of a token; V pieces are 16 tokens of a dimension, so for V a
// lane reads four dimensions of each token (whole rows stay coalesced) and the pieces
// pass through shared memory once, to leave in order.  The maximum is taken over the bits
// of |x|, two bf16 at a time, which also shows whether an infinity or a NaN is there; only
// then are values looked at one by one.  The row that starts a run leads it; others exit, so
// a batch of single tokens is one warp per token and cache, and rows of a long prompt are
// taken sixteen to a warp to spare idle warps.  Bound by latency: 16 tokens of 4 x 128 take
// 2.7 us, 26295 rows 17 us (81 MB, 4.8 TB/s).
//
// Gather: code * scale, one product.  A lane writes 16 bytes of a K row; V's pages are
// shifted into row order, two pages of four dimensions a lane.  64662 rows of 4 x 128 take
// 38 us (199 MB, 5.2 TB/s), 16 rows 2 us.
#include "paged.cuh"

namespace kvs {
namespace {

constexpr int kWarps = 4;

// N consecutive inputs as they are in memory.
template <int IN, int N>
struct Raw {
  static constexpr bool B = IN == KVS_BF16;
  static constexpr int W = B ? N / 2 : N;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const char* p = static_cast<const char*>(base) + elem * (B ? 2 : 4);
    if constexpr (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    }
  }
  // The largest |x| as bits: of float32, or of two bf16 in halves.
  __device__ __forceinline__ uint32_t top(uint32_t so_far) const {
#pragma unroll
    for (int i = 0; i < W; ++i)
      so_far = B ? __vmaxu2(so_far, w[i] & 0x7fff7fffu) : max(so_far, w[i] & 0x7fffffffu);
    return so_far;
  }
  // The same without what is not finite; NaN becomes 0.
  __device__ __forceinline__ uint32_t clean(uint32_t so_far, bool& nan) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (B) {
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
          const uint32_t a = w[i] >> k & 0x7fffu;
          if (a > 0x7f80u) { nan = true; w[i] &= ~(0xffffu << k); }
          if (a < 0x7f80u) so_far = __vmaxu2(so_far, a);
        }
      } else {
        const uint32_t a = w[i] & 0x7fffffffu;
        if (a > 0x7f800000u) { nan = true; w[i] = 0; }
        if (a < 0x7f800000u) so_far = max(so_far, a);
      }
    }
    return so_far;
  }
  __device__ __forceinline__ float at(int i) const {
    return B ? __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
  }
};
template <int IN>
__device__ __forceinline__ float bits_to_float(uint32_t top) {
  return IN == KVS_BF16 ? __uint_as_float(max(top << 16, top & 0xffff0000u)) : __uint_as_float(top);
}
__device__ __forceinline__ bool is_finite(float v) { return __float_as_uint(v) < 0x7f800000u; }

template <int OUT>
__device__ __forceinline__ void store4(void* base, size_t elem, const float v[4]) {
  if constexpr (OUT == KVS_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 raw;
    raw.x = *reinterpret_cast<const uint32_t*>(&a);
    raw.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + elem) = raw;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + elem) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

__device__ __forceinline__ uint32_t requantise4(uint32_t codes, float ratio) {
  const float2 a = e4m3x2_to_float2(codes & 0xffffu), b = e4m3x2_to_float2(codes >> 16);
  return float2_to_e4m3x2(a.x * ratio, a.y * ratio) | (float2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

// The warp's largest |x|, and whether any lane has one that is not finite.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// A run: rows of one page, at most 16.  Lane t < 16 holds the row of slot t in the page (-1: none).
struct Run {
  int page, row;
  uint32_t have;
};

template <int IN, int D>
__device__ void store_k(const PagedDev& d, int layer, int head, const void* x, const Run& run, int lane) {
  constexpr int CH = D / 16;                       // pieces of a token
  constexpr int NP = (16 * CH + 31) / 32;          // pieces of a lane
  const size_t at = (size_t)run.page * d.Hkv + head;
  uint8_t* base = d.k + layer * d.layer_bytes + at * (16 * D);
  float* scale_at = &d.scales[layer * d.layer_scales + at].x;
  const bool fresh = run.have & 1;
  const float old = fresh ? exp2_int(kScaleMinExp) : fmaxf(*scale_at, exp2_int(kScaleMinExp));
  Raw<IN, 16> v[NP];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = i * 32 + lane, t = piece / CH, c = piece % CH;
    const int row = __shfl_sync(0xffffffffu, run.row, t & 15);
    if (piece < 16 * CH && row >= 0) v[i].load(x, ((size_t)row * d.Hkv + head) * D + c * 16);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) top = v[i].top(top);
  float amax = warp_max(bits_to_float<IN>(top));
  if (!is_finite(amax)) {
    bool nan = false;
    top = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) top = v[i].clean(top, nan);
    amax = warp_max(bits_to_float<IN>(top));
    if (nan) paged_error(d, kErrState);
  }
  const float scale = fmaxf(old, exp2_int(scale_exp(amax)));
  const float inv = 1.f / scale, ratio = old * inv;      // powers of two: exact
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = i * 32 + lane, t = piece / CH, c = piece % CH;
    if (piece >= 16 * CH) continue;
    uint4* dst = reinterpret_cast<uint4*>(base + k_code(D, t, c * 16));
    uint4 w = make_uint4(0, 0, 0, 0);
    if (run.have >> t & 1) {
      uint32_t* p = &w.x;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        p[u] = float2_to_e4m3x2(v[i].at(4 * u) * inv, v[i].at(4 * u + 1) * inv) |
               (float2_to_e4m3x2(v[i].at(4 * u + 2) * inv, v[i].at(4 * u + 3) * inv) << 16);
    } else if (!fresh) {
      if (ratio == 1.f) continue;
      w = *dst;
      w.x = requantise4(w.x, ratio); w.y = requantise4(w.y, ratio);
      w.z = requantise4(w.z, ratio); w.w = requantise4(w.w, ratio);
    }
    *dst = w;
  }
  __syncwarp();                                    // every lane has read the old scale
  if (lane == 0) *scale_at = scale;
}

// stage: 16 * D bytes of the warp's shared memory.
template <int IN, int D>
__device__ void store_v(const PagedDev& d, int layer, int head, const void* x, const Run& run, int lane,
                        uint4* stage) {
  const size_t at = (size_t)run.page * d.Hkv + head;
  uint8_t* base = d.v + layer * d.layer_bytes + at * (16 * D);
  float* scale_at = &d.scales[layer * d.layer_scales + at].y;
  const bool fresh = run.have & 1, mine = lane < D / 4;
  const float old = fresh ? exp2_int(kScaleMinExp) : fmaxf(*scale_at, exp2_int(kScaleMinExp));
  Raw<IN, 4> v[16];
  uint32_t top = 0;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const int row = __shfl_sync(0xffffffffu, run.row, t);
    if (row >= 0 && mine) v[t].load(x, ((size_t)row * d.Hkv + head) * D + lane * 4);
    else v[t].zero();
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) top = v[t].top(top);
  float amax = warp_max(bits_to_float<IN>(top));
  if (!is_finite(amax)) {
    bool nan = false;
    top = 0;
#pragma unroll
    for (int t = 0; t < 16; ++t) top = v[t].clean(top, nan);
    amax = warp_max(bits_to_float<IN>(top));
    if (nan) paged_error(d, kErrState);
  }
  const float scale = fmaxf(old, exp2_int(scale_exp(amax)));
  const float inv = 1.f / scale, ratio = old * inv;
  __syncwarp();                                    // the stage's last use, and the old scale's reads
  if (mine) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (!fresh && run.have != 0xffffu) {
        w = reinterpret_cast<const uint4*>(base)[lane * 4 + u];
        if (ratio != 1.f) {
          w.x = requantise4(w.x, ratio); w.y = requantise4(w.y, ratio);
          w.z = requantise4(w.z, ratio); w.w = requantise4(w.w, ratio);
        }
      }
      uint32_t* p = &w.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t codes = float2_to_e4m3x2(v[4 * j].at(u) * inv, v[4 * j + 1].at(u) * inv) |
                               (float2_to_e4m3x2(v[4 * j + 2].at(u) * inv, v[4 * j + 3].at(u) * inv) << 16);
        const uint32_t h = run.have >> (4 * j);
        const uint32_t mask = (h & 1 ? 0xffu : 0) | (h & 2 ? 0xff00u : 0) | (h & 4 ? 0xff0000u : 0) |
                              (h & 8 ? 0xff000000u : 0);
        p[j] = (p[j] & ~mask) | (codes & mask);
      }
      stage[lane * 4 + (u ^ (lane >> 1 & 3))] = w;         // spread over the banks
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < (D + 31) / 32; ++i) {
    const int q = i * 32 + lane, from = q / 4;
    if (q < D) reinterpret_cast<uint4*>(base)[from * 4 + ((q & 3) ^ (from >> 1 & 3))] = stage[q];
  }
  if (lane == 0) *scale_at = scale;
}

// grid: x groups of `per` rows, kWarps to a CTA; y KV heads; z 0 = K, 1 = V.
template <int IN, int D>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const PagedDev d, int layer, int n_rows, int per,
                                                             const int32_t* __restrict__ slots, const void* k,
                                                             const void* v) {
  __shared__ uint4 stage[kWarps][D];
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
  if (first >= n_rows) return;
  // Lane l has the slot of row first - 1 + l: the row before, the warp's rows and what their runs may reach.
  const long long mine = first - 1 + lane;
  const int sl = mine >= 0 && mine < n_rows ? __ldg(slots + mine) : -1;
  const int before = __shfl_up_sync(0xffffffffu, sl, 1);
  const bool leads = lane >= 1 && lane <= per && sl >= 0 && !(before >= 0 && before >> 4 == sl >> 4);
  for (uint32_t todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1, i = (int)first - 1 + l;
    const int page = __shfl_sync(0xffffffffu, sl, l) >> 4;
    if (page >= d.num_pages) {
      if (lane == 0) paged_error(d, kErrState);
      continue;
    }
    // the run: rows i, i + 1, ... while they stay in the page
    const int s = __shfl_sync(0xffffffffu, sl, (l + lane) & 31);
    const uint32_t in = __ballot_sync(0xffffffffu, lane < 16 && l + lane < 32 && s >= 0 && s >> 4 == page);
    const int len = __ffs(~in) - 1;
    Run run{page, -1, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int off = __shfl_sync(0xffffffffu, s, j) & 15;
      if (j < len) {
        if (lane == off && KVS_DCHECK(d, i + j < n_rows)) run.row = i + j;
        run.have |= 1u << off;
      }
    }
    if (blockIdx.z == 0) store_k<IN, D>(d, layer, head, k, run, lane);
    else store_v<IN, D>(d, layer, head, v, run, lane, stage[threadIdx.x >> 5]);
  }
}

// A warp reads the codes of up to 16 rows at a time, run by run.
template <int OUT, int D>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const PagedDev d, int layer, int n_rows, int per,
                                                             const int32_t* __restrict__ slots, void* k, void* v) {
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
  if (first >= n_rows) return;
  const int i0 = (int)first, n = min(per, n_rows - i0);
  int s = lane < n ? __ldg(slots + i0 + lane) : -1;
  if (s >= 0 && (s >> 4) >= d.num_pages) {
    paged_error(d, kErrState);
    s = -1;
  }
  const float2 sc = s >= 0 ? d.scales[layer * d.layer_scales + (size_t)(s >> 4) * d.Hkv + head] : make_float2(0.f, 0.f);
  if (blockIdx.z == 0) {
    // a lane writes 16 bytes of a row
    constexpr int E = OUT == KVS_BF16 ? 8 : 4, LPR = D / E, RPP = 32 / LPR > 0 ? 32 / LPR : 1;
    const uint8_t* kbase = d.k + layer * d.layer_bytes;
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += RPP) {
      if (r0 >= n) break;
      const int j = r0 + lane / LPR, dim = lane % LPR * E;
      const int sj = __shfl_sync(0xffffffffu, s, j & 15);
      const float scale = __shfl_sync(0xffffffffu, sc.x, j & 15);
      if (j >= n || j >= r0 + RPP) continue;
      uint32_t c[E / 4] = {};
      if (sj >= 0) {
        const uint8_t* at = kbase + ((size_t)(sj >> 4) * d.Hkv + head) * (16 * D) + k_code(D, sj & 15, dim);
        if constexpr (E == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
          c[0] = v.x;
          c[1] = v.y;
        } else {
          c[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
        }
      }
      float f[E];
#pragma unroll
      for (int u = 0; u < E / 2; ++u) {
        const float2 v = e4m3x2_to_float2(c[u / 2] >> (u & 1 ? 16 : 0) & 0xffffu);
        f[2 * u] = v.x * scale;
        f[2 * u + 1] = v.y * scale;
      }
      const size_t e = ((size_t)(i0 + j) * d.Hkv + head) * D + dim;
      if constexpr (E == 8) {
        uint4 o;
        uint32_t* p = &o.x;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * u], f[2 * u + 1]);
          p[u] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(k) + e) = o;
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(k) + e) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
    return;
  }
  const bool mine = lane < D / 4;
  const uint8_t* vbase = d.v + layer * d.layer_bytes;
  // Rows in page order, which may pass into another page: the usual case, of whole contexts.  Both pages'
  // bytes are then shifted into row order at once.
  const int s0 = __shfl_sync(0xffffffffu, s, 0), off = s0 & 15, cut = 16 - off;
  const int s1 = __shfl_sync(0xffffffffu, s, cut & 15);
  const bool in_order = lane >= n || s == (lane < cut ? s0 + lane : s1 + lane - cut);
  const bool two = off > 0 && cut < n;
  if (s0 >= 0 && per == 16 && __all_sync(0xffffffffu, in_order) && (!two || (s1 >= 0 && (s1 & 15) == 0))) {
    const float sa = __shfl_sync(0xffffffffu, sc.y, 0), sb = __shfl_sync(0xffffffffu, sc.y, cut & 15);
    if (!mine) return;
    const uint4* pa = reinterpret_cast<const uint4*>(vbase + ((size_t)(s0 >> 4) * d.Hkv + head) * (16 * D)) + lane * 4;
    const uint4* pb = reinterpret_cast<const uint4*>(vbase + ((size_t)((two ? s1 : s0) >> 4) * d.Hkv + head) * (16 * D)) + lane * 4;
    uint32_t c[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 x = __ldg(pa + u), y = two ? __ldg(pb + u) : make_uint4(0, 0, 0, 0);
      c[u][0] = x.x; c[u][1] = x.y; c[u][2] = x.z; c[u][3] = x.w;
      c[u][4] = y.x; c[u][5] = y.y; c[u][6] = y.z; c[u][7] = y.w;
    }
    const int words = off >> 2, bits = (off & 3) * 8;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < words) {
#pragma unroll
          for (int i = 0; i < 7; ++i) c[u][i] = c[u][i + 1];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[u][i] = __funnelshift_r(c[u][i], c[u][i + 1], bits);
    }
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      float2 f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) f[u] = e4m3x2_to_float2(c[u][j / 4] >> (j & 2 ? 16 : 0) & 0xffffu);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (j + k < n) {
          const float scale = j + k < cut ? sa : sb;
          const float o[4] = {(k ? f[0].y : f[0].x) * scale, (k ? f[1].y : f[1].x) * scale,
                              (k ? f[2].y : f[2].x) * scale, (k ? f[3].y : f[3].x) * scale};
          store4<OUT>(v, ((size_t)(i0 + j + k) * d.Hkv + head) * D + lane * 4, o);
        }
    }
    return;
  }
  int page = -2;
  uint4 w[4];
  for (int j = 0; j < n; ++j) {
    const int sj = __shfl_sync(0xffffffffu, s, j);
    const float scale = __shfl_sync(0xffffffffu, sc.y, j);
    if (!mine) continue;
    const int pj = sj < 0 ? -1 : sj >> 4;
    if (pj != page) {
      page = pj;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w[u] = page < 0 ? make_uint4(0, 0, 0, 0)
                        : __ldg(reinterpret_cast<const uint4*>(d.v + layer * d.layer_bytes + ((size_t)page * d.Hkv + head) * (16 * D)) +
                                lane * 4 + u);
    }
    const int word = (sj & 15) >> 2, shift = (sj & 3) * 8;
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t x = word == 0 ? w[u].x : word == 1 ? w[u].y : word == 2 ? w[u].z : w[u].w;
      f[u] = e4m3x2_to_float2((x >> shift) & 0xffu).x * scale;
    }
    store4<OUT>(v, ((size_t)(i0 + j) * d.Hkv + head) * D + lane * 4, f);
  }
}

// Rows of a warp: one up to 8192 warps, else a page's worth.  One prompt's rows, 4 KV heads of 128, append with
// one against sixteen: 256 rows 2.9 against 3.8 us, 1024 alike, 2048 5.2 against 4.2, 8000 12.8 against 6.8;
// 256 single tokens 4.0 against 22, 4000 25 against 36.
int rows_per_warp(int n_rows, int Hkv) { return (long long)n_rows * Hkv * 2 <= 8192 ? 1 : 16; }

template <int DT, int D>
cudaError_t append_d(const PagedDev& d, int layer, int n_rows, const int32_t* slots, const void* k, const void* v,
                     cudaStream_t st) {
  const int per = rows_per_warp(n_rows, d.Hkv);
  const dim3 grid((unsigned)cdiv64(n_rows, (long long)per * kWarps), d.Hkv, 2);
  append_kernel<DT, D><<<grid, kWarps * 32, 0, st>>>(d, layer, n_rows, per, slots, k, v);
  return cudaGetLastError();
}

template <int DT, int D>
cudaError_t gather_d(const PagedDev& d, int layer, int n_rows, const int32_t* slots, void* k, void* v,
                     cudaStream_t st) {
  const int per = rows_per_warp(n_rows, d.Hkv);
  const dim3 grid((unsigned)cdiv64(n_rows, (long long)per * kWarps), d.Hkv, 2);
  gather_kernel<DT, D><<<grid, kWarps * 32, 0, st>>>(d, layer, n_rows, per, slots, k, v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedDev& d, int layer, int n_rows, const int32_t* slots, const void* k,
                                const void* v, cudaStream_t st) {
  const bool b = d.in_dtype == KVS_BF16;
  switch (d.D) {
    case 16: return b ? append_d<KVS_BF16, 16>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 16>(d, layer, n_rows, slots, k, v, st);
    case 32: return b ? append_d<KVS_BF16, 32>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 32>(d, layer, n_rows, slots, k, v, st);
    case 64: return b ? append_d<KVS_BF16, 64>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 64>(d, layer, n_rows, slots, k, v, st);
    default: return b ? append_d<KVS_BF16, 128>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 128>(d, layer, n_rows, slots, k, v, st);
  }
}

cudaError_t launch_paged_gather(const PagedDev& d, int layer, int n_rows, const int32_t* slots, void* k, void* v,
                                cudaStream_t st) {
  const bool b = d.in_dtype == KVS_BF16;
  switch (d.D) {
    case 16: return b ? gather_d<KVS_BF16, 16>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 16>(d, layer, n_rows, slots, k, v, st);
    case 32: return b ? gather_d<KVS_BF16, 32>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 32>(d, layer, n_rows, slots, k, v, st);
    case 64: return b ? gather_d<KVS_BF16, 64>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 64>(d, layer, n_rows, slots, k, v, st);
    default: return b ? gather_d<KVS_BF16, 128>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 128>(d, layer, n_rows, slots, k, v, st);
  }
}

}  // namespace kvs
