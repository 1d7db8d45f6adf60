// Paged attention on the CUDA cores (any head_dim, group and input type) and the block
// masses of either attend kernel.
//
// For query row t of request r at position p, KV head h and its query heads g:
//   s_gj = q_g . k_j / sqrt(D),  m_g = max_j s_gj,  o_g = sum_j 2^(s_gj - m_g) v_j / sum_j 2^(s_gj - m_g)
// (logits in log2 units) over the visible positions max(0, p - window + 1) .. p.
//
// How: a CTA takes one (row, KV head, part of the range); its four warps take pages in
// turn, each with a running maximum, sum and output of eight heads in registers.  For the
// logits a lane pair owns a token; for the output a lane owns dimensions, whose sixteen
// tokens are one 16-byte piece of V.  The range is cut in parts when rows are few, and a
// second kernel joins the parts.  All arithmetic is float32: this is the path of float32
// inputs, whose outputs keep float32 accuracy, and of shapes the tensor-core kernels do
// not take.  Bound by the FMA pipe, not by memory (19 TFLOP/s on a prompt of 8192 tokens,
// a fiftieth of the tensor-core kernel's rate).  The mass kernel reads 4 bytes a head and
// block (64 ragged contexts: 17 MB, a few us behind the attend).
#include "paged.cuh"

namespace kvs {
namespace {

constexpr int kWarps = 4;
constexpr int kHeads = 8;                // query heads of one pass over the range
constexpr float kLog2e = 1.4426950408889634f;

template <int IN>
__device__ __forceinline__ float load1(const void* p, size_t i) {
  if constexpr (IN == KVS_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <int OUT>
__device__ __forceinline__ void store1(void* p, size_t i, float v) {
  if constexpr (OUT == KVS_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// Row t of the call: its request, whether it is computed, and its visible positions [lo, hi).
struct RowRange {
  int r;
  bool live;
  int lo, hi;
};
__device__ __forceinline__ RowRange row_range(const PagedAttend& a, int t) {
  RowRange x{t, true, 0, 0};
  int first = t, n = 1;
  if (a.row_start) {
    if (t < __ldg(a.row_start) || t >= __ldg(a.row_start + a.n_reqs)) { x.live = false; return x; }
    x.r = request_of(a.row_start, a.n_reqs, t);
    first = __ldg(a.row_start + x.r);
    n = __ldg(a.row_start + x.r + 1) - first;
    if (t < first || t - first >= a.max_q_len) { x.live = false; return x; }
  }
  const int len = min(max(__ldg(a.kv_len + x.r), 0), a.table_stride * kBlock);
  const int p = len - n + (t - first);           // the row's position
  x.hi = min(max(p + 1, 0), len);
  x.lo = a.window > 0 ? max(0, x.hi - a.window) : 0;
  return x;
}

// What the one row of request r sees, in a call of single-token rows.
__device__ __forceinline__ RowRange request_range(const PagedAttend& a, int r) {
  RowRange x{r, true, 0, 0};
  int n = 1;
  if (a.row_start) {
    const int first = __ldg(a.row_start + r);
    n = __ldg(a.row_start + r + 1) - first;
    x.live = n > 0 && first >= 0 && first < a.total_q;
  }
  const int len = min(max(__ldg(a.kv_len + r), 0), a.table_stride * kBlock);
  x.hi = min(max(len - n + 1, 0), len);
  x.lo = a.window > 0 ? max(0, x.hi - a.window) : 0;
  return x;
}

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32) general_kernel(const PagedAttend a) {
  constexpr int ND = (D + 31) / 32;              // dimensions of a lane
  constexpr int CH = D / 16;
  __shared__ float s_q[kHeads][D];
  __shared__ float s_p[kWarps][kHeads][16];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ float s_o[kWarps][kHeads][D];
  const PagedDev& d = a.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, head = blockIdx.y, part = blockIdx.z;
  const RowRange x = row_range(a, t);
  if (!x.live) return;
  const int b0 = x.lo / kBlock, b1 = (x.hi + kBlock - 1) / kBlock;
  const int nb = max(b1 - b0, 0);
  const int c0 = b0 + (int)((long long)nb * part / a.splits), c1 = b0 + (int)((long long)nb * (part + 1) / a.splits);
  const float qk = kLog2e / sqrtf((float)D);
  for (int g0 = 0; g0 < d.G; g0 += kHeads) {
    const int ng = min(kHeads, d.G - g0);
    __syncthreads();
    for (int i = threadIdx.x; i < kHeads * D; i += kWarps * 32) {
      const int g = i / D;
      s_q[g][i % D] = g < ng ? load1<DT>(a.q, ((size_t)t * d.Hq + head * d.G + g0 + g) * D + i % D) * qk : 0.f;
    }
    __syncthreads();
    float m[kHeads], l[kHeads], o[kHeads][ND];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[g][i] = 0.f;
    }
    for (int b = c0 + warp; b < c1; b += kWarps) {
      const int page = __ldg(a.table + (size_t)x.r * a.table_stride + b);
      if (page < 0 || page >= d.num_pages) {
        if (lane == 0) paged_error(d, kErrState);
        if (a.blk)
          for (int g = lane; g < ng; g += 32)
            a.blk[((size_t)x.r * a.table_stride + b) * d.Hq + head * d.G + g0 + g] = -INFINITY;
        continue;
      }
      if (!KVS_DCHECK(d, x.r < a.n_reqs && b >= 0 && b < a.table_stride)) continue;
      const size_t at = (size_t)page * d.Hkv + head;
      const float2 sc = d.scales[a.layer * d.layer_scales + at];
      const uint8_t* kb = d.k + a.layer * d.layer_bytes + at * (16 * D);
      const uint8_t* vb = d.v + a.layer * d.layer_bytes + at * (16 * D);
      const int tok = lane >> 1;
      float s[kHeads];
#pragma unroll
      for (int g = 0; g < kHeads; ++g) s[g] = 0.f;
      for (int c = lane & 1; c < CH; c += 2) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(kb + k_code(D, tok, c * 16)));
        const uint32_t* pw = &w.x;
        float kf[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 e = e4m3x2_to_float2(pw[u] & 0xffffu), f = e4m3x2_to_float2(pw[u] >> 16);
          kf[4 * u] = e.x; kf[4 * u + 1] = e.y; kf[4 * u + 2] = f.x; kf[4 * u + 3] = f.y;
        }
#pragma unroll
        for (int g = 0; g < kHeads; ++g)
#pragma unroll
          for (int u = 0; u < 16; ++u) s[g] = fmaf(s_q[g][c * 16 + u], kf[u], s[g]);
      }
      const int pos = b * kBlock + tok;
      const bool seen = pos >= x.lo && pos < x.hi;
      float f[kHeads];
#pragma unroll
      for (int g = 0; g < kHeads; ++g) {
        s[g] += __shfl_xor_sync(0xffffffffu, s[g], 1);
        s[g] = seen ? s[g] * sc.x : -INFINITY;
        float top = s[g];
#pragma unroll
        for (int k = 2; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float now = fmaxf(m[g], top);      // finite: a visited page has a visible token
        f[g] = exp2f(m[g] - now);
        m[g] = now;
        const float p = exp2f(s[g] - now);
        float sum = p;
#pragma unroll
        for (int k = 2; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        l[g] = l[g] * f[g] + sum;
        if (!(lane & 1)) s_p[warp][g][tok] = p;
        if (a.blk && lane == 0 && g < ng)
          a.blk[((size_t)x.r * a.table_stride + b) * d.Hq + head * d.G + g0 + g] = log2f(sum) + now;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int dim = lane + 32 * i;
        if (dim >= D) continue;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(vb + dim * 16));
        const uint32_t* pw = &w.x;
        float vf[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 e = e4m3x2_to_float2(pw[u] & 0xffffu), ff = e4m3x2_to_float2(pw[u] >> 16);
          vf[4 * u] = e.x * sc.y; vf[4 * u + 1] = e.y * sc.y; vf[4 * u + 2] = ff.x * sc.y; vf[4 * u + 3] = ff.y * sc.y;
        }
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
          float acc = o[g][i] * f[g];
#pragma unroll
          for (int u = 0; u < 16; ++u) acc = fmaf(s_p[warp][g][u], vf[u], acc);
          o[g][i] = acc;
        }
      }
      __syncwarp();
    }
    // join the warps
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      if (lane == 0) { s_m[warp][g] = m[g]; s_l[warp][g] = l[g]; }
#pragma unroll
      for (int i = 0; i < ND; ++i)
        if (lane + 32 * i < D) s_o[warp][g][lane + 32 * i] = o[g][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ng * D; i += kWarps * 32) {
      const int g = i / D, dim = i % D;
      float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][g]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float e = exp2f(s_m[w][g] - ref);
        sum += s_l[w][g] * e;
        acc += s_o[w][g][dim] * e;
      }
      const int hq = head * d.G + g0 + g;
      if (a.splits == 1) {
        store1<DT>(a.out, ((size_t)t * d.Hq + hq) * D + dim, sum == 0.f ? 0.f : acc / sum);
        if (a.lse && dim == 0) a.lse[(size_t)x.r * d.Hq + hq] = top + log2f(sum);
      } else {
        const size_t rec = ((size_t)t * d.Hq + hq) * a.splits + part;
        a.part_o[rec * D + dim] = acc;
        if (dim == 0) a.part_ml[rec] = make_float2(top, sum);
      }
    }
  }
}

// Joins the parts of one (row, query head): a warp each.
template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32) general_join_kernel(const PagedAttend a) {
  const PagedDev& d = a.d;
  const int lane = threadIdx.x & 31;
  const long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= (long long)a.total_q * d.Hq) return;
  const int t = (int)(u / d.Hq), hq = (int)(u % d.Hq);
  const RowRange x = row_range(a, t);
  if (!x.live) return;
  const size_t rec = (size_t)u * a.splits;
  float top = -INFINITY, sum = 0.f;
  for (int k = 0; k < a.splits; ++k) top = fmaxf(top, a.part_ml[rec + k].x);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int k = 0; k < a.splits; ++k) sum += a.part_ml[rec + k].y * exp2f(a.part_ml[rec + k].x - ref);
  for (int dim = lane; dim < D; dim += 32) {
    float acc = 0.f;
    for (int k = 0; k < a.splits; ++k) acc += a.part_o[(rec + k) * D + dim] * exp2f(a.part_ml[rec + k].x - ref);
    store1<DT>(a.out, (size_t)u * D + dim, sum == 0.f ? 0.f : acc / sum);
  }
  if (a.lse && lane == 0) a.lse[(size_t)x.r * d.Hq + hq] = top + log2f(sum);
}

// Block masses: the query heads over a warp's lanes, four blocks at a time.  The attend left
// log2 of each head's weight sum in the block and of its whole sum.
constexpr int kMassBlocks = 16;          // of a warp
__global__ void __launch_bounds__(kWarps * 32) mass_kernel(const PagedAttend a) {
  const int lane = threadIdx.x & 31, r = blockIdx.x, Hq = a.d.Hq;
  const RowRange x = request_range(a, r);
  const int b1 = x.live && x.hi > x.lo ? (x.hi + kBlock - 1) / kBlock : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = x.lo / kBlock + (blockIdx.y * kWarps + (threadIdx.x >> 5)) * kMassBlocks;
  for (int i = 0, c = first; c < b1; ++i) {
    uint32_t best[4] = {0u, 0u, 0u, 0u};               // of numbers >= 0, whose bits are in their order
    for (int h = lane; h < Hq; h += 32) {
      const float lse = a.lse[(size_t)r * Hq + h];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float s = c + k < b1 ? a.blk[((size_t)r * a.table_stride + c + k) * Hq + h] : -INFINITY;
        if (s > -INFINITY) best[k] = max(best[k], __float_as_uint(exp2f(s - lse)));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      best[k] = __reduce_max_sync(0xffffffffu, best[k]);
      if (lane == 0 && c + k < b1) a.mass[(size_t)r * a.table_stride + c + k] = __uint_as_float(best[k]);
    }
    c += 4;
    if ((i + 1) % (kMassBlocks / 4) == 0) c += (gridDim.y * kWarps - 1) * kMassBlocks;   // a grid shorter than the table
  }
}

__global__ void check_rows_kernel(const PagedAttend a) { report_rows(a, blockDim.x); }

template <int DT, int D>
cudaError_t general_d(const PagedAttend& a, cudaStream_t st) {
  const dim3 grid(a.total_q, a.d.Hkv, a.splits);
  general_kernel<DT, D><<<grid, kWarps * 32, 0, st>>>(a);
  if (a.splits > 1)
    general_join_kernel<DT, D><<<(unsigned)cdiv64((long long)a.total_q * a.d.Hq, kWarps), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_general(const PagedAttend& a, cudaStream_t st) {
  if (a.row_start) check_rows_kernel<<<1, 256, 0, st>>>(a);
  const bool b = a.d.in_dtype == KVS_BF16;
  switch (a.d.D) {
    case 16: return b ? general_d<KVS_BF16, 16>(a, st) : general_d<KVS_F32, 16>(a, st);
    case 32: return b ? general_d<KVS_BF16, 32>(a, st) : general_d<KVS_F32, 32>(a, st);
    case 64: return b ? general_d<KVS_BF16, 64>(a, st) : general_d<KVS_F32, 64>(a, st);
    default: return b ? general_d<KVS_BF16, 128>(a, st) : general_d<KVS_F32, 128>(a, st);
  }
}

cudaError_t launch_paged_mass(const PagedAttend& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.stream = st;
  const int64_t ctas = cdiv64(a.table_stride, kWarps * kMassBlocks);
  cfg.gridDim = dim3(a.n_reqs, (unsigned)(ctas < 65535 ? ctas : 65535));
  cfg.blockDim = dim3(kWarps * 32);
  return cudaLaunchKernelEx(&cfg, mass_kernel, a);
}

}  // namespace kvs
