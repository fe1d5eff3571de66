// LSE combine: merge n partial attention results of the same rows through their LSEs.
//
// Used for the public lse_merge (shard partials, "vLLM PR #54012 (FlashInfer native CP
// mask)" page, section "实现拆解" step 3: ranks are combined through LSEs in one common
// base) and for the split-KV reduction inside mla_decode (fp32 partials in workspace).
//
// One warp per (row, head): lane j owns dims [8j, 8j+8) and [256+8j, 256+8j+8) of the
// 512, so every load and store of a warp covers 512 contiguous bytes (bf16) or 1 KB
// (fp32).  The row max M of the n LSEs is reduced with warp shuffles; weights are
// 2^(lse*k - M*k) with k = 1 (base-2 LSEs) or log2(e) (natural LSEs).  HBM-bound:
// n * 1 KB (bf16) or n * 2 KB (fp32) read and 1 KB written per row.  Few rows of many
// bf16 shards take 2 or 4 warps per row instead (lse_combine_split_kernel), so that the
// n rounds of loads of a row are spread over more warps.
#include <math.h>

#include <cuda_bf16.h>

#include "internal.h"

namespace mla {
namespace {

constexpr int kDv = 512;
constexpr int kWarps = 8;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(p));
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(h[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// A NaN is the larger: a row none of whose LSEs is a number is no empty row.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
lse_combine_kernel(const T* __restrict__ partials, const float* __restrict__ lses, int n,
                   long long rows, long long shard_stride_rows, float lse_to_log2,
                   float out_lse_mul, __nv_bfloat16* __restrict__ out,
                   float* __restrict__ out_lse) {
  // launched as a dependent of the kernel that wrote the partials
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;

  float m2 = -INFINITY;                       // max LSE, in log2 units
  for (int s = lane; s < n; s += 32)
    m2 = max_nan(m2, __ldg(lses + s * shard_stride_rows + row) * lse_to_log2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m2 = max_nan(m2, __shfl_xor_sync(0xffffffffu, m2, o));

  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  float wsum = 0.f;
  if (m2 != -INFINITY) {
    for (int s = 0; s < n; ++s) {
      const float l2 = __ldg(lses + s * shard_stride_rows + row) * lse_to_log2;
      const float w = exp2f(l2 - m2);
      if (w == 0.f) continue;                 // empty shard: weight 0, partial unread
      wsum += w;
      const T* base = partials + (s * shard_stride_rows + row) * (long long)kDv;
      float v[8];
      load8(base + 8 * lane, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, v[k], acc[k]);
      load8(base + 256 + 8 * lane, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[8 + k] = fmaf(w, v[k], acc[8 + k]);
    }
  }
  const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
  __nv_bfloat16* o = out + row * kDv;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint4 packed;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&packed);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      h[k] = __floats2bfloat162_rn(acc[8 * c + 2 * k] * inv, acc[8 * c + 2 * k + 1] * inv);
    *reinterpret_cast<uint4*>(o + 256 * c + 8 * lane) = packed;
  }
  if (out_lse != nullptr && lane == 0)
    out_lse[row] = wsum != 0.f ? (m2 + log2f(wsum)) * out_lse_mul : -INFINITY;
}

// The same merge for few rows of many shards: S warps per row, warp q of a row taking
// shards q, q + S, q + 2S, ...; the S weighted partial sums are added through shared
// memory by the row's first warp.  With one warp per row such a merge is latency-bound
// (n dependent rounds of loads per warp; 16 shards of 1,024 rows took 13.6 us for 8.4 MB).
template <typename T, int S>
__global__ void __launch_bounds__(kWarps * 32)
lse_combine_split_kernel(const T* __restrict__ partials, const float* __restrict__ lses, int n,
                         long long rows, long long shard_stride_rows, float lse_to_log2,
                         float out_lse_mul, __nv_bfloat16* __restrict__ out,
                         float* __restrict__ out_lse) {
  static_assert(kWarps % S == 0, "whole rows per block");
  __shared__ float s_acc[kWarps][kDv];
  __shared__ float s_w[kWarps];
  // launched as a dependent of the kernel that wrote the partials
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * (kWarps / S) + warp / S;
  const int part = warp % S;
  const bool valid = row < rows;

  float m2 = -INFINITY;                       // max LSE over all shards, in log2 units
  if (valid)
    for (int s = lane; s < n; s += 32)
      m2 = max_nan(m2, __ldg(lses + s * shard_stride_rows + row) * lse_to_log2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m2 = max_nan(m2, __shfl_xor_sync(0xffffffffu, m2, o));

  float acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  float wsum = 0.f;
  if (valid && m2 != -INFINITY) {
    for (int s = part; s < n; s += S) {
      const float w = exp2f(__ldg(lses + s * shard_stride_rows + row) * lse_to_log2 - m2);
      if (w == 0.f) continue;                 // empty shard: weight 0, partial unread
      wsum += w;
      const T* base = partials + (s * shard_stride_rows + row) * (long long)kDv;
      float v[8];
      load8(base + 8 * lane, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, v[k], acc[k]);
      load8(base + 256 + 8 * lane, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[8 + k] = fmaf(w, v[k], acc[8 + k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s_acc[warp][8 * lane + k] = acc[k];
    s_acc[warp][256 + 8 * lane + k] = acc[8 + k];
  }
  if (lane == 0) s_w[warp] = wsum;
  __syncthreads();
  if (part != 0 || !valid) return;
  for (int q = 1; q < S; ++q) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[k] += s_acc[warp + q][8 * lane + k];
      acc[8 + k] += s_acc[warp + q][256 + 8 * lane + k];
    }
    wsum += s_w[warp + q];
  }
  const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
  __nv_bfloat16* o = out + row * kDv;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint4 packed;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&packed);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      h[k] = __floats2bfloat162_rn(acc[8 * c + 2 * k] * inv, acc[8 * c + 2 * k + 1] * inv);
    *reinterpret_cast<uint4*>(o + 256 * c + 8 * lane) = packed;
  }
  if (out_lse != nullptr && lane == 0)
    out_lse[row] = wsum != 0.f ? (m2 + log2f(wsum)) * out_lse_mul : -INFINITY;
}

// Rows of 128 values (the expanded form's outputs): half a warp a row, eight values a lane, four
// shards in flight.  Bound by the way of the LSEs and then the partials: 9 parts of 512 tokens x 8 heads
// (fp32, 19 MB) in 9.6 us, no less with a warp a row and more loads in flight.
constexpr int kDv128 = 128;

// Rows that mla_prefill computed: those of requests in order (none begins before the largest value so far)
// that end within T, as its kernel takes them.  What lies between cu[0] and cu[B] is not enough: the
// workspace holds nothing for a skipped request's rows.  32 requests a round, one a lane, their cu at lo and
// end; both halves of the warp look for their own token (-1: none).
__device__ __forceinline__ bool computed(const int32_t* __restrict__ cu, int B, int T, int token, int lane, int lo,
                                         int end) {
  bool found = token < 0;
  int top = 0;
  for (int b = lane;;) {
    int high = lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, high, o);
      if (lane >= o) high = max(high, v);
    }
    high = max(high, top);
    const bool fine = b < B && lo >= high && end <= T;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = __shfl_sync(0xffffffffu, token, 16 * h);
      if (__any_sync(0xffffffffu, fine && lo <= t && t < end) && (lane >> 4) == h) found = true;
    }
    top = __shfl_sync(0xffffffffu, high, 31);
    b += 32;
    if (b - lane >= B || __all_sync(0xffffffffu, found)) break;
    lo = b < B ? __ldg(cu + b) : 0;
    end = b < B ? __ldg(cu + b + 1) : 0;
  }
  return found && token >= 0;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
lse_combine128_kernel(const T* __restrict__ partials, const float* __restrict__ lses, int n,
                      long long rows, float lse_to_log2, float out_lse_mul,
                      __nv_bfloat16* __restrict__ out, float* __restrict__ out_lse,
                      const int32_t* __restrict__ cu, int B, int H) {
  // launched as a dependent of the kernel that wrote the partials
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, sub = lane & 15;
  const long long row = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * 2 + (lane >> 4);
  const bool live = row < rows;
  int lo = 0, end = 0;
  if (cu != nullptr && lane < B) {
    lo = __ldg(cu + lane);
    end = __ldg(cu + lane + 1);
  }

  float m2 = -INFINITY;                       // max LSE, in log2 units
  if (live)
    for (int s = sub; s < n; s += 16) m2 = max_nan(m2, __ldg(lses + s * rows + row) * lse_to_log2);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m2 = max_nan(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  // (the parts of mla_prefill are few rows, below 2^31)
  if (cu != nullptr && !computed(cu, B, (int)rows / H, live ? (int)row / H : -1, lane, lo, end)) return;
  if (!live) return;

  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  float wsum = 0.f;
  if (m2 != -INFINITY) {
    for (int s0 = 0; s0 < n; s0 += 4) {
      float w[4], v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = s0 + u < n ? exp2f(__ldg(lses + (s0 + u) * rows + row) * lse_to_log2 - m2) : 0.f;
        if (w[u] != 0.f)                      // empty shard: weight 0, partial unread
          load8(partials + ((s0 + u) * rows + row) * (long long)kDv128 + 8 * sub, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (w[u] != 0.f) {
          wsum += w[u];
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[u], v[u][k], acc[k]);
        }
    }
  }
  const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
  uint4 packed;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&packed);
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  *reinterpret_cast<uint4*>(out + row * kDv128 + 8 * sub) = packed;
  if (out_lse != nullptr && sub == 0)
    out_lse[row] = wsum != 0.f ? (m2 + log2f(wsum)) * out_lse_mul : -INFINITY;
}

}  // namespace

cudaError_t launch_lse_combine128(const void* partials, bool partials_fp32, const float* lses, int n,
                                  long long rows, bool in_log2, float out_lse_mul, uint16_t* out,
                                  float* out_lse, const int32_t* cu, int B, int H,
                                  cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const float k = in_log2 ? 1.0f : 1.4426950408889634f;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  DependentLaunch dl(dim3((unsigned)((rows + 2 * kWarps - 1) / (2 * kWarps))), dim3(kWarps * 32), stream);
  if (partials_fp32)
    return cudaLaunchKernelEx(&dl.cfg, lse_combine128_kernel<float>, static_cast<const float*>(partials), lses,
                              n, rows, k, out_lse_mul, o, out_lse, cu, B, H);
  return cudaLaunchKernelEx(&dl.cfg, lse_combine128_kernel<__nv_bfloat16>,
                            static_cast<const __nv_bfloat16*>(partials), lses, n, rows, k, out_lse_mul, o,
                            out_lse, cu, B, H);
}

cudaError_t launch_lse_combine(const void* partials, bool partials_fp32, const float* lses,
                               int n, long long rows, long long shard_stride_rows,
                               bool in_log2, float out_lse_mul, uint16_t* out,
                               float* out_lse, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const float k = in_log2 ? 1.0f : 1.4426950408889634f;
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  // few rows of many bf16 shards: several warps per row (up to 4, at least 4 shards each,
  // at most 4 K warps).  From 2,048 rows on one warp per row has enough warps in flight
  // (2,048 rows of 8 shards: 10.2 us with one warp per row, 11.2 us with two; 1,024 rows
  // of 16 shards: 13.6 us with one, 9.2 us with four; GB300, ncu)
  int S = 1;
  if (rows < 2048)
    while (S < 4 && 2 * S * 4 <= n && rows * 2 * S <= 4096) S *= 2;
  if (!partials_fp32 && S > 1) {
    const long long rpb = kWarps / S;
    DependentLaunch dl(dim3((unsigned)((rows + rpb - 1) / rpb)), dim3(kWarps * 32), stream);
    const __nv_bfloat16* pb = static_cast<const __nv_bfloat16*>(partials);
    if (S == 2)
      return cudaLaunchKernelEx(&dl.cfg, lse_combine_split_kernel<__nv_bfloat16, 2>, pb, lses, n,
                                rows, shard_stride_rows, k, out_lse_mul, o, out_lse);
    return cudaLaunchKernelEx(&dl.cfg, lse_combine_split_kernel<__nv_bfloat16, 4>, pb, lses, n,
                              rows, shard_stride_rows, k, out_lse_mul, o, out_lse);
  }
  const long long blocks = (rows + kWarps - 1) / kWarps;
  DependentLaunch dl(dim3((unsigned)blocks), dim3(kWarps * 32), stream);
  if (partials_fp32)
    return cudaLaunchKernelEx(&dl.cfg, lse_combine_kernel<float>,
                              static_cast<const float*>(partials), lses, n, rows,
                              shard_stride_rows, k, out_lse_mul, o, out_lse);
  return cudaLaunchKernelEx(&dl.cfg, lse_combine_kernel<__nv_bfloat16>,
                            static_cast<const __nv_bfloat16*>(partials), lses, n, rows,
                            shard_stride_rows, k, out_lse_mul, o, out_lse);
}

}  // namespace mla
