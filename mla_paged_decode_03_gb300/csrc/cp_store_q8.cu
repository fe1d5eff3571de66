// cp_store_q8: new KV rows into the 8-bit paged cache -- e4m3 values with one scale for every
// 16 consecutive slots of a page.
//
// Definition: the header's; rows go to the slots of cp_local_slot ("vLLM PR #52188 (DSpark +
// DCP)" page, sections "关键源码片段" and "实现拆解" step 4).  A request's keys on a rank
// fill its pages in order, so its new tokens are the local keys [L0, L1), L0 and L1 the
// rank's share of ctx and total, and local key l lies in slot l % block_size of page
// block_table[l / block_size].  The scale is a power of two: x / s and a later re-encoding by
// s_old / s are exact but for the one rounding to e4m3, whose relative step does not depend
// on the scale, so a finer scale would buy nothing but the last bit of range.
//
// One block of 128 threads per (request, group of 16 slots): it alone reads and writes the
// group, so the maximum, the earlier rows' re-encoding and the new rows need no atomics and
// no second launch.  The group's up to 16 new rows (1,152 bytes each) stay in registers
// between the maximum and the rounding, 16 bytes a load, nine a thread.
//
// HBM for prompts: 1,152 bytes in and 576.25 out per row (16 prompts, 98,000 rows: 33.4 us, 5.1 TB/s;
// 25.0 at the copy rate): a block loads its group, waits for the maximum, rounds and writes, with
// nothing of its own under way meanwhile, and only the SM's seven other blocks cover that.  Few
// rows: the launch and two dependent loads (64 rows 3.1 us).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

constexpr int kD = 576;
constexpr int kGroup = MLA_Q8_GROUP;
constexpr int kThreads = 128;
constexpr int kChunks = kD / 8;                          // 8 values: 16 bytes in, 8 out
constexpr int kPer = kGroup * kChunks / kThreads;        // chunks per thread
static_assert(kPer * kThreads == kGroup * kChunks, "whole chunks per thread");

struct Params {
  const uint4* rows;
  const int32_t *ctx, *total, *table;
  long long bt_stride;
  int max_blocks, N, block_size, rank, il;
  long long span;                                        // cp_size * interleave
  FastDiv div_il;
  int groups;                                            // blocks per request
  uint2* cache;
  float* scales;
  int num_blocks;
  unsigned int* status;
};

__device__ __forceinline__ unsigned int fdiv(unsigned int n, const FastDiv& f) {
  return f.d == 1u ? n : (unsigned int)__umul64hi(f.m, (unsigned long long)n);
}

__device__ __forceinline__ int local_len(const Params& p, int g) {
  const long long q = g / p.span, over = g - q * p.span - (long long)p.rank * p.il;
  return (int)(q * p.il + min(max(over, 0LL), (long long)p.il));
}

// Largest magnitude of 8 bf16 values, as their 15 bits.
__device__ __forceinline__ unsigned int peak8(const uint4& v) {
  const unsigned int k = 0x7fff7fffu;
  const unsigned int m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
  return max(m & 0xffffu, m >> 16);
}
// The same over the finite ones.
__device__ __noinline__ unsigned int finite_peak8(uint4 v) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
  unsigned int m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned int a = (w[k >> 1] >> (16 * (k & 1))) & 0x7fffu;
    if (a < 0x7f80u) m = max(m, a);
  }
  return m;
}

// 8 bf16 values times `mul` as e4m3.
__device__ __forceinline__ uint2 encode8(const uint4& v, float mul) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
  unsigned int o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[k] << 16) * mul,
                                                __uint_as_float(w[k] & 0xffff0000u) * mul),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}
// The same for values that may not be finite (NaN and infinities become NaN) and for a scale
// that is no power of two, whose reciprocal is not exact: x / s.
__device__ __noinline__ uint2 encode8_any(uint4 v, float s) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
  unsigned int o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 x = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    if ((w[k] & 0x7f80u) == 0x7f80u) x.x = __uint_as_float(0x7fc00000u);
    if ((w[k] & 0x7f800000u) == 0x7f800000u) x.y = __uint_as_float(0x7fc00000u);
    o[k] = __nv_cvt_float2_to_fp8x2(make_float2(x.x / s, x.y / s), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// 8 e4m3 values times `ratio`, rounded to e4m3 again.
__device__ __forceinline__ uint2 again8(uint2 v, float ratio) {
  unsigned int o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned int w = k < 2 ? v.x : v.y;
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(k & 1 ? w >> 16 : w & 0xffffu);
    const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    o[k] = __nv_cvt_float2_to_fp8x2(make_float2(x.x * ratio, x.y * ratio), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// (eight blocks an SM: with the 80 registers that the compiler takes otherwise, 33.4 instead of
// 29.6 us for 16 prompts of up to 8,192 rows that are the same, and half in L2, in every call)
__global__ void __launch_bounds__(kThreads, 8) cp_store_q8_kernel(const Params p) {
  __shared__ unsigned int s_peak[kThreads / 32];
  __shared__ long long s_src[kGroup];                    // where each new row begins, in 16 bytes
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.groups, gi = blockIdx.x - b * p.groups;
  const int ctx = __ldg(p.ctx + b);
  long long fresh = (long long)__ldg(p.total + b) - ctx;
  if (ctx < 0 || fresh > p.N) {
    if (tid == 0 && gi == 0) atomicOr(p.status, MLA_STATUS_BAD_STEP);
    if (ctx < 0) return;
    fresh = p.N;
  }
  if (fresh <= 0) return;
  const int l0 = local_len(p, ctx), l1 = local_len(p, ctx + (int)fresh);
  // (compared as groups: past the last one the first key may lie beyond 2^31)
  const int group = l0 / kGroup + gi;
  if (l1 <= l0 || group > (l1 - 1) / kGroup) return;
  const int g0 = group * kGroup;                         // the group's first local key
  const int vb = g0 / p.block_size;
  if (vb >= p.max_blocks) {
    if (tid == 0) atomicOr(p.status, MLA_STATUS_BAD_VBLOCK);
    return;
  }
  const int page = __ldg(p.table + (long long)b * p.bt_stride + vb);
  if (page < 0 || page >= p.num_blocks) {
    if (tid == 0) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return;
  }
  const long long slot0 = (long long)page * p.block_size + (g0 - vb * p.block_size);
  const int lo = max(l0 - g0, 0), hi = min(l1 - g0, kGroup);   // new rows [lo, hi) of the group

  // ---- new rows into registers; the largest magnitude ----------------------------------
  if (tid >= lo && tid < hi) {
    const unsigned int l = (unsigned int)(g0 + tid);
    const unsigned int seg = fdiv(l, p.div_il);
    const long long pos = seg * p.span + (long long)p.rank * p.il + (l - seg * (unsigned int)p.il);
    s_src[tid] = ((long long)b * p.N + (pos - ctx)) * kChunks;
  }
  const float old_raw = lo > 0 ? p.scales[slot0 / kGroup] : 0.f;
  __syncthreads();
  uint4 v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + i * kThreads;
    const int r = c / kChunks;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) v[i] = __ldcs(p.rows + s_src[r] + (c - r * kChunks));
  }
  unsigned int peak = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) peak = max(peak, peak8(v[i]));
  const bool wild = peak >= 0x7f80u;                     // this thread has a NaN or an infinity
  if (wild) {
    peak = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) peak = max(peak, finite_peak8(v[i]));
  }
  peak = __reduce_max_sync(0xffffffffu, peak);
  if ((tid & 31) == 0) s_peak[tid >> 5] = peak;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) peak = max(peak, s_peak[w]);

  // ---- scale: 448 = 1.75 * 2^8, so a value m * 2^x (1 <= m < 2) needs 2^(x-8) when
  // m <= 1.75 (mantissa bits <= 96 of 128), else 2^(x-7) ----------------------------------
  int e = (int)(peak >> 7) - 127 - 8 + ((peak & 0x7fu) > 96u ? 1 : 0);
  e = min(max(e, -32), 64);
  float s = __int_as_float((e + 127) << 23);
  float s_old = old_raw;
  if (lo > 0) {
    if (!(s_old >= MLA_Q8_SCALE_MIN && s_old <= MLA_Q8_SCALE_MAX)) {
      s_old = 1.f;
      if (tid == 0) atomicOr(p.status, MLA_STATUS_BAD_SCALE);
    }
    s = fmaxf(s, s_old);
  }
  const bool plain = !wild && (__float_as_int(s) & 0x7fffff) == 0;   // 1 / s is exact
  const float inv = 1.f / s;

  uint2* dst = p.cache + slot0 * kChunks;
  if (lo > 0 && s != s_old) {
    const float ratio = s_old / s;
    for (int c = tid; c < lo * kChunks; c += kThreads) dst[c] = again8(dst[c], ratio);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + i * kThreads;
    const int r = c / kChunks;
    if (r >= lo && r < hi) dst[c] = plain ? encode8(v[i], inv) : encode8_any(v[i], s);
  }
  if (tid == 0 && (lo == 0 || s != old_raw)) p.scales[slot0 / kGroup] = s;
}

}  // namespace

cudaError_t launch_cp_store_q8(const StoreQ8Args& a, cudaStream_t stream) {
  Params p;
  p.rows = reinterpret_cast<const uint4*>(a.kv_new);
  p.ctx = a.ctx;
  p.total = a.total;
  p.table = a.table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.N = a.N;
  p.block_size = a.block_size;
  p.rank = a.cp_rank;
  p.il = a.interleave;
  p.span = (long long)a.cp_size * a.interleave;
  p.div_il = make_fastdiv((unsigned int)a.interleave);
  p.cache = reinterpret_cast<uint2*>(a.cache);
  p.scales = a.scales;
  p.num_blocks = a.num_blocks;
  p.status = a.status;
  // a rank holds at most `most` of N consecutive positions: a segment's share of each whole
  // round and at most one segment (or two parts of less) of the rest.  n keys in a row touch
  // at most (n + 14) / 16 + 1 groups, which is never above n, so the grid stays within B * N
  const long long rest = a.N % p.span;
  const long long most = a.N / p.span * a.interleave + (rest < a.interleave ? rest : a.interleave);
  if (most == 0) return cudaSuccess;
  p.groups = (int)((most + kGroup - 2) / kGroup + 1);
  const long long blocks = (long long)a.B * p.groups;
  cp_store_q8_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
