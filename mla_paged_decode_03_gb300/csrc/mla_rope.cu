// Rotary positions: the rope part of queries (mla_rope), and the append of new tokens to the
// paged cache with their rope key rotated on the way (cp_rope_store).
//
// A rope part is 64 dims, 32 pairs: (2i, 2i+1), or (i, i+32) in the halves layout.  At position p
// pair i turns by the angle 2 pi frac(p f_i), f_i the turns a position:
//   y0 = m (x0 cos a - x1 sin a),  y1 = m (x0 sin a + x1 cos a).
//
// f_i comes as a 64-bit fixed-point fraction (units of 2^-64 turns), so that p f_i mod 1 is a
// wrapping 64-bit product: exact at any position up to 2^63, where an angle in single precision
// is off by p 2^-24 radians, and without the double-precision arithmetic that this GPU has little
// of.  The upper 32 bits of the fraction are kept (2^-33 turns), sincospif takes them from there.
//
// HBM-bound: 128 bytes in and out for each head of a token, 1152 for a stored token; a lane turns
// eight pairs of one token, so that its eight sines and cosines serve all heads that its warp
// takes.  Four lanes hold a rope part: two 16-byte chunks each, 64 bytes apart in either layout.
//
// Measured in graphs: 8,192 tokens x 128 heads out of rows of 192 in 47 us (5.8 TB/s, 86% of a copy's rate;
// the 128 bytes read of each 384 are whole lines); 64 tokens x 128 heads in 3.0 us.  One head leaves 28 of a
// warp's lanes idle: 8,192 tokens in 7.2 us, 65,536 in 42, where their 17 MB would pass in 2.5.  Stores: some
// 24,500 rows of 49,200 positions in 12.9 us (4.4 TB/s), 64 in 2.8.
#include <cuda_bf16.h>

#include "internal.h"
#include "slots.cuh"
#include "sm100.cuh"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

constexpr int kLatentChunks = 64;              // 16-byte chunks of a row's latent part
constexpr int kRowChunks = 72;                 // and of the whole row

// Cosines and sines of the eight pairs of lane quarter j (0..3).  Pairs layout: the quarter's
// chunks hold dims 8j.. and 32+8j.., so pairs 4j..4j+3 and 16+4j..; halves: pairs 8j..8j+7.
struct Turns {
  float c[8], s[8];
  __device__ __forceinline__ void set(long long pos, const unsigned long long* __restrict__ freqs,
                                      int j, bool half, float mscale) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = half ? 8 * j + k : (k < 4 ? 4 * j + k : 12 + 4 * j + k);
      const unsigned long long turn = (unsigned long long)pos * __ldg(freqs + i);
      // the fraction as a signed 32-bit number of 2^-32 turns; sincospif's unit is half a turn
      const float x = (float)(int)(turn >> 32) * 4.656612873077393e-10f;
      sincospif(x, &s[k], &c[k]);
      c[k] *= mscale;
      s[k] *= mscale;
    }
  }
};

__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Turns a quarter's two chunks in place.
__device__ __forceinline__ void turn(uint4& a, uint4& b, const Turns& t, bool half) {
  uint32_t* u = &a.x;
  uint32_t* v = &b.x;
  if (half) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = lo16(u[k]), x1 = lo16(v[k]), z0 = hi16(u[k]), z1 = hi16(v[k]);
      const int e = 2 * k, o = 2 * k + 1;
      u[k] = pack(x0 * t.c[e] - x1 * t.s[e], z0 * t.c[o] - z1 * t.s[o]);
      v[k] = pack(x0 * t.s[e] + x1 * t.c[e], z0 * t.s[o] + z1 * t.c[o]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = lo16(u[k]), x1 = hi16(u[k]), z0 = lo16(v[k]), z1 = hi16(v[k]);
      u[k] = pack(x0 * t.c[k] - x1 * t.s[k], x0 * t.s[k] + x1 * t.c[k]);
      v[k] = pack(z0 * t.c[4 + k] - z1 * t.s[4 + k], z0 * t.s[4 + k] + z1 * t.c[4 + k]);
    }
  }
}

// A warp takes `heads` consecutive heads (a multiple of 8) of one token, eight at a time.
__global__ void __launch_bounds__(256) mla_rope_kernel(RopeArgs p, int heads, int groups) {
  sm100::grid_wait();
  sm100::grid_release();
  const int lane = threadIdx.x & 31, j = lane & 3;
  const long long w = (blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5;
  const long long tok = w / groups;
  if (tok >= p.T) return;
  const long long pos = __ldg(reinterpret_cast<const long long*>(p.positions) + tok);
  if (pos < 0) return;                          // a rejected token's rows stay as they are
  const int h0 = (int)(w - tok * groups) * heads + (lane >> 2);
  const int h1 = min((int)(w - tok * groups) * heads + heads, p.H);
  Turns t;
  t.set(pos, reinterpret_cast<const unsigned long long*>(p.freqs), j, p.half, p.mscale);
  const uint16_t* x = p.x + tok * p.x_t + 8 * j;
  uint16_t* o = p.out + tok * p.out_t + 8 * j;
  // four heads of a lane in flight; x and out may be the same rows, so a round's loads come
  // before its stores
  for (int h = h0; h < h1; h += 32) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (h + 8 * u < h1) {
        const uint16_t* r = x + (long long)(h + 8 * u) * p.x_h;
        a[u] = __ldcs(reinterpret_cast<const uint4*>(r));
        b[u] = __ldcs(reinterpret_cast<const uint4*>(r + 32));
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (h + 8 * u < h1) {
        turn(a[u], b[u], t, p.half);
        uint16_t* r = o + (long long)(h + 8 * u) * p.out_h;
        *reinterpret_cast<uint4*>(r) = a[u];
        *reinterpret_cast<uint4*>(r + 32) = b[u];
      }
  }
}

// A warp takes `group` (1 to 32) consecutive positions: lanes map one each, then the warp writes
// the rows of the owned ones, four a round: 64 latent chunks, two a lane, and the rope part by
// four lanes (lanes 4u .. 4u+3 that of the round's row u).
__global__ void __launch_bounds__(256) cp_rope_store_kernel(RopeStoreArgs a, SlotParams p,
                                                            FastDiv div_row, int group) {
  sm100::grid_wait();
  sm100::grid_release();
  const int lane = threadIdx.x & 31;
  const long long total = (long long)a.B * a.N;
  const long long rows = (long long)a.num_blocks * a.block_size;
  bool bad_vb = false, bad_page = false;
  const long long first = ((blockIdx.x * (long long)blockDim.x + threadIdx.x) >> 5) * group;
  if (first >= total) return;
  const long long i = first + lane;
  long long slot = MLA_PAD_SLOT_ID, pos = -1;
  if (lane < group && i < total) {
    pos = __ldg(reinterpret_cast<const long long*>(a.positions) + i);
    int page;
    unsigned int local;
    if (locate(pos, (int)fdiv((unsigned int)i, div_row), p, bad_vb, page, local)) {
      slot = (long long)page * p.block_size + local;
      if (a.slots != nullptr) a.slots[i] = slot;
      if (page < 0 || slot >= rows) {
        bad_page = true;
        slot = MLA_PAD_SLOT_ID;
      }
    } else if (a.slots != nullptr) {
      a.slots[i] = MLA_PAD_SLOT_ID;
    }
  }
  unsigned int own = __ballot_sync(0xffffffffu, slot >= 0);
  while (own != 0u) {
    int src[4], nr = 0;
    long long dst[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      src[u] = 0;
      if (own != 0u) {
        src[u] = __ffs(own) - 1;
        own &= own - 1u;
        nr = u + 1;
      }
      dst[u] = __shfl_sync(0xffffffffu, slot, src[u]);
    }
    uint4 v[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (u < nr) {
        const uint4* r = reinterpret_cast<const uint4*>(a.latent + (first + src[u]) * a.latent_t);
        v[u][0] = __ldcs(r + lane);
        v[u][1] = __ldcs(r + 32 + lane);
      }
    const int u = (lane >> 2) & 3, j = lane & 3;
    const int mine = u == 0 ? src[0] : u == 1 ? src[1] : u == 2 ? src[2] : src[3];
    const long long at = u == 0 ? dst[0] : u == 1 ? dst[1] : u == 2 ? dst[2] : dst[3];
    const long long where = __shfl_sync(0xffffffffu, pos, mine);
    if (lane < 4 * nr) {
      const uint16_t* r = a.k_rope + (first + mine) * a.k_rope_t + 8 * j;
      uint4 x = __ldcs(reinterpret_cast<const uint4*>(r));
      uint4 y = __ldcs(reinterpret_cast<const uint4*>(r + 32));
      Turns t;
      t.set(where, reinterpret_cast<const unsigned long long*>(a.freqs), j, a.half, a.mscale);
      turn(x, y, t, a.half);
      uint4* o = reinterpret_cast<uint4*>(a.cache) + at * kRowChunks + kLatentChunks + j;
      o[0] = x;
      o[4] = y;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < nr) {
        uint4* o = reinterpret_cast<uint4*>(a.cache) + dst[k] * kRowChunks;
        o[lane] = v[k][0];
        o[32 + lane] = v[k][1];
      }
  }
  if (__any_sync(0xffffffffu, bad_vb) && lane == 0) atomicOr(a.status, MLA_STATUS_BAD_VBLOCK);
  if (__any_sync(0xffffffffu, bad_page) && lane == 0) atomicOr(a.status, MLA_STATUS_BAD_PAGE);
}

}  // namespace

cudaError_t launch_mla_rope(const RopeArgs& a, cudaStream_t stream) {
  // heads a warp: all of a token's when that gives every SM 32 warps, else fewer, so that few
  // tokens spread over the GPU (the sines are then computed more than once)
  int heads = (a.H + 7) / 8 * 8;
  while (heads > 8 && (long long)a.T * ((a.H + heads - 1) / heads) < 32LL * a.num_sms)
    heads = (heads / 2 + 7) / 8 * 8;
  const int groups = (a.H + heads - 1) / heads;
  const long long warps = (long long)a.T * groups;
  DependentLaunch dl(dim3((unsigned)((warps + 7) / 8)), dim3(256), stream);
  return cudaLaunchKernelEx(&dl.cfg, mla_rope_kernel, a, heads, groups);
}

cudaError_t launch_cp_rope_store(const RopeStoreArgs& a, cudaStream_t stream) {
  const long long total = (long long)a.B * a.N;
  const SlotParams p = make_slot_params(a.block_table, a.bt_stride, a.max_blocks, a.block_size,
                                        a.cp_size, a.cp_rank, a.interleave, a.status);
  // a position a warp while that keeps all warps resident, then 32.  us in a graph, one rank (one of two), by
  // positions a warp:
  //   positions       1              8              32
  //          64    3.2 (3.2)      4.7 (3.7)      8.6 (5.6)
  //       4,864    6.6 (6.0)      5.4 (4.1)     12.7 (7.9)
  //       8,192   10.3 (9.5)      5.9 (4.4)     12.9 (8.0)
  //      16,384   17.5 (15.7)     8.1 (5.6)     13.4 (8.2)
  //      32,768   33.5 (28.9)    16.0 (9.6)     17.3 (9.1)
  //      65,536   65.9 (56.1)    28.3 (17.6)    27.9 (15.4)
  // so both ends are served, and 8 would be the better choice from a thousand to 32,000 positions: with 32 they
  // are on few SMs (4,865 positions on 20 blocks, every SM has one from 38,900 on).
  const int group = total <= 32LL * a.num_sms ? 1 : 32;
  const long long warps = (total + group - 1) / group;
  DependentLaunch dl(dim3((unsigned)((warps + 7) / 8)), dim3(256), stream);
  return cudaLaunchKernelEx(&dl.cfg, cp_rope_store_kernel, a, p, make_fastdiv((unsigned int)a.N), group);
}

}  // namespace mla
