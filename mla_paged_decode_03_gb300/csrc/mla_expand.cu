// Keys and values of all heads from the pages' latent rows (the expanded form of latent
// attention): for row r of the output, that request b's local key l gives (r = kv_starts[b] + l),
//   kv[h, r, 0:256] = W[h] c,   k_rope[r] = c[512:576],
// with c the key's cache row (times its scale in the 8-bit form) and W[h] the 256 x 512 weights of
// head h (128 dims of its key, then 128 of its value).
//
// A matrix product of K = 512 with gathered rows: 1,024 operations for each 2-byte output, so
// bound by the tensor cores, with an output stream of over half the memory's rate beside it.
//
// Design.  A tile is 128 rows x 128 output dims (half of a head).  The gathered rows are the A
// operand and stay in tensor memory (512 dims are 256 columns), since each is used for all heads;
// the other 256 columns are two accumulators, so that one is written out while the other is
// computed.  Only W passes through shared memory: 16 KB chunks of 128 dims x 64 in a ring of 12, by
// TMA.  A pair of SMs (a cluster of two) works on two neighbouring row tiles with the same W: each
// loads half of a chunk and multicasts it to both, which halves what W takes of the L2's rate (32
// bytes a clock and SM).  The tiles of all row pairs are one sequence, row pair after row pair, cut
// evenly over the clusters; a cluster gathers rows only when its row pair changes.
//
// Rows are gathered by four warps, a thread a row, straight into tensor memory: any page size and
// any start, and the 8-bit form's conversion costs nothing but there.
//
// Safety: every wait is bounded (sm100.cuh); rows of no request, and pages or lengths out of range,
// are read as zeros and not written (the latter flagged).
#include <math.h>
#include <stdint.h>

#include <functional>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "internal.h"
#include "sm100.cuh"
#include "tma_map.h"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kLatent = 512, kRow = 576;
constexpr int kM = 128, kN = 128;
constexpr int kChunkBytes = kN * 128;              // 128 dims of W x 64 latent dims, bf16
constexpr int kChunks = kLatent / 64;
constexpr int kStages = 12;
constexpr int kThreads = 384;                      // warp 0 TMA, 1 MMA; 4-7 epilogue; 8-11 rows
constexpr uint32_t kColD = 256;                    // accumulators; A is columns 0..255

constexpr int kOffStage = kStages * kChunkBytes;   // 4 warps x 32 rows x 256 bytes
constexpr int kOffBar = kOffStage + 4 * 32 * 256;
constexpr int kOffMisc = kOffBar + 512;
constexpr int kSmemBytes = kOffMisc + 64 + 1024;

enum Bar : int {
  B_FULL = 0,                    // [12] W chunk here (both halves)
  B_EMPTY = B_FULL + kStages,    // [12] both SMs have used it
  B_AFULL = B_EMPTY + kStages,   // [8] 64 dims of the rows in tensor memory
  B_AFREE = B_AFULL + kChunks,   // the row tile's last product is done
  B_DFULL = B_AFREE + 1,         // [2]
  B_DFREE = B_DFULL + 2,         // [2]
  B_DRAIN = B_DFREE + 2,
  B_COUNT = B_DRAIN + 1
};
static_assert(B_COUNT * 8 <= 512, "barriers");

struct ExpandParams {
  ExpandArgs a;
  int col_tiles;                 // 2 H
};

struct Ctx {
  uint32_t base;
  volatile int* abort;
  unsigned int* status;
  unsigned long long wait_ns;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + kOffBar + 8 * i; }
  __device__ __forceinline__ bool wait(int i, uint32_t parity, bool cluster = false) const {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, status, wait_ns, cluster));
  }
};

// The key that output row r holds: the request is the last one that starts at r or before.
struct Key {
  const uint8_t* row;            // null: none
  float scale;
};

template <bool kQ8>
__device__ __forceinline__ Key find_key(const ExpandArgs& a, long long r, unsigned& flags) {
  Key k{nullptr, 0.f};
  if (r >= a.S) return k;
  int lo = 0, hi = a.B;          // starts[lo - 1] <= r < starts[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.starts + mid) <= r) lo = mid + 1;
    else hi = mid;
  }
  if (lo == 0) return k;
  const int b = lo - 1;
  const long long l = r - __ldg(a.starts + b);
  long long have = __ldg(a.seq_lens + b);
  if (have > (long long)a.max_blocks * a.block_size) {
    have = (long long)a.max_blocks * a.block_size;
    flags |= MLA_STATUS_SEQ_TOO_LONG;
  }
  if (l >= have) return k;
  const int blk = (int)(l / a.block_size), off = (int)(l - (long long)blk * a.block_size);
  const int page = __ldg(a.block_table + (long long)b * a.bt_stride + blk);
  if (page < 0 || page >= a.num_blocks) {
    flags |= MLA_STATUS_BAD_PAGE;
    k.row = nullptr;
    k.scale = -1.f;              // a row of the request all the same: zeros are written
    return k;
  }
  const long long slot = (long long)page * a.block_size + off;
  k.row = static_cast<const uint8_t*>(a.cache) + slot * (kQ8 ? kRow : 2 * kRow);
  k.scale = 1.f;
  if (kQ8) {
    k.scale = __ldg(a.scales + (long long)page * (a.block_size / MLA_Q8_GROUP) + off / MLA_Q8_GROUP);
    if (!(k.scale >= MLA_Q8_SCALE_MIN && k.scale <= MLA_Q8_SCALE_MAX)) {
      k.scale = 1.f;
      flags |= MLA_STATUS_BAD_SCALE;
    }
  }
  return k;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 dims of a row, from dim `d`, as 32 words of two bf16.
template <bool kQ8>
__device__ __forceinline__ void load64(const Key& k, int d, uint32_t (&v)[32]) {
  if (k.row == nullptr) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0;
  } else if (!kQ8) {
    const uint4* s = reinterpret_cast<const uint4*>(k.row + 2 * d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = __ldg(s + i);
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
    }
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(k.row + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = __ldg(s + i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t h;
        const uint16_t two = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[8 * i + q] = pack(f.x * k.scale, f.y * k.scale);
      }
    }
  }
}

// W chunk: 64 rows (output dims) x 64 latent dims into both SMs of the pair.
__device__ __forceinline__ void tma_load_2d_both_warp(uint32_t dst, const CUtensorMap* map, int x,
                                                      int y, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".multicast::cluster [%0], [%1, {%2, %3}], [%4], %5;\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "h"((uint16_t)3)
      : "memory");
}

template <bool kQ8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_expand_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sp = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cr = cluster_ctarank();
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sp + kOffMisc);
  Ctx s;
  s.base = smem_u32(sp);
  s.abort = reinterpret_cast<volatile int*>(misc + 1);
  s.status = p.a.status;
  s.wait_ns = p.a.wait_ns;

  if (tid == 0) {
    *s.abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(s.bar(B_FULL + i), 1);
      mbar_init(s.bar(B_EMPTY + i), 2);
    }
    for (int i = 0; i < kChunks; ++i) mbar_init(s.bar(B_AFULL + i), 4);
    mbar_init(s.bar(B_AFREE), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s.bar(B_DFULL + i), 1);
      mbar_init(s.bar(B_DFREE + i), 4);
    }
    mbar_init(s.bar(B_DRAIN), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s.base + kOffMisc, 512);
    tmem_relinquish();
  }
  // rows in use: the last request's end (requests are in the order of their rows)
  long long rows = 0;
  if (p.a.B > 0)
    rows = (long long)__ldg(p.a.starts + p.a.B - 1) + max(0, __ldg(p.a.seq_lens + p.a.B - 1));
  rows = rows < 0 ? 0 : rows > p.a.S ? p.a.S : rows;
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  const long long units = (rows + 2 * kM - 1) / (2 * kM) * p.col_tiles;
  const long long C = nclusters_x(), c = cluster_id_x();
  const long long u0 = units * c / C, u1 = units * (c + 1) / C;
  unsigned flags = 0;

  if (warp == 0) {
    // ---- W chunks ---------------------------------------------------------------------
    int st = 0;
    uint32_t par = 1;
    long long issued = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok; ++u) {
      const int n0 = (int)(u % p.col_tiles) * kN + 64 * (int)cr;
      for (int k = 0; k < kChunks; ++k) {
        ok = s.wait(B_EMPTY + st, par, true);
        if (!ok) break;
        mbar_arrive_expect_tx_warp(s.bar(B_FULL + st), kChunkBytes);
        tma_load_2d_both_warp(s.base + st * kChunkBytes + cr * (kChunkBytes / 2), &wmap, 64 * k, n0,
                              s.bar(B_FULL + st));
        ++issued;
        if (++st == kStages) {
          st = 0;
          par ^= 1u;
        }
      }
    }
    // the peer's last releases arrive here before this SM ends; after an abort, the copies do
    for (long long m = issued > kStages ? issued - kStages : 0; m < issued; ++m) {
      const int i = (int)(m % kStages);
      const uint32_t ph = (uint32_t)((m / kStages) & 1);
      if (!ok || !s.wait(B_EMPTY + i, ph, true)) mbar_wait_drain(s.bar(B_FULL + i), ph);
    }
  } else if (warp == 1) {
    // ---- products ---------------------------------------------------------------------
    const uint32_t idesc = idesc_bf16(kM, kN, false, false);
    int st = 0;
    uint32_t par = 0, apar = 0;
    bool ok = true;
    long long n = 0;
    for (long long u = u0; u < u1 && ok; ++u, ++n) {
      const bool fresh = u == u0 || u % p.col_tiles == 0;
      const bool last = u + 1 == u1 || (u + 1) % p.col_tiles == 0;
      const int g = (int)(n & 1);
      ok = s.wait(B_DFREE + g, (uint32_t)(((n >> 1) + 1) & 1));
      for (int k = 0; k < kChunks && ok; ++k) {
        if (fresh) ok = s.wait(B_AFULL + k, apar);
        ok = ok && s.wait(B_FULL + st, par, true);
        if (!ok) break;
        tc_fence_after();
        mma4_ts_warp(tmem + kColD + g * kN, tmem + 32 * k,
                     smem_desc(s.base + st * kChunkBytes, 16, 1024, kSwizzle128B), idesc, k != 0);
        mma_commit_multicast_warp(s.bar(B_EMPTY + st), (uint16_t)3);
        if (++st == kStages) {
          st = 0;
          par ^= 1u;
        }
      }
      if (!ok) break;
      mma_commit_warp(s.bar(B_DFULL + g));
      if (fresh) apar ^= 1u;
      if (last) mma_commit_warp(s.bar(B_AFREE));
    }
    mma_commit_warp(s.bar(B_DRAIN));
    mbar_wait_drain(s.bar(B_DRAIN), 0);
  } else if (warp >= 8) {
    // ---- rows into tensor memory: thread = row ------------------------------------------
    const uint32_t ta = tmem + ((uint32_t)(warp & 3) << 21);
    bool ok = true;
    long long m = 0;
    for (long long u = u0; u < u1 && ok; u = (u / p.col_tiles + 1) * p.col_tiles, ++m) {
      const long long r = (u / p.col_tiles * 2 + cr) * kM + (warp & 3) * 32 + lane;
      const Key key = find_key<kQ8>(p.a, r, flags);
      ok = s.wait(B_AFREE, (uint32_t)((m + 1) & 1));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < kChunks; k += 2) {
        uint32_t v[32], w[32];
        load64<kQ8>(key, 64 * k, v);
        load64<kQ8>(key, 64 * k + 64, w);
        tmem_st32(ta + 32 * k, v);
        tmem_st32(ta + 32 * k + 32, w);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s.bar(B_AFULL + k));
          mbar_arrive(s.bar(B_AFULL + k + 1));
        }
      }
      // the cluster that has a row tile's first unit copies its rope keys
      if (u % p.col_tiles == 0 && (key.row != nullptr || key.scale != 0.f)) {
        uint32_t v[32];
        load64<kQ8>(key, kLatent, v);
        uint4* o = reinterpret_cast<uint4*>(p.a.k_rope + r * 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  } else if (warp >= 4) {
    // ---- outputs: accumulator rows (thread = row) -> 256 bytes a row in shared memory ->
    // half a warp a row to memory
    const int q = warp & 3;
    uint8_t* stage = sp + kOffStage + q * 32 * 256;
    const uint32_t td = tmem + kColD + ((uint32_t)q << 21);
    unsigned valid = 0;                           // the warp's rows that are somebody's
    bool ok = true;
    long long n = 0, m0 = -1;
    for (long long u = u0; u < u1 && ok; ++u, ++n) {
      const long long mp = u / p.col_tiles;
      const int nt = (int)(u - mp * p.col_tiles);
      const long long r0 = (mp * 2 + cr) * kM + q * 32;
      if (mp != m0) {
        unsigned f = 0;
        const Key key = find_key<kQ8>(p.a, r0 + lane, f);
        valid = __ballot_sync(0xffffffffu, key.row != nullptr || key.scale != 0.f);
        m0 = mp;
      }
      const int g = (int)(n & 1);
      ok = s.wait(B_DFULL + g, (uint32_t)((n >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32], w[32];
        tmem_ld32(td + g * kN + 64 * h, v);
        tmem_ld32(td + g * kN + 64 * h + 32, w);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t* x = i < 4 ? v + 8 * i : w + 8 * (i - 4);
          uint4 o;
          o.x = pack(__uint_as_float(x[0]), __uint_as_float(x[1]));
          o.y = pack(__uint_as_float(x[2]), __uint_as_float(x[3]));
          o.z = pack(__uint_as_float(x[4]), __uint_as_float(x[5]));
          o.w = pack(__uint_as_float(x[6]), __uint_as_float(x[7]));
          *reinterpret_cast<uint4*>(stage + lane * 256 + (((8 * h + i) ^ (lane & 7)) << 4)) = o;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s.bar(B_DFREE + g));
      uint16_t* out = p.a.kv + ((long long)(nt >> 1) * p.a.S + r0) * 256 + (nt & 1) * 128;
#pragma unroll 8
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4), ch = lane & 15;
        if (valid >> r & 1u)
          *reinterpret_cast<uint4*>(out + (long long)r * 256 + ch * 8) =
              *reinterpret_cast<const uint4*>(stage + r * 256 + ((ch ^ (r & 7)) << 4));
      }
      __syncwarp();
    }
  }
  if (flags) atomicOr(p.a.status, flags);
  // an SM that gave up stops the other one too
  if (*s.abort && lane == 0) st_cluster_u32(mapa(smem_u32((const void*)(sp + kOffMisc + 4)), cr ^ 1), 1);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Set once per device: the shared-memory attributes and how many clusters run at a time.
struct ExpandDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int clusters = 0;
};
constexpr int kMaxDevices = 64;
ExpandDevice g_dev[kMaxDevices];

void device_setup(ExpandDevice& d) {
  d.err = cudaFuncSetAttribute(mla_expand_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmemBytes);
  if (d.err == cudaSuccess)
    d.err = cudaFuncSetAttribute(mla_expand_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes);
  if (d.err != cudaSuccess) return;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  d.err = cudaOccupancyMaxActiveClusters(&d.clusters, mla_expand_kernel<false>, &cfg);
  if (d.err == cudaSuccess && d.clusters < 1) d.err = cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_mla_expand(const ExpandArgs& a, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(g_dev[dev].once, device_setup, std::ref(g_dev[dev]));
  if (g_dev[dev].err != cudaSuccess) return g_dev[dev].err;
  ExpandParams p;
  p.a = a;
  p.col_tiles = 2 * a.H;
  CUtensorMap wmap;
  const uint64_t dims[2] = {(uint64_t)kLatent, (uint64_t)a.H * 256}, strides[1] = {kLatent * 2};
  const uint32_t box[2] = {64, 64};
  if (!encode_tile_map(&wmap, a.w, 2, dims, strides, box)) return cudaErrorInvalidValue;
  const long long units = ((long long)a.S + 2 * kM - 1) / (2 * kM) * p.col_tiles;
  const int clusters = (int)(units < g_dev[dev].clusters ? units : g_dev[dev].clusters);
  if (a.scales != nullptr)
    mla_expand_kernel<true><<<2 * clusters, kThreads, kSmemBytes, stream>>>(wmap, p);
  else
    mla_expand_kernel<false><<<2 * clusters, kThreads, kSmemBytes, stream>>>(wmap, p);
  return cudaGetLastError();
}

}  // namespace mla
