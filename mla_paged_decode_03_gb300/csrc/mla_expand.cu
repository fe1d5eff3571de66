// Keys and values of all heads from the pages' latent rows (the expanded form of latent
// attention): for row r of the output, that request b's local key l gives (r = kv_starts[b] + l),
//   kv[h, r, 0:256] = W[h] c,   k_rope[r] = c[512:576],
// with c the key's cache row (times its scale in the 8-bit form) and W[h] the 256 x 512 weights of
// head h (128 dims of its key, then 128 of its value).
//
// A matrix product of K = 512 with gathered rows: 1,024 operations for each 2-byte output, so
// bound by the tensor cores, with an output stream of over half the memory's rate beside it.
//
// Design.  A pair of SMs (a cluster of two, cta_group::2) computes tiles of 256 rows x 128 output dims
// (half of a head).  The gathered rows are the A operand and stay in tensor memory, 128 rows an SM
// (512 dims are 256 columns), since each is used for all heads; 256 more columns are two accumulators,
// so that one is written out while the other is computed.  Only W passes through shared memory, by
// TMA, 64 of a tile's 128 dims on each SM: 32 KB (64 dims x 256 latent dims) in a ring of five, 32 bytes
// a clock and SM at the full rate of the products (a tile of 128 rows on each SM by itself takes twice
// that, and was bound by it: 223 us for 8,192 rows and 128 heads).  The tiles of all row pairs are one
// sequence, row pair after row pair, cut evenly over the clusters; a cluster gathers rows only when
// its row pair changes.  The first SM of a pair issues all products.
//
// Rows are gathered by eight warps (two sets, which take 128 dims in turn), eight lanes a row so that a
// load reads whole lines, and turned by lane exchanges into a lane a row for tensor memory: any page
// size and any start, and the 8-bit form's conversion costs nothing but there.  Outputs leave by two
// sets of four warps, a set an accumulator, through shared memory as rows of 256 bytes.
//
// Measured: 8,192 rows x 128 heads in 170 to 189 us (1.46 to 1.62 PFLOP/s by the clock that the power
// limit leaves, 3 TB/s written), 67,583 8-bit rows x 32 heads in 300 to 352 (1.89 to 1.61 PFLOP/s);
// 2,064 rows x 8 heads in 10.6, nearly all of it the way of the first rows and weights and the last outputs.
//
// Safety: every wait is bounded (sm100.cuh); rows of no request, and pages or lengths out of range,
// are read as zeros and not written (the latter flagged).
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <functional>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "internal.h"
#include "lanes.cuh"
#include "sm100.cuh"
#include "tma_map.h"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kLatent = 512, kRow = 576;
constexpr int kM = 128, kN = 128;                  // rows an SM, output dims of a tile
constexpr int kStageDims = 256;                    // latent dims of a stage of W
constexpr int kBoxBytes = (kN / 2) * 128;          // 64 dims of W x 64 latent dims, bf16
constexpr int kStageBytes = kStageDims / 64 * kBoxBytes;
constexpr int kStages = 5;
constexpr int kRowDims = 128;                      // latent dims that are handed over with a row tile
constexpr int kRowSteps = kLatent / kRowDims;
// warp 0 TMA, 1 MMA; 4-7 and 8-11 outputs, a set an accumulator; 12-15 and 16-19 rows, a set every other
// 128 dims
constexpr int kThreads = 640;
constexpr uint32_t kColD = 256;                    // accumulators; A is columns 0..255

constexpr int kOffStage = kStages * kStageBytes;   // 8 warps x 32 rows x 256 bytes
constexpr int kOffBar = kOffStage + 8 * 32 * 256;
constexpr int kOffMisc = kOffBar + 512;
constexpr int kSmemBytes = kOffMisc + 64 + 1024;

// Those marked "pair" are the first SM's, for both; commits arrive on the others in both SMs.
enum Bar : int {
  B_FULL = 0,                    // [5] pair: W here, both SMs' parts
  B_EMPTY = B_FULL + kStages,    // [5] the products have read it
  B_AFULL = B_EMPTY + kStages,   // [4] pair: 128 dims of the rows in tensor memory
  B_AFREE = B_AFULL + kRowSteps,    // [4] the row tile's last product of these dims is done
  B_DFULL = B_AFREE + kRowSteps,    // [2]
  B_DFREE = B_DFULL + 2,         // [2] pair
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
    if (__all_sync(0xffffffffu, cluster ? mbar_try_wait_cluster(bar(i), parity) : mbar_try_wait(bar(i), parity)))
      return true;
    return __all_sync(0xffffffffu, mbar_wait_slow(bar(i), parity, abort, status, wait_ns, cluster));
  }
};

// The key that output row r holds (a row a lane): the request is the last one that starts at r or before.
struct Key {
  const uint8_t* row;            // null: none
  float scale;
};

template <bool kQ8>
__device__ __forceinline__ Key find_key(const ExpandArgs& a, int r, int lane, unsigned& flags) {
  Key k{nullptr, 0.f};
  int lo = 0, start = 0, have = 0;              // requests that start at r or before
  if (a.B <= 32) {
    // a request a lane, one round trip
    const int mine = lane < a.B ? __ldg(a.starts + lane) : INT_MAX;
    const int lens = lane < a.B ? __ldg(a.seq_lens + lane) : 0;
    for (int b = 0; b < a.B; ++b) lo += __shfl_sync(0xffffffffu, mine, b) <= r;
    start = __shfl_sync(0xffffffffu, mine, max(lo - 1, 0));
    have = __shfl_sync(0xffffffffu, lens, max(lo - 1, 0));
  } else {
    int hi = a.B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.starts + mid) <= r) lo = mid + 1;
      else hi = mid;
    }
    if (lo > 0) {
      start = __ldg(a.starts + lo - 1);
      have = __ldg(a.seq_lens + lo - 1);
    }
  }
  if (lo == 0 || r >= a.S) return k;
  const int b = lo - 1;
  const unsigned l = (unsigned)r - (unsigned)start;                    // r >= start
  if (have > a.max_blocks * a.block_size) {                            // (below 2^31)
    have = a.max_blocks * a.block_size;
    flags |= MLA_STATUS_SEQ_TOO_LONG;
  }
  if (have < 0 || l >= (unsigned)have) return k;
  const unsigned blk = l / (unsigned)a.block_size, off = l - blk * (unsigned)a.block_size;
  const int page = __ldg(a.block_table + (long long)b * a.bt_stride + blk);
  if (page < 0 || page >= a.num_blocks) {
    flags |= MLA_STATUS_BAD_PAGE;
    k.row = nullptr;
    k.scale = -1.f;              // a row of the request all the same: zeros are written
    return k;
  }
  const long long slot = (long long)page * a.block_size + (int)off;
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

// A scale (positive, normal) is 2^e f, 1 <= f < 2: e4m3 values times 2^e are exact in bf16, and f multiplies the
// row's fp32 sums, so that no scale adds a rounding.  Warps whose rows all have f = 1, as the store makes them, skip
// that product (67,583 rows x 32 heads in a graph: 299 us, with it 308).
__device__ __forceinline__ float scale_power(float s) { return __uint_as_float(__float_as_uint(s) & 0xff800000u); }
__device__ __forceinline__ float scale_rest(float s) { return __uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u); }

// 128 bytes of the rows of a warp's lanes, from byte `at` on, each lane its own row's; absent rows
// give zeros.  Eight lanes read a row's.
__device__ __forceinline__ void load_rows(const uint8_t* row, int at, int lane, uint32_t (&v)[32]) {
  const unsigned long long mine = reinterpret_cast<unsigned long long>(row);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, (lane & 24) + r));
    uint4 x = make_uint4(0, 0, 0, 0);
    if (src != nullptr) x = __ldg(reinterpret_cast<const uint4*>(src + at) + (lane & 7));
    v[4 * r] = x.x;
    v[4 * r + 1] = x.y;
    v[4 * r + 2] = x.z;
    v[4 * r + 3] = x.w;
  }
}
// 64 e4m3 values from word kFirst on, times the scale, as 32 words of two bf16 (exact for powers of two).
template <int kFirst>
__device__ __forceinline__ void widen(const uint32_t (&v)[32], float scale, uint32_t (&o)[32]) {
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    uint32_t h;
    const uint16_t two = (uint16_t)(v[kFirst + (q >> 1)] >> (16 * (q & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[q] = pack(f.x * scale, f.y * scale);
  }
}

// A cluster's tiles: of row pair `pair` from output tile `col` on, `n` of them, row pair after row pair.
struct Range {
  int pair, col, n;
};
// Tiles are cut evenly over the C clusters; or each row pair's over clusters of its own, where that
// gives none more than kGather tiles more: the rows of a second row pair are gathered in about that
// time.  (76 clusters, 128 heads; tiles of the busiest cluster cut evenly and by row pairs, times:
// 2,048 rows 27 and 29, 52.4 and 47.5 us; 2,816 rows 38 and 43, 63.5 and 63.8; 4,096 rows 54 and 64,
// 90 and 97.)
constexpr int kGather = 6;
__device__ __forceinline__ Range cut(unsigned pairs, unsigned cols, unsigned C, unsigned c) {
  const unsigned all = pairs * cols;             // below 2^31 - 256
  unsigned u0 = 0, u1 = 0;
  if (pairs > 0 && pairs <= C && (cols + C / pairs - 1) / (C / pairs) <= all / C + kGather) {
    const unsigned mp = ((c + 1) * pairs - 1) / C;             // its clusters: from c0, before c1
    const unsigned c0 = mp * C / pairs, c1 = (mp + 1) * C / pairs;
    u0 = mp * cols + cols * (c - c0) / (c1 - c0);
    u1 = mp * cols + cols * (c + 1 - c0) / (c1 - c0);
  } else {
    u0 = (unsigned)((unsigned long long)all * c / C);
    u1 = (unsigned)((unsigned long long)all * (c + 1) / C);
  }
  Range r;
  r.pair = (int)(u0 / cols);
  r.col = (int)(u0 - (u0 / cols) * cols);
  r.n = (int)(u1 - u0);
  return r;
}

// ---- instructions of a pair of SMs ------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive on a barrier at a shared::cluster address.  What is handed over lies in tensor memory, which
// tcgen05's own waits and fences order; with .release.cluster the arrival waited until the output
// rows stored before it had reached the L2 (2,000 clocks and more a tile).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// A tile into this SM's shared memory, its bytes counted by the barrier at a shared::cluster address
// (the pair's first SM's).  Warp-collective.
__device__ __forceinline__ void tma_load_2d_pair_warp(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                      uint32_t cluster_bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}
// Eight products along K (A: tensor memory columns +8 each; B: +32 bytes each, the second four in the
// next box), 256 rows on two SMs; `add` applies to the first.  Warp-collective, one election.
__device__ __forceinline__ void mma8_pair_warp(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 y;\n .reg .b64 k;\n"
      " setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
      " add.u32 y, %1, 8; add.u64 k, %2, 2;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 16; add.u64 k, %2, 4;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 24; add.u64 k, %2, 6;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 32; add.u64 k, %2, 512;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 40; add.u64 k, %2, 514;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 48; add.u64 k, %2, 516;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n"
      " add.u32 y, %1, 56; add.u64 k, %2, 518;\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], [y], k, %3, t;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// An arrival on `bar` in both SMs once all products before are done.
__device__ __forceinline__ void commit_pair_warp(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::
          "r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
static_assert(kBoxBytes / 16 == 512, "the second box's descriptors");

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
      mbar_init(s.bar(B_EMPTY + i), 1);
    }
    for (int i = 0; i < kRowSteps; ++i) {
      mbar_init(s.bar(B_AFULL + i), 8);
      mbar_init(s.bar(B_AFREE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s.bar(B_DFULL + i), 1);
      mbar_init(s.bar(B_DFREE + i), 8);
    }
    mbar_init(s.bar(B_DRAIN), 1);
    fence_mbar_init();
  }
  if (tid == 32) prefetch_tensormap(&wmap);
  if (warp == 1) {
    tmem_alloc_pair(s.base + kOffMisc, 512);
    tmem_relinquish_pair();
  }
  grid_wait();
  grid_release();
  // rows in use: the last request's end (requests are in the order of their rows)
  long long end = (long long)__ldg(p.a.starts + p.a.B - 1) + max(0, __ldg(p.a.seq_lens + p.a.B - 1));
  const int rows = (int)(end < 0 ? 0 : end > p.a.S ? p.a.S : end);
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();        // the barriers are initialised (fence_mbar_init) in both SMs
  tc_fence_after();
  const uint32_t tmem = misc[0];

  const Range range = cut((rows + 2 * kM - 1) / (2 * kM), p.col_tiles, nclusters_x(), cluster_id_x());
  unsigned flags = 0;

  if (warp == 0) {
    // ---- W: this SM's 64 of a tile's 128 dims ---------------------------------------------
    int st = 0;
    uint32_t par = 1;
    unsigned issued = 0;
    bool ok = true;
    int col = range.col;
    for (int i = 0; i < range.n && ok; ++i, col = col + 1 == p.col_tiles ? 0 : col + 1) {
      const int n0 = col * kN + (kN / 2) * (int)cr;
      for (int k = 0; k < kLatent; k += kStageDims) {
        ok = s.wait(B_EMPTY + st, par, true);
        if (!ok) break;
        if (cr == 0) mbar_arrive_expect_tx_warp(s.bar(B_FULL + st), 2 * kStageBytes);
        const uint32_t full = mapa(s.bar(B_FULL + st), 0), dst = s.base + st * kStageBytes;
#pragma unroll
        for (int c = 0; c < kStageDims / 64; ++c)
          tma_load_2d_pair_warp(dst + c * kBoxBytes, &wmap, k + 64 * c, n0, full);
        ++issued;
        if (++st == kStages) {
          st = 0;
          par ^= 1u;
        }
      }
    }
    // the last releases arrive here, and so all copies have, before this SM ends
    for (unsigned m = issued > kStages ? issued - kStages : 0; m < issued && ok; ++m)
      ok = s.wait(B_EMPTY + (int)(m % kStages), m / kStages & 1, true);
    if (!ok) {
      // after an abort: the first SM waits for the copies that it counts, the other one, whose copies
      // are counted there, for as long as any copy takes
      for (unsigned m = issued > kStages ? issued - kStages : 0; m < issued && cr == 0; ++m)
        mbar_wait_drain(s.bar(B_FULL + (int)(m % kStages)), m / kStages & 1);
      const unsigned long long t0 = globaltimer();
      while (globaltimer() - t0 < 100000ull) {
      }
    }
  } else if (warp == 1) {
    // ---- products (the first SM's warp, for both) -------------------------------------------
    const uint32_t idesc = idesc_bf16(2 * kM, kN, false, false);
    const uint64_t wd = smem_desc(s.base, 16, 1024, kSwizzle128B);
    int st = 0;
    uint32_t par = 0, apar = 0;
    bool ok = cr == 0;
    int col = range.col;
    for (int n = 0; n < range.n && ok; ++n, col = col + 1 == p.col_tiles ? 0 : col + 1) {
      const bool fresh = n == 0 || col == 0;
      const bool last = n + 1 == range.n || col + 1 == p.col_tiles;
      const int g = n & 1;
      ok = s.wait(B_DFREE + g, (uint32_t)(((n >> 1) + 1) & 1), true);
#pragma unroll
      for (int k = 0; k < kRowSteps && ok; ++k) {
        const bool stage = k % (kStageDims / kRowDims) == 0;        // W's next stage begins
        if (fresh) ok = s.wait(B_AFULL + k, apar, true);
        if (stage) ok = ok && s.wait(B_FULL + st, par, true);
        if (!ok) break;
        if (fresh || stage) tc_fence_after();
        mma8_pair_warp(tmem + kColD + g * kN, tmem + 64 * k,
                       wd + st * (kStageBytes / 16) + (stage ? 0 : 2 * kBoxBytes / 16), idesc, k != 0);
        if (last) commit_pair_warp(s.bar(B_AFREE + k));
        if (stage) continue;
        commit_pair_warp(s.bar(B_EMPTY + st));
        if (++st == kStages) {
          st = 0;
          par ^= 1u;
        }
      }
      if (!ok) break;
      commit_pair_warp(s.bar(B_DFULL + g));
      if (fresh) apar ^= 1u;
    }
    if (cr == 0) commit_pair_warp(s.bar(B_DRAIN));
  } else if (warp >= 12) {
    // ---- rows into tensor memory: thread = row ------------------------------------------
    const uint32_t ta = tmem + ((uint32_t)(warp & 3) << 21);
    const int set = warp >= 16;
    bool ok = true;
    uint32_t m = 0;
    // its row pairs: the first from output tile range.col on, the others from 0
    for (int col = range.col, left = range.n; left > 0 && ok; left -= p.col_tiles - col, col = 0, ++m) {
      const int r = ((range.pair + (int)m) * 2 + (int)cr) * kM + (warp & 3) * 32 + lane;
      const Key key = find_key<kQ8>(p.a, r, lane, flags);
#pragma unroll 1
      for (int k = set; k < kRowSteps; k += 2) {
        // 128 dims of the row: 128 bytes of e4m3 or twice that of bf16
        uint32_t v[32], w[32];
        load_rows(key.row, kRowDims * (kQ8 ? 1 : 2) * k, lane, v);
        if (!kQ8) load_rows(key.row, kRowDims * 2 * k + 128, lane, w);
        ok = s.wait(B_AFREE + k, (m + 1) & 1, true);
        if (!ok) break;
        tc_fence_after();
        transpose8(v, lane);
        if (kQ8) {
          uint32_t o[32];
          widen<0>(v, scale_power(key.scale), o);
          tmem_st32(ta + 64 * k, o);
          widen<16>(v, scale_power(key.scale), o);
          tmem_st32(ta + 64 * k + 32, o);
        } else {
          tmem_st32(ta + 64 * k, v);
          transpose8(w, lane);
          tmem_st32(ta + 64 * k + 32, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(mapa(s.bar(B_AFULL + k), 0));
      }
      if (!ok) break;
      // the cluster that has a row tile's first unit copies its rope keys
      if (set == 0 && col == 0) {
        const bool mine = key.row != nullptr || key.scale != 0.f;
        uint8_t* out = reinterpret_cast<uint8_t*>(p.a.k_rope + (long long)r * 64);
        if (kQ8) {
          if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(out);
            const uint4* src = reinterpret_cast<const uint4*>(key.row + kLatent);
            uint32_t v[32], o[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x = key.row != nullptr ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
              v[4 * i] = x.x;
              v[4 * i + 1] = x.y;
              v[4 * i + 2] = x.z;
              v[4 * i + 3] = x.w;
            }
            widen<0>(v, key.scale, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        } else {
          // bit for bit, eight lanes a row
          uint32_t v[32];
          load_rows(key.row, 2 * kLatent, lane, v);
          const unsigned rows_here = __ballot_sync(0xffffffffu, mine);
          out -= (lane & 7) * 128 - (lane & 7) * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (rows_here >> ((lane & 24) + i) & 1u)
              *reinterpret_cast<uint4*>(out + i * 128) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    }
  } else if (warp >= 4) {
    // ---- outputs: accumulator rows (thread = row) -> 256 bytes a row in shared memory ->
    // half a warp a row to memory
    const int q = warp & 3, g = (warp >> 2) - 1;  // the set's accumulator: every other tile
    uint8_t* stage = sp + kOffStage + (warp - 4) * 32 * 256;
    const uint32_t td = tmem + kColD + g * kN + ((uint32_t)q << 21);
    unsigned valid = 0;                           // the warp's rows that are somebody's
    float rest = 1.f;                             // scale_rest of the thread's row
    bool powers = true;                           // and whether the warp's are all 1
    bool ok = true;
    int m0 = -1, mp = range.pair, nt = range.col + g;
    for (int n = 0; 2 * n + g < range.n && ok; ++n, nt += 2) {
      while (nt >= p.col_tiles) {
        nt -= p.col_tiles;
        ++mp;
      }
      const int r0 = (mp * 2 + (int)cr) * kM + q * 32;
      if (mp != m0) {
        unsigned f = 0;
        const Key key = find_key<kQ8>(p.a, r0 + lane, lane, f);
        valid = __ballot_sync(0xffffffffu, key.row != nullptr || key.scale != 0.f);
        if (kQ8) {
          rest = scale_rest(key.scale);
          powers = __all_sync(0xffffffffu, rest == 1.f);
        }
        m0 = mp;
      }
      ok = s.wait(B_DFULL + g, n & 1, true);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t v[32];
        tmem_ld32(td + 32 * h, v);
        tmem_wait_ld();
        if (kQ8 && !powers) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * rest);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 o;
          o.x = pack(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1]));
          o.y = pack(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3]));
          o.z = pack(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5]));
          o.w = pack(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7]));
          *reinterpret_cast<uint4*>(stage + lane * 256 + (((4 * h + i) ^ (lane & 7)) << 4)) = o;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(mapa(s.bar(B_DFREE + g), 0));
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
  if (*s.abort && lane == 0) {
    st_cluster_u32(mapa(smem_u32((const void*)(sp + kOffMisc + 4)), cr ^ 1), 1);
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // every product is done before either SM ends (it reads both SMs' memory)
  if (warp == 1) mbar_wait_drain(s.bar(B_DRAIN), 0);
  __syncwarp();
  cluster_sync_relaxed();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
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
  const int units = (a.S + 2 * kM - 1) / (2 * kM) * p.col_tiles;
  const int clusters = units < g_dev[dev].clusters ? units : g_dev[dev].clusters;
  DependentLaunch dl(dim3(2 * clusters), dim3(kThreads), stream, kSmemBytes);
  if (a.scales != nullptr) return cudaLaunchKernelEx(&dl.cfg, mla_expand_kernel<true>, wmap, p);
  return cudaLaunchKernelEx(&dl.cfg, mla_expand_kernel<false>, wmap, p);
}

}  // namespace mla
