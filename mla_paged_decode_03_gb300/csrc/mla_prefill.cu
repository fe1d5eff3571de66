// Attention of chunks of new tokens (ragged) over the heads' expanded keys and values, sm_103a.
//
// Query row i of the n that request b brings sees L_i of its local keys (mla_decode's bound: the
// global prefix G_i = G_b - (n-1-i), of which this shard holds local_len(G_i); all keys where the
// block is not causal):
//   s_l = scale (<q[0:128], k_nope_l> + <q[128:192], k_rope_l>),
//   out = sum_l softmax(s)_l v_l,  lse = log sum_l exp(s_l).
// k_rope is shared by the heads and read as it is, so that a head's keys are 128 wide in memory.
//
// Bound by the tensor cores on long chunks (640 operations a row and key against 512 bytes a key
// and head), by memory on chunks below some 150 rows.
//
// Design.  A block takes 256 query rows of one request and head, as two streams of 128 rows that
// share every key and value tile (128 keys); per tile and stream 12 products of 128 x 128 x 16 for
// S = Q K^T (768 clocks) and 8 for O += P V (512).  Tensor memory holds S (then P in its place) and
// O of both streams: 4 x 128 columns.  One warp issues PV of a stream's tile j-1 and QK of its tile j
// back to back and then turns to the other stream: while a stream's softmax (128 threads, a row
// each) works, the tensor cores work for the other.  Products complete in the order of issue, so
// that S of tile j, once there, says that PV of tile j-1 is done: the softmax threads may rescale O
// then without another barrier, which they do only where a row's maximum rose by more than 2^8.
// Shared memory: Q of both streams (96 KB) and a ring of eight 16 KB slots: three of keys (128 keys
// x 64 dims) and two of values (64 keys x 128 dims) a tile.
//
// Blocks run the last (longest) rows of a request first; neighbouring blocks share a head's keys in
// the L2.  Where all blocks would not fill the SMs, each request's tiles are cut into parts whose
// partial results (fp32) the LSE combine joins.
//
// Safety: every wait is bounded (sm100.cuh); lengths and starts out of range are clamped and
// flagged; value rows behind a request's last key are zeroed in shared memory before they meet P
// (they may hold anything), rows of other requests are computed but not stored.
#include <math.h>
#include <stdint.h>

#include <functional>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>

#include "internal.h"
#include "sm100.cuh"
#include "tma_map.h"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kM = 128;                       // rows a stream
constexpr int kTile = 128;                    // keys a tile
constexpr int kSlotBytes = 16384;
constexpr int kSlots = 8;
constexpr int kQChunks = 3, kKSlots = 3, kVSlots = 2;
// Group 2j is tile j's keys, group 2j + 1 its values; the slots they take one after another make
// group n's slots free once group n - 3 has been used.
constexpr int kGroups = 3;
constexpr int kThreads = 384;                 // warp 0 TMA; 1, 2 MMA and 4-7, 8-11 softmax of a stream
constexpr float kRise = 8.0f;                 // log2 units that a maximum may rise before O is rescaled

constexpr int kOffQ = 0;                                     // 2 x 48 KB, then the output's staging
constexpr int kOffRing = 2 * kQChunks * kSlotBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kOffMisc = kOffBar + 256;
constexpr int kSmemBytes = kOffMisc + 128 + 1024;

enum Bar : int {
  B_QFULL = 0,                   // [2]
  B_FULL = 2,                    // [3] keys or values of a tile
  B_EMPTY = B_FULL + kGroups,    // [3] both streams have used them
  B_SFULL = B_EMPTY + kGroups,   // [2] S of a stream's tile computed (and all products before)
  B_PFULL = B_SFULL + 2,         // [2][2] P of half a tile in tensor memory, O rescaled
  B_OFULL = B_PFULL + 4,         // [2] the stream's last product is done
  B_TURN = B_OFULL + 2,          // [2] a stream's products may be issued
  B_DRAIN = B_TURN + 2,          // [2]
  B_COUNT = B_DRAIN + 2
};
static_assert(B_COUNT * 8 <= 256, "barriers");

struct Ctx {
  uint32_t base;
  volatile int* abort;
  unsigned int* status;
  unsigned long long wait_ns;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + kOffBar + 8 * i; }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, status, wait_ns));
  }
};

// What a block works on.
struct Unit {
  int row0, n;                   // first row (of q) of the request's chunk, its rows
  int first;                     // the block's first row within the chunk
  int key0, keys;                // first key row, keys of the shard
  int global;                    // global length
};

// One warp: the request and rows of tile x.  False: there is no such tile.
__device__ bool find_unit(const PrefillArgs& a, int x, int lane, Unit& un) {
  unsigned flags = 0;
  int before = 0;                // tiles of the requests before this round's
  bool found = false;
  for (int b0 = 0; b0 < a.B && !found; b0 += 32) {
    const int b = b0 + lane;
    int row0 = 0, n = 0;
    if (b < a.B) {
      row0 = __ldg(a.cu + b);
      const int end = __ldg(a.cu + b + 1);
      if (row0 < 0 || end < row0 || end > a.T) flags |= MLA_STATUS_BAD_STEP;
      else n = end - row0;
    }
    const int tiles = (n + 2 * kM - 1) / (2 * kM);
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int at = x - (before + incl - tiles);
    const unsigned hit = __ballot_sync(0xffffffffu, at >= 0 && at < tiles);
    before += __shfl_sync(0xffffffffu, incl, 31);
    if (hit) {
      found = true;
      const int who = __ffs(hit) - 1;
      un.row0 = __shfl_sync(0xffffffffu, row0, who);
      un.n = __shfl_sync(0xffffffffu, n, who);
      // the last rows, which see the most keys, first
      un.first = 2 * kM * __shfl_sync(0xffffffffu, tiles - 1 - at, who);
      const int r = b0 + who;
      int keys = __ldg(a.seq_lens + r), key0 = __ldg(a.starts + r), g = keys;
      if (a.gseq != nullptr) g = __ldg(a.gseq + r);
      if (keys < 0 || key0 < 0 || keys > a.S - key0) {
        flags |= MLA_STATUS_BAD_STEP;
        key0 = min(max(key0, 0), a.S);
        keys = min(max(keys, 0), a.S - key0);
      }
      un.key0 = key0;
      un.keys = keys;
      un.global = g;
    }
  }
  if (flags) atomicOr(a.status, flags);
  return found;
}

// Keys that row i of the chunk sees.
__device__ __forceinline__ int seen(const PrefillArgs& a, const Unit& u, int i) {
  if (!a.causal) return u.keys;
  const long long g = (long long)u.global - (u.n - 1 - i);
  if (g <= 0) return 0;
  long long l = g;
  if (a.cp > 1) {
    const long long span = (long long)a.cp * a.il;
    const long long rem = g % span - (long long)a.rank * a.il;
    l = g / span * a.il + (rem < 0 ? 0 : rem > a.il ? a.il : rem);
  }
  return (int)(l < u.keys ? l : u.keys);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two single-precision multiply-adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__global__ void __launch_bounds__(kThreads, 1)
mla_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sp = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // blocks of one group of heads after another; in a group all heads' longest tiles first
  const unsigned per = (unsigned)a.tiles * a.group;
  const unsigned grp = blockIdx.x / per, in = blockIdx.x - grp * per;
  const unsigned heads = min((unsigned)a.group, (unsigned)a.H - grp * a.group);
  const int tile_x = (int)(in / heads), head = (int)(grp * a.group + in % heads);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sp + kOffMisc);
  Unit* su = reinterpret_cast<Unit*>(sp + kOffMisc + 16);
  Ctx s;
  s.base = smem_u32(sp);
  s.abort = reinterpret_cast<volatile int*>(misc + 1);
  s.status = a.status;
  s.wait_ns = a.wait_ns;

  if (warp == 0) {
    Unit u;
    const bool any = find_unit(a, tile_x, lane, u);
    if (lane == 0) {
      misc[2] = any;
      if (any) *su = u;
    }
  } else if (warp == 1) {
    tmem_alloc(s.base + kOffMisc, 512);
    tmem_relinquish();
  } else if (tid == 96) {
    *s.abort = 0;
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(s.bar(i), i >= B_PFULL && i < B_PFULL + 4 ? 4 : i >= B_EMPTY && i < B_EMPTY + kGroups ? 2 : 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const bool any = misc[2] != 0;

  if (any) {
    const Unit un = *su;
    // tiles of each stream: the bound grows with the row, so a stream's last row has the most
    int begin = 0, tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int i0 = un.first + t * kM;
      tiles[t] = i0 < un.n ? (seen(a, un, min(i0 + kM, un.n) - 1) + kTile - 1) / kTile : 0;
    }
    if (a.splits > 1) {
      const int most = max(tiles[0], tiles[1]);
      begin = (int)((long long)most * blockIdx.y / a.splits);
      const int end = (int)((long long)most * (blockIdx.y + 1) / a.splits);
      tiles[0] = max(min(tiles[0], end), begin);
      tiles[1] = max(min(tiles[1], end), begin);
    }
    const int most = max(max(tiles[0], tiles[1]), begin);

    if (warp == 0) {
      // ---- loads --------------------------------------------------------------------------
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (tiles[t] > begin) {
          mbar_arrive_expect_tx_warp(s.bar(B_QFULL + t), kQChunks * kSlotBytes);
          for (int c = 0; c < kQChunks; ++c)
            tma_load_3d_warp(s.base + kOffQ + (t * kQChunks + c) * kSlotBytes, &qmap, 64 * c, head,
                             un.row0 + un.first + t * kM, s.bar(B_QFULL + t));
        }
      int sl = 0, g = 0, issued = 0;
      uint32_t par = 1;
      bool ok = true;
      for (int j = begin; j < most && ok; ++j) {
        const int y = un.key0 + j * kTile;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          ok = s.wait(B_EMPTY + g, par);
          if (!ok) break;
          const uint32_t fb = s.bar(B_FULL + g);
          mbar_arrive_expect_tx_warp(fb, (part == 0 ? kKSlots : kVSlots) * kSlotBytes);
#pragma unroll
          for (int c = 0; c < (part == 0 ? kKSlots : kVSlots); ++c) {
            const uint32_t dst = s.base + kOffRing + sl * kSlotBytes;
            if (part == 1) {
              tma_load_3d_warp(dst, &vmap, 0, head, y + 64 * c, fb);
              tma_load_3d_warp(dst + kSlotBytes / 2, &vmap, 64, head, y + 64 * c, fb);
            } else if (c < 2) {
              tma_load_3d_warp(dst, &kmap, 64 * c, head, y, fb);
            } else {
              tma_load_2d_warp(dst, &rmap, 0, y, fb);
            }
            sl = (sl + 1) % kSlots;
          }
          ++issued;
          if (++g == kGroups) {
            g = 0;
            par ^= 1u;
          }
        }
      }
      if (*s.abort) {
        // let loads in flight land before the block ends
        for (int m = issued > kGroups ? issued - kGroups : 0; m < issued; ++m)
          mbar_wait_drain(s.bar(B_FULL + m % kGroups), (uint32_t)((m / kGroups) & 1));
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (tiles[t] > begin) mbar_wait_drain(s.bar(B_QFULL + t), 0);
      }
    } else if (warp <= 2) {
      // ---- products of a stream, the streams in turn ------------------------------------------
      const int t = warp - 1;
      const uint32_t id_qk = idesc_bf16(kM, kTile, false, false), id_pv = idesc_bf16(kM, 128, false, true);
      const uint64_t qd = smem_desc(s.base + kOffQ + t * kQChunks * kSlotBytes, 16, 1024, kSwizzle128B);
      const uint64_t kd = smem_desc(s.base + kOffRing, 16, 1024, kSwizzle128B);
      const uint64_t vd = smem_desc(s.base + kOffRing, kSlotBytes / 2, 1024, kSwizzle128B);
      constexpr unsigned kStep = kSlotBytes / 16;
      const uint32_t ds = tmem + t * 128, d_o = ds + 256;
      const int mine = tiles[t];
      bool ok = begin >= mine || s.wait(B_QFULL + t, 0);
      unsigned sl = 0;                          // slot of tile j's keys
      int g = 0;                                // its group's barriers, and their parity
      uint32_t par = 0, ph = 0;                 // parity of the tile before, and of the turn
      for (int j = begin; j <= most && ok; ++j) {
        const int gv = g == 0 ? kGroups - 1 : g - 1;      // tile j - 1's values: the group and slots before
        const unsigned v0 = (sl + kSlots - 2) % kSlots, v1 = (sl + kSlots - 1) % kSlots;
        const bool pv = j > begin && j <= mine, qk = j < mine;
        if (pv) {
          ok = s.wait(B_FULL + gv, g == 0 ? par ^ 1u : par);
          const int left = un.keys - (j - 1) * kTile;
          if (ok && left < kTile) {
            // rows behind the last key: P is zero there, the values may be anything
            for (int h = 0; h < kVSlots; ++h) {
              uint8_t* v = sp + kOffRing + (h == 0 ? v0 : v1) * kSlotBytes;
              for (int i = max(left - 64 * h, 0) * 8 + lane; i < 64 * 8; i += 32) {
                *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(v + kSlotBytes / 2 + i * 16) = make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          ok = ok && s.wait(B_PFULL + 2 * t, ph ^ 1u);
        }
        // the other stream's products are issued
        if (t == 1 || j > begin) ok = ok && s.wait(B_TURN + t, t == 1 ? ph : ph ^ 1u);
        if (!ok) break;
        tc_fence_after();
        if (pv) {
          mma4_ts_mn_warp(d_o, ds, vd + v0 * kStep, id_pv, j - 1 > begin);
          ok = s.wait(B_PFULL + 2 * t + 1, ph ^ 1u);
          if (!ok) break;
          tc_fence_after();
          mma4_ts_mn_warp(d_o, ds + 32, vd + v1 * kStep, id_pv, 1);
        }
        if (j > begin) mma_commit_warp(s.bar(B_EMPTY + gv));
        if (qk) {
          ok = s.wait(B_FULL + g, par);
          if (!ok) break;
          tc_fence_after();
          mma12_ss_warp(ds, qd, kd + sl * kStep, kd + (sl + 1) % kSlots * kStep, kd + (sl + 2) % kSlots * kStep, id_qk);
          mma_commit_warp(s.bar(B_SFULL + t));
        }
        if (lane == 0) mbar_arrive(s.bar(B_TURN + (t ^ 1)));
        __syncwarp();
        if (pv && j == mine) mma_commit_warp(s.bar(B_OFULL + t));
        if (j < most) mma_commit_warp(s.bar(B_EMPTY + g));
        sl = (sl + kKSlots + kVSlots) % kSlots;
        ph ^= 1u;
        g += 2;
        if (g >= kGroups) {
          g -= kGroups;
          par ^= 1u;
        }
      }
      mma_commit_warp(s.bar(B_DRAIN + t));
      mbar_wait_drain(s.bar(B_DRAIN + t), 0);
    } else if (warp >= 4) {
      // ---- softmax: thread = row ------------------------------------------------------------
      const int t = (warp >> 2) - 1, q = warp & 3;
      const int i0 = un.first + t * kM + q * 32;               // the warp's first row in the chunk
      const int mine = seen(a, un, min(i0 + lane, un.n - 1));  // rows behind the chunk: not stored
      const int least = __shfl_sync(0xffffffffu, mine, 0);
      const uint32_t ts = tmem + ((uint32_t)q << 21) + t * 128, to = ts + 256;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      const int n_tiles = tiles[t];
      for (int j = begin; j < n_tiles; ++j) {
        ok = s.wait(B_SFULL + t, (uint32_t)((j - begin) & 1));
        if (!ok) break;
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
        tmem_wait_ld();
        if (least < (j + 1) * kTile) {
          const int lim = mine - j * kTile;
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = c < lim ? x[c] : -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], x[c + 2 * k], x[c + 2 * k + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], x[124 + k]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        // the reference moves where a maximum rose too far (from nothing at the first)
        const bool moves = top > m + kRise;
        if (__any_sync(0xffffffffu, moves)) {
          const float f = moves ? exp2_fast(m - top) : 1.f;
          if (moves) m = top;
          l *= f;
          if (j > begin)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(to + 32 * c, o);
            }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 mul = make_float2(a.scale_log2, a.scale_log2), sub = make_float2(-ref, -ref);
        const float2 one = make_float2(1.f, 1.f);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // P of 64 keys, then of the other 64: the first half's product starts meanwhile
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 e = fma2(make_float2(x[64 * h + 2 * k], x[64 * h + 2 * k + 1]), mul, sub);
            const float2 p = make_float2(exp2_fast(e.x), exp2_fast(e.y));
            sum[k & 1] = fma2(p, one, sum[k & 1]);
            pk[k] = pack(p.x, p.y);
          }
          tmem_st32(ts + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s.bar(B_PFULL + 2 * t + h));
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (ok && n_tiles > begin) {
        ok = s.wait(B_OFULL + t, 0);
        tc_fence_after();
      }
      const int rows = un.n - i0;                              // the warp's rows that are stored
      if (ok && rows > 0) {
        const long long row = (long long)(un.row0 + i0) * a.H + head;
        const bool none = l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        uint8_t* stage = sp + kOffQ + t * kQChunks * kSlotBytes + q * 32 * 256;
        if (a.splits == 1) {
          if (a.lse != nullptr && lane < rows)
            a.lse[row + (long long)lane * a.H] = none ? -INFINITY : (m + log2f(l)) * a.lse_mul;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[64];
            if (n_tiles > begin) {
              tmem_ld32(to + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(v));
              tmem_ld32(to + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
              tmem_wait_ld();
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = none ? 0u : pack(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 256 + (((8 * h + k) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const int r = 2 * k + (lane >> 4), ch = lane & 15;
            if (r < rows)
              *reinterpret_cast<uint4*>(a.out + (row + (long long)r * a.H) * 128 + ch * 8) =
                  *reinterpret_cast<const uint4*>(stage + r * 256 + ((ch ^ (r & 7)) << 4));
          }
        } else {
          const long long part = (long long)blockIdx.y * a.T * a.H;
          if (lane < rows) a.ws_lse[part + row + (long long)lane * a.H] = none ? -INFINITY : m + log2f(l);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[64];
            if (n_tiles > begin) {
              tmem_ld32(to + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(v));
              tmem_ld32(to + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
              tmem_wait_ld();
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = none ? 0u : __float_as_uint(__uint_as_float(v[4 * k + e]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 256 + ((k ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll 4
            for (int k = 0; k < 16; ++k) {
              const int r = 2 * k + (lane >> 4), ch = lane & 15;
              if (r < rows)
                *reinterpret_cast<uint4*>(a.ws_o + (part + row + (long long)r * a.H) * 128 + 64 * h + ch * 4) =
                    *reinterpret_cast<const uint4*>(stage + r * 256 + ((ch ^ (r & 7)) << 4));
            }
            __syncwarp();
          }
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

struct PrefillDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
constexpr int kMaxDevices = 64;
PrefillDevice g_dev[kMaxDevices];

void device_setup(PrefillDevice& d) {
  d.err = cudaFuncSetAttribute(mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

long long row_tiles(int T, int B) { return (long long)T / (2 * kM) + (B < T ? B : T); }

// Parts that each request's keys are cut into: as many as fill the SMs, each of 256 keys or more
// if a request had all key rows.
int parts(int T, int B, int H, int S, int num_sms) {
  const long long blocks = row_tiles(T, B) * H;
  long long n = num_sms / (blocks > 0 ? blocks : 1);
  if (n > S / 256) n = S / 256;
  return n < 1 ? 1 : (int)n;
}

// Heads whose blocks run at a time, longest tiles first: as many as have their keys and values in half
// of the L2 together.
int head_group(int S, int H) {
  const long long n = (64LL << 20) / ((long long)S * 512);
  return n < 1 ? 1 : n < H ? (int)n : H;
}

size_t lse_bytes(int n, int T, int H) { return ((size_t)n * T * H * sizeof(float) + 255) / 256 * 256; }

}  // namespace

bool prefill_grid_ok(int T, int B, int H) { return row_tiles(T, B) * H < (1LL << 31); }

size_t prefill_workspace_size(int T, int B, int H, int S, int num_sms) {
  const int n = parts(T, B, H, S, num_sms);
  return n == 1 ? 0 : lse_bytes(n, T, H) + (size_t)n * T * H * 128 * sizeof(float);
}

cudaError_t launch_mla_prefill(PrefillArgs a, const PrefillTensors& x, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(g_dev[dev].once, device_setup, std::ref(g_dev[dev]));
  if (g_dev[dev].err != cudaSuccess) return g_dev[dev].err;
  a.splits = parts(a.T, a.B, a.H, a.S, a.num_sms);
  if (a.splits > 1) {
    if (x.workspace == nullptr || x.workspace_bytes < prefill_workspace_size(a.T, a.B, a.H, a.S, a.num_sms)) {
      a.splits = 1;
    } else {
      a.ws_lse = static_cast<float*>(x.workspace);
      a.ws_o = reinterpret_cast<float*>(static_cast<char*>(x.workspace) + lse_bytes(a.splits, a.T, a.H));
    }
  }
  // [rows][heads][dims] of q and v and of the keys' first part, boxes of one head; rope keys [rows][64]
  CUtensorMap qmap, kmap, rmap, vmap;
  const uint64_t H = (uint64_t)a.H, T = (uint64_t)a.T, S = (uint64_t)a.S;
  const uint64_t qd[3] = {192, H, T}, kd[3] = {128, H, S}, rd[2] = {64, S};
  // strides in bytes; that of a dimension of one is any
  const auto by = [](uint64_t n, int64_t stride) { return n > 1 ? (uint64_t)stride * 2 : (uint64_t)16; };
  const uint64_t qs[2] = {by(H, x.q_h), by(T, x.q_t)}, ks[2] = {by(H, x.k_h), by(S, x.k_s)},
                 vs[2] = {by(H, x.v_h), by(S, x.v_s)}, rs[1] = {by(S, x.r_s)};
  const uint32_t box[3] = {64, 1, 128}, vbox[3] = {64, 1, 64}, rbox[2] = {64, 128};
  if (!encode_tile_map(&qmap, x.q, 3, qd, qs, box) || !encode_tile_map(&kmap, x.k_nope, 3, kd, ks, box) ||
      !encode_tile_map(&rmap, x.k_rope, 2, rd, rs, rbox) || !encode_tile_map(&vmap, x.v, 3, kd, vs, vbox))
    return cudaErrorInvalidValue;
  a.tiles = (int)row_tiles(a.T, a.B);
  a.group = head_group(a.S, a.H);
  const dim3 grid((unsigned)a.tiles * (unsigned)a.H, (unsigned)a.splits);
  mla_prefill_kernel<<<grid, kThreads, kSmemBytes, stream>>>(qmap, kmap, rmap, vmap, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_lse_combine128(a.ws_o, true, a.ws_lse, a.splits, (long long)a.T * a.H, true, a.lse_mul, a.out,
                               a.lse, a.cu, a.B, a.H, stream);
}

}  // namespace mla
