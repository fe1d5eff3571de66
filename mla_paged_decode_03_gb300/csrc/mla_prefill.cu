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
// Design.  A unit of work is 256 query rows of one request and head, as two streams of 128 rows that
// share every key and value tile (128 keys); per tile and stream 12 products of 128 x 128 x 16 for
// S = Q K^T (768 clocks) and 8 for O += P V (512).  Tensor memory holds S (then P in its place) and
// O of both streams: 4 x 128 columns.  A warp a stream issues PV of tile j-1 and QK of tile j back to
// back, and the two warps do so in turn (issued as each is ready, both streams' softmax fell into step
// and the tensor cores idled): while a stream's softmax (128 threads, a row each) works, the tensor
// cores work for the other.  Products complete in the order of issue, so that S of tile j, once there,
// says that PV of tile j-1 is done: the softmax threads may rescale O then without another barrier,
// which they do only where a row's maximum rose by more than 2^8.  The first half's weights are
// computed beside the maximum, by the reference so far (at first the largest of four scores: none would
// mean all weights of a unit's first tile twice), and its PV starts before the second half's.
// Shared memory: Q of both streams (96 KB) and a ring of eight 16 KB slots: three of keys (128 keys
// x 64 dims, waited for one by one) and two of values (64 keys x 128 dims) a tile.
//
// Units are the grid's blocks, one of which runs on an SM for as long as there are others: it asks the
// launch for blocks that have not begun (clusterlaunchcontrol), so that the next unit's loads overlap
// the last one's output and long and short units even out.  It asks late, when a unit's last but one
// tile is on its way; asked for at a unit's start, the last units ran on a few SMs.  The last (longest)
// rows of a request come first; neighbouring units share a head's keys in the L2.  Where all units
// would not fill the SMs, each request's tiles are cut into parts whose partial results (fp32) the LSE
// combine joins.  Units of up to 128 rows take the streams by turns.  Outputs go
// from a row a thread to whole lines by lane exchanges.
//
// Measured, in a graph and as calls for a second: one prompt of 8,192 tokens x 128 heads in 1.47 and 1.68 ms
// (1.9 and 1.6 PFLOP/s of masked work; the clock falls to 1.4 GHz under the power limit); 512 tokens
// behind 32,256 x 8 heads in 60 and 63 us (1.4 PFLOP/s with the combine); 24 requests of 1 to 700 tokens,
// 32 heads, in 282 and 306, whose units of few tiles spend 4,000 to 7,000 clocks each on what no tile hides.
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
#include "lanes.cuh"
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
// Tiles take the ring's slots one after another: three of keys, two of values.  Tile g's first keys
// slot is free once the keys of tile g - 2 have been used, the other two once its values have, its
// values' once the keys of tile g - 1 have.
constexpr int kThreads = 384;                 // warp 0 TMA; 1, 2 MMA and 4-7, 8-11 softmax of a stream; 3 units
constexpr float kRise = 8.0f;                 // log2 units that a maximum may rise before O is rescaled

constexpr int kOffQ = 0;                                     // 2 x 48 KB
constexpr int kOffRing = 2 * kQChunks * kSlotBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kOffMisc = kOffBar + 320;
constexpr int kSmemBytes = kOffMisc + 160 + 1024;

enum Bar : int {
  B_QFULL = 0,                   // [2]
  B_QEMPTY = 2,                  // [2] the unit's last QK of a stream is done
  B_KFULL = 4,                   // [3][2] 64 dims of the keys of an even, an odd tile
  B_SFULL = B_KFULL + 6,         // [2] S of a stream's tile computed (and all products before)
  B_PFULL = B_SFULL + 2,         // [2][2] P of half a tile in tensor memory, O rescaled
  B_OFULL = B_PFULL + 4,         // [2] the unit's last product of a stream is done
  B_OFREE = B_OFULL + 2,         // [2] O read
  B_TURN = B_OFREE + 2,          // [2] a stream's products may be issued
  B_UFULL = B_TURN + 2,          // the next unit is known
  B_UEMPTY = B_UFULL + 1,        // every role has read it
  B_ASK = B_UEMPTY + 1,          // the unit's last but one tile is on its way
  B_NEXT = B_ASK + 1,            // the answer about the next block of the grid is here
  B_DRAIN = B_NEXT + 1,          // [2]
  B_VFULL = B_DRAIN + 2,         // [2] the values of an even, an odd tile
  B_KEMPTY = B_VFULL + 2,        // [2] both streams have used its keys
  B_VEMPTY = B_KEMPTY + 2,       // [2] and its values
  B_COUNT = B_VEMPTY + 2
};
static_assert(B_COUNT * 8 <= 320, "barriers");
constexpr int kReaders = 11;     // warps that read a unit: loads, products (2), softmax (8)
constexpr int kOffNext = kOffMisc + 16, kOffUnit = kOffMisc + 32;

extern __shared__ uint8_t smem_raw[];
__device__ __forceinline__ uint8_t* smem_1024(uint8_t* raw) { return raw + ((1024 - (smem_u32(raw) & 1023)) & 1023); }

// Warps that compute rows again (redo_rows): those at it in the lower half, those that began in the upper.  (Looked up
// where it is used: handed over as an argument, it cost every call 1 to 2% through the compiler's schedule.)
__device__ __forceinline__ unsigned* redo_word() { return reinterpret_cast<unsigned*>(smem_1024(smem_raw) + kOffMisc + 8); }
constexpr unsigned kRedoBegins = 0x10001u, kRedoEnds = 0xffffffffu;

// mbar_wait_slow with a limit that starts anew while rows are computed again, or were since the last look:
// that takes as long as the keys are many, and ends by itself.  The word lies behind `abort`.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, unsigned int* status,
                                              unsigned long long limit_ns) {
  unsigned redo = (unsigned)abort[1];
  unsigned long long t0 = globaltimer();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if ((i & 63u) == 63u && globaltimer() - t0 > limit_ns) {
      const unsigned now = (unsigned)abort[1];
      if (now == redo && (now & 0xffffu) == 0) {
        *abort = 1;
        atomicOr(status, MLA_STATUS_WAIT_TIMEOUT);
        return false;
      }
      redo = now;
      t0 = globaltimer();
    }
  }
}

struct Ctx {
  uint32_t base;
  volatile int* abort;           // and redo_word() behind it
  unsigned int* status;
  unsigned long long wait_ns;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + kOffBar + 8 * i; }
  // Without waiting (try_wait may suspend the warp).
  __device__ __forceinline__ bool ready(int i, uint32_t parity) const {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar(i)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, done != 0);
  }
  __device__ __forceinline__ bool wait(int i, uint32_t parity) const {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
    return __all_sync(0xffffffffu, wait_slow(bar(i), parity, abort, status, wait_ns));
  }
};

// What a block works on at a time.
struct Unit {
  int row0, n;                   // first row (of q) of the request's chunk, its rows
  int first, from;               // first row of the streams within the chunk, of those to be stored
  int key0, keys;                // first key row, keys of the shard
  int global;                    // global length
  int head, part;                // -1: no more units
  int begin, end0, end1;         // first tile of keys, the streams' ends
  __device__ __forceinline__ int end(int t) const { return t == 0 ? end0 : end1; }
  __device__ __forceinline__ int most() const { return max(max(end0, end1), begin); }
};
static_assert(kOffUnit + 2 * (int)sizeof(Unit) <= kOffMisc + 160, "units");

// 32 requests, one a lane: rows and keys, checked, and the row tiles before them.
struct Round {
  int row0, n, key0, keys, global;
  int tiles, before;             // its tiles, those of the requests before it (of its kind)
  bool early;                    // runs before the others, for all heads
  int base, top, from, all;      // of the round: its first request, the end of the rows so far, tiles
                                 // before it and with it
  int early_tiles;               // of all early ones

  // The round behind the one at hand.
  __device__ void next(const PrefillArgs& a, int lane) {
    base += 32;
    from = all;
    load(a, lane);
  }
  __device__ void first(const PrefillArgs& a, int lane) {
    base = top = from = 0;
    load(a, lane);
  }
  __device__ void load(const PrefillArgs& a, int lane) {
    unsigned flags = 0;
    const int b = base + lane;
    int end = 0;
    row0 = n = key0 = keys = global = 0;
    if (b < a.B) {
      row0 = __ldg(a.cu + b);
      end = __ldg(a.cu + b + 1);
      keys = __ldg(a.seq_lens + b);
      key0 = __ldg(a.starts + b);
      global = a.gseq != nullptr ? __ldg(a.gseq + b) : keys;
      if (keys < 0 || key0 < 0 || keys > a.S - key0) {
        flags |= MLA_STATUS_BAD_STEP;
        key0 = min(max(key0, 0), a.S);
        keys = min(max(keys, 0), a.S - key0);
      }
    }
    // rows in order: none before the largest value so far
    int high = row0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, high, o);
      if (lane >= o) high = max(high, v);
    }
    high = max(high, top);
    if (b < a.B) {
      if (row0 < high || end < row0 || end > a.T) flags |= MLA_STATUS_BAD_STEP;
      else n = end - row0;
    }
    top = __shfl_sync(0xffffffffu, max(high, end), 31);
    tiles = (n + 2 * kM - 1) / (2 * kM);
    // Where a request's longest unit is over a third of what an SM gets in all, it begins with the
    // first: behind other heads' units it would run on by itself (requests of 3,000, 500, 1,500 and 200
    // tokens behind 0, 8,000, 3,000 and 16,000, 32 heads: 380 us in the order of heads, 268 so).  All
    // units by length, whatever the head, would read equal requests' keys more often (4 x 2,048 behind
    // 4,096: 527 us instead of 479).
    early = false;
    if (a.B > 1 && a.B <= 32 && a.splits == 1 && gridDim.x > (unsigned)a.num_sms) {
      float load = (float)tiles * (float)(keys - min(keys, a.causal ? n / (2 * a.cp) : 0));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) load += __shfl_xor_sync(0xffffffffu, load, o);
      early = tiles > 0 && 3.f * (float)keys * (float)a.num_sms > load * (float)a.H;
    }
    const unsigned some = __ballot_sync(0xffffffffu, early);
    early_tiles = __reduce_add_sync(0xffffffffu, early ? tiles : 0);
    int incl = early ? 0 : tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    before = from + incl - tiles;
    all = from + __shfl_sync(0xffffffffu, incl, 31);
    if (some != 0) {
      int e = early ? tiles : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, e, o);
        if (lane >= o) e += v;
      }
      if (early) before = e - tiles;
    }
    if (flags) atomicOr(a.status, flags);
  }
  // The unit of row tile x, whose request may lie in another round: a block's tiles mostly grow, so
  // that it goes on from where it is.  False: there is none.
  __device__ __forceinline__ bool find(const PrefillArgs& a, int x, bool of_early, int lane, Unit& un) {
    if (x < from) first(a, lane);
    while (x >= all && base + 32 < a.B) next(a, lane);
    const int at = x - before;
    const unsigned hit = __ballot_sync(0xffffffffu, early == of_early && at >= 0 && at < tiles);
    if (hit == 0) return false;
    const int who = __ffs(hit) - 1;
    un.row0 = __shfl_sync(0xffffffffu, row0, who);
    un.n = __shfl_sync(0xffffffffu, n, who);
    // the last rows, which see the most keys, first
    un.first = 2 * kM * __shfl_sync(0xffffffffu, tiles - 1 - at, who);
    un.key0 = __shfl_sync(0xffffffffu, key0, who);
    un.keys = __shfl_sync(0xffffffffu, keys, who);
    un.global = __shfl_sync(0xffffffffu, global, who);
    return true;
  }
};

// Keys that row i of the chunk sees.
__device__ __forceinline__ int seen(const PrefillArgs& a, const Unit& u, int i) {
  if (!a.causal) return u.keys;
  if (u.global <= 0) return 0;
  const int g = u.global - (u.n - 1 - i);
  if (g <= 0) return 0;
  int l = g;
  if (a.cp > 1) {
    // cp * il < 2^31; a round's positions before this rank's segment, those of its segment
    const unsigned span = (unsigned)a.cp * (unsigned)a.il, rounds = (unsigned)g / span;
    const long long rem = (long long)((unsigned)g - rounds * span) - (long long)a.rank * a.il;
    l = (int)rounds * a.il + (int)(rem < 0 ? 0 : rem > a.il ? a.il : rem);
  }
  return min(l, u.keys);
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

// Two weights 2^(s mul + sub), added to `sum`, as two bf16.  The values are bf16, and both operands of a product
// have one type, so a weight has 8 bits there: with 16 (two bf16 words, the products twice) PV would take
// twice its time, 40% more products in all.  The rounding is unbiased, at most 2^-8 of each term; beside the output's own it
// makes the mean error sqrt(2) times what that alone would (0.0022 of the values instead of 0.0016).  The sum
// keeps 32 bits, and so does the LSE.
__device__ __forceinline__ uint32_t weights(float2 s, float2 mul, float sub, float2& sum) {
  const float2 e = fma2(s, mul, make_float2(sub, sub));
  const float2 p = make_float2(exp2_fast(e.x), exp2_fast(e.y));
  sum = fma2(p, make_float2(1.f, 1.f), sum);
  return pack(p.x, p.y);
}

// Descriptors here are lower words; the upper ones are the same for all operands of a kind.
// O (+)= P V of 64 keys: four products, P at tensor memory `p`, one election.
__device__ __forceinline__ void pv_half(uint32_t d, uint32_t p, uint32_t v, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred e, ac, on;\n .reg .b32 x, y;\n .reg .b64 k;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 ac, %5, 0;\n setp.eq.b32 on, 0, 0;\n"
      " add.u32 x, %2, 0; mov.b64 k, {x, %3}; add.u32 y, %1, 0;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, ac;\n"
      " add.u32 x, %2, 128; mov.b64 k, {x, %3}; add.u32 y, %1, 8;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " add.u32 x, %2, 256; mov.b64 k, {x, %3}; add.u32 y, %1, 16;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " add.u32 x, %2, 384; mov.b64 k, {x, %3}; add.u32 y, %1, 24;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      "}" ::"r"(d), "r"(p), "r"(v), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}
// S (+)= Q K^T of 64 dims: four products, one election.
__device__ __forceinline__ void qk_chunk(uint32_t d, uint32_t q, uint32_t k, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred e, ac, on;\n .reg .b32 x, y;\n .reg .b64 k, q;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 ac, %5, 0;\n setp.eq.b32 on, 0, 0;\n"
      " add.u32 x, %2, 0; mov.b64 k, {x, %3}; add.u32 y, %1, 0; mov.b64 q, {y, %3};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %4, ac;\n"
      " add.u32 x, %2, 2; mov.b64 k, {x, %3}; add.u32 y, %1, 2; mov.b64 q, {y, %3};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %4, on;\n"
      " add.u32 x, %2, 4; mov.b64 k, {x, %3}; add.u32 y, %1, 4; mov.b64 q, {y, %3};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %4, on;\n"
      " add.u32 x, %2, 6; mov.b64 k, {x, %3}; add.u32 y, %1, 6; mov.b64 q, {y, %3};\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %4, on;\n"
      "}" ::"r"(d), "r"(q), "r"(k), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}

// The rest of a turn whose keys are all here: the second half of O += P V, the release of V, S = Q K^T
// (three chunks of 64 dims, Q's 16 KB apart), the other stream's turn, S's barrier, under one election
// (apart from one another, with a wait between, 200 clocks more).
__device__ __forceinline__ void pv_qk_turn(uint32_t d_o, uint32_t p, uint32_t v, uint32_t vhi, uint32_t id_pv,
                                           uint32_t b_v, uint32_t d, uint32_t q, uint32_t k0, uint32_t k1, uint32_t k2,
                                           uint32_t hi, uint32_t idesc, uint32_t b_turn, uint32_t b_s) {
  asm volatile(
      "{\n .reg .pred e, on;\n .reg .b32 x, y;\n .reg .b64 k, q;\n elect.sync _|e, 0xffffffff;\n"
      " setp.eq.b32 on, 0, 0;\n"
      " add.u32 x, %2, 0; mov.b64 k, {x, %3}; add.u32 y, %1, 0;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " add.u32 x, %2, 128; mov.b64 k, {x, %3}; add.u32 y, %1, 8;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " add.u32 x, %2, 256; mov.b64 k, {x, %3}; add.u32 y, %1, 16;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " add.u32 x, %2, 384; mov.b64 k, {x, %3}; add.u32 y, %1, 24;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], k, %4, on;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
      " add.u32 x, %8, 0; mov.b64 k, {x, %11}; add.u32 y, %7, 0; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, !on;\n"
      " add.u32 x, %8, 2; mov.b64 k, {x, %11}; add.u32 y, %7, 2; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %8, 4; mov.b64 k, {x, %11}; add.u32 y, %7, 4; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %8, 6; mov.b64 k, {x, %11}; add.u32 y, %7, 6; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %9, 0; mov.b64 k, {x, %11}; add.u32 y, %7, 1024; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %9, 2; mov.b64 k, {x, %11}; add.u32 y, %7, 1026; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %9, 4; mov.b64 k, {x, %11}; add.u32 y, %7, 1028; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %9, 6; mov.b64 k, {x, %11}; add.u32 y, %7, 1030; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %10, 0; mov.b64 k, {x, %11}; add.u32 y, %7, 2048; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %10, 2; mov.b64 k, {x, %11}; add.u32 y, %7, 2050; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %10, 4; mov.b64 k, {x, %11}; add.u32 y, %7, 2052; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " add.u32 x, %10, 6; mov.b64 k, {x, %11}; add.u32 y, %7, 2054; mov.b64 q, {y, %11};\n @e tcgen05.mma.cta_group::1.kind::f16 [%6], q, k, %12, on;\n"
      " @e mbarrier.arrive.shared::cta.b64 _, [%13];\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%14];\n}" ::"r"(d_o),
      "r"(p), "r"(v), "r"(vhi), "r"(id_pv), "r"(b_v), "r"(d), "r"(q), "r"(k0), "r"(k1), "r"(k2), "r"(hi), "r"(idesc),
      "r"(b_turn), "r"(b_s)
      : "memory");
}

// Asks for a block of the grid that has not begun: its index, or that there is none, comes into 16
// bytes of shared memory.
__device__ __forceinline__ void ask_next(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool read_next(uint32_t src, uint32_t& x, uint32_t& y) {
  uint32_t some;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n .reg .b32 z, w;\n"
      " ld.shared.b128 h, [%3];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
      " selp.u32 %0, 1, 0, p;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, z, w}, h;\n}"
      : "=r"(some), "=r"(x), "=r"(y)
      : "r"(src)
      : "memory");
  // the read is done before the next answer is written there
  fence_proxy_async_smem();
  return some != 0;
}

// One warp: O's 32 rows at tensor memory `to` times `inv` (0: nothing was seen, zeros), as fp32 or
// bf16, to `dst` and on, a token's H heads apart; the first `rows` are stored.  Arrives on `free` once
// O is read.  True: the thread's row holds a NaN or an infinity.  Out of line: inlined, its registers
// spill the tile loop's.
template <bool kFp32>
__device__ __noinline__ bool write_rows(uint32_t to, bool any, float inv, uint8_t* dst, int H, int rows, int lane,
                                        uint32_t free) {
  constexpr int kPasses = kFp32 ? 4 : 2;          // 128 bytes of each row at a time
  const long long step = (long long)H * (128 * kPasses);
  dst += (lane & 24) * step + (lane & 7) * 16;
  const bool none = inv == 0.f || !any;
  float2 zero = make_float2(0.f, 0.f);            // 0 x each value
#pragma unroll 1
  for (int c = 0; c < kPasses; ++c) {
    uint32_t v[32];
    if (kFp32) {
      tmem_ld32(to + 32 * c, v);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; i += 2) zero = fma2(make_float2(0.f, 0.f), make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), zero);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = none ? 0u : __float_as_uint(__uint_as_float(v[i]) * inv);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[32];
        tmem_ld32(to + 64 * c + 32 * h, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) zero = fma2(make_float2(0.f, 0.f), make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), zero);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[16 * h + i] = none ? 0u : pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
      }
    }
    if (c == kPasses - 1 && any) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(free);
    }
    transpose8(v, lane);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if ((lane & 24) + r < rows)
        *reinterpret_cast<uint4*>(dst + r * step + c * 128) = make_uint4(v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]);
  }
  return !none && zero.x + zero.y != 0.f;
}

// A key that some rows of a tile do not see has the weight 0 there, and 0 times a value that is NaN or
// infinite is NaN.  One warp: its rows `bad` (with such outputs) once more, over their own keys alone,
// where a value of a key that not every row sees is the reason; else they stay.  Scores: lane = key, the
// row's query is read by all lanes; values: lane = 4 dims.  Slow, by the loads' latency (256 rows, 8,448
// keys, 16 heads: 28 ms instead of 0.14): where all values are finite it costs only the test, 64
// multiply-adds a row.  Running the unit again on the tensor cores with such values cleared, in a second
// copy of the block's code, took 0.3 ms here but 3 to 6% of every other call's time.
// m, inv: the row's reference and 1 / (sum of weights).
template <bool kFp32>
__device__ __noinline__ void redo_rows(const PrefillArgs& a, const Unit& u, int begin, int end, int least, int mine,
                                       float m, float inv, unsigned bad, int row0, uint8_t* dst, int lane) {
  unsigned* const redo = redo_word();
  if (lane == 0) atomicAdd(redo, kRedoBegins);
  const PrefillTensors& x = a.x;
  const uint16_t* v = static_cast<const uint16_t*>(x.v) + (long long)u.key0 * x.v_s + u.head * x.v_h + 4 * lane;
  const uint16_t* k = static_cast<const uint16_t*>(x.k_nope) + (long long)u.key0 * x.k_s + u.head * x.k_h;
  const uint16_t* kr = static_cast<const uint16_t*>(x.k_rope) + (long long)u.key0 * x.r_s;
  bool found = false;
#pragma unroll 4
  for (int l = max(least, begin); l < end; ++l) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(v + l * x.v_s));
    found = found || (((w.x & 0x7fff7fffu) + 0x00800080u) | ((w.y & 0x7fff7fffu) + 0x00800080u)) & 0x80008000u;
  }
  if (!__any_sync(0xffffffffu, found)) bad = 0;
  for (; bad != 0; bad &= bad - 1) {
    const int r = __ffs(bad) - 1;
    const int keys = min(__shfl_sync(0xffffffffu, mine, r), end);
    const float ref = __shfl_sync(0xffffffffu, m, r), f = __shfl_sync(0xffffffffu, inv, r);
    const uint16_t* q = static_cast<const uint16_t*>(x.q) + (long long)(row0 + r) * x.q_t + u.head * x.q_h;
    float o[2][4] = {};
    for (int l0 = begin; l0 < keys; l0 += 32) {
      float p = 0.f;
      if (l0 + lane < keys) {
        // eight sums of 24 products
        const uint16_t* kn = k + (l0 + lane) * x.k_s;
        const uint16_t* rope = kr + (l0 + lane) * x.r_s;
        float2 t[4] = {};
#pragma unroll 12
        for (int c = 0; c < 24; ++c) {
          const uint4 qa = __ldg(reinterpret_cast<const uint4*>(q + 8 * c));
          const uint4 ka = __ldg(reinterpret_cast<const uint4*>(c < 16 ? kn + 8 * c : rope + 8 * (c - 16)));
          const uint32_t qw[4] = {qa.x, qa.y, qa.z, qa.w}, kw[4] = {ka.x, ka.y, ka.z, ka.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            t[i] = fma2(make_float2(__uint_as_float(qw[i] << 16), __uint_as_float(qw[i] & 0xffff0000u)),
                        make_float2(__uint_as_float(kw[i] << 16), __uint_as_float(kw[i] & 0xffff0000u)), t[i]);
        }
        const float s = ((t[0].x + t[0].y) + (t[1].x + t[1].y)) + ((t[2].x + t[2].y) + (t[3].x + t[3].y));
        // rounded as where it meets the values on the tensor cores
        p = __bfloat162float(__float2bfloat16_rn(exp2_fast(fmaf(s, a.scale_log2, -ref))));
      }
      // sixteen keys' values in flight
#pragma unroll 1
      for (int i0 = 0; i0 < min(32, keys - l0); i0 += 16) {
        uint2 b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          b[i] = l0 + i0 + i < keys ? __ldg(reinterpret_cast<const uint2*>(v + (l0 + i0 + i) * x.v_s)) : make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float w = __shfl_sync(0xffffffffu, p, i0 + i);
          o[i & 1][0] = fmaf(w, __uint_as_float(b[i].x << 16), o[i & 1][0]);
          o[i & 1][1] = fmaf(w, __uint_as_float(b[i].x & 0xffff0000u), o[i & 1][1]);
          o[i & 1][2] = fmaf(w, __uint_as_float(b[i].y << 16), o[i & 1][2]);
          o[i & 1][3] = fmaf(w, __uint_as_float(b[i].y & 0xffff0000u), o[i & 1][3]);
        }
      }
    }
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (o[0][i] + o[1][i]) * f;
    uint8_t* const to = dst + (long long)r * a.H * (kFp32 ? 512 : 256);
    if (kFp32)
      *reinterpret_cast<float4*>(to + 16 * lane) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(to + 8 * lane) = make_uint2(pack(y[0], y[1]), pack(y[2], y[3]));
  }
  if (lane == 0) atomicAdd(redo, kRedoEnds);
}

__global__ void __launch_bounds__(kThreads, 1)
mla_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ PrefillArgs a) {
  uint8_t* sp = smem_1024(smem_raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sp + kOffMisc);
  Unit* su = reinterpret_cast<Unit*>(sp + kOffUnit);
  Ctx s;
  s.base = smem_u32(sp);
  s.abort = reinterpret_cast<volatile int*>(misc + 1);
  s.status = a.status;
  s.wait_ns = a.wait_ns;

  Round requests;                // warp 3's
  if (warp == 1) {
    tmem_alloc(s.base + kOffMisc, 512);
    tmem_relinquish();
  } else if (warp == 3) {
    grid_wait();
    requests.first(a, lane);
  } else if (tid < 4) {
    prefetch_tensormap(tid == 0 ? &qmap : tid == 1 ? &kmap : tid == 2 ? &rmap : &vmap);
  } else if (tid == 64) {
    s.abort[0] = s.abort[1] = 0;
    for (int i = 0; i < B_COUNT; ++i) {
      const bool of_warps = (i >= B_PFULL && i < B_PFULL + 4) || i == B_OFREE || i == B_OFREE + 1;
      mbar_init(s.bar(i), of_warps ? 4 : i >= B_KEMPTY ? 2 : i == B_UEMPTY ? kReaders : 1);
    }
    fence_mbar_init();
  }
  grid_wait();
  grid_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);

  // Every role goes through the same units: next() waits for the k-th one.  False: there is none, or
  // a wait has run out.
  // A unit stays where it is until the role has asked for the one after it.
  const auto next = [&](uint32_t& k, const Unit*& u) {
    if (!s.wait(B_UFULL, k & 1)) return false;
    u = su + (k & 1);
    __syncwarp();
    if (lane == 0) mbar_arrive(s.bar(B_UEMPTY));
    ++k;
    return u->head >= 0;
  };

  if (warp == 3) {
    // ---- units: this block's own, then those of blocks that have not begun ---------------------
    uint32_t x = blockIdx.x, y = blockIdx.y, asked = 0, k = 0;
    bool some = true, ok = true;
    while (ok) {
      Unit u;
      u.head = -1;
      if (some) {
        // early requests' blocks; then one group of heads after another, in a group all heads' longest
        // tiles first
        const unsigned es = (unsigned)requests.early_tiles * (unsigned)a.H;
        const bool of_early = x < es;
        const unsigned per = ((unsigned)a.tiles - (unsigned)requests.early_tiles) * (unsigned)a.group;
        const unsigned grp = of_early ? 0 : (x - es) / max(per, 1u), in = of_early ? x : x - es - grp * per;
        const unsigned heads = of_early ? (unsigned)a.H : min((unsigned)a.group, (unsigned)a.H - grp * a.group);
        if (requests.find(a, (int)(in / heads), of_early, lane, u)) {
          u.head = (int)(grp * a.group + in % heads);
          u.part = (int)y;
          u.from = u.first;
          u.begin = 0;
          // the bound grows with the row, so a stream's last row has the most tiles
          u.end0 = (seen(a, u, min(u.first + kM, u.n) - 1) + kTile - 1) / kTile;
          u.end1 = u.first + kM < u.n ? (seen(a, u, min(u.first + 2 * kM, u.n) - 1) + kTile - 1) / kTile : 0;
          if (a.splits > 1) {
            const int most = u.most();
            u.begin = (int)((long long)most * y / a.splits);
            const int end = (int)((long long)most * (y + 1) / a.splits);
            u.end0 = max(min(u.end0, end), u.begin);
            u.end1 = max(min(u.end1, end), u.begin);
          }
          if (u.n - u.first <= kM && (k & 1) != 0) {
            // rows of one stream alone: units take the streams in turn, so that one's output is written
            // while the other works
            u.end1 = u.end0;
            u.end0 = u.begin;
            u.first -= kM;
          }
        }
      }
      if (u.head >= 0 || !some) {
        ok = s.wait(B_UEMPTY, (k & 1) ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          su[k & 1] = u;
          mbar_arrive(s.bar(B_UFULL));
        }
        __syncwarp();
        ++k;
        if (!some) break;
        // requests behind the last row tile's, which nobody looks for, are checked here
        if (x + 1 == gridDim.x && y == 0)
          while (requests.base + 32 < a.B) requests.next(a, lane);
        // the next one only when this one is nearly loaded: what is asked for early runs late
        ok = s.wait(B_ASK, (k & 1) ^ 1u);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(s.bar(B_NEXT), 16);
        ask_next(s.base + kOffNext, s.bar(B_NEXT));
      }
      __syncwarp();
      ok = s.wait(B_NEXT, asked & 1);
      ++asked;
      some = ok && read_next(s.base + kOffNext, x, y);
    }
    if (!ok && asked > 0) mbar_wait_drain(s.bar(B_NEXT), (asked - 1) & 1);
  } else if (warp == 0) {
    // ---- loads ------------------------------------------------------------------------------
    const Unit* unit;
    uint32_t k = 0, nq[2] = {0, 0};
    int sl = 0;
    uint32_t g = 0;                             // tiles so far
    bool ok = true;
    const auto slot = [&]() {
      const uint32_t dst = s.base + kOffRing + sl * kSlotBytes;
      sl = (sl + 1) % kSlots;
      return dst;
    };
    while (ok && next(k, unit)) {
      const Unit u = *unit;
      const int most = u.most();
      if (most == u.begin && lane == 0) mbar_arrive(s.bar(B_ASK));
      // its queries into the L2: their place is free only when the unit before has no more products
      for (int t = 0; t < 2; ++t)
        if (u.end(t) > u.begin)
          for (int c = 0; c < kQChunks; ++c)
            tma_prefetch_3d_warp(&qmap, 64 * c, u.head, u.row0 + u.first + t * kM);
      for (int j = u.begin; j < most && ok; ++j, ++g) {
        if (j == max(u.begin, most - 2) && lane == 0) mbar_arrive(s.bar(B_ASK));
        const int y = u.key0 + j * kTile;
        const uint32_t e = g & 1, use = g >> 1 & 1;           // even or odd tile; parity of its phase
        ok = s.wait(B_KEMPTY + e, use ^ 1u);
        if (!ok) break;
        mbar_arrive_expect_tx_warp(s.bar(B_KFULL + e), kSlotBytes);
        tma_load_3d_warp(slot(), &kmap, 0, u.head, y, s.bar(B_KFULL + e));
        ok = s.wait(B_VEMPTY + e, use ^ 1u);
        if (!ok) {
          ++g;
          break;
        }
        mbar_arrive_expect_tx_warp(s.bar(B_KFULL + 2 + e), kSlotBytes);
        tma_load_3d_warp(slot(), &kmap, 64, u.head, y, s.bar(B_KFULL + 2 + e));
        mbar_arrive_expect_tx_warp(s.bar(B_KFULL + 4 + e), kSlotBytes);
        tma_load_2d_warp(slot(), &rmap, 0, y, s.bar(B_KFULL + 4 + e));
        if (j == u.begin) {
          // the unit's queries, after its first keys
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (u.end(t) > u.begin) {
              ok = ok && s.wait(B_QEMPTY + t, (nq[t] & 1) ^ 1u);
              if (!ok) break;
              mbar_arrive_expect_tx_warp(s.bar(B_QFULL + t), kQChunks * kSlotBytes);
              for (int c = 0; c < kQChunks; ++c)
                tma_load_3d_warp(s.base + kOffQ + (t * kQChunks + c) * kSlotBytes, &qmap, 64 * c, u.head,
                                 u.row0 + u.first + t * kM, s.bar(B_QFULL + t));
              ++nq[t];
            }
        }
        if (ok && g > 0) ok = s.wait(B_KEMPTY + (e ^ 1), (g - 1) >> 1 & 1);
        if (!ok) {
          ++g;
          break;
        }
        mbar_arrive_expect_tx_warp(s.bar(B_VFULL + e), kVSlots * kSlotBytes);
#pragma unroll
        for (int c = 0; c < kVSlots; ++c) {
          const uint32_t dst = slot();
          tma_load_3d_warp(dst, &vmap, 0, u.head, y + 64 * c, s.bar(B_VFULL + e));
          tma_load_3d_warp(dst + kSlotBytes / 2, &vmap, 64, u.head, y + 64 * c, s.bar(B_VFULL + e));
        }
      }
    }
    if (*s.abort) {
      // let loads in flight land before the block ends (those that were not issued are not waited for
      // longer than a drain's limit)
      for (uint32_t m = g > 2 ? g - 2 : 0; m < g; ++m) {
        for (int c = 0; c < kKSlots; ++c) mbar_wait_drain(s.bar(B_KFULL + 2 * c + (int)(m & 1)), m >> 1 & 1);
        mbar_wait_drain(s.bar(B_VFULL + (int)(m & 1)), m >> 1 & 1);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (nq[t] > 0) mbar_wait_drain(s.bar(B_QFULL + t), (nq[t] - 1) & 1);
    }
  } else if (warp <= 2) {
    // ---- products of a stream, the streams in turn ----------------------------------------------
    const int t = warp - 1;
    const uint32_t id_qk = idesc_bf16(kM, kTile, false, false), id_pv = idesc_bf16(kM, 128, false, true);
    const uint64_t qd = smem_desc(s.base + kOffQ + t * kQChunks * kSlotBytes, 16, 1024, kSwizzle128B);
    const uint32_t kd = (uint32_t)smem_desc(s.base + kOffRing, 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(s.base + kOffRing, kSlotBytes / 2, 1024, kSwizzle128B);
    constexpr unsigned kStep = kSlotBytes / 16;
    const uint32_t ds = tmem + t * 128, d_o = ds + 256, hi = (uint32_t)(qd >> 32), vhi = (uint32_t)(vd >> 32);
    const Unit* unit;
    uint32_t k = 0;
    unsigned sl = 0;                            // slot of tile j's keys
    uint32_t g = 0;                             // tiles before it
    uint32_t units = 0, pv_tiles = 0;           // units and tiles of this stream so far
    uint32_t turn = 0;
    bool ok = true;
    while (ok && next(k, unit)) {
      const Unit u = *unit;
      const int most = u.most(), mine = u.end(t);
      if (u.begin < mine) ok = s.wait(B_QFULL + t, units & 1);
      for (int j = u.begin; j <= most && ok; ++j) {
        // barriers and phases of tile j's keys and of tile j - 1's values, whose slots are the two before
        const int e = (int)(g & 1), ev = e ^ 1;
        const uint32_t use = g >> 1 & 1, vuse = (g - 1) >> 1 & 1;
        const unsigned v0 = (sl + kSlots - 2) % kSlots, v1 = (sl + kSlots - 1) % kSlots;
        const bool pv = j > u.begin && j <= mine, qk = j < mine, first = j - 1 == u.begin;
        if (pv) {
          ok = s.wait(B_VFULL + ev, vuse);
          const int left = u.keys - (j - 1) * kTile;
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
          if (first) ok = ok && s.wait(B_OFREE + t, (units & 1) ^ 1u);
          ok = ok && s.wait(B_PFULL + 2 * t, pv_tiles & 1);
        }
        const bool keys = qk && s.ready(B_KFULL + e, use) && s.ready(B_KFULL + 2 + e, use) && s.ready(B_KFULL + 4 + e, use);
        // the other stream's products are issued
        if (t == 1 || turn > 0) ok = ok && s.wait(B_TURN + t, t == 1 ? turn & 1 : (turn & 1) ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t k0 = kd + sl * kStep, k1 = kd + (sl + 1) % kSlots * kStep, k2 = kd + (sl + 2) % kSlots * kStep;
        if (pv) {
          pv_half(d_o, ds, (uint32_t)vd + v0 * kStep, vhi, id_pv, !first);
          ok = s.wait(B_PFULL + 2 * t + 1, pv_tiles & 1);
          if (!ok) break;
          tc_fence_after();
          ++pv_tiles;
        }
        if (pv && keys) {
          pv_qk_turn(d_o, ds + 32, (uint32_t)vd + v1 * kStep, vhi, id_pv, s.bar(B_VEMPTY + ev), ds, (uint32_t)qd, k0, k1,
                     k2, hi, id_qk, s.bar(B_TURN + (t ^ 1)), s.bar(B_SFULL + t));
        } else {
          if (pv) pv_half(d_o, ds + 32, (uint32_t)vd + v1 * kStep, vhi, id_pv, 1);
          if (j > u.begin) mma_commit_warp(s.bar(B_VEMPTY + ev));
          if (qk) {
            // a chunk at a time, as they come
            ok = s.wait(B_KFULL + e, use);
            if (!ok) break;
            tc_fence_after();
            qk_chunk(ds, (uint32_t)qd, k0, hi, id_qk, 0);
            ok = s.wait(B_KFULL + 2 + e, use);
            if (!ok) break;
            tc_fence_after();
            qk_chunk(ds, (uint32_t)qd + kStep, k1, hi, id_qk, 1);
            ok = s.wait(B_KFULL + 4 + e, use);
            if (!ok) break;
            tc_fence_after();
            qk_chunk(ds, (uint32_t)qd + 2 * kStep, k2, hi, id_qk, 1);
            if (lane == 0) mbar_arrive(s.bar(B_TURN + (t ^ 1)));
            __syncwarp();
            mma_commit_warp(s.bar(B_SFULL + t));
          } else {
            if (lane == 0) mbar_arrive(s.bar(B_TURN + (t ^ 1)));
            __syncwarp();
          }
        }
        ++turn;
        if (pv && j == mine) mma_commit_warp(s.bar(B_OFULL + t));
        if (qk && j + 1 == mine) mma_commit_warp(s.bar(B_QEMPTY + t));
        if (j == most) break;
        mma_commit_warp(s.bar(B_KEMPTY + e));
        sl = (sl + kKSlots + kVSlots) % kSlots;
        ++g;
      }
      if (u.begin < mine) ++units;
    }
    mma_commit_warp(s.bar(B_DRAIN + t));
    mbar_wait_drain(s.bar(B_DRAIN + t), 0);
  } else {
    // ---- softmax and output: thread = row ---------------------------------------------------------
    const int t = (warp >> 2) - 1, q = warp & 3;
    const uint32_t ts = tmem + ((uint32_t)q << 21) + t * 128, to = ts + 256;
    const Unit* u;
    uint32_t k = 0, s_tiles = 0, units = 0;
    bool ok = true;
    while (ok && next(k, u)) {
      // keys that the row sees (rows behind the chunk are not stored), the fewest of the warp
      const int mine = seen(a, *u, min(u->first + t * kM + q * 32 + lane, u->n - 1));
      const int least = __shfl_sync(0xffffffffu, mine, 0);
      float m = -INFINITY, l = 0.f;
      const int begin = u->begin, n_tiles = u->end(t);
      for (int j = begin; j < n_tiles; ++j, ++s_tiles) {
        ok = s.wait(B_SFULL + t, s_tiles & 1);
        if (!ok) break;
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
        tmem_wait_ld();
        if (least < (j + 1) * kTile) {
          const int lim = mine - j * kTile, all = least - j * kTile;    // the row's and the warp's bound
#pragma unroll
          for (int b = 0; b < 128; b += 32) {
            if (all >= b + 32) continue;
#pragma unroll
            for (int c = b; c < b + 32; ++c) x[c] = c < lim ? x[c] : -INFINITY;
          }
        }
        // P of the first 64 keys by the reference so far, beside the maximum: it seldom moves.  The first
        // one is that of four keys
        const float2 mul = make_float2(a.scale_log2, a.scale_log2);
        if (j == begin) m = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * a.scale_log2;
        float ref = m == -INFINITY ? 0.f : m;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[32];
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[c + 2 * i], x[c + 2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[124 + i]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = weights(make_float2(x[2 * i], x[2 * i + 1]), mul, -ref, sum[i & 1]);
        // the reference moves where a maximum rose too far
        const bool moves = top > m + kRise;
        if (__any_sync(0xffffffffu, moves)) {
          const float f = moves ? exp2_fast(m - top) : 1.f;
          if (moves) m = top;
          l *= f;
          if (j > begin)
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16(to + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(to + 16 * c, o);
            }
          // and P again, from S
          ref = m == -INFINITY ? 0.f : m;
          sum[0] = sum[1] = make_float2(0.f, 0.f);
          const int lim = mine - j * kTile;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t y[32];
            tmem_ld32(ts + 32 * c, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int d = 32 * c + 2 * i;
              pk[16 * c + i] = weights(make_float2(d < lim ? __uint_as_float(y[2 * i]) : -INFINITY,
                                                   d + 1 < lim ? __uint_as_float(y[2 * i + 1]) : -INFINITY),
                                       mul, -ref, sum[i & 1]);
            }
          }
        }
        // the first half's product starts while P of the other is computed
        tmem_st32(ts, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s.bar(B_PFULL + 2 * t));
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = weights(make_float2(x[64 + 2 * i], x[65 + 2 * i]), mul, -ref, sum[i & 1]);
        tmem_st32(ts + 32, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s.bar(B_PFULL + 2 * t + 1));
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      const bool any = n_tiles > begin;
      if (any) {
        ok = s.wait(B_OFULL + t, units & 1);
        if (!ok) break;
        tc_fence_after();
        ++units;
      }
      // O / l: bf16, or fp32 where the keys are split
      const int i0 = u->first + t * kM + q * 32;             // the warp's first row in the chunk
      const int rows = i0 < u->from ? 0 : u->n - i0;         // the warp's rows that are stored
      const long long row0 = (long long)(u->row0 + i0) * a.H + u->head, row = row0 + (long long)lane * a.H;
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const bool split = a.splits > 1;
      const long long part = (long long)u->part * a.T * a.H;
      if (lane < rows) {
        if (split) a.ws_lse[part + row] = none ? -INFINITY : m + log2f(l);
        else if (a.lse != nullptr) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * a.lse_mul;
      }
      uint8_t* const dst = split ? reinterpret_cast<uint8_t*>(a.ws_o + (part + row0) * 128)
                                 : reinterpret_cast<uint8_t*>(a.out + row0 * 128);
      if (rows <= 0) {
        if (any && lane == 0) mbar_arrive(s.bar(B_OFREE + t));
        continue;
      }
      const bool odd = split ? write_rows<true>(to, any, inv, dst, a.H, rows, lane, s.bar(B_OFREE + t))
                             : write_rows<false>(to, any, inv, dst, a.H, rows, lane, s.bar(B_OFREE + t));
      const unsigned bad = __ballot_sync(0xffffffffu, odd && lane < rows);
      const int end = min(n_tiles * kTile, u->keys);
      if (bad != 0 && least < end) {
        if (split) redo_rows<true>(a, *u, begin * kTile, end, least, mine, m, inv, bad, u->row0 + i0, dst, lane);
        else redo_rows<false>(a, *u, begin * kTile, end, least, mine, m, inv, bad, u->row0 + i0, dst, lane);
      }
    }
  }
  __syncwarp();
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

// Row tiles at most: sum ceil(n_b / 256) <= sum (n_b + 255) / 256, requests without rows left out.
long long row_tiles(int T, int B) { return (T + (2LL * kM - 1) * (B < T ? B : T)) / (2 * kM); }

// Parts that each request's keys are cut into: as many as fill the SMs, each of 256 keys or more
// if a request had all key rows.
int parts(int T, int B, int H, int S, int num_sms) {
  const long long blocks = row_tiles(T, B) * H;
  long long n = num_sms / (blocks > 0 ? blocks : 1);
  if (n > S / 256) n = S / 256;
  return n < 1 ? 1 : (int)n;
}

// Heads whose units run at a time, longest first: enough for four units an SM, so that the last ones
// to run are short (two shards' prompts of 64 heads: 169 us; for one an SM 181, two 172, 16 169), unless
// their keys and values would not stay in half of the L2; in equal groups.
int head_group(int tiles, int S, int H, int num_sms) {
  long long n = (4LL * num_sms + tiles - 1) / tiles;
  const long long fit = (64LL << 20) / ((long long)(S > 0 ? S : 1) * 512);
  n = n < fit ? n : fit;
  const long long groups = n < 1 ? H : n < H ? H / n : 1;
  return (int)((H + groups - 1) / groups);
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
  a.x = x;
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
  // (without key rows the maps of the keys stand on q; nothing is loaded through them)
  const bool keys = a.S > 0;
  const uint64_t H = (uint64_t)a.H, T = (uint64_t)a.T, S = keys ? (uint64_t)a.S : 1;
  const uint64_t qd[3] = {192, H, T}, kd[3] = {128, H, S}, rd[2] = {64, S};
  // strides in bytes; that of a dimension of one is any
  const auto by = [](uint64_t n, int64_t stride) { return n > 1 ? (uint64_t)stride * 2 : (uint64_t)16; };
  const uint64_t qs[2] = {by(H, x.q_h), by(T, x.q_t)}, ks[2] = {by(H, x.k_h), by(S, x.k_s)},
                 vs[2] = {by(H, x.v_h), by(S, x.v_s)}, rs[1] = {by(S, x.r_s)};
  const uint32_t box[3] = {64, 1, 128}, vbox[3] = {64, 1, 64}, rbox[2] = {64, 128};
  if (!encode_tile_map(&qmap, x.q, 3, qd, qs, box) || !encode_tile_map(&kmap, keys ? x.k_nope : x.q, 3, kd, ks, box) ||
      !encode_tile_map(&rmap, keys ? x.k_rope : x.q, 2, rd, rs, rbox) ||
      !encode_tile_map(&vmap, keys ? x.v : x.q, 3, kd, vs, vbox))
    return cudaErrorInvalidValue;
  a.tiles = (int)row_tiles(a.T, a.B);
  a.group = head_group(a.tiles, a.S, a.H, a.num_sms);
  const dim3 grid((unsigned)a.tiles * (unsigned)a.H, (unsigned)a.splits);
  DependentLaunch dl(grid, dim3(kThreads), stream, kSmemBytes);
  e = cudaLaunchKernelEx(&dl.cfg, mla_prefill_kernel, qmap, kmap, rmap, vmap, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  return launch_lse_combine128(a.ws_o, true, a.ws_lse, a.splits, (long long)a.T * a.H, true, a.lse_mul, a.out,
                               a.lse, a.cu, a.B, a.H, stream);
}

}  // namespace mla
