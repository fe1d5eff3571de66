// Paged MLA decode over the 8-bit cache on the Blackwell tensor cores (tcgen05 + TMEM + TMA).
//
// What it computes: mla_decode's shard-local attention (row bounds and LSE as there: "vLLM PR
// #52188 (DSpark + DCP)" page, section "关键源码片段"; "vLLM PR #54012" page, section
// "实现拆解" step 3) with key l = S_l k8_l, k8 the row's 576 e4m3 values and S_l the scale of
// its group of 16 slots:
//   t_l = scale S_l <q, k8_l>,  out = sum_l 2^(t'_l - m) S_l v8_l / sum_l 2^(t'_l - m)  (t' in log2).
//
// Two forms of the products.  A unit is kN query rows of one request, 64 or 32 (rows_per_unit).
// The tile of 128 keys lies in shared memory once, as TMA brings it (128-byte rows of 128 dims,
// 128-byte swizzle); QK reads it K-major, PV reads the same bytes M-major (the transpose bit of
// the instruction).  PV is O^T [512 dims x rows] += V8^T [512 x 128] P^T in both: the time goes
// with the number of rows, where rows as M would always pay for 128, and O^T of 64 rows takes
// 256 of the 512 tensor-memory columns, so that a unit needs no second SM.
//   64 rows: S [hi and lo of 64 rows x 128 keys] = Q K8^T.  Q's latent dims are the tensor-memory
//     operand, 128 columns beside O^T and one S (QK then reads keys and nothing else: 80 KB of
//     shared memory a tile where Q in shared memory took 144), its rope dims are in shared memory.
//   32 rows: S^T [128 keys x hi and lo of 32 rows] = K8 Q^T, Q in shared memory, two S^T: such
//     units are bound by HBM or by their start, and rows as M = 128 would double QK's time.
//
// 8-bit operands in two parts.  Both factors of a product must be 8-bit types, and
// a query or a weight rounded to one e4m3 value would be off by up to 2^-4.  So:
//   * q, times a power of two that puts its row's maximum in [128, 256), is the sum of two
//     e4m3 values hi + lo: a bf16 has 8 significant bits, each e4m3 holds 4, and hi's residue
//     is at most 8 units of q's last place; exact for elements within 2^-9 of the maximum,
//     off by at most 2^-10 (2^-17 of the maximum) below.  hi and lo are columns of one
//     product with N = 2 kN (the keys are read once), added when S is read.
//   * a weight p = S_l 2^(t'_l - m) is an e5m2 value (3 bits, range to 2^-16) plus its residue,
//     two products into the same accumulator.  The residue is an e4m3 value: p is off by at
//     most 2^-8 p, or 2^-10 below 2^-2.  Where some row's largest p of 16 keys is below 2^-3 (and
//     not below 2^-22), the residues of a tile are e5m2 values for all the unit's rows: off by
//     at most 2^-7 p, or 2^-17 below 2^-10.  Both have a dither of up to half the type's smallest
//     step, spread evenly over the keys, so that the sum of many small weights comes out right:
//     thousands of equal ones far below one large one may be most of the output (with e4m3 alone
//     and without dithers, 16,384 of e^-8 of the largest lost 5 % of the output, of e^-15 40 %).
// An e4m3 residue (at most 448) serves p up to 2^12.  m is set 2^6 below a tile's largest S_l 2^t'_l
// and moved (then O, l and m move together) only when a tile exceeds 2^12.  Nearer to 2^12 small
// weights would have more of the range, but a move costs half a tile's time (2^10 / 2^8 / 2^6 / 2^5
// below: 64 x 128 rows of 32k keys 404 / 383 / 376 / 373 us, 8 x 256 of 512..4k 27.2 / 25.5 / 24.6 /
// 24.3); at 2^12 where a segment has but one tile.  Where a tile's largest stands alone (as first
// tokens do, with nearly all the weight and little value), the rest counts: that is set to 2^3 or
// more, as far as 2^12 for the largest allows.  All this takes 2 to 8 % of the time (e4m3 residues
// alone, without dithers, set 2^5 below: 368 us, with outliers 565).
//
// Roles (20 warps, 12 for 32 rows): warp 0 loads tiles (TMA, four 16 KB chunks of latent dims
// and one of rope dims each, chunk by chunk as PV frees them), warp 1 issues the QK products and
// warp 2 the PV products, each when its inputs have come (one warp for both in a fixed order
// waits for the later of two inputs: 8 % of 64 x 32k; one that polls both takes issue slots from the
// softmax warps of its scheduler), warp 3 walks the schedule, passes the block's
// segments on and looks the tiles' scales up, the others take 32 keys and 16 rows each: they
// read S, scale, mask, exponentiate and write P^T; they also prepare Q and write the output.
//
// Bounds: few rows by the cache's bytes (64 x 16 rows of 1k..16k keys: 67 us, 47.7 at the copy
// rate); 64 rows by shared-memory bandwidth: a tile's QK reads 16 x 4 + 2 x (4 + 4) KB and its
// PV 32 x (4 + 2) KB, TMA writes 72 KB and the softmax 16 KB, 2,880 cycles at 128 bytes a cycle of
// the 3,150 that it takes, against 2,176 of tensor time.  64 x 128 rows of 32,768 keys: 376 us
// (430 call after call, at the power limit), 1.55 PFLOP/s, twice that as issued; 4 x 256 rows of
// 256k..512k with outliers: 608 us (616); 32 x 512 rows of 1k..16k: 214 us (227).
//
// Work split, partials and the combine: as in mla_decode_tc.cu (tiles of all requests on one
// line, equal ranges, units cut between blocks merged by a second kernel); a block has at most
// two partials, the unit it continues and the unit it does not finish.
//
// Safety: every wait is bounded; one that runs out sets the block's abort word, every later
// wait then returns at once, the softmax warps go through their remaining tiles without
// waiting (their barriers stay balanced), the other roles leave, copies in flight and
// issued products are waited for (bounded), and the block frees its tensor memory.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <functional>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "internal.h"
#include "sm100.cuh"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kD = 576;
constexpr int kDv = 512;
constexpr int kTile = 128;                 // keys per tile
constexpr int kChunkBytes = kTile * 128;   // 128 keys x 128 dims
constexpr int kRopeBytes = kTile * 64;
constexpr int kR = 16;                     // query rows per softmax warp
// log2 of the largest weight that a reference may stay with, of where a new reference puts a tile's
// largest, and of the excess that moves a row's when some row's weights pass the first
// (2^12.125: hi's residue is below 448 up to 2^12.149)
constexpr float kTop = 12.125f, kPlace = 6.f, kMove = 9.f;
// A largest weight that stands alone in its tile is put higher, so that the rest is at 2^kRest, up to
// 2^kAlone: below kTop, or another key of the same score would move the reference
constexpr float kRest = 3.f, kAlone = 12.f;
// A tile has fine weights where some row's largest of 16 keys is between 2^kNone and 2^kFine (see above)
constexpr float kNone = -22.f, kFine = -3.f;

// One segment of a block: tiles [t_begin, t_end) of a request's unit (b < 0: no more).
struct __align__(16) Seg {
  int b, t_begin, t_end, keys;    // keys: of the unit
  int cap, g, rank, single;       // the request's lengths; 1: the segment is the whole unit
};
constexpr int kSegRing = 4;
// Tiles whose mark of fine weights is kept.  That of tile n is read before its PV is over; the softmax
// warps wait for that PV in tile n + 2, before they come to tile n + 4's mark.
constexpr int kFineRing = 4;

template <int kN>
struct Cfg {
  static constexpr int kSoftWarps = 4 * (kN / kR);         // 4 x 32 keys, kR rows each
  static constexpr int kThreads = 128 + 32 * kSoftWarps;   // warps 0-2: loads, QK, PV
  static constexpr bool kQTmem = kN == 64;                 // Q's latent dims in tensor memory
  static constexpr int kSBufs = kQTmem ? 1 : 2;            // S buffers
  static constexpr int kQChunk = 2 * kN * 128;             // hi and lo rows of 128 dims
  static constexpr int kOffQRope = kQTmem ? 0 : 4 * kQChunk;
  static constexpr int kSegTiles = kN == 64 ? 3 : 6;       // cost of starting a segment, in tiles
  static constexpr int kSlots = kN == 64 ? 11 : 10;        // latent chunks in the ring (one rope chunk)
  static constexpr int kPBufs = 2;
  static constexpr int kPHalf = kTile * kN;                // hi or lo of P^T
  static constexpr int kOffK = kOffQRope + 2 * kN * 64;
  static constexpr int kOffRope = kOffK + kSlots * kChunkBytes;
  static constexpr int kOffP = kOffRope + kRopeBytes;
  static constexpr int kOffBar = kOffP + kPBufs * 2 * kPHalf;
  static constexpr int kOffRow = kOffBar + 384;            // five words for each row (softmax warps)
  static constexpr int kOffMisc = kOffRow + 20 * kN;       // tmem base, abort, scan result
  static constexpr int kOffSeg = kOffMisc + 48;            // Seg[kSegRing]
  static constexpr int kOffScale = kOffSeg + 32 * kSegRing;   // float4 [kSBufs tiles][8 groups of 16 keys]
  static constexpr int kOffFine = kOffScale + 128 * kSBufs;   // int [kFineRing]
  static constexpr int kSmem = kOffFine + 4 * kFineRing + 1008;   // + alignment slack
  // tensor memory: O^T, then S, then Q
  static constexpr uint32_t kColS = 4 * kN, kColQ = kColS + 128;
  static constexpr uint32_t kTmemCols = 8 * kN;
  static_assert(kOffK % 1024 == 0 && kOffRope % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static_assert(kSmem <= 232448, "shared memory of a block");
};

enum Bar : int {
  B_KF = 0,        // [12] latent chunk loaded
  B_KE = 12,       // [12] its PV done
  B_SF = 24,       // [2] S and the tile's scales written
  B_SE = 26,       // [2] both read (the softmax warps)
  B_PF = 28,       // [2] P^T written (the softmax warps)
  B_PE = 30,       // [2] its PV done
  B_RF = 32,       // rope chunk loaded
  B_RE = 33,       // its QK done
  B_QF = 34,       // the segment's Q written (the softmax warps)
  B_DRAIN = 35,    // [2] the QK / PV warp's last operations
  B_NEVER = 37,    // never arrived at (tests of the timeout path)
  B_GF = 38,       // [4] a segment has been written
  B_GE = 42,       // [4] and read by every role (three warps and the softmax warps)
  B_COUNT = 46
};

// 2^32 / the golden ratio: the upper bytes of its multiples are spread evenly over any run of keys
constexpr uint32_t kTurn = 0x9E3779B1u;

struct Params {
  const uint16_t* q;
  const float* scales;
  const int32_t* bt;
  long long bt_stride;
  const int32_t* seq_lens;
  const int32_t* gseq;
  int B, H, q_len, bs, num_blocks, max_blocks, rank;
  int causal, il;
  int span;                    // cp * il
  FastDiv div_H, div_span, div_rt, div_groups;
  unsigned long long wait_ns;
  int stall_test;
  int seg_tiles;               // start-up share of a request on the split line, in tiles
  int shard_B;
  unsigned shard_mul;          // as in mla_decode_tc.cu
  int rows;                    // H * q_len
  int row_tiles;               // R
  int units;
  int groups;                  // G: blocks g*R .. g*R + R-1 take the g-th range of the line
  int comb_blocks, comb_warps; // combine: blocks a unit, warps a row
  int whole_units;             // no workspace: requests go round the groups uncut
  int box_rows;                // rows per TMA box (a page is whole boxes)
  FastDiv div_bs;
  int tile_pages, tile_rest;   // 128 keys = tile_pages pages and tile_rest slots
  float scale_log2, lse_mul;
  uint16_t* out;
  float* lse;
  unsigned int* hdr;           // [0] = T
  int2* meta;                  // [units] first / last group of each unit
  float2* ws_lse;              // [2 * blocks][kN] LSE (base 2), sum of weights / l
  uint16_t* ws_o;              // [2 * blocks][kN][512] O / sum of weights, half precision
  unsigned int* status;
};

// ---- small device helpers ------------------------------------------------------------------
__device__ __forceinline__ unsigned int fdiv(unsigned int n, const FastDiv& f) {
  return f.d == 1u ? n : (unsigned int)__umul64hi(f.m, (unsigned long long)n);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Named barrier 1 over the softmax warps, alone and with an OR across them.
template <int kN>
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * Cfg<kN>::kSoftWarps) : "memory");
}
template <int kN>
__device__ __forceinline__ bool soft_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(32 * Cfg<kN>::kSoftWarps)
      : "memory");
  return r != 0;
}
// 16 lanes x 16 columns of tensor memory: a thread gets lanes lane / 4 (registers 0, 1, 4, 5) and
// lane / 4 + 8 (2, 3, 6, 7), columns 2 (lane % 4) and the next (0-3) and those 8 further (4-7).
__device__ __forceinline__ void tmem_load_16x16(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(addr)
               : "memory");
}
// Four 8 x 8 matrices of 16-bit elements; lane l holds elements 2 (l % 4) and the next of row l / 4
// of each, and gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
// The same layout over 16 lanes x 32 columns (four registers for eight columns), and written over
// 16 x 16.
__device__ __forceinline__ void tmem_load_16x32(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_16x16(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Four 16 x 8 matrices of bytes, stored transposed (8 lines of 16 bytes): lane l holds rows l / 4
// (bytes 0, 1) and l / 4 + 8 (bytes 2, 3), columns 2 (l % 4) and the next, of each, and gives the
// address of line l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_t_x4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m16n8.x4.trans.shared.b8 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, stored transposed: lane l holds elements 2 (l % 4) and the
// next of row l / 4 of each, and gives the address of column l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_t16_x4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Cut towards 0.
__device__ __forceinline__ uint32_t half2_cut(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^-16 (x 2^-32 - 1/2), by way of a float 1 + x 2^-32; its last bit set, so that half a step, 2^-17,
// is not reached on either side (a weight of 0 stays 0)
__device__ __forceinline__ float dither_of(uint32_t x) {
  return fmaf(__uint_as_float((x >> 9) | 0x3f800001u), 0x1p-16f, -0x1.8p-16f);
}
// 2^-9 (x 2^-16 - 1/2) for two 16-bit x, of their upper bytes, by way of halves 1024 + byte.  `minus`:
// kDown or kUp for each, which are off by half a step of a byte, 2^-18, either way.
constexpr uint32_t kDown = 0xa080u, kUp = 0xa07fu;         // -1152 and -1151 times 2^-17
__device__ __forceinline__ uint32_t dither2_of(uint32_t x, uint32_t minus) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(__byte_perm(x, 0x64u, 0x4341)), "r"(0x00800080u), "r"(minus));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Is a half of v between kNone and kFine?  (not so: NaN, -inf)
__device__ __forceinline__ bool any_fine(uint32_t v) {
  constexpr float kMid = (kFine + kNone) / 2, kHalf = (kFine - kNone) / 2;
  return fabsf(__uint_as_float(v << 16) - kMid) < kHalf || fabsf(__uint_as_float(v & 0xffff0000u) - kMid) < kHalf;
}
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t a) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)a));
  return r;
}
// Two halves as e4m3 bytes (the low one in the low byte), to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_of_half2(uint32_t a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(a));
  return r;
}

// Largest magnitude of 8 bf16 values, as their 15 bits.
__device__ __forceinline__ uint32_t peak8(const uint4& v) {
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
  return max(m & 0xffffu, m >> 16);
}
// 8 bf16 values times a power of two as e4m3 hi + lo; in half precision every scaled element is
// exact but for what lies below 2^-24.
__device__ __forceinline__ void split8(const uint4& w, float f, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  const uint64_t f2 = f32x2(f, f);
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x0, x1;
    f32x2_split(mul2(f32x2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u)), f2), x0, x1);
    const uint32_t u = half2_of(x0, x1);
    h[k] = e4m3x2_of_half2(u);
    l[k] = e4m3x2_of_half2(sub_half2(u, half2_of_e4m3x2(h[k])));
  }
  hi[0] = h[0] | h[1] << 16;
  hi[1] = h[2] | h[3] << 16;
  lo[0] = l[0] | l[1] << 16;
  lo[1] = l[2] | l[3] << 16;
}

// Instruction descriptor of kind::f8f6f4 with an fp32 accumulator; formats 0 = e4m3, 1 = e5m2;
// mn: both operands are stored M- (N-) major.
__host__ __device__ constexpr uint32_t idesc_f8(int N, uint32_t b_format, bool mn) {
  return (1u << 4) | (b_format << 10) | ((mn ? 1u : 0u) << 15) | ((mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
constexpr uint32_t kSwizzle64B = 4, kSwizzle32B = 6;

// A matrix descriptor (sm100.cuh) is passed as its two words: the high one holds the strides and
// the swizzle and is the same for every operand of a kind, the low one moves with the address
// (in 16 bytes).  Built whole for each product, descriptors took more instructions than anything
// else the issuing warps do.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | (1u << 16);           // leading stride 16 bytes (not used here)
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}

// kSteps products along K under one election, operands 32 bytes apart (K-major rows).
template <int kSteps>
__device__ __forceinline__ void qk_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                       uint32_t acc) {
  static_assert(kSteps == 2 || kSteps == 4, "chunks of 64 or 128 dims");
  if constexpr (kSteps == 4)
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 u, v;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " setp.ne.b32 t, %6, 0;\n elect.sync _|e, 0xffffffff;\n"
        " mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n"
        " add.u32 u, %1, 2; add.u32 v, %2, 2; mov.b64 x, {u, %3}; mov.b64 y, {v, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n"
        " add.u32 u, %1, 4; add.u32 v, %2, 4; mov.b64 x, {u, %3}; mov.b64 y, {v, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n"
        " add.u32 u, %1, 6; add.u32 v, %2, 6; mov.b64 x, {u, %3}; mov.b64 y, {v, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n"
        "}" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(1u)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 u, v;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n"
        " setp.ne.b32 t, %6, 0;\n elect.sync _|e, 0xffffffff;\n"
        " mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n"
        " add.u32 u, %1, 2; add.u32 v, %2, 2; mov.b64 x, {u, %3}; mov.b64 y, {v, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, t;\n"
        "}" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(1u)
        : "memory");
}

// Four products along K under one election, A in tensor memory (32 bytes of K are eight columns).
__device__ __forceinline__ void qk_mma_t(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 u, v;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n"
      " setp.ne.b32 t, %6, 0;\n elect.sync _|e, 0xffffffff;\n"
      " mov.b64 y, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], y, %4, p;\n"
      " add.u32 u, %1, 8; add.u32 v, %2, 2; mov.b64 y, {v, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [u], y, %4, t;\n"
      " add.u32 u, %1, 16; add.u32 v, %2, 4; mov.b64 y, {v, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [u], y, %4, t;\n"
      " add.u32 u, %1, 24; add.u32 v, %2, 6; mov.b64 y, {v, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [u], y, %4, t;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc), "r"(1u)
      : "memory");
}

// One product over 32 keys: values times one part of the weights.
__device__ __forceinline__ void pv_mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " mov.b64 x, {%1, %2}; mov.b64 y, {%3, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n"
      "}" ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}

// ---- row bounds and the work split (as in mla_decode_tc.cu, with units of kN rows and tiles
// of 128 keys) ---------------------------------------------------------------------------------
// All of it in 32 bits, with reciprocals from the host: lengths, cp * il and the split line are
// below 2^31 (the entry point and q8_supported see to it), and every block goes through this
// code before its first load (with 64-bit divisions that took 5 us).
__device__ __forceinline__ int shard_of(const Params& p, int b) {
  return (int)__umulhi((unsigned)b, p.shard_mul);
}
// A request's keys on its shard, its global length and its rank.
struct Lens {
  int cap, g, rank;
};
__device__ __forceinline__ Lens lens_of(const Params& p, int b) {
  const int sh = shard_of(p, b);
  Lens n;
  n.cap = max(min(__ldg(p.seq_lens + b), p.max_blocks * p.bs), 0);
  n.g = p.causal ? max(__ldg(p.gseq + (b - sh * p.shard_B)), 0) : 0;
  n.rank = p.rank + sh;
  return n;
}
// Keys that row r (0-based within the request's q_len*H rows) sees: the shard's share of the
// row's global prefix, at most its keys.
__device__ __forceinline__ int row_keys(const Params& p, const Lens& n, int r) {
  if (!p.causal) return n.cap;
  const int i = (int)fdiv((unsigned)r, p.div_H);
  const int g = max(n.g - (p.q_len - 1 - i), 0);
  const int q = (int)fdiv((unsigned)g, p.div_span);
  const int over = g - q * p.span - n.rank * p.il;
  return min(n.cap, q * p.il + min(max(over, 0), p.il));
}
template <int kN>
__device__ __forceinline__ int unit_keys(const Params& p, const Lens& n, int rt) {
  return row_keys(p, n, min((rt + 1) * kN, p.rows) - 1);     // its last row sees the most
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }
// A request's length on the split line: its tiles after the start-up share.
template <int kN>
__device__ __forceinline__ unsigned int req_span(const Params& p, const Lens& n) {
  const int nt = tiles_of(unit_keys<kN>(p, n, p.row_tiles - 1));
  return nt > 0 ? (unsigned)(nt + p.seg_tiles) : 0u;
}
// floor(T * c / G) for 0 <= c <= G (G <= 2^15)
__device__ __forceinline__ unsigned int range_start(const Params& p, unsigned int T, int c) {
  const unsigned int q = fdiv(T, p.div_groups), rest = T - q * (unsigned)p.groups;
  return q * (unsigned)c + fdiv(rest * (unsigned)c, p.div_groups);
}
// The group whose range holds position x < T.
__device__ __forceinline__ int owner_of(const Params& p, unsigned int x, unsigned int T) {
  return (int)((((unsigned long long)x + 1) * (unsigned)p.groups - 1) / T);
}

// The block's segments in order (walked by one warp, which passes them on).
template <int kN>
struct SegIter {
  int rt, grp;
  int nt, req_nt;                 // tiles of the unit, of the request (of its last unit)
  unsigned int g0, g_end;         // the request's first tile and the range's end on the line
  Seg seg;

  // request seg.b, of lengths n, from tile tb of it on
  __device__ bool set(const Params& p, const Lens& n, int tb) {
    req_nt = tiles_of(unit_keys<kN>(p, n, p.row_tiles - 1));
    seg.keys = unit_keys<kN>(p, n, rt);
    seg.cap = n.cap;
    seg.g = n.g;
    seg.rank = n.rank;
    nt = tiles_of(seg.keys);
    int te = nt;
    // a range may end inside the start-up share, before the request's first tile
    if (!p.whole_units) te = min(te, (int)(g_end - g0));
    if (tb >= te) return false;
    seg.t_begin = tb;
    seg.t_end = te;
    seg.single = tb == 0 && te == nt;
    return true;
  }
  __device__ bool next(const Params& p) {
    for (;;) {
      if (!p.whole_units) {
        // past the request; one without a tile has no place on the line
        if (req_nt > 0) g0 += req_nt + p.seg_tiles;
        if (g0 >= g_end) return false;
      }
      seg.b += p.whole_units ? p.groups : 1;
      if (seg.b >= p.B) return false;
      if (set(p, lens_of(p, seg.b), 0)) return true;
    }
  }
  // scan: the request that holds the range's first position, where its tiles begin, its lengths
  __device__ bool first(const Params& p, unsigned int T, const int* scan) {
    grp = (int)fdiv(blockIdx.x, p.div_rt);
    rt = blockIdx.x - grp * p.row_tiles;
    if (p.whole_units) {
      g0 = g_end = 0;
      seg.b = grp;
      if (seg.b >= p.B) return false;
      return set(p, lens_of(p, seg.b), 0) || next(p);
    }
    const unsigned int a = range_start(p, T, grp);
    g_end = range_start(p, T, grp + 1);
    if (a >= g_end || scan[0] < 0) return false;
    seg.b = scan[0];
    g0 = (unsigned)scan[1];
    return set(p, Lens{scan[2], scan[3], scan[4]}, a > g0 ? (int)(a - g0) : 0) || next(p);
  }
};

struct Ctx {
  uint32_t base;                 // shared address of the aligned base
  uint8_t* ptr;
  volatile int* abort;
};

template <int kN>
__device__ __forceinline__ uint32_t bar(const Ctx& s, int i) {
  return s.base + Cfg<kN>::kOffBar + 8 * i;
}
template <int kN>
__device__ __forceinline__ bool wait(const Ctx& s, int i, uint32_t parity, const Params& p) {
  return mbar_wait(bar<kN>(s, i), parity, s.abort, p.status, p.wait_ns);
}
__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }

// The i-th segment of the block, for one warp; false after the last one or when a wait gave up.
template <int kN>
__device__ __forceinline__ bool take_segment(const Ctx& s, uint32_t i, const Params& p, Seg& seg) {
  const uint32_t slot = i % kSegRing;
  const bool ok = warp_all(wait<kN>(s, B_GF + slot, (i / kSegRing) & 1, p));
  const int4* src = reinterpret_cast<const int4*>(s.ptr + Cfg<kN>::kOffSeg) + 2 * slot;
  const int4 a = src[0], b = src[1];
  seg = Seg{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar<kN>(s, B_GE + slot));
  return ok && seg.b >= 0;
}

// Four warps' part of a segment's output: the 128 dims of chunk col / kN (32 a warp) and twice 32
// rows of O^T, which go through 8 KB of shared memory (their share of P^T, which no product reads
// then) to become rows of 256 bytes (64 bytes, a warp by itself: 2 us more for 228 x 768 rows of 66
// keys, 163 us).
// The unit's output (bf16) is O / l.  A partial is O / w, w the sum of the weights (scales
// included): a mean of e4m3 values, at most 448, so that half precision holds it to 2^-11 in half
// the bytes of fp32; w / l goes with the row's LSE.  (A function of its own, so that its registers
// do not weigh on the loop over the tiles.)
template <int kN>
__device__ __noinline__ void store_rows(uint32_t tmem, uint8_t* stage, const float* inv, uint16_t* dst, int quad,
                                        int part, int nrow, bool single) {
  using C = Cfg<kN>;
  static_assert(C::kPBufs * 2 * C::kPHalf >= 2048 * C::kSoftWarps, "2 KB a warp");
  const int lane = threadIdx.x & 31, c4 = lane & 3;
  auto sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(2 + part) : "memory"); };
#pragma unroll 1
  for (int c32 = 0; c32 < 2; ++c32) {
    const int col = part * 64 + c32 * 32, r0 = col % kN;
    uint32_t v[2][16];                     // [h]: dims 16 h + lane / 4 and + 8
    tmem_load_16x32(tmem + (uint32_t)col, v[0]);
    tmem_load_16x32(tmem + (16u << 16) + (uint32_t)col, v[1]);
    tmem_wait_ld();
    if (c32) sync();                       // the rows before have been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = *reinterpret_cast<const float2*>(inv + r0 + 8 * i + 2 * c4);
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __uint_as_float(v[k >> 1][4 * i + 2 * (k & 1)]) * f.x;
        const float b = __uint_as_float(v[k >> 1][4 * i + 2 * (k & 1) + 1]) * f.y;
        const __nv_bfloat162 o2 = __floats2bfloat162_rn(a, b);
        u[k] = single ? *reinterpret_cast<const uint32_t*>(&o2) : half2_of(a, b);
      }
      // lane l gives the address of row l % 8 of the eight, dims 32 quad + 8 (l / 8) ..
      const int r = 8 * i + (lane & 7);
      stmatrix_t16_x4(smem_u32(stage) + r * 256 + ((4 * quad + (lane >> 3)) ^ (lane & 7)) * 16, u);
    }
    sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * quad + 2 * i + (lane >> 4), unit = lane & 15;
      const uint4 o = *reinterpret_cast<const uint4*>(stage + r * 256 + (unit ^ (r & 7)) * 16);
      if (r0 + r < nrow) *reinterpret_cast<uint4*>(dst + (r0 + r) * kDv + col / kN * 128 + unit * 8) = o;
    }
  }
}

// ---------------------------------------------------------------------------------------------
template <int kN>
__global__ void __launch_bounds__(Cfg<kN>::kThreads, 1)
    mla_decode_q8_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap rmap, const Params p) {
  using C = Cfg<kN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Ctx s;
  s.ptr = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  s.base = smem_u32(s.ptr);
  uint32_t* misc = reinterpret_cast<uint32_t*>(s.ptr + C::kOffMisc);   // [0] tmem base, [1] abort
  s.abort = reinterpret_cast<volatile int*>(misc + 1);
  int* s_scan = reinterpret_cast<int*>(misc + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- setup: barriers, tensor memory, schedule scan --------------------------------------------
  if (tid == 64) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&rmap);
  }
  if (warp == 2) {
    if (lane == 0) *s.abort = 0;
    for (int i = lane; i < B_COUNT; i += 32) {
      const bool by_warps = i == B_SE || i == B_SE + 1 || i == B_PF || i == B_PF + 1 || i == B_QF;
      const bool by_all = i >= B_GE && i < B_GE + kSegRing;
      const int count = by_all ? C::kSoftWarps + 3 : by_warps ? C::kSoftWarps : i == B_SF || i == B_SF + 1 ? 2 : 1;
      mbar_init(bar<kN>(s, i), count);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s.base + C::kOffMisc, C::kTmemCols);
    tmem_relinquish();
  }
  // a dependent launch (as the combine): nothing before this line touches global memory
  asm volatile("griddepcontrol.wait;" ::: "memory");
  unsigned int T = 0;
  {
    // T = length of the split line; the request that holds this group's first position.  The
    // per-warp sums use the P buffer, which nothing else touches yet.
    unsigned int* s_warp = reinterpret_cast<unsigned int*>(s.ptr + C::kOffP);
    constexpr int kThreads = C::kThreads, kWarps = kThreads / 32;
    if (tid == 0) s_scan[0] = -1;
    // inclusive sum over the block; `before` is what the earlier warps add to it
    auto scan = [&](unsigned int n, unsigned int& total) {
      unsigned int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      const unsigned int w = lane < kWarps ? s_warp[lane] : 0u;
      total = __reduce_add_sync(0xffffffffu, w);
      incl += __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
      __syncthreads();
      return incl;
    };
    Lens own{0, 0, 0};
    if (tid < p.B) own = lens_of(p, tid);
    unsigned int n = tid < p.B ? req_span<kN>(p, own) : 0u, total;
    unsigned int end = scan(n, total);
    T = total;
    for (int b0 = kThreads; b0 < p.B; b0 += kThreads) {
      scan(b0 + tid < p.B ? req_span<kN>(p, lens_of(p, b0 + tid)) : 0u, total);
      T += total;
    }
    if (!p.whole_units && T > 0) {
      const unsigned int a = range_start(p, T, (int)fdiv(blockIdx.x, p.div_rt));
      unsigned int running = 0;
      for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        if (p.B > kThreads) {                      // more requests than threads: summed again
          if (b0 + tid < p.B) own = lens_of(p, b0 + tid);
          n = b0 + tid < p.B ? req_span<kN>(p, own) : 0u;
          end = scan(n, total);
        }
        const unsigned int excl = running + end - n;
        if (n > 0 && excl <= a && a < excl + n) {
          s_scan[0] = b0 + tid;
          s_scan[1] = (int)(excl + p.seg_tiles);
          s_scan[2] = own.cap;
          s_scan[3] = own.g;
          s_scan[4] = own.rank;
        }
        running += total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  if (blockIdx.x == 0 && tid == 0 && !p.whole_units) p.hdr[0] = T;

  const int rt = (int)(blockIdx.x - fdiv(blockIdx.x, p.div_rt) * (unsigned)p.row_tiles);   // this block's units
  Seg it;
  uint32_t nseg = 0;                        // segments taken
  if (warp == 0) {
    // ================= loads: per tile four latent chunks and the rope chunk ====================
    const int nbox = kTile / p.box_rows;
    const uint32_t box_lat = (uint32_t)p.box_rows * 128, box_rope = (uint32_t)p.box_rows * 64;
    bool ok = true, bad = false;
    int slot = 0;
    uint32_t kpar = 1;                      // a slot's first use passes at once
    long long chunks = 0, ropes = 0;
    while (ok && take_segment<kN>(s, nseg++, p, it)) {
        const int32_t* btrow = p.bt + (long long)it.b * p.bt_stride;
        // cache row of the segment's box i; a missing or invalid page becomes a row past the
        // cache, which TMA fills with zeros
        auto row_of = [&](int i) {
          const int tok = i * p.box_rows;          // below 2^31: see q8_supported
          int y = p.num_blocks * p.bs;
          if (tok < it.keys) {
            const int pg = (int)fdiv((unsigned)tok, p.div_bs);
            const int page = __ldg(btrow + pg);
            if (page >= 0 && page < p.num_blocks)
              y = page * p.bs + (tok - pg * p.bs);
            else
              bad = true;
          }
          return y;
        };
        // lane l holds box i0 + l of the current window, the next window one ahead
        int i0 = it.t_begin * nbox;
        int cur = row_of(i0 + lane), nxt = row_of(i0 + 32 + lane);
        // the segment's Q rows (consecutive bytes) on their way to L2: the softmax warps come to them
        // up to a segment later
        if (lane == 0) {
          const int sh = shard_of(p, it.b);
          const long long row = (long long)(it.b - sh * p.shard_B) * p.rows + rt * kN;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.q + row * kD),
                       "r"(min(kN, p.rows - rt * kN) * kD * 2)
                       : "memory");
        }
        for (int t = it.t_begin; t < it.t_end && ok; ++t) {
          if (t * nbox >= i0 + 32) {
            i0 += 32;
            cur = nxt;
            nxt = row_of(i0 + 32 + lane);
          }
          // lane l < nbox issues the tile's box l
          const int y = __shfl_sync(0xffffffffu, cur, (t * nbox + lane - i0) & 31);
          for (int c = 0; c < 4; ++c) {
            ok = warp_all(wait<kN>(s, B_KE + slot, kpar, p));
            if (!ok) break;
            const uint32_t fb = bar<kN>(s, B_KF + slot);
            if (lane == 0) mbar_arrive_expect_tx(fb, kChunkBytes);
            __syncwarp();
            if (lane < nbox)
              tma_load_2d(s.base + C::kOffK + slot * kChunkBytes + lane * box_lat, &kmap, c * 128, y, fb);
            ++chunks;
            if (++slot == C::kSlots) {
              slot = 0;
              kpar ^= 1u;
            }
          }
          if (!ok) break;
          ok = warp_all(wait<kN>(s, B_RE, (uint32_t)((ropes + 1) & 1), p));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar<kN>(s, B_RF), kRopeBytes);
          __syncwarp();
          if (lane < nbox)
            tma_load_2d(s.base + C::kOffRope + lane * box_rope, &rmap, kDv, y, bar<kN>(s, B_RF));
          ++ropes;
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    if (*s.abort && lane == 0) {
      // loads already issued land before the block exits
      for (long long m = chunks > C::kSlots ? chunks - C::kSlots : 0; m < chunks; ++m)
        mbar_wait_drain(bar<kN>(s, B_KF + (int)(m % C::kSlots)), (uint32_t)((m / C::kSlots) & 1));
      if (ropes > 0) mbar_wait_drain(bar<kN>(s, B_RF), (uint32_t)((ropes - 1) & 1));
    }
  } else if (warp == 1) {
    // ================= QK ========================================================================
    constexpr uint32_t id_qk = idesc_f8(2 * kN, 0, false);
    const uint32_t ka = desc_lo(s.base + C::kOffK), qa = desc_lo(s.base);
    bool ok = true;
    if (p.stall_test) ok = warp_all(wait<kN>(s, B_NEVER, 0, p));
    long long n = 0;
    int slot = 0;
    uint32_t par = 0;
    while (ok && take_segment<kN>(s, nseg++, p, it)) {
        ok = warp_all(wait<kN>(s, B_QF, (nseg - 1) & 1, p));
        for (int t = it.t_begin; t < it.t_end && ok; ++t, ++n) {
          const int g = (int)(n % C::kSBufs);
          ok = warp_all(wait<kN>(s, B_SE + g, (uint32_t)((n / C::kSBufs + 1) & 1), p));   // S read
          const uint32_t d = tmem + C::kColS + g * 2 * kN;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ok = ok && warp_all(wait<kN>(s, B_KF + slot, par, p));
            if (!ok) break;
            tc_fence_after();
            if constexpr (C::kQTmem)
              qk_mma_t(d, tmem + C::kColQ + c * 32, ka + slot * (kChunkBytes / 16), desc_hi(1024, kSwizzle128B), id_qk,
                       c != 0);
            else
              qk_mma<4>(d, ka + slot * (kChunkBytes / 16), qa + c * (C::kQChunk / 16),
                        desc_hi(1024, kSwizzle128B), id_qk, c != 0);
            if (++slot == C::kSlots) {
              slot = 0;
              par ^= 1u;
            }
          }
          ok = ok && warp_all(wait<kN>(s, B_RF, (uint32_t)(n & 1), p));
          if (!ok) break;
          tc_fence_after();
          const uint32_t kr = desc_lo(s.base + C::kOffRope), qr = qa + C::kOffQRope / 16;
          qk_mma<2>(d, C::kQTmem ? qr : kr, C::kQTmem ? kr : qr, desc_hi(512, kSwizzle64B), id_qk, 1);
          mma_commit_warp(bar<kN>(s, B_RE));
          mma_commit_warp(bar<kN>(s, B_SF + g));
        }
    }
    // every operation issued here completes before the block tears down
    mma_commit_warp(bar<kN>(s, B_DRAIN));
    mbar_wait_drain(bar<kN>(s, B_DRAIN), 0);
  } else if (warp == 2) {
    // ================= PV ========================================================================
    constexpr uint32_t id_hi = idesc_f8(kN, 1, true), id_lo = idesc_f8(kN, 0, true);
    constexpr uint32_t p_hi = desc_hi(8 * kN, kN == 64 ? kSwizzle64B : kSwizzle32B);
    const uint32_t va = desc_lo(s.base + C::kOffK), pa0 = desc_lo(s.base + C::kOffP);
    bool ok = true;
    long long n = 0;
    int slot = 0;
    while (ok && take_segment<kN>(s, nseg++, p, it)) {
        for (int t = it.t_begin; t < it.t_end; ++t, ++n) {
          const int pb = (int)(n % C::kPBufs);
          ok = warp_all(wait<kN>(s, B_PF + pb, (uint32_t)((n / C::kPBufs) & 1), p));
          if (!ok) break;
          tc_fence_after();
          const uint32_t pa = pa0 + pb * (2 * C::kPHalf / 16);
          // (comes while the first products, which it does not concern, are issued)
          const int fine = reinterpret_cast<const int*>(s.ptr + C::kOffFine)[n % kFineRing];
          // chunk c of the values (dims 128 c ..), step k of 32 keys: the weights' first part, or the second
          auto product = [&](int c, int k, bool second, uint32_t id) {
            pv_mma(tmem + c * kN, va + slot * (kChunkBytes / 16) + k * (4096 / 16), desc_hi(1024, kSwizzle128B),
                   pa + ((second ? C::kPHalf : 0) + k * 32 * kN) / 16, p_hi, id,
                   (t == it.t_begin && k == 0 && !second) ? 0u : 1u);
          };
          auto release = [&]() {
            mma_commit_warp(bar<kN>(s, B_KE + slot));
            if (++slot == C::kSlots) slot = 0;
          };
          // the steps that hold keys, in straight code for each count: a branch between two products
          // costs more than a product (3 % of a long request, 2,500 cycles of a short one)
          auto run = [&](auto steps) {
            constexpr int kSteps = decltype(steps)::value;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) product(0, k, false, id_hi);
            auto rest = [&](uint32_t id) {
#pragma unroll
              for (int k = 0; k < kSteps; ++k) product(0, k, true, id);
              release();
#pragma unroll 1
              for (int c = 1; c < 4; ++c) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                  product(c, k, false, id_hi);
                  product(c, k, true, id);
                }
                release();
              }
            };
            rest(fine ? id_hi : id_lo);
          };
          const int left = it.keys - t * kTile;
          if (left > 96)
            run(std::integral_constant<int, 4>{});
          else if (left > 64)
            run(std::integral_constant<int, 3>{});
          else if (left > 32)
            run(std::integral_constant<int, 2>{});
          else
            run(std::integral_constant<int, 1>{});
          mma_commit_warp(bar<kN>(s, B_PE + pb));
        }
    }
    mma_commit_warp(bar<kN>(s, B_DRAIN + 1));
    mbar_wait_drain(bar<kN>(s, B_DRAIN + 1), 0);
  } else if (warp == 3) {
    // ================= the schedule and the tiles' scales =========================================
    // Passes the block's segments on, one ahead of the tiles, and writes each tile's eight scales
    // (lane l < 8: those of keys 16 l ..), with their logarithms and reciprocals, for the softmax
    // warps, which otherwise looked them up 4 (kN / 16) times over.
    SegIter<kN> walk;
    const int groups_per_page = p.bs / MLA_Q8_GROUP;
    bool have = walk.first(p, T, s_scan), bad_scale = false, ok = true;
    uint32_t n = 0;
    // the next segment's description into the ring (b = -1: no more)
    auto publish = [&]() {
      const uint32_t slot = nseg % kSegRing;
      ok = ok && warp_all(wait<kN>(s, B_GE + slot, ((nseg / kSegRing) + 1) & 1, p));
      if (!ok) return;
      ++nseg;
      if (lane == 0) {
        int4* dst = reinterpret_cast<int4*>(s.ptr + C::kOffSeg) + 2 * slot;
        dst[0] = make_int4(have ? walk.seg.b : -1, walk.seg.t_begin, walk.seg.t_end, walk.seg.keys);
        dst[1] = make_int4(walk.seg.cap, walk.seg.g, walk.seg.rank, walk.seg.single);
        mbar_arrive(bar<kN>(s, B_GF + slot));
        // the owner of a unit's first tile records which groups hold the unit
        if (have && walk.seg.t_begin == 0 && !p.whole_units)
          p.meta[walk.seg.b * p.row_tiles + rt] = make_int2(walk.grp, owner_of(p, walk.g0 + walk.nt - 1, T));
      }
      __syncwarp();
    };
    publish();
    while (have && ok) {
      it = walk.seg;
      // group l of a tile is at slot `at` of the request: page pg, offset off; the page is looked up
      // two tiles ahead, the scale one
      const int32_t* btrow = p.bt + (long long)it.b * p.bt_stride;
      const int at_end = lane < 8 ? min(it.keys, it.t_end * kTile) : 0;
      int at = it.t_begin * kTile + lane * MLA_Q8_GROUP;
      int pg = (int)fdiv((unsigned)at, p.div_bs), off = at - pg * p.bs;
      auto page_here = [&]() { return at < at_end ? __ldg(btrow + pg) : -1; };
      auto scale_in = [&](int page) {
        return page >= 0 && page < p.num_blocks
                   ? __ldg(p.scales + (long long)page * groups_per_page + (off >> 4))
                   : 1.f;
      };
      auto step = [&]() {
        at += kTile;
        pg += p.tile_pages;
        off += p.tile_rest;
        if (off >= p.bs) {
          off -= p.bs;
          ++pg;
        }
      };
      float sc_next = scale_in(page_here());
      step();
      int page_next = page_here();
      have = walk.next(p);
      publish();
      for (int t = it.t_begin; t < it.t_end && ok; ++t, ++n) {
        const uint32_t g = n % C::kSBufs;
        float sc = sc_next;
        sc_next = scale_in(page_next);
        step();
        page_next = page_here();
        if (!(sc >= MLA_Q8_SCALE_MIN && sc <= MLA_Q8_SCALE_MAX)) {
          bad_scale = true;
          sc = 1.f;
        }
        const float4 v = make_float4(sc, fast_log2(sc), fast_rcp(sc), 0.f);
        ok = warp_all(wait<kN>(s, B_SE + g, (n / C::kSBufs + 1) & 1, p));
        if (lane < 8) reinterpret_cast<float4*>(s.ptr + C::kOffScale)[g * 8 + lane] = v;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar<kN>(s, B_SF + g));
      }
    }
    if (__any_sync(0xffffffffu, bad_scale) && lane == 0) atomicOr(p.status, MLA_STATUS_BAD_SCALE);
  } else if (warp >= 4) {
    // ================= softmax ===================================================================
    // A warp has 32 keys of a tile (from 32 kq) and 16 rows of the unit (from 16 rg).  S is read
    // so that a thread's values need no exchange and leave as words of P^T:
    //   64 rows: lanes of tensor memory are rows (16 hi, 16 lo for each 16 rows), columns keys.  A
    //     thread has rows lane / 4 and + 8, keys 2 (lane % 4) and the next of each eight;
    //   32 rows: lanes are keys, columns rows (hi, then lo).  A thread has keys lane / 4 + 8 i; Q's
    //     rows are laid out so that its columns are rows 4 (lane % 4) .. + 3.
    // y[i][k] is then row k / 2, key 8 i + k % 2, or key i, row k.
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const int kq = C::kQTmem ? part : quad, rg = C::kQTmem ? quad : part;
    const int c4 = lane & 3;
    const int my_rows = C::kQTmem ? 16 * rg + (lane >> 2) : 16 * rg + 4 * c4;
    const int my_keys = kq * 32 + (C::kQTmem ? 2 * c4 : lane >> 2);
    const int key = kq * 32 + lane;                // the key whose 16 bytes of P^T this thread addresses
    const int st = tid - 128;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    float* row_a = reinterpret_cast<float*>(s.ptr + C::kOffRow);     // log2 units per unit of S
    float* row_nm = row_a + kN;                                      // minus the reference
    float* shift = row_nm + kN;                                      // its move; later 1 / l
    float* factor = shift + kN;                                      // 2^shift
    int* lim = reinterpret_cast<int*>(factor + kN);                  // keys the row sees
    // the thread's rows' values of a row array (by k of y[i][k])
    auto of_rows = [&](const auto* v) {
      using T = std::remove_cv_t<std::remove_reference_t<decltype(*v)>>;
      using T4 = std::conditional_t<std::is_same_v<T, float>, float4, int4>;
      if constexpr (C::kQTmem) {
        const T a = v[my_rows], b = v[my_rows + 8];
        return T4{a, a, b, b};
      } else {
        return *reinterpret_cast<const T4*>(v + my_rows);
      }
    };
    // v, combined over the warp's keys, into row array `to`
    auto over_keys = [&](float4 v, auto op, float* to) {
      if constexpr (C::kQTmem) {
        float a = op(v.x, v.y), b = op(v.z, v.w);
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          a = op(a, __shfl_xor_sync(0xffffffffu, a, o));
          b = op(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        if (c4 == 0) {
          to[my_rows] = a;
          to[my_rows + 8] = b;
        }
      } else {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          v.x = op(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
          v.y = op(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
          v.z = op(v.z, __shfl_xor_sync(0xffffffffu, v.z, o));
          v.w = op(v.w, __shfl_xor_sync(0xffffffffu, v.w, o));
        }
        if (lane < 4) *reinterpret_cast<float4*>(to + my_rows) = v;
      }
    };
    // 2^up puts a maximum with exponent ex in [128, 256) (one below 2^-119 less far up); the row's
    // constants
    auto set_row = [&](int r, int ex) {
      const int up = min(134 - ex, 126);
      const float a = __int_as_float((127 - up) << 23) * p.scale_log2;
      row_a[r] = ex == 255 ? __int_as_float(0x7fc00000) : a;          // NaN or infinity: a NaN row
      row_nm[r] = 0.f;
    };
    auto q_factor = [](int ex) { return __int_as_float((min(134 - ex, 126) + 127) << 23); };
    uint32_t n = 0;
    // The order of a block's segments: Q of the next one is prepared (and its first QK may run)
    // before the output of the one before is written, which waits for its last PV.
    uint64_t w01 = 0, w23 = 0;                     // sums of weights by k of y[i][k]
    uint64_t l01 = 0, l23 = 0;                     // sums of weights / S
    bool have = !soft_or<kN>(!take_segment<kN>(s, nseg++, p, it)), pending = false;
    // of the segment whose output is to be written: its request, whether it is a whole unit, which of
    // the block's two partials it is
    int out_b = 0, out_part = 0;
    bool out_single = false;
    float out_nm = 0.f;
    for (;;) {
      if (have) {
        const int row0 = rt * kN;
        const int sh = shard_of(p, it.b);
        const uint16_t* q0 = p.q + ((long long)(it.b - sh * p.shard_B) * p.rows + row0) * kD;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if (st < kN) lim[st] = row0 + st < p.rows ? row_keys(p, Lens{it.cap, it.g, it.rank}, row0 + st) : it.keys;
        if constexpr (C::kQTmem) {
          // ---- Q into tensor memory, rope dims into shared memory; a warp has its 16 rows' dims
          // 128 kq .. + 127, a thread eight dims of each 32 of two rows, and eight rope dims of one ---
          static_assert(kN == 64, "16 rows for each quarter of the lanes");
          const bool v0 = row0 + my_rows < p.rows, v1 = row0 + my_rows + 8 < p.rows, second = c4 >= 2;
          const uint16_t *s0 = q0 + (v0 ? my_rows : 0) * kD, *s1 = q0 + (v1 ? my_rows + 8 : 0) * kD;
          uint4 w[2][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int dim = kq * 128 + k * 32 + c4 * 8;
            w[0][k] = v0 ? __ldg(reinterpret_cast<const uint4*>(s0 + dim)) : zero;
            w[1][k] = v1 ? __ldg(reinterpret_cast<const uint4*>(s1 + dim)) : zero;
          }
          const int piece = 2 * kq + (c4 & 1);     // of the row's eight pieces of 8 rope dims
          const uint4 wr =
              (second ? v1 : v0) ? __ldg(reinterpret_cast<const uint4*>((second ? s1 : s0) + kDv + piece * 8)) : zero;
          uint32_t m0 = second ? 0u : peak8(wr), m1 = second ? peak8(wr) : 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            m0 = max(m0, peak8(w[0][k]));
            m1 = max(m1, peak8(w[1][k]));
          }
#pragma unroll
          for (int o = 1; o <= 2; o <<= 1) {
            m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          }
          uint8_t* ex = reinterpret_cast<uint8_t*>(shift);            // [4][kN] exponents; shift is free here
          if (c4 == 0) {
            ex[kq * kN + my_rows] = (uint8_t)(m0 >> 7);
            ex[kq * kN + my_rows + 8] = (uint8_t)(m1 >> 7);
          }
          soft_sync<kN>();
          int e0 = 0, e1 = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e0 = max(e0, (int)ex[k * kN + my_rows]);
            e1 = max(e1, (int)ex[k * kN + my_rows + 8]);
          }
          if (kq == 0 && c4 == 0) {
            set_row(my_rows, e0);
            set_row(my_rows + 8, e1);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[2], l[2];
              split8(w[k & 1][2 * half + (k >> 1)], q_factor(k & 1 ? e1 : e0), h, l);
              hi[2 * k] = h[0];
              hi[2 * k + 1] = h[1];
              lo[2 * k] = l[0];
              lo[2 * k + 1] = l[1];
            }
            const uint32_t dst = tmem + lane_off + C::kColQ + kq * 32 + half * 16;
            tmem_store_16x16(dst, hi);
            tmem_store_16x16(dst + (16u << 16), lo);
          }
          {
            uint32_t h[2], l[2];
            split8(wr, q_factor(second ? e1 : e0), h, l);
            const int line = 32 * rg + (lane >> 2) + (second ? 8 : 0);            // of hi; lo is 16 on
            uint8_t* dst = s.ptr + C::kOffQRope + line * 64 + (((piece >> 1) ^ ((line >> 1) & 3)) << 4) +
                           (piece & 1) * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
            *reinterpret_cast<uint2*>(dst + 16 * 64) = make_uint2(l[0], l[1]);
          }
          tmem_wait_st();
          tc_fence_before();
        } else {
          // ---- Q into shared memory: eight lanes a row ------------------------------------------
          static_assert(kN == 4 * C::kSoftWarps, "four rows a warp");
          const int r = (warp - 4) * 4 + (lane >> 3), l8 = lane & 7;
          const bool valid = row0 + r < p.rows;
          const uint4* src = reinterpret_cast<const uint4*>(q0 + (valid ? r : 0) * kD) + l8;
          uint4 w[9];                              // elements 8 (l8 + 8 i) .. + 7
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 9; ++i) w[i] = valid ? __ldg(src + 8 * i) : zero;
#pragma unroll
          for (int i = 0; i < 9; ++i) m = max(m, peak8(w[i]));
#pragma unroll
          for (int o = 1; o <= 4; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int ex = (int)(m >> 7);
          if (l8 == 0) set_row(r, ex);
          const int col = (r & ~15) + ((r & 2) << 2) + ((r & 12) >> 1) + (r & 1);   // its column of S^T
          uint8_t* lat = s.ptr + col * 128 + (l8 & 1) * 8;
          uint8_t* rope = s.ptr + C::kOffQRope + col * 64 + (((l8 >> 1) ^ ((col >> 1) & 3)) << 4) + (l8 & 1) * 8;
#pragma unroll
          for (int i = 0; i < 9; ++i) {
            uint32_t h[2], l[2];
            split8(w[i], q_factor(ex), h, l);
            uint8_t* dst = i < 8 ? lat + (i >> 1) * C::kQChunk + ((((i & 1) * 4 + (l8 >> 1)) ^ (col & 7)) << 4)
                                 : rope;
            *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
            *reinterpret_cast<uint2*>(dst + (i < 8 ? kN * 128 : kN * 64)) = make_uint2(l[0], l[1]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar<kN>(s, B_QF));
      }
      if (pending) {
        const int out_row0 = rt * kN;
        const long long out_row = (long long)out_b * p.rows + out_row0, out_slot = 2ll * blockIdx.x + out_part;
        // ---- the segment's output ---------------------------------------------------------------
        wait<kN>(s, B_PE + (n - 1) % C::kPBufs, ((n - 1) / C::kPBufs) & 1, p);
        tc_fence_after();
        {
          float* xs = reinterpret_cast<float*>(s.ptr + C::kOffP);        // [2][4][kN]
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float4 sum;
            f32x2_split(v ? w01 : l01, sum.x, sum.y);
            f32x2_split(v ? w23 : l23, sum.z, sum.w);
            over_keys(sum, [](float a, float b) { return a + b; }, xs + (v * 4 + kq) * kN);
          }
          soft_sync<kN>();
          if (st < kN) {
            const float l = (xs[st] + xs[kN + st]) + (xs[2 * kN + st] + xs[3 * kN + st]);
            const float* xw = xs + 4 * kN;
            const float w = (xw[st] + xw[kN + st]) + (xw[2 * kN + st] + xw[3 * kN + st]);
            const float lse2 = l == 0.f ? -INFINITY : log2f(l) - out_nm;
            const float by = out_single ? l : w;
            shift[st] = by == 0.f ? 0.f : 1.f / by;                       // NaN stays NaN
            if (!out_single) {
              p.ws_lse[out_slot * kN + st] = make_float2(lse2, l == 0.f ? 0.f : w / l);
            } else if (p.lse != nullptr && out_row0 + st < p.rows) {
              p.lse[out_row + st] = lse2 * p.lse_mul;
            }
          }
          soft_sync<kN>();
          const int nrow = min(kN, p.rows - out_row0);
          uint16_t* dst = out_single ? p.out + out_row * kDv : p.ws_o + out_slot * kN * kDv;
          store_rows<kN>(tmem + lane_off, s.ptr + C::kOffP + part * 8192, shift, dst, quad, part, nrow, out_single);
          tc_fence_before();
        }
      }
      if (!have) break;
      soft_sync<kN>();                             // row constants and limits; shift is free again
      const int all_see = lim[0];                // every row of the unit sees this many keys
      const float4 a4 = of_rows(row_a);
      float4 nm4 = make_float4(0.f, 0.f, 0.f, 0.f);

      w01 = w23 = l01 = l23 = 0;
      for (int t = it.t_begin; t < it.t_end; ++t, ++n) {
        const uint32_t g = n % C::kSBufs, pb = n % C::kPBufs;
        wait<kN>(s, B_SF + g, (n / C::kSBufs) & 1, p);
        tc_fence_after();
        float y[4][4];
        float inv_g[2];
        {
          uint32_t hi[2][8], lo[2][8];             // [j]: group of keys j
          const uint32_t src = tmem + lane_off + C::kColS + g * 2 * kN + (C::kQTmem ? 32 * kq : kR * rg);
          if constexpr (C::kQTmem) {
            tmem_load_16x32(src, reinterpret_cast<uint32_t(&)[16]>(hi));
            tmem_load_16x32(src + (16u << 16), reinterpret_cast<uint32_t(&)[16]>(lo));
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              tmem_load_16x16(src + ((uint32_t)(16 * j) << 16), hi[j]);
              tmem_load_16x16(src + ((uint32_t)(16 * j) << 16) + kN, lo[j]);
            }
          }
          // t' = acc * (a S) + (log2 S - m), for the group of keys i = 0, 1 and that of 2, 3
          uint64_t A[2][2], Bc[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 v = reinterpret_cast<const float4*>(s.ptr + C::kOffScale)[g * 8 + 2 * kq + j];
            inv_g[j] = v.z;
            A[j][0] = mul2(f32x2(a4.x, a4.y), f32x2(v.x, v.x));
            A[j][1] = mul2(f32x2(a4.z, a4.w), f32x2(v.x, v.x));
            Bc[j][0] = add2(f32x2(nm4.x, nm4.y), f32x2(v.y, v.y));
            Bc[j][1] = add2(f32x2(nm4.z, nm4.w), f32x2(v.y, v.y));
          }
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar<kN>(s, B_SE + g));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = i >> 1, r = C::kQTmem ? (i & 1) * 4 + k * 2 : (i & 1) * 2 + k * 4;
              const uint64_t acc =
                  add2(f32x2(__uint_as_float(hi[j][r]), __uint_as_float(hi[j][r + 1])),
                       f32x2(__uint_as_float(lo[j][r]), __uint_as_float(lo[j][r + 1])));
              f32x2_split(fma2(acc, A[j][k], Bc[j][k]), y[i][2 * k], y[i][2 * k + 1]);
            }
        }
        if ((t + 1) * kTile > all_see) {
          // a key that a row does not see weighs nothing, whatever its slot holds
          const int4 l4 = of_rows(lim);
          constexpr int kStep = C::kQTmem ? 1 : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k_abs = t * kTile + my_keys + 8 * i;
            if (k_abs >= l4.x) y[i][0] = -INFINITY;
            if (k_abs + kStep >= l4.y) y[i][1] = -INFINITY;
            if (k_abs >= l4.z) y[i][2] = -INFINITY;
            if (k_abs + kStep >= l4.w) y[i][3] = -INFINITY;
          }
        }
        // the rows' largest of this thread's keys (by k of y[i][k])
        float4 m4;
        if constexpr (C::kQTmem) {
          m4.x = m4.y = fmax3(fmax3(fmax3(y[0][0], y[0][1], y[1][0]), y[1][1], y[2][0]),
                              fmax3(y[2][1], y[3][0], y[3][1]), -INFINITY);
          m4.z = m4.w = fmax3(fmax3(fmax3(y[0][2], y[0][3], y[1][2]), y[1][3], y[2][2]),
                              fmax3(y[2][3], y[3][2], y[3][3]), -INFINITY);
        } else {
          m4.x = fmaxf(fmax3(y[0][0], y[1][0], y[2][0]), y[3][0]);
          m4.y = fmaxf(fmax3(y[0][1], y[1][1], y[2][1]), y[3][1]);
          m4.z = fmaxf(fmax3(y[0][2], y[1][2], y[2][2]), y[3][2]);
          m4.w = fmaxf(fmax3(y[0][3], y[1][3], y[2][3]), y[3][3]);
        }
        // does a row's largest of 16 keys, this thread's and its neighbours', ask for fine weights?
        auto asks = [&]() {
          if constexpr (C::kQTmem) {
            uint32_t v = bf16x2_of(m4.x, m4.z);
            v = max_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, 1));
            return any_fine(v);
          } else {
            uint32_t v = bf16x2_of(m4.x, m4.y), w = bf16x2_of(m4.z, m4.w);
#pragma unroll
            for (int o = 4; o <= 8; o <<= 1) {
              v = max_bf16x2(v, __shfl_xor_sync(0xffffffffu, v, o));
              w = max_bf16x2(w, __shfl_xor_sync(0xffffffffu, w, o));
            }
            return any_fine(v) || any_fine(w);
          }
        };
        // one barrier in most tiles; where that finds something, another tells whether references have to
        // move (those tiles have fine weights in any case: to ask again would take one more)
        const bool first = t == it.t_begin, ask = !first && asks();
        const bool over = fmaxf(fmax3(m4.x, m4.y, m4.z), m4.w) > kTop;
        bool fine = !first && soft_or<kN>(ask || over);
        const bool move = first || (fine && soft_or<kN>(over));
        if (move) {
          // ---- set or move the references ---------------------------------------------------
          wait<kN>(s, B_PE + pb, ((n / C::kPBufs) + 1) & 1, p);          // this P^T (xm) is free
          float* xm = reinterpret_cast<float*>(s.ptr + C::kOffP + pb * 2 * C::kPHalf);   // [4][kN]
          over_keys(m4, [](float a, float b) { return fmaxf(a, b); }, xm + kq * kN);
          soft_sync<kN>();
          if (st < kN) {
            const float x0 = xm[st], x1 = xm[kN + st], x2 = xm[2 * kN + st], x3 = xm[3 * kN + st];
            const float m = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)), rest = fmaxf(fminf(x0, x1), fminf(x2, x3));
            const bool one = it.t_end - it.t_begin == 1;
            float by = 0.f;
            if (m != -INFINITY && (first || m > kMove))
              by = (one ? kAlone : rest == -INFINITY ? kPlace : fminf(fmaxf(kPlace, kRest + (m - rest)), kAlone)) - m;
            shift[st] = by;
            factor[st] = first ? 1.f : fast_exp2(by);   // (a first reference may lie far down: 0 * inf)
            row_nm[st] += by;
          }
          soft_sync<kN>();
          const float4 by = of_rows(shift);
          nm4 = of_rows(row_nm);
          const float4 f4 = of_rows(factor);
          const uint64_t b01 = f32x2(f4.x, f4.y), b23 = f32x2(f4.z, f4.w);
          l01 = mul2(l01, b01);
          l23 = mul2(l23, b23);
          w01 = mul2(w01, b01);
          w23 = mul2(w23, b23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i][0] += by.x;
            y[i][1] += by.y;
            y[i][2] += by.z;
            y[i][3] += by.w;
          }
          if (first) {
            m4 = make_float4(m4.x + by.x, m4.y + by.y, m4.z + by.z, m4.w + by.w);
            fine = soft_or<kN>(asks());
          }
        }
        if (st == 0) reinterpret_cast<int*>(s.ptr + C::kOffFine)[n % kFineRing] = fine;
        // ---- weights, their sums, and their two 8-bit parts ------------------------------------
        // In half precision (11 bits): h = the value rounded to e5m2, that is to its upper byte;
        // the residue is exact, and goes to e4m3 or (fine) e5m2, with a dither of up to half of that
        // type's smallest step (0 stays 0).  The e4m3 residue's is added in half precision;
        // the e5m2 residue's, whose step is 2^8 of half precision's last, to the weight before, which
        // is then cut to half precision, so that this rounding does not move the sum either.
        uint32_t ph[4], pl[4];
        auto weights = [&](auto is_fine) {
          const uint32_t key0 = (uint32_t)(t * kTile + my_keys);
          // 16-bit multiples of 2^16 / the golden ratio for the keys of a pair (a carry between them
          // is one of 2^16)
          const uint32_t pair = (key0 * (kTurn >> 16) & 0xffffu) * 0x10001u + (C::kQTmem ? kTurn & 0xffff0000u : 0u);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint64_t s01 = 0, s23 = 0;
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2; ++i) {
              float e0 = fast_exp2(y[i][0]), e1 = fast_exp2(y[i][1]);
              float e2 = fast_exp2(y[i][2]), e3 = fast_exp2(y[i][3]);
              s01 = add2(s01, f32x2(e0, e1));
              s23 = add2(s23, f32x2(e2, e3));
              if constexpr (is_fine) {
                const float da = dither_of((key0 + 8 * i) * kTurn);
                const float db = C::kQTmem ? dither_of((key0 + 8 * i + 1) * kTurn) : da;
                e0 += da;
                e1 += db;
                e2 += da;
                e3 += db;
              }
              const uint32_t u = is_fine ? half2_cut(e0, e1) : half2_of(e0, e1);
              const uint32_t v = is_fine ? half2_cut(e2, e3) : half2_of(e2, e3);
              const uint32_t hu = (u + 0x00800080u) & 0xff00ff00u, hv = (v + 0x00800080u) & 0xff00ff00u;
              const uint32_t ru = sub_half2(u, hu), rv = sub_half2(v, hv);
              ph[i] = __byte_perm(hu, hv, 0x7531);
              if constexpr (is_fine) {
                // (a residue of minus half a step, from a weight of half a step, stays: + 0x7f)
                pl[i] = __byte_perm(ru + 0x007f007fu, rv + 0x007f007fu, 0x7531);
              } else {
                const uint32_t d = dither2_of(pair + i * (8 * (kTurn >> 16) & 0xffffu) * 0x10001u,
                                              C::kQTmem ? kDown | kUp << 16 : (i & 1 ? kUp : kDown) * 0x10001u);
                pl[i] = __byte_perm(e4m3x2_of_half2(add_half2(ru, d)), e4m3x2_of_half2(add_half2(rv, d)), 0x5410);
              }
            }
            const uint64_t ij = f32x2(inv_g[j], inv_g[j]);
            l01 = fma2(s01, ij, l01);
            l23 = fma2(s23, ij, l23);
            w01 = add2(w01, s01);
            w23 = add2(w23, s23);
          }
        };
        if (fine)
          weights(std::true_type{});
        else
          weights(std::false_type{});
        if (!move) wait<kN>(s, B_PE + pb, ((n / C::kPBufs) + 1) & 1, p);
        {
          // lane l gives the address of key 32 kq + l's 16 bytes rg
          const uint32_t dst = s.base + C::kOffP + pb * 2 * C::kPHalf + key * kN +
                               16 * (rg ^ (kN == 64 ? (key >> 1) & 3 : (key >> 2) & 1));
          if constexpr (C::kQTmem) {
            stmatrix_t_x4(dst, ph);
            stmatrix_t_x4(dst + C::kPHalf, pl);
          } else {
            stmatrix_x4(dst, ph);
            stmatrix_x4(dst + C::kPHalf, pl);
          }
        }
        if (t * kTile + kq * 32 + 32 > all_see) {
          // a weight of 0 does not keep a NaN out of O (0 * NaN): behind the request's last key,
          // where slots may hold anything, a key's values become 0; a key that only some
          // rows see loses its NaN (the rows that see it have a NaN score, so their whole
          // output is NaN in any case).  Four keys a time, eight lanes to a key's 128 bytes of a
          // chunk; the four chunks are shared out to the groups of rows.
          constexpr int kShare = 64 / kN;
          const int k0 = t * kTile + kq * 32;      // of the warp's 32 keys: those before `some` are
          const int some = max(all_see - k0, 0), gone = max(it.keys - k0, 0);   // seen by every row
#pragma unroll 1
          for (int c = 0; c < kShare; ++c) {
            const uint32_t vs = (4 * n + kShare * rg + c) % C::kSlots;
            uint4* row = reinterpret_cast<uint4*>(s.ptr + C::kOffK + vs * kChunkBytes + kq * 32 * 128) + (lane & 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 4 * i + (lane >> 3);
              if (k >= gone) row[8 * k] = make_uint4(0, 0, 0, 0);
            }
            for (int k = some + (lane >> 3); k < min(gone, 32); k += 4) {
              uint4 v = row[8 * k];
              v.x &= ~__vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu);
              v.y &= ~__vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
              v.z &= ~__vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu);
              v.w &= ~__vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
              row[8 * k] = v;
            }
          }
        }
        if (move && !first) {
          // ---- O^T (columns are rows; 64 of them a warp) moves with the references: nothing may
          // write to it meanwhile, so after the PV before, which has run since S was read --------
          wait<kN>(s, B_PE + (n - 1) % C::kPBufs, ((n - 1) / C::kPBufs) & 1, p);
          tc_fence_after();
#pragma unroll 1
          for (int c32 = 0; c32 < 2; ++c32) {
            const uint32_t col = (uint32_t)(part * 64 + c32 * 32);
            if (!__any_sync(0xffffffffu, shift[col % kN + lane] != 0.f)) continue;
            uint32_t v[32];
            tmem_ld32(tmem + lane_off + col, v);
            tmem_wait_ld();
            const float4* by = reinterpret_cast<const float4*>(factor + col % kN);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 f = by[k];
              v[4 * k] = __float_as_uint(__uint_as_float(v[4 * k]) * f.x);
              v[4 * k + 1] = __float_as_uint(__uint_as_float(v[4 * k + 1]) * f.y);
              v[4 * k + 2] = __float_as_uint(__uint_as_float(v[4 * k + 2]) * f.z);
              v[4 * k + 3] = __float_as_uint(__uint_as_float(v[4 * k + 3]) * f.w);
            }
            tmem_st32(tmem + lane_off + col, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar<kN>(s, B_PF + pb));
      }

      out_b = it.b;
      out_single = it.single != 0;
      out_part = it.t_begin == 0 ? 1 : 0;
      if (st < kN) out_nm = row_nm[st];            // written by this thread
      pending = true;
      // (all of them go on together, also when a wait of some gave up)
      have = !soft_or<kN>(!take_segment<kN>(s, nseg++, p, it) || *s.abort != 0);
    }
  }

  // ---- teardown ----------------------------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merges the partials of units cut between blocks; a unit with no key gets out = 0, lse = -inf.
// comb_blocks blocks a unit, comb_warps warps a row, which share its partials.  The unit's first
// holder wrote its slot 1, the others, which continue the unit, their slot 0.
// (kMany: more than one warp a row.  Then a warp loads four partials at a time, which takes 80
// registers; with one warp a row and few partials that cost 2 us of 50 in fewer resident blocks.)
template <int kN, bool kMany>
__global__ void __launch_bounds__(256) mla_q8_combine_kernel(const Params p) {
  __shared__ int s_nt;
  __shared__ int2 s_m;
  __shared__ unsigned int s_T;
  extern __shared__ float s_part[];                 // [8][kDv] sums and [8] (kMany)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int u = blockIdx.x / p.comb_blocks, rb = blockIdx.x - u * p.comb_blocks;
  const int b = (int)fdiv((unsigned)u, p.div_rt), rt = u - b * p.row_tiles;
  const int rows = kN / p.comb_blocks;              // the block's, from rb * rows on
  if (rt * kN + rb * rows >= p.rows) return;        // rows of no request
  if (threadIdx.x == 0) {
    if (rt == 0 && rb == 0 && __ldg(p.seq_lens + b) > p.max_blocks * p.bs)
      atomicOr(p.status, MLA_STATUS_SEQ_TOO_LONG);
    s_nt = tiles_of(unit_keys<kN>(p, lens_of(p, b), rt));
  } else if (threadIdx.x == 32) {
    // (three threads, so that the loads do not wait for one another)
    int2 m = make_int2(0, 0);
    if (!p.whole_units) {
      m = p.meta[u];
      // inside [0, groups) whatever a decode that gave up early left there; not set for no keys
      m.x = min(max(m.x, 0), p.groups - 1);
      m.y = min(max(m.y, m.x), p.groups - 1);
    }
    s_m = m;
  } else if (threadIdx.x == 64) {
    s_T = p.whole_units ? 0u : p.hdr[0];
  }
  __syncthreads();
  const int2 m = s_m;
  const bool empty = s_nt == 0;
  if (!empty && m.x == m.y) return;                 // one block wrote the result
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = kMany ? p.comb_warps : 1, at_once = 8 / W, mine = warp % W;
  const unsigned int T = s_T;
  auto holds = [&](int g) { return range_start(p, T, g) < range_start(p, T, g + 1); };
  for (int r0 = 0; r0 < rows; r0 += at_once) {
    const int r = rb * rows + r0 + warp / W, row = rt * kN + r;
    const bool valid = row < p.rows;
    const long long grow = (long long)b * p.rows + row;
    uint16_t* o = p.out + grow * kDv;
    if (empty) {
      if (valid && mine == 0) {
        *reinterpret_cast<uint4*>(o + 8 * lane) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(o + 256 + 8 * lane) = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr && lane == 0) p.lse[grow] = -INFINITY;
      }
      continue;
    }
    auto slot_of = [&](int g) { return (2ll * (g * p.row_tiles + rt) + (g == m.x ? 1 : 0)) * kN + r; };
    float mx = -INFINITY;
    bool nan = false;
    for (int g0 = m.x; g0 <= m.y; g0 += 32) {
      const int g = g0 + lane;
      if (valid && g <= m.y && holds(g)) {
        const float l = p.ws_lse[slot_of(g)].x;
        nan |= l != l;
        mx = fmaxf(mx, l);
      }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if (__any_sync(0xffffffffu, nan)) mx = __int_as_float(0x7fc00000);
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
    float wsum = 0.f;
    if (mx != -INFINITY) {
      for (int g0 = m.x; g0 <= m.y; g0 += 32) {
        const int g = g0 + lane;
        float2 lw = make_float2(-INFINITY, 0.f);
        if (g <= m.y && holds(g)) lw = p.ws_lse[slot_of(g)];
        const float wl = exp2f(lw.x - mx), fl = wl * lw.y;
        const int nh = min(32, m.y - g0 + 1);
        constexpr int kAhead = kMany ? 4 : 1;       // partials whose loads are in flight together
        for (int k0 = mine; k0 < nh; k0 += kAhead * W) {
          float f[kAhead];
          uint4 v[kAhead][2];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int k = min(k0 + i * W, 31);
            const float w = __shfl_sync(0xffffffffu, wl, k);
            f[i] = __shfl_sync(0xffffffffu, fl, k);
            // (what has no weight is not read: nothing there, or nothing that counts)
            const bool use = k0 + i * W < nh && w != 0.f;
            const uint4* src = reinterpret_cast<const uint4*>(p.ws_o + slot_of(g0 + k) * kDv) + lane;
            if (use) wsum += w;
#pragma unroll
            for (int j = 0; j < 2; ++j) v[i][j] = use ? __ldcs(src + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
            if (!use) f[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t x[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
                acc[8 * j + 2 * e] = fmaf(f[i], t.x, acc[8 * j + 2 * e]);
                acc[8 * j + 2 * e + 1] = fmaf(f[i], t.y, acc[8 * j + 2 * e + 1]);
              }
            }
        }
      }
    }
    if constexpr (kMany) {
      // lane l has dims 8 l .. + 7 and 256 further; in shared memory as four words for each lane, so
      // that a warp's access is 512 consecutive bytes
      float4* to = reinterpret_cast<float4*>(s_part + warp * kDv) + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        to[32 * k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
      if (lane == 0) s_part[8 * kDv + warp] = wsum;
      __syncthreads();
      if (mine == 0) {
        for (int q = 1; q < W; ++q) {
          const float4* from = reinterpret_cast<const float4*>(s_part + (warp + q) * kDv) + lane;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 a = from[32 * k];
            acc[4 * k] += a.x;
            acc[4 * k + 1] += a.y;
            acc[4 * k + 2] += a.z;
            acc[4 * k + 3] += a.w;
          }
          wsum += s_part[8 * kDv + warp + q];
        }
      }
      __syncthreads();
    }
    if (mine != 0 || !valid) continue;
    const float inv = mx == -INFINITY ? 0.f : 1.f / wsum;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[8 * j + 2 * e] * inv, acc[8 * j + 2 * e + 1] * inv);
        w4[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(o + 256 * j + 8 * lane) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
    }
    if (p.lse != nullptr && lane == 0)
      p.lse[grow] = mx == -INFINITY ? -INFINITY : (mx + log2f(wsum)) * p.lse_mul;
  }
}

// ---- host ---------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 lookup_encoder() {
  cudaDriverEntryPointQueryResult q;
  void* f = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
          cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  return nullptr;
}
PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = lookup_encoder();
  return fn;
}

// Rows per unit: 32 or 64.  A tile costs a unit of 32 rows 0.8 of what it costs one of 64, so
// two of them take 1.6 times as long, but their start (Q, first loads) and output are 3 to 4 us
// shorter.  32 where a request has no more rows, and where full tables would give a block fewer
// than 5 tiles in units of 64 (units of 32 / 64, 8 x 128 rows of 1,024 keys 14.8 / 17.3 us, of
// 4,096 21.5 / 21.4, of 8,192 29.9 / 27.9; 64 x 128 of 512 25.6 / 26.4, of 1,024 35.4 / 33.5;
// 1 x 128 of 8,192 15.6 / 18.7; 16 x 80 of 1,024 17.8 / 19.3, of 16,384 72.7 / 60.7); else 64.
int rows_per_unit(long long B, long long rows, long long max_keys, int num_sms) {
  if (rows <= 32) return 32;
  if ((rows + 31) / 32 > num_sms) return 64;
  return B * ((rows + 63) / 64) * ((max_keys + kTile - 1) / kTile) < 5LL * num_sms ? 32 : 64;
}
int rows_per_unit(const DecodeArgs& a) {
  return rows_per_unit(a.B, (long long)a.H * a.q_len, (long long)a.max_blocks * a.block_size, a.num_sms);
}

size_t ws_bytes(size_t units, int blocks, int kN) {
  size_t b = 256;                                                    // header
  b += (units * sizeof(int2) + 255) / 256 * 256;
  b += (2 * (size_t)blocks * kN * sizeof(float2) + 255) / 256 * 256;
  return b + 2 * (size_t)blocks * kN * kDv * sizeof(uint16_t);
}

struct Q8Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
constexpr int kMaxDevices = 64;
Q8Device g_q8_dev[kMaxDevices];

void device_setup(Q8Device& d) {
  d.err = cudaFuncSetAttribute(mla_decode_q8_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Cfg<32>::kSmem);
  if (d.err == cudaSuccess)
    d.err = cudaFuncSetAttribute(mla_decode_q8_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<64>::kSmem);
}

template <int kN>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& rmap, const Params& p, int blocks,
                   cudaStream_t stream) {
  DependentLaunch dk(dim3((unsigned)blocks), dim3(Cfg<kN>::kThreads), stream);
  dk.cfg.dynamicSmemBytes = Cfg<kN>::kSmem;
  const cudaError_t e = cudaLaunchKernelEx(&dk.cfg, mla_decode_q8_kernel<kN>, kmap, rmap, p);
  if (e != cudaSuccess) return e;
  DependentLaunch dl(dim3((unsigned)p.units * (unsigned)p.comb_blocks), dim3(256), stream);
  if (p.comb_warps == 1) return cudaLaunchKernelEx(&dl.cfg, mla_q8_combine_kernel<kN, false>, p);
  dl.cfg.dynamicSmemBytes = 8 * (kDv + 1) * sizeof(float);
  return cudaLaunchKernelEx(&dl.cfg, mla_q8_combine_kernel<kN, true>, p);
}

}  // namespace

const char* q8_limit(const DecodeArgs& a) {
  const int rows = a.H * a.q_len, n = rows_per_unit(a);
  const long long tiles = (rows + n - 1) / n;
  // a block for every row tile of a request
  if (tiles > a.num_sms) return "ceil(q_len*H / 64) row tiles of a request are more than the SMs";
  // token and cache row numbers, with the look-ahead of the page window, fit 32 bits
  if ((long long)a.num_blocks * a.block_size >= (1LL << 31) - 65536)
    return "num_blocks*block_size must stay below 2^31 - 65536";
  if ((long long)a.max_blocks * a.block_size >= (1LL << 31) - 65536)
    return "max_blocks*block_size must stay below 2^31 - 65536";
  if (a.B * tiles > 0x7fffffffLL / 8) return "requests (of all shards) times row tiles must stay below 2^28";
  // the split line, were every request as long as its table
  if (a.B * ((long long)a.max_blocks * a.block_size / kTile + 1 + Cfg<32>::kSegTiles) >= (1LL << 31))
    return "requests (of all shards) times (max_blocks*block_size / 128 + 7) must stay below 2^31";
  return nullptr;
}

bool q8_driver_ok() { return get_encoder() != nullptr; }

size_t q8_workspace_size(int B, int H, int q_len, int num_sms) {
  const long long rows = (long long)H * q_len;
  const size_t a = ws_bytes((size_t)B * ((rows + 31) / 32), num_sms, 32);
  if (rows <= 32) return a;
  return std::max(a, ws_bytes((size_t)B * ((rows + 63) / 64), num_sms, 64));   // whichever a call takes
}

cudaError_t launch_decode_q8(const DecodeArgs& a, cudaStream_t stream) {
  Params p;
  p.q = a.q;
  p.scales = a.kv_scales;
  p.bt = a.block_table;
  p.bt_stride = a.bt_stride;
  p.seq_lens = a.seq_lens;
  p.gseq = a.gseq;
  p.B = a.B;
  p.H = a.H;
  p.q_len = a.q_len;
  p.bs = a.block_size;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.rank = a.cp_rank;
  p.causal = a.causal ? 1 : 0;
  p.il = a.interleave;
  p.span = a.cp_world * a.interleave;
  p.wait_ns = a.wait_ns;
  p.stall_test = a.stall_test;
  p.shard_B = a.shard_B;
  p.shard_mul = a.shard_B == a.B ? 0u
                                 : (unsigned)((0x100000000ull + (unsigned long long)a.shard_B - 1) /
                                              (unsigned long long)a.shard_B);
  p.rows = a.H * a.q_len;
  const int n = rows_per_unit(a);
  p.row_tiles = (p.rows + n - 1) / n;
  p.units = a.B * p.row_tiles;
  p.box_rows = a.block_size % 128 == 0 ? 128 : a.block_size % 64 == 0 ? 64 : a.block_size % 32 == 0 ? 32 : 16;
  p.div_bs = make_fastdiv((unsigned)a.block_size);
  p.tile_pages = kTile / a.block_size;
  p.tile_rest = kTile % a.block_size;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.lse_mul = a.lse_base_e ? 0.6931471805599453f : 1.0f;
  p.out = a.out;
  p.lse = a.lse;
  p.status = a.status;
  p.seg_tiles = n == 32 ? Cfg<32>::kSegTiles : Cfg<64>::kSegTiles;

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  Q8Device& qd = g_q8_dev[dev];
  std::call_once(qd.once, device_setup, std::ref(qd));
  if (qd.err != cudaSuccess) return qd.err;

  p.groups = a.num_sms / p.row_tiles;
  if (a.workspace != nullptr && a.workspace_bytes >= ws_bytes(p.units, a.num_sms, n)) {
    char* ws = static_cast<char*>(a.workspace);
    p.hdr = reinterpret_cast<unsigned int*>(ws);
    ws += 256;
    p.meta = reinterpret_cast<int2*>(ws);
    ws += ((size_t)p.units * sizeof(int2) + 255) / 256 * 256;
    p.ws_lse = reinterpret_cast<float2*>(ws);
    ws += (2 * (size_t)a.num_sms * n * sizeof(float2) + 255) / 256 * 256;
    p.ws_o = reinterpret_cast<uint16_t*>(ws);
    p.whole_units = 0;
  } else {
    p.hdr = nullptr;
    p.meta = nullptr;
    p.ws_lse = nullptr;
    p.ws_o = nullptr;
    p.whole_units = 1;
    if (p.groups > a.B) p.groups = a.B;
  }
  const int blocks = p.groups * p.row_tiles;
  // The combine: a unit has about groups / B partials.  Enough warps a row that each has few of
  // them, and as many blocks as give every row its warps, but not many more than can be resident
  // at once (most units have nothing to merge, and a block's start is all they cost).
  const int parts = p.whole_units ? 1 : p.groups / a.B;
  p.comb_warps = parts >= 24 ? 8 : parts >= 12 ? 4 : parts >= 6 ? 2 : 1;
  p.comb_blocks = n * p.comb_warps / 8;
  while (p.comb_blocks > 1 && (long long)p.units * p.comb_blocks > 16LL * a.num_sms) p.comb_blocks /= 2;
  p.div_H = make_fastdiv((unsigned)a.H);
  p.div_span = make_fastdiv((unsigned)p.span);
  p.div_rt = make_fastdiv((unsigned)p.row_tiles);
  p.div_groups = make_fastdiv((unsigned)p.groups);

  // the cache as rows of 576 bytes: boxes of 128 latent bytes (x = 0, 128, 256, 384; 128-byte
  // swizzle) and of the 64 rope bytes (x = 512; 64-byte swizzle)
  CUtensorMap kmap, rmap;
  cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)a.num_blocks * a.block_size};
  cuuint64_t strides[1] = {(cuuint64_t)kD};
  cuuint32_t es[2] = {1, 1};
  for (int i = 0; i < 2; ++i) {
    cuuint32_t box[2] = {i == 0 ? 128u : 64u, (cuuint32_t)p.box_rows};
    const CUresult r = get_encoder()(
        i == 0 ? &kmap : &rmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint16_t*>(a.kv), dims, strides,
        box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
        i == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return n == 32 ? launch<32>(kmap, rmap, p, blocks, stream) : launch<64>(kmap, rmap, p, blocks, stream);
}

}  // namespace mla
