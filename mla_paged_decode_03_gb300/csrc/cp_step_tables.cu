// cp_step_tables: a serving step's tables from request lengths (pages taken from and given
// back to a ring, block-table entries, global and shard-local lengths, positions, slots).
//
// Definition: the header's formulas; the page of a position is block_table[pos //
// (block_size * CP_SIZE)] and its slot cp_local_slot's ("vLLM PR #52188 (DSpark + DCP)"
// page, sections "关键源码片段" and "实现拆解" step 4).  Integer work, bit-exact.
//
// One launch.  Which pages a request takes depends on the requests before it through two
// prefix sums (pages taken, which decides who is granted; then pages given back).  Every
// block computes them by itself over the requests up to its own (12 bytes a request, from L2
// after the first block), so that no block waits for another and no scratch is needed:
// inputs and outputs are disjoint, pops read ring entries [head, head + count) and pushes
// write entries behind them.  A block then serves a tile of `tile` positions: whole requests
// when a request's N positions fit, else one request's next `tile` positions.
//
// Bound: the launch and the chain lengths -> scan -> table or ring -> slot of dependent L2
// accesses (8 requests, a token each: 3.2 us; 256 requests of 4 tokens on 8 ranks, 32 of them
// finished: 5.5; 32 prompts of up to 8,192: 7.0 for 4.2 MB of positions and slots, 0.6 at
// the copy rate).
#include <cuda_runtime.h>

#include "internal.h"
#include "../../include/mla_decode.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxReq = 256;             // requests per block
constexpr int kMaxTile = 2048;           // positions per block

struct Params {
  const int32_t *prev, *ctx, *fresh;
  int B, N;
  int32_t* table;
  long long bt_stride;
  int max_blocks;
  int32_t* ring;
  int cap;
  const int32_t* state;
  int32_t* state_out;
  unsigned int vbs;                      // block_size * cp_size
  int block_size, cp_size, cp_rank, n_ranks, il;
  FastDiv div_vbs, div_n, div_il, div_cp, div_span, div_req;
  int32_t *total, *seq;
  long long *positions, *slots;
  int req;                               // requests per block (1 when chunks > 1)
  int chunks;                            // blocks per request
  int tile;
  unsigned int* status;
};

__device__ __forceinline__ unsigned int fdiv(unsigned int n, const FastDiv& f) {
  return f.d == 1u ? n : (unsigned int)__umul64hi(f.m, (unsigned long long)n);
}

// What phase 2 needs of a request.
struct Req {
  int ctx, fresh, total; // cached tokens; new tokens (0 when not granted); length after the step
  int held, keep, take;  // pages held before, kept, taken
  int take0, give0;      // pages taken / given back by the requests before
};

// Inclusive prefix sum over the block; `total` receives the block's sum.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp,
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  unsigned long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  __syncthreads();
  return v + before;
}

__global__ void __launch_bounds__(kThreads) cp_step_tables_kernel(const Params p) {
  __shared__ Req s_req[kMaxReq];
  __shared__ unsigned long long s_warp[kWarps];
  const int tid = threadIdx.x;
  const int first = p.chunks > 1 ? blockIdx.x / p.chunks : blockIdx.x * p.req;
  const int chunk = p.chunks > 1 ? blockIdx.x - first * p.chunks : 0;
  const int last = min(first + p.req, p.B);          // this block's requests [first, last)
  unsigned int flags = 0;

  int head = p.state[0], count = p.state[1];
  if (head < 0 || head >= p.cap || count < 0 || count > p.cap) {
    head = 0;
    count = 0;
    if (blockIdx.x == 0) flags |= MLA_STATUS_BAD_STEP;
  }

  // ---- phase 1: the prefix sums, up to this block's requests (block 0: over all, for the
  // ring's new state).  In most steps of a decode loop no request of a round of 256 takes or gives
  // a page, and the sums are skipped. ---------------------------------------------------------
  unsigned long long asked = 0, moved = 0;           // by the requests before these 256: asked for; given, taken
  const int upto = blockIdx.x == 0 ? p.B : last;
  for (int base = 0; base < upto; base += kThreads) {
    const int b = base + tid;
    bool fits = true, bad = false;
    int held = 0, prev = 0, ctx = 0, fresh = 0, take = 0;
    if (b < upto) {
      prev = __ldg(p.prev + b);
      ctx = __ldg(p.ctx + b);
      fresh = __ldg(p.fresh + b);
      bad = prev < 0 || ctx < 0 || fresh < 0 || fresh > p.N;
      prev = max(prev, 0);
      ctx = max(ctx, 0);
      fresh = min(max(fresh, 0), p.N);
      unsigned int hp = fdiv((unsigned int)prev + p.vbs - 1u, p.div_vbs);
      if (hp > (unsigned int)p.max_blocks) {
        hp = p.max_blocks;
        bad = true;
      }
      held = (int)hp;
      const long long len = (long long)ctx + fresh;
      fits = len <= 0x7fffffffLL;
      if (fits) {
        const unsigned int want = fdiv((unsigned int)len + p.vbs - 1u, p.div_vbs);
        fits = want <= (unsigned int)p.max_blocks;
        if (fits) take = max((int)want - held, 0);
      }
    }
    bool granted = fits;
    unsigned long long asked0 = asked;               // asked for by the requests before b
    if (__syncthreads_or(take > 0)) {
      unsigned long long sum;
      const unsigned long long incl = asked + block_scan((unsigned long long)take, s_warp, sum);
      granted = fits && (take == 0 || incl <= (unsigned long long)count);
      asked0 = incl - take;
      asked += sum;
    }
    const int total = granted ? ctx + fresh : min(ctx, prev);
    const int keep = min((int)fdiv((unsigned int)total + p.vbs - 1u, p.div_vbs), p.max_blocks);
    const int give = max(held - keep, 0);
    // pages given (upper half) and taken (lower): neither exceeds the ring in consistent tables
    const unsigned long long mine = (unsigned long long)give << 32 | (unsigned)(granted ? take : 0);
    unsigned long long moved0 = moved;
    if (__syncthreads_or(mine != 0)) {
      unsigned long long sum;
      moved0 += block_scan(mine, s_warp, sum) - mine;
      moved += sum;
    }
    if (b >= first && b < last) {
      Req r;
      const unsigned int give0 = (unsigned int)(moved0 >> 32);
      r.ctx = ctx;
      r.fresh = granted ? fresh : 0;
      r.held = held;
      r.keep = keep;
      r.take = granted ? take : 0;
      r.take0 = (int)min(asked0, (unsigned long long)p.cap);
      r.give0 = (int)min(give0, (unsigned int)p.cap);
      r.total = total;
      s_req[b - first] = r;
      if (chunk == 0) {
        if (bad) flags |= MLA_STATUS_BAD_STEP;
        if (!fits) flags |= MLA_STATUS_SEQ_TOO_LONG;
        if (fits && !granted) flags |= MLA_STATUS_OUT_OF_PAGES;
        if (give > 0 && (unsigned long long)give0 + give > (unsigned long long)(p.cap - count))
          flags |= MLA_STATUS_BAD_STEP;
        p.total[b] = total;
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    // pages that a full ring cannot hold were dropped (below)
    const unsigned int taken = (unsigned int)moved, given = (unsigned int)(moved >> 32);
    const unsigned int h = (unsigned int)head + taken;
    p.state_out[0] = (int)(h >= (unsigned int)p.cap ? h - p.cap : h);
    p.state_out[1] = count - (int)taken + (int)min(given, (unsigned int)(p.cap - count));
  }
  __syncthreads();

  // ---- phase 2: shard-local lengths ---------------------------------------------------
  if (p.seq != nullptr && chunk == 0) {
    const int reqs = last - first;
    for (int k = tid; k < reqs * p.n_ranks; k += kThreads) {
      // (whole blocks of requests have p.req of them; the last may have fewer)
      const int rk = reqs == p.req ? (int)fdiv((unsigned int)k, p.div_req) : k / reqs, i = k - rk * reqs;
      const int total = s_req[i].total;
      const int q = (int)fdiv((unsigned int)total, p.div_span);
      const int over = total - q * (p.cp_size * p.il) - (p.cp_rank + rk) * p.il;
      p.seq[(long long)rk * p.B + first + i] = q * p.il + min(max(over, 0), p.il);
    }
  }

  // ---- phase 2: pages ---------------------------------------------------------------
  auto ring_at = [&](int i) {                        // entry i behind the head, i < cap
    const unsigned int x = (unsigned int)head + (unsigned int)i;
    return x >= (unsigned int)p.cap ? x - p.cap : x;
  };
  {
    const int lane = tid & 31, warp = tid >> 5;
    // one request: the whole block (and the request's other blocks) stride over its pages;
    // several: a warp each
    const bool one = p.req == 1;
    for (int i = one ? 0 : warp; i < last - first; i += one ? 1 : kWarps) {
      const Req r = s_req[i];
      int32_t* row = p.table + (long long)(first + i) * p.bt_stride;
      const long long k0 = one ? (long long)chunk * kThreads + tid : lane;
      const long long step = one ? (long long)p.chunks * kThreads : 32;
      // eight pages a thread at a time: the loads of a round do not wait for one another
      constexpr int kAhead = 8;
      for (long long k = k0; k < r.take; k += kAhead * step) {
        int v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + j * step < r.take) v[j] = p.ring[ring_at((int)(r.take0 + k + j * step))];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + j * step < r.take) row[r.held + k + j * step] = v[j];
      }
      // (pages behind a full ring are dropped)
      const int give = min(r.held - r.keep, max(p.cap - count - r.give0, 0));
      for (long long k = k0; k < give; k += kAhead * step) {
        int v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + j * step < give) v[j] = row[r.keep + k + j * step];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + j * step < give) p.ring[ring_at((int)(count + r.give0 + k + j * step))] = v[j];
      }
    }
  }

  // ---- phase 2: positions and slots --------------------------------------------------
  if ((p.positions != nullptr || p.slots != nullptr) && first < p.B) {
    const int n0 = chunk * p.tile;
    const int items = p.chunks > 1 ? min(p.tile, p.N - n0) : (last - first) * p.N;
    const long long bn = (long long)p.B * p.N;
    const long long out0 = (long long)first * p.N + n0;
    for (int k = tid; k < items; k += kThreads) {
      const int i = p.chunks > 1 ? 0 : (int)fdiv((unsigned int)k, p.div_n);
      const int n = p.chunks > 1 ? n0 + k : k - i * p.N;
      const Req& r = s_req[i];
      const bool live = n < r.fresh;
      const unsigned int pos = (unsigned int)(r.ctx + n);
      if (p.positions != nullptr) p.positions[out0 + k] = live ? (long long)pos : -1ll;
      if (p.slots == nullptr) continue;
      long long slot = MLA_PAD_SLOT_ID;
      int owner = -1;
      if (live) {
        const unsigned int vb = fdiv(pos, p.div_vbs);
        const unsigned int off = pos - vb * p.vbs;
        const unsigned int seg = fdiv(off, p.div_il);
        const unsigned int rnd = fdiv(seg, p.div_cp);
        owner = (int)(seg - rnd * (unsigned int)p.cp_size) - p.cp_rank;
        if (owner >= 0 && owner < p.n_ranks) {
          // a page taken in this call is read where it comes from
          const int page = (int)vb < r.held
                               ? p.table[(long long)(first + i) * p.bt_stride + vb]
                               : p.ring[ring_at(r.take0 + (int)vb - r.held)];
          slot = (long long)page * p.block_size + rnd * (unsigned int)p.il +
                 (off - seg * (unsigned int)p.il);
        }
      }
      for (int q = 0; q < p.n_ranks; ++q)
        p.slots[q * bn + out0 + k] = q == owner ? slot : (long long)MLA_PAD_SLOT_ID;
    }
  }
  if (flags != 0u) atomicOr(p.status, flags);
}

}  // namespace

cudaError_t launch_cp_step_tables(const StepArgs& a, cudaStream_t stream) {
  Params p;
  p.prev = a.prev;
  p.ctx = a.ctx;
  p.fresh = a.fresh;
  p.B = a.B;
  p.N = a.N;
  p.table = a.table;
  p.bt_stride = a.bt_stride;
  p.max_blocks = a.max_blocks;
  p.ring = a.ring;
  p.cap = a.cap;
  p.state = a.state;
  p.state_out = a.state_out;
  p.vbs = (unsigned int)a.block_size * (unsigned int)a.cp_size;
  p.block_size = a.block_size;
  p.cp_size = a.cp_size;
  p.cp_rank = a.cp_rank;
  p.n_ranks = a.n_ranks;
  p.il = a.interleave;
  p.div_vbs = make_fastdiv(p.vbs);
  p.div_n = make_fastdiv((unsigned int)(a.N > 0 ? a.N : 1));
  p.div_il = make_fastdiv((unsigned int)a.interleave);
  p.div_cp = make_fastdiv((unsigned int)a.cp_size);
  p.div_span = make_fastdiv((unsigned int)(a.cp_size * a.interleave));
  p.total = a.total;
  p.seq = a.seq;
  p.positions = reinterpret_cast<long long*>(a.positions);
  p.slots = reinterpret_cast<long long*>(a.slots);
  p.status = a.status;
  // tiles of 256 positions (one a thread) until they give four blocks to every SM, then
  // larger ones up to 2,048, so that the repeated prefix sums stay few
  long long tile = ((long long)a.B * a.N / (4LL * a.num_sms) + kThreads - 1) / kThreads * kThreads;
  tile = tile < kThreads ? kThreads : (tile > kMaxTile ? kMaxTile : tile);
  p.tile = (int)tile;
  p.chunks = a.N > tile ? (int)((a.N + tile - 1) / tile) : 1;
  p.req = p.chunks > 1 ? 1 : (a.N > 0 ? (int)(tile / a.N) : kMaxReq);
  if (p.req > kMaxReq) p.req = kMaxReq;
  if (p.req < 1) p.req = 1;
  p.div_req = make_fastdiv((unsigned int)p.req);
  const long long blocks = p.chunks > 1 ? (long long)a.B * p.chunks : ((long long)a.B + p.req - 1) / p.req;
  cp_step_tables_kernel<<<(unsigned)(blocks > 0 ? blocks : 1), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
