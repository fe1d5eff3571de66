// The DCP slot mapping of one position, shared by the kernels that map, scatter and append.
#pragma once

#include "internal.h"
#include "../../include/mla_decode.h"

namespace mla {

struct SlotParams {
  const int32_t* block_table;
  int64_t bt_stride;
  int max_blocks, block_size, cp_size, cp_rank, interleave;
  unsigned int vbs;          // block_size * cp_size (checked < 2^31 on the host)
  FastDiv div_vbs, div_il, div_cp;
  unsigned int* status;
};

__device__ __forceinline__ unsigned int fdiv(unsigned int n, const FastDiv& f) {
  return f.d == 1u ? n : (unsigned int)__umul64hi(f.m, (unsigned long long)n);
}

// Where `pos` lies if this rank owns it: the page that the table names and the offset in it.
// False if another rank owns it, the position is negative, or its virtual block lies past the
// table (then `bad` is set and the table is not read).
__device__ __forceinline__ bool locate(long long pos, int b, const SlotParams& p, bool& bad,
                                       int& page, unsigned int& local) {
  if (pos < 0) return false;
  long long vb;
  unsigned int off;
  if (pos <= 0xffffffffLL) {
    const unsigned int q = fdiv((unsigned int)pos, p.div_vbs);
    vb = q;
    off = (unsigned int)pos - q * p.vbs;
  } else {
    vb = pos / p.vbs;
    off = (unsigned int)(pos - vb * p.vbs);
  }
  if (vb >= p.max_blocks) {
    bad = true;
    return false;
  }
  if (p.cp_size == 1) {
    local = off;
  } else {
    // segment of `interleave` positions, its owner (segment mod cp) and its round
    const unsigned int seg = fdiv(off, p.div_il);
    const unsigned int rin = off - seg * (unsigned int)p.interleave;
    const unsigned int rnd = fdiv(seg, p.div_cp);
    if ((int)(seg - rnd * (unsigned int)p.cp_size) != p.cp_rank) return false;
    local = rnd * (unsigned int)p.interleave + rin;
  }
  page = __ldg(p.block_table + (long long)b * p.bt_stride + vb);
  return true;
}

// Slot of `pos` on this rank, or MLA_PAD_SLOT_ID if it has none (see locate).
__device__ __forceinline__ long long map_one(long long pos, int b, const SlotParams& p,
                                             bool& bad) {
  int page;
  unsigned int local;
  if (!locate(pos, b, p, bad, page, local)) return MLA_PAD_SLOT_ID;
  return (long long)page * p.block_size + local;
}

inline SlotParams make_slot_params(const int32_t* block_table, int64_t bt_stride, int max_blocks,
                       int block_size, int cp_size, int cp_rank, int interleave,
                       unsigned int* status) {
  SlotParams p;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.max_blocks = max_blocks;
  p.block_size = block_size;
  p.cp_size = cp_size;
  p.cp_rank = cp_rank;
  p.interleave = interleave;
  p.vbs = (unsigned int)block_size * (unsigned int)cp_size;
  p.div_vbs = make_fastdiv(p.vbs);
  p.div_il = make_fastdiv((unsigned int)interleave);
  p.div_cp = make_fastdiv((unsigned int)cp_size);
  p.status = status;
  return p;
}

}  // namespace mla
