// C ABI of libmla_decode.so (declared in include/mla_decode.h): host-side argument
// validation, error reporting and kernel launches.  Nothing here allocates memory.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <functional>
#include <mutex>

#include <cuda_runtime.h>

#include "internal.h"
#include "sm100.cuh"
#include "tma_map.h"
#include "../../include/mla_decode.h"

namespace {

// One status word per device; kernels OR MLA_STATUS_* bits into it.
__device__ unsigned int g_mla_status = 0;

thread_local char t_err[512] = {0};

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_err, sizeof(t_err), fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  t_err[0] = 0;
  return MLA_OK;
}

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  const char* what = "";
  int num_sms = 0;
  unsigned int* status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];

void device_setup(DeviceInfo& d, int dev) {
  int sms = 0;
  d.err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (d.err != cudaSuccess) {
    d.what = "cudaDeviceGetAttribute";
    return;
  }
  void* p = nullptr;
  d.err = cudaGetSymbolAddress(&p, g_mla_status);
  if (d.err != cudaSuccess) {
    d.what = "cudaGetSymbolAddress(status)";
    return;
  }
  d.num_sms = sms;
  d.status = static_cast<unsigned int*>(p);
}

// Resolves the current device's SM count and status-word address (once per device, also
// when several host threads make their first call at the same time).
int device_info(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(MLA_ERR_UNSUPPORTED, "device index %d", dev);
  DeviceInfo& d = g_dev[dev];
  std::call_once(d.once, device_setup, std::ref(d), dev);
  if (d.err != cudaSuccess) return fail(MLA_ERR_CUDA, "%s: %s", d.what, cudaGetErrorString(d.err));
  *out = &d;
  return MLA_OK;
}

// Process-wide settings of the diagnostic entry points.
std::atomic<unsigned long long> g_wait_ns{0};   // 0: the default limit
std::atomic<int> g_stall_test{0};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

namespace mla {
int api_fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_err, sizeof(t_err), fmt, ap);
  va_end(ap);
  return code;
}
}  // namespace mla

extern "C" {

int mla_abi_version(void) { return MLA_ABI_VERSION; }

int mla_set_decode_kernel(int choice) {
  static std::atomic<int> current{0};
  if (choice < 0 || choice > 2)
    return fail(MLA_ERR_INVALID_ARGUMENT, "mla_set_decode_kernel: choice %d not in 0..2", choice);
  mla::set_decode_kernel_choice(choice);
  return current.exchange(choice);
}

int mla_set_rescale_budget(int choice) {
  static std::atomic<int> current{0};
  if (choice < 0 || choice > 2)
    return fail(MLA_ERR_INVALID_ARGUMENT, "mla_set_rescale_budget: choice %d not in 0..2", choice);
  mla::set_rescale_budget_choice(choice);
  return current.exchange(choice);
}

int mla_set_test_stall(int on) {
  if (on != 0 && on != 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "mla_set_test_stall: %d is neither 0 nor 1", on);
  return g_stall_test.exchange(on);
}

int64_t mla_set_wait_limit_ns(int64_t ns) {
  if (ns < 0) return fail(MLA_ERR_INVALID_ARGUMENT, "mla_set_wait_limit_ns: ns=%lld < 0",
                          (long long)ns);
  return (int64_t)g_wait_ns.exchange((unsigned long long)ns);
}

const char* mla_last_error(void) { return t_err; }

size_t mla_decode_workspace_size(int B, int H, int q_len, int num_sms) {
  if (B <= 0 || H <= 0 || q_len <= 0 || num_sms <= 0) return 0;
  return mla::decode_workspace_size(B, H, q_len, num_sms);
}

size_t mla_decode_q8_workspace_size(int B, int H, int q_len, int num_sms) {
  if (B <= 0 || H <= 0 || q_len <= 0 || num_sms <= 0) return 0;
  return mla::q8_workspace_size(B, H, q_len, num_sms);
}

}  // extern "C"

namespace mla {

// Shared by mla_decode (n_shards == 1, the given rank), mla_decode_shards (ranks
// 0 .. n_shards-1 of cp_world == n_shards, shard-major tables and outputs), their forms over
// the 8-bit cache (q8: kv_cache is e4m3 and kv_scales its scales) and mla_decode_noalloc
// (require_full_split: the workspace must hold the scratch of the full split-KV schedule, else
// the call is refused after every other check).
int decode_entry(const char* fn, const void* q, const void* kv_cache, bool q8,
                 const float* kv_scales, const int32_t* block_table, int64_t bt_stride,
                 const int32_t* seq_lens, const int32_t* causal_seqlens_global, int B, int H,
                 int q_len, int causal, int block_size, int num_blocks, int max_blocks,
                 int cp_world, int cp_rank, int interleave, int n_shards, float scale, void* out,
                 float* lse, int lse_base_e, void* workspace, size_t workspace_bytes,
                 bool require_full_split, mla_stream_t stream) {
  if (B < 0) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: B=%d < 0", fn, B);
  if (H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: H=%d < 1", fn, H);
  if (q_len < 1 || q_len > MLA_MAX_Q_LEN)
    return fail(q_len < 1 ? MLA_ERR_INVALID_ARGUMENT : MLA_ERR_UNSUPPORTED,
                "%s: q_len=%d outside [1, %d]", fn, q_len, MLA_MAX_Q_LEN);
  if (block_size < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size < 1", fn);
  if (q8 && block_size % MLA_Q8_GROUP != 0)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size (%d) must be a multiple of %d", fn,
                block_size, MLA_Q8_GROUP);
  if (num_blocks < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: num_blocks < 1", fn);
  if (max_blocks < 1 || bt_stride < max_blocks)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 1 <= max_blocks (%d) <= bt_stride (%lld)",
                fn, max_blocks, (long long)bt_stride);
  if ((long long)max_blocks * block_size > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: max_blocks*block_size exceeds 2^31-1", fn);
  if ((long long)num_blocks * block_size > (1LL << 40))
    return fail(MLA_ERR_UNSUPPORTED, "%s: cache too large", fn);
  if (cp_world < 1 || cp_rank < 0 || cp_rank >= cp_world)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 0 <= cp_rank (%d) < cp_world (%d)", fn,
                cp_rank, cp_world);
  if (interleave < 1 || block_size % interleave != 0)
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: interleave (%d) must be >= 1 and divide block_size (%d)", fn, interleave,
                block_size);
  if ((long long)cp_world * interleave > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: cp_world*interleave exceeds 2^31-1", fn);
  if (!isfinite(scale) || !(scale > 0.f))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: scale must be finite and > 0", fn);
  if (B == 0) return ok();
  if (!q || !kv_cache || !block_table || !seq_lens || !out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null q/kv_cache/block_table/seq_lens/out", fn);
  if (q8 && !kv_scales) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null kv_scales", fn);
  if (causal_seqlens_global == nullptr && cp_world != 1 && causal)
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: causal_seqlens_global is required when cp_world > 1", fn);
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: q, kv_cache and out must be 16-byte aligned", fn);
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      (causal_seqlens_global && !aligned(causal_seqlens_global, 4)) || (lse && !aligned(lse, 4)) ||
      (q8 && !aligned(kv_scales, 4)))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned int32/float argument", fn);
  if (workspace && !aligned(workspace, 256))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  if ((long long)n_shards * B * q_len * H > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: too many query rows", fn);

  DeviceInfo* dev = nullptr;
  int rc = device_info(&dev);
  if (rc != MLA_OK) return rc;

  mla::DecodeArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.kv = static_cast<const uint16_t*>(kv_cache);
  a.kv_scales = q8 ? kv_scales : nullptr;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.gseq = causal_seqlens_global ? causal_seqlens_global : seq_lens;
  a.B = n_shards * B;
  a.shard_B = B;
  a.H = H;
  a.q_len = q_len;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.cp_world = cp_world;
  a.cp_rank = cp_rank;
  a.causal = causal ? 1 : 0;
  a.interleave = interleave;
  const unsigned long long wait_ns = g_wait_ns.load();
  a.wait_ns = wait_ns ? wait_ns : mla::sm100::kDefaultWaitNs;
  a.stall_test = g_stall_test.load();
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.lse_base_e = lse_base_e ? 1 : 0;
  a.workspace = workspace;
  a.workspace_bytes = workspace ? workspace_bytes : 0;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  const mla::DecodeKernel k = mla::choose_decode_kernel(a);
  if (k == mla::kDecodeNone && q8)
    return fail(MLA_ERR_UNSUPPORTED,
                "%s: %s (B=%d%s, q_len*H=%d, max_blocks=%d, num_blocks=%d, block_size=%d, %d SMs)", fn,
                mla::q8_limit(a), a.B, n_shards > 1 ? " over all shards" : "", q_len * H, max_blocks,
                num_blocks, block_size, dev->num_sms);
  if (k == mla::kDecodeQ8 && !mla::q8_driver_ok())
    return fail(MLA_ERR_CUDA, "%s: the CUDA driver has no cuTensorMapEncodeTiled", fn);
  if (k == mla::kDecodeNone)
    return fail(MLA_ERR_UNSUPPORTED,
                "%s: no decode kernel for this layout (block_size %d: the tcgen05 kernel takes "
                "16, 32 or a multiple of 64; q_len*H = %d rows need at most %d row tiles of 128)",
                fn, block_size, q_len * H, dev->num_sms / 2);
  if (require_full_split) {
    const size_t need = mla::decode_workspace_for(n_shards * B, H, q_len, dev->num_sms, block_size);
    if (need > workspace_bytes)
      return fail(MLA_ERR_UNSUPPORTED,
                  "%s: B=%d H=%d q_len=%d needs %zu bytes of split-KV scratch, more than the "
                  "library's fixed %zu; use mla_decode with a caller workspace",
                  fn, B, H, q_len, need, workspace_bytes);
  }
  cudaError_t e = mla::launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

}  // namespace mla

extern "C" {

int mla_decode(const void* q, const void* kv_cache, const int32_t* block_table,
               int64_t bt_stride, const int32_t* seq_lens,
               const int32_t* causal_seqlens_global, int B, int H, int q_len, int causal,
               int block_size, int num_blocks, int max_blocks, int cp_world, int cp_rank,
               int interleave, float scale, void* out, float* lse, int lse_base_e,
               void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  return mla::decode_entry("mla_decode", q, kv_cache, false, nullptr, block_table, bt_stride,
                           seq_lens, causal_seqlens_global, B, H, q_len, causal, block_size,
                           num_blocks, max_blocks, cp_world, cp_rank, interleave, 1, scale, out,
                           lse, lse_base_e, workspace, workspace_bytes, false, stream);
}

int mla_decode_shards(const void* q, const void* kv_cache, const int32_t* block_table,
                      int64_t bt_stride, const int32_t* seq_lens,
                      const int32_t* causal_seqlens_global, int B, int H, int q_len,
                      int causal, int block_size, int num_blocks, int max_blocks, int n_shards,
                      int interleave, float scale, void* out, float* lse, int lse_base_e,
                      void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  if (n_shards < 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "mla_decode_shards: n_shards=%d < 1", n_shards);
  if (n_shards > 1 && B > 0 && (unsigned long long)n_shards * B * B >= (1ull << 32))
    return fail(MLA_ERR_UNSUPPORTED, "mla_decode_shards: n_shards * B^2 must stay below 2^32");
  return mla::decode_entry("mla_decode_shards", q, kv_cache, false, nullptr, block_table,
                           bt_stride, seq_lens, causal_seqlens_global, B, H, q_len, causal,
                           block_size, num_blocks, max_blocks, n_shards, 0, interleave, n_shards,
                           scale, out, lse, lse_base_e, workspace, workspace_bytes, false,
                           stream);
}

int mla_decode_q8(const void* q, const void* kv_cache, const float* kv_scales,
                  const int32_t* block_table, int64_t bt_stride, const int32_t* seq_lens,
                  const int32_t* causal_seqlens_global, int B, int H, int q_len, int causal,
                  int block_size, int num_blocks, int max_blocks, int cp_world, int cp_rank,
                  int interleave, float scale, void* out, float* lse, int lse_base_e,
                  void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  return mla::decode_entry("mla_decode_q8", q, kv_cache, true, kv_scales, block_table, bt_stride,
                           seq_lens, causal_seqlens_global, B, H, q_len, causal, block_size,
                           num_blocks, max_blocks, cp_world, cp_rank, interleave, 1, scale, out,
                           lse, lse_base_e, workspace, workspace_bytes, false, stream);
}

int mla_decode_shards_q8(const void* q, const void* kv_cache, const float* kv_scales,
                         const int32_t* block_table, int64_t bt_stride,
                         const int32_t* seq_lens, const int32_t* causal_seqlens_global, int B,
                         int H, int q_len, int causal, int block_size, int num_blocks,
                         int max_blocks, int n_shards, int interleave, float scale, void* out,
                         float* lse, int lse_base_e, void* workspace, size_t workspace_bytes,
                         mla_stream_t stream) {
  if (n_shards < 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "mla_decode_shards_q8: n_shards=%d < 1", n_shards);
  if (n_shards > 1 && B > 0 && (unsigned long long)n_shards * B * B >= (1ull << 32))
    return fail(MLA_ERR_UNSUPPORTED,
                "mla_decode_shards_q8: n_shards * B^2 must stay below 2^32");
  return mla::decode_entry("mla_decode_shards_q8", q, kv_cache, true, kv_scales, block_table,
                           bt_stride, seq_lens, causal_seqlens_global, B, H, q_len, causal,
                           block_size, num_blocks, max_blocks, n_shards, 0, interleave, n_shards,
                           scale, out, lse, lse_base_e, workspace, workspace_bytes, false,
                           stream);
}

int lse_merge(const void* partials, int partials_fp32, const float* lses, int n_shards,
              int T, int H, void* out, float* out_lse, int lse_base_e, mla_stream_t stream) {
  if (n_shards < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "lse_merge: n_shards=%d < 1", n_shards);
  if (T < 0 || H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "lse_merge: need T >= 0, H >= 1");
  if (T == 0) return ok();
  if (!partials || !lses || !out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "lse_merge: null partials/lses/out");
  if (!aligned(partials, 16) || !aligned(out, 16) || !aligned(lses, 4) ||
      (out_lse && !aligned(out_lse, 4)))
    return fail(MLA_ERR_INVALID_ARGUMENT, "lse_merge: partials/out need 16-byte alignment");
  const long long rows = (long long)T * H;
  cudaError_t e = mla::launch_lse_combine(partials, partials_fp32 != 0, lses, n_shards, rows,
                                          rows, !lse_base_e, lse_base_e ? 0.6931471805599453f : 1.f,
                                          static_cast<uint16_t*>(out), out_lse,
                                          reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "lse_merge launch: %s", cudaGetErrorString(e));
  return ok();
}

static int slot_args_check(const char* fn, int B, int N, int block_size, int cp_size,
                           int cp_rank, int interleave, int max_blocks, int64_t bt_stride) {
  if (B < 0 || N < 0) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: B, N must be >= 0", fn);
  if (block_size < 1 || cp_size < 1 || interleave < 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size, cp_size, interleave >= 1", fn);
  if (cp_rank < 0 || cp_rank >= cp_size)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 0 <= cp_rank < cp_size", fn);
  if (block_size % interleave != 0)
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: block_size (%d) must be a multiple of interleave (%d)", fn, block_size,
                interleave);
  if (max_blocks < 1 || bt_stride < max_blocks)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 1 <= max_blocks <= bt_stride", fn);
  if ((long long)block_size * cp_size > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: block_size*cp_size exceeds 2^31-1", fn);
  if ((long long)B * N > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: B*N exceeds 2^31-1 positions", fn);
  return MLA_OK;
}

int cp_local_slot(const int64_t* positions, const int32_t* block_table, int64_t bt_stride,
                  int max_blocks, int B, int N, int block_size, int cp_size, int cp_rank,
                  int interleave, int64_t* slots, mla_stream_t stream) {
  int rc = slot_args_check("cp_local_slot", B, N, block_size, cp_size, cp_rank, interleave,
                           max_blocks, bt_stride);
  if (rc != MLA_OK) return rc;
  if ((long long)B * N == 0) return ok();
  if (!positions || !block_table || !slots)
    return fail(MLA_ERR_INVALID_ARGUMENT, "cp_local_slot: null positions/block_table/slots");
  if (!aligned(positions, 8) || !aligned(slots, 8) || !aligned(block_table, 4))
    return fail(MLA_ERR_INVALID_ARGUMENT, "cp_local_slot: misaligned pointer");
  DeviceInfo* dev = nullptr;
  rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  cudaError_t e = mla::launch_cp_local_slot(positions, block_table, bt_stride, max_blocks, B, N,
                                            block_size, cp_size, cp_rank, interleave, slots,
                                            dev->status, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(MLA_ERR_CUDA, "cp_local_slot launch: %s", cudaGetErrorString(e));
  return ok();
}

int cp_local_slot_scatter(const int64_t* positions, const void* kv_new,
                          const int32_t* block_table, int64_t bt_stride, int max_blocks, int B,
                          int N, int block_size, int cp_size, int cp_rank, int interleave,
                          void* kv_cache, int num_blocks, int64_t* slots, mla_stream_t stream) {
  int rc = slot_args_check("cp_local_slot_scatter", B, N, block_size, cp_size, cp_rank,
                           interleave, max_blocks, bt_stride);
  if (rc != MLA_OK) return rc;
  if (num_blocks < 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "cp_local_slot_scatter: num_blocks < 1");
  if ((long long)B * N == 0) return ok();
  if (!positions || !kv_new || !block_table || !kv_cache)
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "cp_local_slot_scatter: null positions/kv_new/block_table/kv_cache");
  if (!aligned(positions, 8) || (slots && !aligned(slots, 8)) || !aligned(block_table, 4) ||
      !aligned(kv_new, 16) || !aligned(kv_cache, 16))
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "cp_local_slot_scatter: misaligned pointer (kv_new and kv_cache need 16 bytes)");
  DeviceInfo* dev = nullptr;
  rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  cudaError_t e = mla::launch_cp_local_slot_scatter(
      positions, static_cast<const uint16_t*>(kv_new), block_table, bt_stride, max_blocks, B, N,
      block_size, cp_size, cp_rank, interleave, static_cast<uint16_t*>(kv_cache), num_blocks,
      slots, dev->status, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(MLA_ERR_CUDA, "cp_local_slot_scatter launch: %s", cudaGetErrorString(e));
  return ok();
}

int cp_step_tables(const int32_t* prev_lens, const int32_t* ctx_lens, const int32_t* new_lens,
                   int B, int N, int32_t* block_table, int64_t bt_stride, int max_blocks,
                   int32_t* free_pages, int free_cap, const int32_t* free_state,
                   int32_t* free_state_out, int block_size, int cp_size, int cp_rank,
                   int n_ranks, int interleave, int32_t* total_lens, int32_t* seq_lens,
                   int64_t* positions, int64_t* slots, mla_stream_t stream) {
  const char* fn = "cp_step_tables";
  int rc = slot_args_check(fn, B, N, block_size, cp_size, cp_rank, interleave, max_blocks,
                           bt_stride);
  if (rc != MLA_OK) return rc;
  if (n_ranks < 1 || n_ranks > cp_size - cp_rank)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 1 <= n_ranks (%d) <= cp_size - cp_rank (%d)",
                fn, n_ranks, cp_size - cp_rank);
  if ((long long)B * N > ((1LL << 31) - 1) / n_ranks || (long long)B * n_ranks > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: n_ranks*B*N exceeds 2^31-1", fn);
  if (free_cap < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: free_cap=%d < 1", fn, free_cap);
  if (!free_pages || !free_state || !free_state_out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null free_pages/free_state/free_state_out", fn);
  if (B > 0 && (!prev_lens || !ctx_lens || !new_lens || !block_table || !total_lens))
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: null prev_lens/ctx_lens/new_lens/block_table/total_lens", fn);
  const void* words[] = {prev_lens, ctx_lens, new_lens, block_table, free_pages, free_state,
                         free_state_out, total_lens, seq_lens};
  for (const void* w : words)
    if (!aligned(w, 4)) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned int32 argument", fn);
  if (!aligned(positions, 8) || !aligned(slots, 8))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned int64 argument", fn);
  // no output (the two updated in place included) may touch an input or another output
  struct Range {
    const void* p;
    unsigned long long bytes;
    bool written;
  };
  const unsigned long long b4 = 4ull * B, bn8 = 8ull * B * N;
  const Range ranges[] = {
      {prev_lens, b4, false},
      {ctx_lens, b4, false},
      {new_lens, b4, false},
      {free_state, 8, false},
      {block_table, B > 0 ? 4ull * ((unsigned long long)(B - 1) * bt_stride + max_blocks) : 0, true},
      {free_pages, 4ull * free_cap, true},
      {free_state_out, 8, true},
      {total_lens, b4, true},
      {seq_lens, b4 * n_ranks, true},
      {positions, bn8, true},
      {slots, bn8 * n_ranks, true}};
  const int nr = (int)(sizeof(ranges) / sizeof(ranges[0]));
  for (int i = 0; i < nr; ++i)
    for (int j = 0; j < i; ++j) {
      const Range &x = ranges[i], &y = ranges[j];
      if (!x.p || !y.p || x.bytes == 0 || y.bytes == 0 || !(x.written || y.written)) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
      if (a < b + y.bytes && b < a + x.bytes)
        return fail(MLA_ERR_INVALID_ARGUMENT, "%s: an output overlaps another argument", fn);
    }
  DeviceInfo* dev = nullptr;
  rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  mla::StepArgs a;
  a.prev = prev_lens;
  a.ctx = ctx_lens;
  a.fresh = new_lens;
  a.B = B;
  a.N = N;
  a.table = block_table;
  a.bt_stride = bt_stride;
  a.max_blocks = max_blocks;
  a.ring = free_pages;
  a.cap = free_cap;
  a.state = free_state;
  a.state_out = free_state_out;
  a.block_size = block_size;
  a.cp_size = cp_size;
  a.cp_rank = cp_rank;
  a.n_ranks = n_ranks;
  a.interleave = interleave;
  a.total = total_lens;
  a.seq = seq_lens;
  a.positions = positions;
  a.slots = slots;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  cudaError_t e = mla::launch_cp_step_tables(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

int cp_store_q8(const void* kv_new, const int32_t* ctx_lens, const int32_t* total_lens,
                const int32_t* block_table, int64_t bt_stride, int max_blocks, int B, int N,
                int block_size, int cp_size, int cp_rank, int interleave, void* kv_cache,
                float* kv_scales, int num_blocks, mla_stream_t stream) {
  const char* fn = "cp_store_q8";
  int rc = slot_args_check(fn, B, N, block_size, cp_size, cp_rank, interleave, max_blocks,
                           bt_stride);
  if (rc != MLA_OK) return rc;
  if (block_size % MLA_Q8_GROUP != 0)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size (%d) must be a multiple of %d", fn,
                block_size, MLA_Q8_GROUP);
  if (num_blocks < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: num_blocks < 1", fn);
  if ((long long)B * N == 0) return ok();
  if (!kv_new || !ctx_lens || !total_lens || !block_table || !kv_cache || !kv_scales)
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: null kv_new/ctx_lens/total_lens/block_table/kv_cache/kv_scales", fn);
  if (!aligned(kv_new, 16) || !aligned(kv_cache, 16) || !aligned(ctx_lens, 4) ||
      !aligned(total_lens, 4) || !aligned(block_table, 4) || !aligned(kv_scales, 4))
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: misaligned pointer (kv_new and kv_cache need 16 bytes)", fn);
  DeviceInfo* dev = nullptr;
  rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  mla::StoreQ8Args a;
  a.kv_new = static_cast<const uint16_t*>(kv_new);
  a.ctx = ctx_lens;
  a.total = total_lens;
  a.table = block_table;
  a.bt_stride = bt_stride;
  a.max_blocks = max_blocks;
  a.B = B;
  a.N = N;
  a.block_size = block_size;
  a.cp_size = cp_size;
  a.cp_rank = cp_rank;
  a.interleave = interleave;
  a.cache = static_cast<uint8_t*>(kv_cache);
  a.scales = kv_scales;
  a.num_blocks = num_blocks;
  a.status = dev->status;
  cudaError_t e = mla::launch_cp_store_q8(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

int lse_merge_v(const void* partials, int partials_fp32, const float* lses, int n_shards, int T,
                int H, int dv, void* out, float* out_lse, int lse_base_e, mla_stream_t stream) {
  const char* fn = "lse_merge_v";
  if (dv != 128 && dv != MLA_HEAD_DIM_V)
    return fail(MLA_ERR_UNSUPPORTED, "%s: dv=%d is neither 128 nor %d", fn, dv, MLA_HEAD_DIM_V);
  if (dv == MLA_HEAD_DIM_V)
    return lse_merge(partials, partials_fp32, lses, n_shards, T, H, out, out_lse, lse_base_e, stream);
  if (n_shards < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: n_shards=%d < 1", fn, n_shards);
  if (T < 0 || H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need T >= 0, H >= 1", fn);
  if (T == 0) return ok();
  if (!partials || !lses || !out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null partials/lses/out", fn);
  if (!aligned(partials, 16) || !aligned(out, 16) || !aligned(lses, 4) ||
      (out_lse && !aligned(out_lse, 4)))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: partials/out need 16-byte alignment", fn);
  const long long rows = (long long)T * H;
  if (rows > (1LL << 34)) return fail(MLA_ERR_UNSUPPORTED, "%s: too many rows", fn);
  cudaError_t e = mla::launch_lse_combine128(partials, partials_fp32 != 0, lses, n_shards, rows, !lse_base_e,
                                             lse_base_e ? 0.6931471805599453f : 1.f,
                                             static_cast<uint16_t*>(out), out_lse, nullptr, 0, H,
                                             reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

// Row strides in elements of a tensor whose rows start on 16 bytes.
static bool strides_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < (1LL << 36); }

int mla_rope(const void* x, int64_t x_stride_t, int64_t x_stride_h, const int64_t* positions,
             const int64_t* freqs, int T, int H, int half, float mscale, void* out,
             int64_t out_stride_t, int64_t out_stride_h, mla_stream_t stream) {
  const char* fn = "mla_rope";
  if (T < 0 || H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need T >= 0 (%d), H >= 1 (%d)", fn, T, H);
  if (!isfinite(mscale)) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: mscale must be finite", fn);
  if (!strides_ok(x_stride_t) || !strides_ok(x_stride_h) || !strides_ok(out_stride_t) || !strides_ok(out_stride_h))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: strides must be multiples of 8 elements, 0 <= stride < 2^36", fn);
  {
    // the rows of out may lie in any order, but apart
    const bool by_t = out_stride_t >= out_stride_h;
    const int64_t wide = by_t ? out_stride_t : out_stride_h, narrow = by_t ? out_stride_h : out_stride_t;
    const int64_t n_wide = by_t ? T : H, n_narrow = by_t ? H : T;
    if ((n_narrow > 1 && narrow < 64) || (n_wide > 1 && wide < (n_narrow > 1 ? narrow * (n_narrow - 1) : 0) + 64))
      return fail(MLA_ERR_INVALID_ARGUMENT, "%s: out's rows overlap (strides %lld, %lld)", fn,
                  (long long)out_stride_t, (long long)out_stride_h);
  }
  if (T == 0) return ok();
  if (!x || !positions || !freqs || !out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null x/positions/freqs/out", fn);
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 8) || !aligned(freqs, 8))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned pointer (x and out need 16 bytes)", fn);
  DeviceInfo* dev = nullptr;
  int rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  mla::RopeArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.x_t = x_stride_t;
  a.x_h = x_stride_h;
  a.out = static_cast<uint16_t*>(out);
  a.out_t = out_stride_t;
  a.out_h = out_stride_h;
  a.positions = positions;
  a.freqs = freqs;
  a.T = T;
  a.H = H;
  a.half = half != 0;
  a.mscale = mscale;
  a.num_sms = dev->num_sms;
  cudaError_t e = mla::launch_mla_rope(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

int cp_rope_store(const void* latent, int64_t latent_stride, const void* k_rope, int64_t k_rope_stride,
                  const int64_t* positions, const int64_t* freqs, const int32_t* block_table,
                  int64_t bt_stride, int max_blocks, int B, int N, int block_size, int cp_size,
                  int cp_rank, int interleave, int half, float mscale, void* kv_cache, int num_blocks,
                  int64_t* slots, mla_stream_t stream) {
  const char* fn = "cp_rope_store";
  int rc = slot_args_check(fn, B, N, block_size, cp_size, cp_rank, interleave, max_blocks, bt_stride);
  if (rc != MLA_OK) return rc;
  if (num_blocks < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: num_blocks < 1", fn);
  if (!isfinite(mscale)) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: mscale must be finite", fn);
  if (!strides_ok(latent_stride) || !strides_ok(k_rope_stride))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: strides must be multiples of 8 elements, 0 <= stride < 2^36", fn);
  if ((long long)B * N == 0) return ok();
  if (!latent || !k_rope || !positions || !freqs || !block_table || !kv_cache)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null latent/k_rope/positions/freqs/block_table/kv_cache", fn);
  if (!aligned(latent, 16) || !aligned(k_rope, 16) || !aligned(kv_cache, 16) || !aligned(positions, 8) ||
      !aligned(freqs, 8) || !aligned(block_table, 4) || (slots && !aligned(slots, 8)))
    return fail(MLA_ERR_INVALID_ARGUMENT,
                "%s: misaligned pointer (latent, k_rope and kv_cache need 16 bytes)", fn);
  DeviceInfo* dev = nullptr;
  rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  mla::RopeStoreArgs a;
  a.latent = static_cast<const uint16_t*>(latent);
  a.k_rope = static_cast<const uint16_t*>(k_rope);
  a.latent_t = latent_stride;
  a.k_rope_t = k_rope_stride;
  a.positions = positions;
  a.freqs = freqs;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.max_blocks = max_blocks;
  a.B = B;
  a.N = N;
  a.block_size = block_size;
  a.cp_size = cp_size;
  a.cp_rank = cp_rank;
  a.interleave = interleave;
  a.half = half != 0;
  a.mscale = mscale;
  a.cache = static_cast<uint16_t*>(kv_cache);
  a.num_blocks = num_blocks;
  a.slots = slots;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  cudaError_t e = mla::launch_cp_rope_store(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

int mla_expand(const void* kv_cache, const float* kv_scales, const int32_t* block_table,
               int64_t bt_stride, const int32_t* seq_lens, const int32_t* kv_starts, int B,
               int block_size, int num_blocks, int max_blocks, const void* w_kv, int H, int S, void* kv,
               void* k_rope, mla_stream_t stream) {
  const char* fn = "mla_expand";
  if (B < 0 || S < 0) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: B, S must be >= 0", fn);
  if (H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: H=%d < 1", fn, H);
  if (block_size < 1 || num_blocks < 1)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size and num_blocks must be >= 1", fn);
  if (kv_scales && block_size % MLA_Q8_GROUP != 0)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: block_size (%d) must be a multiple of %d", fn, block_size,
                MLA_Q8_GROUP);
  if (max_blocks < 1 || bt_stride < max_blocks)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 1 <= max_blocks (%d) <= bt_stride (%lld)", fn, max_blocks,
                (long long)bt_stride);
  if ((long long)max_blocks * block_size > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: max_blocks*block_size exceeds 2^31-1", fn);
  if (S > INT_MAX - 512 || (S / 256 + 1LL) * 2 * H > INT_MAX - 512)
    return fail(MLA_ERR_UNSUPPORTED, "%s: S or (S/256 + 1) * 2 H too close to 2^31", fn);
  if (B == 0 || S == 0) return ok();
  if (!kv_cache || !block_table || !seq_lens || !kv_starts || !w_kv || !kv || !k_rope)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null kv_cache/block_table/seq_lens/kv_starts/w_kv/kv/k_rope", fn);
  if (!aligned(kv_cache, 16) || !aligned(w_kv, 16) || !aligned(kv, 16) || !aligned(k_rope, 16))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: kv_cache, w_kv, kv and k_rope must be 16-byte aligned", fn);
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(kv_starts, 4) ||
      (kv_scales && !aligned(kv_scales, 4)))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned int32/float argument", fn);
  DeviceInfo* dev = nullptr;
  int rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  if (!mla::tile_maps_ok()) return fail(MLA_ERR_CUDA, "%s: the CUDA driver has no cuTensorMapEncodeTiled", fn);
  mla::ExpandArgs a;
  a.cache = kv_cache;
  a.scales = kv_scales;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.seq_lens = seq_lens;
  a.starts = kv_starts;
  a.B = B;
  a.w = static_cast<const uint16_t*>(w_kv);
  a.H = H;
  a.S = S;
  a.kv = static_cast<uint16_t*>(kv);
  a.k_rope = static_cast<uint16_t*>(k_rope);
  const unsigned long long wait_ns = g_wait_ns.load();
  a.wait_ns = wait_ns ? wait_ns : mla::sm100::kDefaultWaitNs;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  cudaError_t e = mla::launch_mla_expand(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

size_t mla_prefill_workspace_size(int T, int B, int H, int S, int num_sms) {
  if (T <= 0 || B <= 0 || H <= 0 || S <= 0 || num_sms <= 0) return 0;
  return mla::prefill_workspace_size(T, B, H, S, num_sms);
}

int mla_prefill(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_nope,
                int64_t k_stride_s, int64_t k_stride_h, const void* k_rope, int64_t k_rope_stride,
                const void* v, int64_t v_stride_s, int64_t v_stride_h, const int32_t* cu_q_lens,
                const int32_t* kv_starts, const int32_t* seq_lens,
                const int32_t* causal_seqlens_global, int T, int B, int H, int S, int causal,
                int cp_world, int cp_rank, int interleave, float scale, void* out, float* lse,
                int lse_base_e, void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  const char* fn = "mla_prefill";
  if (T < 0 || B < 0 || S < 0) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: T, B, S must be >= 0", fn);
  if (H < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: H=%d < 1", fn, H);
  if (cp_world < 1 || cp_rank < 0 || cp_rank >= cp_world)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: need 0 <= cp_rank (%d) < cp_world (%d)", fn, cp_rank, cp_world);
  if (interleave < 1) return fail(MLA_ERR_INVALID_ARGUMENT, "%s: interleave=%d < 1", fn, interleave);
  if ((long long)cp_world * interleave > (1LL << 31) - 1)
    return fail(MLA_ERR_UNSUPPORTED, "%s: cp_world*interleave exceeds 2^31-1", fn);
  if (!isfinite(scale) || !(scale > 0.f))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: scale must be finite and > 0", fn);
  const struct {
    int64_t stride;
    int size;
  } dims[] = {{q_stride_t, T}, {q_stride_h, H}, {k_stride_s, S}, {k_stride_h, H}, {k_rope_stride, S},
              {v_stride_s, S}, {v_stride_h, H}};
  for (const auto& d : dims)
    if (!strides_ok(d.stride) || (d.size > 1 && d.stride == 0))
      return fail(MLA_ERR_INVALID_ARGUMENT, "%s: strides must be multiples of 8 elements, 0 < stride < 2^36", fn);
  if (T == 0 || B == 0) return ok();
  if (!q || (S > 0 && (!k_nope || !k_rope || !v)) || !cu_q_lens || !kv_starts || !seq_lens || !out)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: null q/k_nope/k_rope/v/cu_q_lens/kv_starts/seq_lens/out", fn);
  if (!causal) causal_seqlens_global = nullptr;            // not read, whatever it holds
  if (causal_seqlens_global == nullptr && cp_world != 1 && causal)
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: causal_seqlens_global is required when cp_world > 1", fn);
  if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16) || !aligned(out, 16))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: q, k_nope, k_rope, v and out must be 16-byte aligned", fn);
  if (!aligned(cu_q_lens, 4) || !aligned(kv_starts, 4) || !aligned(seq_lens, 4) ||
      !aligned(causal_seqlens_global, 4) || !aligned(lse, 4))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: misaligned int32/float argument", fn);
  if (workspace && !aligned(workspace, 256))
    return fail(MLA_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
  if (!mla::prefill_grid_ok(T, B, H)) return fail(MLA_ERR_UNSUPPORTED, "%s: (T/256 + B) * H exceeds 2^31-1", fn);
  if (S > INT_MAX - 256 || T > INT_MAX - 512)
    return fail(MLA_ERR_UNSUPPORTED, "%s: T or S too close to 2^31", fn);
  DeviceInfo* dev = nullptr;
  int rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  if (!mla::tile_maps_ok()) return fail(MLA_ERR_CUDA, "%s: the CUDA driver has no cuTensorMapEncodeTiled", fn);
  mla::PrefillArgs a = {};
  a.cu = cu_q_lens;
  a.starts = kv_starts;
  a.seq_lens = seq_lens;
  a.gseq = causal_seqlens_global;
  a.T = T;
  a.B = B;
  a.H = H;
  a.S = S;
  a.causal = causal ? 1 : 0;
  a.cp = cp_world;
  a.rank = cp_rank;
  a.il = interleave;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.lse_mul = lse_base_e ? 0.6931471805599453f : 1.f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const unsigned long long wait_ns = g_wait_ns.load();
  a.wait_ns = wait_ns ? wait_ns : mla::sm100::kDefaultWaitNs;
  a.num_sms = dev->num_sms;
  a.status = dev->status;
  mla::PrefillTensors x;
  x.q = q;
  x.q_t = q_stride_t;
  x.q_h = q_stride_h;
  x.k_nope = k_nope;
  x.k_s = k_stride_s;
  x.k_h = k_stride_h;
  x.k_rope = k_rope;
  x.r_s = k_rope_stride;
  x.v = v;
  x.v_s = v_stride_s;
  x.v_h = v_stride_h;
  x.workspace = workspace;
  x.workspace_bytes = workspace_bytes;
  cudaError_t e = mla::launch_mla_prefill(a, x, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}

int mla_get_device_status(mla_stream_t stream, uint32_t* bits_out) {
  DeviceInfo* dev = nullptr;
  int rc = device_info(&dev);
  if (rc != MLA_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess)
    return fail(MLA_ERR_CUDA, "mla_get_device_status: %s", cudaGetErrorString(e));
  unsigned int bits = 0;
  e = cudaMemcpyFromSymbol(&bits, g_mla_status, sizeof(bits));
  if (e == cudaSuccess) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_mla_status, &zero, sizeof(zero));
  }
  if (e != cudaSuccess)
    return fail(MLA_ERR_CUDA, "mla_get_device_status: %s", cudaGetErrorString(e));
  if (bits_out) *bits_out = bits;
  if (bits == 0) return ok();
  return fail(MLA_ERR_DEVICE, "device status 0x%x:%s%s%s%s%s%s%s", bits,
              (bits & MLA_STATUS_BAD_PAGE) ? " bad block_table entry;" : "",
              (bits & MLA_STATUS_SEQ_TOO_LONG) ? " seq_len beyond max_blocks*block_size;" : "",
              (bits & MLA_STATUS_BAD_VBLOCK) ? " virtual block beyond max_blocks;" : "",
              (bits & MLA_STATUS_WAIT_TIMEOUT) ? " on-chip wait timed out;" : "",
              (bits & MLA_STATUS_BAD_SCALE) ? " 8-bit cache scale out of range;" : "",
              (bits & MLA_STATUS_OUT_OF_PAGES) ? " too few free pages;" : "",
              (bits & MLA_STATUS_BAD_STEP) ? " length or ring state out of range;" : "");
}

}  // extern "C"
