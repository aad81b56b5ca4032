// launch.h -- internal launch entry points of libattn.so (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <stdint.h>

namespace sdpa {

// Raises a kernel's limit of dynamic shared memory, once per device (`ready`: a bit for each), to the most that
// any call of it needs. The limit belongs to the kernel and not to a launch: set to what each call needs, it could
// be lowered by another host thread between this one's setting it and its launch, which then fails.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return e;
}

// Internal mask mode of attn_fwd_sinks, beside the attn_mask values: row i at position
// p = i + sk - sq sees key j iff j <= p and (j >= p - pre or j < sinks).
constexpr int kMaskSinks = 4;

struct FwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu_q;   // TND only
  const int32_t* cu_kv;  // TND only
  int B, Sq, Skv, Nq, Nkv, D;
  int Dv;  // value / output head size (== D except through attn_fwd_masked)
  float scale;
  int mask_mode, layout, dtype;
  int pre, next;               // band limits (mask_mode ATTN_MASK_BAND), clamped to +-2^30;
                               // kMaskSinks: pre = window - 1
  int sinks;                   // kMaskSinks: first keys that stay visible
  const uint8_t* mask;         // explicit mask, 1 = excluded (null: none)
  int64_t mask_bs, mask_rs;    // its batch and row strides in bytes
  bool mask_vec;               // mask, mask_bs and mask_rs all 16-byte aligned
  int acc_mode;  // 0: plain output; 1: overwrite an accumulator; 2: merge into it
  void* out;     // output, or the accumulator's output (merge layouts) when acc_mode != 0
  float* smax;   // statistics (may be null with ssum when acc_mode == 0), or the accumulator's
  float* ssum;   // [.., 8]-lane statistics when acc_mode != 0
  int* status;  // device status word
  int num_sms;
};

struct CsrArgs {
  const float* q;
  const float* k;
  const float* v;
  const int32_t* offset;
  const int32_t* columns;
  int B, H, S, D;
  int64_t nnz_cap;
  bool cols_vec;  // columns 16-byte aligned and nnz_cap % 4 == 0: read 4 indices at a time
  float* out;
  int* status;
  int num_sms;   // SMs of the device (the tiled kernel sizes its blocks to fill whole rounds)
};

struct CsrTcArgs {  // attn_sparse_csr_tc: 16-bit q, k, v, out [B, H, S, D]
  const void* q;
  const void* k;
  const void* v;
  const int32_t* offset;   // unused with a plan
  const int32_t* columns;  // unused with a plan
  const uint8_t* plan;     // a plan of the pattern (csr_plan.cuh), or null: build per block
  int B, H, S, D, dtype;
  int64_t nnz_cap;
  bool cols_vec;  // columns 16-byte aligned and nnz_cap % 4 == 0: read 4 indices at a time
  void* out;
  int* status;
};

struct CsrPlanArgs {  // attn_csr_plan: the pattern of a CSR call and the plan buffer to fill
  const int32_t* offset;
  const int32_t* columns;
  int B, H, S;
  int64_t nnz_cap;
  bool cols_vec;
  uint8_t* plan;
  int* status;
};

struct MergeArgs {
  const void* prev_out;
  const float* prev_max;
  const float* prev_sum;
  const void* cur_out;
  const float* cur_max;
  const float* cur_sum;
  int S, B, N, D, dtype, layout;
  const int64_t* seq_qlen;  // TND only, may be null
  void* out;
  float* out_max;
  float* out_sum;
  int* status;
};

// A paged key/value cache (paged.cuh) and the rows of its page table.
struct PagedArgs {
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* seq_lens;    // [B]
  int B, num_pages, page_size, max_pages;
  int64_t page_stride, tok_stride, head_stride;  // elements
  uint32_t div_mul;           // division by page_size (page_of)
  int div_shift;
};

struct DecodeArgs {
  PagedArgs p;
  const void* q;  // [B, Nq, D]
  const void* k;
  const void* v;
  int Nq, Nkv, D, dtype;
  float scale;
  int window, sinks;  // clamped to 2^30
  int rows, groups;   // query heads a unit works on; units a KV head's query heads are cut into
  float* part;        // workspace: partial results
  unsigned* ctr;      // workspace: arrival counters, 0 between calls
  void* out;          // [B, Nq, D]
  float* smax;        // [B, Nq], may be null with ssum
  float* ssum;
  int* status;
  int num_sms;
};

struct AppendArgs {
  PagedArgs p;
  const void* k_new;          // [T, Nkv, D]
  const void* v_new;
  const int32_t* cu;          // [B] cumulative new tokens, or null: one per row
  int T, Nkv, D, dtype;
  void* k;
  void* v;
  int* status;
  int num_sms;
};

constexpr int kMaxTableRows = 8192;  // rows of a page table in the calls that change it

struct ForkArgs {
  const int32_t* table;
  const int32_t* src;
  const int32_t* ref;
  const int32_t* lens;      // may be null with lens_out
  int rows_in, rows_out, max_pages, num_pages;
  int32_t* table_out;
  int32_t* ref_out;
  int32_t* lens_out;
  int* status;
};

struct ReserveArgs {
  int32_t* table;
  int32_t* ref;
  const int32_t* lens;
  const int32_t* new_tokens;  // null: one per row
  int32_t* copies;            // [B, 2]
  int32_t* lens_out;          // attn_cache_grow: lens; null with new_lens otherwise
  int32_t* new_lens;          // [B]
  bool live_only;             // without new_tokens: empty rows get none
  int B, max_pages, num_pages, page_size;
  int* status;
};

struct EvictArgs {
  int32_t* table;
  int32_t* ref;
  const int32_t* lens;
  int B, max_pages, num_pages, page_size;
  int window, sinks;  // clamped to 2^30
  int* status;
};

struct CompactArgs {
  const int32_t* table;
  const int32_t* ref;
  int rows, max_pages, num_pages;
  int32_t* table_out;
  int32_t* ref_out;
  int32_t* page_map;  // [num_pages]
  int32_t* copies;    // [num_pages / 2, 2]
  int32_t* live;      // [1]
  int* status;
};

struct PageCopyArgs {
  const int32_t* copies;  // [n, 2]
  int n, num_pages;
  int64_t page_bytes, stride_bytes;
  void* k;
  void* v;
  int* status;
  int num_sms;
};

// Workspace of attn_decode_paged: partial results of at most kDecodeMaxCtas blocks (two each: the
// unit a block's range starts in and the one it ends in) of `rows` query heads, and the counters.
constexpr int kDecodeMaxCtas = 512;
int decode_rows(int dtype, int Nq, int Nkv, int D);
int64_t decode_workspace_bytes(int rows, int D);

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);
cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t st);
cudaError_t launch_cache_reserve(const ReserveArgs& a, cudaStream_t st);
cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st);
cudaError_t launch_cache_copy(const PageCopyArgs& a, cudaStream_t st);
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t st);
cudaError_t launch_fwd_f32(const FwdArgs& a, cudaStream_t st);
cudaError_t launch_fwd_bf16(const FwdArgs& a, cudaStream_t st);
cudaError_t launch_sparse_csr(const CsrArgs& a, cudaStream_t st);
bool sparse_csr_tiled_supported(const CsrArgs& a);
cudaError_t launch_sparse_csr_tiled(const CsrArgs& a, cudaStream_t st);
cudaError_t launch_sparse_csr_tc(const CsrTcArgs& a, cudaStream_t st);
cudaError_t launch_csr_plan(const CsrPlanArgs& a, cudaStream_t st);

}  // namespace sdpa
