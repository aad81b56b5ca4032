// attn_api.cu -- the C ABI of libattn.so: argument checks, the device status word, dispatch.
//
// Argument limits follow the constraints of "aclnnFlashAttentionVarLenScore" (CANN 8.5 API
// doc, 约束说明): Nq/Nkv a nonzero integer with 1 <= Nq <= 256, head dim at most 768, at most
// 1M packed tokens and 2K cumulative-length entries. The host never reads device data, so
// data-dependent checks happen in the kernels, which record them in the status word below.
#include <cuda_runtime.h>
#include <stdint.h>

#include <math.h>

#include <mutex>

#include "attn.h"
#include "csr_plan.cuh"
#include "launch.h"

namespace {

// One status word per device; kernels record the first device-side error here. Beside it, the
// slot attn_get_last_error reads the word into (exchanging it for 0 in one atomic step).
__device__ int g_status_word;
__device__ int g_status_read;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
std::mutex g_read_mu[kMaxDevices];  // one status reader at a time per device (the read slot)
int* g_status_ptr[kMaxDevices] = {};
int* g_read_ptr[kMaxDevices] = {};
int g_num_sms[kMaxDevices] = {};

// Device addresses of this device's status word and read slot, and its SM count (looked up
// once per device, with that device current).
int device_state(int** status, int* num_sms, int** read_slot = nullptr, int* device = nullptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_status_ptr[dev] == nullptr) {
    void* p = nullptr;
    void* r = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return ATTN_ERR_CUDA;
    if (cudaGetSymbolAddress(&r, g_status_read) != cudaSuccess) return ATTN_ERR_CUDA;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return ATTN_ERR_CUDA;
    g_read_ptr[dev] = static_cast<int*>(r);
    g_num_sms[dev] = sms;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  *status = g_status_ptr[dev];
  *num_sms = g_num_sms[dev];
  if (read_slot != nullptr) *read_slot = g_read_ptr[dev];
  if (device != nullptr) *device = dev;
  return ATTN_OK;
}

// Reads the status word and clears it in one step, so an error a kernel on another stream
// records meanwhile is kept for the next read instead of being lost between a read and a clear.
__global__ void read_and_clear_status(int* word, int* slot) { *slot = atomicExch(word, 0); }

constexpr int64_t kMaxTokens = 1 << 20;  // "1M"
constexpr int kMaxCu = 2048;             // "2K" cumulative-length entries

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" {

int attn_abi_version(void) { return (1 << 16) | 5; }  // 1.5: attn_cache_grow

const char* attn_status_string(int s) {
  switch (s) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported by this library";
    case ATTN_ERR_CUDA: return "CUDA runtime error";
    case ATTN_ERR_DATA: return "bad device data (cumulative lengths, CSR indices or page tables)";
    case ATTN_ERR_TIMEOUT: return "pipeline wait timed out";
    case ATTN_ERR_PAGES: return "not enough free pages";
    default: return "unknown status";
  }
}

}  // extern "C"

namespace {

// The masked-call extras of fwd_impl (band limits, explicit mask, value head size).
struct Extras {
  bool allow_band = false;
  bool window = false;  // attn_fwd_sinks: `pre` holds window - 1
  int64_t sinks = 0;
  int Dv = -1;  // -1: same as D
  int64_t pre = 0, next = 0;
  const uint8_t* mask = nullptr;
  int64_t mask_bs = 0, mask_rs = 0;
};

int clamp30(int64_t x) {
  const int64_t lim = int64_t(1) << 30;
  return (int)(x < -lim ? -lim : (x > lim ? lim : x));
}

int fwd_impl(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
             const int32_t* cu_seqlens_kv, int B, int Sq, int Skv, int Nq, int Nkv, int D,
             float scale, int mask_mode, int dtype, int layout, void* out, float* softmax_max,
             float* softmax_sum, int acc_mode, void* stream, const Extras& x = Extras()) {
  if (layout != ATTN_BHSD && layout != ATTN_TND) return ATTN_ERR_INVALID;
  if (dtype != ATTN_BF16 && dtype != ATTN_F32 && dtype != ATTN_F16) return ATTN_ERR_INVALID;
  const int max_mode = x.allow_band ? ATTN_MASK_BAND : ATTN_MASK_CAUSAL_BOTTOMRIGHT;
  if (mask_mode < ATTN_MASK_NONE || mask_mode > max_mode) return ATTN_ERR_INVALID;
  if (mask_mode == ATTN_MASK_BAND && (int64_t)clamp30(x.pre) + clamp30(x.next) < 0) return ATTN_ERR_INVALID;
  const int Dv = x.Dv < 0 ? D : x.Dv;
  if (Dv < 1 || Dv > D) return ATTN_ERR_INVALID;
  if (x.mask != nullptr && (x.mask_bs < 0 || x.mask_rs < 0)) return ATTN_ERR_INVALID;
  if (x.mask != nullptr && layout == ATTN_BHSD && x.mask_rs < Skv) return ATTN_ERR_INVALID;
  if (B < 0 || Sq < 0 || Skv < 0) return ATTN_ERR_INVALID;
  if (Nq < 1 || Nq > 256 || Nkv < 1 || Nq % Nkv != 0) return ATTN_ERR_INVALID;
  if (D < 1 || D > 768) return ATTN_ERR_INVALID;
  if (!(scale > 0.f) || scale == INFINITY) return ATTN_ERR_INVALID;  // finite and positive
  if ((softmax_max == nullptr) != (softmax_sum == nullptr)) return ATTN_ERR_INVALID;
  if (acc_mode != 0 && softmax_max == nullptr) return ATTN_ERR_INVALID;
  if (layout == ATTN_TND) {
    if (B > kMaxCu || Sq > kMaxTokens || Skv > kMaxTokens) return ATTN_ERR_INVALID;
    if (B > 0 && (cu_seqlens_q == nullptr || cu_seqlens_kv == nullptr)) return ATTN_ERR_INVALID;
  } else if (cu_seqlens_q != nullptr || cu_seqlens_kv != nullptr) {
    return ATTN_ERR_INVALID;
  }
  const bool empty_q = B == 0 || Sq == 0;
  if (empty_q) return ATTN_OK;
  if (q == nullptr || out == nullptr) return ATTN_ERR_INVALID;
  if (Skv > 0 && (k == nullptr || v == nullptr)) return ATTN_ERR_INVALID;
  if (dtype == ATTN_F32 && D > 256) return ATTN_ERR_UNSUPPORTED;
  if (dtype == ATTN_BF16 || dtype == ATTN_F16) {
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (Dv != D && !(D == 128 && Dv == 64)) return ATTN_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return ATTN_ERR_INVALID;
  }

  sdpa::FwdArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu_q = cu_seqlens_q;
  a.cu_kv = cu_seqlens_kv;
  a.B = B;
  a.Sq = Sq;
  a.Skv = Skv;
  a.Nq = Nq;
  a.Nkv = Nkv;
  a.D = D;
  a.Dv = Dv;
  a.scale = scale;
  a.mask_mode = x.window ? sdpa::kMaskSinks : mask_mode;
  a.sinks = clamp30(x.sinks);
  a.pre = clamp30(x.pre);
  a.next = clamp30(x.next);
  a.mask = x.mask;
  a.mask_bs = x.mask_bs;
  a.mask_rs = x.mask_rs;
  a.mask_vec = x.mask != nullptr && aligned16(x.mask) && (x.mask_bs & 15) == 0 && (x.mask_rs & 15) == 0;
  a.layout = layout;
  a.dtype = dtype;
  a.acc_mode = acc_mode;
  a.out = out;
  a.smax = softmax_max;
  a.ssum = softmax_sum;
  int rc = device_state(&a.status, &a.num_sms);
  if (rc != ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == ATTN_F32 ? sdpa::launch_fwd_f32(a, st) : sdpa::launch_fwd_bf16(a, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
             const int32_t* cu_seqlens_kv, int B, int Sq, int Skv, int Nq, int Nkv, int D,
             float scale, int mask_mode, int dtype, int layout, void* out, float* softmax_max,
             float* softmax_sum, void* stream) {
  return fwd_impl(q, k, v, cu_seqlens_q, cu_seqlens_kv, B, Sq, Skv, Nq, Nkv, D, scale, mask_mode,
                  dtype, layout, out, softmax_max, softmax_sum, 0, stream);
}

int attn_fwd_accumulate(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                        const int32_t* cu_seqlens_kv, int B, int Sq, int Skv, int Nq, int Nkv,
                        int D, float scale, int mask_mode, int dtype, int layout, int first,
                        void* acc_out, float* acc_max, float* acc_sum, void* stream) {
  if (acc_out == nullptr || acc_max == nullptr || acc_sum == nullptr) return ATTN_ERR_INVALID;
  if (first != 0 && first != 1) return ATTN_ERR_INVALID;
  // the tensor-core epilogue moves a row's 8 statistic lanes as two 16-byte vectors
  if ((dtype == ATTN_BF16 || dtype == ATTN_F16) && (!aligned16(acc_max) || !aligned16(acc_sum)))
    return ATTN_ERR_INVALID;
  return fwd_impl(q, k, v, cu_seqlens_q, cu_seqlens_kv, B, Sq, Skv, Nq, Nkv, D, scale, mask_mode,
                  dtype, layout, acc_out, acc_max, acc_sum, first ? 1 : 2, stream);
}

int attn_fwd_masked(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                    const int32_t* cu_seqlens_kv, int B, int Sq, int Skv, int Nq, int Nkv, int Dqk,
                    int Dv, float scale, int mask_mode, int64_t pre_tokens, int64_t next_tokens,
                    const uint8_t* atten_mask, int64_t mask_batch_stride, int64_t mask_row_stride,
                    int dtype, int layout, void* out, float* softmax_max, float* softmax_sum,
                    void* stream) {
  Extras x;
  x.allow_band = true;
  x.Dv = Dv < 1 ? 0 : Dv;  // 0 is rejected as out of range
  x.pre = pre_tokens;
  x.next = next_tokens;
  x.mask = atten_mask;
  x.mask_bs = mask_batch_stride;
  x.mask_rs = mask_row_stride;
  return fwd_impl(q, k, v, cu_seqlens_q, cu_seqlens_kv, B, Sq, Skv, Nq, Nkv, Dqk, scale, mask_mode,
                  dtype, layout, out, softmax_max, softmax_sum, 0, stream, x);
}

int attn_fwd_sinks(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                   const int32_t* cu_seqlens_kv, int B, int Sq, int Skv, int Nq, int Nkv, int D,
                   float scale, int64_t window_tokens, int64_t sink_tokens, int dtype, int layout,
                   void* out, float* softmax_max, float* softmax_sum, void* stream) {
  if (window_tokens < 1 || sink_tokens < 0) return ATTN_ERR_INVALID;
  // positions are 32-bit sums of a row and the two lengths, and a window of 2^30 is one of every key
  if (Sq > 1 << 30 || Skv > 1 << 30) return ATTN_ERR_UNSUPPORTED;
  Extras x;
  x.window = true;
  x.pre = window_tokens - 1;
  x.sinks = sink_tokens;
  return fwd_impl(q, k, v, cu_seqlens_q, cu_seqlens_kv, B, Sq, Skv, Nq, Nkv, D, scale,
                  ATTN_MASK_CAUSAL_BOTTOMRIGHT, dtype, layout, out, softmax_max, softmax_sum, 0, stream, x);
}

int attn_sparse_csr(const float* q, const float* k, const float* v, const int32_t* csr_offset,
                    const int32_t* csr_columns, int B, int H, int S, int D, int64_t nnz_cap,
                    float* out, void* stream) {
  if (B < 0 || H < 0 || S < 0 || nnz_cap < 0) return ATTN_ERR_INVALID;
  if (D < 1) return ATTN_ERR_INVALID;
  if ((int64_t)B * H * S == 0) return ATTN_OK;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || csr_offset == nullptr)
    return ATTN_ERR_INVALID;
  if (nnz_cap > 0 && csr_columns == nullptr) return ATTN_ERR_INVALID;
  if (D > 256) return ATTN_ERR_UNSUPPORTED;
  sdpa::CsrArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.offset = csr_offset;
  a.columns = csr_columns;
  a.B = B;
  a.H = H;
  a.S = S;
  a.D = D;
  a.nnz_cap = nnz_cap;
  a.cols_vec = csr_columns != nullptr && aligned16(csr_columns) && nnz_cap % 4 == 0;
  a.out = out;
  int rc = device_state(&a.status, &a.num_sms);
  if (rc != ATTN_OK) return rc;
  // D = 64 or 128 with 16-byte aligned tensors: tiled over each block's union of columns;
  // otherwise a warp per row gathering its own entries
  const cudaError_t e = sdpa::sparse_csr_tiled_supported(a)
                            ? sdpa::launch_sparse_csr_tiled(a, static_cast<cudaStream_t>(stream))
                            : sdpa::launch_sparse_csr(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_sparse_csr_tc(const void* q, const void* k, const void* v, const int32_t* csr_offset,
                       const int32_t* csr_columns, int B, int H, int S, int D, int64_t nnz_cap,
                       int dtype, void* out, void* stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID;
  if (B < 0 || H < 0 || S < 0 || nnz_cap < 0) return ATTN_ERR_INVALID;
  if (D < 1) return ATTN_ERR_INVALID;
  if ((int64_t)B * H * S == 0) return ATTN_OK;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || csr_offset == nullptr)
    return ATTN_ERR_INVALID;
  if (nnz_cap > 0 && csr_columns == nullptr) return ATTN_ERR_INVALID;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (S > 32768) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return ATTN_ERR_INVALID;
  sdpa::CsrTcArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.offset = csr_offset;
  a.columns = csr_columns;
  a.B = B;
  a.H = H;
  a.S = S;
  a.D = D;
  a.dtype = dtype;
  a.nnz_cap = nnz_cap;
  a.cols_vec = csr_columns != nullptr && aligned16(csr_columns) && nnz_cap % 4 == 0;
  a.out = out;
  int sms = 0;
  int rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  const cudaError_t e = sdpa::launch_sparse_csr_tc(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_csr_plan_size(int B, int H, int S, int64_t nnz_cap, int64_t* bytes) {
  if (bytes == nullptr || B < 0 || H < 0 || S < 0 || nnz_cap < 0) return ATTN_ERR_INVALID;
  if (S > 32768) return ATTN_ERR_UNSUPPORTED;
  const int64_t n = sdpa::plan_bytes(B, H, S, nnz_cap);
  if (n < 0) return ATTN_ERR_UNSUPPORTED;
  *bytes = n;
  return ATTN_OK;
}

int attn_csr_plan(const int32_t* csr_offset, const int32_t* csr_columns, int B, int H, int S,
                  int64_t nnz_cap, void* plan, int64_t plan_bytes, void* stream) {
  int64_t need = 0;
  const int rc0 = attn_csr_plan_size(B, H, S, nnz_cap, &need);
  if (rc0 != ATTN_OK) return rc0;
  if ((int64_t)B * H * S == 0) return ATTN_OK;
  if (csr_offset == nullptr || plan == nullptr) return ATTN_ERR_INVALID;
  if (nnz_cap > 0 && csr_columns == nullptr) return ATTN_ERR_INVALID;
  if (plan_bytes < need || !aligned16(plan)) return ATTN_ERR_INVALID;
  sdpa::CsrPlanArgs a{};
  a.offset = csr_offset;
  a.columns = csr_columns;
  a.B = B;
  a.H = H;
  a.S = S;
  a.nnz_cap = nnz_cap;
  a.cols_vec = csr_columns != nullptr && aligned16(csr_columns) && nnz_cap % 4 == 0;
  a.plan = static_cast<uint8_t*>(plan);
  int sms = 0;
  int rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  const cudaError_t e = sdpa::launch_csr_plan(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_sparse_csr_tc_planned(const void* q, const void* k, const void* v, const void* plan,
                               int64_t plan_bytes, int B, int H, int S, int D, int64_t nnz_cap,
                               int dtype, void* out, void* stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F16) return ATTN_ERR_INVALID;
  int64_t need = 0;
  const int rc0 = attn_csr_plan_size(B, H, S, nnz_cap, &need);
  if (rc0 != ATTN_OK) return rc0;
  if (D < 1) return ATTN_ERR_INVALID;
  if ((int64_t)B * H * S == 0) return ATTN_OK;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || plan == nullptr)
    return ATTN_ERR_INVALID;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (plan_bytes < need || !aligned16(plan)) return ATTN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return ATTN_ERR_INVALID;
  sdpa::CsrTcArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.plan = static_cast<const uint8_t*>(plan);
  a.B = B;
  a.H = H;
  a.S = S;
  a.D = D;
  a.dtype = dtype;
  a.nnz_cap = nnz_cap;
  a.out = out;
  int sms = 0;
  int rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  const cudaError_t e = sdpa::launch_sparse_csr_tc(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_merge(const void* prev_out, const float* prev_max, const float* prev_sum,
               const void* cur_out, const float* cur_max, const float* cur_sum, int S, int B,
               int N, int D, int dtype, int layout, const int64_t* actual_seq_qlen, void* out,
               float* out_max, float* out_sum, void* stream) {
  if (dtype != ATTN_BF16 && dtype != ATTN_F32 && dtype != ATTN_F16) return ATTN_ERR_INVALID;
  if (layout != ATTN_BHSD && layout != ATTN_TND) return ATTN_ERR_INVALID;
  if (S < 0 || B < 0 || N < 1 || D < 1) return ATTN_ERR_INVALID;
  if (layout == ATTN_BHSD && actual_seq_qlen != nullptr) return ATTN_ERR_INVALID;
  if (layout == ATTN_TND && actual_seq_qlen != nullptr && (B < 1 || B > kMaxCu)) return ATTN_ERR_INVALID;
  const int64_t rows = layout == ATTN_TND ? (int64_t)S * N : (int64_t)S * B;
  if (rows == 0) return ATTN_OK;
  if (layout == ATTN_BHSD && ((int64_t)B * N > 0x7fffffffLL || S > 65535LL * 8)) return ATTN_ERR_UNSUPPORTED;
  if (layout == ATTN_TND && rows > 0x7fffffffLL * 8) return ATTN_ERR_UNSUPPORTED;
  if (!prev_out || !prev_max || !prev_sum || !cur_out || !cur_max || !cur_sum || !out ||
      !out_max || !out_sum)
    return ATTN_ERR_INVALID;
  sdpa::MergeArgs a{};
  a.prev_out = prev_out;
  a.prev_max = prev_max;
  a.prev_sum = prev_sum;
  a.cur_out = cur_out;
  a.cur_max = cur_max;
  a.cur_sum = cur_sum;
  a.S = S;
  a.B = B;
  a.N = N;
  a.D = D;
  a.dtype = dtype;
  a.layout = layout;
  a.seq_qlen = actual_seq_qlen;
  a.out = out;
  a.out_max = out_max;
  a.out_sum = out_sum;
  int sms = 0;
  int rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  const cudaError_t e = sdpa::launch_merge(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"

namespace {

int elem_size(int dtype) { return dtype == ATTN_F32 ? 4 : 2; }

bool is_dtype(int dtype) { return dtype == ATTN_BF16 || dtype == ATTN_F32 || dtype == ATTN_F16; }

// The sizes of a paged cache and its addressing. *page_stride = 0 stands for dense pages.
int page_args(const int32_t* page_table, const int32_t* seq_lens, int B, int Nkv, int D, int num_pages,
              int page_size, int max_pages, int64_t page_stride, int layout, sdpa::PagedArgs* p) {
  if (layout != ATTN_BHSD && layout != ATTN_TND) return ATTN_ERR_INVALID;
  if (B < 0 || Nkv < 1 || Nkv > 256 || D < 1 || D > 768) return ATTN_ERR_INVALID;
  if (num_pages < 0 || page_size < 1 || max_pages < 0) return ATTN_ERR_INVALID;
  const int64_t dense = (int64_t)page_size * Nkv * D;
  if (page_stride != 0 && page_stride < dense) return ATTN_ERR_INVALID;
  if (B > 0 && (seq_lens == nullptr || (page_table == nullptr && max_pages > 0))) return ATTN_ERR_INVALID;
  if ((int64_t)max_pages * page_size > (int64_t(1) << 30)) return ATTN_ERR_UNSUPPORTED;  // positions
  if (B > 1 << 30) return ATTN_ERR_UNSUPPORTED;  // rows are divided and searched in 32-bit integers
  p->page_table = page_table;
  p->seq_lens = seq_lens;
  p->B = B;
  p->num_pages = num_pages;
  p->page_size = page_size;
  p->max_pages = max_pages;
  p->page_stride = page_stride != 0 ? page_stride : dense;
  p->tok_stride = layout == ATTN_TND ? (int64_t)Nkv * D : D;
  p->head_stride = layout == ATTN_TND ? D : (int64_t)page_size * D;
  int l = 0;
  while ((int64_t(1) << l) < page_size) ++l;
  p->div_mul = (uint32_t)((((uint64_t(1) << l) - page_size) << 32) / page_size + 1);
  p->div_shift = l;
  return ATTN_OK;
}

int table_args(int rows, int max_pages, int num_pages) {
  if (rows < 0 || max_pages < 0 || num_pages < 0) return ATTN_ERR_INVALID;
  if (rows > sdpa::kMaxTableRows || (int64_t)rows * max_pages > (int64_t(1) << 29)) return ATTN_ERR_UNSUPPORTED;
  if (num_pages > 1 << 30) return ATTN_ERR_UNSUPPORTED;  // the kernels' walks over the pool count in 32 bits
  return ATTN_OK;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// attn_cache_reserve, and with lens_out and new_lens attn_cache_grow
int reserve_impl(int32_t* page_table, int32_t* ref_count, const int32_t* seq_lens, const int32_t* new_tokens, int B,
                 int max_pages, int num_pages, int page_size, int32_t* copies, int32_t* lens_out, int32_t* new_lens,
                 bool live_only, void* stream) {
  int rc = table_args(B, max_pages, num_pages);
  if (rc != ATTN_OK) return rc;
  if (page_size < 1) return ATTN_ERR_INVALID;
  if ((int64_t)max_pages * page_size > (int64_t(1) << 30)) return ATTN_ERR_UNSUPPORTED;
  if (B == 0) return ATTN_OK;
  if (seq_lens == nullptr || copies == nullptr) return ATTN_ERR_INVALID;
  if (max_pages > 0 && page_table == nullptr) return ATTN_ERR_INVALID;
  if (num_pages > 0 && ref_count == nullptr) return ATTN_ERR_INVALID;
  sdpa::ReserveArgs a{};
  a.table = page_table;
  a.ref = ref_count;
  a.lens = seq_lens;
  a.new_tokens = new_tokens;
  a.copies = copies;
  a.lens_out = lens_out;
  a.new_lens = new_lens;
  a.live_only = live_only;
  a.B = B;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page_size = page_size;
  int sms = 0;
  rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_reserve(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int attn_decode_workspace_size(int Nq, int Nkv, int D, int dtype, int64_t* bytes) {
  if (bytes == nullptr || !is_dtype(dtype)) return ATTN_ERR_INVALID;
  if (Nq < 1 || Nq > 256 || Nkv < 1 || Nq % Nkv != 0 || D < 1 || D > 768) return ATTN_ERR_INVALID;
  if (D > 256) return ATTN_ERR_UNSUPPORTED;
  *bytes = sdpa::decode_workspace_bytes(sdpa::decode_rows(dtype, Nq, Nkv, D), D);
  return ATTN_OK;
}

int attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                      const int32_t* seq_lens, int B, int Nq, int Nkv, int D, int num_pages, int page_size,
                      int max_pages, int64_t page_stride, float scale, int64_t window_tokens,
                      int64_t sink_tokens, int dtype, int layout, void* workspace, int64_t workspace_bytes,
                      void* out, float* softmax_max, float* softmax_sum, void* stream) {
  if (!is_dtype(dtype)) return ATTN_ERR_INVALID;
  sdpa::DecodeArgs a{};
  int rc = page_args(page_table, seq_lens, B, Nkv, D, num_pages, page_size, max_pages, page_stride, layout, &a.p);
  if (rc != ATTN_OK) return rc;
  if (window_tokens < 1 || sink_tokens < 0) return ATTN_ERR_INVALID;
  if (!(scale > 0.f) || scale == INFINITY) return ATTN_ERR_INVALID;
  if ((softmax_max == nullptr) != (softmax_sum == nullptr)) return ATTN_ERR_INVALID;
  int64_t need = 0;
  rc = attn_decode_workspace_size(Nq, Nkv, D, dtype, &need);
  if (rc != ATTN_OK) return rc;
  if (B == 0) return ATTN_OK;
  if (q == nullptr || out == nullptr || workspace == nullptr) return ATTN_ERR_INVALID;
  if (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return ATTN_ERR_INVALID;
  if (workspace_bytes < need || !aligned16(workspace)) return ATTN_ERR_INVALID;
  a.rows = sdpa::decode_rows(dtype, Nq, Nkv, D);
  a.groups = (Nq / Nkv + a.rows - 1) / a.rows;
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.Nq = Nq;
  a.Nkv = Nkv;
  a.D = D;
  a.dtype = dtype;
  a.scale = scale;
  a.window = clamp30(window_tokens);
  a.sinks = clamp30(sink_tokens);
  a.ctr = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(a.ctr + 2 * sdpa::kDecodeMaxCtas);
  a.out = out;
  a.smax = softmax_max;
  a.ssum = softmax_sum;
  rc = device_state(&a.status, &a.num_sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

int attn_cache_append(const void* k, const void* v, const int32_t* page_table, const int32_t* seq_lens,
                      const int32_t* cu_seqlens, int T, int B, int Nkv, int D, int num_pages, int page_size,
                      int max_pages, int64_t page_stride, int dtype, int layout, void* k_cache, void* v_cache,
                      void* stream) {
  if (!is_dtype(dtype)) return ATTN_ERR_INVALID;
  sdpa::AppendArgs a{};
  int rc = page_args(page_table, seq_lens, B, Nkv, D, num_pages, page_size, max_pages, page_stride, layout, &a.p);
  if (rc != ATTN_OK) return rc;
  if (T < 0 || (cu_seqlens == nullptr && T != B)) return ATTN_ERR_INVALID;
  if (T > 1 << 30) return ATTN_ERR_UNSUPPORTED;  // the kernel steps over the tokens in 32-bit integers
  if (T == 0) return ATTN_OK;
  if (B == 0) return ATTN_ERR_INVALID;
  if (k == nullptr || v == nullptr || k_cache == nullptr || v_cache == nullptr) return ATTN_ERR_INVALID;
  a.k_new = k;
  a.v_new = v;
  a.cu = cu_seqlens;
  a.T = T;
  a.Nkv = Nkv;
  a.D = D;
  a.dtype = dtype;
  a.k = k_cache;
  a.v = v_cache;
  rc = device_state(&a.status, &a.num_sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

int attn_cache_fork(const int32_t* page_table, const int32_t* src_rows, const int32_t* ref_count,
                    const int32_t* seq_lens, int rows_in, int rows_out, int max_pages, int num_pages,
                    int32_t* page_table_out, int32_t* ref_count_out, int32_t* seq_lens_out, void* stream) {
  int rc = table_args(rows_in, max_pages, num_pages);
  if (rc == ATTN_OK) rc = table_args(rows_out, max_pages, num_pages);
  if (rc != ATTN_OK) return rc;
  if ((seq_lens == nullptr) != (seq_lens_out == nullptr)) return ATTN_ERR_INVALID;
  if (max_pages < 1) return ATTN_ERR_INVALID;
  if (page_table_out != nullptr && page_table_out == page_table && rows_in != rows_out) return ATTN_ERR_INVALID;
  if (rows_in > 0 && page_table == nullptr) return ATTN_ERR_INVALID;
  if (rows_out > 0 && (src_rows == nullptr || page_table_out == nullptr)) return ATTN_ERR_INVALID;
  if (num_pages > 0 && (ref_count == nullptr || ref_count_out == nullptr)) return ATTN_ERR_INVALID;
  sdpa::ForkArgs a{};
  a.table = page_table;
  a.src = src_rows;
  a.ref = ref_count;
  a.lens = seq_lens;
  a.rows_in = rows_in;
  a.rows_out = rows_out;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.table_out = page_table_out;
  a.ref_out = ref_count_out;
  a.lens_out = seq_lens_out;
  int sms = 0;
  rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_fork(a, static_cast<cudaStream_t>(stream)));
}

int attn_cache_reserve(int32_t* page_table, int32_t* ref_count, const int32_t* seq_lens,
                       const int32_t* new_tokens, int B, int max_pages, int num_pages, int page_size,
                       int32_t* copies, void* stream) {
  return reserve_impl(page_table, ref_count, seq_lens, new_tokens, B, max_pages, num_pages, page_size, copies,
                      nullptr, nullptr, false, stream);
}

int attn_cache_grow(int32_t* page_table, int32_t* ref_count, int32_t* seq_lens, const int32_t* new_tokens,
                    int live_only, int B, int max_pages, int num_pages, int page_size, int32_t* copies,
                    int32_t* new_lens, void* stream) {
  if (live_only != 0 && live_only != 1) return ATTN_ERR_INVALID;
  if (B > 0 && (new_lens == nullptr || new_lens == seq_lens || new_lens == new_tokens)) return ATTN_ERR_INVALID;
  return reserve_impl(page_table, ref_count, seq_lens, new_tokens, B, max_pages, num_pages, page_size, copies,
                      seq_lens, new_lens, live_only != 0, stream);
}

int attn_cache_evict(int32_t* page_table, int32_t* ref_count, const int32_t* seq_lens, int B, int max_pages,
                     int num_pages, int page_size, int64_t window_tokens, int64_t sink_tokens, void* stream) {
  int rc = table_args(B, max_pages, num_pages);
  if (rc != ATTN_OK) return rc;
  if (page_size < 1 || window_tokens < 1 || sink_tokens < 0) return ATTN_ERR_INVALID;
  if ((int64_t)max_pages * page_size > (int64_t(1) << 30)) return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)B * max_pages == 0) return ATTN_OK;
  if (seq_lens == nullptr || page_table == nullptr) return ATTN_ERR_INVALID;
  if (num_pages > 0 && ref_count == nullptr) return ATTN_ERR_INVALID;
  sdpa::EvictArgs a{};
  a.table = page_table;
  a.ref = ref_count;
  a.lens = seq_lens;
  a.B = B;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.window = clamp30(window_tokens);
  a.sinks = clamp30(sink_tokens);
  int sms = 0;
  rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_evict(a, static_cast<cudaStream_t>(stream)));
}

int attn_cache_compact(const int32_t* page_table, const int32_t* ref_count, int rows, int max_pages,
                       int num_pages, int32_t* page_table_out, int32_t* ref_count_out, int32_t* page_map,
                       int32_t* copies, int32_t* live_pages, void* stream) {
  const int rc0 = table_args(rows, max_pages, num_pages);
  if (rc0 != ATTN_OK) return rc0;
  const int64_t n = (int64_t)rows * max_pages;
  if (live_pages == nullptr) return ATTN_ERR_INVALID;
  if (n > 0 && (page_table == nullptr || page_table_out == nullptr)) return ATTN_ERR_INVALID;
  if (num_pages > 0 && (ref_count == nullptr || ref_count_out == nullptr || page_map == nullptr))
    return ATTN_ERR_INVALID;
  if (num_pages > 1 && copies == nullptr) return ATTN_ERR_INVALID;
  sdpa::CompactArgs a{};
  a.table = page_table;
  a.ref = ref_count;
  a.rows = rows;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.table_out = page_table_out;
  a.ref_out = ref_count_out;
  a.page_map = page_map;
  a.copies = copies;
  a.live = live_pages;
  int sms = 0;
  const int rc = device_state(&a.status, &sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_compact(a, static_cast<cudaStream_t>(stream)));
}

int attn_cache_copy(const int32_t* copies, int n_copies, int num_pages, int64_t page_elems, int64_t page_stride,
                    int dtype, void* k_cache, void* v_cache, void* stream) {
  if (!is_dtype(dtype)) return ATTN_ERR_INVALID;
  if (n_copies < 0 || num_pages < 0 || page_elems < 1) return ATTN_ERR_INVALID;
  if (page_stride != 0 && page_stride < page_elems) return ATTN_ERR_INVALID;
  if (n_copies == 0) return ATTN_OK;
  if (copies == nullptr || (reinterpret_cast<uintptr_t>(copies) & 7u) != 0) return ATTN_ERR_INVALID;
  if (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return ATTN_ERR_INVALID;
  if (page_elems > (int64_t(1) << 34)) return ATTN_ERR_UNSUPPORTED;
  const int64_t es = elem_size(dtype);
  sdpa::PageCopyArgs a{};
  a.copies = copies;
  a.n = n_copies;
  a.num_pages = num_pages;
  a.page_bytes = page_elems * es;
  a.stride_bytes = (page_stride != 0 ? page_stride : page_elems) * es;
  a.k = k_cache;
  a.v = v_cache;
  const int rc = device_state(&a.status, &a.num_sms);
  if (rc != ATTN_OK) return rc;
  return from_cuda(sdpa::launch_cache_copy(a, static_cast<cudaStream_t>(stream)));
}

int attn_get_last_error(void* stream, int* device_status) {
  if (device_status == nullptr) return ATTN_ERR_INVALID;
  int* word = nullptr;
  int* slot = nullptr;
  int sms = 0, dev = 0;
  int rc = device_state(&word, &sms, &slot, &dev);
  if (rc != ATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lk(g_read_mu[dev]);
  int host = 0;
  read_and_clear_status<<<1, 1, 0, st>>>(word, slot);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (cudaMemcpyAsync(&host, slot, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return ATTN_ERR_CUDA;
  *device_status = host;
  return ATTN_OK;
}

}  // extern "C"
