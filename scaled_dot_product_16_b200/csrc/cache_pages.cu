// cache_pages.cu -- the pages of a key/value cache: writing new tokens into them, and the bookkeeping
// that forks, frees, reserves and compacts them.
//
// The state is a page table [rows, max_pages] (-1: no page) and a reference count per page (0: free).
// Everything is decided on the device from these arrays, so a serving step never waits for the host
// and can be captured into a graph. All arithmetic on them is on integers, so the order of atomics
// does not change a result; pages are handed out lowest index first in the order of rows and columns.
// Which pages' contents have to move is returned as a list of (source, destination) pairs that
// attn_cache_copy carries out, once for each layer that shares the page table.
#include "paged.cuh"

namespace sdpa {
namespace {

// ---- attn_cache_append ---------------------------------------------------------------------------
// A warp writes one token's key and value rows (all heads), in vectors of type V. Bound by HBM for
// whole prompts (each new element is read and written once), by latency for one token per row.
constexpr int kAppendWarps = 4;

template <typename V>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(AppendArgs a, int vec_per_head) {
  const int lane = threadIdx.x & 31;
  const int n_warps = gridDim.x * kAppendWarps;
  if (a.cu != nullptr && blockIdx.x == 0) {
    // the cumulative lengths as a whole: non-decreasing, ending at T
    for (int b = threadIdx.x; b < a.p.B; b += blockDim.x) {
      const int lo = b == 0 ? 0 : __ldg(a.cu + b - 1), hi = __ldg(a.cu + b);
      if (hi < lo || (b == a.p.B - 1 && hi != a.T)) report(a.status, ATTN_ERR_DATA);
    }
  }
  const V* kn = static_cast<const V*>(a.k_new);
  const V* vn = static_cast<const V*>(a.v_new);
  V* kc = static_cast<V*>(a.k);
  V* vc = static_cast<V*>(a.v);
  const int per_row = a.Nkv * vec_per_head;
  for (int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5); t < a.T; t += n_warps) {
    int b = t, left = 1;  // row of token t; tokens of the row from t on
    if (a.cu != nullptr) {
      int lo = 0, hi = a.p.B;  // first row whose end lies behind t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid + 1;
        else hi = mid;
      }
      b = lo;
      if (b == a.p.B) continue;  // behind the last row: reported above
      left = __ldg(a.cu + b) - t;
    }
    const int64_t pos = (int64_t)__ldg(a.p.seq_lens + b) - left;
    if (pos < 0 || pos >= (int64_t)a.p.max_pages * a.p.page_size) {
      if (lane == 0) report(a.status, ATTN_ERR_DATA);
      continue;
    }
    const int pi = page_of(a.p, (int)pos);
    const int page = __ldg(a.p.page_table + (int64_t)b * a.p.max_pages + pi);
    if (page < 0 || page >= a.p.num_pages) {
      if (lane == 0) report(a.status, ATTN_ERR_DATA);
      continue;
    }
    // strides in vectors here
    const int64_t at = page * a.p.page_stride + ((int)pos - pi * a.p.page_size) * a.p.tok_stride;
    const int64_t from = (int64_t)t * per_row;
    for (int x = lane; x < per_row; x += 32) {
      const int h = x / vec_per_head;
      const int64_t to = at + h * a.p.head_stride + (x - h * vec_per_head);
      kc[to] = kn[from + x];
      vc[to] = vn[from + x];
    }
  }
}

template <typename V>
cudaError_t launch_append(AppendArgs a, int es, cudaStream_t st) {
  const int per = (int)sizeof(V) / es;
  a.p.page_stride /= per;
  a.p.tok_stride /= per;
  a.p.head_stride /= per;
  const int blocks = min((a.T + kAppendWarps - 1) / kAppendWarps, a.num_sms * 16);
  append_kernel<V><<<blocks, kAppendWarps * 32, 0, st>>>(a, a.D / per);
  return cudaGetLastError();
}

// ---- attn_cache_copy -----------------------------------------------------------------------------
// Each block takes (pair, chunk) items in turn; bound by HBM (a page's bytes read and written once).
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // vectors a thread holds at once

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(PageCopyArgs a, int64_t page_vecs, int64_t stride_vecs,
                                                            int chunks) {
  const int64_t items = (int64_t)a.n * chunks;
  for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
    const int pair = (int)(x / chunks);
    const int64_t v0 = (x - (int64_t)pair * chunks) * (kCopyThreads * kCopyVecs) + threadIdx.x;
    const int2 sd = __ldg(reinterpret_cast<const int2*>(a.copies) + pair);
    if (sd.x < 0 && sd.y < 0) continue;  // an unused pair
    if (sd.x < 0 || sd.y < 0 || sd.x >= a.num_pages || sd.y >= a.num_pages) {
      if (threadIdx.x == 0) report(a.status, ATTN_ERR_DATA);
      continue;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      V* base = static_cast<V*>(kv == 0 ? a.k : a.v);
      const V* src = base + sd.x * stride_vecs;
      V* dst = base + sd.y * stride_vecs;
      V r[kCopyVecs];
#pragma unroll
      for (int i = 0; i < kCopyVecs; ++i)
        if (v0 + i * kCopyThreads < page_vecs) r[i] = src[v0 + i * kCopyThreads];
#pragma unroll
      for (int i = 0; i < kCopyVecs; ++i)
        if (v0 + i * kCopyThreads < page_vecs) dst[v0 + i * kCopyThreads] = r[i];
    }
  }
}

template <typename V>
cudaError_t launch_copy(const PageCopyArgs& a, cudaStream_t st) {
  const int64_t vecs = a.page_bytes / (int64_t)sizeof(V);
  const int64_t per = kCopyThreads * kCopyVecs;
  const int64_t chunks = (vecs + per - 1) / per;
  const int64_t items = a.n * chunks;
  const int blocks = (int)(items < a.num_sms * 8LL ? items : a.num_sms * 8LL);
  copy_kernel<V><<<blocks, kCopyThreads, 0, st>>>(a, vecs, a.stride_bytes / (int64_t)sizeof(V), (int)chunks);
  return cudaGetLastError();
}

// ---- attn_cache_fork -----------------------------------------------------------------------------
// Row r of the new table is row src[r] of the old one (or empty). A page's count changes by
// (children of the row - 1) for each row that holds it. A block owns a range of columns: it reads
// them for all rows before it writes them, so the new table may be the old one.
constexpr int kForkThreads = 256;
constexpr int kForkEntries = 8192;  // staged entries per block

__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkArgs a, int cols) {
  extern __shared__ int32_t sm[];
  int32_t* kids = sm;               // [rows_in] rows that take this one's pages
  int32_t* old = sm + a.rows_in;    // [rows_in][cols]
  const int c0 = blockIdx.x * cols, nc = min(cols, a.max_pages - c0);
  for (int r = threadIdx.x; r < a.rows_in; r += kForkThreads) kids[r] = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < a.rows_out; r += kForkThreads) {
    const int s = __ldg(a.src + r);
    if (s >= 0 && s < a.rows_in) atomicAdd(kids + s, 1);
    else if (s >= a.rows_in && blockIdx.x == 0) report(a.status, ATTN_ERR_DATA);
  }
  for (int x = threadIdx.x; x < a.rows_in * nc; x += kForkThreads) {
    const int r = x / nc, c = x - r * nc;
    old[r * cols + c] = a.table[(int64_t)r * a.max_pages + c0 + c];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < a.rows_in * nc; x += kForkThreads) {
    const int r = x / nc, c = x - r * nc;
    const int page = old[r * cols + c];
    if (page >= a.num_pages) {
      report(a.status, ATTN_ERR_DATA);
      old[r * cols + c] = -1;
    } else if (page >= 0 && kids[r] != 1) {
      atomicAdd(a.ref_out + page, kids[r] - 1);
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < a.rows_out * nc; x += kForkThreads) {
    const int r = x / nc, c = x - r * nc;
    const int s = __ldg(a.src + r);
    a.table_out[(int64_t)r * a.max_pages + c0 + c] = s >= 0 && s < a.rows_in ? old[s * cols + c] : -1;
  }
  if (blockIdx.x == 0 && a.lens != nullptr) {
    __syncthreads();
    for (int r = threadIdx.x; r < a.rows_in; r += kForkThreads) kids[r] = a.lens[r];
    __syncthreads();
    for (int r = threadIdx.x; r < a.rows_out; r += kForkThreads) {
      const int s = __ldg(a.src + r);
      a.lens_out[r] = s >= 0 && s < a.rows_in ? kids[s] : 0;
    }
  }
}

// ---- attn_cache_reserve --------------------------------------------------------------------------
// One block. A slot is a (row, column) whose page the row's next tokens go to: it needs a free page
// if it has none, or if its page is shared (count > 1). Where every holder of a page asks for it in
// the same call the first of them, in slot order, keeps it. Nothing is changed unless enough pages
// are free.
//
// The counts themselves carry the bookkeeping between the passes (all counts are below 2^17 and there
// are at most 8192 slots of one page, one per row): every asking slot takes 2^17 off its shared page's
// count, which makes it negative and keeps both the count and the number k of askers readable; where
// k is the count, the slots replace it by the smallest of -2^31 + slot, below every such value.
constexpr int kResThreads = 1024;
constexpr int kResWarps = kResThreads / 32;
constexpr int kAsk = 1 << 17;
constexpr int kOwned = -(1 << 30);  // below: the keeper's slot; kOwned and above, negative: asked for

struct ResSmem {
  int warp[kResWarps];
  int bad;
  int taken;   // free pages found so far
  int free_page[kResThreads];
};

// Exclusive prefix sum over the block; *total gets the sum. Ends with a barrier before reuse of w.
__device__ __forceinline__ int block_scan(int v, int* w, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) w[warp] = incl;
  __syncthreads();
  int before = 0, sum = 0;
  for (int i = 0; i < kResWarps; ++i) {
    if (i < warp) before += w[i];
    sum += w[i];
  }
  __syncthreads();
  *total = sum;
  return before + incl - v;
}

__global__ void __launch_bounds__(kResThreads) reserve_kernel(ReserveArgs a) {
  __shared__ ResSmem s;
  extern __shared__ int32_t prefix[];  // [B] first slot of each row
  const int tid = threadIdx.x;
  if (tid == 0) {
    s.bad = 0;
    s.taken = 0;
  }
  __syncthreads();
  auto span = [&](int b, int* start, int* i0) -> int {  // slots of row b
    const int len = a.lens[b], add = a.new_tokens != nullptr ? a.new_tokens[b] : 1;
    if (add < 0 || len < add || (int64_t)len > (int64_t)a.max_pages * a.page_size) {
      s.bad = 1;
      return 0;
    }
    *start = len - add;
    *i0 = *start / a.page_size;
    return add == 0 ? 0 : (len - 1) / a.page_size - *i0 + 1;
  };
  // the slots of each row, and the first slot of it
  int slots = 0;
  for (int b0 = 0; b0 < a.B; b0 += kResThreads) {
    const int b = b0 + tid;
    int start = 0, i0 = 0, n = 0, sum;
    if (b < a.B) n = span(b, &start, &i0);
    const int before = block_scan(n, s.warp, &sum);
    if (b < a.B) {
      prefix[b] = slots + before;
      a.copies[2 * b] = a.copies[2 * b + 1] = -1;
    }
    slots += sum;
  }
  __syncthreads();
  if (s.bad) {
    if (tid == 0) report(a.status, ATTN_ERR_DATA);
    return;
  }
  auto entry = [&](int slot, int* b, int* i) -> int32_t* {  // table entry of a slot
    int lo = 0, hi = a.B;  // the last row that begins at or before the slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= slot) lo = mid;
      else hi = mid;
    }
    int start = 0, i0 = 0;
    span(lo, &start, &i0);
    *b = lo;
    *i = i0 + slot - prefix[lo];
    return a.table + (int64_t)lo * a.max_pages + *i;
  };
  int b, i;
  // 1: every slot of a shared page asks for it
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *entry(x, &b, &i);
    if (page >= a.num_pages) s.bad = 1;
    else if (page >= 0 && a.ref[page] != 1) {
      // a page that is held has a count; 0 here would be handed out a second time
      if (a.ref[page] == 0) s.bad = 1;
      else atomicSub(a.ref + page, kAsk);
    }
  }
  __syncthreads();
  // 2: where all holders ask, the first slot owns the page
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *entry(x, &b, &i);
    if (page < 0 || page >= a.num_pages) continue;
    const int v = *(volatile int32_t*)(a.ref + page);
    if (v >= 0) continue;
    const int k = (-v + kAsk - 1) / kAsk;
    if (v < kOwned || v + k * kAsk == k) atomicMin(a.ref + page, INT32_MIN + x);
    else if (v + k * kAsk < k) s.bad = 1;  // more rows hold the page than its count says
  }
  __syncthreads();
  // 3: how many pages are needed, and whether that many are free
  int needed = 0;
  for (int x0 = 0; x0 < slots; x0 += kResThreads) {
    const int x = x0 + tid;
    int need = 0, sum;
    if (x < slots) {
      const int page = *entry(x, &b, &i);
      if (page < 0) need = 1;
      else if (page < a.num_pages) {
        const int v = a.ref[page];
        need = v < 0 && v != INT32_MIN + x;
      }
    }
    block_scan(need, s.warp, &sum);
    needed += sum;
  }
  int have = 0;
  for (int p0 = 0; p0 < a.num_pages && have < needed; p0 += kResThreads) {
    int sum;
    block_scan(p0 + tid < a.num_pages && a.ref[p0 + tid] == 0, s.warp, &sum);
    have += sum;
  }
  __syncthreads();
  if (s.bad || have < needed) {
    // undo: an owned page's count is the number of slots that ask for it
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *entry(x, &b, &i);
      if (page >= 0 && page < a.num_pages && a.ref[page] == INT32_MIN + x) a.ref[page] = INT32_MIN;
    }
    __syncthreads();
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *entry(x, &b, &i);
      if (page < 0 || page >= a.num_pages) continue;
      const int v = *(volatile int32_t*)(a.ref + page);
      if (v < kOwned) atomicAdd(a.ref + page, 1);
      else if (v < 0) atomicAdd(a.ref + page, kAsk);
    }
    __syncthreads();
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *entry(x, &b, &i);
      if (page >= 0 && page < a.num_pages && a.ref[page] < kOwned) atomicAnd(a.ref + page, INT32_MAX);
    }
    if (tid == 0) report(a.status, s.bad ? ATTN_ERR_DATA : ATTN_ERR_PAGES);
    return;
  }
  // 4: hand out the pages, kResThreads slots at a time
  int p0 = 0;  // pages below it have been looked at
  for (int x0 = 0; x0 < slots; x0 += kResThreads) {
    const int x = x0 + tid;
    int need = 0, v = 0, page = -1, sum;
    int32_t* e = nullptr;
    if (x < slots) {
      e = entry(x, &b, &i);
      page = *e;
      if (page >= 0) v = a.ref[page];
      need = page < 0 || (v < 0 && v != INT32_MIN + x);
    }
    const int rank = block_scan(need, s.warp, &sum);
    // the next `sum` free pages, in order; a page found but not needed here is found again
    int found = 0;
    while (found < sum && p0 < a.num_pages) {
      const bool is_free = p0 + tid < a.num_pages && a.ref[p0 + tid] == 0;
      int n;
      const int at = found + block_scan(is_free, s.warp, &n);
      if (is_free && at < sum) {
        s.free_page[at] = p0 + tid;
        a.ref[p0 + tid] = 1;
      }
      found += n;
      if (found <= sum) p0 += kResThreads;
      __syncthreads();
    }
    __syncthreads();
    if (need) {
      const int to = s.free_page[rank];
      *e = to;
      if (page >= 0) {
        if (v >= kOwned) atomicAdd(a.ref + page, kAsk - 1);
        int start = 0, i0 = 0;
        span(b, &start, &i0);
        // only the first page of a row's slots can hold earlier tokens
        if (i == i0 && start % a.page_size != 0) {
          a.copies[2 * b] = page;
          a.copies[2 * b + 1] = to;
        }
      }
    }
    __syncthreads();
  }
  // 5: a kept page has one holder
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *entry(x, &b, &i);
    if (a.ref[page] == INT32_MIN + x) a.ref[page] = 1;
  }
}

// ---- attn_cache_compact --------------------------------------------------------------------------
// One block scans the counts: with n live pages, the k-th live page at or above n moves to the k-th
// free page below n. A second kernel renames the pages in the table.
__global__ void __launch_bounds__(kResThreads) compact_kernel(CompactArgs a) {
  __shared__ int w[kResWarps];
  const int tid = threadIdx.x;
  const int pairs = a.num_pages / 2;
  int live = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kResThreads) {
    int sum;
    block_scan(p0 + tid < a.num_pages && a.ref[p0 + tid] > 0, w, &sum);
    live += sum;
  }
  int holes = 0, moved = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kResThreads) {
    const int p = p0 + tid;
    const int ref = p < a.num_pages ? a.ref[p] : 0;
    const bool hole = p < live && ref <= 0, high = p >= live && ref > 0;
    int nh, nm;
    const int h = holes + block_scan(hole, w, &nh);
    const int m = moved + block_scan(high, w, &nm);
    if (hole) a.copies[2 * h + 1] = p;
    __syncthreads();  // the holes of these pages are listed before their movers look them up
    if (p < a.num_pages) {
      if (high) {
        const int to = *(volatile int32_t*)(a.copies + 2 * m + 1);
        a.copies[2 * m] = p;
        a.page_map[p] = to;
        a.ref_out[to] = ref;
        a.ref_out[p] = 0;
      } else {
        a.page_map[p] = ref > 0 ? p : -1;
        if (!hole) a.ref_out[p] = ref > 0 ? ref : 0;  // a hole's count is its mover's
      }
    }
    holes += nh;
    moved += nm;
  }
  for (int x = moved + tid; x < pairs; x += kResThreads) a.copies[2 * x] = a.copies[2 * x + 1] = -1;
  if (tid == 0) *a.live = live;
}

__global__ void __launch_bounds__(256) rename_kernel(CompactArgs a, int64_t n) {
  for (int64_t x = blockIdx.x * 256LL + threadIdx.x; x < n; x += gridDim.x * 256LL) {
    const int page = a.table[x];
    int to = -1;
    if (page >= 0) {
      if (page < a.num_pages) to = a.page_map[page];
      if (to < 0) report(a.status, ATTN_ERR_DATA);  // a page outside the pool, or one without a count
    }
    a.table_out[x] = to;
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  const int es = a.dtype == ATTN_F32 ? 4 : 2;
  const uintptr_t bases = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new) |
                          reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  // 16-byte vectors where every row starts on one
  if (((bases | (uintptr_t)(a.p.page_stride * es) | (uintptr_t)((int64_t)a.D * es)) & 15u) == 0)
    return launch_append<uint4>(a, es, st);
  return es == 4 ? launch_append<uint32_t>(a, es, st) : launch_append<uint16_t>(a, es, st);
}

cudaError_t launch_cache_copy(const PageCopyArgs& a, cudaStream_t st) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        (uintptr_t)a.page_bytes | (uintptr_t)a.stride_bytes;
  return (all & 15u) == 0 ? launch_copy<uint4>(a, st) : launch_copy<uint16_t>(a, st);
}

cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t st) {
  if (a.ref_out != a.ref) {
    const cudaError_t e = cudaMemcpyAsync(a.ref_out, a.ref, sizeof(int32_t) * (size_t)a.num_pages,
                                          cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
  }
  const int rows = a.rows_in > 0 ? a.rows_in : 1;
  int cols = kForkEntries / rows;
  cols = cols < 1 ? 1 : (cols > 32 ? 32 : cols);
  const int smem = (int)sizeof(int32_t) * (a.rows_in + a.rows_in * cols);
  cudaError_t e = cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fork_kernel<<<(a.max_pages + cols - 1) / cols, kForkThreads, smem, st>>>(a, cols);
  return cudaGetLastError();
}

cudaError_t launch_cache_reserve(const ReserveArgs& a, cudaStream_t st) {
  reserve_kernel<<<1, kResThreads, sizeof(int32_t) * a.B, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  compact_kernel<<<1, kResThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  const int64_t n = (int64_t)a.rows * a.max_pages;
  if (e != cudaSuccess || n == 0) return e;
  const int64_t blocks = (n + 255) / 256;
  rename_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, st>>>(a, n);
  return cudaGetLastError();
}

}  // namespace sdpa
