// cache_pages.cu -- the pages of a key/value cache: writing new tokens into them, and the bookkeeping
// that forks, frees, reserves, evicts and compacts them.
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
constexpr int kAppendVecs = 4;  // vectors a lane holds of each of k and v

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
    // the first vectors of the token are on their way while its place is looked up
    const V* ks = kn + (int64_t)t * per_row;
    const V* vs = vn + (int64_t)t * per_row;
    V rk[kAppendVecs], rv[kAppendVecs];
    auto load = [&](int x0) {
#pragma unroll
      for (int i = 0; i < kAppendVecs; ++i)
        if (x0 + 32 * i < per_row) {
          rk[i] = ks[x0 + 32 * i];
          rv[i] = vs[x0 + 32 * i];
        }
    };
    load(lane);
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
    const int len = __ldg(a.p.seq_lens + b);
    if (len == 0) continue;  // no new tokens after all (attn_cache_grow)
    const int64_t pos = (int64_t)len - left;
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
    for (int x0 = lane; x0 < per_row; x0 += 32 * kAppendVecs) {
      if (x0 != lane) load(x0);
#pragma unroll
      for (int i = 0; i < kAppendVecs; ++i) {
        const int x = x0 + 32 * i;
        if (x < per_row) {
          const int h = x / vec_per_head;
          const int64_t to = at + h * a.p.head_stride + (x - h * vec_per_head);
          kc[to] = rk[i];
          vc[to] = rv[i];
        }
      }
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
constexpr int kCopyVecs = 8;  // vectors a thread holds of each of k and v

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
    const V* ks = static_cast<const V*>(a.k) + sd.x * stride_vecs;
    const V* vs = static_cast<const V*>(a.v) + sd.x * stride_vecs;
    V* kd = static_cast<V*>(a.k) + sd.y * stride_vecs;
    V* vd = static_cast<V*>(a.v) + sd.y * stride_vecs;
    V rk[kCopyVecs], rv[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (v0 + i * kCopyThreads < page_vecs) {
        rk[i] = ks[v0 + i * kCopyThreads];
        rv[i] = vs[v0 + i * kCopyThreads];
      }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (v0 + i * kCopyThreads < page_vecs) {
        kd[v0 + i * kCopyThreads] = rk[i];
        vd[v0 + i * kCopyThreads] = rv[i];
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
constexpr int kForkEntries = 1024;  // staged entries per block, where a column has no more

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
// are free. attn_cache_grow is the same with the lengths kept here too, so that what follows on the device (append)
// can tell a step that was refused.
//
// The counts themselves carry the bookkeeping between the passes (a count is at most kMaxCount, and at most kMaxAsk
// slots may ask for one page: one for each row a table can have): every asking slot takes 2^17 off its shared page's
// count, which makes it negative and keeps both the count and the number k of askers readable; where
// k is the count, the slots replace it by the smallest of -2^31 + slot, below every such value.
constexpr int kResThreads = 1024;
constexpr int kResWarps = kResThreads / 32;
constexpr int kAsk = 1 << 17;
constexpr int kMaxCount = 1 << 16;
constexpr int kMaxAsk = kMaxTableRows;
static_assert(kMaxAsk * (int64_t)kAsk == 1 << 30 && kMaxCount < kAsk, "counts less what kMaxAsk slots take stay above kOwned");
constexpr int kOwned = -(1 << 30);  // below: the keeper's slot; kOwned and above, negative: asked for

struct ResSmem {
  int warp[kResWarps];
  int bad;
  int free_page[kResThreads];
};

// Exclusive prefix sum over the block; *total gets the sum. w [kResWarps] may be used again at once.
__device__ __forceinline__ int block_scan(int v, int* w, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();  // the last scan's sums have been read
  if (lane == 31) w[warp] = incl;
  __syncthreads();
  int sums = w[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += t;
  }
  *total = __shfl_sync(0xffffffffu, sums, 31);
  const int before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + incl - v;
}

// kScan counts in a row per thread (beyond n: fill).
constexpr int kScan = 8;
__device__ __forceinline__ void load_counts(const int32_t* ref, int p, int n, int fill, int (&r)[kScan]) {
  if (p + kScan <= n && (reinterpret_cast<uintptr_t>(ref) & 15u) == 0) {  // p is a multiple of kScan
#pragma unroll
    for (int i = 0; i < kScan; i += 4) *reinterpret_cast<int4*>(r + i) = *reinterpret_cast<const int4*>(ref + p + i);
  } else {
#pragma unroll
    for (int i = 0; i < kScan; ++i) r[i] = p + i < n ? ref[p + i] : fill;
  }
}

// GROW: attn_cache_grow, whose lengths come without the new tokens.
template <bool GROW>
__global__ void __launch_bounds__(kResThreads, 1) reserve_kernel(ReserveArgs a) {
  __shared__ ResSmem s;
  extern __shared__ int32_t prefix[];  // [B] first slot of each row
  const int tid = threadIdx.x;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  auto added = [&](int b) -> int {
    return a.new_tokens != nullptr ? a.new_tokens[b] : GROW && a.live_only ? a.lens[b] > 0 : 1;
  };
  auto span = [&](int b, int* start, int* i0) -> int {  // slots of row b
    const int add = added(b);
    const int64_t first = GROW ? (int64_t)a.lens[b] : (int64_t)a.lens[b] - add;
    if (add < 0 || first < 0 || first + add > (int64_t)a.max_pages * a.page_size) {
      s.bad = 1;
      return 0;
    }
    *start = (int)first;
    *i0 = *start / a.page_size;
    return add == 0 ? 0 : (*start + add - 1) / a.page_size - *i0 + 1;
  };
  auto refuse = [&](int status) {
    if (tid == 0) report(a.status, status);
    if constexpr (GROW)
      for (int b = tid; b < a.B; b += kResThreads) a.new_lens[b] = 0;
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
    refuse(ATTN_ERR_DATA);
    return;
  }
  // A slot: its row and table entry, and whether an earlier token of the row lies in its page. Each
  // thread keeps its first one (with one token per row there is no other).
  struct Slot {
    int b;
    bool partial;
    int32_t* e;
  };
  auto find = [&](int slot) -> Slot {
    int lo = 0, hi = a.B;  // the last row that begins at or before the slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= slot) lo = mid;
      else hi = mid;
    }
    int start = 0, i0 = 0;
    span(lo, &start, &i0);
    const int i = i0 + slot - prefix[lo];
    return {lo, i == i0 && start != i0 * a.page_size, a.table + (int64_t)lo * a.max_pages + i};
  };
  Slot mine{0, false, nullptr};
  if (tid < slots) mine = find(tid);
  auto slot_at = [&](int x) -> Slot { return x == tid ? mine : find(x); };
  // 0: every entry is a page or none, and every page has a count (one that is held with a count of 0
  // would be handed out a second time)
  bool mine_shared = false;
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *slot_at(x).e;
    if (page < 0) continue;
    const int v = page < a.num_pages ? a.ref[page] : 0;
    if (v < 1 || v > kMaxCount) s.bad = 1;
    if (x == tid) mine_shared = v > 1;
  }
  __syncthreads();
  if (s.bad) {
    refuse(ATTN_ERR_DATA);
    return;
  }
  // 1: every slot of a shared page asks for it. Only among more than kMaxAsk slots can too many ask for one page
  // (waiting for what the atomics return and for each other took 0.9 us).
  auto asks = [&](int x, int page) -> bool {
    return page >= 0 && (x == tid ? mine_shared : *(volatile int32_t*)(a.ref + page) != 1);
  };
  if (__builtin_expect(slots > kMaxAsk, 0)) {
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *slot_at(x).e;
      if (asks(x, page) && atomicSub(a.ref + page, kAsk) - kAsk <= kOwned) {  // rows hold the page many times
        atomicAdd(a.ref + page, kAsk);
        s.bad = 1;
      }
    }
    __syncthreads();
    if (s.bad) {
      // undo: as many steps for each page as slots asked for it (more of them may hold it)
      for (int x = tid; x < slots; x += kResThreads) {
        const int page = *slot_at(x).e;
        if (page < 0) continue;
        for (int v = *(volatile int32_t*)(a.ref + page); v < 0;) {
          const int was = atomicCAS(a.ref + page, v, v + kAsk);
          if (was == v) break;
          v = was;
        }
      }
      refuse(ATTN_ERR_DATA);
      return;
    }
  } else {
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *slot_at(x).e;
      if (asks(x, page)) atomicSub(a.ref + page, kAsk);
    }
    __syncthreads();
  }
  // 2: where all holders ask, the first slot owns the page
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *slot_at(x).e;
    if (page < 0) continue;
    const int v = *(volatile int32_t*)(a.ref + page);
    if (v >= 0) continue;
    const int k = (-v + kAsk - 1) / kAsk;
    if (v < kOwned || v + k * kAsk == k) atomicMin(a.ref + page, INT32_MIN + x);
    else if (v + k * kAsk < k) s.bad = 1;  // more rows hold the page than its count says
  }
  __syncthreads();
  auto needs = [&](int x, int page) -> bool {  // slot x needs a free page
    if (page < 0) return true;
    const int v = a.ref[page];
    return v < 0 && v != INT32_MIN + x;
  };
  // 3: how many pages are needed, and whether that many are free. The first kResThreads of them are
  // listed on the way.
  int needed = 0;
  for (int x0 = 0; x0 < slots; x0 += kResThreads) {
    const int x = x0 + tid;
    int sum;
    block_scan(x < slots && needs(x, *slot_at(x).e), s.warp, &sum);
    needed += sum;
  }
  int have = 0;
  for (int p0 = 0; p0 < a.num_pages && have < needed; p0 += kResThreads * kScan) {
    int r[kScan], n = 0, sum;
    load_counts(a.ref, p0 + tid * kScan, a.num_pages, 1, r);
#pragma unroll
    for (int i = 0; i < kScan; ++i) n += r[i] == 0;
    int at = have + block_scan(n, s.warp, &sum);
#pragma unroll
    for (int i = 0; i < kScan; ++i)
      if (r[i] == 0) {
        if (at < kResThreads) s.free_page[at] = p0 + tid * kScan + i;
        ++at;
      }
    have += sum;
  }
  __syncthreads();
  if (s.bad || have < needed) {
    // undo: an owned page's count is the number of slots that ask for it
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *slot_at(x).e;
      if (page >= 0 && a.ref[page] == INT32_MIN + x) a.ref[page] = INT32_MIN;
    }
    __syncthreads();
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *slot_at(x).e;
      if (page < 0) continue;
      const int v = *(volatile int32_t*)(a.ref + page);
      if (v < kOwned) atomicAdd(a.ref + page, 1);
      else if (v < 0) atomicAdd(a.ref + page, kAsk);
    }
    __syncthreads();
    for (int x = tid; x < slots; x += kResThreads) {
      const int page = *slot_at(x).e;
      if (page >= 0 && a.ref[page] < kOwned) atomicAnd(a.ref + page, INT32_MAX);
    }
    refuse(s.bad ? ATTN_ERR_DATA : ATTN_ERR_PAGES);
    return;
  }
  // 4: hand out the pages, kResThreads slots at a time
  int given = 0;              // pages handed out
  int listed = 0;             // s.free_page holds free pages listed .. listed + kResThreads - 1
  for (int x0 = 0; x0 < slots; x0 += kResThreads) {
    const int x = x0 + tid;
    Slot t = mine;
    int page = -1, sum;
    bool need = false;
    if (x < slots) {
      t = slot_at(x);
      page = *t.e;
      need = needs(x, page);
    }
    const int rank = given + block_scan(need, s.warp, &sum);
    if (given + sum > listed + kResThreads) {
      // list free pages given .. given + kResThreads - 1, or as many as are still needed, and not only this step's: the
      // next steps take theirs from here too. Those handed out so far are no longer free.
      int found = given;
      const int upto = min(given + kResThreads, needed);
      for (int p0 = 0; p0 < a.num_pages && found < upto; p0 += kResThreads * kScan) {
        int r[kScan], n = 0, more;
        load_counts(a.ref, p0 + tid * kScan, a.num_pages, 1, r);
#pragma unroll
        for (int i = 0; i < kScan; ++i) n += r[i] == 0;
        int at = found - given + block_scan(n, s.warp, &more);
#pragma unroll
        for (int i = 0; i < kScan; ++i)
          if (r[i] == 0) {
            if (at < kResThreads) s.free_page[at] = p0 + tid * kScan + i;
            ++at;
          }
        found += more;
      }
      listed = given;
      __syncthreads();
    }
    if (need) {
      const int to = s.free_page[rank - listed];
      *t.e = to;
      a.ref[to] = 1;
      if (page >= 0) {
        // the count of an owned page is its owner's to set
        if (a.ref[page] >= kOwned) atomicAdd(a.ref + page, kAsk - 1);
        if (t.partial) {
          a.copies[2 * t.b] = page;
          a.copies[2 * t.b + 1] = to;
        }
      }
    }
    given += sum;
    __syncthreads();
  }
  // 5: a kept page has one holder
  for (int x = tid; x < slots; x += kResThreads) {
    const int page = *slot_at(x).e;
    if (a.ref[page] == INT32_MIN + x) a.ref[page] = 1;
  }
  if constexpr (GROW) {
    __syncthreads();  // the old lengths have been read
    for (int b = tid; b < a.B; b += kResThreads) {
      const int add = added(b), len = a.lens[b] + add;
      a.lens_out[b] = len;
      a.new_lens[b] = add > 0 ? len : 0;
    }
  }
}

// ---- attn_cache_evict ----------------------------------------------------------------------------
// One thread per table entry; only those between the sinks and the window look at the table.
__global__ void __launch_bounds__(256) evict_kernel(EvictArgs a, int64_t n) {
  for (int64_t x = blockIdx.x * 256LL + threadIdx.x; x < n; x += gridDim.x * 256LL) {
    const int b = (int)(x / a.max_pages), i = (int)(x - (int64_t)b * a.max_pages);
    const int len = __ldg(a.lens + b);
    if (len < 0 || len > a.max_pages * a.page_size) {
      if (i == 0) report(a.status, ATTN_ERR_DATA);
      continue;
    }
    const int p0 = i * a.page_size;
    if (len <= a.window || p0 < a.sinks || p0 + a.page_size > len - a.window) continue;
    const int page = a.table[x];
    if (page < 0) continue;
    if (page >= a.num_pages) {
      report(a.status, ATTN_ERR_DATA);
      continue;
    }
    a.table[x] = -1;
    atomicSub(a.ref + page, 1);
  }
}

// ---- attn_cache_compact --------------------------------------------------------------------------
// One block scans the counts: with n live pages, the k-th live page at or above n moves to the k-th
// free page below n. It renames the pages of a small table too; a second kernel, of more blocks, those of
// a larger one. The call is bound by the latency of that chain (8,192 pages, 4,928 entries: 10 us).
constexpr int kHoles = 8192;             // holes listed in shared memory; further ones are looked up in copies
constexpr int64_t kRenameHere = 32768;   // table entries that the one block renames itself

__device__ __forceinline__ int renamed(const CompactArgs& a, int page) {
  int to = -1;
  if (page >= 0) {
    if (page < a.num_pages) to = *(volatile int32_t*)(a.page_map + page);
    if (to < 0) report(a.status, ATTN_ERR_DATA);  // a page outside the pool, or one without a count
  }
  return to;
}

__global__ void __launch_bounds__(kResThreads) compact_kernel(CompactArgs a, int64_t entries) {
  __shared__ int w[kResWarps];
  __shared__ int hole_page[kHoles];
  // a warp looks at kScan * 32 pages in a row, 32 at a time, so that its accesses are whole lines; ranks
  // come from ballots
  constexpr int kStep = kResThreads * kScan;
  const int tid = threadIdx.x, lane = tid & 31;
  const int p_warp = (tid >> 5) * (kScan * 32) + lane;
  const unsigned below = (1u << lane) - 1u;
  const int pairs = a.num_pages / 2;
  int live = 0, r[kScan];
  auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int p = p0 + p_warp + 32 * i;
      r[i] = p < a.num_pages ? a.ref[p] : 0;
    }
  };
  for (int p0 = 0; p0 < a.num_pages; p0 += kStep) {
    int n = 0, sum;
    load(p0);
#pragma unroll
    for (int i = 0; i < kScan; ++i) n += r[i] > 0;
    block_scan(n, w, &sum);
    live += sum;
  }
  int holes = 0, moved = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kStep) {
    if (a.num_pages > kStep) load(p0);  // else still there
    // holes below n and live pages from n on, counted in the halves of a word (at most kStep each)
    unsigned is_hole[kScan], is_high[kScan];
    int n = 0, sum;
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int p = p0 + p_warp + 32 * i;
      is_hole[i] = __ballot_sync(0xffffffffu, p < live && r[i] <= 0);
      is_high[i] = __ballot_sync(0xffffffffu, p >= live && r[i] > 0);
      n += __popc(is_hole[i]) + (__popc(is_high[i]) << 16);
    }
    const int before = block_scan(lane == 31 ? n : 0, w, &sum);  // of the warps before, except in lane 31
    const int base = __shfl_sync(0xffffffffu, before, 0);
    int h = holes + (base & 0xffff), m = moved + (base >> 16);
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      if (is_hole[i] >> lane & 1) {
        const int at = h + __popc(is_hole[i] & below);
        if (at < kHoles) hole_page[at] = p0 + p_warp + 32 * i;
        a.copies[2 * at + 1] = p0 + p_warp + 32 * i;
      }
      h += __popc(is_hole[i]);
    }
    __syncthreads();  // the holes of these pages are listed before their movers look them up
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int p = p0 + p_warp + 32 * i;
      if (is_high[i] >> lane & 1) {
        const int at = m + __popc(is_high[i] & below);
        const int to = at < kHoles ? hole_page[at] : *(volatile int32_t*)(a.copies + 2 * at + 1);
        a.copies[2 * at] = p;
        a.page_map[p] = to;
        a.ref_out[to] = r[i];
        a.ref_out[p] = 0;
      } else if (p < a.num_pages) {
        a.page_map[p] = r[i] > 0 ? p : -1;
        if (p >= live) a.ref_out[p] = 0;
        else if (r[i] > 0) a.ref_out[p] = r[i];  // a hole's count is its mover's
      }
      m += __popc(is_high[i]);
    }
    holes += sum & 0xffff;
    moved += sum >> 16;
  }
  for (int x = moved + tid; x < pairs; x += kResThreads) a.copies[2 * x] = a.copies[2 * x + 1] = -1;
  if (tid == 0) *a.live = live;
  __syncthreads();  // the map is complete
  for (int64_t x = tid; x < entries; x += kResThreads) a.table_out[x] = renamed(a, a.table[x]);
}

__global__ void __launch_bounds__(256) rename_kernel(CompactArgs a, int64_t n) {
  for (int64_t x = blockIdx.x * 256LL + threadIdx.x; x < n; x += gridDim.x * 256LL) a.table_out[x] = renamed(a, a.table[x]);
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
  if (smem > 48 * 1024) {  // a column of more than 6,144 rows
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fork_kernel), 2 * kMaxTableRows * (int)sizeof(int32_t), ready);
    if (e != cudaSuccess) return e;
  }
  fork_kernel<<<(a.max_pages + cols - 1) / cols, kForkThreads, smem, st>>>(a, cols);
  return cudaGetLastError();
}

cudaError_t launch_cache_reserve(const ReserveArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(int32_t) * a.B;
  if (a.new_lens != nullptr)
    reserve_kernel<true><<<1, kResThreads, smem, st>>>(a);
  else
    reserve_kernel<false><<<1, kResThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * a.max_pages, blocks = (n + 255) / 256;
  evict_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, st>>>(a, n);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.rows * a.max_pages;
  compact_kernel<<<1, kResThreads, 0, st>>>(a, n <= kRenameHere ? n : 0);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || n <= kRenameHere) return e;
  const int64_t blocks = (n + 255) / 256;
  rename_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, st>>>(a, n);
  return cudaGetLastError();
}

}  // namespace sdpa
