// decode_paged.cu -- attention of one new token per sequence over a paged key/value cache.
//
// out[b, h] = softmax_j(scale q[b, h] . k_j) v over the keys j that position len_b - 1 sees: all of
// them, or a window of the newest keys and the first `sinks` ones. Every key and value is read once
// for all query heads that share it, so the call is bound by HBM: 2 * keys * Nkv * D elements.
//
// Division of the work: a unit is one sequence's KV head with up to `rows` of its query heads. The
// units' tiles (of kWarps times what a warp works on at once) are laid end to end and cut into equal ranges, one per block, so that
// one long sequence and many short ones load the GPU alike. Lengths are read on the device (the
// host never sees them, and the call can be captured into a graph); every block finds its own range
// by a scan over them. A unit inside one block is finished there. A unit cut between blocks leaves
// partial results (the sum of e^(s - m) v, m and the sum of e^(s - m)) in the workspace, and the
// last of its blocks to arrive joins them in the blocks' order:
//   m = max m_i, l = sum l_i e^(m_i - m), out = sum o_i e^(m_i - m) / l.
// Which block comes last does not change the result. The arrival counters wrap to 0 by themselves,
// so a workspace that was zero before the first call is ready for the next one after each.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGenericKeys = 16;             // keys of a tile that one warp works on, one at a time
constexpr int kJoin = 16;                    // parts of a unit that one block joins
constexpr int kGenericRows = 4;              // query heads of a unit outside the tensor-core kernel

// The blocks' ranges of the T tiles: the first T % n blocks have one more than the others.
struct Split {
  int64_t base, rem;  // T / n, T % n
  __device__ __forceinline__ void set(int64_t T, int n) {
    base = T / n;
    rem = T - base * n;
  }
  __device__ __forceinline__ int64_t begin(int c) const { return c * base + (c < rem ? c : rem); }
  __device__ __forceinline__ int owner(int64_t t) const {
    const int64_t wide = rem * (base + 1);
    return (int)(t < wide ? t / (base + 1) : rem + (t - wide) / base);
  }
};

// Shared-memory words of the range search.
struct SchedSmem {
  long long warp_sum[kWarps];
  long long total;
  long long unit_first;  // first tile of the sequence that holds the range's first tile
  int b;
  int last;              // this block is the last to arrive at a unit
};

// Finds the sequence that holds this block's first tile. Every sequence has units_b * nt_b tiles.
// Returns the number of blocks that take part (this block does not if its index is not below it).
template <int TILE>
__device__ __forceinline__ int find_range(const DecodeArgs& a, SchedSmem* s, Split* sp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = a.Nkv * a.groups;
  const int each = (a.p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, a.p.B), b1 = min(b0 + each, a.p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    KeySpan ks;
    ks.set(row_length(a.p, b, a.status), a.window, a.sinks, TILE);
    mine += (long long)ks.nt * per_seq;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s->warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s->warp_sum[w];
    total += s->warp_sum[w];
  }
  const int n = (int)(total < gridDim.x ? total : (long long)gridDim.x);
  sp->set(total, n);
  if ((int)blockIdx.x < n) {
    const long long want = sp->begin(blockIdx.x);
    long long at = before + incl - mine;
    if (want >= at && want < at + mine) {
      for (int b = b0;; ++b) {
        KeySpan ks;
        ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, TILE);
        const long long here = (long long)ks.nt * per_seq;
        if (want < at + here) {
          s->b = b;
          s->unit_first = at;
          break;
        }
        at += here;
      }
    }
  }
  __syncthreads();
  return n;
}

// A walk over the tiles (of TILE keys) of a block's range, unit by unit.
template <int TILE>
struct Cursor {
  KeySpan ks;
  int b, u;       // sequence, unit within it
  int t, t_end;   // tile within the unit; end of this block's part of the unit
  int t_begin;    // start of that part
  int64_t left;   // tiles of the range not yet handed out, this unit's part included
  int64_t first;  // index of the unit's tile 0 among all tiles

  __device__ __forceinline__ void open(const DecodeArgs& a, const SchedSmem* s, const Split& sp) {
    b = s->b;
    ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, TILE);
    const int64_t begin = sp.begin(blockIdx.x);
    const int64_t off = begin - s->unit_first;
    u = (int)(off / ks.nt);
    t = t_begin = (int)(off - (int64_t)u * ks.nt);
    first = begin - t;
    left = sp.begin(blockIdx.x + 1) - begin;
    t_end = (int)min((int64_t)ks.nt, t + left);
  }
  // On to the next unit of the range; false past its end.
  __device__ __forceinline__ bool next_unit(const DecodeArgs& a) {
    left -= t_end - t_begin;
    if (left <= 0) return false;
    first += ks.nt;
    if (++u == a.Nkv * a.groups) {
      u = 0;
      ++b;
      ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, TILE);
    }
    t = t_begin = 0;
    t_end = (int)min((int64_t)ks.nt, left);
    return true;
  }
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// e^(scale (m - to)) of raw scores m <= to: the factor that takes sums relative to m to sums relative
// to `to`. -inf stands for no key (factor 0, where `to` is -inf too); NaN stays NaN.
__device__ __forceinline__ float shrink(float m, float to, float scale_log2) {
  return exp2f((m - (to == -INFINITY ? 0.f : to)) * scale_log2);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* dst, const float (&o)[V]) {
  T t[V];
#pragma unroll
  for (int i = 0; i < V; ++i) t[i] = from_f<T>(o[i]);
  if constexpr (V == 4 && sizeof(T) == 2)
    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(t);
  else
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = t[i];
}

// The end of a unit's part in this block. Each warp's o (sum of e^(s - m) v), m (largest raw score) and
// l of the unit's query heads lie in shared memory: s_w [kWarps][rows][ld], s_wml [kWarps][rows] (m, l).
// They are merged, and written out if the unit is whole; else left in the workspace, where the last
// block to arrive joins the unit's parts. A thread takes V columns at a time.
template <typename T, int V, int TILE>
__device__ __forceinline__ void finish_unit(const DecodeArgs& a, const Cursor<TILE>& c, const Split& sp, SchedSmem* s,
                                            float* s_w, const float2* s_wml, int ld, float scale_log2) {
  const int G = a.Nq / a.Nkv, D = a.D, per_row = D / V;
  const int hk = c.u / a.groups, g0 = (c.u - hk * a.groups) * a.rows;
  const int n_rows = min(a.rows, G - g0);
  const int64_t row0 = (int64_t)c.b * a.Nq + (int64_t)hk * G + g0;
  const int64_t slot_floats = (int64_t)a.rows * (D + 4);  // o [rows][D], then (m, l) [rows], 16-byte aligned
  const bool whole = c.t_begin == 0 && c.t_end == c.ks.nt;
  float2* s_join = reinterpret_cast<float2*>(s_w);  // the warps' results are no longer needed there
  float* slot = a.part + (2 * (int64_t)blockIdx.x + (c.t_begin > 0 ? 0 : 1)) * slot_floats;
  auto write = [&](int r, int d, float m, float l, float (&o)[V]) {
    const float inv = l != 0.f ? 1.f / l : 0.f;  // l = 0: no key was seen
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= inv;
    store_row<T, V>(static_cast<T*>(a.out) + (row0 + r) * D + d, o);
    if (d == 0 && a.smax != nullptr) {
      a.smax[row0 + r] = l != 0.f ? m * a.scale : -INFINITY;
      a.ssum[row0 + r] = l;
    }
  };
  for (int x = threadIdx.x; x < n_rows * per_row; x += kThreads) {
    const int r = x / per_row, d = (x - r * per_row) * V;
    float2 ml[kWarps];
    float m = -INFINITY, l = 0.f, o[V] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = s_wml[w * a.rows + r];
      m = fmaxf(m, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = shrink(ml[w].x, m, scale_log2);
      const float* ow = s_w + (w * a.rows + r) * ld + d;
      l = fmaf(ml[w].y, f, l);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(ow[i], f, o[i]);
    }
    if (whole) {
      write(r, d, m, l, o);
    } else {
      if constexpr (V == 4)
        __stcg(reinterpret_cast<float4*>(slot + r * D + d), make_float4(o[0], o[1], o[2], o[3]));
      else
#pragma unroll
        for (int i = 0; i < V; ++i) __stcg(slot + r * D + d + i, o[i]);
      if (d == 0) __stcg(reinterpret_cast<float2*>(slot + a.rows * D) + r, make_float2(m, l));
    }
  }
  if (whole) return;
  // Part i of the unit is the tail of block c0 (i = 0) or the head of block c0 + i. Up to kJoin parts
  // are joined by the last block to arrive among them; of more, each kJoin in a row first become one
  // (in the slot of the first of them), and the last block to finish such a group joins the groups. One
  // block joining all parts of a long sequence alone took longer than reading its keys.
  const int c0 = sp.owner(c.first), parts = sp.owner(c.first + c.ks.nt - 1) - c0 + 1;
  const int groups = (parts + kJoin - 1) / kJoin;
  auto part_slot = [&](int i) { return a.part + (2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0)) * slot_floats; };
  // whether this block is the last of n to arrive at a counter
  auto last_of = [&](unsigned* ctr, int n) -> bool {
    if (n == 1) return true;
    __syncthreads();
    if (threadIdx.x == 0) {
      // releases the block's writes before its barrier and acquires those of the blocks that came earlier (fences
      // in every thread instead took 34 and not 32.5 us for two sequences of 131,072 and 81,007 keys)
      unsigned was;
      asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(was) : "l"(ctr), "r"((unsigned)n - 1) : "memory");
      s->last = was == (unsigned)n - 1;
    }
    __syncthreads();
    return s->last;
  };
  // joins n parts i0, i0 + step, ...; the result replaces part i0, or is the unit's
  auto join = [&](int i0, int n, int step, bool final) {
    for (int x = threadIdx.x; x < n_rows * per_row; x += kThreads) {
      const int r = x / per_row, d = (x - r * per_row) * V;
      float m = -INFINITY, l = 0.f, o[V] = {};
      constexpr int kAhead = 8;  // parts loaded at once
      for (int j0 = 0; j0 < n; j0 += kAhead) {
        float2 ml[kAhead];
        float po[kAhead][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          ml[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int k = 0; k < V; ++k) po[j][k] = 0.f;
          if (j0 + j < n) {
            const float* p = part_slot(i0 + (j0 + j) * step);
            ml[j] = __ldcg(reinterpret_cast<const float2*>(p + a.rows * D) + r);
            if constexpr (V == 4) {
              const float4 t = __ldcg(reinterpret_cast<const float4*>(p + r * D + d));
              po[j][0] = t.x; po[j][1] = t.y; po[j][2] = t.z; po[j][3] = t.w;
            } else {
#pragma unroll
              for (int k = 0; k < V; ++k) po[j][k] = __ldcg(p + r * D + d + k);
            }
          }
        }
        float mn = m;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) mn = fmaxf(mn, ml[j].x);
        const float f = shrink(m, mn, scale_log2);
        m = mn;
        l *= f;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] *= f;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float g = shrink(ml[j].x, m, scale_log2);
          l = fmaf(ml[j].y, g, l);
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = fmaf(po[j][k], g, o[k]);
        }
      }
      if (final) {
        write(r, d, m, l, o);
      } else {
        float* p = part_slot(i0);
#pragma unroll
        for (int k = 0; k < V; ++k) __stcg(p + r * D + d + k, o[k]);
        s_join[x] = make_float2(m, l);
      }
    }
    if (!final) {
      // (m, l) of part i0 is still read above by the other columns of its row
      __syncthreads();
      for (int r = threadIdx.x; r < n_rows; r += kThreads)
        __stcg(reinterpret_cast<float2*>(part_slot(i0) + a.rows * D) + r, s_join[r * per_row]);
    }
  };
  const int i0 = ((int)blockIdx.x - c0) / kJoin * kJoin, n = min(kJoin, parts - i0);
  if (!last_of(a.ctr + c0 + i0, n)) return;
  if (groups == 1) {
    join(0, parts, 1, true);
    return;
  }
  if (n > 1) join(i0, n, 1, false);
  if (last_of(a.ctr + kDecodeMaxCtas + c0, groups)) join(0, groups, kJoin, true);
}

// Any type, head size up to 32 * DT, any alignment: a warp takes a key at a time, lane = column.
template <typename T, int DT, int R>
__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeArgs a, float scale_log2) {
  __shared__ SchedSmem sched;
  extern __shared__ float smem[];
  const int D = a.D;
  float* s_w = smem;                                                    // [kWarps][R][D]
  float2* s_wml = reinterpret_cast<float2*>(s_w + kWarps * R * D);      // [kWarps][R] (kWarps * R is even)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTile = kWarps * kGenericKeys;
  Split sp;
  const int n = find_range<kTile>(a, &sched, &sp);
  if ((int)blockIdx.x >= n) return;
  Cursor<kTile> c;
  c.open(a, &sched, sp);
  const int G = a.Nq / a.Nkv;
  const T* K = static_cast<const T*>(a.k);
  const T* V = static_cast<const T*>(a.v);
  do {
    const int hk = c.u / a.groups, g0 = (c.u - hk * a.groups) * R;
    const int n_rows = min(R, G - g0);
    const T* Q = static_cast<const T*>(a.q) + ((int64_t)c.b * a.Nq + (int64_t)hk * G + g0) * D;
    float q[R][DT], o[R][DT], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const int d = lane + 32 * t;
        q[r][t] = r < n_rows && d < D ? to_f(Q[r * D + d]) : 0.f;
        o[r][t] = 0.f;
      }
    }
    for (; c.t < c.t_end; ++c.t) {
      const int k0 = c.ks.start(c.t, kTile) + warp * kGenericKeys;
      for (int j = k0; j < k0 + kGenericKeys; ++j) {
        if (!c.ks.sees(j)) continue;  // a key that is not seen is not read: its page may be anyone's
        const int pi = page_of(a.p, j);
        const int page = __ldg(a.p.page_table + (int64_t)c.b * a.p.max_pages + pi);
        if (page < 0 || page >= a.p.num_pages) {
          if (lane == 0) report(a.status, ATTN_ERR_DATA);
          continue;
        }
        const int64_t at = page * a.p.page_stride + (int64_t)(j - pi * a.p.page_size) * a.p.tok_stride +
                           hk * a.p.head_stride;
        float kk[DT], vv[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const int d = lane + 32 * t;
          kk[t] = d < D ? to_f(K[at + d]) : 0.f;
          vv[t] = d < D ? to_f(V[at + d]) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float sc = 0.f;
#pragma unroll
          for (int t = 0; t < DT; ++t) sc = fmaf(q[r][t], kk[t], sc);
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, x);
          const float mn = fmaxf(m[r], sc);
          const float p = shrink(sc, mn, scale_log2), f = shrink(m[r], mn, scale_log2);
          m[r] = mn;
          l[r] = l[r] * f + p;
#pragma unroll
          for (int t = 0; t < DT; ++t) o[r][t] = fmaf(p, vv[t], o[r][t] * f);
        }
      }
    }
    // merge the warps
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const int d = lane + 32 * t;
        if (d < D) s_w[(warp * R + r) * D + d] = o[r][t];
      }
      if (lane == 0) s_wml[warp * R + r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    finish_unit<T, 1>(a, c, sp, &sched, s_w, s_wml, D, scale_log2);
    __syncthreads();
  } while (c.next_unit(a));
}

// ---- streaming keys and values into shared memory ---------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros instead where !ok (src is then not read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's ring of shared-memory stages. A stage holds KEYS keys and as many values, rows of CHUNKS
// 16-byte chunks, chunk c of row r at place KSwz(r, c) (values: VSwz) of its row, so that the reads of
// the products fall into different banks. Stages are filled STAGES - 1 steps ahead with asynchronous
// copies, past the ends of units, so that HBM is never waited for between them. Keys that are not seen
// are not read: their rows become zeros, and s_seen tells the seen ones.
template <int KEYS, int CHUNKS, int STAGES, int ES, typename KSwz, typename VSwz>
struct Feeder {
  static constexpr int kTile = kWarps * KEYS;
  static constexpr int kRowBytes = CHUNKS * 16;
  static constexpr int kHalf = KEYS * kRowBytes;   // bytes of a stage's keys (or values)
  static constexpr int kRing = STAGES * 2 * kHalf;
  static constexpr int kRpi = 32 / CHUNKS;         // rows a warp copies per instruction
  static_assert(32 % CHUNKS == 0 && KEYS % kRpi == 0 && KEYS <= 32, "rows of a copy");
  Cursor<kTile> p;  // the tile being fetched
  uint32_t ring;    // shared-memory address of the warp's ring
  unsigned* seen_bits;  // [STAGES]
  int key, page, real;  // lane r looks after key r mod KEYS: its page, looked up a step ahead
  bool seen, more;

  __device__ __forceinline__ void open(const DecodeArgs& a, const Cursor<kTile>& c, uint32_t ring_addr, unsigned* bits,
                                       int real_chunks) {
    p = c;
    ring = ring_addr;
    seen_bits = bits;
    real = real_chunks;
    key = 0;
    page = -1;
    more = true;
    look_up(a);
    for (int i = 0; i < STAGES - 1; ++i) fetch(a, i);
  }
  __device__ __forceinline__ void look_up(const DecodeArgs& a) {
    key = p.ks.start(p.t, kTile) + (threadIdx.x >> 5) * KEYS + ((threadIdx.x & 31) & (KEYS - 1));
    seen = p.ks.sees(key);
    if (seen) page = __ldg(a.p.page_table + (int64_t)p.b * a.p.max_pages + page_of(a.p, key));
  }
  __device__ __forceinline__ void fetch(const DecodeArgs& a, int stage) {
    const int lane = threadIdx.x & 31;
    if (more) {
      const bool ok = seen && page >= 0 && page < a.p.num_pages;
      if (seen && !ok && lane < KEYS) report(a.status, ATTN_ERR_DATA);
      const int hk = p.u / a.groups;
      const int64_t off = ok ? page * a.p.page_stride +
                                   (int64_t)(key - page_of(a.p, key) * a.p.page_size) * a.p.tok_stride + hk * a.p.head_stride
                             : 0;
      const unsigned oks = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) seen_bits[stage] = oks;
      const uint32_t dst = ring + stage * 2 * kHalf;
      const uint8_t* K = static_cast<const uint8_t*>(a.k);
      const uint8_t* V = static_cast<const uint8_t*>(a.v);
#pragma unroll
      for (int i = 0; i < KEYS / kRpi; ++i) {
        const int row = i * kRpi + lane / CHUNKS, chunk = lane % CHUNKS;
        const int64_t at = __shfl_sync(0xffffffffu, off, row) * ES + chunk * 16;
        const bool v = ((oks >> row) & 1) && chunk < real;
        const uint32_t to = dst + row * kRowBytes;
        cp_async16(to + KSwz::at(row, chunk) * 16, K + (v ? at : 0), v);
        cp_async16(to + kHalf + VSwz::at(row, chunk) * 16, V + (v ? at : 0), v);
      }
      if (++p.t == p.t_end) more = p.next_unit(a);
      if (more) look_up(a);
    }
    cp_commit();
  }
  // Waits for the stage of the current step and fetches into the one that the last step has left.
  __device__ __forceinline__ void step(const DecodeArgs& a, int stage) {
    cp_wait<STAGES - 2>();
    __syncwarp();
    fetch(a, stage == 0 ? STAGES - 1 : stage - 1);
  }
};
struct SwzNone {
  __device__ static __forceinline__ int at(int, int c) { return c; }
};
struct SwzRow8 {  // eight rows at one chunk (ldmatrix)
  __device__ static __forceinline__ int at(int r, int c) { return c ^ (r & 7); }
};
struct SwzPair {  // two rows at four chunks in a row
  __device__ static __forceinline__ int at(int r, int c) { return c ^ ((r & 1) << 2); }
};

// ---- the tensor-core kernel ------------------------------------------------------------------------
// bf16 or fp16, head size 64 or 128. Each warp works on 16 MB keys of a tile on its own: it brings them
// into its ring of shared-memory stages with 16-byte asynchronous copies (kStages - 1 steps ahead, over
// the ends of units, so that HBM is never waited for between them), and multiplies
//   S^T [16 MB keys x 8 NB heads] = K Q^T      (K by ldmatrix, Q held in registers)
//   O^T [D x 8 NB heads] += V^T P^T            (V by ldmatrix.trans, P^T from S^T by movmatrix)
// with m16n8k16 products and fp32 sums. Keys are the rows of the first product, so a group of up to
// 8 query heads costs 8 columns and not 16. The blocks' warps meet only at the end of a unit.
// P in 16 bits would keep 2^-8 (bf16) or 2^-11 (fp16) of a weight, so it goes in as two terms, p and what
// rounding left of it (2^-16; fp16 2^-22): the second product is free, the call waits for HBM. A weight relative to
// the largest one may be tiny and still count, as there may be many like it behind one key that takes most of
// the weight. fp16 has no normal numbers below 2^-14, so its weights are kept times 2^15 until the unit ends: the
// largest is 2^15, normal ones reach down to 2^-29 of it, and the two terms together end at 2^-40 of it. (Kept as they are, keys below 2^-25 of their warp's
// largest one counted in the sum of e^(s - m) and not in that of e^(s - m) v. Windows of 4,096 keys over 16
// sequences take 46.4 us either way.)
// tcgen05 would pad the 1 to 16 rows of queries to 64 or 128 and fill its operands through the same
// shared memory; at most 16 rows of heads, mma.sync is far from its limit here.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  T t[2] = {from_f<T>(x), from_f<T>(y)};
  return *reinterpret_cast<uint32_t*>(t);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  const T* t = reinterpret_cast<const T*>(&x);
  return make_float2(to_f(t[0]), to_f(t[1]));
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int NB>
struct TcCfg {
  // 16-key blocks that a warp works on at once: as many as make 8 KB of keys and values, so that the
  // fixed cost of a step (the copies' addresses, the maximum's shuffles) is spread alike
  static constexpr int kMb = 128 / D;
  static constexpr int kWarpKeys = 16 * kMb;
  static constexpr int kRows = 8 * NB;                       // query heads of a unit
  static constexpr int kStages = 3;                          // ring stages of a warp
  using Feed = Feeder<kWarpKeys, D / 8, kStages, 2, SwzRow8, SwzRow8>;
  static constexpr int kTile = Feed::kTile;
  static constexpr int kHalf = Feed::kHalf;
  static constexpr int kRing = kWarps * Feed::kRing;
  static constexpr int kLd = D + 4;                          // padded row of the merge area
  static constexpr int kMerge = kWarps * kRows * kLd * 4;
  static constexpr int kSmem = kRing + kMerge + kWarps * kRows * 8;
};

template <typename T, int D, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) decode_tc_kernel(DecodeArgs a, float scale_log2) {
  using C = TcCfg<D, NB>;
  constexpr bool kF16 = sizeof(T) == 2 && std::is_same<T, __half>::value;
  constexpr int kTile = C::kTile, kMb = C::kMb;
  constexpr float kBias = kF16 ? 15.f : 0.f, kUnbias = kF16 ? 0x1p-15f : 1.f;  // weights are kept times 2^kBias
  extern __shared__ __align__(128) uint8_t tc_smem[];
  __shared__ SchedSmem sched;
  __shared__ unsigned s_seen[kWarps][C::kStages];  // bit r: key r of the stage is visible
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* s_w = reinterpret_cast<float*>(tc_smem + C::kRing);
  float2* s_wml = reinterpret_cast<float2*>(tc_smem + C::kRing + C::kMerge);
  const uint32_t ring0 = smem_addr(tc_smem + warp * C::Feed::kRing);

  Split sp;
  const int n = find_range<kTile>(a, &sched, &sp);
  if ((int)blockIdx.x >= n) return;
  Cursor<kTile> c;  // the tile being multiplied
  c.open(a, &sched, sp);
  typename C::Feed feed;
  feed.open(a, c, ring0, s_seen[warp], D / 8);
  const int G = a.Nq / a.Nkv;

  int stage = 0;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  // ldmatrix rows of this lane: keys (lane & 7) + 8 * bit 3 and columns 8 * bit 4 for K; keys
  // (lane & 7) + 8 * bit 4 and columns 8 * bit 3 for V
  const int krow = (lane & 7) + (lane & 8), kcol = lane >> 4;
  const int vrow = (lane & 7) + ((lane >> 1) & 8), vcol = (lane >> 3) & 1;
  do {
    const int hk = c.u / a.groups, g0 = (c.u - hk * a.groups) * C::kRows;
    const int n_rows = min(C::kRows, G - g0);
    uint32_t q[NB][D / 16][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 8 * b + g;
      const T* Q = static_cast<const T*>(a.q) + ((int64_t)c.b * a.Nq + (int64_t)hk * G + g0 + r) * D + t2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[b][k][0] = r < n_rows ? __ldg(reinterpret_cast<const uint32_t*>(Q + 16 * k)) : 0u;
        q[b][k][1] = r < n_rows ? __ldg(reinterpret_cast<const uint32_t*>(Q + 16 * k + 8)) : 0u;
      }
    }
    float o[NB][D / 16][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      m[b][0] = m[b][1] = -INFINITY;
      l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[b][k][i] = 0.f;
    }
    for (; c.t < c.t_end; ++c.t) {
      feed.step(a, stage);
      const uint32_t sk = ring0 + stage * 2 * C::kHalf, sv = sk + C::kHalf;
      const unsigned seen_now = s_seen[warp][stage];
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      float s[NB][kMb][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < kMb; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[b][j][i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int j = 0; j < kMb; ++j) {
          uint32_t kf[4];
          ldsm4(kf, sk + (16 * j + krow) * (D * 2) + (((2 * k + kcol) ^ (krow & 7)) << 4));
#pragma unroll
          for (int b = 0; b < NB; ++b) mma16816<kF16>(s[b][j], kf, q[b][k][0], q[b][k][1]);
        }
      }
      uint32_t ph[NB][kMb][2], pl[NB][kMb][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // the largest score of each head's keys; the running one only moves where it is exceeded
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < kMb; ++j) {
          if (!((seen_now >> (16 * j + g)) & 1)) s[b][j][0] = s[b][j][1] = -INFINITY;
          if (!((seen_now >> (16 * j + g + 8)) & 1)) s[b][j][2] = s[b][j][3] = -INFINITY;
          x0 = fmaxf(x0, fmaxf(s[b][j][0], s[b][j][2]));
          x1 = fmaxf(x1, fmaxf(s[b][j][1], s[b][j][3]));
        }
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, i));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, i));
        }
        if (__any_sync(0xffffffffu, x0 > m[b][0] || x1 > m[b][1])) {
          const float n0 = fmaxf(m[b][0], x0), n1 = fmaxf(m[b][1], x1);
          const float f0 = shrink(m[b][0], n0, scale_log2), f1 = shrink(m[b][1], n1, scale_log2);
          m[b][0] = n0;
          m[b][1] = n1;
          l[b][0] *= f0;
          l[b][1] *= f1;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            o[b][k][0] *= f0;
            o[b][k][1] *= f1;
            o[b][k][2] *= f0;
            o[b][k][3] *= f1;
          }
        }
        const float u0 = m[b][0] == -INFINITY ? 0.f : m[b][0], u1 = m[b][1] == -INFINITY ? 0.f : m[b][1];
        const float c0 = -u0 * scale_log2, c1 = -u1 * scale_log2;
#pragma unroll
        for (int j = 0; j < kMb; ++j) {
          float e[4];
          if constexpr (kF16) {
            // the difference first: rounding scale m may not take a weight above 2^15 (fp16 ends at 65,504)
            e[0] = ex2_approx(fmaf(s[b][j][0] - u0, scale_log2, kBias));
            e[1] = ex2_approx(fmaf(s[b][j][1] - u1, scale_log2, kBias));
            e[2] = ex2_approx(fmaf(s[b][j][2] - u0, scale_log2, kBias));
            e[3] = ex2_approx(fmaf(s[b][j][3] - u1, scale_log2, kBias));
          } else {
            e[0] = ex2_approx(fmaf(s[b][j][0], scale_log2, c0));
            e[1] = ex2_approx(fmaf(s[b][j][1], scale_log2, c1));
            e[2] = ex2_approx(fmaf(s[b][j][2], scale_log2, c0));
            e[3] = ex2_approx(fmaf(s[b][j][3], scale_log2, c1));
          }
          l[b][0] += e[0] + e[2];
          l[b][1] += e[1] + e[3];
          const uint32_t h0 = pack2<T>(e[0], e[1]), h1 = pack2<T>(e[2], e[3]);
          ph[b][j][0] = transpose8(h0);
          ph[b][j][1] = transpose8(h1);
          const float2 r0 = unpack2<T>(h0), r1 = unpack2<T>(h1);
          pl[b][j][0] = transpose8(pack2<T>(e[0] - r0.x, e[1] - r0.y));
          pl[b][j][1] = transpose8(pack2<T>(e[2] - r1.x, e[3] - r1.y));
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int j = 0; j < kMb; ++j) {
          uint32_t vf[4];
          ldsm4t(vf, sv + (16 * j + vrow) * (D * 2) + (((2 * k + vcol) ^ (vrow & 7)) << 4));
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma16816<kF16>(o[b][k], vf, ph[b][j][0], ph[b][j][1]);
            mma16816<kF16>(o[b][k], vf, pl[b][j][0], pl[b][j][1]);
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        l[b][0] += __shfl_xor_sync(0xffffffffu, l[b][0], i);
        l[b][1] += __shfl_xor_sync(0xffffffffu, l[b][1], i);
      }
      float* w0 = s_w + (warp * C::kRows + 8 * b + t2) * C::kLd + g;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        w0[16 * k] = o[b][k][0] * kUnbias;
        w0[16 * k + C::kLd] = o[b][k][1] * kUnbias;
        w0[16 * k + 8] = o[b][k][2] * kUnbias;
        w0[16 * k + 8 + C::kLd] = o[b][k][3] * kUnbias;
      }
      if (g == 0) {
        s_wml[warp * C::kRows + 8 * b + t2] = make_float2(m[b][0], l[b][0] * kUnbias);
        s_wml[warp * C::kRows + 8 * b + t2 + 1] = make_float2(m[b][1], l[b][1] * kUnbias);
      }
    }
    __syncthreads();
    finish_unit<T, 4>(a, c, sp, &sched, s_w, s_wml, C::kLd, scale_log2);
    __syncthreads();
  } while (c.next_unit(a));
  cp_wait<0>();
}

// ---- the fp32 kernel -----------------------------------------------------------------------------
// float32 with rows of whole 16-byte chunks, head size up to DM. As above a warp streams its keys
// (8 at a time) through its ring. Scores: four lanes share a key, each multiplies every fourth chunk of
// the row with all query heads (from shared memory); exchanging halves of the heads, then quarters,
// leaves lane 4 k + r with the score of key k and head r (R = 8: and r + 4), so that each exponential is
// computed once. Values: a lane owns a chunk of columns and takes the weights from shared memory. With
// 4 heads a KV head a key costs about 50 instructions a warp: the call waits for HBM.
template <int DM, int R>
struct F32Cfg {
  static constexpr int kKeys = 8, kStages = 3, kChunks = DM / 4;
  using Feed = Feeder<kKeys, kChunks, kStages, 4, SwzPair, SwzNone>;
  static constexpr int kTile = Feed::kTile;
  static constexpr int kLd = DM;
  static constexpr int kRing = kWarps * Feed::kRing;
  static constexpr int kQ = kWarps * R * DM * 4;       // query heads, a copy per warp
  static constexpr int kP = kWarps * kKeys * R * 4;    // weights
  static constexpr int kMerge = kWarps * R * kLd * 4;  // over the ring's size: rings stay in flight
  static constexpr int kSmem = kRing + kQ + kP + kMerge + kWarps * R * 8;
};

template <int DM, int R>
__global__ void __launch_bounds__(kThreads) decode_f32_kernel(DecodeArgs a, float scale_log2) {
  using C = F32Cfg<DM, R>;
  constexpr int kTile = C::kTile, kKeys = C::kKeys;
  constexpr int RG = R / 4;            // groups of four heads
  constexpr int kParts = 32 / C::kChunks;  // keys whose values the lanes take at once (1 or 2)
  extern __shared__ __align__(128) uint8_t tc_smem[];
  __shared__ SchedSmem sched;
  __shared__ unsigned s_seen[kWarps][C::kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* ring = tc_smem + warp * C::Feed::kRing;
  float* s_q = reinterpret_cast<float*>(tc_smem + C::kRing) + warp * R * DM;
  float* s_p = reinterpret_cast<float*>(tc_smem + C::kRing + C::kQ) + warp * kKeys * R;
  float* s_w = reinterpret_cast<float*>(tc_smem + C::kRing + C::kQ + C::kP);
  float2* s_wml = reinterpret_cast<float2*>(tc_smem + C::kRing + C::kQ + C::kP + C::kMerge);
  Split sp;
  const int n = find_range<kTile>(a, &sched, &sp);
  if ((int)blockIdx.x >= n) return;
  Cursor<kTile> c;
  c.open(a, &sched, sp);
  typename C::Feed feed;
  feed.open(a, c, smem_addr(ring), s_seen[warp], a.D / 4);
  const int G = a.Nq / a.Nkv;
  int stage = 0;
  const int kk = lane >> 2, qr = lane & 3;              // key and chunk quarter of the scores
  const int vk = lane / C::kChunks, vc = lane % C::kChunks;  // key parity and chunk of the values
  do {
    const int hk = c.u / a.groups, g0 = (c.u - hk * a.groups) * R;
    const int n_rows = min(R, G - g0);
    const float* Q = static_cast<const float*>(a.q) + ((int64_t)c.b * a.Nq + (int64_t)hk * G + g0) * a.D;
    // every load of the heads before the first store, or the unit begins with several trips to memory (61 MB of
    // keys and values in 32 units: 25.3 -> 23.4 us); Q is 16-byte aligned and a.D a multiple of 4
    float4 q[R * C::kChunks / 32];
#pragma unroll
    for (int i = 0; i < R * C::kChunks / 32; ++i) {
      const int x = lane + 32 * i, r = x / C::kChunks, d = x % C::kChunks * 4;
      q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n_rows && d < a.D) q[i] = __ldg(reinterpret_cast<const float4*>(Q + r * a.D + d));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < R * C::kChunks / 32; ++i) reinterpret_cast<float4*>(s_q)[lane + 32 * i] = q[i];
    __syncwarp();
    float o[R][4], m[RG], l[RG];
#pragma unroll
    for (int r = 0; r < R; ++r) o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    for (; c.t < c.t_end; ++c.t) {
      feed.step(a, stage);
      const float4* sk = reinterpret_cast<const float4*>(ring + stage * 2 * C::Feed::kHalf);
      const float4* sv = sk + kKeys * C::kChunks;
      const bool see = (s_seen[warp][stage] >> kk) & 1;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll
      for (int i = 0; i < C::kChunks / 4; ++i) {
        const float4 kv = sk[kk * C::kChunks + SwzPair::at(kk, 4 * i + qr)];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(s_q + r * DM + (4 * i + qr) * 4);
          s[r] = fmaf(qv.x, kv.x, s[r]);
          s[r] = fmaf(qv.y, kv.y, s[r]);
          s[r] = fmaf(qv.z, kv.z, s[r]);
          s[r] = fmaf(qv.w, kv.w, s[r]);
        }
      }
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        // lanes qr and qr ^ 2 exchange two heads each, then qr and qr ^ 1 one: head qr is left
        const bool hi = qr & 2, odd = qr & 1;
        const float* t = s + 4 * i;
        float a0 = hi ? t[2] : t[0], a1 = hi ? t[3] : t[1];
        a0 += __shfl_xor_sync(0xffffffffu, hi ? t[0] : t[2], 2);
        a1 += __shfl_xor_sync(0xffffffffu, hi ? t[1] : t[3], 2);
        float sc = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
        if (!see) sc = -INFINITY;
        float x = sc;
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
        if (__any_sync(0xffffffffu, x > m[i])) {
          const float mn = fmaxf(m[i], x);
          const float f = shrink(m[i], mn, scale_log2);
          m[i] = mn;
          l[i] *= f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f, r);
#pragma unroll
            for (int y = 0; y < 4; ++y) o[4 * i + r][y] *= fr;
          }
        }
        const float e = shrink(sc, m[i], scale_log2);
        l[i] += e;
        s_p[kk * R + 4 * i + qr] = e;
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kKeys / kParts; ++k) {
        const int key = k * kParts + vk;
        const float4 v = sv[key * C::kChunks + vc];
#pragma unroll
        for (int i = 0; i < RG; ++i) {
          const float4 p4 = *reinterpret_cast<const float4*>(s_p + key * R + 4 * i);
          const float pr[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[4 * i + r][0] = fmaf(pr[r], v.x, o[4 * i + r][0]);
            o[4 * i + r][1] = fmaf(pr[r], v.y, o[4 * i + r][1]);
            o[4 * i + r][2] = fmaf(pr[r], v.z, o[4 * i + r][2]);
            o[4 * i + r][3] = fmaf(pr[r], v.w, o[4 * i + r][3]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (kParts == 2) {
#pragma unroll
        for (int y = 0; y < 4; ++y) o[r][y] += __shfl_xor_sync(0xffffffffu, o[r][y], 16);
      }
      if (vk == 0)
        *reinterpret_cast<float4*>(s_w + (warp * R + r) * C::kLd + vc * 4) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
    }
#pragma unroll
    for (int i = 0; i < RG; ++i) {
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], y);
      if (kk == 0) s_wml[warp * R + 4 * i + qr] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    finish_unit<float, 4>(a, c, sp, &sched, s_w, s_wml, C::kLd, scale_log2);
    __syncthreads();
  } while (c.next_unit(a));
  cp_wait<0>();
}

template <typename T, int D, int NB>
cudaError_t launch_tc(const DecodeArgs& a, cudaStream_t st) {
  using C = TcCfg<D, NB>;
  auto kernel = decode_tc_kernel<T, D, NB>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use that much shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, ready);
  if (e != cudaSuccess) return e;
  const int grid = min((NB == 1 ? 2 : 1) * a.num_sms, kDecodeMaxCtas);
  kernel<<<grid, kThreads, C::kSmem, st>>>(a, a.scale * 1.4426950408889634f);
  return cudaGetLastError();
}

template <int DM, int R>
cudaError_t launch_f32(const DecodeArgs& a, cudaStream_t st) {
  using C = F32Cfg<DM, R>;
  auto kernel = decode_f32_kernel<DM, R>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::kSmem, ready);
  if (e != cudaSuccess) return e;
  const int per_sm = 2 * (C::kSmem + 1280) <= 228 * 1024 ? 2 : 1;  // with what the block reserves
  kernel<<<min(per_sm * a.num_sms, kDecodeMaxCtas), kThreads, C::kSmem, st>>>(a, a.scale * 1.4426950408889634f);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_tc_t(const DecodeArgs& a, cudaStream_t st) {
  if (a.D == 64) return a.rows == 8 ? launch_tc<T, 64, 1>(a, st) : launch_tc<T, 64, 2>(a, st);
  return a.rows == 8 ? launch_tc<T, 128, 1>(a, st) : launch_tc<T, 128, 2>(a, st);
}

template <typename T, int DT>
cudaError_t launch_dt(const DecodeArgs& a, cudaStream_t st) {
  constexpr int R = kGenericRows;
  const int smem = (int)sizeof(float) * (kWarps * R * a.D + 2 * R * kWarps);
  const int grid = min(2 * a.num_sms, kDecodeMaxCtas);
  decode_kernel<T, DT, R><<<grid, kThreads, smem, st>>>(a, a.scale * 1.4426950408889634f);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t st) {
  if (a.D <= 64) return launch_dt<T, 2>(a, st);
  if (a.D <= 128) return launch_dt<T, 4>(a, st);
  return launch_dt<T, 8>(a, st);
}

bool tensor_shape(int dtype, int D) { return dtype != ATTN_F32 && (D == 64 || D == 128); }

}  // namespace

int decode_rows(int dtype, int Nq, int Nkv, int D) {
  if (tensor_shape(dtype, D)) return Nq / Nkv <= 8 ? 8 : 16;
  return dtype == ATTN_F32 && D <= 128 && Nq / Nkv > 4 ? 8 : kGenericRows;
}

int64_t decode_workspace_bytes(int rows, int D) {
  return 2LL * kDecodeMaxCtas * rows * (D + 4) * (int64_t)sizeof(float) + 2 * kDecodeMaxCtas * (int64_t)sizeof(unsigned);
}

cudaError_t launch_decode(const DecodeArgs& args, cudaStream_t st) {
  DecodeArgs a = args;
  const int es = a.dtype == ATTN_F32 ? 4 : 2;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                        reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.p.page_stride * es);
  if (tensor_shape(a.dtype, a.D) && (all & 15u) == 0)
    return a.dtype == ATTN_F16 ? launch_tc_t<__half>(a, st) : launch_tc_t<__nv_bfloat16>(a, st);
  if (a.dtype == ATTN_F32 && a.D <= 128 && (all & 15u) == 0 && a.D % 4 == 0) {
    if (a.D <= 64) return a.rows == 4 ? launch_f32<64, 4>(a, st) : launch_f32<64, 8>(a, st);
    return a.rows == 4 ? launch_f32<128, 4>(a, st) : launch_f32<128, 8>(a, st);
  }
  // the workspace for the rows of the kernels above is as large as this one's or larger
  a.rows = kGenericRows;
  a.groups = (a.Nq / a.Nkv + a.rows - 1) / a.rows;
  if (a.dtype == ATTN_F32) return launch_t<float>(a, st);
  return a.dtype == ATTN_F16 ? launch_t<__half>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sdpa
