// decode_paged.cu -- attention of one new token per sequence over a paged key/value cache.
//
// out[b, h] = softmax_j(scale q[b, h] . k_j) v over the keys j that position len_b - 1 sees: all of
// them, or a window of the newest keys and the first `sinks` ones. Every key and value is read once
// for all query heads that share it, so the call is bound by HBM: 2 * keys * Nkv * D elements.
//
// Division of the work: a unit is one sequence's KV head with up to `rows` of its query heads. The
// units' tiles (of kTile keys) are laid end to end and cut into equal ranges, one per block, so that
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

#include <atomic>
#include <type_traits>

#include "paged.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpKeys = 16;                // keys of a tile that one warp works on
constexpr int kTile = kWarps * kWarpKeys;    // keys per tile
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
__device__ __forceinline__ int find_range(const DecodeArgs& a, SchedSmem* s, Split* sp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = a.Nkv * a.groups;
  const int each = (a.p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, a.p.B), b1 = min(b0 + each, a.p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    KeySpan ks;
    ks.set(row_length(a.p, b, a.status), a.window, a.sinks, kTile);
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
        ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, kTile);
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

// A walk over the tiles of a block's range, unit by unit.
struct Cursor {
  KeySpan ks;
  int b, u;       // sequence, unit within it
  int t, t_end;   // tile within the unit; end of this block's part of the unit
  int t_begin;    // start of that part
  int64_t left;   // tiles of the range not yet handed out, this unit's part included
  int64_t first;  // index of the unit's tile 0 among all tiles

  __device__ __forceinline__ void open(const DecodeArgs& a, const SchedSmem* s, const Split& sp) {
    b = s->b;
    ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, kTile);
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
      ks.set(row_length(a.p, b, nullptr), a.window, a.sinks, kTile);
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
template <typename T, int V>
__device__ __forceinline__ void finish_unit(const DecodeArgs& a, const Cursor& c, const Split& sp, SchedSmem* s,
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
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s->last = atomicInc(ctr, (unsigned)n - 1) == (unsigned)n - 1;
    __syncthreads();
    const bool last = s->last;
    __threadfence();
    return last;
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
  Split sp;
  const int n = find_range(a, &sched, &sp);
  if ((int)blockIdx.x >= n) return;
  Cursor c;
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
      const int k0 = c.ks.start(c.t, kTile) + warp * kWarpKeys;
      for (int j = k0; j < k0 + kWarpKeys; ++j) {
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

// ---- the tensor-core kernel ------------------------------------------------------------------------
// bf16 or fp16, head size 64 or 128. Each warp works on 16 keys of a tile on its own: it brings them
// into its ring of shared-memory stages with 16-byte asynchronous copies (kStages - 1 steps ahead, over
// the ends of units, so that HBM is never waited for between them), and multiplies
//   S^T [16 keys x 8 NB heads] = K Q^T         (K by ldmatrix, Q held in registers)
//   O^T [D x 8 NB heads] += V^T P^T            (V by ldmatrix.trans, P^T from S^T by movmatrix)
// with m16n8k16 products and fp32 sums. Keys are the rows of the first product, so a group of up to
// 8 query heads costs 8 columns and not 16. The blocks' warps meet only at the end of a unit.
// P in 16 bits: fp16 keeps 2^-11 of a weight; bf16 would keep 2^-8, so it goes in as two terms, p and
// what rounding left of it (2^-16): the second product is free, the call waits for HBM.
// tcgen05 would pad the 1 to 16 rows of queries to 64 or 128 and fill its operands through the same
// shared memory; at most 16 rows of heads, mma.sync is far from its limit here.
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
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int NB>
struct TcCfg {
  static constexpr int kRows = 8 * NB;                       // query heads of a unit
  static constexpr int kStages = D == 128 ? 3 : 6;           // ring stages of a warp
  static constexpr int kHalf = kWarpKeys * D * 2;            // bytes of a stage's keys (or values)
  static constexpr int kRing = kWarps * kStages * 2 * kHalf;
  static constexpr int kLd = D + 4;                          // padded row of the merge area
  static constexpr int kMerge = kWarps * kRows * kLd * 4;
  static constexpr int kSmem = kRing + kMerge + kWarps * kRows * 8;
};

template <typename T, int D, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) decode_tc_kernel(DecodeArgs a, float scale_log2) {
  using C = TcCfg<D, NB>;
  constexpr bool kF16 = sizeof(T) == 2 && std::is_same<T, __half>::value;
  constexpr int kCpr = D / 8;        // 16-byte chunks per row
  constexpr int kRpi = 32 / kCpr;    // rows a warp copies per instruction
  constexpr int kSteps = kWarpKeys / kRpi;
  extern __shared__ __align__(128) uint8_t tc_smem[];
  __shared__ SchedSmem sched;
  __shared__ unsigned s_seen[kWarps][C::kStages];  // bit r: key r of the stage is visible
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = tc_smem + warp * C::kStages * 2 * C::kHalf;
  float* s_w = reinterpret_cast<float*>(tc_smem + C::kRing);
  float2* s_wml = reinterpret_cast<float2*>(tc_smem + C::kRing + C::kMerge);
  const uint32_t ring0 = smem_addr(ring);

  Split sp;
  const int n = find_range(a, &sched, &sp);
  if ((int)blockIdx.x >= n) return;
  Cursor c, p;  // the tile being multiplied, the tile being fetched
  c.open(a, &sched, sp);
  p = c;
  bool more = true;
  const int G = a.Nq / a.Nkv;
  const uint8_t* K = static_cast<const uint8_t*>(a.k);
  const uint8_t* V = static_cast<const uint8_t*>(a.v);

  // lane r (and r + 16) looks after key r of the warp's 16: its page, looked up a step ahead
  int key = 0, page = -1;
  bool seen = false;
  auto look_up = [&]() {
    key = p.ks.start(p.t, kTile) + warp * kWarpKeys + (lane & 15);
    seen = p.ks.sees(key);
    if (seen) page = __ldg(a.p.page_table + (int64_t)p.b * a.p.max_pages + page_of(a.p, key));
  };
  auto fetch = [&](int stage) {
    if (more) {
      bool ok = seen && page >= 0 && page < a.p.num_pages;
      if (seen && !ok && lane < 16) report(a.status, ATTN_ERR_DATA);
      const int hk = p.u / a.groups;
      const int64_t off = ok ? page * a.p.page_stride +
                                   (int64_t)(key - page_of(a.p, key) * a.p.page_size) * a.p.tok_stride + hk * a.p.head_stride
                             : 0;
      const unsigned oks = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) s_seen[warp][stage] = oks;
      const uint32_t dst = ring0 + stage * 2 * C::kHalf;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int row = i * kRpi + lane / kCpr, chunk = lane % kCpr;
        const int64_t o = (__shfl_sync(0xffffffffu, off, row) + chunk * 8) * 2;
        const bool v = (oks >> row) & 1;
        const uint32_t at = dst + row * (D * 2) + ((chunk ^ (row & 7)) << 4);
        cp_async16(at, K + (v ? o : 0), v);
        cp_async16(at + C::kHalf, V + (v ? o : 0), v);
      }
      if (++p.t == p.t_end) more = p.next_unit(a);
      if (more) look_up();
    }
    cp_commit();
  };
  look_up();
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) fetch(s);

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
      cp_wait<C::kStages - 2>();
      __syncwarp();  // this step's copies of all lanes are there, and the last step's stage is free
      fetch(stage == 0 ? C::kStages - 1 : stage - 1);
      const uint32_t sk = ring0 + stage * 2 * C::kHalf, sv = sk + C::kHalf;
      const unsigned seen_now = s_seen[warp][stage];
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      float s[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[b][i] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t kf[4];
        ldsm4(kf, sk + krow * (D * 2) + (((2 * k + kcol) ^ (krow & 7)) << 4));
#pragma unroll
        for (int b = 0; b < NB; ++b) mma16816<kF16>(s[b], kf, q[b][k][0], q[b][k][1]);
      }
      const bool see0 = (seen_now >> g) & 1, see1 = (seen_now >> (g + 8)) & 1;
      uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (!see0) s[b][0] = s[b][1] = -INFINITY;
        if (!see1) s[b][2] = s[b][3] = -INFINITY;
        // the largest score of each head's 16 keys; the running one only moves where it is exceeded
        float x0 = fmaxf(s[b][0], s[b][2]), x1 = fmaxf(s[b][1], s[b][3]);
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
        const float c0 = m[b][0] == -INFINITY ? 0.f : -m[b][0] * scale_log2;
        const float c1 = m[b][1] == -INFINITY ? 0.f : -m[b][1] * scale_log2;
        float e[4];
        e[0] = ex2_approx(fmaf(s[b][0], scale_log2, c0));
        e[1] = ex2_approx(fmaf(s[b][1], scale_log2, c1));
        e[2] = ex2_approx(fmaf(s[b][2], scale_log2, c0));
        e[3] = ex2_approx(fmaf(s[b][3], scale_log2, c1));
        l[b][0] += e[0] + e[2];
        l[b][1] += e[1] + e[3];
        const uint32_t h0 = pack2<T>(e[0], e[1]), h1 = pack2<T>(e[2], e[3]);
        ph[b][0] = transpose8(h0);
        ph[b][1] = transpose8(h1);
        if constexpr (!kF16) {
          const float2 r0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
          const float2 r1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
          pl[b][0] = transpose8(pack2<T>(e[0] - r0.x, e[1] - r0.y));
          pl[b][1] = transpose8(pack2<T>(e[2] - r1.x, e[3] - r1.y));
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t vf[4];
        ldsm4t(vf, sv + vrow * (D * 2) + (((2 * k + vcol) ^ (vrow & 7)) << 4));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          mma16816<kF16>(o[b][k], vf, ph[b][0], ph[b][1]);
          if constexpr (!kF16) mma16816<kF16>(o[b][k], vf, pl[b][0], pl[b][1]);
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
        w0[16 * k] = o[b][k][0];
        w0[16 * k + C::kLd] = o[b][k][1];
        w0[16 * k + 8] = o[b][k][2];
        w0[16 * k + 8 + C::kLd] = o[b][k][3];
      }
      if (g == 0) {
        s_wml[warp * C::kRows + 8 * b + t2] = make_float2(m[b][0], l[b][0]);
        s_wml[warp * C::kRows + 8 * b + t2 + 1] = make_float2(m[b][1], l[b][1]);
      }
    }
    __syncthreads();
    finish_unit<T, 4>(a, c, sp, &sched, s_w, s_wml, C::kLd, scale_log2);
    __syncthreads();
  } while (c.next_unit(a));
  cp_wait<0>();
}

// Raises a kernel's limit of dynamic shared memory, once per device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return e;
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
  return tensor_shape(dtype, D) ? (Nq / Nkv <= 8 ? 8 : 16) : kGenericRows;
}

int64_t decode_workspace_bytes(int rows, int D) {
  return 2LL * kDecodeMaxCtas * rows * (D + 4) * (int64_t)sizeof(float) + 2 * kDecodeMaxCtas * (int64_t)sizeof(unsigned);
}

cudaError_t launch_decode(const DecodeArgs& args, cudaStream_t st) {
  DecodeArgs a = args;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                        reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(a.p.page_stride * 2);
  if (tensor_shape(a.dtype, a.D) && (all & 15u) == 0)
    return a.dtype == ATTN_F16 ? launch_tc_t<__half>(a, st) : launch_tc_t<__nv_bfloat16>(a, st);
  // the tensor-core kernel's workspace is larger than this one's
  a.rows = kGenericRows;
  a.groups = (a.Nq / a.Nkv + a.rows - 1) / a.rows;
  if (a.dtype == ATTN_F32) return launch_t<float>(a, st);
  return a.dtype == ATTN_F16 ? launch_t<__half>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sdpa
