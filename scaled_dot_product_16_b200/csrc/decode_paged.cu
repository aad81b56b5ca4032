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
#include <math.h>

#include "paged.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpKeys = 16;                // keys of a tile that one warp works on
constexpr int kTile = kWarps * kWarpKeys;    // keys per tile

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

// The unit's result o (sum of e^(s - m) v), m (largest raw score) and l of its `rows` query heads,
// merged over the block's warps, lies in shared memory: written out if the unit is whole, else left
// in the workspace, where the last block to arrive joins the unit's parts.
// s_o [rows][D], s_ml [rows][2].
template <typename T>
__device__ void finish_unit(const DecodeArgs& a, const Cursor& c, const Split& sp, SchedSmem* s, float* s_o,
                            float* s_ml, float scale_log2) {
  const int G = a.Nq / a.Nkv;
  const int hk = c.u / a.groups, g0 = (c.u - hk * a.groups) * a.rows;
  const int n_rows = min(a.rows, G - g0);
  const int64_t row0 = (int64_t)c.b * a.Nq + (int64_t)hk * G + g0;
  const int D = a.D;
  const int64_t slot_floats = (int64_t)a.rows * (D + 2);
  const bool whole = c.t_begin == 0 && c.t_end == c.ks.nt;
  int c0 = 0, parts = 0;
  if (!whole) {
    c0 = sp.owner(c.first);
    parts = sp.owner(c.first + c.ks.nt - 1) - c0 + 1;
    float* slot = a.part + (2 * (int64_t)blockIdx.x + (c.t_begin > 0 ? 0 : 1)) * slot_floats;
    for (int x = threadIdx.x; x < n_rows * D; x += kThreads) __stcg(slot + x, s_o[x]);
    for (int x = threadIdx.x; x < 2 * n_rows; x += kThreads) __stcg(slot + (int64_t)a.rows * D + x, s_ml[x]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s->last = atomicInc(a.ctr + c0, (unsigned)parts - 1) == (unsigned)parts - 1;
    __syncthreads();
    if (!s->last) return;
    __threadfence();
  }
  for (int x = threadIdx.x; x < n_rows * D; x += kThreads) {
    const int r = x / D;
    float m, l, o;
    if (whole) {
      m = s_ml[2 * r];
      l = s_ml[2 * r + 1];
      o = s_o[x];
    } else {
      m = -INFINITY;
      l = o = 0.f;
      for (int i = 0; i < parts; ++i) {
        const float* slot = a.part + (2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0)) * slot_floats;
        const float mi = __ldcg(slot + (int64_t)a.rows * D + 2 * r);
        const float li = __ldcg(slot + (int64_t)a.rows * D + 2 * r + 1);
        const float oi = __ldcg(slot + x);
        if (li == 0.f) continue;  // a part without a visible key
        const float mn = fmaxf(m, mi);
        const float f = shrink(m, mn, scale_log2), fi = shrink(mi, mn, scale_log2);
        o = o * f + oi * fi;
        l = l * f + li * fi;
        m = mn;
      }
    }
    const bool any = l != 0.f;  // some key was seen (a NaN sum among them)
    static_cast<T*>(a.out)[(row0 + r) * D + (x - r * D)] = from_f<T>(any ? o / l : 0.f);
    if (x == r * D && a.smax != nullptr) {
      a.smax[row0 + r] = any ? m * a.scale : -INFINITY;
      a.ssum[row0 + r] = any ? l : 0.f;
    }
  }
}

// Any type, head size up to 32 * DT, any alignment: a warp takes a key at a time, lane = column.
template <typename T, int DT, int R>
__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeArgs a, float scale_log2) {
  __shared__ SchedSmem sched;
  extern __shared__ float smem[];
  const int D = a.D;
  float* s_o = smem;                        // [R][D] merged over the warps
  float* s_w = s_o + R * D;                 // [kWarps][R][D]
  float* s_ml = s_w + kWarps * R * D;       // [R][2]
  float* s_wml = s_ml + 2 * R;              // [kWarps][R][2]
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
      if (lane == 0) {
        s_wml[(warp * R + r) * 2] = m[r];
        s_wml[(warp * R + r) * 2 + 1] = l[r];
      }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < R * D; x += kThreads) {
      const int r = x / D;
      float mm = -INFINITY, ll = 0.f, oo = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_wml[(w * R + r) * 2]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = shrink(s_wml[(w * R + r) * 2], mm, scale_log2);
        ll += s_wml[(w * R + r) * 2 + 1] * f;
        oo += s_w[w * R * D + x] * f;
      }
      s_o[x] = oo;
      if (x == r * D) {
        s_ml[2 * r] = mm;
        s_ml[2 * r + 1] = ll;
      }
    }
    __syncthreads();
    finish_unit<T>(a, c, sp, &sched, s_o, s_ml, scale_log2);
    __syncthreads();
  } while (c.next_unit(a));
}

template <typename T, int DT>
cudaError_t launch_dt(const DecodeArgs& a, cudaStream_t st) {
  constexpr int R = 4;
  const int smem = (int)sizeof(float) * (R * a.D * (kWarps + 1) + 2 * R * (kWarps + 1));
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

}  // namespace

int decode_rows(int dtype, int Nq, int Nkv, int D) {
  (void)dtype;
  (void)Nq;
  (void)Nkv;
  (void)D;
  return 4;
}

int64_t decode_workspace_bytes(int rows, int D) {
  return 2LL * kDecodeMaxCtas * rows * (D + 2) * (int64_t)sizeof(float) + kDecodeMaxCtas * (int64_t)sizeof(unsigned);
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
  if (a.dtype == ATTN_F32) return launch_t<float>(a, st);
  return a.dtype == ATTN_F16 ? launch_t<__half>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace sdpa
